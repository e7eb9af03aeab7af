"""Shared by the tests of the paged cache: ragged batches over shuffled pages, and the operators'
definitions in 64 bits."""
from __future__ import annotations

import math
from dataclasses import replace

import numpy as np
import torch

from cross_token_latent_b200 import RLTModel
from workloads import TINY

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}        # eps / 2, relative to the value


def op_model(dtype: str, hd: int, max_pos: int, V: int = 64) -> RLTModel:
    """A handle with this type, head width and rotary table (its weights are never set)."""
    cfg = replace(TINY.model, V=V, d=hd, n_heads=1, head_dim=hd, L_E=1, L_D=1, F=16, dtype=dtype)
    return RLTModel(cfg, max_pos=max_pos)


class Ragged:
    """Sequences of q[b] new tokens at the end of kv[b], on shuffled pages, `pad` rows behind them."""

    def __init__(self, q, kv, page: int, pad: int = 0, seed: int = 0, spare: int = 2, max_q=None, max_kv=None,
                 n_pages=None):
        self.q, self.kv, self.page, self.pad = list(q), list(kv), page, pad
        self.B, self.N = len(q), sum(q) + pad
        need = [-(-k // page) for k in kv]
        self.n_pages = sum(need) + spare if n_pages is None else n_pages
        ids = np.random.default_rng(seed).permutation(self.n_pages)
        table = np.full((self.B, max(max(need), 1)), -7, np.int32)          # entries nobody may read
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table_np = table
        self.starts = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        self.max_q = max(max(q), 1) if max_q is None else max_q
        self.max_kv = max(max(kv), self.max_q) if max_kv is None else max_kv
        cols = -(-self.max_kv // page)
        if cols > table.shape[1]:
            table = np.concatenate([table, np.full((self.B, cols - table.shape[1]), -7, np.int32)], 1)
        self.table = torch.from_numpy(table).cuda()
        self.q_start = torch.from_numpy(self.starts).cuda()
        self.kv_len = torch.from_numpy(np.asarray(kv, np.int32)).cuda()

    def batch(self, model, Hkv):
        return model.paged_batch(self.table, self.q_start, self.kv_len, self.N, self.max_q, self.max_kv, self.page, Hkv)

    def rows(self):
        """(sequence, position) of every row that belongs to one."""
        return [(b, self.kv[b] - n + i) for b, n in enumerate(self.q) for i in range(n)]

    def place(self, b, t):
        return int(self.table_np[b, t // self.page]), t % self.page


def gather(pool, r: Ragged, b: int, n: int):
    """Keys and values [Hkv, n, hd] (float64) of sequence b's first n tokens."""
    pages = torch.from_numpy(r.table_np[b, :-(-n // r.page)].astype(np.int64)).to(pool.device)
    x = pool[pages].permute(1, 2, 0, 3, 4).flatten(2, 3)
    return x[0, :, :n].double(), x[1, :, :n].double()


def attention_ref(pool, r: Ragged, q, scale=None):
    """(out, tolerance) in 64 bits for every row of a sequence, [rows, H, hd].

    The tolerance is a bound on what the arithmetic allows: with the score error ds (products of
    float32 sums), every probability is off by a relative ds + 2^-21 (exponential; 2^-13 for the
    polynomial of the bf16 kernels), on the tensor cores by a rounding to bf16 more; numerator and denominator both carry it, weighted by
    A = sum p |v|; sums of n terms add n 2^-24; the result is rounded once."""
    H, hd = q.shape[1], q.shape[2]
    Hkv = pool.shape[2]
    g = H // Hkv
    scale = hd ** -0.5 if scale is None else scale
    dtype = "bf16" if pool.dtype == torch.bfloat16 else "f32"
    half = HALF_STEP[dtype]
    outs, tols = [], []
    for b, n in enumerate(r.q):
        if n == 0:
            continue
        k, v = gather(pool, r, b, r.kv[b])
        x = q[r.starts[b]:r.starts[b] + n].double().permute(1, 0, 2).unflatten(0, (Hkv, g))     # [Hkv, g, n, hd]
        s = torch.einsum("hgqd,hkd->hgqk", x, k) * scale
        mag = torch.einsum("hgqd,hkd->hgqk", x.abs(), k.abs()) * scale
        at = torch.arange(r.kv[b] - n, r.kv[b], device=q.device)
        ahead = torch.arange(r.kv[b], device=q.device) > at[:, None]
        p = torch.softmax(s.masked_fill(ahead, -math.inf), -1)
        o = torch.einsum("hgqk,hkd->hgqd", p, v)
        A = torch.einsum("hgqk,hkd->hgqd", p, v.abs())
        ds = mag.masked_fill(ahead, 0).amax(-1, keepdim=True) * (hd + 4) * 2.0 ** -24
        rel = 2 * (ds + 2.0 ** (-13 if dtype == "bf16" else -21) + r.kv[b] * 2.0 ** -24) + (2 * 2.0 ** -8 if dtype == "bf16" else 0)
        tol = half * o.abs() + rel * A * 1.01 + 1e-30
        outs.append(o.flatten(0, 1).permute(1, 0, 2))
        tols.append(tol.flatten(0, 1).permute(1, 0, 2))
    return torch.cat(outs), torch.cat(tols)


def rotate_ref(x, pos, base=10000.0):
    """(x rotated by its positions, sum of the magnitudes of the two products) in 64 bits; x [N, heads, hd]."""
    hd = x.shape[-1]
    f = base ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, device=x.device) / hd)
    a = (pos.double()[:, None] * f)[:, None]
    lo, hi = x[..., :hd // 2].double(), x[..., hd // 2:].double()
    c, s = a.cos(), a.sin()
    y = torch.cat([lo * c - hi * s, lo * s + hi * c], -1)
    mag = torch.cat([(lo * c).abs() + (hi * s).abs(), (lo * s).abs() + (hi * c).abs()], -1)
    return y, mag
