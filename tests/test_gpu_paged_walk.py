"""Calls of more rows than the append, and the scatter of encoded rows, have blocks for: every block walks
through several rows with the next one's elements on their way."""
from dataclasses import replace

import numpy as np
import pytest
import torch

import test_gpu_paged as paged
from gpu_util import build_model, to_np
from paged_util import Ragged, op_model
from workloads import TINY, make_weights

pytestmark = pytest.mark.gpu

APPEND = [
    # dtype, source, heads, kv heads, hd, page, blocks per row, rows of padding
    ("bf16", "bf16", 32, 8, 128, 16, 2, 5),
    ("bf16", "f32", 16, 16, 64, 64, 2, 0),
    ("bf16", "f32", 5, 5, 64, 128, 1, 37),
    ("bf16", "bf16", 3, 1, 16, 32, 1, 1),
    ("f32", "f32", 4, 4, 16, 16, 1, 2),
    ("f32", "f32", 20, 4, 128, 64, 2, 3),
]


def lengths(dtype_src, H, Hkv, hd, blocks, times):
    """Ragged lengths of a call with `times` rows and a bit for every block: 4096 threads per SM, items of 16
    bytes of the source."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    items = (H + 2 * Hkv) * hd // 2 // (16 // (2 if dtype_src == "bf16" else 4))
    assert -(-items // 256) == blocks
    threads = -(-(-(-items // blocks)) // 32) * 32
    most = -(-4096 * sms // (blocks * threads))
    n = times * most + most // 3 + 7
    q = [n // 2 + 1, 0, 1, n // 3, 17, 1]
    q.append(n - sum(q))
    return q, [k + ctx for k, ctx in zip(q, (0, 5, 700, 33, 0, 0, 2))]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[:6])))
def test_append_of_many_rows(case):
    dtype, src, H, Hkv, hd, page, blocks, pad = case
    q_len, kv_len = lengths(src, H, Hkv, hd, blocks, 2)
    paged.test_append_rotates_and_places_every_row((dtype, src, H, Hkv, hd, page, q_len, kv_len, pad))


@pytest.mark.parametrize("dtype,H,Hkv,hd,blocks", [("bf16", 32, 8, 128, 2), ("f32", 4, 4, 16, 1)])
def test_append_of_many_rows_in_place(dtype, H, Hkv, hd, blocks):
    """q_out is q: a block writes a row while the next one, of the same tensor, is already loaded."""
    q_len, kv_len = lengths(dtype, H, Hkv, hd, blocks, 3)
    r = Ragged(q_len, kv_len, 64, pad=9)
    model = op_model(dtype, hd, r.max_kv)
    pool = torch.zeros((r.n_pages, 2, Hkv, 64, hd), dtype=model.sdtype, device="cuda")
    other = pool.clone()
    q, k, v = (paged.randn((r.N, h, hd), model.sdtype, i) for i, h in enumerate((H, Hkv, Hkv)))
    batch = r.batch(model, Hkv)
    out = model.paged_append(batch, pool, k, v, q=q, q_out=torch.full_like(q, 5.0))
    again = q.clone()
    model.paged_append(batch, other, k, v, q=again, q_out=again)
    assert model.last_error() == 0
    n = r.N - r.pad
    assert torch.equal(out[:n], again[:n]) and torch.equal(pool, other)
    assert bool((out[n:] == 5.0).all()) and torch.equal(again[n:], q[n:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_chunk_of_many_rows_is_scattered_whole(dtype):
    """The encoder over two ragged calls of more rows than the scatters have blocks (8 per SM), against the
    same tokens in calls of a few rows, which other tests hold against the definition: float32 within
    summation order, bf16 within four of its steps at magnitudes between 2 and 4 (2^-6 each)."""
    cfg = replace(TINY.model, dtype=dtype, G=2)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = 5
    T = -(-(8 * sms * 5 // 2) // B) + 11
    T_alloc = T + 8
    model = build_model(cfg, max_pos=T_alloc, weights=make_weights(cfg))
    tok = np.random.default_rng(6).integers(0, cfg.V, size=(B, T)).astype(np.int32)
    head = np.array([T - 1, T - 40, T, T - 3, 60])
    e, M = paged.chunked_encoding(model, tok, [head, T - head], 16, T_alloc, pad=3)
    few = [np.full(B, 150)] * (T // 150) + [np.full(B, T % 150)]
    e_few, M_few = paged.chunked_encoding(model, tok, few, 16, T_alloc)
    assert bool((e[:, T:] == 0).all()) and bool((M[:, :, :, :, T:] == 0).all())
    limit = 1e-5 if dtype == "f32" else 2.0 ** -4
    assert np.abs(to_np(e) - to_np(e_few)).max() <= limit
    assert np.abs(to_np(M) - to_np(M_few)).max() <= limit
