"""Logits before a draw on the GPU: penalties, bias, mask, temperature and the log-softmax against
their definition in 64 bits, and the generation loop that uses them."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from cross_token_latent_b200 import RLTError
from oracle import RLTOracle
from workloads import TINY, make_weights
from gpu_util import build_model, to_np
from paged_util import op_model

pytestmark = pytest.mark.gpu

RLT_EDEVICE = 6


def bits(allowed):
    """Rows of truth values as int32 words, bit v % 32 of word v / 32."""
    B, V = allowed.shape
    padded = np.zeros((B, -(-V // 32) * 32), bool)
    padded[:, :V] = allowed
    return torch.from_numpy(np.packbits(padded, axis=1, bitorder="little").view(np.int32)).cuda()


def reference(x, lse=None, bias=None, allowed=None, tokens=None, tok_len=None, gen_start=None, repetition=None,
              presence=None, frequency=None, tau=None):
    """(out, log-sum-exp, tolerance) in 64 bits.  The tolerance counts float32 roundings of 2^-24: x + lse,
    the penalties, the bias and the temperature round once or twice each at the magnitudes they have; the
    log-sum-exp carries the largest such error, an exponential's 2^-22 and the sum's."""
    z = x.astype(np.float64)
    B, V = z.shape
    mag = np.abs(z)
    if lse is not None:
        z = z + lse[:, None].astype(np.float64)
        mag = np.maximum(mag, np.abs(lse[:, None]))
    mag = mag + np.abs(z)
    if tokens is not None:
        for b in range(B):
            n = tokens.shape[1] if tok_len is None else tok_len[b]
            g = 0 if gen_start is None else gen_start[b]
            seen = np.bincount(tokens[b, :n], minlength=V) > 0
            c = np.bincount(tokens[b, max(0, min(g, n)):n], minlength=V).astype(np.float64)
            if repetition is not None:
                r = np.float64(repetition[b])
                z[b] = np.where(seen, np.where(z[b] > 0, z[b] / r, z[b] * r), z[b])
                mag[b] *= np.where(seen, max(r, 1 / r), 1)
            drop = (0 if presence is None else np.float64(presence[b])) * (c > 0) + \
                (0 if frequency is None else np.float64(frequency[b])) * c
            z[b] -= drop
            mag[b] += 3 * np.abs(drop)
    if bias is not None:
        z = z + bias
        mag = mag + np.abs(bias)
    if allowed is not None:
        z = np.where(allowed, z, -np.inf)
    if tau is not None:
        z = z / tau[:, None].astype(np.float64)
        mag = mag / tau[:, None] + 2 * np.abs(np.where(np.isfinite(z), z, 0))
    err = np.where(np.isfinite(z), 4 * mag * 2.0 ** -24, 0)
    top = z.max(1, keepdims=True)
    safe = np.where(np.isfinite(top), top, 0)
    with np.errstate(divide="ignore"):
        total = safe + np.log(np.exp(z - safe).sum(1, keepdims=True))
    with np.errstate(invalid="ignore"):
        out = np.where(np.isneginf(z), -np.inf, z - total)
    lse_err = err.max(1, keepdims=True) + 2.0 ** -21 + 4 * np.abs(np.where(np.isfinite(total), total, 0)) * 2.0 ** -24
    tol = err + lse_err + np.where(np.isfinite(out), np.abs(out), 0) * 2.0 ** -23
    return out, total[:, 0], tol


def check(got, want, tol):
    got = to_np(got)
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and not np.isnan(got).any()
    fin = np.isfinite(want)
    d = np.abs(got[fin] - want[fin])
    assert (d <= tol[fin]).all(), float((d / tol[fin]).max())


def inputs(B, V, hist, seed):
    r = np.random.default_rng([seed, B, V])
    x = (r.standard_normal((B, V)) * 4).astype(np.float32)
    tokens = np.minimum((V * r.random((B, max(hist, 1))) ** 3).astype(np.int32), V - 1)
    tok_len = r.integers(0, hist + 1, B).astype(np.int32)
    gen = (tok_len * r.random(B)).astype(np.int32)
    par = {k: r.uniform(*lim, B).astype(np.float32) for k, lim in
           (("repetition", (0.7, 1.6)), ("presence", (-0.6, 1.0)), ("frequency", (-0.1, 0.6)), ("tau", (0.3, 1.7)))}
    return r, x, tokens, tok_len, gen, par


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


CASES = [
    # V, rows, history, with lse, bias rows, mask
    (8, 1, 0, False, 0, False),
    (40, 3, 5, True, 0, True),
    (512, 7, 100, True, 1, True),
    (4104, 1, 3000, False, 1, False),
    (8200, 33, 64, True, 33, True),
    (32000, 5, 700, True, 0, True),
    (32768, 130, 40, False, 130, False),
    (49152, 2, 1, True, 1, True),
    (131072, 1, 500, False, 1, True),
    (262144, 3, 64, True, 0, True),
]


@pytest.mark.parametrize("V,B,hist,with_lse,bias_rows,with_mask", CASES)
def test_matches_the_definition(V, B, hist, with_lse, bias_rows, with_mask):
    model = op_model("f32", 16, 8, V=V)
    r, x, tokens, tok_len, gen, par = inputs(B, V, hist, 1)
    lse = r.uniform(5, 12, B).astype(np.float32) if with_lse else None
    x = x - lse[:, None] if with_lse else x
    bias = (r.standard_normal((bias_rows, V)) * (r.random((bias_rows, V)) < 0.1)).astype(np.float32) if bias_rows else None
    allowed = r.random((B, V)) < 0.4 if with_mask else None
    if with_mask:
        allowed[:, V // 2] = True
        allowed[0] = False
        allowed[0, V - 1] = True                                     # one token left
    kw = dict(tokens=tokens, tok_len=tok_len, gen_start=gen, **par) if hist else dict(tau=par["tau"])
    want, total, tol = reference(x, lse=lse, bias=bias, allowed=allowed, **kw)
    out_lse = torch.empty(B, device="cuda")
    out = model.process_logits(dev(x), lse=dev(lse), bias=dev(bias), mask=None if allowed is None else bits(allowed),
                               out_lse=out_lse, **{k: dev(v) for k, v in kw.items()})
    assert model.last_error() == 0
    check(out, want, tol)
    assert (np.abs(to_np(out_lse) - total) <= tol.max(1)).all()
    # in place, and the same bits again
    y = dev(x)
    model.process_logits(y, out=y, lse=dev(lse), bias=dev(bias), mask=None if allowed is None else bits(allowed),
                         **{k: dev(v) for k, v in kw.items()})
    assert torch.equal(y, out)


@pytest.mark.parametrize("V,n", [(512, 70000), (40000, 66000)])
def test_a_long_history_of_one_token(V, n):
    """More occurrences than 16 bits count, and as many as they do."""
    model = op_model("f32", 16, 8, V=V)
    r, x, _, _, _, par = inputs(2, V, 0, 10)
    tokens = np.full((2, n), V - 3, np.int32)
    tokens[:, :100] = r.integers(0, V, (2, 100))
    for lens in ([n, n], [65534, 65000]):
        for m in (n, max(lens)):
            kw = dict(tokens=tokens[:, :m], tok_len=np.array(lens, np.int32), gen_start=np.array([0, 50], np.int32), **par)
            want, _, tol = reference(x, **kw)
            check(model.process_logits(dev(x), **{k: dev(v) for k, v in kw.items()}), want, tol)
    assert model.last_error() == 0


@pytest.mark.parametrize("only", ["repetition", "presence", "frequency", "tau", "none", "nothing but a history"])
def test_each_parameter_alone(only):
    V, B = 512, 4
    model = op_model("f32", 16, 8, V=V)
    _, x, tokens, tok_len, gen, par = inputs(B, V, 60, 2)
    kw = dict(tokens=tokens, tok_len=tok_len, gen_start=gen) if only != "none" else {}
    if only in par:
        kw[only] = par[only]
    want, _, tol = reference(x, **kw)
    check(model.process_logits(dev(x), **{k: dev(v) for k, v in kw.items()}), want, tol)
    assert model.last_error() == 0


@pytest.mark.parametrize("offset", [0, 1, 4])
def test_strides_and_alignment(offset):
    """Rows with gaps, at addresses that vectors cannot take, a history stored token-major, and mask and
    bias rows with gaps."""
    V, B, hist = 1000, 6, 50
    model = op_model("f32", 16, 8, V=V)
    r, x, tokens, tok_len, gen, par = inputs(B, V, hist, 3)
    bias = (r.standard_normal((B, V)) * (r.random((B, V)) < 0.2)).astype(np.float32)
    allowed = r.random((B, V)) < 0.5
    want, _, tol = reference(x, bias=bias, allowed=allowed, tokens=tokens, tok_len=tok_len, gen_start=gen, **par)

    def wide(a, gap):
        t = torch.full((a.shape[0], offset + a.shape[1] + gap), 77, dtype=torch.from_numpy(a[:1]).dtype, device="cuda")
        v = t[:, offset:offset + a.shape[1]]
        v.copy_(torch.from_numpy(a))
        return t, v

    _, xv = wide(x, 3 + offset)
    _, bv = wide(bias, 1)
    _, mv = wide(bits(allowed).cpu().numpy(), 2)
    whole, ov = wide(np.zeros((B, V), np.float32), 5)
    th = dev(tokens.T.copy()).t()
    model.process_logits(xv, out=ov, bias=bv, mask=mv, tokens=th, tok_len=dev(tok_len), gen_start=dev(gen),
                         **{k: dev(v) for k, v in par.items()})
    assert model.last_error() == 0
    check(ov, want, tol)
    whole[:, offset:offset + V] = 77
    assert bool((whole == 77).all())


@pytest.mark.parametrize("V,B", [(512, 2), (2000, 3), (4000, 3), (8000, 300), (20000, 160), (30000, 2), (60000, 2), (100000, 2),
                                 (200000, 1)])
def test_unaligned_rows_of_every_size(V, B):
    """Rows at odd addresses, with all that a call can have, for every split of a row."""
    hist = 40
    model = op_model("f32", 16, 8, V=V)
    r, x, tokens, tok_len, gen, par = inputs(B, V, hist, 9)
    bias = (r.standard_normal((B, V)) * (r.random((B, V)) < 0.2)).astype(np.float32)
    allowed = r.random((B, V)) < 0.5
    allowed[:, 1] = True
    want, _, tol = reference(x, bias=bias, allowed=allowed, tokens=tokens, tok_len=tok_len, gen_start=gen, **par)
    rows = [torch.zeros((B, V + 3), device="cuda")[:, 1:V + 1] for _ in range(3)]
    rows[0].copy_(torch.from_numpy(x))
    rows[1].copy_(torch.from_numpy(bias))
    model.process_logits(rows[0], out=rows[2], bias=rows[1], mask=bits(allowed), tokens=dev(tokens), tok_len=dev(tok_len),
                         gen_start=dev(gen), **{k: dev(v) for k, v in par.items()})
    assert model.last_error() == 0
    check(rows[2], want, tol)


@pytest.mark.parametrize("V,B", [(520, 3), (32768, 2), (16384, 300)])
def test_rows_of_the_types_lowest_and_highest_value(V, B):
    """A row of equal values is uniform whatever they are: V ones add up exactly, their logarithm is off
    by an ulp, and the difference rounds once."""
    model = op_model("f32", 16, 8, V=V)
    x = np.zeros((B, V), np.float32)
    top = np.float32(3.4028235e38)
    tol = 2.0 ** -22 * np.log(V)
    for value in (-top, top, np.float32(-1e30), np.float32(1e4)):
        got = to_np(model.process_logits(dev(x + value)))
        assert np.abs(got + np.log(V)).max() <= tol
        got = to_np(model.process_logits(dev(x), bias=dev(x[:1] + value)))
        assert np.abs(got + np.log(V)).max() <= tol
    x[:, ::2], x[:, 1::2] = top, -top
    got = to_np(model.process_logits(dev(x)))
    assert np.abs(got[:, ::2] + np.log(V / 2)).max() <= tol and (got[:, 1::2] < -1e38).all()
    assert model.last_error() == 0


def test_what_masked_places_hold_does_not_matter():
    V, B = 2056, 4
    model = op_model("f32", 16, 8, V=V)
    r, x, *_ = inputs(B, V, 0, 4)
    allowed = r.random((B, V)) < 0.5
    bias = np.zeros((1, V), np.float32)
    want, _, tol = reference(x, allowed=allowed)
    for bad in (np.nan, np.inf, -np.inf, 3e38, -3.4028235e38):
        y = np.where(allowed, x, np.float32(bad)).astype(np.float32)
        check(model.process_logits(dev(y), bias=dev(bias), mask=bits(allowed)), want, tol)
    # a mask made of the type's lowest value works as one too, short of the -inf: such tokens have no mass
    low = np.where(allowed, 0, -3.4028235e38).astype(np.float32)
    got = to_np(model.process_logits(dev(x), bias=dev(low)))
    assert (np.abs(got - want)[allowed] <= tol[allowed]).all() and (got[~allowed] < -1e38).all()
    # unmasked infinities: -inf is a token without mass
    y = np.where(allowed, x, -np.inf).astype(np.float32)
    check(model.process_logits(dev(y)), want, tol)
    # a NaN that counts makes its row NaN and no other
    y = x.copy()
    y[1, 7] = np.nan
    got = to_np(model.process_logits(dev(y)))
    assert np.isnan(got[1]).all() and not np.isnan(np.delete(got, 1, 0)).any()
    y[2] = np.nan
    assert np.isnan(to_np(model.process_logits(dev(y)))[2]).all()
    assert model.last_error() == 0


@pytest.mark.parametrize("V,B", [(40, 3), (32768, 200), (262144, 2)])
def test_a_row_without_any_token_is_latched_and_the_others_hold(V, B):
    model = op_model("f32", 16, 8, V=V)
    r, x, *_ = inputs(B, V, 0, 5)
    allowed = r.random((B, V)) < 0.5
    allowed[:, 0] = True
    allowed[1] = False
    want, _, tol = reference(x, allowed=allowed)
    lse = torch.zeros(B, device="cuda")
    out = model.process_logits(dev(x), mask=bits(allowed), out_lse=lse)
    assert model.last_error() == RLT_EDEVICE and model.last_error() == 0
    check(out, want, tol)
    assert np.isneginf(to_np(lse)[1])


def test_bad_parameters_and_ids_are_latched():
    V, B = 64, 3
    model = op_model("f32", 16, 8, V=V)
    _, x, tokens, *_ = inputs(B, V, 6, 6)
    two, one = np.full(B, 2.0, np.float32), np.ones(B, np.float32)
    for bad in (0.0, -1.0, np.nan):
        for name in ("repetition", "tau"):
            par = {"repetition": two.copy(), "tau": two.copy()}
            par[name][1] = bad
            got = model.process_logits(dev(x), tokens=dev(tokens), **{k: dev(v) for k, v in par.items()})
            assert model.last_error() == RLT_EDEVICE
            par[name][1] = 1.0
            want, _, tol = reference(x, tokens=tokens, **par)
            check(got, want, tol)
    for bad in (-1, V, 2**31 - 1, -2**31):
        t = tokens.copy()
        t[0, 3] = bad
        got = model.process_logits(dev(x), tokens=dev(t), frequency=dev(one))
        assert model.last_error() == RLT_EDEVICE
        want, _, tol = reference(x, tokens=tokens, frequency=one)
        assert (np.abs(to_np(got)[1:] - want[1:]) <= tol[1:]).all()
        keep = np.delete(tokens[:1], 3, axis=1)
        want, _, tol = reference(x[:1], tokens=keep, frequency=one[:1])
        check(got[:1], want, tol)
    got = model.process_logits(dev(x), tokens=dev(tokens), tok_len=dev(np.array([7, -1, 2], np.int32)), frequency=dev(one))
    assert model.last_error() == RLT_EDEVICE
    want, _, tol = reference(x, tokens=tokens, tok_len=[6, 0, 2], frequency=one)
    check(got, want, tol)
    assert model.last_error() == 0


def test_refusals():
    V, B = 64, 3
    model = op_model("f32", 16, 8, V=V)
    x = torch.zeros((B, V), device="cuda")
    v = torch.ones(B, device="cuda")
    ids = torch.zeros((B, 4), dtype=torch.int32, device="cuda")
    for kw in (dict(lse=v[:2]), dict(tau=v.double()), dict(tau=v.cpu()), dict(bias=torch.zeros((2, V), device="cuda")),
               dict(bias=torch.zeros((B, V - 1), device="cuda")), dict(mask=torch.zeros((B, 3), dtype=torch.int32, device="cuda")),
               dict(mask=torch.zeros((B, 2), dtype=torch.int64, device="cuda")), dict(tokens=ids.long()), dict(tokens=ids[:2]),
               dict(tok_len=ids[:, 0].contiguous()), dict(gen_start=ids[:, 0].contiguous()), dict(out=x[:2]),
               dict(tokens=ids, tok_len=ids[:, 0]), dict(out=torch.zeros((V, B), device="cuda").t())):
        with pytest.raises(ValueError):
            model.process_logits(x, **kw)
    for bad in (x[:, :40], x.double(), x.cpu(), torch.zeros((V, B), device="cuda").t()):
        with pytest.raises(ValueError):
            model.process_logits(bad)
    with pytest.raises(RLTError):                        # a vocabulary beyond what a row's cluster holds
        big = op_model("f32", 16, 8, V=262152)
        big.process_logits(torch.zeros((1, 262152), device="cuda"))
    torch.cuda.synchronize()
    assert model.last_error() == 0


def test_a_captured_call_reads_what_the_buffers_hold_then():
    V, B, hist = 4096, 5, 30
    model = op_model("f32", 16, 8, V=V)
    _, x, tokens, tok_len, gen, par = inputs(B, V, hist, 7)
    buf = {k: dev(v) for k, v in dict(x=x, tokens=tokens, tok_len=tok_len, gen_start=gen, **par).items()}
    out = torch.empty((B, V), device="cuda")

    def call():
        model.process_logits(buf["x"], out=out, **{k: v for k, v in buf.items() if k != "x"})

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    _, x, tokens, tok_len, gen, par = inputs(B, V, hist, 8)
    for k, v in dict(x=x, tokens=tokens, tok_len=tok_len, gen_start=gen, **par).items():
        buf[k].copy_(torch.from_numpy(v))
    graph.replay()
    torch.cuda.synchronize()
    want, _, tol = reference(x, tokens=tokens, tok_len=tok_len, gen_start=gen, **par)
    check(out, want, tol)


def test_generation_under_penalties_a_bias_and_a_mask():
    """Float32 model: the draws of generate() are those of the oracle's distribution under the same
    penalties, bias and mask; behaviour log-probs agree within 1e-4; no token leaves the mask, and with a
    presence penalty that outweighs every logit no generated token occurs twice."""
    from oracle import sample_token

    cfg = TINY.model
    w = make_weights(cfg)
    model = build_model(cfg, max_pos=40, weights=w)
    B, P, n_new, tau = 3, 10, 12, 0.8
    rng = np.random.default_rng(11)
    prompt = rng.integers(0, cfg.V, size=(B, P)).astype(np.int32)
    u = rng.random((n_new, B)).astype(np.float32)
    bias = np.zeros((1, cfg.V), np.float32)
    bias[0, 5:25] = 1.5
    even, odd = (np.arange(cfg.V)[None] % 2 == i for i in (0, 1))
    masks = [bits(even), bits(odd)]
    seen_steps = []

    def grammar(step, tokens):
        assert tokens.shape == (B, P + step)
        seen_steps.append(step)
        return masks[step % 2]

    toks, blp, _, _ = model.generate(dev(prompt), n_new, dev(u), tau=tau, top_k=30, top_p=0.9, repetition=1.2,
                                     presence=100.0, frequency=0.3, bias=dev(bias), mask=grammar)
    assert model.last_error() == 0 and seen_steps == list(range(n_new))
    toks, blp = toks.cpu().numpy(), to_np(blp)
    assert (toks[:, P:] % 2 == np.arange(n_new) % 2).all()
    assert all(len(set(toks[b, P:])) == n_new for b in range(B))
    oracle = RLTOracle(cfg, w)
    same = 0
    e, M = oracle.encode(toks)
    state = oracle.init_state(B)
    for t in range(1, P + n_new):
        state, logp = oracle.step(state, e[:, t - 1], M, 1.0)
        if t < P:
            continue
        z = np.asarray(logp, np.float64)
        # logp is z - lse: the penalty needs z itself
        z = np.asarray(state.s, np.float64) @ np.asarray(w["unembed"], np.float64).T
        par = {k: np.full(B, x, np.float32) for k, x in (("repetition", 1.2), ("presence", 100.0), ("frequency", 0.3),
                                                         ("tau", tau))}
        want, _, _ = reference(z, bias=bias, allowed=np.broadcast_to((even, odd)[(t - P) % 2], (B, cfg.V)),
                               tokens=toks[:, :t], gen_start=np.full(B, P), **par)
        for b in range(B):
            picks = {sample_token(want[b].astype(np.float32), float(np.clip(u[t - P, b] + d, 0, 1 - 1e-7)), 30, 0.9)
                     for d in (-1e-5, 0.0, 1e-5)}
            by = dict(picks)
            assert int(toks[b, t]) in by, (b, t)
            same += 1
            assert abs(blp[b, t - P] - by[int(toks[b, t])]) <= 1e-4
    assert same == B * n_new
