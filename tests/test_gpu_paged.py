"""The paged key/value cache on the GPU: appending with the rotation on the way, the attention of
new tokens over it, and the encoder that runs on both, against definitions in 64 bits, the
token-parallel encoder and the CPU oracle."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from cross_token_latent_b200 import RLTError
from oracle import RLTOracle
from workloads import SMALL, TINY, make_weights
from gpu_util import build_model, cosine, to_np
from paged_util import HALF_STEP, TYPES, Ragged, attention_ref, op_model, rotate_ref

pytestmark = pytest.mark.gpu

RLT_EDEVICE = 6


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


# ------------------------------------------------------------------ append
APPEND = [
    # dtype, source, heads, kv heads, hd, page, new tokens, tokens in all, rows of padding
    ("bf16", "f32", 16, 16, 64, 64, [1], [1], 0),
    ("bf16", "f32", 4, 4, 32, 16, [1, 1, 1], [1, 16, 17], 0),
    ("bf16", "bf16", 32, 8, 128, 16, [1, 0, 33, 16], [700, 0, 33, 32], 5),
    ("bf16", "bf16", 7, 1, 128, 256, [300, 1], [300, 4000], 1),
    ("bf16", "f32", 6, 2, 16, 32, [0, 0, 45], [0, 9, 77], 0),
    ("bf16", "f32", 5, 5, 64, 128, [129, 127, 1, 257], [129, 511, 128, 1000], 3),
    ("f32", "f32", 4, 4, 16, 16, [31, 1, 2], [31, 600, 17], 2),
    ("f32", "f32", 3, 1, 128, 64, [65, 64], [65, 8000], 0),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[:6])))
def test_append_rotates_and_places_every_row(case):
    dtype, src, H, Hkv, hd, page, q_len, kv_len, pad = case
    r = Ragged(q_len, kv_len, page, pad, seed=1)
    model = op_model(dtype, hd, r.max_kv)
    dt = TYPES[dtype]
    pool = randn((r.n_pages, 2, Hkv, page, hd), dt, 2)
    before = pool.clone()
    # column ranges of one projection, with a few columns of something else behind them
    rows = randn((r.N, (H + 2 * Hkv) * hd + 24), TYPES[src], 3)
    q = rows[:, :H * hd].unflatten(1, (H, hd))
    k = rows[:, H * hd:(H + Hkv) * hd].unflatten(1, (Hkv, hd))
    v = rows[:, (H + Hkv) * hd:(H + 2 * Hkv) * hd].unflatten(1, (Hkv, hd))
    out = torch.full((r.N, H, hd), 9.0, dtype=dt, device="cuda")
    got = model.paged_append(r.batch(model, Hkv), pool, k, v, q=q, q_out=out)
    assert got is out and model.last_error() == 0
    where = r.rows()
    n = len(where)
    pos = torch.tensor([t for _, t in where], device="cuda")
    # a rotated element is two products of float32 values with table entries rounded once, and a sum:
    # three roundings of 2^-24 of the products' magnitudes; then the one rounding to the stored type
    def close(x, y, mag):
        tol = HALF_STEP[dtype] * (y.abs() + 3 * 2.0 ** -24 * mag) + 3 * 2.0 ** -24 * mag
        assert bool(((x.double() - y).abs() <= tol).all())
    close(out[:n], *rotate_ref(q[:n], pos))
    assert bool((out[n:] == 9.0).all())
    page_of = torch.tensor([r.place(b, t)[0] for b, t in where], device="cuda")
    slot_of = torch.tensor([r.place(b, t)[1] for b, t in where], device="cuda")
    close(pool[page_of, 0, :, slot_of], *rotate_ref(k[:n], pos))
    assert torch.equal(pool[page_of, 1, :, slot_of], v[:n].to(dt))
    # every other slot is as it was
    pool[page_of, :, :, slot_of] = before[page_of, :, :, slot_of]
    assert torch.equal(pool, before)


def test_append_in_place_and_without_queries():
    r = Ragged([3, 40], [10, 40], 16)
    model = op_model("bf16", 64, 64)
    pool = torch.zeros((r.n_pages, 2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    other = pool.clone()
    q, k, v = (randn((r.N, h, 64), torch.bfloat16, i) for i, h in enumerate((4, 2, 2)))
    batch = r.batch(model, 2)
    out = model.paged_append(batch, pool, k, v, q=q)
    again = q.clone()
    model.paged_append(batch, other, k, v, q=again, q_out=again)
    assert torch.equal(out, again) and torch.equal(pool, other)
    third = torch.zeros_like(pool)
    assert model.paged_append(batch, third, k, v) is None
    assert torch.equal(pool, third)


def test_append_and_attention_behind_two_to_the_32_bytes_and_elements():
    """Pages whose elements lie beyond 2^32: offsets take 64 bits."""
    page, Hkv, hd = 256, 8, 128
    n_pages = (1 << 32) // (2 * Hkv * page * hd) + 3
    model = op_model("bf16", hd, 600)
    pool = torch.empty((n_pages, 2, Hkv, page, hd), dtype=torch.bfloat16, device="cuda")
    r = Ragged([20, 1], [20, 513], page, n_pages=n_pages)
    r.table_np[:, :] = np.array([[n_pages - 1, -7, -7], [n_pages - 2, 0, n_pages - 3]], np.int32)
    r.table = torch.from_numpy(r.table_np).cuda()
    for p in (0, n_pages - 3, n_pages - 2, n_pages - 1):
        pool[p] = randn(pool.shape[1:], torch.bfloat16, p % 97)
    q, k, v = (randn((r.N, h, hd), torch.bfloat16, 50 + h) for h in (16, 8, 8))
    batch = r.batch(model, Hkv)
    q = model.paged_append(batch, pool, k, v, q=q)
    assert torch.equal(pool[n_pages - 1, 1, :, :20].transpose(0, 1), v[:20])
    out = model.paged_attention(batch, pool, q)
    assert model.last_error() == 0
    ref, tol = attention_ref(pool, r, q)
    assert bool(((out.double() - ref).abs() <= tol).all())


# ------------------------------------------------------------------ attention
ATTEND = [
    # dtype, heads, kv heads, hd, page, new tokens, tokens in all, rows of padding
    ("bf16", 16, 16, 64, 64, [1], [1], 0),
    ("bf16", 16, 16, 64, 64, [1], [171], 0),
    ("bf16", 16, 16, 128, 128, [1, 1, 1, 1], [1, 127, 128, 4096], 0),
    ("bf16", 32, 8, 128, 16, [1, 1, 0, 1, 1], [33, 2049, 0, 15, 700], 2),
    ("bf16", 7, 1, 64, 32, [1, 2, 1], [5000, 64, 1], 0),
    ("bf16", 64, 1, 128, 16, [1, 3], [300, 1000], 0),
    ("bf16", 4, 4, 32, 16, [5, 1, 100], [5, 16, 333], 1),
    ("bf16", 8, 2, 16, 256, [64, 17], [64, 900], 0),
    ("bf16", 16, 16, 64, 64, [128, 129, 1, 300], [128, 129, 640, 301], 7),
    ("bf16", 16, 16, 128, 16, [200, 1, 16], [1500, 1500, 16], 0),
    ("bf16", 12, 4, 128, 32, [257, 43], [257, 2100], 0),
    ("bf16", 5, 1, 64, 16, [400], [411], 0),
    ("bf16", 2, 2, 64, 256, [700, 65], [3000, 65], 0),
    ("bf16", 2, 1, 128, 64, [40], [20000], 0),
    ("bf16", 1, 1, 64, 128, [1], [30000], 0),
    # many sequences: more than a warp, and more than a block, looks at in one go
    ("bf16", 6, 2, 64, 16, [(0, 1, 2, 30, 0, 1, 9)[i % 7] for i in range(700)], [(i * 37) % 290 + 31 for i in range(700)], 4),
    ("bf16", 4, 4, 128, 32, [1 + i % 2 for i in range(90)], [(i * 131) % 2000 + 2 for i in range(90)], 0),
    # more tiles than a warp looks at in one go, of a group that does not divide a tile
    ("bf16", 3, 1, 64, 64, [1, 5000, 40], [7000, 9000, 40], 1),
    ("f32", 2, 2, 16, 16, [i % 3 for i in range(100)], [(i * 53) % 500 + 3 for i in range(100)], 2),
    ("f32", 4, 4, 16, 16, [1, 9, 100], [400, 9, 250], 1),
    ("f32", 6, 2, 32, 32, [1, 1], [5000, 3], 0),
    ("f32", 2, 1, 64, 64, [33, 1], [33, 900], 0),
    ("f32", 3, 3, 128, 128, [70], [600], 0),
    ("f32", 1, 1, 128, 16, [2, 1], [9000, 1], 0),
]


def attend_case(case, seed=0, scale_q=2.0, garbage=float("nan")):
    dtype, H, Hkv, hd, page, q_len, kv_len, pad = case
    r = Ragged(q_len, kv_len, page, pad, seed=seed + 5)
    model = op_model(dtype, hd, r.max_kv)
    pool = randn((r.n_pages, 2, Hkv, page, hd), TYPES[dtype], seed)
    q = randn((r.N, H, hd), TYPES[dtype], seed + 1, scale_q)
    q[r.N - pad:] = garbage
    # slots that hold no token, and pages that belong to nobody, hold anything
    used = torch.zeros((r.n_pages, page), dtype=torch.bool, device="cuda")
    for b, n in enumerate(r.kv):
        for c in range(-(-n // page)):
            used[r.table_np[b, c], :min(page, n - c * page)] = True
    pool = torch.where(used[:, None, None, :, None], pool, torch.tensor(garbage, dtype=pool.dtype, device="cuda"))
    return r, model, pool, q


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c[:5])) + f"-{len(c[5])}x{max(c[5])}-{max(c[6])}")
def test_attention_matches_the_definition(case):
    r, model, pool, q = attend_case(case)
    out = torch.full_like(q, 3.0)
    batch = r.batch(model, pool.shape[2])
    got = model.paged_attention(batch, pool, q, out=out)
    assert got is out and model.last_error() == 0
    ref, tol = attention_ref(pool, r, q)
    n = ref.shape[0]
    bad = (out[:n].double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((out[:n].double() - ref).abs().max()))
    assert bool((out[n:] == 3.0).all())
    # the same call again gives the same bits
    again = model.paged_attention(batch, pool, q, out=torch.full_like(q, 3.0))
    assert torch.equal(again, out)


@pytest.mark.parametrize("case", [ATTEND[3], ATTEND[8], ATTEND[19]], ids=["step", "chunk", "f32"])
def test_attention_takes_strided_rows_a_scale_and_large_scores(case):
    r, model, pool, q = attend_case(case, seed=7, scale_q=30.0, garbage=float("inf"))
    H, hd = q.shape[1:]
    wide_q = torch.empty((r.N, H * hd + 40), dtype=q.dtype, device="cuda")
    wide_q[:, 16:16 + H * hd] = q.flatten(1)
    wide_o = torch.full((r.N, H * hd + 8), 5.0, dtype=q.dtype, device="cuda")
    qs, os = wide_q[:, 16:16 + H * hd].unflatten(1, (H, hd)), wide_o[:, :H * hd].unflatten(1, (H, hd))
    model.paged_attention(r.batch(model, pool.shape[2]), pool, qs, out=os, scale=0.3)
    assert model.last_error() == 0
    ref, tol = attention_ref(pool, r, q, scale=float(np.float32(0.3)))
    n = ref.shape[0]
    assert bool(((os[:n].double() - ref).abs() <= tol).all())
    assert bool((wide_o[:, H * hd:] == 5.0).all()) and bool((os[n:] == 5.0).all())


def test_sequences_that_share_pages():
    """Two sequences with a common prefix on the same pages, each with its own last page."""
    r = Ragged([4, 1], [100, 90], 16)
    r.table_np[1, :5] = r.table_np[0, :5]
    r.table = torch.from_numpy(r.table_np).cuda()
    model = op_model("bf16", 64, 128)
    pool, q = randn((r.n_pages, 2, 2, 16, 64), torch.bfloat16, 1), randn((r.N, 8, 64), torch.bfloat16, 2)
    out = model.paged_attention(r.batch(model, 2), pool, q)
    ref, tol = attention_ref(pool, r, q)
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("hd,chunk", [(64, 1), (64, 200), (32, 3)])
def test_a_captured_call_is_replayed_with_other_lengths(hd, chunk):
    """Append and attention captured once under bounds; the replays see other lengths, starts and pages."""
    B, page, H, Hkv, max_kv = 3, 16, 4, 2, 600
    N = B * chunk
    model = op_model("bf16", hd, max_kv)
    pages = 3 * (-(-max_kv // page))
    pool = randn((pages, 2, Hkv, page, hd), torch.bfloat16, 0)
    table = torch.zeros((B, -(-max_kv // page)), dtype=torch.int32, device="cuda")
    q_start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    batch = model.paged_batch(table, q_start, kv_len, N, chunk, max_kv, page, Hkv)
    k, v, q = (randn((N, h, hd), torch.bfloat16, 3 + h) for h in (Hkv, Hkv, H))
    rot, out = torch.zeros_like(q), torch.zeros_like(q)

    def call():
        model.paged_append(batch, pool, k, v, q=q, q_out=rot)
        model.paged_attention(batch, pool, rot, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i, (ql, kl) in enumerate([([chunk] * 3, [chunk, 333, 600]), ([0, 1, chunk], [0, 1, 431]), ([0, 0, 0], [0, 5, 0]),
                                  ([1, 1, 1], [600, 600, 600])]):
        r = Ragged(ql, kl, page, pad=N - sum(ql), seed=20 + i, max_q=chunk, max_kv=max_kv, n_pages=pages)
        table.copy_(r.table.clamp(min=0))
        q_start.copy_(r.q_start)
        kv_len.copy_(r.kv_len)
        out.fill_(4.0)
        graph.replay()
        torch.cuda.synchronize()
        assert model.last_error() == 0
        n = sum(ql)
        if n:
            ref, tol = attention_ref(pool, r, rot)
            assert bool(((out[:n].double() - ref).abs() <= tol).all())
        assert bool((out[n:] == 4.0).all())


def test_calls_on_two_streams_do_not_share_a_workspace():
    """Two long-context calls in flight at once, on streams of their own, give what they give alone."""
    r = Ragged([1], [30000], 64)
    model = op_model("bf16", 128, 30000)
    pools = [randn((r.n_pages, 2, 2, 64, 128), torch.bfloat16, i) for i in range(2)]
    qs = [randn((1, 16, 128), torch.bfloat16, 9 + i) for i in range(2)]
    batch = r.batch(model, 2)
    alone = [model.paged_attention(batch, p, q) for p, q in zip(pools, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(model.paged_attention(batch, pools[i], qs[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone[i]) for i in range(2) for o in outs[i])


# ------------------------------------------------------------------ what the device refuses
def test_bad_pages_and_lengths_are_latched_and_leave_the_rest_right():
    """The kernels check every page id and length against the call's bounds before they use it."""
    H, Hkv, hd, page = 4, 2, 64, 16
    model = op_model("bf16", hd, 200)
    good = Ragged([2, 5, 3], [50, 60, 70], page, seed=3)
    pool = randn((good.n_pages, 2, Hkv, page, hd), torch.bfloat16, 1)
    q, k, v = (randn((good.N, h, hd), torch.bfloat16, h) for h in (H, Hkv, Hkv))
    ref, tol = attention_ref(pool, good, q)

    def others_hold(out, b):
        keep = [i for i in range(good.N) if not good.starts[b] <= i < good.starts[b + 1]]
        assert bool(((out[keep].double() - ref[keep]).abs() <= tol[keep]).all())

    for page_id in (-1, good.n_pages, 2**31 - 1, -2**31):
        table = good.table.clone()
        table[1, 1] = page_id
        batch = model.paged_batch(table, good.q_start, good.kv_len, good.N, 5, 80, page, Hkv)
        out = model.paged_attention(batch, pool, q)
        assert model.last_error() == RLT_EDEVICE and model.last_error() == 0
        others_hold(out, 1)
        # an append whose page is bad is dropped; the sequence's other rows are placed
        table = good.table.clone()
        table[0, 3] = page_id                              # row 1 of sequence 0 is at position 49, row 0 at 48: both there
        batch = model.paged_batch(table, good.q_start, good.kv_len, good.N, 5, 80, page, Hkv)
        other = pool.clone()
        model.paged_append(batch, other, k, v)
        assert model.last_error() == RLT_EDEVICE
        assert torch.equal(other[int(good.table_np[0, 3])], pool[int(good.table_np[0, 3])])
        p, s = good.place(1, 59)
        assert torch.equal(other[p, 1, :, s], v[6])
    # (sequence that is wrong, q_start, kv_len): lengths beyond the bounds, below the new tokens, decreasing starts
    for b, qs, kl in [(1, [0, 2, 7, 10], [50, 81, 70]), (1, [0, 2, 7, 10], [50, -1, 70]), (1, [0, 2, 7, 10], [50, 4, 70]),
                      (2, [0, 2, 7, 13], [50, 60, 70]), (2, [0, 2, 7, 6], [50, 60, 70]), (2, [0, 2, 7, -4], [50, 60, 70])]:
        batch = model.paged_batch(good.table, torch.tensor(qs, dtype=torch.int32, device="cuda"),
                                  torch.tensor(kl, dtype=torch.int32, device="cuda"), good.N, 5, 80, page, Hkv)
        out = torch.full_like(q, 2.0)
        model.paged_attention(batch, pool, q, out=out)
        assert model.last_error() == RLT_EDEVICE
        others_hold(out, b)
        rows = slice(int(good.starts[b]), int(good.starts[b + 1]))
        assert bool((out[rows] == 2.0).all())
        other = pool.clone()
        model.paged_append(batch, other, k, v)
        assert model.last_error() == RLT_EDEVICE
        for t in range(good.kv[b] - good.q[b], good.kv[b]):
            p, s = good.place(b, t)
            assert torch.equal(other[p, :, :, s], pool[p, :, :, s])
    assert model.last_error() == 0


@pytest.mark.parametrize("dtype,hd,rows", [("bf16", 64, 5), ("bf16", 128, 40), ("f32", 32, 5)])
def test_starts_that_overlap_are_latched_and_nothing_else_is_touched(dtype, hd, rows):
    """Starts that go back and forth count the same rows many times, more than the host sized for; the
    kernels leave out what does not fit, and the handle stays usable."""
    H, Hkv, page, kv, B = 4, 2, 16, 3000, 64
    model = op_model(dtype, hd, kv)
    cols = -(-kv // page)
    pool = randn((cols, 2, Hkv, page, hd), TYPES[dtype], 1)
    table = torch.arange(cols, dtype=torch.int32, device="cuda").repeat(B, 1)
    starts = torch.tensor([0, rows] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    kv_len = torch.full((B,), kv, dtype=torch.int32, device="cuda")
    whole = randn((rows + 64, H, hd), TYPES[dtype], 2)
    out = torch.full_like(whole, 3.0)
    batch = model.paged_batch(table, starts, kv_len, rows, rows, kv, page, Hkv)
    before = pool.clone()
    model.paged_attention(batch, pool, whole[:rows], out=out[:rows])
    assert model.last_error() == RLT_EDEVICE
    assert bool((out[rows:] == 3.0).all()) and torch.equal(pool, before)
    good = model.paged_batch(table[:1], torch.tensor([0, rows], dtype=torch.int32, device="cuda"), kv_len[:1], rows, rows, kv,
                             page, Hkv)
    r = Ragged([rows], [kv], page, n_pages=cols)
    r.table_np[0] = np.arange(cols)
    got = model.paged_attention(good, pool, whole[:rows])
    assert model.last_error() == 0
    ref, tol = attention_ref(pool, r, whole[:rows])
    assert bool(((got.double() - ref).abs() <= tol).all())


def test_refusals():
    r = Ragged([2, 3], [20, 30], 16)
    model = op_model("bf16", 64, 64)
    batch = r.batch(model, 2)
    pool = torch.zeros((r.n_pages, 2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((5, 2, 64), device="cuda")
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16, device="cuda")
    ids = dict(table=r.table, q_start=r.q_start, kv_len=r.kv_len, N=5, max_q=3, max_kv=30, page_size=16, n_kv_heads=2)
    for kw in (dict(max_q=0), dict(max_q=6), dict(max_kv=2), dict(max_kv=33), dict(N=2), dict(table=r.table.long()),
               dict(kv_len=r.kv_len[:1]), dict(q_start=r.q_start[:2]), dict(table=r.table.cpu()),
               dict(table=r.table.t().contiguous().t())):
        with pytest.raises(ValueError):
            model.paged_batch(**{**ids, **kw})
    with pytest.raises(RLTError):                       # 48 is no page size
        odd = model.paged_batch(**{**ids, "page_size": 48})
        model.paged_attention(odd, torch.zeros((4, 2, 2, 48, 64), dtype=torch.bfloat16, device="cuda"), q)
    for call in (lambda: model.paged_append(batch, pool, kv[:4], kv),
                 lambda: model.paged_append(batch, pool.float(), kv, kv),
                 lambda: model.paged_append(batch, pool, kv.half(), kv.half()),
                 lambda: model.paged_append(batch, pool, kv, kv.bfloat16()),
                 lambda: model.paged_append(batch, pool, kv, kv, q_out=q),
                 lambda: model.paged_append(batch, pool, kv, kv, q=q),
                 lambda: model.paged_append(batch, pool[:, :, :1], kv, kv),
                 lambda: model.paged_append(batch, pool.transpose(2, 3).contiguous().transpose(2, 3), kv, kv),
                 lambda: model.paged_append(batch, pool, kv.transpose(1, 2).contiguous().transpose(1, 2), kv),
                 lambda: model.paged_attention(batch, pool, q.float()),
                 lambda: model.paged_attention(batch, pool, q[:4]),
                 lambda: model.paged_attention(batch, pool, q, out=q[:, :2]),
                 lambda: op_model("bf16", 64, 64).paged_attention(batch, pool, q)):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros((5, 4 * 64 + 4), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: model.paged_attention(batch, pool, torch.zeros((5, 3, 64), dtype=torch.bfloat16, device="cuda")),
                 lambda: model.paged_attention(batch, pool, q, scale=-1.0),
                 lambda: model.paged_attention(batch, pool, q, scale=float("nan")),
                 lambda: model.paged_attention(batch, pool, q, scale=float("inf")),
                 lambda: model.paged_attention(batch, pool, wide[:, :256].unflatten(1, (4, 64))),   # stride not of 8
                 lambda: model.paged_attention(batch, pool, wide[:, 2:258].unflatten(1, (4, 64))),
                 lambda: model.paged_attention(batch, pool, wide[:, 4:].unflatten(1, (4, 64)))):
        with pytest.raises(RLTError):
            call()
    torch.cuda.synchronize()
    assert model.last_error() == 0


# ------------------------------------------------------------------ the encoder over pages
ENCODERS = {
    "tiny-f32": TINY.model,
    "small-bf16": SMALL.model,
    "hd64-bf16": replace(TINY.model, dtype="bf16", d=256, n_heads=4, head_dim=64, F=512, W=8),
    "hd128-bf16-G2": replace(TINY.model, dtype="bf16", d=256, n_heads=2, head_dim=128, F=512, W=8, G=2),
}


def chunked_encoding(model, tok, plan, page, T_alloc, pad=0):
    """Encode tok [B, T] in the ragged calls of `plan` (new tokens of every sequence, call by call)."""
    B, T = tok.shape
    e, M = model.alloc_encoder_outputs(B, T_alloc)
    e.fill_(0)
    M.fill_(0)
    cols = -(-T_alloc // page)
    pools = model.alloc_pages(B * cols, page)
    pools.fill_(float("nan"))
    table = torch.randperm(B * cols, generator=torch.Generator().manual_seed(1)).int().view(B, cols).cuda()
    done = np.zeros(B, np.int64)
    for step in plan:
        step = np.asarray(step)
        new = np.concatenate([tok[b, done[b]:done[b] + n] for b, n in enumerate(step)] + [np.zeros(pad, np.int32)])
        done += step
        batch = model.paged_batch(table, torch.from_numpy(np.concatenate([[0], np.cumsum(step)]).astype(np.int32)).cuda(),
                                  torch.from_numpy(done.astype(np.int32)).cuda(), len(new), int(step.max()),
                                  int(max(done.max(), step.max())), page)
        model.encode_chunk(batch, pools, torch.from_numpy(new.astype(np.int32)).cuda(), e, M)
    assert (done == T).all()
    torch.cuda.synchronize()
    assert model.last_error() == 0
    return e, M


@pytest.mark.parametrize("name", list(ENCODERS))
def test_chunked_encoding_equals_token_parallel_encoding(name):
    cfg = ENCODERS[name]
    w = make_weights(cfg)
    B, T, T_alloc = 3, 150, 160
    model = build_model(cfg, max_pos=T_alloc, weights=w)
    tok = np.random.default_rng(4).integers(0, cfg.V, size=(B, T)).astype(np.int32)
    plan = [(30, 1, 0), (1, 1, 140), (64, 17, 1), (0, 130, 0), (55, 1, 9)]
    e, M = chunked_encoding(model, tok, plan, 16, T_alloc, pad=3)
    assert bool((e[:, T:] == 0).all()) and bool((M[:, :, :, :, T:] == 0).all())
    e, M = e[:, :T], M[:, :, :, :, :T]
    e_full, M_full = model.encode(torch.from_numpy(tok).cuda())
    e_o, M_o = RLTOracle(cfg, w).encode(tok)
    M_np = to_np(M).transpose(0, 1, 2, 4, 3, 5).reshape(cfg.G, 2, B, T, cfg.d)
    if cfg.dtype == "f32":
        assert np.abs(to_np(e) - to_np(e_full)).max() <= 1e-5 and np.abs(to_np(M) - to_np(M_full)).max() <= 1e-5
        assert np.abs(to_np(e) - e_o).max() <= 1e-5 and np.abs(M_np - M_o).max() <= 1e-5
    else:
        assert cosine(to_np(e).reshape(-1, cfg.d), to_np(e_full).reshape(-1, cfg.d)).min() >= 0.999
        assert cosine(to_np(e).reshape(-1, cfg.d), e_o.reshape(-1, cfg.d)).min() >= 0.999
        assert cosine(M_np.reshape(-1, cfg.d), M_o.reshape(-1, cfg.d)).min() >= 0.999


def test_chunk_refusals():
    cfg = ENCODERS["hd64-bf16"]
    model = build_model(cfg, max_pos=64)
    r = Ragged([2, 3], [20, 30], 16)
    batch = r.batch(model, cfg.n_heads)
    pools = model.alloc_pages(r.n_pages, 16)
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    e, M = model.alloc_encoder_outputs(2, 32)
    for args in ((pools[:1], tok, e, M), (pools, tok[:4], e, M), (pools, tok.long(), e, M), (pools, tok, e[:1], M),
                 (pools, tok, e, M[:, :1]), (pools, tok, e.float(), M)):
        with pytest.raises(ValueError):
            model.encode_chunk(batch, *args)
    with pytest.raises(RLTError):                       # e and M are shorter than the longest sequence
        model.encode_chunk(batch, pools, tok, *model.alloc_encoder_outputs(2, 29))
    with pytest.raises(RLTError):                       # no weights yet
        from cross_token_latent_b200 import RLTModel
        bare = RLTModel(cfg, max_pos=64)
        bare.encode_chunk(r.batch(bare, cfg.n_heads), pools, tok, e, M)
    assert model.last_error() == 0


def test_next_turn_of_a_conversation_f32():
    """The operators together: a paged prompt, decoder steps, tokens drawn under penalties and a mask,
    a second turn as one ragged chunk, and more draws.  Every next-token distribution equals the
    oracle's over the same tokens, and no draw leaves the mask."""
    cfg = TINY.model
    w = make_weights(cfg)
    model = build_model(cfg, max_pos=64, weights=w)
    B, page, T_alloc = 2, 16, 64
    rng = np.random.default_rng(3)
    prompts = [list(rng.integers(0, cfg.V, 9)), list(rng.integers(0, cfg.V, 4))]
    turns = [list(rng.integers(0, cfg.V, 5)), list(rng.integers(0, cfg.V, 12))]
    pools = model.alloc_pages(B * 4, page)
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4).flip(1).contiguous()
    e, M = model.alloc_encoder_outputs(B, T_alloc)
    allowed = np.zeros((1, cfg.V), bool)
    allowed[:, ::3] = True
    mask = torch.from_numpy(np.packbits(allowed, axis=1, bitorder="little").view(np.int32)).cuda()
    text = [list(p) for p in prompts]
    state = [model.new_state(1) for _ in range(B)]
    taken = [0] * B
    row, lse = torch.empty((1, cfg.V), device="cuda"), torch.empty(1, device="cuda")
    one = torch.ones(1, device="cuda")

    def encode(new):
        for b in range(B):
            text[b] += new[b]
        q, kv = [len(n) for n in new], [len(t) for t in text]
        batch = model.paged_batch(table, torch.tensor([0, q[0], q[0] + q[1]], dtype=torch.int32, device="cuda"),
                                  torch.tensor(kv, dtype=torch.int32, device="cuda"), sum(q), max(q), max(kv), page)
        flat = torch.tensor(sum(new, []), dtype=torch.int32, device="cuda")
        model.encode_chunk(batch, pools, flat, e, M)

    def advance(b):
        """Decoder steps of sequence b through all its tokens; the last one's distribution stays in row, lse."""
        eb, Mb = e[b:b + 1].contiguous(), M[:, :, b:b + 1].contiguous()
        while taken[b] < len(text[b]):
            model.decode_step(state[b], eb, Mb, lse=lse, logp_full=row)
            taken[b] += 1

    text = [[] for _ in range(B)]
    encode(prompts)
    oracle = RLTOracle(cfg, w)
    for turn in (turns, None):
        for _ in range(4):
            new = []
            for b in range(B):
                advance(b)
                ref = oracle.replay(np.asarray([text[b] + [0]], np.int32), 1, 1.0)
                history = torch.tensor([text[b]], dtype=torch.int32, device="cuda")
                z = to_np(row[0]).astype(np.float64) + float(lse)
                out = model.process_logits(row, lse=lse, mask=mask, tokens=history, repetition=one * 1.3, tau=one * 0.7)
                seen = np.zeros(cfg.V, bool)
                seen[text[b]] = True
                z = np.where(seen, np.where(z > 0, z / np.float32(1.3), z * np.float32(1.3)), z) / np.float32(0.7)
                z[~allowed[0]] = -np.inf
                want = z - np.log(np.exp(z - z.max()).sum()) - z.max()
                got = to_np(out[0])
                assert np.abs(got[allowed[0]] - want[allowed[0]]).max() <= 2e-5
                assert np.isneginf(got[~allowed[0]]).all()
                draw = int(model.sample(out, torch.tensor([0.37], device="cuda"))[0])
                assert allowed[0, draw]
                # the distribution itself is the oracle's over the same text
                lp_next = float(row[0, 0])
                assert abs(lp_next - float(ref[1][0, len(text[b]) - 1])) <= 1e-4
                new.append([draw])
            encode(new)
        if turn:
            encode(turn)
    assert model.last_error() == 0
