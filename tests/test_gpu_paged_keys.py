"""Every key of the paged attention counts once, in every row that sees it: at the ends of pages, tiles,
units and shares, and at the causal end."""
import pytest
import torch

from paged_util import TYPES, Ragged, attention_ref, op_model

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, heads, kv heads, hd, page, new tokens, tokens in all
    ("bf16", 8, 8, 64, 64, [1, 1, 1], [5000, 1025, 4097]),
    ("bf16", 32, 8, 128, 16, [1] * 12, [700, 2049, 257, 8000, 1, 255, 256, 511, 3000, 1023, 64, 65]),
    ("bf16", 2, 2, 128, 128, [1], [30000]),
    ("bf16", 1, 1, 16, 16, [1, 20], [4000, 900]),
    ("bf16", 4, 4, 32, 32, [130, 1], [1500, 2000]),
    ("bf16", 4, 4, 64, 64, [300, 77, 129, 1], [3000, 1500, 129, 600]),
    ("bf16", 16, 16, 64, 16, [700, 200, 100, 400, 1, 300], [4000, 3400, 600, 2100, 77, 300]),
    ("bf16", 4, 4, 128, 256, [300, 77, 129], [3000, 1500, 129]),
    ("bf16", 3, 1, 128, 64, [1000, 40], [5000, 9000]),
    ("bf16", 1, 1, 64, 64, [513], [12000]),
    ("bf16", 2, 2, 128, 64, [128, 256], [384, 512]),
    ("f32", 2, 2, 64, 16, [1, 40], [5000, 300]),
    ("f32", 4, 1, 16, 32, [9, 1], [2000, 4000]),
    ("f32", 1, 1, 128, 64, [70, 1], [1100, 9000]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + f"-{len(c[5])}x{max(c[5])}-{max(c[6])}")
def test_every_key_counts_once(case):
    """Queries of zero give every key the weight 1.  Value element c of key j is 1 where j = c + offset
    (mod m), else 0, so a row at position t is the number of such keys up to t divided by t + 1.

    Counts and t + 1 are whole numbers below 2^24, exact in float32; the division is off by two roundings of
    2^-24 and the result by half a step.  With m >= t / 60 a count is 61 at most, and one key more or less
    changes the row by at least 1 / 61, four times the half step of bf16."""
    dtype, H, Hkv, hd, page, q_len, kv_len = case
    r = Ragged(q_len, kv_len, page, seed=3)
    model = op_model(dtype, hd, r.max_kv)
    m = max(hd, -(-r.max_kv // 60))
    q = torch.zeros((r.N, H, hd), dtype=TYPES[dtype], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.empty((r.n_pages, 2, Hkv, page, hd), dtype=TYPES[dtype], device="cuda").normal_(generator=g)
    batch = r.batch(model, Hkv)
    half = torch.finfo(TYPES[dtype]).eps / 2
    cols = torch.arange(hd, device="cuda")
    for offset in range(0, m, hd):
        for b, n in enumerate(r.kv):
            keys = torch.arange(-(-n // page) * page, device="cuda")
            mark = (keys[:, None] % m == (cols + offset) % m).to(pool.dtype)
            mark[n:] = float("nan")
            pages = torch.from_numpy(r.table_np[b, :-(-n // page)]).long().cuda()
            pool[pages, 1] = mark.view(-1, 1, page, hd)
        out = model.paged_attention(batch, pool, q)
        assert model.last_error() == 0
        at = torch.tensor([t for _, t in r.rows()], device="cuda")
        residue = (cols + offset) % m
        count = torch.where(at[:, None] >= residue, (at[:, None] - residue) // m + 1, 0)
        want = (count.double() / (at[:, None] + 1))[:, None]
        bad = (out.double() - want).abs() > want * (half + 2 * 2.0 ** -24) * (1 + 2.0 ** -8)
        assert not bool(bad.any()), (offset, bad.nonzero()[:4].tolist())


LONG = [
    ("bf16", 8, 8, 64, 64, [1] * 6, [5000, 1025, 8000, 9000, 2000, 7000]),
    ("bf16", 16, 4, 128, 16, [1] * 4, [20000, 5000, 12000, 30000]),
    ("bf16", 8, 8, 64, 64, [300, 129, 60], [5000, 6000, 20000]),
    ("bf16", 4, 4, 128, 32, [200, 129, 60], [5000, 6000, 20000]),
    ("bf16", 4, 4, 32, 32, [100], [6000]),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c[:5])) + f"-{len(c[5])}x{max(c[5])}-{max(c[6])}")
def test_the_error_of_long_contexts_is_that_of_the_roundings(case):
    """Norm of the error over the norm of the result.  A rounding to bf16 has a relative error of at most
    2^-8, evenly spread, so 2^-8 / sqrt(3) = 0.0023 in the mean square at most.  The result is rounded
    once; rounded weights change a weighted mean of independent values by as much again at most: 0.0032
    together, and 0.005 leaves room for few rows.  (A key left out of 5000 costs some 0.014.)"""
    dtype, H, Hkv, hd, page, q_len, kv_len = case
    r = Ragged(q_len, kv_len, page, seed=4)
    model = op_model(dtype, hd, r.max_kv)
    g = torch.Generator(device="cuda").manual_seed(9)
    pool = torch.empty((r.n_pages, 2, Hkv, page, hd), dtype=TYPES[dtype], device="cuda").normal_(generator=g)
    q = torch.empty((r.N, H, hd), dtype=TYPES[dtype], device="cuda").normal_(generator=g)
    out = model.paged_attention(r.batch(model, Hkv), pool, q)
    assert model.last_error() == 0
    for b, n in enumerate(r.q):             # the reference holds one sequence's scores at a time
        one = Ragged([n], [r.kv[b]], page, n_pages=r.n_pages)
        one.table_np = r.table_np[b:b + 1]
        rows = slice(int(r.starts[b]), int(r.starts[b + 1]))
        ref, _ = attention_ref(pool, one, q[rows])
        assert float((out[rows].double() - ref).norm() / ref.norm()) <= 0.005, b
