"""Scores of the paged attention that are no numbers show in the outputs that they belong to, and in no
others."""
import pytest
import torch

from paged_util import TYPES, Ragged, attention_ref, op_model

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, heads, kv heads, hd, page, new tokens, tokens in all
    ("bf16", 2, 2, 64, 64, [200], [500]),
    ("bf16", 4, 2, 128, 16, [150], [700]),
    ("bf16", 4, 2, 128, 32, [1, 40], [300, 300]),
    ("bf16", 4, 2, 64, 16, [1], [300]),
    ("bf16", 2, 1, 16, 16, [9], [200]),
    ("f32", 2, 1, 32, 16, [9], [200]),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + f"-{max(c[5])}-{max(c[6])}")
def test_a_score_that_is_no_number_makes_its_rows_nan(case, bad):
    """One key at a time holds a bad element that every query meets with a positive factor, so that its
    scores are NaN or +inf.  Rows that see the key are NaN throughout (inf - inf is NaN); rows in front of
    it, the other key heads' and the other sequences' are what they are without it."""
    dtype, H, Hkv, hd, page, q_len, kv_len = case
    r = Ragged(q_len, kv_len, page, seed=2)
    model = op_model(dtype, hd, r.max_kv)
    g = torch.Generator(device="cuda").manual_seed(5)
    pool = torch.empty((r.n_pages, 2, Hkv, page, hd), dtype=TYPES[dtype], device="cuda").normal_(generator=g)
    q = torch.empty((r.N, H, hd), dtype=TYPES[dtype], device="cuda").normal_(generator=g)
    q[..., 3] = q[..., 3].abs() + 0.5
    batch = r.batch(model, Hkv)
    ref, tol = attention_ref(pool, r, q)
    b = r.B - 1
    n, kv, group = r.q[b], r.kv[b], H // Hkv
    head = Hkv - 1
    # every place in a block of 32 keys, and the ends
    for key in sorted({*range(64, 96), 0, 1, kv - n, kv - 1 - n // 2, kv - 2, kv - 1}):
        p, s = r.place(b, key)
        kept = pool[p, 0, head, s, 3].clone()
        pool[p, 0, head, s, 3] = bad
        out = model.paged_attention(batch, pool, q)
        pool[p, 0, head, s, 3] = kept
        hit = torch.zeros((r.N, H), dtype=torch.bool, device="cuda")
        first = int(r.starts[b]) + max(0, key - (kv - n))           # the first row that sees it
        hit[first:int(r.starts[b + 1]), head * group:] = True
        nan = torch.isnan(out)
        assert bool((nan.all(-1) == hit).all()) and bool((nan.any(-1) == hit).all()), (key, int(hit.sum()),
                                                                                      int(nan.all(-1).sum()))
        assert bool((((out.double() - ref).abs() <= tol) | hit[..., None]).all()), key
    assert model.last_error() == 0
