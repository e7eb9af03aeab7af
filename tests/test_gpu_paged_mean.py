"""The paged attention's result is a weighted mean of the values: the weights that are summed are the
weights that multiply."""
import pytest
import torch

from paged_util import Ragged, op_model

pytestmark = pytest.mark.gpu

CASES = [
    # heads, kv heads, hd, page, new tokens, tokens in all
    (4, 4, 64, 64, [300, 129], [300, 900]),
    (4, 4, 128, 16, [300, 129], [300, 900]),
    (6, 2, 128, 32, [257, 43], [257, 1800]),
    (3, 1, 64, 128, [700], [1500]),
    (4, 4, 64, 16, [1, 1, 5], [1, 900, 70]),
    (16, 2, 128, 64, [1, 1], [3, 1900]),
    (4, 4, 32, 16, [40, 1], [40, 700]),
    (2, 2, 16, 16, [33], [400]),
]


@pytest.mark.parametrize("H,Hkv,hd,page,q_len,kv_len", CASES)
def test_equal_values_come_back_as_they_are(H, Hkv, hd, page, q_len, kv_len):
    """All values of a key head are one number c of the largest bf16 significand: the mean is c.

    The products w c of bf16 weights are exact in float32; numerator and denominator are off by n 2^-23
    each for n < 2000 summands, and by one rounding for each rescale and for the division: less than 2^-10
    together, while the result would have to be off by half a step, 2^-9 of c, to be rounded to another
    number."""
    r = Ragged(q_len, kv_len, page)
    model = op_model("bf16", hd, r.max_kv)
    g = torch.Generator(device="cuda").manual_seed(hd + H)
    pool = torch.empty((r.n_pages, 2, Hkv, page, hd), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    c = torch.tensor([1.9921875, -0.99609375, 3.984375, -1.9921875], device="cuda")[:Hkv].bfloat16()
    pool[:, 1] = c[None, :, None, None]
    q = torch.empty((r.N, H, hd), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    for scale in (0.05, 0.3):
        out = model.paged_attention(r.batch(model, Hkv), pool, q, scale=scale)
        assert model.last_error() == 0
        want = c.repeat_interleave(H // Hkv)[None, :, None].expand_as(out)
        assert torch.equal(out, want), (int((out != want).sum()), out[out != want][:4].tolist())
