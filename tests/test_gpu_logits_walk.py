"""Logits of more rows than clusters fit on the GPU: every cluster walks through four rows at least, each with
a history, a bias and a mask of its own."""
import numpy as np
import pytest
import torch

from paged_util import op_model
from test_gpu_logits import bits, check, dev, inputs, reference

pytestmark = pytest.mark.gpu

WALKS = [
    # V, CTAs per row, CTAs per SM, history, offset of the rows from a 16-byte boundary in elements
    (520, 1, 4, 30, 0),
    (520, 1, 4, 30, 1),
    (2056, 1, 4, 1100, 0),
    (4096, 1, 4, 1500, 0),
    (4160, 1, 2, 1300, 0),
    (4160, 1, 2, 1300, 3),
    (9008, 1, 2, 1200, 0),
    (9008, 1, 2, 100, 1),
    (16416, 2, 2, 1200, 0),
]


@pytest.mark.parametrize("V,n_cta,per_sm,hist,offset", WALKS)
def test_rows_behind_rows(V, n_cta, per_sm, hist, offset):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = 3 * (sms * per_sm // n_cta) + 5
    model = op_model("f32", 16, 8, V=V)
    r, x, tokens, tok_len, gen, par = inputs(B, V, hist, 21)
    bias = (r.standard_normal((B, V)) * (r.random((B, V)) < 0.2)).astype(np.float32)
    allowed = r.random((B, V)) < 0.5
    allowed[:, V // 2] = True
    lse = r.uniform(5, 12, B).astype(np.float32)
    want, _, tol = reference(x, lse=lse, bias=bias, allowed=allowed, tokens=tokens, tok_len=tok_len, gen_start=gen, **par)
    wide = [torch.zeros((B, V + 8), device="cuda")[:, offset:offset + V] for _ in range(3)]
    wide[0].copy_(torch.from_numpy(x))
    wide[1].copy_(torch.from_numpy(bias))
    kw = dict(lse=dev(lse), bias=wide[1], mask=bits(allowed), tokens=dev(tokens), tok_len=dev(tok_len), gen_start=dev(gen),
              **{k: dev(v) for k, v in par.items()})
    model.process_logits(wide[0], out=wide[2], **kw)
    assert model.last_error() == 0
    check(wide[2], want, tol)
    # in place, and the same bits again
    model.process_logits(wide[0], out=wide[0], **kw)
    assert torch.equal(wide[0], wide[2])


@pytest.mark.parametrize("V,rows,hist", [(262144, 40, 200), (40000, 160, 66000)])
def test_rows_behind_rows_with_counters_of_32_bits(V, rows, hist):
    """Vocabularies or histories for which the counters take 32 bits; row b's history is the one buffer from its
    token 7 b on, so that histories overlap and differ."""
    model = op_model("f32", 16, 8, V=V)
    r, x, tokens, _, _, par = inputs(1, V, hist + 7 * rows, 22)
    x = np.tile(x, (rows, 1)) + np.arange(rows, dtype=np.float32)[:, None] * np.float32(0.125)
    par = {k: np.linspace(v[0] * 0.9, v[0] * 1.1, rows).astype(np.float32) for k, v in par.items()}
    histories = np.lib.stride_tricks.as_strided(tokens[0], (rows, hist), (28, 4))
    tok_len = r.integers(hist // 2, hist + 1, rows).astype(np.int32)
    gen = (tok_len * r.random(rows)).astype(np.int32)
    allowed = np.tile(r.random((1, V)) < 0.5, (rows, 1))
    allowed[1::2] ^= True
    buffer = dev(tokens[0])
    out = model.process_logits(dev(x), mask=bits(allowed), tokens=buffer.as_strided((rows, hist), (7, 1)), tok_len=dev(tok_len),
                               gen_start=dev(gen), **{k: dev(v) for k, v in par.items()})
    assert model.last_error() == 0
    for b in range(rows):                                   # (a row at a time: the reference holds many copies)
        one = slice(b, b + 1)
        want, _, tol = reference(x[one], allowed=allowed[one], tokens=histories[one], tok_len=tok_len[one], gen_start=gen[one],
                                 **{k: v[one] for k, v in par.items()})
        check(out[one], want, tol)
