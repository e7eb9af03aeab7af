"""Draws from rows that a mask leaves without a token, or with few: defined, latched, and never a forbidden
token."""
import numpy as np
import pytest
import torch

from cross_token_latent_b200 import RLTError
from workloads import TINY, make_weights
from gpu_util import build_model, to_np
from paged_util import op_model
from test_gpu_logits import RLT_EDEVICE, bits, dev

pytestmark = pytest.mark.gpu


def draw(model, rows, u, **kw):
    blp = torch.full((rows.shape[0],), 7.0, device="cuda")
    tok = model.sample(dev(rows), dev(np.asarray(u, np.float32)), behaviour_logp=blp, **kw)
    return tok.cpu().numpy(), to_np(blp)


@pytest.mark.parametrize("kw", [{}, dict(top_p=0.9), dict(top_k=5), dict(top_k=3, top_p=0.5)], ids=str)
@pytest.mark.parametrize("V", [8, 1000, 32768])
def test_a_row_without_probability(V, kw):
    model = op_model("f32", 16, 8, V=V)
    r = np.random.default_rng(V)
    rows = np.log(r.dirichlet(np.ones(V), 3)).astype(np.float32)
    u = [0.2, 0.7, 0.9]
    want = draw(model, rows, u, **kw)
    assert model.last_error() == 0
    for bad, log_p in ((-np.inf, -np.inf), (np.nan, np.nan)):
        x = rows.copy()
        x[1] = bad
        tok, blp = draw(model, x, u, **kw)
        assert model.last_error() == RLT_EDEVICE and model.last_error() == 0
        assert tok[1] == 0 and np.array_equal(blp[1], np.float32(log_p), equal_nan=True)
        assert tok[0] == want[0][0] and tok[2] == want[0][2] and blp[0] == want[1][0] and blp[2] == want[1][2]


@pytest.mark.parametrize("kw", [{}, dict(top_p=0.999), dict(top_k=7)], ids=str)
def test_a_token_without_probability_is_never_drawn(kw):
    """Uniforms at the very end of their range, and at it, with forbidden ids behind the last allowed one and in
    front of the first; fewer allowed ids than top_k keeps."""
    V = 5000
    model = op_model("f32", 16, 8, V=V)
    allowed = [1234, 1236, 4000]
    rows = np.full((4, V), -np.inf, np.float32)
    rows[:, allowed] = np.log(np.float32(1 / 3))
    tok, blp = draw(model, rows, [0.0, 0.5, 1 - 2.0 ** -24, 1.0], **kw)
    assert model.last_error() == 0
    assert tok.tolist() == [1234, 1236, 4000, 4000]
    assert np.abs(blp - np.log(1 / 3)).max() <= 1e-6


def test_generation_whose_grammar_leaves_a_row_empty_raises():
    cfg = TINY.model
    model = build_model(cfg, max_pos=24, weights=make_weights(cfg))
    prompt = np.random.default_rng(2).integers(0, cfg.V, size=(2, 4)).astype(np.int32)
    u = torch.rand((6, 2), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    everything = np.ones((2, cfg.V), bool)
    nothing = everything.copy()
    nothing[1] = False
    seen = []

    def grammar(step, tokens):
        seen.append(tokens)
        return bits(nothing if step == 3 else everything)

    with pytest.raises(RLTError) as e:
        model.generate(dev(prompt), 6, u, mask=grammar)
    assert e.value.code == RLT_EDEVICE and len(seen) == 6 and model.last_error() == 0
    toks = seen[-1].cpu().numpy()
    assert toks[1, 4 + 3] == 0                            # the draw from nothing
    # a bias that forbids everything does the same; the handle goes on
    with pytest.raises(RLTError):
        model.generate(dev(prompt), 2, u[:2], bias=torch.full((1, cfg.V), -torch.inf, device="cuda"))
    again, blp, _, _ = model.generate(dev(prompt), 6, u, mask=bits(everything))
    assert model.last_error() == 0 and bool(torch.isfinite(blp).all())
    plain, blp0, _, _ = model.generate(dev(prompt), 6, u)
    assert torch.equal(again, plain) and float((blp - blp0).abs().max()) <= 1e-5


def test_a_controlled_generation_can_be_captured():
    cfg = TINY.model
    model = build_model(cfg, max_pos=24, weights=make_weights(cfg))
    prompt = dev(np.random.default_rng(2).integers(0, cfg.V, size=(2, 4)).astype(np.int32))
    u = torch.rand((5, 2), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    allowed = np.ones((2, cfg.V), bool)
    allowed[:, ::2] = False
    mask = bits(allowed)
    toks, blp, *_ = model.generate(prompt, 5, u, repetition=1.3, mask=mask)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = model.generate(prompt, 5, u, repetition=1.3, mask=mask)
    graph.replay()
    torch.cuda.synchronize()
    assert model.last_error() == 0
    assert torch.equal(kept[0], toks) and torch.equal(kept[1], blp)
    mask[1] = 0
    graph.replay()
    assert model.last_error() == RLT_EDEVICE and model.last_error() == 0
    assert torch.equal(kept[0][0], toks[0]) and bool((kept[0][1, 4:] == 0).all())
