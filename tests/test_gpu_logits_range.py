"""Temperatures and penalties at the ends of float32's range give numbers, and those that have no finite
reciprocal are refused."""
import numpy as np
import pytest
import torch

from paged_util import op_model
from test_gpu_logits import RLT_EDEVICE, check, dev, reference
from gpu_util import to_np

pytestmark = pytest.mark.gpu

SHAPES = [(64, 3), (8200, 40), (20008, 3), (140000, 2)]


def rows(V, B, seed):
    r = np.random.default_rng([seed, V])
    x = (r.standard_normal((B, V)) * 4).astype(np.float32)
    x[:, V // 3] = 0.0                                      # zeros, and a greatest logit of zero
    x[0] = -np.abs(x[0])
    x[1, 5] = x[1, V - 2] = np.float32(30.0)                # two that share the maximum
    return x


@pytest.mark.parametrize("with_lse", [False, True])
@pytest.mark.parametrize("V,B", SHAPES)
def test_temperatures_at_the_ends_of_the_range(V, B, with_lse):
    """out = (z - max) / tau - log sum: z - max is off by a rounding, the reciprocal, the product and the sum
    by one each, 2^-24 of what they round; the logarithm by 2^-21 (its sum's exponentials have 2^-22).  With lse,
    x is given less lse, rounded once at the size of the greater."""
    model = op_model("f32", 16, 8, V=V)
    x = rows(V, B, 1)
    lse = np.linspace(1, 9, B).astype(np.float32) if with_lse else None
    given = x - lse[:, None] if with_lse else x
    z = given.astype(np.float64)
    for tau in (2.0 ** -126, 1e-37, 1e-30, 1e-6, 1e6, 1e30, 3.4e38):
        t = np.full(B, tau, np.float32)
        out_lse = torch.empty(B, device="cuda")
        got = to_np(model.process_logits(dev(given), lse=dev(lse), tau=dev(t), out_lse=out_lse))
        assert model.last_error() == 0
        d = (z - z.max(1, keepdims=True)) / np.float64(t[0])
        want = d - np.log(np.exp(d).sum(1, keepdims=True))
        assert not np.isnan(got).any() and not np.isnan(to_np(out_lse)).any()
        inside = want > -3.4e38                             # what lies beyond is -inf in float32
        err = np.abs(got[inside] - want[inside])
        assert (err <= 5 * 2.0 ** -24 * np.abs(want[inside]) + 2.0 ** -21).all(), (tau, float(err.max()))
        assert (got[~inside] < -3.3e38).all()


@pytest.mark.parametrize("V,B", SHAPES)
def test_repetitions_at_the_ends_of_the_range(V, B):
    model = op_model("f32", 16, 8, V=V)
    x = rows(V, B, 2)
    x[:, 3], x[:, 4] = 20.0, -20.0
    tokens = np.tile(np.array([[3, V // 3]], np.int32), (B, 1))          # a logit above 0, and one of 0
    for rep in (2.0 ** -100, 2.0 ** -126, 2.0 ** 100, 3.4e38):
        for ids in (tokens, np.full((B, 2), 4, np.int32)):
            r = np.full(B, rep, np.float32)
            got = to_np(model.process_logits(dev(x), tokens=dev(ids), repetition=dev(r)))
            assert model.last_error() == 0 and not np.isnan(got).any()
            z = x.astype(np.float64)
            for v in set(ids[0].tolist()):
                z[:, v] = np.where(z[:, v] > 0, z[:, v] / np.float64(r[0]), z[:, v] * np.float64(r[0]))
            z = z.clip(-3.4028234663852886e38, 3.4028234663852886e38)
            d = z - z.max(1, keepdims=True)
            want = d - np.log(np.exp(d).sum(1, keepdims=True))
            err = np.abs(got - want)
            # 4 roundings of the difference, and the logarithm's 2^-21
            ok = err <= 2.0 ** -22 * np.abs(want) + 2.0 ** -21
            assert (ok | ((got < -3.3e38) & (want < -3.3e38))).all(), (rep, float(err[~ok].max()))


def test_the_only_token_left_survives_its_penalty():
    """A penalty beyond the range leaves the token that a mask allows: the row is not empty."""
    V = 64
    model = op_model("f32", 16, 8, V=V)
    x = np.full((1, V), -20.0, np.float32)
    allowed = np.full((1, 2), 0, np.int32)
    allowed[0, 0] = 1 << 4
    got = model.process_logits(dev(x), mask=dev(allowed), tokens=dev(np.array([[4]], np.int32)),
                               repetition=dev(np.array([3.4e38], np.float32)))
    assert model.last_error() == 0
    got = to_np(got)
    assert got[0, 4] == 0.0 and np.isneginf(np.delete(got[0], 4)).all()


@pytest.mark.parametrize("V,B", SHAPES)
def test_values_without_a_finite_reciprocal_are_latched_and_taken_as_one(V, B):
    model = op_model("f32", 16, 8, V=V)
    x = rows(V, B, 3)
    tokens = np.tile(np.arange(6, dtype=np.int32), (B, 1))
    for bad in (1e-39, 1e-45, np.inf, -np.inf, -1e-40, 0.0, np.nan):
        for name in ("repetition", "tau"):
            par = {"repetition": np.full(B, 1.5, np.float32), "tau": np.full(B, 0.75, np.float32)}
            par[name][1] = bad
            got = model.process_logits(dev(x), tokens=dev(tokens), **{k: dev(v) for k, v in par.items()})
            assert model.last_error() == RLT_EDEVICE and model.last_error() == 0
            par[name][1] = 1.0
            want, _, tol = reference(x, tokens=tokens, **par)
            check(got, want, tol)
