"""Lengths of a history without tokens are checked like those of any other."""
import ctypes

import numpy as np
import pytest
import torch

from cross_token_latent_b200 import lib
from cross_token_latent_b200.rlt import LogitsArgs
from paged_util import op_model
from test_gpu_logits import RLT_EDEVICE, check, dev, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [64, 140000])
def test_lengths_without_tokens(V):
    B = 3
    model = op_model("f32", 16, 8, V=V)
    x = np.random.default_rng(1).standard_normal((B, V)).astype(np.float32)
    want, _, tol = reference(x)
    none = torch.empty((B, 0), dtype=torch.int32, device="cuda")
    for lens, status in (([0, 0, 0], 0), ([0, 1, 0], RLT_EDEVICE), ([0, 0, -1], RLT_EDEVICE)):
        got = model.process_logits(dev(x), tokens=none, tok_len=dev(np.array(lens, np.int32)))
        assert model.last_error() == status and model.last_error() == 0
        check(got, want, tol)
    # n_tokens says nothing where there are no tokens
    out = torch.zeros((B, V), device="cuda")
    given = dev(x)
    a = LogitsArgs(x=given.data_ptr(), x_stride=V, out=out.data_ptr(), out_stride=V, n_tokens=-5)
    assert lib().rlt_process_logits(model.handle, ctypes.byref(a), B, None) == 0
    assert model.last_error() == 0
    check(out, want, tol)
