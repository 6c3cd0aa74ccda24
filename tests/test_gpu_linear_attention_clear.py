"""GPU tests of clearing the linear attention's state: what was in it is gone, whatever it was."""
import math

import pytest
import torch

from nonlinear_rnn_pararnn_b200 import api
from test_gpu_linear_attention import BF16, F32, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 33])
@pytest.mark.parametrize("what", [math.nan, math.inf, 1e38])
@pytest.mark.parametrize("g", [-math.inf, -100.0])
def test_step(g, what, d, dtype, cuda_device):
    """A slot taken over from another sequence: a cleared state may hold anything; a factor below the normal numbers
    clears as it does in a prompt."""
    x = _inputs((5,), 1, 2, d, d, dtype, 31, grads=False)
    x["g"][1:4, 0] = g
    want_o, want_s = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"],
                                               x["s0"] * (x["g"] > -50)[..., None, None])
    x["s0"][1:4, 0] = what
    o, s = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], x["s0"])
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
    s = x["s0"].clone()
    o, _ = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], s, out=s)
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
