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


CASES = [
    # dtype, d_k, d_v, T, where the state is cleared, packed
    (F32, 40, 33, 150, [70], False),
    (F32, 64, 64, 100, [0], True),
    (BF16, 64, 64, 150, [0], False),
    (BF16, 128, 72, 300, [37, 201], False),
    (BF16, 128, 128, 300, [127], True),
    (BF16, 64, 128, 3000, [900, 901, 1700], False),   # segments
    (BF16, 33, 20, 150, [131], False),
]


@pytest.mark.parametrize("dtype,dk,dv,T,at,packed", CASES)
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_in_chunks(what, dtype, dk, dv, T, at, packed, cuda_device):
    """Behind a clear everything is as if the state in front of it had been nothing; and in front of the last one
    the gradients are as if that of the final state had been."""
    x = _inputs((1, T), 1, 2, dk, dv, dtype, 32 + T)
    x["g"][:, at] = -math.inf
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def run(s0, dsT):
        q, k, v, g, dO = (x[n][0] if packed else x[n] for n in ("q", "k", "v", "g", "dO"))
        if packed:
            o, sT = api.linear_attention_forward_varlen(q, k, v, g, s0, cu)
            out = api.linear_attention_backward_varlen(q, k, v, g, s0, cu, dO, dsT)
        else:
            o, sT = api.linear_attention_forward(q, k, v, g, s0)
            out = api.linear_attention_backward(q, k, v, g, s0, dO, dsT)
        out.update(o=o, sT=sT)
        return {n: y if n in ("sT", "ds0") else y.view(T, *y.shape[-2:] if y.dim() > 3 - packed else y.shape[-1:])
                for n, y in out.items()}

    zero = torch.zeros_like(x["s0"])
    want, got = run(zero, x["dsT"]), run(zero + what, x["dsT"])
    for n in ("sT", "ds0", "dk", "dv"):
        assert torch.equal(got[n], want[n]), n
    for n in ("o", "dq", "dg"):
        assert torch.equal(got[n][at[0]:], want[n][at[0]:]), n
        assert at[0] == 0 or not torch.isfinite(got[n][:at[0]]).all(), n
    want, got = run(x["s0"], zero), run(x["s0"], zero + what)
    for n in ("o", "sT", "dq", "ds0"):
        assert torch.equal(got[n], want[n]), n
    for n in ("dk", "dv"):
        assert torch.equal(got[n][:at[-1]], want[n][:at[-1]]), n
    assert torch.equal(got["dg"][:at[-1] + 1], want["dg"][:at[-1] + 1])
    assert not torch.isfinite(got["dk"][at[-1]:]).all()
