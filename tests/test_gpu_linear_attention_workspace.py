"""GPU tests of the workspaces and states that a caller of the linear attention brings."""
import pytest
import torch

from nonlinear_rnn_pararnn_b200 import api
from test_gpu_linear_attention import BF16, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("with_k", [False, True])
def test_keys_of_another_spacing(with_k, packed, cuda_device):
    """q and v whose tokens lie multiples of 8 apart, and k a slice whose do not: other kernels, which need more."""
    x = _inputs((300,) if packed else (2, 150), 1, 2, 64, 64, BF16, 51, nseq=2)
    wide = torch.zeros(*x["k"].shape[:-1], 67, dtype=BF16, device="cuda")
    wide[..., 3:] = x["k"]
    k = wide[..., 3:]
    kw = {"k": k} if with_k else {}
    ws = [api.linear_attention_workspace(x["q"], x["v"], x["g"], backward=b, n_seq=2 if packed else 0, **kw)
          for b in (False, True)]
    a = [x["q"], k, x["v"], x["g"], x["s0"]]
    if packed:
        a.append(torch.tensor([0, 90, 300], dtype=torch.int32, device="cuda"))
    fwd = api.linear_attention_forward_varlen if packed else api.linear_attention_forward
    bwd = api.linear_attention_backward_varlen if packed else api.linear_attention_backward
    for y, z in zip(fwd(*a), fwd(*a, ws=ws[0])):
        assert torch.equal(y, z)
    want, got = bwd(*a, x["dO"], x["dsT"]), bwd(*a, x["dO"], x["dsT"], ws=ws[1])
    assert all(torch.equal(want[n], got[n]) for n in want)
    # and k like q
    a[1] = x["k"]
    fwd(*a, ws=api.linear_attention_workspace(x["q"], x["v"], x["g"], n_seq=2 if packed else 0))


def test_misaligned_states(cuda_device):
    """A slot of a cache of odd states may start on no 16 bytes: refused by name, wherever a state is taken."""
    x = _inputs((1, 5), 1, 1, 3, 3, torch.float32, 52)
    q, k, v, g = (x[n] for n in ("q", "k", "v", "g"))
    s = torch.zeros(3, 1, 3, 3, device="cuda")[1:2]
    one = [t[:, 0].contiguous() for t in (q, k, v, g)]
    for name, call in (("s0", lambda: api.linear_attention_forward(q, k, v, g, s)),
                       ("sT", lambda: api.linear_attention_forward(q, k, v, g, sT=s)),
                       ("s0", lambda: api.linear_attention_backward(q, k, v, g, s, x["dO"])),
                       ("dsT", lambda: api.linear_attention_backward(q, k, v, g, None, x["dO"], s)),
                       ("ds0", lambda: api.linear_attention_backward(q, k, v, g, None, x["dO"], out={
                           "dq": q.clone(), "dk": q.clone(), "dv": v.clone(), "ds0": s})),
                       ("s_prev", lambda: api.linear_attention_step(*one, s)),
                       ("out", lambda: api.linear_attention_step(*one, out=s))):
        with pytest.raises(ValueError, match=f"{name} must be 16-byte aligned"):
            call()
    o, _ = api.linear_attention_forward(q, k, v, g, s.clone())
    assert torch.equal(o, api.linear_attention_forward(q, k, v, g)[0])
