"""GPU tests of the linear attention on long rows: several of them shared out in segments, and gradients of tensors of
more than 2^31 elements."""
import pytest
import torch

import la_reference as ref
from nonlinear_rnn_pararnn_b200 import api
from test_gpu_linear_attention import BF16, _check, _dense, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,dk,dv,per_head", [(3, 1500, 2, 64, 64, False), (2, 2500, 1, 128, 72, True),
                                                  (5, 2500, 2, 32, 128, False), (14, 1100, 2, 32, 128, False)])
def test_several_rows_in_segments(B, T, H, dk, dv, per_head, cuda_device):
    """Few heads of a batch of long rows: each is cut into segments of four chunks or more, one of them ragged (the
    rows of the last case stay whole)."""
    x = _inputs((B, T), 1, H, dk, dv, BF16, 71, per_head=per_head, resets=0 if per_head else 700)
    want, size = _dense(x, 0.125)
    _check(_run(x, 0.125), want, size, BF16, T, dk, dv, H)


@pytest.mark.parametrize("H,dk,dv,dtype", [(16, 128, 128, BF16), (16, 8, 250, BF16)])
def test_gradients_beyond_32_bits(H, dk, dv, dtype, cuda_device):
    """The last sequence of more than 2^31 elements has the gradients that it has alone, in the rows of its own."""
    last, wide = 500, H * max(dk, dv)
    total = 2 ** 31 // wide + 1000
    tail = _inputs((last,), H, H, dk, dv, dtype, 72, nseq=1)
    x = {}
    for n in ("q", "k", "v", "g", "dO"):
        x[n] = torch.zeros(total, *tail[n].shape[1:], dtype=tail[n].dtype, device="cuda")
        x[n][-last:] = tail[n]
    cu = torch.tensor([0, total - last, total], dtype=torch.int32, device="cuda")
    s0, dsT = (torch.cat([torch.zeros_like(tail[n]), tail[n]]) for n in ("s0", "dsT"))
    got = api.linear_attention_backward_varlen(x["q"], x["k"], x["v"], x["g"], s0, cu, x["dO"], dsT)
    want = api.linear_attention_backward_varlen(*(tail[n] for n in ("q", "k", "v", "g", "s0")),
                                                torch.tensor([0, last], dtype=torch.int32, device="cuda"),
                                                tail["dO"], tail["dsT"])
    assert torch.equal(got["ds0"][1:], want["ds0"]) and (got["ds0"][0] == 0).all()
    for n in ("dq", "dk", "dv", "dg"):
        assert not got[n][:-last].any(), n
        # On the CUDA cores many chunks take blocks of 128 threads and few of 256, and <S, dS> of a chunk is summed by
        # thread: d_k d_v / 128 or / 256 fp32 terms in turn, then over the threads.  dg is held against 64 bits there.
        if n != "dg" or dv % 8 == 0:
            assert torch.equal(got[n][-last:], want[n]), n
    exact, size = ref.values({n: (y[0] if n in ("s0", "dsT") else y) for n, y in tail.items()}, dk ** -0.5)
    _check({n: got[n][-last:] for n in ("dq", "dk", "dv", "dg")}, exact, size, dtype, last, dk, dv, 1)
