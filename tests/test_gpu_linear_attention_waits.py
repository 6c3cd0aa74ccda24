"""GPU tests of the linear attention's bounded waits on the tensor cores: where one runs out, the outputs that hang on
it are NaN, and the others are what they always are.  The waits run out because the kernels' loading warp stops
(debug_fault); nothing on the device faults or hangs."""
import ctypes

import pytest
import torch

from nonlinear_rnn_pararnn_b200 import _lib, api
from test_gpu_linear_attention import BF16, _inputs

pytestmark = pytest.mark.gpu


def _call(x, fault, backward, packed, mark):
    lead, (Hqk, dk), (H, dv) = x["q"].shape[:-2], x["q"].shape[-2:], x["v"].shape[-2:]
    per_head = x["g"].dim() == 1
    cfg = _lib.LinearAttentionConfig(H, Hqk, dk, dv, _lib.SLSTM_BF16,
                                     _lib.SLSTM_DECAY_HEAD if per_head else _lib.SLSTM_DECAY_TOKEN, 0.125, Hqk * dk,
                                     Hqk * dk, H * dv, fault, 1000 if fault else 0)
    lib, c = _lib.load(), ctypes.byref(cfg)
    cu = torch.tensor(packed, dtype=torch.int32, device="cuda") if packed else None
    B, T = (len(packed) - 1, lead[0]) if packed else lead
    n = lib.slstm_linear_attention_workspace_size(c, B, T, 1 if packed else 0, 1 if backward else 0)
    ws = torch.full((n // 4,), mark, device="cuda")

    def new(shape, dtype):
        return torch.full(shape, mark, dtype=dtype, device="cuda")

    if backward:
        out = {"dq": new(x["q"].shape, BF16), "dk": new(x["q"].shape, BF16), "dv": new(x["v"].shape, BF16),
               "dg": new(x["g"].shape, torch.float32), "ds0": new(x["s0"].shape, torch.float32)}
        fn = lib.slstm_linear_attention_backward_varlen if packed else lib.slstm_linear_attention_backward
        more = [x["dO"], x["dsT"]]
    else:
        out = {"o": new(x["v"].shape, BF16), "sT": new(x["s0"].shape, torch.float32)}
        fn = lib.slstm_linear_attention_forward_varlen if packed else lib.slstm_linear_attention_forward
        more = []
    p = [api._at(t) for t in [x[i] for i in ("q", "k", "v", "g", "s0")]]
    p += [api._at(cu), B] if packed else []
    p += [api._at(t) for t in more + list(out.values())] + [c] + ([T] if packed else [B, T])
    assert fn(*p, api._at(ws), ws.nbytes, api._stream()) == _lib.SLSTM_OK
    torch.cuda.synchronize()
    return out


CASES = [
    # B, T, Hqk, H, dk, dv, per_head, packed
    (2, 400, 2, 2, 64, 64, False, None),
    (2, 400, 1, 2, 128, 128, True, None),
    (1, 900, 1, 4, 128, 40, False, [0, 300, 300, 877]),
    (1, 3000, 1, 1, 64, 128, False, None),     # segments
    (40, 256, 2, 4, 64, 64, False, None),      # several chunks a block of the gradients
    (40, 256, 4, 4, 128, 64, True, None),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("fault", [1, 2, 3])
@pytest.mark.parametrize("B,T,Hqk,H,dk,dv,per_head,packed", CASES)
def test_expired_waits(B, T, Hqk, H, dk, dv, per_head, packed, fault, backward, cuda_device):
    x = _inputs((T,) if packed else (B, T), Hqk, H, dk, dv, BF16, 41, per_head=per_head,
                nseq=len(packed) - 1 if packed else B)
    want = _call(x, 0, backward, packed, 3.0)
    got = _call(x, fault, backward, packed, 7.0)
    lost = 0
    for n, y in got.items():
        z = want[n]
        bad = torch.isnan(y)
        outside = (z == 3.0) & (y == 7.0)     # packed: rows of no sequence
        assert (bad | (y == z) | outside).all(), n
        lost += int(bad.sum())
        if fault == 1 and n in ("o", "dq", "dk", "dv", "dg"):
            assert torch.isnan(y[packed[0]:packed[-1]] if packed else y).all(), n
    chunks = ((577 if packed else T) - 1) // 128 + 1
    if fault <= chunks or (backward and B == 40):   # 320 chunks and heads on 148 blocks, of two chunks a sequence
        assert lost > 0
    # and nothing is left behind
    again = _call(x, 0, backward, packed, 3.0)
    for n in want:
        assert torch.equal(again[n], want[n]), n
