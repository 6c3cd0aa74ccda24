"""GPU tests of the guards that the bounds-checked build holds over the linear attention's and the layer norm's outputs:
with every extent taken one element short, the store to the last element of each output is skipped and reported; with
the extents as they are, nothing is."""
import ctypes

import pytest
import torch

from nonlinear_rnn_pararnn_b200 import _lib, api
from test_gpu_linear_attention import BF16, F32, _inputs

pytestmark = pytest.mark.gpu

MARK = 77.0


def _marked(shape, dtype):
    return torch.full(tuple(shape), MARK, dtype=dtype, device="cuda")


def _attention(x, cu):
    q, k, v, g, s0 = (x[n] for n in ("q", "k", "v", "g", "s0"))
    o, sT = _marked(v.shape, v.dtype), _marked(s0.shape, F32)
    out = {"dq": _marked(q.shape, q.dtype), "dk": _marked(q.shape, q.dtype), "dv": _marked(v.shape, v.dtype),
           "dg": _marked(g.shape, F32), "ds0": _marked(s0.shape, F32)}
    if cu is None:
        api.linear_attention_forward(q, k, v, g, s0, o=o, sT=sT)
        api.linear_attention_backward(q, k, v, g, s0, x["dO"], x["dsT"], out=out)
    else:
        api.linear_attention_forward_varlen(q, k, v, g, s0, cu, o=o, sT=sT)
        api.linear_attention_backward_varlen(q, k, v, g, s0, cu, x["dO"], x["dsT"], out=out)
    return {"o": o, "sT": sT, **out}


def _step(x):
    o, s = _marked(x["v"].shape, x["v"].dtype), _marked(x["s0"].shape, F32)
    api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], x["s0"], o=o, out=s)
    return {"o": o, "s": s}


def _forward_norm(z, w, groups):
    y = _marked(z.shape, z.dtype)
    _, m, r = api.layer_norm_forward(z, w, groups=groups, y=y)
    return y, m, r


def _backward_norm(z, w, dy, m, r, groups):
    out = {"dx": _marked(z.shape, z.dtype), "dw": _marked(w.shape, F32), "db": _marked(w.shape, F32)}
    return api.layer_norm_backward(z, w, dy, m, r, groups=groups, out=out)


class _short:
    """The checked library with its extents taken short; `seen` says what it has reported."""

    def __init__(self, elements):
        self.elements = elements

    def __enter__(self):
        self.ctx = _lib.checked_library()
        self.lib = self.ctx.__enter__()
        assert self.lib.slstm_check_clear() == _lib.SLSTM_OK
        assert self.lib.slstm_check_plant(self.elements) == _lib.SLSTM_OK
        return self

    def seen(self):
        out = (ctypes.c_longlong * 4)()
        assert self.lib.slstm_check_status(out) == _lib.SLSTM_OK
        assert self.lib.slstm_check_clear() == _lib.SLSTM_OK
        return out[0]

    def __exit__(self, *exc):
        assert self.lib.slstm_check_plant(0) == _lib.SLSTM_OK
        assert self.lib.slstm_check_clear() == _lib.SLSTM_OK
        return self.ctx.__exit__(*exc)


CASES = [
    # dtype, rows, Hqk, H, dk, dv, per_head, offsets
    (F32, (2, 70), 2, 2, 33, 40, False, None),
    (F32, (100,), 1, 3, 16, 20, True, [0, 30, 30, 100]),
    (BF16, (2, 150), 2, 2, 64, 40, False, None),
    (BF16, (1, 150), 1, 2, 128, 128, True, None),
    (BF16, (1, 3000), 1, 1, 64, 64, False, None),
    (BF16, (200,), 1, 2, 24, 128, False, [0, 10, 200]),
    (BF16, (200,), 1, 2, 64, 64, False, [0, 200, 200]),
]


@pytest.mark.parametrize("dtype,rows,Hqk,H,dk,dv,per_head,offsets", CASES)
def test_attention(dtype, rows, Hqk, H, dk, dv, per_head, offsets, cuda_device):
    x = _inputs(rows, Hqk, H, dk, dv, dtype, 61, per_head=per_head, nseq=len(offsets) - 1 if offsets else None)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda") if offsets else None
    with _short(1) as c:
        out = _attention(x, cu)
        assert c.seen() > 0
        for n, y in out.items():
            assert y.view(-1)[-1] == MARK and y.view(-1)[0] != MARK, n
    with _short(0) as c:
        want = _attention(x, cu)
        assert c.seen() == 0
    for n, y in _attention(x, cu).items():
        assert torch.equal(y, want[n]), n


@pytest.mark.parametrize("dtype,dv", [(F32, 32), (BF16, 33)])
def test_step(dtype, dv, cuda_device):
    x = _inputs((3,), 1, 2, 24, dv, dtype, 62, grads=False)
    with _short(1) as c:
        for n, y in _step(x).items():
            assert y.view(-1)[-1] == MARK and y.view(-1)[0] != MARK, n
        assert c.seen() >= 2
    with _short(0) as c:
        _step(x)
        assert c.seen() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("groups,d", [(1, 100), (2, 64), (1, 1030)])
def test_norm(groups, d, dtype, cuda_device):
    z = torch.randn(33, groups * d, device="cuda").to(dtype)
    w = torch.ones(groups * d, device="cuda")
    _, m, r = api.layer_norm_forward(z, w, groups=groups)
    with _short(1) as c:
        y, _, _ = _forward_norm(z, w, groups)
        assert c.seen() >= 2   # y, and mean and rstd together
        assert y.view(-1)[-1] == MARK and y.view(-1)[0] != MARK
        for n, t in _backward_norm(z, w, z, m, r, groups).items():
            assert t.view(-1)[-1] == MARK and t.view(-1)[0] != MARK, n
        assert c.seen() >= 4   # dx, the partial sums, dw and db
    with _short(0) as c:
        _backward_norm(z, w, z, *_forward_norm(z, w, groups)[1:], groups)
        assert c.seen() == 0


def test_nothing_to_plant_in_the_normal_build(cuda_device):
    lib = _lib.load()
    assert lib.slstm_check_plant(-1) == _lib.SLSTM_ERR_INVALID_ARG
    assert lib.slstm_check_plant(1) == _lib.SLSTM_OK
    x = _inputs((1, 30), 1, 1, 16, 16, F32, 63)
    for n, y in _attention(x, None).items():
        assert y.view(-1)[-1] != MARK, n
    assert lib.slstm_check_plant(0) == _lib.SLSTM_OK
