"""GPU tests of the layer norm, forward and backward, against fp64."""
import pytest
import torch

import la_reference as ref
from nonlinear_rnn_pararnn_b200 import api

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


CASES = [(1, 1, 1), (1, 1, 8), (5, 1, 7), (3, 4, 16), (700, 8, 64), (33, 3, 100), (1000, 2, 128), (9, 1, 250),
         (2500, 1, 256), (4, 1, 513), (17, 1, 1000), (600, 1, 1024), (3, 5, 1030), (5, 1, 2048), (7, 1, 4096),
         (3, 1, 5001), (2, 2, 8192), (2, 1, 16384), (3, 1, 16383)]


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,groups,d", CASES)
def test_layer_norm(rows, groups, d, xt, yt, cuda_device):
    gen = torch.Generator(device="cuda").manual_seed(rows + d)
    D, eps = groups * d, 1e-5
    # each slice with an offset of its own, some of them large beside their spread
    x = torch.randn(rows, D, generator=gen, device="cuda") + torch.randn(rows, 1, generator=gen, device="cuda") * 5
    x = x.to(xt)
    w = torch.randn(D, generator=gen, device="cuda")
    b = torch.randn(D, generator=gen, device="cuda") if rows % 2 else None
    dy = torch.randn(rows, D, generator=gen, device="cuda").to(yt)
    y, mean, rstd = api.layer_norm_forward(x, w, b, groups=groups, eps=eps, y_dtype=yt)
    Y, M, R = ref.layer_norm(x, w, b, groups, eps)
    xg = x.double().view(rows, groups, d)
    # a sum of d terms in the order of a tree over threads that each add up to 64: 64 + 16 roundings
    n = 80
    big = xg.abs().mean(-1)
    assert ((mean.double() - M).abs() <= n * U * big).all()
    # the variance: deviations off by the mean's error and one rounding, squares summed
    dev = n * U * big + U * xg.abs().amax(-1)
    var = ((xg - M[..., None]) ** 2).mean(-1)
    rel = (n * U * var + 2 * dev * var.sqrt() + dev ** 2) / (var + eps) + 4 * U
    assert ((rstd.double() - R).abs() <= rel * R).all()
    unit = ((xg - M[..., None]) * R[..., None]).abs()
    tol = (unit * (rel[..., None] + 4 * U) + (dev * R)[..., None]).flatten(1) * w.double().abs()
    tol = tol + 2 * U * Y.abs() + _half_step(yt) * Y.abs() + 1e-30
    if b is not None:
        tol = tol + U * b.double().abs()
    assert ((y.double() - Y).abs() <= tol * (1 + _half_step(yt)) + 1e-30).all()

    out = api.layer_norm_backward(x, w, dy, mean, rstd, groups=groups)
    # the formula at the given mean and rstd
    m, r = mean.double()[..., None], rstd.double()[..., None]
    xh = (xg - m) * r
    p = (dy.double() * w.double()).view(rows, groups, d)
    mp, mx = p.mean(-1, keepdim=True), (p * xh).mean(-1, keepdim=True)
    DX = r * (p - mp - xh * mx)
    size = r * (p.abs() + p.abs().mean(-1, keepdim=True) + xh.abs() * (p * xh).abs().mean(-1, keepdim=True))
    # xhat carries the cancellation of x - mean
    slip = 4 * U * (xg.abs() + m.abs()) * r
    size2 = r * (slip * mx.abs() + xh.abs() * (p.abs() * slip).mean(-1, keepdim=True))
    off = (out["dx"].double().view_as(DX) - DX).abs()
    assert (off <= (n + 8) * U * size + 2 * size2 + _half_step(xt) * DX.abs() * (1 + 1e-3) + 1e-30).all()
    dyd = dy.double().view(rows, groups, d)
    for name, terms, extra in (("dw", dyd * xh, dyd.abs() * slip), ("db", dyd, 0 * dyd)):
        # rows in turn within a block, the blocks within eight shares, eight shares
        total = terms.sum(0).flatten()
        chain = rows // 100 + 64 + 80 + 16
        tol = chain * U * terms.abs().sum(0).flatten() + extra.sum(0).flatten() + 1e-30
        assert ((out[name].double() - total).abs() <= tol).all(), name
    again = api.layer_norm_backward(x, w, dy, mean, rstd, groups=groups)
    assert all(torch.equal(out[i], again[i]) for i in out)


def test_gradient_against_differences(cuda_device):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w, dy = (torch.randn(s, generator=gen, device="cuda") for s in ((3, 24), (24,), (3, 24)))
    _, mean, rstd = api.layer_norm_forward(x, w, groups=2)
    out = api.layer_norm_backward(x, w, dy, mean, rstd, groups=2)

    def loss(x, w):
        return float((ref.layer_norm(x, w, None, 2, 1e-5)[0] * dy.double()).sum())

    h = 1e-5
    for name, t, i in [("dx", x, i) for i in range(0, 72, 5)] + [("dw", w, i) for i in range(24)]:
        up, down = t.double().clone(), t.double().clone()
        up.view(-1)[i] += h
        down.view(-1)[i] -= h
        d = (loss(up, w) - loss(down, w)) / (2 * h) if name == "dx" else (loss(x, up) - loss(x, down)) / (2 * h)
        # differences: h^2 of the third derivative; fp32: a few hundred roundings of terms of this size
        assert abs(d - float(out[name].view(-1)[i])) <= 1e-4, (name, i)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_misaligned_in_place_and_graph(dtype, cuda_device):
    gen = torch.Generator(device="cuda").manual_seed(2)
    flat = torch.randn(40 * 64 + 1, generator=gen, device="cuda").to(dtype)
    x = flat[1:].view(40, 64)     # aligned to its elements alone
    w, dy = torch.randn(64, generator=gen, device="cuda"), torch.randn(40, 64, generator=gen, device="cuda").to(dtype)
    y, m, r = api.layer_norm_forward(x, w)
    ya, ma, ra = api.layer_norm_forward(x.clone(), w)
    # the two column orders add in different orders: as many roundings as a slice has terms
    assert torch.allclose(m, ma, rtol=0, atol=64 * U * float(x.abs().max()))
    assert torch.allclose(y.float(), ya.float(), rtol=4 * _half_step(dtype), atol=1e-4)
    ref_out = api.layer_norm_backward(x, w, dy, m, r)
    z = x.clone()
    api.layer_norm_forward(z, w, y=z)
    assert torch.equal(z, ya)
    g = dy.clone()
    out = {"dx": g, "dw": torch.empty(64, device="cuda"), "db": torch.empty(64, device="cuda")}
    want = api.layer_norm_backward(x.clone(), w, dy, ma, ra)
    api.layer_norm_backward(x.clone(), w, g, ma, ra, out=out)
    assert all(torch.equal(out[i], want[i]) for i in out)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        c, cm, cr = api.layer_norm_forward(x, w)
        cb = api.layer_norm_backward(x, w, dy, cm, cr)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, y) and all(torch.equal(cb[i], ref_out[i]) for i in cb)


def test_constant_rows(cuda_device):
    """No spread at all: y is b, and the gradient stays finite."""
    x, w, b = torch.full((4, 32), 3.0, device="cuda"), torch.ones(32, device="cuda"), torch.arange(32.0, device="cuda")
    y, mean, rstd = api.layer_norm_forward(x, w, b)
    assert torch.equal(y, b.expand(4, 32)) and (mean == 3).all()
    out = api.layer_norm_backward(x, w, torch.ones(4, 32, device="cuda"), mean, rstd)
    assert all(torch.isfinite(v).all() for v in out.values())


def test_refusals(cuda_device):
    x, w = torch.zeros(4, 32, device="cuda"), torch.ones(32, device="cuda")
    y, m, r = api.layer_norm_forward(x, w)
    for call in (lambda: api.layer_norm_forward(x.half(), w), lambda: api.layer_norm_forward(x.cpu(), w),
                 lambda: api.layer_norm_forward(x.t(), w), lambda: api.layer_norm_forward(x, w[:31]),
                 lambda: api.layer_norm_forward(x, w, groups=5), lambda: api.layer_norm_forward(x, w, groups=0),
                 lambda: api.layer_norm_forward(x, w.double()), lambda: api.layer_norm_forward(x[:0], w),
                 lambda: api.layer_norm_forward(x, w, y_dtype=torch.float16),
                 lambda: api.layer_norm_forward(torch.zeros(1, 16385, device="cuda"),
                                                torch.zeros(16385, device="cuda")),
                 lambda: api.layer_norm_backward(x, w, y[:3], m, r), lambda: api.layer_norm_backward(x, w, y, m[:3], r),
                 lambda: api.layer_norm_backward(x, w, y, m, r, groups=2),
                 lambda: api.layer_norm_backward(x, w, y, m, r, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):
        api.layer_norm_forward(x, w, eps=-1.0)


def test_offsets_beyond_32_bits(cuda_device):
    """More than 2^31 elements: the last rows as they are alone."""
    D, rows = 1024, 2 ** 21 + 100
    x = torch.zeros(rows, D, dtype=BF16, device="cuda")
    tail = torch.randn(64, D, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(BF16)
    x[-64:] = tail
    w = torch.ones(D, device="cuda")
    y, m, r = api.layer_norm_forward(x, w)
    y1, m1, r1 = api.layer_norm_forward(tail, w)
    assert torch.equal(y[-64:], y1) and torch.equal(m[-64:], m1) and torch.equal(r[-64:], r1)
    out = api.layer_norm_backward(x, w, x, m, r)
    out1 = api.layer_norm_backward(tail, w, tail, m1, r1)
    assert torch.equal(out["dx"][-64:], out1["dx"]) and (out["dx"][:-64] == 0).all()
    # the other rows add nothing, the order of the others may change: 64 terms
    assert torch.allclose(out["db"], out1["db"], rtol=0, atol=64 * 64 * U * 6)
