"""GPU tests of how many bits the linear attention keeps in bf16 on the tensor cores: fp32 outputs are those of fp32
arithmetic, bf16 outputs too, up to the numbers held as two bf16 terms, rounded once.

A number held as two bf16 terms loses at most 2^-17 of itself: the upper term is off by half a step, 2^-8 at most of
the power of two below the number, and the lower one by half a step of that.  bf16 outputs are rounded once, half a
step: 2^-8 of the value."""
import pytest
import torch

import la_reference as ref
from nonlinear_rnn_pararnn_b200 import api
from test_gpu_linear_attention import BF16, F32, _dense, _inputs, _row, _run

pytestmark = pytest.mark.gpu

# numbers of two terms in the products that an output is made of: a weight, a state in front of o, its gradient in
# front of dv.  (What a state sums, and the states in front of the other gradients, have three terms, which are all of
# an fp32 number.)
TERMS = {"o": 1, "sT": 0, "dq": 1, "dk": 1, "dv": 1, "dg": 0, "ds0": 0}


def _bound(name, size, exact, T, dk, dv, rep):
    tol = (ref.units(T, dk, dv) + rep) * 2.0 ** -24 * size + TERMS[name] * 2.0 ** -17 * size
    if name in ("o", "dq", "dk", "dv"):
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * exact.abs()
    return tol + 1e-30


CASES = [
    # B, T, Hqk, H, dk, dv, more: a token or two of shared heads, whose gradients of q and k nearly cancel
    (4, 1, 1, 8, 64, 64, {}),
    (4, 2, 1, 8, 64, 128, {"s0": False}),
    (2, 64, 2, 4, 128, 64, {}),
    (2, 129, 2, 2, 128, 128, {"resets": 40}),
    (1, 400, 1, 3, 64, 64, {"per_head": True}),
    (1, 260, 2, 2, 96, 40, {"fused": True}),
]


def _within(got, want, size, T, dk, dv, rep):
    for name, y in got.items():
        tol = _bound(name, size[name], want[name], T, dk, dv, rep)
        worst = float(((y.double() - want[name]).abs() / tol).max())
        assert worst <= 1.0, (name, worst)


@pytest.mark.parametrize("B,T,Hqk,H,dk,dv,more", CASES)
def test_outputs_and_states(B, T, Hqk, H, dk, dv, more, cuda_device):
    x = _inputs((B, T), Hqk, H, dk, dv, BF16, 101 + T, grads=False, **more)
    scale = dk ** -0.5
    want, size = _dense(x, scale)
    _within(_run(x, scale), want, size, T, dk, dv, H // Hqk)


@pytest.mark.parametrize("B,T,Hqk,H,dk,dv,more", CASES)
def test_gradients(B, T, Hqk, H, dk, dv, more, cuda_device):
    x = _inputs((B, T), Hqk, H, dk, dv, BF16, 201 + T, **more)
    scale = dk ** -0.5
    want, size = _dense(x, scale)
    got = _run(x, scale)
    _within({n: got[n] for n in ("dq", "dk", "dv", "ds0")}, want, size, T, dk, dv, H // Hqk)


@pytest.mark.parametrize("strong,times", [(-80.0, 20), (-40.0, 10), (-20.0, 16), (-87.0, 31)])
@pytest.mark.parametrize("block", [0, 1, 3])
def test_behind_strong_decays(strong, times, block, cuda_device):
    """Strong decays that clear nothing, in front of mild ones in the same 32 tokens: the sums of the log decays
    are large there, and the weights come from their differences."""
    T = 128
    x = _inputs((2, T), 1, 2, 64, 64, BF16, 300 + times)
    x["g"] = x["g"] * 0.25
    x["g"][:, 32 * block:32 * block + times] = strong
    want, size = _dense(x, 0.125)
    got = _run(x, 0.125)
    if block == 3:
        # the states are sums over the n tokens behind the strong ones: the roundings of the sum, the exponentials
        # of numbers below 16
        n = T - 96 - times
        off = float((got["sT"].double() - want["sT"]).norm() / want["sT"].norm())
        assert off <= (n + 16 + 8) * 2.0 ** -24, off
    _within(got, want, size, T, 64, 64, 2)


def _dg_sizes(case, scale):
    """For each token and head of one sequence, the root of the sum of the squares of the products that dg is made of:
    dg_t is a sum over the 128 tokens of t's chunk, of q_i S_i dO_i from t on and of k_j dS_j v_j before it, and of
    S dS where the chunk begins."""
    q, k, v, g, s = ref._double(case)
    dO, T, H = case["dO"].double(), q.shape[0], v.shape[1]
    a = torch.exp(g)[..., None, None]
    states = [s]
    for t in range(T):
        states.append(a[t] * states[-1] + k[t][:, :, None] * v[t][:, None, :])
    ds = case["dsT"].double()
    u, w, grads = torch.empty(T, H, dtype=torch.float64, device="cuda"), torch.empty_like(g.contiguous()), [None] * T
    for t in range(T - 1, -1, -1):
        ds = ds + scale * q[t][:, :, None] * dO[t][:, None, :]
        u[t] = ((scale * q[t][:, :, None] * states[t + 1] * dO[t][:, None, :]) ** 2).sum((1, 2))
        w[t] = ((k[t][:, :, None] * ds * v[t][:, None, :]) ** 2).sum((1, 2))
        ds = a[t] * ds
        grads[t] = ds
    out = torch.empty_like(u)
    for c in range(0, T, 128):
        e = min(T, c + 128)
        # the gradient of the state that leaves the chunk, times the chunk's decay: no more than at its first token
        edge = ((states[c] * grads[c]) ** 2).sum((1, 2))
        back = u[c:e].flip(0).cumsum(0).flip(0)
        front = w[c:e].cumsum(0) - w[c:e]
        out[c:e] = back + front + edge
    return out.sqrt()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hqk,H,dk,dv,more", CASES)
def test_gradient_of_the_decays(B, T, Hqk, H, dk, dv, more, dtype, cuda_device):
    """dg in the 2-norm, which a bound for each element on its own has to leave far too wide: its terms, of which some
    hundreds cancel, are off independently of one another."""
    x = _inputs((B, T), Hqk, H, dk, dv, dtype, 401 + T, **more)
    scale = dk ** -0.5
    want, _ = _dense(x, scale)
    got = api.linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["s0"],
                                        x["dO"], x["dsT"], scale=scale)["dg"].double()
    rows = [_row(x, b) for b in range(B)]
    for r in rows:
        if r["s0"] is None:
            r["s0"] = torch.zeros(H, dk, dv, device="cuda")
    size = torch.stack([_dg_sizes(r, scale) for r in rows])
    if x["g"].dim() == 1:
        size = (size ** 2).sum((0, 1)).sqrt() * 128 ** 0.5   # the tokens of a chunk share their errors
    # a term's error: the roundings of a sum of some 200 fp32 terms and of the states, which sum as many, the root of
    # 400 half units; four times that for the whole
    eps = 400 ** 0.5 * 2.0 ** -24
    off = float((got - want["dg"]).norm())
    assert off <= 4 * eps * float(size.norm()), (off / float(want["dg"].norm()), off / float(size.norm()) / eps)
    # which is far below dg itself
    assert 4 * eps * float(size.norm()) <= 0.02 * float(want["dg"].norm())


def test_one_rounding(cuda_device):
    """bf16 outputs of a longer sequence in the 2-norm: the rounding of each, of half a step at most and anywhere in it,
    and the numbers of two terms."""
    T, d = 1000, 128
    x = _inputs((1, T), 1, 2, d, d, BF16, 501)
    want, size = _dense(x, d ** -0.5)
    got = _run(x, d ** -0.5)
    for n in ("o", "dq", "dk", "dv"):
        off = float((got[n].double() - want[n]).norm())
        tol = 2.0 ** -8 * 3 ** -0.5 * float(want[n].norm())
        tol += (2.0 ** -17 + 200 ** 0.5 * 2.0 ** -24) * float(size[n].norm())
        assert off <= tol, (n, off / float(want[n].norm()))
