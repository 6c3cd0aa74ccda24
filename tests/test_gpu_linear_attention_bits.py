"""GPU tests of how many bits the linear attention keeps in bf16 on the tensor cores: every output is that of
fp32 arithmetic up to the numbers held as two bf16 terms, rounded once.

A number held as two bf16 terms loses at most 2^-17 of itself: the upper term is off by half a step, 2^-8 at most of
the power of two below the number, and the lower one by half a step of that.  bf16 outputs are rounded once, half a
step: 2^-8 of the value."""
import pytest
import torch

import la_reference as ref
from nonlinear_rnn_pararnn_b200 import api
from test_gpu_linear_attention import BF16, _dense, _inputs, _run

pytestmark = pytest.mark.gpu

# numbers of two terms on the way into an output: the weighted rows that a state sums and the state itself, of S and
# of its gradient; in o, dq, dk and dv also the weights, in place of the states
TERMS = {"o": 2, "sT": 1, "dq": 2, "dk": 2, "dv": 2, "dg": 4, "ds0": 1}


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
        # the states are sums over the n tokens behind the strong ones: a row of v in two terms, the roundings of
        # the sum, the exponentials of numbers below 16
        n = T - 96 - times
        off = float((got["sT"].double() - want["sT"]).norm() / want["sT"].norm())
        assert off <= 2.0 ** -17 + (n + 16 + 8) * 2.0 ** -24, off
    _within(got, want, size, T, 64, 64, 2)
