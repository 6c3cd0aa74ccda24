"""CPU tests of the fp64 reference of the linear attention and the layer norm:
its gradients against central differences of its forward pass, and the invariants
of the recurrence (a cleared state forgets, a sequence in two halves is the
sequence)."""
import math

import pytest
import torch

import la_reference as ref


def _case(T, Hqk, H, dk, dv, seed, per_head=False):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    return {"q": r(T, Hqk, dk), "k": r(T, Hqk, dk), "v": r(T, H, dv),
            "g": -torch.rand(H, generator=g, dtype=torch.float64) if per_head
            else -torch.rand(T, H, generator=g, dtype=torch.float64),
            "s0": r(H, dk, dv), "dO": r(T, H, dv), "dsT": r(H, dk, dv)}


def _loss(case, scale):
    out, _ = ref.values({n: x for n, x in case.items() if n not in ("dO", "dsT")}, scale)
    return float((out["o"] * case["dO"]).sum() + (out["sT"] * case["dsT"]).sum())


@pytest.mark.parametrize("Hqk,H,per_head", [(2, 2, False), (1, 3, False), (2, 4, True)])
def test_gradients_against_differences(Hqk, H, per_head):
    case = _case(5, Hqk, H, 3, 2, 1, per_head)
    out, _ = ref.values(case, 0.7)
    h = 1e-5
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "ds0")):
        flat = case[name].view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = _loss(case, 0.7)
            flat[i] = keep - h
            down = _loss(case, 0.7)
            flat[i] = keep
            assert abs((up - down) / (2 * h) - out[grad].reshape(-1)[i].item()) < 1e-7, (name, i)


def test_halves_and_clears():
    case = _case(8, 2, 2, 3, 4, 2)
    out, _ = ref.values(case, 1.0)
    first, _ = ref.values({n: (x[:3] if n in "qkvg" else x) for n, x in case.items() if n != "dO"}, 1.0)
    second, _ = ref.values({**{n: case[n][3:] for n in "qkvg"}, "s0": first["sT"]}, 1.0)
    assert torch.allclose(torch.cat([first["o"], second["o"]]), out["o"], rtol=1e-13, atol=1e-13)
    assert torch.allclose(second["sT"], out["sT"], rtol=1e-13, atol=1e-13)
    case["g"][3] = -math.inf
    out, _ = ref.values(case, 1.0)
    alone, _ = ref.values({**{n: case[n][3:] for n in "qkvg"}, "s0": None}, 1.0)
    assert torch.allclose(out["o"][3:], alone["o"], rtol=1e-13, atol=1e-13)
    assert (out["ds0"] * 0 == 0).all() and (out["dg"][3] == 0).all()
