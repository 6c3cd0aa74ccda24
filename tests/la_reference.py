"""The linear attention with a decay for each head and the layer norm in fp64,
token by token from their definitions, and bounds for the error that a
computation in chunks may make.

The gradients are the recurrences' own, not an automatic differentiation; the
CPU tests hold them against differences.
"""
import torch


def forward(q, k, v, g, s0, scale):
    """q, k (T, H, dk), v (T, H, dv), g (T, H), s0 (H, dk, dv), all fp64: o, sT."""
    s, o = s0, torch.empty_like(v)
    a = torch.exp(g)
    for t in range(q.shape[0]):
        s = a[t][:, None, None] * s + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * (s * q[t][:, :, None]).sum(1)
    return o, s


def backward(q, k, v, g, s0, dO, dsT, scale):
    """The gradients of sum dO o + sum dsT sT: dq, dk, dv, dg, ds0."""
    T = q.shape[0]
    a = torch.exp(g)
    states, s = [], s0
    for t in range(T):
        states.append(s)
        s = a[t][:, None, None] * s + k[t][:, :, None] * v[t][:, None, :]
    states.append(s)
    dq, dk, dv, dg = (torch.empty_like(x) for x in (q, k, v, g))
    ds = dsT
    for t in range(T - 1, -1, -1):
        ds = ds + scale * q[t][:, :, None] * dO[t][:, None, :]
        dq[t] = scale * (states[t + 1] * dO[t][:, None, :]).sum(2)
        dk[t] = (ds * v[t][:, None, :]).sum(2)
        dv[t] = (ds * k[t][:, :, None]).sum(1)
        dg[t] = a[t] * (ds * states[t]).sum((1, 2))
        ds = a[t][:, None, None] * ds
    return dq, dk, dv, dg, ds


def _double(case):
    """One sequence's tensors in fp64 with the heads repeated and g spread out."""
    q, k, v, g = (case[n].double() for n in ("q", "k", "v", "g"))
    rep = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    H, dk, dv = v.shape[1], q.shape[2], v.shape[2]
    s0 = case["s0"].double() if case.get("s0") is not None else torch.zeros(H, dk, dv, dtype=torch.float64,
                                                                            device=q.device)
    return q, k, v, g.expand(v.shape[:2]), s0


def values(case, scale):
    """The exact outputs of one sequence and, for each, the sum of the magnitudes
    of the products it is made of (the same recurrences on the absolute values).
    case: q, k, v, g, s0 and for the gradients dO, dsT."""
    q, k, v, g, s0 = _double(case)
    ab = [x.abs() for x in (q, k, v)]
    out, size = {}, {}
    out["o"], out["sT"] = forward(q, k, v, g, s0, scale)
    size["o"], size["sT"] = forward(*ab, g, s0.abs(), scale)
    if case.get("dO") is None:
        return out, size
    dO = case["dO"].double()
    dsT = case["dsT"].double() if case.get("dsT") is not None else torch.zeros_like(s0)
    names = ("dq", "dk", "dv", "dg", "ds0")
    out.update(zip(names, backward(q, k, v, g, s0, dO, dsT, scale)))
    size.update(zip(names, backward(*ab, g, s0.abs(), dO.abs(), dsT.abs(), scale)))
    # dg is the difference of sums over (at most) 128 rows of its chunk
    T, H = g.shape
    row = (ab[0] * size["dq"]).sum(-1) + (ab[1] * size["dk"]).sum(-1)
    n = (T + 127) // 128
    chunk = torch.nn.functional.pad(row, (0, 0, 0, n * 128 - T)).view(n, 128, H).sum(1)
    size["dg"] = size["dg"] + chunk.repeat_interleave(128, 0)[:T]
    # the heads that share a query and key head
    Hqk = case["q"].shape[1]
    for part in (out, size):
        for name in ("dq", "dk"):
            part[name] = part[name].unflatten(1, (Hqk, H // Hqk)).sum(2)
        if case["g"].dim() == 1:
            part["dg"] = part["dg"].sum(0)
    return out, size


def units(T, dk, dv):
    """Relative error, in units of 2^-24 of the sum of magnitudes, of one fp32
    evaluation: each rounding of a running sum is at most one unit (a half) of
    it, so as many units as terms are added one after another, in the longest
    chain: a product over d_k, one over d_v, one over the rows of a chunk (128),
    the states over the chunks (three roundings each), and 64 for the
    exponentials: 2 to the x has the relative error of x, |x| < 128 where the
    factor is not zero, in half units, at most twice along the way through a
    chunk.  Through a chain of chunks a factor counts each chunk's |x|, 256 in
    all where the product is not zero."""
    return dk + dv + 128 + 3 * ((T + 63) // 64) + 64 + 256


def tolerance(name, size, exact, dtype, T, dk, dv, rep):
    """The error an output may have."""
    tol = (units(T, dk, dv) + rep) * 2.0 ** -24 * size
    if dtype == torch.bfloat16:
        if name in ("o", "dq", "dk", "dv"):
            # the weights D (q k) and the states are rounded to bf16 on their way
            # into a product (half a step each), and the result is
            tol = tol + 2 * 2.0 ** -8 * size + 2.0 ** -8 * exact.abs()
        else:
            # two bf16 terms for a number: 2^-17 of it left; in S and in dS,
            # and in each weighted row that they sum
            tol = tol + 4 * 2.0 ** -17 * size
    return tol + 1e-30


def layer_norm(x, w, b, groups, eps):
    x = x.double().unflatten(-1, (groups, -1))
    mean = x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    rstd = 1.0 / torch.sqrt(var + eps)
    y = ((x - mean[..., None]) * rstd[..., None]).flatten(-2) * w.double()
    return y if b is None else y + b.double(), mean, rstd
