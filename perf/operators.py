"""The gated linear attention and the layer norm: cases, inputs, plain forms and exact values.

Linear attention with a decay for each head, per batch row (or packed sequence) and value head:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T        S: (d_k, d_v), fp32, S_{-1} = s0 or 0
    o_t = scale * S_t^T q_t

g is the log decay, one per token and head (B, T, H) or one per head (H,); -inf clears the state.
H value heads share H_qk query and key heads (H a multiple of H_qk).

Layer norm over each of `groups` equal slices of a row: y = (x - mean) * rstd * w + b.

With `own` false, run() computes in elementary torch operations in fp32, rounded once at the end; with
`own` true it calls the package.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}
EPS = 1e-5


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------
def listed():
    return [
        # the prompt or forward pass of a training step at the flagship shape (8 rows of 8192 steps, 1024
        # features as 8 heads of 128), q, k and v being slices of one fused projection
        {"name": "la_fwd_train", "op": "la_fwd", "dtype": BF16, "B": 8, "T": 8192, "H": 8, "Hqk": 8, "dk": 128,
         "dv": 128, "decay": "token", "fused": True, "resets": 0, "s0": False},
        # one long prompt of 65536 steps, documents packed into the row (the state is cleared between them)
        {"name": "la_fwd_long", "op": "la_fwd", "dtype": BF16, "B": 1, "T": 65536, "H": 16, "Hqk": 4, "dk": 64,
         "dv": 128, "decay": "token", "fused": False, "resets": 5000, "s0": True},
        # a short prompt in fp32 with one fixed decay for each head, odd length
        {"name": "la_fwd_short_f32", "op": "la_fwd", "dtype": F32, "B": 2, "T": 777, "H": 4, "Hqk": 4, "dk": 64,
         "dv": 64, "decay": "head", "fused": False, "resets": 0, "s0": True},
        # the backward pass of the training step
        {"name": "la_bwd_train", "op": "la_bwd", "dtype": BF16, "B": 8, "T": 8192, "H": 8, "Hqk": 8, "dk": 128,
         "dv": 128, "decay": "token", "fused": True, "resets": 0, "s0": False},
        # a backward pass in fp32 (8 rows of 1024 steps, 256 features as 4 heads of 64), a decay for each head
        {"name": "la_bwd_f32", "op": "la_bwd", "dtype": F32, "B": 8, "T": 1024, "H": 4, "Hqk": 4, "dk": 64, "dv": 64,
         "decay": "head", "fused": False, "resets": 0, "s0": True},
        # ragged prompts packed end to end, as a server prefills them
        {"name": "la_varlen_fwd", "op": "la_vfwd", "dtype": BF16, "n": 37, "total": 16384, "H": 8, "Hqk": 8, "dk": 128,
         "dv": 128, "decay": "token", "s0": True},
        # the same for a training step on packed ragged sequences, heads of 64 sharing two query and key heads
        {"name": "la_varlen_bwd", "op": "la_vbwd", "dtype": BF16, "n": 21, "total": 12345, "H": 8, "Hqk": 2, "dk": 64,
         "dv": 64, "decay": "token", "s0": True},
        # one token for each of 128 sequences being decoded
        {"name": "la_step_batch", "op": "la_step", "dtype": BF16, "B": 128, "H": 8, "Hqk": 8, "dk": 128, "dv": 128,
         "decay": "token"},
        # one token of a single sequence: latency
        {"name": "la_step_one", "op": "la_step", "dtype": BF16, "B": 1, "H": 8, "Hqk": 8, "dk": 64, "dv": 64,
         "decay": "token"},
        # the norm in front of a layer's projections, fp32 residual stream in, bf16 operand out
        {"name": "ln_fwd_train", "op": "ln_fwd", "dtype": F32, "ydtype": BF16, "rows": 65536, "groups": 1, "d": 1024,
         "bias": True},
        # the backward pass of the norm of each head behind the attention
        {"name": "ln_bwd_heads", "op": "ln_bwd", "dtype": BF16, "ydtype": BF16, "rows": 65536, "groups": 8, "d": 128,
         "bias": True},
        # a few rows of an odd width, both passes of which are latency
        {"name": "ln_bwd_few", "op": "ln_bwd", "dtype": F32, "ydtype": F32, "rows": 37, "groups": 1, "d": 1000,
         "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_bwd", "la_vfwd", "la_vbwd", "la_step", "ln_fwd", "ln_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    if op.startswith("ln"):
        groups = rng.choice([1, 1, 4, 8, 13])
        d = _log(rng, 16, 4096 if groups == 1 else 256)
        rows = min(_log(rng, 1, 65536), max(1, (1 << 26) // (groups * d)))
        return {"op": op, "dtype": dtype, "ydtype": rng.choice([dtype, BF16]), "rows": rows, "groups": groups, "d": d,
                "bias": rng.random() < 0.7}
    Hqk = rng.choice([1, 2, 3, 4, 8])
    H = Hqk * rng.choice([1, 1, 2, 4])
    sizes = [16, 24, 32, 40, 64, 64, 80, 96, 128, 128] + ([20, 33] if op in ("la_fwd", "la_step") else [])
    c = {"op": op, "dtype": dtype, "H": H, "Hqk": Hqk, "dk": rng.choice(sizes), "dv": rng.choice(sizes),
         "decay": rng.choice(["token", "token", "head"])}
    if op == "la_step":
        c["B"] = _log(rng, 1, 256)
        return c
    # at most the tokens * heads of half the training case, a quarter in fp32
    most = (131072 if dtype == F32 else 262144) // H
    c["s0"] = rng.random() < 0.5
    if op in ("la_vfwd", "la_vbwd"):
        c["total"] = min(_log(rng, 64, 16384), most)
        c["n"] = min(_log(rng, 1, 64), c["total"])
        return c
    c["B"] = rng.choice([1, 2, 3, 8])
    c["T"] = min(_log(rng, 1, 16384), max(1, most // c["B"]))
    c["fused"] = rng.random() < 0.5
    c["resets"] = rng.choice([0, 0, 300])
    return c


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _lengths(case, seed):
    """The lengths of the packed sequences: uneven, some of them a token or nothing."""
    g = torch.Generator().manual_seed(seed + 77)
    n, total = case["n"], case["total"]
    w = torch.rand(n, generator=g) ** 3
    cuts = torch.floor(torch.cumsum(w, 0) / w.sum() * total).to(torch.int64)
    cuts[-1] = total
    return torch.diff(cuts, prepend=torch.zeros(1, dtype=torch.int64)).tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"].startswith("ln"):
        rows, D = case["rows"], case["groups"] * case["d"]
        x = (randn(rows, D) * 1.5 + 0.3).to(dt)
        st = {"case": case, "x": x, "w": 1.0 + 0.2 * randn(D), "b": 0.2 * randn(D) if case["bias"] else None}
        if case["op"] == "ln_bwd":
            # what the forward pass has left behind
            xg = x.double().view(rows, case["groups"], case["d"])
            mean = xg.mean(-1)
            var = ((xg - mean[..., None]) ** 2).mean(-1)
            st["mean"], st["rstd"] = mean.float(), ((var + EPS) ** -0.5).float()
            st["dy"] = randn(rows, D).to(_DT[case["ydtype"]])
        return st

    H, Hqk, dk, dv = case["H"], case["Hqk"], case["dk"], case["dv"]
    packed = case["op"] in ("la_vfwd", "la_vbwd")
    if packed:
        lead, nseq = (case["total"],), case["n"]
    elif case["op"] == "la_step":
        lead, nseq = (case["B"],), case["B"]
    else:
        lead, nseq = (case["B"], case["T"]), case["B"]
    # queries and keys at the scale of a projection; keys of unit length on average
    wide = randn(*lead, 2 * Hqk * dk + H * dv)
    wide[..., Hqk * dk:2 * Hqk * dk] *= dk ** -0.5
    wide = wide.to(dt)
    q, k, v = wide.split([Hqk * dk, Hqk * dk, H * dv], dim=-1)
    if not case.get("fused"):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    st = {"case": case, "q": q.view(*lead, Hqk, dk), "k": k.view(*lead, Hqk, dk), "v": v.view(*lead, H, dv),
          "scale": dk ** -0.5}
    # forget gates with the biases 3 to 6 of the framework's workloads, or one decay for each head
    if case["decay"] == "head":
        st["g"] = torch.log1p(-torch.pow(2.0, -4.0 - 4.0 * torch.arange(H, device="cuda") / max(H, 1)))
    else:
        st["g"] = torch.nn.functional.logsigmoid(randn(*lead, H) + torch.linspace(3.0, 6.0, H, device="cuda"))
        if case.get("resets"):
            hit = torch.rand(*lead, 1, generator=gen, device="cuda") < 1.0 / case["resets"]
            st["g"] = st["g"].masked_fill(hit, -math.inf)
    st["s0"] = randn(nseq, H, dk, dv) if case.get("s0") or case["op"] == "la_step" else None
    if packed:
        lens = _lengths(case, seed)
        cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        st["cu"] = cu.to(torch.int32).cuda()
        st["longest"] = max(lens)
    if case["op"] in ("la_bwd", "la_vbwd"):
        st["dO"] = randn(*lead, H, dv).to(dt)
        st["dsT"] = 0.1 * randn(nseq, H, dk, dv)
    return st


# ---------------------------------------------------------------------------------------------------
# the plain forms: chunks of C tokens, all of them at once
# ---------------------------------------------------------------------------------------------------
def _sums(g):
    """L[..., i, j] = g[j+1] + ... + g[i] for i >= j, -inf for i < j (no differences: g may be -inf)."""
    n = g.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=g.device).tril(-1)
    L = torch.cumsum(torch.where(low, g[..., :, None], 0.0), dim=-2)
    return torch.where(low | torch.eye(n, dtype=torch.bool, device=g.device), L, -math.inf)


def _chunks(x, C, N):
    """(B, T, H, d) -> (B, H, N, C, d) in fp32, zeros behind the end."""
    B, T, H, d = x.shape
    x = torch.nn.functional.pad(x.float().transpose(1, 2), (0, 0, 0, N * C - T))
    return x.reshape(B, H, N, C, d)


def _lay(q, k, v, g, s0):
    B, T, Hqk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    C = 64 if T <= 8192 else 256
    N = (T + C - 1) // C
    q, k = [t.repeat_interleave(H // Hqk, dim=2) for t in (q, k)]
    q, k, v = [_chunks(t, C, N) for t in (q, k, v)]
    g = g.expand(B, T, H)
    g = torch.nn.functional.pad(g.transpose(1, 2), (0, N * C - T)).reshape(B, H, N, C)
    D = torch.exp(_sums(g))
    E = torch.exp(torch.cumsum(g, -1))[..., None]                                   # from the chunk's entry to i
    after = torch.nn.functional.pad(g[..., 1:], (0, 1))
    F = torch.exp(torch.flip(torch.cumsum(torch.flip(after, [-1]), -1), [-1]))[..., None]   # from j to its exit
    M = torch.exp(_sums(torch.nn.functional.pad(g.sum(-1), (1, 0))))                # between the chunks' entries
    first = torch.zeros(B, H, dk, dv, device=q.device) if s0 is None else s0
    X = torch.cat([first[:, :, None], (k * F).transpose(-1, -2) @ v], 2)
    S = (M @ X.flatten(-2)).view(X.shape)                                           # the state that enters each chunk
    return q, k, v, D, E, F, M, S


def _rows(x, T):
    """(B, H, N, C, d) -> (B, T, H, d)."""
    return x.flatten(2, 3)[:, :, :T].transpose(1, 2)


def _plain_forward(q, k, v, g, s0, scale):
    T, dt = q.shape[1], q.dtype
    q, k, v, D, E, F, M, S = _lay(q, k, v, g, s0)
    o = (D * (q @ k.transpose(-1, -2))) @ v + E * (q @ S[:, :, :-1])
    return _rows(o * scale, T).to(dt).contiguous(), S[:, :, -1].contiguous()


def _plain_backward(q, k, v, g, s0, scale, dO, dsT):
    (B, T, Hqk, dk), dt, H = q.shape, q.dtype, v.shape[2]
    gshape = g.shape
    q, k, v, D, E, F, M, S = _lay(q, k, v, g, s0)
    C, N = q.shape[3], q.shape[2]
    do = _chunks(dO, C, N) * scale
    Y = torch.cat([(q * E).transpose(-1, -2) @ do, dsT[:, :, None]], 2)
    dS = (M.transpose(-1, -2) @ Y.flatten(-2)).view(Y.shape)
    ds0, dS, S = dS[:, :, 0], dS[:, :, 1:], S[:, :, :-1]
    P, dP = D * (q @ k.transpose(-1, -2)), do @ v.transpose(-1, -2)
    dq_in = E * (do @ S.transpose(-1, -2))
    dk_in = F * (v @ dS.transpose(-1, -2))
    W = (P * dP).tril(-1)
    dP = D * dP
    dq, dk_ = dP @ k + dq_in, dP.transpose(-1, -2) @ q + dk_in
    dv_ = P.transpose(-1, -2) @ do + F * (k @ dS)
    u, w = (q * dq_in).sum(-1), (k * dk_in).sum(-1)
    back = torch.flip(torch.cumsum(torch.flip(W.sum(-1) - W.sum(-2) + u, [-1]), -1), [-1])
    tot = torch.diagonal(M, offset=-1, dim1=-2, dim2=-1)
    dg = back + torch.cumsum(w, -1) - w + (tot * (S * dS).sum((-1, -2)))[..., None]
    dg = dg.flatten(2)[:, :, :T].transpose(1, 2)
    dg = dg if len(gshape) == 3 else dg.sum((0, 1))
    share = [_rows(t, T).reshape(B, T, Hqk, H // Hqk, dk).sum(3).to(dt) for t in (dq, dk_)]
    return {"dq": share[0], "dk": share[1], "dv": _rows(dv_, T).to(dt).contiguous(), "dg": dg.contiguous(),
            "ds0": ds0.contiguous()}


def _dense(st):
    """Packed rows laid out as one row for each sequence: the index of each packed token, and a layout function."""
    cu, longest = st["cu"].long(), max(1, st["longest"])
    n, total = cu.numel() - 1, st["q"].shape[0]
    t = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = seq * longest + t - cu[seq]

    def lay(x):
        y = torch.zeros(n * longest, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[at] = x
        return y.view(n, longest, *x.shape[1:])

    return at, lay


def _ln_plain_forward(st):
    c = st["case"]
    x = st["x"].float().view(c["rows"], c["groups"], c["d"])
    mean = x.mean(-1)
    xc = x - mean[..., None]
    rstd = ((xc * xc).mean(-1) + EPS) ** -0.5
    y = (xc * rstd[..., None]).flatten(1) * st["w"]
    y = y if st["b"] is None else y + st["b"]
    return {"y": y.to(_DT[c["ydtype"]]), "mean": mean, "rstd": rstd}


def _ln_plain_backward(st):
    c = st["case"]
    shape = (c["rows"], c["groups"], c["d"])
    xhat = (st["x"].float().view(shape) - st["mean"][..., None]) * st["rstd"][..., None]
    dy = st["dy"].float()
    dxhat = (dy * st["w"]).view(shape)
    dx = (dxhat - dxhat.mean(-1, keepdim=True) - xhat * (dxhat * xhat).mean(-1, keepdim=True)) * st["rstd"][..., None]
    return {"dx": dx.flatten(1).to(st["x"].dtype), "dw": (dy * xhat.flatten(1)).sum(0), "db": dy.sum(0)}


def _plain(st):
    op = st["case"]["op"]
    if op == "ln_fwd":
        return _ln_plain_forward(st)
    if op == "ln_bwd":
        return _ln_plain_backward(st)
    q, k, v, g, s0, scale = (st[n] for n in ("q", "k", "v", "g", "s0", "scale"))
    if op == "la_step":
        H, Hqk = v.shape[1], q.shape[1]
        qf, kf = [t.float().repeat_interleave(H // Hqk, dim=1) for t in (q, k)]
        s = torch.exp(g.expand(v.shape[0], H))[..., None, None] * s0 + kf[..., :, None] * v.float()[..., None, :]
        return {"o": ((qf[..., None, :] @ s)[..., 0, :] * scale).to(v.dtype), "s": s}
    if op == "la_fwd":
        o, sT = _plain_forward(q, k, v, g, s0, scale)
        return {"o": o, "sT": sT}
    if op == "la_bwd":
        return _plain_backward(q, k, v, g, s0, scale, st["dO"], st["dsT"])
    at, lay = _dense(st)
    # a row's decay is 1 behind its last token: the state stands still there
    gd = g if g.dim() == 2 else g.expand(q.shape[0], g.numel())
    if op == "la_vfwd":
        o, sT = _plain_forward(lay(q), lay(k), lay(v), lay(gd), s0, scale)
        return {"o": o.flatten(0, 1)[at], "sT": sT}
    r = _plain_backward(lay(q), lay(k), lay(v), lay(gd), s0, scale, lay(st["dO"]), st["dsT"])
    out = {n: r[n].flatten(0, 1)[at] for n in ("dq", "dk", "dv", "dg")}
    out["dg"] = out["dg"] if g.dim() == 2 else out["dg"].sum(0)
    out["ds0"] = r["ds0"]
    return out


# ---------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------
def _own(st):
    from nonlinear_rnn_pararnn_b200 import api
    c = st["case"]
    op = c["op"]
    if op == "ln_fwd":
        y, mean, rstd = api.layer_norm_forward(st["x"], st["w"], st["b"], groups=c["groups"], eps=EPS,
                                               y_dtype=_DT[c["ydtype"]])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        return api.layer_norm_backward(st["x"], st["w"], st["dy"], st["mean"], st["rstd"], groups=c["groups"])
    q, k, v, g, s0, scale = (st[n] for n in ("q", "k", "v", "g", "s0", "scale"))
    if op == "la_step":
        o, s = api.linear_attention_step(q, k, v, g, s0, scale=scale)
        return {"o": o, "s": s}
    if op == "la_fwd":
        o, sT = api.linear_attention_forward(q, k, v, g, s0, scale=scale)
        return {"o": o, "sT": sT}
    if op == "la_bwd":
        return api.linear_attention_backward(q, k, v, g, s0, st["dO"], st["dsT"], scale=scale)
    if op == "la_vfwd":
        o, sT = api.linear_attention_forward_varlen(q, k, v, g, s0, st["cu"], scale=scale)
        return {"o": o, "sT": sT}
    return api.linear_attention_backward_varlen(q, k, v, g, s0, st["cu"], st["dO"], st["dsT"], scale=scale)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------
def work(case):
    size = {F32: 4, BF16: 2}
    e = size[case["dtype"]]
    if case["op"].startswith("ln"):
        n, D = case["rows"] * case["groups"], case["groups"] * case["d"]
        x, y = case["rows"] * D * e, case["rows"] * D * size[case["ydtype"]]
        if case["op"] == "ln_fwd":
            return {"bytes": x + y + 8 * n + 4 * D * (2 if case["bias"] else 1), "flops": 8 * case["rows"] * D}
        return {"bytes": 2 * x + y + 8 * n + 12 * D, "flops": 14 * case["rows"] * D}
    H, Hqk, dk, dv = case["H"], case["Hqk"], case["dk"], case["dv"]
    packed = case["op"] in ("la_vfwd", "la_vbwd")
    tokens = case["total"] if packed else case["B"] * case.get("T", 1)
    nseq = case["n"] if packed else case["B"]
    state = 4 * nseq * H * dk * dv
    g = 4 * (H if case["decay"] == "head" else tokens * H)
    qk, vo = tokens * Hqk * dk * e, tokens * H * dv * e
    if case["op"] == "la_step":
        return {"bytes": 2 * qk + 2 * vo + g + 2 * state, "flops": 5 * tokens * H * dk * dv}
    s0 = state if case["s0"] else 0
    if case["op"] in ("la_fwd", "la_vfwd"):
        return {"bytes": 2 * qk + 2 * vo + g + s0 + state, "flops": 4 * tokens * H * dk * dv}
    return {"bytes": 4 * qk + 3 * vo + 2 * g + s0 + 2 * state, "flops": 12 * tokens * H * dk * dv}


# ---------------------------------------------------------------------------------------------------
# exact values: the recurrences token by token in fp64
# ---------------------------------------------------------------------------------------------------
def _exact_ln(st):
    c = st["case"]
    shape = (c["rows"], c["groups"], c["d"])
    x, w = st["x"].double().view(shape), st["w"].double().view(shape[1:])
    if c["op"] == "ln_fwd":
        var, mean = torch.var_mean(x, dim=-1, correction=0)
        y = (x - mean[..., None]) / torch.sqrt(var + EPS)[..., None] * w
        y = y if st["b"] is None else y + st["b"].double().view(shape[1:])
        return {"y": y.flatten(1), "mean": mean, "rstd": 1.0 / torch.sqrt(var + EPS)}
    # y = xhat(x) w with the given mean and rstd as the row's own: the gradient through both
    r, dy = st["rstd"].double()[..., None], st["dy"].double().view(shape)
    n = (x - st["mean"].double()[..., None]) * r
    p = dy * w
    dx = r * p - r * p.sum(-1, keepdim=True) / c["d"] - r * n * (p * n).sum(-1, keepdim=True) / c["d"]
    return {"dx": dx.flatten(1), "dw": torch.einsum("rgd,rgd->gd", dy, n).flatten(), "db": dy.sum(0).flatten()}


def exact(case, seed):
    def _exact_row(q, k, v, g, s, scale, dO, dsT):
        """Rows of one length: q, k (B, T, H, dk) fp64, heads repeated; the values of both passes."""
        T = q.shape[1]
        a = torch.exp(g)[..., None, None]
        qc, kc = q[..., :, None], k[..., :, None]
        vr = v[..., None, :]
        if dO is None:
            o = torch.empty_like(v)
            for t in range(T):
                s = s * a[:, t] + kc[:, t] * vr[:, t]
                o[:, t] = (qc[:, t] * s).sum(-2)
            return o * scale, s
        # states kept at every `hold`-th token, rebuilt from there on the way back
        hold = max(1, int(math.sqrt(T)))
        kept = []
        for t in range(T):
            if t % hold == 0:
                kept.append(s)
            s = s * a[:, t] + kc[:, t] * vr[:, t]
        dr, ds = (dO * scale)[..., None, :], dsT
        dq, dk_, dv_, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g)
        for block in range(len(kept) - 1, -1, -1):
            lo, hi = block * hold, min(T, (block + 1) * hold)
            before = [kept[block]]
            for t in range(lo, hi):
                before.append(before[-1] * a[:, t] + kc[:, t] * vr[:, t])
            for t in range(hi - 1, lo - 1, -1):
                ds = ds + qc[:, t] * dr[:, t]
                dq[:, t] = (before[t - lo + 1] * dr[:, t]).sum(-1)
                dk_[:, t] = (ds * vr[:, t]).sum(-1)
                dv_[:, t] = (ds * kc[:, t]).sum(-2)
                ds = ds * a[:, t]
                dg[:, t] = (ds * before[t - lo]).sum((-1, -2))
        return dq, dk_, dv_, dg, ds

    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("ln"):
        return _exact_ln(st)
    H, Hqk = case["H"], case["Hqk"]
    rep = H // Hqk
    q, k, v, g = (st[n].double() for n in ("q", "k", "v", "g"))
    q, k = [torch.repeat_interleave(t, rep, dim=-2) for t in (q, k)]
    per_head = g.dim() == 1
    g = g.expand(*v.shape[:-1])
    scale = st["scale"]
    nseq = case["n"] if op in ("la_vfwd", "la_vbwd") else case["B"]
    s0 = torch.zeros(nseq, H, case["dk"], case["dv"], dtype=torch.float64, device="cuda")
    s0 = s0 if st["s0"] is None else st["s0"].double()
    if op == "la_step":
        o, s = _exact_row(q[:, None], k[:, None], v[:, None], g[:, None], s0, scale, None, None)
        return {"o": o[:, 0], "s": s}
    back = op in ("la_bwd", "la_vbwd")
    dO, dsT = (st["dO"].double(), st["dsT"].double()) if back else (None, None)
    if op in ("la_fwd", "la_bwd"):
        out = list(_exact_row(q, k, v, g, s0, scale, dO, dsT))
    else:
        parts = []
        cu = st["cu"].tolist()
        for i in range(nseq):
            at = slice(cu[i], cu[i + 1])
            parts.append(_exact_row(q[None, at], k[None, at], v[None, at], g[None, at], s0[i:i + 1], scale,
                                    dO[None, at] if back else None, dsT[i:i + 1] if back else None))
        cols = list(zip(*parts))
        out = [torch.cat([x[0] for x in col]) for col in cols[:-1]] + [torch.cat(cols[-1])]
    if not back:
        return {"o": out[0], "sT": out[1]}
    dq, dk_, dv_, dg, ds0 = out
    dq, dk_ = [t.unflatten(-2, (Hqk, rep)).sum(-2) for t in (dq, dk_)]
    if per_head:
        dg = dg.flatten(0, -2).sum(0)
    return {"dq": dq, "dk": dk_, "dv": dv_, "dg": dg, "ds0": ds0}
