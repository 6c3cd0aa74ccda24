"""GPU tests of the linear attention with a decay for each head: every form
against the fp64 recurrence, with bounds from the roundings made."""
import math

import pytest
import torch

import la_reference as ref
from nonlinear_rnn_pararnn_b200 import api

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _inputs(lead, Hqk, H, dk, dv, dtype, seed, *, per_head=False, nseq=None, s0=True, resets=0, fused=False,
            grads=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    wide = r(*lead, 2 * Hqk * dk + H * dv).to(dtype)
    q, k, v = wide.split([Hqk * dk, Hqk * dk, H * dv], dim=-1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nseq = lead[0] if nseq is None else nseq
    if per_head:
        g = -torch.rand(H, generator=gen, device="cuda") * 0.2
    else:
        g = torch.nn.functional.logsigmoid(r(*lead, H) * 1.5 + 3.0)
        if resets:
            g = g.masked_fill(torch.rand(*lead, H, generator=gen, device="cuda") < 1.0 / resets, -math.inf)
    x = {"q": q.view(*lead, Hqk, dk), "k": k.view(*lead, Hqk, dk), "v": v.view(*lead, H, dv), "g": g,
         "s0": r(nseq, H, dk, dv) if s0 else None}
    if grads:
        x["dO"] = r(*lead, H, dv).to(dtype)
        x["dsT"] = r(nseq, H, dk, dv)
    return x


def _check(got, want, size, dtype, T, dk, dv, rep, what=""):
    for name, y in got.items():
        assert torch.isfinite(y).all(), (what, name)
        off = (y.double() - want[name]).abs()
        tol = ref.tolerance(name, size[name], want[name], dtype, T, dk, dv, rep)
        worst = float((off / tol).max()) if y.numel() else 0.0
        assert worst <= 1.0, (what, name, worst, float(off.max()))


def _row(x, b):
    """Sequence b of a dense case."""
    return {n: (y if y is None or (n == "g" and y.dim() == 1) else y[b]) for n, y in x.items()}


def _dense(x, scale):
    """The exact values and sizes of a dense case, stacked."""
    parts = [ref.values(_row(x, b), scale) for b in range(x["q"].shape[0])]
    out, size = ({n: torch.stack([p[i][n] for p in parts]) for n in parts[0][i]} for i in (0, 1))
    if x["g"].dim() == 1 and "dg" in out:
        out["dg"], size["dg"] = out["dg"].sum(0), size["dg"].sum(0)
    return out, size


def _run(x, scale, **kw):
    o, sT = api.linear_attention_forward(x["q"], x["k"], x["v"], x["g"], x["s0"], scale=scale)
    got = {"o": o, "sT": sT}
    if x.get("dO") is not None:
        got.update(api.linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["s0"], x["dO"], x["dsT"],
                                                 scale=scale, **kw))
    return got


CASES = [
    # B, T, Hqk, H, dk, dv, more
    (1, 1, 1, 1, 1, 1, {}),
    (2, 1, 2, 4, 64, 64, {}),
    (1, 2, 1, 2, 128, 128, {"s0": False}),
    (2, 63, 1, 1, 16, 32, {"resets": 5}),
    (1, 64, 2, 2, 64, 128, {}),
    (1, 65, 2, 2, 128, 64, {"per_head": True}),
    (2, 127, 1, 3, 24, 40, {"fused": True}),
    (1, 128, 2, 2, 128, 128, {"fused": True, "s0": False}),
    (2, 129, 2, 2, 128, 128, {"resets": 3}),
    (1, 300, 2, 6, 96, 80, {"per_head": True, "fused": True}),
    (3, 257, 1, 2, 33, 20, {"fused": True}),
    (1, 700, 1, 1, 64, 64, {"resets": 100}),
    (1, 130, 1, 2, 256, 136, {}),
    (1, 70, 1, 1, 8, 256, {"s0": False}),
    (1, 1025, 1, 1, 32, 16, {}),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hqk,H,dk,dv,more", CASES)
def test_dense(B, T, Hqk, H, dk, dv, more, dtype, cuda_device):
    x = _inputs((B, T), Hqk, H, dk, dv, dtype, 3 * T + dk, **more)
    scale = dk ** -0.5
    want, size = _dense(x, scale)
    got = _run(x, scale)
    _check(got, want, size, dtype, T, dk, dv, H // Hqk)
    # again: the same bits
    for n, y in _run(x, scale).items():
        assert torch.equal(y, got[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fill", [-math.inf, -100.0, -60.0, 0.0, 0.05])
def test_extreme_decays(fill, dtype, cuda_device):
    """Every token cleared, factors no normal number or nearly none, none, growth."""
    x = _inputs((1, 200), 1, 2, 64, 64, dtype, 5)
    x["g"] = torch.full_like(x["g"], fill)
    want, size = _dense(x, 0.3)
    got = _run(x, 0.3)
    if fill == -100.0:
        # the factors are below the normal numbers and count as zero: what they carry is less than this
        for n in size:
            size[n] = size[n] + 1e-25
    _check(got, want, size, dtype, 200, 64, 64, 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_mixed_decays(dtype, cuda_device):
    """Cleared and nearly cleared tokens among ordinary ones, the first and last among them."""
    x = _inputs((2, 333), 2, 2, 64, 64, dtype, 6)
    for i, val in enumerate((-math.inf, -50.0, -87.0, -math.inf)):
        x["g"][:, i::11, i % 2] = val
    x["g"][0, 0] = -math.inf
    x["g"][1, -1] = -math.inf
    x["g"][0, 120:140] = -math.inf
    want, size = _dense(x, 0.3)
    got = _run(x, 0.3)
    _check(got, want, size, dtype, 333, 64, 64, 1)
    cleared = x["g"] == -math.inf
    assert (got["dg"][cleared] == 0).all()
    assert (got["ds0"][0] == 0).all()   # nothing passes a cleared first token


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_optional_arguments(dtype, cuda_device):
    """No dsT, no dg, the final state over the first, given outputs and workspaces."""
    x = _inputs((2, 150), 1, 2, 64, 64, dtype, 7)
    full = _run(x, 0.2)
    s = x["s0"].clone()
    o, sT = api.linear_attention_forward(x["q"], x["k"], x["v"], x["g"], s, scale=0.2, sT=s,
                                         ws=api.linear_attention_workspace(x["q"], x["v"], x["g"]))
    assert sT is s and torch.equal(s, full["sT"]) and torch.equal(o, full["o"])
    args = (x["q"], x["k"], x["v"], x["g"], x["s0"], x["dO"])
    z = api.linear_attention_backward(*args, torch.zeros_like(x["dsT"]), scale=0.2)
    n = api.linear_attention_backward(*args, scale=0.2, with_dg=False,
                                      ws=api.linear_attention_workspace(x["q"], x["v"], x["g"], backward=True))
    assert "dg" not in n
    for name in ("dq", "dk", "dv", "ds0"):
        assert torch.equal(z[name], n[name]), name


PACKED = [
    # lengths, Hqk, H, dk, dv, per_head
    ([1], 1, 1, 64, 64, False),
    ([128, 0, 1, 129, 0, 300, 64], 2, 4, 64, 64, False),
    ([0, 0, 257, 3, 0], 1, 2, 128, 128, True),
    ([5] * 40, 2, 2, 32, 128, False),
    ([700, 31], 1, 3, 33, 24, False),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,Hqk,H,dk,dv,per_head", PACKED)
def test_packed(lens, Hqk, H, dk, dv, per_head, dtype, cuda_device):
    """Packed sequences, with rows in front of the first and behind the last left as they were and
    values there that are not finite."""
    front, behind = 3, 70
    total = front + sum(lens) + behind
    x = _inputs((total,), Hqk, H, dk, dv, dtype, sum(lens), per_head=per_head, nseq=len(lens))
    cu = [front]
    for n in lens:
        cu.append(cu[-1] + n)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    outside = torch.ones(total, dtype=torch.bool, device="cuda")
    outside[cu[0]:cu[-1]] = False
    for n in ("q", "k", "v", "dO"):
        x[n][outside] = float("nan")
    if not per_head:
        x["g"][outside] = float("nan")
    scale = dk ** -0.5
    mark = 7.0
    o = torch.full((total, H, dv), mark, dtype=dtype, device="cuda")
    got = {"o": o}
    _, got["sT"] = api.linear_attention_forward_varlen(x["q"], x["k"], x["v"], x["g"], x["s0"], cut, scale=scale, o=o)
    out = {"dq": torch.full((total, Hqk, dk), mark, dtype=dtype, device="cuda"),
           "dk": torch.full((total, Hqk, dk), mark, dtype=dtype, device="cuda"),
           "dv": torch.full((total, H, dv), mark, dtype=dtype, device="cuda"),
           "dg": torch.full(x["g"].shape, mark, device="cuda"), "ds0": torch.empty_like(x["s0"])}
    got.update(api.linear_attention_backward_varlen(x["q"], x["k"], x["v"], x["g"], x["s0"], cut, x["dO"], x["dsT"],
                                                    scale=scale, out=out))
    for n in ("o", "dq", "dk", "dv") + (() if per_head else ("dg",)):
        assert (got[n][outside] == mark).all(), n
    dg, dgs = 0.0, 0.0
    for i, n in enumerate(lens):
        at = slice(cu[i], cu[i + 1])
        one = {m: (y if m == "g" and per_head else y[at]) for m, y in x.items() if m in ("q", "k", "v", "g", "dO")}
        want, size = ref.values({**one, "s0": x["s0"][i], "dsT": x["dsT"][i]}, scale)
        part = {m: got[m][at] for m in ("o", "dq", "dk", "dv")}
        part.update({m: got[m][i] for m in ("sT", "ds0")})
        if per_head:
            dg, dgs = dg + want["dg"], dgs + size["dg"]
        else:
            part["dg"] = got["dg"][at]
        _check(part, want, size, dtype, max(n, 1), dk, dv, H // Hqk, i)
    if per_head:
        _check({"dg": got["dg"]}, {"dg": dg}, {"dg": dgs}, dtype, total, dk, dv, 1)


def test_malformed_offsets_stay_in_range(cuda_device):
    """Offsets out of range or falling are clamped: the calls return, rows they do not reach stay."""
    x = _inputs((200,), 1, 2, 64, 64, BF16, 9, nseq=4)
    for cu in ([0, 500, -3, 100, 200], [-7, 50, 20, 80, 190], [200, 100, 0, 0, 0]):
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, sT = api.linear_attention_forward_varlen(x["q"], x["k"], x["v"], x["g"], x["s0"], cut)
        api.linear_attention_backward_varlen(x["q"], x["k"], x["v"], x["g"], x["s0"], cut, x["dO"], x["dsT"])
        torch.cuda.synchronize()
        if cu[0] == 200:
            assert torch.equal(sT, x["s0"])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_other_sequences_stay_clean(dtype, cuda_device):
    """A row of the batch that is not finite spoils itself alone."""
    x = _inputs((3, 90), 1, 1, 64, 64, dtype, 10)
    want = _run(x, 1.0)
    for n in ("q", "k", "v", "dO"):
        x[n][1] = float("nan")
    got = _run(x, 1.0)
    for n, y in got.items():
        assert torch.equal(y[0], want[n][0]) and torch.equal(y[2], want[n][2]), n
        assert torch.isnan(y[1]).any(), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Hqk,H,dk,dv,per_head", [(1, 1, 1, 1, 1, False), (3, 2, 4, 64, 64, False),
                                                    (40, 8, 8, 128, 128, True), (2, 1, 3, 33, 20, False),
                                                    (5, 1, 2, 256, 136, False), (200, 1, 1, 16, 250, False)])
def test_step(B, Hqk, H, dk, dv, per_head, dtype, cuda_device):
    x = _inputs((B,), Hqk, H, dk, dv, dtype, B + dk, per_head=per_head, grads=False, fused=True)
    if not per_head:
        x["g"][0, 0] = -math.inf
    scale = dk ** -0.5
    o, s = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], x["s0"], scale=scale)
    parts = [ref.values({n: (y if n == "g" and per_head else y[b:b + 1]) if n != "s0" else y[b]
                         for n, y in x.items()}, scale) for b in range(B)]
    for b, (want, size) in enumerate(parts):
        # fp32 throughout: the sums over d_k and the exponential; the result rounded once
        for name, y in (("o", o[b:b + 1]), ("sT", s[b])):
            tol = (dk + 8) * 2.0 ** -24 * size[name] + 1e-30
            if name == "o" and dtype == BF16:
                tol = tol + 2.0 ** -8 * want["o"].abs()
            assert float(((y.double() - want[name]).abs() / tol).max()) <= 1.0, (b, name)
    # in place, and from nothing
    t = x["s0"].clone()
    o2, t2 = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], t, scale=scale, out=t)
    assert t2 is t and torch.equal(t, s) and torch.equal(o, o2)
    o3, s3 = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], scale=scale)
    o4, s4 = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], torch.zeros_like(x["s0"]), scale=scale)
    assert torch.equal(s3, s4) and torch.equal(o3, o4)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_then_tokens(dtype, cuda_device):
    """A prompt and then single tokens, as a server runs them, is the whole sequence."""
    T, cut = 140, 131
    x = _inputs((2, T), 1, 2, 64, 64, dtype, 11, grads=False)
    want, size = _dense(x, 0.125)
    o, s = api.linear_attention_forward(*(x[n][:, :cut].contiguous() for n in ("q", "k", "v", "g")), x["s0"])
    outs = [o]
    for t in range(cut, T):
        o, s = api.linear_attention_step(*(x[n][:, t].contiguous() for n in ("q", "k", "v", "g")), s, out=s)
        outs.append(o[:, None])
    # the steps' roundings come on top: three a token
    _check({"o": torch.cat(outs, 1), "sT": s}, want, size, dtype, T + 64 * (T - cut), 64, 64, 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graphs_and_streams(dtype, cuda_device):
    """Both passes and the step captured and replayed on new inputs, two graphs at once on streams of
    their own, each with its own workspace."""
    a, b = (_inputs((2, 200), 1, 2, 64, 64, dtype, s) for s in (12, 13))
    want = [_run(x, 0.125) for x in (a, b)]
    buf = [{n: y.clone() for n, y in a.items()} for _ in range(2)]
    outs, graphs = [], []
    for x in buf:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            _run(x, 0.125)
        torch.cuda.current_stream().wait_stream(st)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_run(x, 0.125))
        graphs.append(gr)
    for order in ((a, b), (b, a)):
        for x, src in zip(buf, order):
            for n in x:
                x[n].copy_(src[n])
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        for got, src in zip(outs, order):
            for n, y in got.items():
                assert torch.equal(y, want[0 if src is a else 1][n]), n


def test_offsets_beyond_32_bits(cuda_device):
    """More than 2^31 elements in q, k, v and o: the last sequence against itself alone."""
    H, d, last = 16, 128, 500
    total = 2 ** 31 // (H * d) + 1000
    x = {n: torch.zeros(total, H, d, dtype=BF16, device="cuda") for n in ("q", "k", "v")}
    tail = _inputs((last,), H, H, d, d, BF16, 14, nseq=1, grads=False)
    for n in ("q", "k", "v"):
        x[n][-last:] = tail[n]
    g = torch.zeros(total, H, device="cuda")
    g[-last:] = tail["g"]
    cu = torch.tensor([0, total - last, total], dtype=torch.int32, device="cuda")
    s0 = torch.cat([torch.zeros_like(tail["s0"]), tail["s0"]])
    o, sT = api.linear_attention_forward_varlen(x["q"], x["k"], x["v"], g, s0, cu)
    o1, s1 = api.linear_attention_forward_varlen(tail["q"], tail["k"], tail["v"], tail["g"], tail["s0"],
                                                 torch.tensor([0, last], dtype=torch.int32, device="cuda"))
    want, size = ref.values({n: (y[0] if n == "s0" else y) for n, y in tail.items()}, d ** -0.5)
    _check({"o": o[-last:], "sT": sT[1]}, want, size, BF16, last, d, d, 1)
    _check({"o": o1, "sT": s1[0]}, want, size, BF16, last, d, d, 1)
    assert (o[:-last] == 0).all() and (sT[0] == 0).all()


def test_refusals(cuda_device):
    x = _inputs((2, 10), 2, 4, 16, 16, F32, 15)
    a = [x[n] for n in ("q", "k", "v", "g", "s0")]

    def bad(i, y, *more):
        b = list(a)
        b[i] = y
        with pytest.raises(ValueError):
            api.linear_attention_forward(*b)

    bad(0, x["q"].half())
    bad(0, x["q"].cpu())
    bad(0, x["q"][0])
    bad(1, x["k"][:, :9])
    bad(1, x["k"].to(BF16))
    bad(1, x["k"].transpose(2, 3))
    bad(2, x["v"][:, :, :3])                      # 3 value heads of 2 query heads
    bad(2, x["v"].transpose(0, 1).contiguous().transpose(0, 1))   # sequences inside tokens
    bad(2, x["v"][:, :1].expand(2, 10, 4, 16))    # tokens on top of one another
    bad(3, x["g"].double())
    bad(3, x["g"][..., :3])
    bad(4, x["s0"][:1])
    bad(0, torch.zeros(2, 10, 2, 300, device="cuda"))
    with pytest.raises(ValueError):
        api.linear_attention_forward(*a, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        api.linear_attention_backward(*a, x["dO"][:, :5], x["dsT"])
    with pytest.raises(ValueError):
        api.linear_attention_backward(*a, x["dO"].transpose(1, 2).contiguous().transpose(1, 2), x["dsT"])
    with pytest.raises(ValueError):
        api.linear_attention_forward_varlen(*(y[0] for y in a[:4]), a[4], torch.tensor([0, 5, 10], device="cuda"))
    with pytest.raises(ValueError):
        api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], x["s0"])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_with_the_norms(dtype, cuda_device):
    """As a layer runs them: norm, q, k and v as slices of one projection, attention, the norm of each
    head, and back, against fp64 autograd of the same formulas."""
    B, T, H, dk, dv, D = 2, 150, 2, 32, 64, 96
    gen = torch.Generator(device="cuda").manual_seed(16)

    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    x, w1, b1 = r(B, T, D), 1 + 0.1 * r(D), 0.1 * r(D)
    W = (r(D, 2 * H * dk + H * dv) * D ** -0.5).to(dtype)
    w2, b2, dy = 1 + 0.1 * r(H * dv), 0.1 * r(H * dv), r(B, T, H * dv).to(dtype)
    g = torch.nn.functional.logsigmoid(r(B, T, H) + 3)
    n, m1, r1 = api.layer_norm_forward(x, w1, b1, y_dtype=dtype)
    wide = n @ W
    q, k, v = wide.split([H * dk, H * dk, H * dv], dim=-1)
    q, k, v = q.view(B, T, H, dk), k.view(B, T, H, dk), v.view(B, T, H, dv)
    o, _ = api.linear_attention_forward(q, k, v, g)
    y, m2, r2 = api.layer_norm_forward(o.view(B, T, -1), w2, b2, groups=H)
    back = api.layer_norm_backward(o.view(B, T, -1), w2, dy, m2, r2, groups=H)
    la = api.linear_attention_backward(q, k, v, g, None, back["dx"].view_as(o))
    dn = torch.cat([la[i].flatten(2) for i in ("dq", "dk", "dv")], -1) @ W.t()
    first = api.layer_norm_backward(x, w1, dn, m1, r1)

    X, W1, B1, G, W2, B2 = (t.double().cpu().requires_grad_() for t in (x, w1, b1, g, w2, b2))
    N = torch.nn.functional.layer_norm(X, (D,), W1, B1, 1e-5)
    Q, K, V = (N @ W.double().cpu()).split([H * dk, H * dk, H * dv], dim=-1)
    s, outs = torch.zeros(B, H, dk, dv, dtype=torch.float64), []
    for t in range(T):
        s = torch.exp(G[:, t])[..., None, None] * s + K[:, t].view(B, H, dk, 1) * V[:, t].view(B, H, 1, dv)
        outs.append((s * Q[:, t].view(B, H, dk, 1)).sum(2) * dk ** -0.5)
    O = torch.stack(outs, 1)
    Y = torch.nn.functional.layer_norm(O, (dv,), None, None, 1e-5).flatten(2) * W2 + B2
    (Y * dy.double().cpu()).sum().backward()
    # a dozen stages, whose roundings in the 2-norm add up at most: half a step of bf16 each, or the
    # 300 terms of a sum in fp32
    bound = 12 * 2.0 ** -8 if dtype == BF16 else 12 * 300 * 2.0 ** -24
    pairs = {"y": (y, Y), "dx": (first["dx"], X.grad), "dw1": (first["dw"], W1.grad), "db1": (first["db"], B1.grad),
             "dg": (la["dg"], G.grad), "dw2": (back["dw"], W2.grad), "db2": (back["db"], B2.grad)}
    for name, (a, b) in pairs.items():
        b = b.detach()
        err = float((a.double().cpu() - b).norm() / b.norm())
        assert err <= bound, (name, err)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [-0.7, 0.0])
def test_scales(scale, dtype, cuda_device):
    x = _inputs((1, 200), 1, 2, 64, 64, dtype, 17)
    want, _ = _dense(x, scale)
    _, size = _dense(x, abs(scale))
    got = _run(x, scale)
    _check(got, want, size, dtype, 200, 64, 64, 1)
    if scale == 0.0:
        assert (got["o"] == 0).all() and (got["dq"] == 0).all()


@pytest.mark.parametrize("dk,dv,per_head", [(64, 128, False), (128, 64, True)])
def test_long_rows_in_segments(dk, dv, per_head, cuda_device):
    """One long row of few heads, dense and packed: its chunks are shared out in segments, whose first
    states come from a pass of their own."""
    T = 3000
    x = _inputs((1, T), 1, 2, dk, dv, BF16, 18, per_head=per_head, resets=0 if per_head else 900)
    scale = dk ** -0.5
    want, size = _dense(x, scale)
    got = _run(x, scale)
    _check(got, want, size, BF16, T, dk, dv, 2)
    p = {n: (y if n in ("s0", "dsT") or (n == "g" and per_head) else y[0]) for n, y in x.items()}
    # packed behind a short sequence and an empty one, which are one segment and none
    cut = 40
    cu = torch.tensor([0, cut, cut, T], dtype=torch.int32, device="cuda")
    s0 = torch.cat([x["s0"]] * 3)
    dsT = torch.cat([x["dsT"]] * 3)
    got = {}
    got["o"], got["sT"] = api.linear_attention_forward_varlen(p["q"], p["k"], p["v"], p["g"], s0, cu, scale=scale)
    got.update(api.linear_attention_backward_varlen(p["q"], p["k"], p["v"], p["g"], s0, cu, p["dO"], dsT, scale=scale))
    assert torch.equal(got["sT"][1], s0[1]) and torch.equal(got["ds0"][1], dsT[1])
    total = [0.0, 0.0]
    for i, at in ((0, slice(0, cut)), (2, slice(cut, T))):
        one = {n: (y if n == "g" and per_head else y[at]) for n, y in p.items() if n in ("q", "k", "v", "g", "dO")}
        want, size = ref.values({**one, "s0": s0[i], "dsT": dsT[i]}, scale)
        part = {m: got[m][at] for m in ("o", "dq", "dk", "dv")}
        part.update({m: got[m][i] for m in ("sT", "ds0")})
        if per_head:
            total = [total[0] + want["dg"], total[1] + size["dg"]]
        else:
            part["dg"] = got["dg"][at]
        _check(part, want, size, BF16, T, dk, dv, 2, i)
    if per_head:
        _check({"dg": got["dg"]}, {"dg": total[0]}, {"dg": total[1]}, BF16, T, dk, dv, 2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_short_sequences(dtype, cuda_device):
    """Thousands of sequences of no or a few tokens, as many offsets as several rounds of the table."""
    gen = torch.Generator().manual_seed(19)
    lens = torch.randint(0, 4, (3001,), generator=gen)
    cu = torch.zeros(3002, dtype=torch.int64)
    cu[1:] = torch.cumsum(lens, 0)
    total = int(cu[-1])
    x = _inputs((total,), 1, 1, 16, 16, dtype, 20, nseq=3001, grads=False)
    cut = cu.to(torch.int32).cuda()
    o, sT = api.linear_attention_forward_varlen(x["q"], x["k"], x["v"], x["g"], x["s0"], cut, scale=0.25)
    # all sequences at once, padded to three tokens whose decay is none and whose key is nothing
    at = (torch.arange(3)[None] + cu[:-1, None]).clamp(max=total - 1).cuda()
    live = (torch.arange(3)[None] < lens[:, None]).cuda()
    q, k, v, g = (x[n].double()[at] for n in ("q", "k", "v", "g"))
    k, g = k * live[..., None, None], g * live[..., None]
    s, mag = x["s0"].double(), x["s0"].double().abs()
    for t in range(3):
        a = torch.exp(g[:, t])[..., None, None]
        s = a * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        mag = a * mag + (k[:, t, :, :, None] * v[:, t, :, None, :]).abs()
        want = 0.25 * (s * q[:, t, :, :, None]).sum(2)
        size = 0.25 * (mag * q[:, t, :, :, None].abs()).sum(2)
        on = live[:, t]
        _check({"o": o[at[:, t]][on]}, {"o": want[on]}, {"o": size[on]}, dtype, 3, 16, 16, 1)
    _check({"sT": sT}, {"sT": s}, {"sT": mag}, dtype, 3, 16, 16, 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_in_a_graph_and_on_another_stream(dtype, cuda_device):
    x = _inputs((6,), 2, 4, 64, 64, dtype, 21, grads=False)
    want_o, want_s = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], x["s0"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = {n: t.clone() for n, t in x.items() if t is not None}   # made on that stream
        o, s = api.linear_attention_step(y["q"], y["k"], y["v"], y["g"], y["s0"])
    st.synchronize()
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
    state = x["s0"].clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        o, _ = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], state, out=state)
    state.copy_(x["s0"])
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and torch.equal(state, want_s)
    gr.replay()   # a token more
    torch.cuda.synchronize()
    o2, s2 = api.linear_attention_step(x["q"], x["k"], x["v"], x["g"], want_s)
    assert torch.equal(o, o2) and torch.equal(state, s2)


def test_misaligned_rows(cuda_device):
    """Rows that start on no 16 bytes: refused where the tensor cores would take them, taken elsewhere."""
    x = _inputs((2, 20), 1, 1, 16, 16, BF16, 22)
    wide = torch.zeros(2, 20, 24, dtype=BF16, device="cuda")
    wide[..., 4:20] = x["q"][:, :, 0]
    with pytest.raises(ValueError, match="aligned"):
        api.linear_attention_forward(wide[..., 4:20].unsqueeze(2), x["k"], x["v"], x["g"], x["s0"])
    odd = torch.zeros(2, 20, 19, dtype=BF16, device="cuda")
    odd[..., 3:] = x["q"][:, :, 0]
    o, sT = api.linear_attention_forward(odd[..., 3:].unsqueeze(2), x["k"], x["v"], x["g"], x["s0"], scale=0.25)
    want, size = _dense(x, 0.25)
    _check({"o": o, "sT": sT}, want, size, BF16, 20, 16, 16, 1)


def test_checked_build_runs_clean(cuda_device):
    """The bounds-checked build sees no access out of range on ragged sizes."""
    import ctypes

    from nonlinear_rnn_pararnn_b200 import _lib
    with _lib.checked_library() as lib:
        assert lib.slstm_check_clear() == _lib.SLSTM_OK
        for dtype in (F32, BF16):
            for d in (24, 33):
                x = _inputs((2, 133), 1, 2, d, d, dtype, 23, fused=True)
                _run(x, 1.0)
                api.linear_attention_step(*(x[n][:, 0].contiguous() for n in ("q", "k", "v", "g")), x["s0"])
            x = _inputs((90,), 1, 1, 40, 40, dtype, 24, nseq=3)
            cu = torch.tensor([2, 2, 70, 88], dtype=torch.int32, device="cuda")
            api.linear_attention_forward_varlen(x["q"], x["k"], x["v"], x["g"], x["s0"], cu)
            api.linear_attention_backward_varlen(x["q"], x["k"], x["v"], x["g"], x["s0"], cu, x["dO"], x["dsT"])
            for D in (64, 100):
                z = torch.randn(33, D, device="cuda").to(dtype)
                w = torch.ones(D, device="cuda")
                y, m, r = api.layer_norm_forward(z, w)
                api.layer_norm_backward(z, w, y, m, r)
        out = (ctypes.c_longlong * 4)()
        assert lib.slstm_check_status(out) == _lib.SLSTM_OK and out[0] == 0, list(out)
