"""C-ABI boundary checks of the linear attention and the layer norm that need no
GPU: host-side validation rejects bad arguments before anything is enqueued."""
import ctypes

from nonlinear_rnn_pararnn_b200 import _lib

P = ctypes.c_void_p(0x10000)      # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10001)    # aligned to nothing
NULL = ctypes.c_void_p(0)
BIG = ctypes.c_size_t(1 << 40)
E = _lib.SLSTM_ERR_INVALID_ARG


def _cfg(**kw):
    c = dict(H=4, H_qk=2, d_k=64, d_v=64, dtype=_lib.SLSTM_BF16, decay=_lib.SLSTM_DECAY_TOKEN, scale=1.0, ld_q=128,
             ld_k=128, ld_v=256)
    c.update(kw)
    return _lib.LinearAttentionConfig(**c)


BAD_CONFIGS = [dict(H=0), dict(H_qk=0), dict(H=5), dict(d_k=0), dict(d_v=257), dict(dtype=2), dict(decay=2),
               dict(ld_q=127), dict(ld_k=1), dict(ld_v=255), dict(ld_v=1 << 40)]


def test_linear_attention_rejects_bad_arguments():
    lib = _lib.load()

    def fwd(q=P, k=P, v=P, g=P, s0=NULL, o=P, sT=P, cfg=None, B=2, T=100, ws=P, wb=BIG):
        c = _cfg() if cfg is None else cfg
        return lib.slstm_linear_attention_forward(q, k, v, g, s0, o, sT, ctypes.byref(c), B, T, ws, wb, NULL)

    def bwd(q=P, dO=P, dsT=NULL, dq=P, dk=P, dv=P, dg=P, ds0=P, cfg=None, B=2, T=100, ws=P, wb=BIG):
        c = _cfg() if cfg is None else cfg
        return lib.slstm_linear_attention_backward(q, P, P, P, NULL, dO, dsT, dq, dk, dv, dg, ds0, ctypes.byref(c), B,
                                                   T, ws, wb, NULL)

    for kw in BAD_CONFIGS:
        c = _cfg(**kw)
        assert fwd(cfg=c) == E and bwd(cfg=c) == E, kw
        assert lib.slstm_linear_attention_workspace_size(ctypes.byref(c), 2, 100, 0, 1) == 0
        assert lib.slstm_linear_attention_step(P, P, P, P, NULL, P, P, ctypes.byref(c), 2, NULL) == E
    for call in (fwd, bwd):
        assert call(B=0) == E and call(T=0) == E and call(B=1 << 20, T=1 << 20) == E
        assert call(ws=NULL) == E and call(wb=ctypes.c_size_t(16)) == E and call(q=NULL) == E and call(q=MIS) == E
    for name in ("k", "v", "g", "o"):
        assert fwd(**{name: NULL}) == E and fwd(**{name: MIS}) == E
    assert fwd(sT=MIS) == E and fwd(s0=MIS) == E
    for name in ("dO", "dq", "dk", "dv"):
        assert bwd(**{name: NULL}) == E and bwd(**{name: MIS}) == E
    assert bwd(dsT=MIS) == E and bwd(ds0=MIS) == E and bwd(dg=MIS) == E
    c = _cfg()
    none = ctypes.POINTER(_lib.LinearAttentionConfig)()
    assert lib.slstm_linear_attention_forward(P, P, P, P, NULL, P, P, none, 2, 100, P, BIG, NULL) == E
    for cu in (NULL, MIS):
        assert lib.slstm_linear_attention_forward_varlen(P, P, P, P, NULL, cu, 2, P, P, ctypes.byref(c), 100, P, BIG,
                                                         NULL) == E
        assert lib.slstm_linear_attention_backward_varlen(P, P, P, P, NULL, cu, 2, P, NULL, P, P, P, P, P,
                                                          ctypes.byref(c), 100, P, BIG, NULL) == E
    assert lib.slstm_linear_attention_forward_varlen(P, P, P, P, NULL, P, 0, P, P, ctypes.byref(c), 100, P, BIG,
                                                     NULL) == E
    assert lib.slstm_linear_attention_step(P, P, P, P, NULL, NULL, P, ctypes.byref(c), 2, NULL) == E
    assert lib.slstm_linear_attention_step(P, P, P, P, NULL, P, P, ctypes.byref(c), 0, NULL) == E


def test_linear_attention_workspace_sizes():
    lib = _lib.load()
    c = ctypes.byref(_cfg())
    size = lib.slstm_linear_attention_workspace_size
    assert 0 < size(c, 2, 100, 0, 0) <= size(c, 2, 1000, 0, 0)
    assert size(c, 2, 1000, 0, 0) <= size(c, 2, 1000, 0, 1)
    assert size(c, 5, 100, 1, 0) > 0            # more sequences than a chunk each
    assert size(c, 2, 100, 0, 0) % 256 == 0


def test_layer_norm_rejects_bad_arguments():
    lib = _lib.load()
    F, H = _lib.SLSTM_F32, _lib.SLSTM_BF16

    def fwd(x=P, xt=F, w=P, b=NULL, y=P, yt=H, mean=P, rstd=P, rows=4, groups=1, d=32, eps=1e-5):
        return lib.slstm_layer_norm_forward(x, xt, w, b, y, yt, mean, rstd, rows, groups, d, eps, NULL)

    def bwd(x=P, xt=F, w=P, dy=P, yt=H, mean=P, rstd=P, dx=P, dw=P, db=P, rows=4, groups=1, d=32, ws=P, wb=BIG):
        return lib.slstm_layer_norm_backward(x, xt, w, dy, yt, mean, rstd, dx, dw, db, rows, groups, d, ws, wb, NULL)

    for call in (fwd, bwd):
        assert call(xt=2) == E and call(yt=-1) == E
        assert call(rows=0) == E and call(groups=0) == E and call(d=0) == E and call(d=16385) == E
        assert call(rows=1 << 31) == E and call(rows=1 << 20, groups=1 << 12) == E and call(groups=65536) == E
        for name in ("x", "w", "mean", "rstd"):
            assert call(**{name: NULL}) == E and call(**{name: MIS}) == E
    assert fwd(y=NULL) == E and fwd(b=MIS) == E and fwd(eps=-1.0) == E and fwd(eps=float("nan")) == E
    for name in ("dy", "dx", "dw", "db"):
        assert bwd(**{name: NULL}) == E and bwd(**{name: MIS}) == E
    assert bwd(ws=NULL) == E and bwd(wb=ctypes.c_size_t(8)) == E
    assert lib.slstm_layer_norm_workspace_size(4, 1, 0) == 0
    assert lib.slstm_layer_norm_workspace_size(4, 2, 32) > 0
