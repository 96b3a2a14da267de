"""Argument checks of the gated block's operators: every refusal happens on the host, before any HIP
call, and names its argument.  Runs where no GPU is visible, so that even a check that failed could
not send a made-up address to a kernel."""
import ctypes
import os

import pytest

from tensor_transformer_mlp_03_amd import _lib as L


def _gpu_visible():
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:
        return False


pytestmark = [
    pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="libtpmlp.so not built"),
    pytest.mark.skipif(_gpu_visible(), reason="made-up device addresses are only passed where no GPU is visible"),
]

OK, NULL, SHAPE, ALIGN, WS, SHARDS, HIP, UNSUP, ALIAS, NO_FORWARD = range(10)
PASSED = (HIP, UNSUP)  # every check passed: the next step is the device's
F32, BF16 = 0, 1


def _p(i, off=0):
    return (1 << 40) + i * (1 << 34) + off


def _err():
    return L.lib().tpmlp_last_error().decode()


def _call(fn, defaults, kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    st = getattr(L.lib(), fn)(*{**defaults, **kw}.values(), None)
    return st, _err()


def _refused(call, cases):
    for kw, status, text in cases:
        st, msg = call(**kw)
        assert st == status and text in msg, (kw, st, msg)


# --- the gated MLP --------------------------------------------------------------------------------
def glu_fwd(**kw):
    return _call("tpmlp_glu_fwd", dict(X=_p(0), A=_p(1), B=_p(2), Z=_p(3), t=F32, P=_p(4), act=1, M=33, H=64, F=40, ws=_p(5),
                                       n=1 << 30), kw)


def glu_bwd(**kw):
    return _call("tpmlp_glu_bwd", dict(dZ=_p(0), X=_p(1), A=_p(2), B=_p(3), P=_p(4), dX=_p(5), xt=F32, dA=_p(6), dB=_p(7),
                                       wt=BF16, act=1, M=33, H=64, F=40, ws=_p(8), n=1 << 30), kw)


def test_glu_accepts():
    for act in (1, 2, 3, 4):
        assert glu_fwd(act=act)[0] in PASSED and glu_bwd(act=act)[0] in PASSED
    for M in (1, 7, 8, 1 << 23):
        assert glu_fwd(M=M, n=1 << 60)[0] in PASSED and glu_bwd(M=M, P=None, n=1 << 60)[0] in PASSED, M
    assert glu_fwd(P=None, t=BF16)[0] in PASSED
    assert glu_fwd(M=0, X=None, Z=None, P=None, ws=None, n=0)[0] == OK      # no tokens
    assert glu_bwd(M=0, dZ=None, X=None, P=None, dX=None, ws=None, n=0)[0] in PASSED  # dA and dB are zeroed


def test_glu_refuses():
    for call in (glu_fwd, glu_bwd):
        _refused(call, [(dict(M=-1), SHAPE, "M outside"), (dict(M=(1 << 23) + 1), SHAPE, "M outside"), (dict(H=60), SHAPE, "H"),
                        (dict(H=0), SHAPE, "H"), (dict(F=4), SHAPE, "F"), (dict(F=(1 << 22) + 8), SHAPE, "F"),
                        (dict(act=0), SHAPE, "act"), (dict(act=5), SHAPE, "act"), (dict(X=None), NULL, "X"),
                        (dict(A=None), NULL, "A"), (dict(B=None), NULL, "B"), (dict(X=_p(0, 8)), ALIGN, "X"),
                        (dict(P=_p(4, 2)), ALIGN, "P"), (dict(ws=None), NULL, "ws"), (dict(ws=_p(5, 4)), ALIGN, "ws"),
                        (dict(n=16), WS, "workspace_bytes")])
    _refused(glu_fwd, [(dict(t=2), SHAPE, "z_type"), (dict(Z=None), NULL, "Z"), (dict(Z=_p(0, 16)), ALIAS, "Z overlaps X"),
                       (dict(P=_p(1)), ALIAS, "P_save overlaps A"), (dict(ws=_p(3)), ALIAS, "ws")])
    _refused(glu_bwd, [(dict(xt=-1), SHAPE, "dx_type"), (dict(wt=2), SHAPE, "dw_type"), (dict(dA=None), NULL, "dA"),
                       (dict(dB=None, M=0), NULL, "dB"), (dict(dX=_p(0)), ALIAS, "dX overlaps dZ"),
                       (dict(dA=_p(7, 32)), ALIAS, "dA"), (dict(dB=_p(4)), ALIAS, "dB overlaps P_saved")])


def test_glu_workspace():
    q, b = L.lib().tpmlp_glu_fwd_workspace_bytes, L.lib().tpmlp_glu_bwd_workspace_bytes
    for bad in ((0, 64, 64), (-1, 64, 64), (8, 63, 64), (8, 64, 0), ((1 << 23) + 1, 64, 64)):
        assert q(*bad) == 0 and b(*bad, 1) == 0
    for M, H, F in ((1, 64, 64), (33, 264, 1368), (2048, 4096, 2048), (32768, 3584, 3584)):
        n = q(M, H, F)
        assert n >= 2 * M * F
        assert b(M, H, F, 1) >= b(M, H, F, 0) + 4 * M * F - 512
        assert glu_fwd(M=M, H=H, F=F, n=n)[0] in PASSED and glu_fwd(M=M, H=H, F=F, n=n - 1)[0] == WS
        assert glu_bwd(M=M, H=H, F=F, P=None, n=b(M, H, F, 1))[0] in PASSED
        assert glu_bwd(M=M, H=H, F=F, P=None, n=b(M, H, F, 1) - 1)[0] == WS


# --- dropout ------------------------------------------------------------------------------------------
def drop_fwd(**kw):
    return _call("tpmlp_dropout_fwd", dict(y=_p(0), yt=F32, ly=0, b=_p(1), bt=BF16, r=_p(2), lr=0, out=_p(3), ot=BF16, lo=0, M=16,
                                           H=65, p=0.1, state=_p(4), site=0, first=0), kw)


def drop_bwd(**kw):
    return _call("tpmlp_dropout_bwd", dict(d=_p(0), ot=BF16, ld=0, dy=_p(1), yt=F32, ly=0, db=_p(2), M=16, H=65, p=0.1, state=_p(3),
                                           site=0, first=0, ws=_p(4), n=1 << 30), kw)


def test_dropout_accepts():
    for p in (0.0, 0.5, 1.0):
        assert drop_fwd(p=p)[0] in PASSED and drop_bwd(p=p)[0] in PASSED
    assert drop_fwd(b=None, r=None)[0] in PASSED
    assert drop_fwd(out=_p(2))[0] in PASSED                         # over r
    assert drop_fwd(out=_p(0), ot=F32, r=None)[0] in PASSED         # over y of its type
    assert drop_fwd(ly=70, lr=66, lo=67, y=_p(0, 4))[0] in PASSED
    assert drop_fwd(M=1 << 23, first=(1 << 32) - (1 << 23))[0] in PASSED
    assert drop_fwd(M=0, y=None, r=None, out=None)[0] == OK
    assert drop_bwd(db=None, ws=None, n=0)[0] in PASSED
    assert drop_bwd(dy=_p(0), yt=BF16)[0] in PASSED                 # over dout of its type
    assert drop_bwd(M=0, d=None, dy=None, db=None)[0] == OK
    assert drop_bwd(M=0, d=None, dy=None)[0] in PASSED              # db is zeroed


def test_dropout_refuses():
    for call in (drop_fwd, drop_bwd):
        _refused(call, [(dict(M=-1), SHAPE, "M outside"), (dict(M=(1 << 23) + 1), SHAPE, "M outside"), (dict(H=0), SHAPE, "H outside"),
                        (dict(H=(1 << 23) + 1), SHAPE, "H outside"), (dict(p=-0.1), SHAPE, "p must"), (dict(p=1.1), SHAPE, "p must"),
                        (dict(p=float("nan")), SHAPE, "p must"), (dict(first=-1), SHAPE, "first_row"),
                        (dict(first=(1 << 32) - 15), SHAPE, "first_row"), (dict(state=None), NULL, "state"),
                        (dict(state=_p(4, 4)), ALIGN, "state"), (dict(yt=2), SHAPE, "y_type"), (dict(ot=2), SHAPE, "out_type"),
                        (dict(ly=64), SHAPE, "ld of")])
    _refused(drop_fwd, [(dict(bt=3), SHAPE, "bias_type"), (dict(y=None), NULL, "y"), (dict(out=None), NULL, "out"),
                        (dict(out=_p(3, 1)), ALIGN, "out"), (dict(out=_p(0)), ALIAS, "out overlaps y"),  # another type
                        (dict(out=_p(2), lo=66), ALIAS, "out overlaps r"), (dict(b=_p(3)), ALIAS, "out overlaps bias"),
                        (dict(state=_p(3)), ALIAS, "out overlaps state")])
    _refused(drop_bwd, [(dict(d=None), NULL, "dout"), (dict(dy=None), NULL, "dy"), (dict(ws=None), NULL, "ws"),
                        (dict(ws=_p(4, 8)), ALIGN, "ws"), (dict(n=4), WS, "tpmlp_dropout_bwd_workspace_bytes"),
                        (dict(db=_p(1)), ALIAS, "overlaps"), (dict(db=_p(0)), ALIAS, "db overlaps dout"),
                        (dict(dy=_p(0), yt=BF16, db=_p(0, 128)), ALIAS, "overlaps"), (dict(dy=_p(0)), ALIAS, "dy overlaps dout"),
                        (dict(ws=_p(3)), ALIAS, "ws overlaps state")])


# --- the edge in 8 bits -----------------------------------------------------------------------------------
def edge8(d=None, **kw):
    a = dict(M=16, H=64, post=1, pre=1, y_type=0, r_type=0, param_type=1, alpha=1.0, eps=1e-5, w_post=_p(10), b_post=None,
             w_pre=_p(11), b_pre=None, gate=None, gate_rows=0, ld_gate=0)
    a.update(d or {})
    return _call("tpmlp_edge_fwd_fp8", dict(e=ctypes.byref(L.EdgeDesc(**a)), y=_p(0), ly=0, r=_p(1), lr=0, ro=_p(2), lo=0, c=_p(3),
                                            lc=0, s=_p(4), ls=0, kind=0), kw)


def test_edge8_accepts():
    assert edge8()[0] in PASSED and edge8(kind=1)[0] in PASSED
    assert edge8(ro=_p(1))[0] in PASSED and edge8(ro=None)[0] in PASSED
    assert edge8(dict(H=65), lc=67, c=_p(3, 1))[0] in PASSED
    assert edge8(dict(H=96), kind=1, ls=5, s=_p(4, 1))[0] in PASSED
    assert edge8(dict(post=0, w_post=None), y=None)[0] in PASSED
    assert edge8(dict(M=0), y=None, r=None, ro=None, c=None, s=None)[0] == OK


def test_edge8_refuses():
    _refused(edge8, [(dict(d=dict(H=65), kind=1), SHAPE, "multiple of 32"), (dict(kind=2), SHAPE, "scale_kind"),
                     (dict(ls=4), SHAPE, "ld_scales"), (dict(kind=1, ls=1), SHAPE, "scales"), (dict(c=None), NULL, "codes"),
                     (dict(s=None), NULL, "scales"), (dict(s=_p(4, 2)), ALIGN, "scales"),
                     (dict(d=dict(pre=0, w_pre=None)), SHAPE, "norm before"), (dict(s=_p(3, 64)), ALIAS, "codes overlaps scales"),
                     (dict(c=_p(1)), ALIAS, "codes overlaps r"), (dict(s=_p(0)), ALIAS, "scales overlaps y"),
                     (dict(d=dict(H=7)), SHAPE, "H outside"), (dict(lc=63), SHAPE, "codes")])
    assert L.lib().tpmlp_edge_fwd_fp8(None, *[None, 0] * 5, 0, None) == NULL


# --- 4-bit products ---------------------------------------------------------------------------------------
def quantize(**kw):
    return _call("tpmlp_fp4_quantize", dict(W=_p(0), ld=0, K=64, N=9, c=_p(1), s=_p(2)), kw)


def fp4(**kw):
    return _call("tpmlp_fp4_fwd", dict(X=_p(0), kind=0, lx=0, xs=None, p=_p(1), Y=_p(3), yt=F32, ly=0, act=0, gated=0, M=5, N=9,
                                       K=64), kw)


def pack(**kw):
    return _call("tpmlp_fp4_pack", dict(c=_p(1), s=_p(2), p=_p(3), gated=0, N=9, K=64), kw)


def test_fp4_accepts():
    assert quantize()[0] in PASSED and quantize(ld=10, W=_p(0, 2))[0] in PASSED
    for act in range(5):
        assert fp4(act=act, gated=act % 2)[0] in PASSED
    assert fp4(kind=1, xs=_p(4))[0] in PASSED and fp4(kind=2, xs=_p(4, 1))[0] in PASSED
    assert fp4(lx=72, ly=11, Y=_p(3, 4), yt=BF16)[0] in PASSED and fp4(M=1 << 23)[0] in PASSED
    assert fp4(M=0, X=None, Y=None)[0] == OK and fp4(M=0, X=None, Y=None, kind=1)[0] == OK
    assert pack()[0] in PASSED and pack(gated=1, s=_p(2, 1))[0] in PASSED
    assert fp4(lx=1 << 30)[0] in PASSED


def test_fp4_sizes():
    packed = L.lib().tpmlp_fp4_packed_bytes
    for bad in ((0, 64), (9, 0), (9, 48), ((1 << 23) + 1, 64), (9, (1 << 23) + 32)):
        assert packed(*bad, 0) == 0
    assert packed(9, 64, 0) == 1024 + 64 and packed(9, 64, 1) == 2 * packed(9, 64, 0)
    assert packed(17, 544, 0) == 2 * 5 * (1024 + 64)
    assert packed(1 << 23, 1 << 23, 1) > 1 << 45


def test_fp4_refuses():
    for call in (quantize, fp4, pack):
        _refused(call, [(dict(N=0), SHAPE, "N outside"), (dict(N=(1 << 23) + 1), SHAPE, "N outside"), (dict(K=0), SHAPE, "K"),
                        (dict(K=48), SHAPE, "K"), (dict(K=(1 << 23) + 32), SHAPE, "K")])
    for call in (quantize, pack):
        _refused(call, [(dict(c=None), NULL, "codes"), (dict(s=None), NULL, "scales"), (dict(c=_p(1, 8)), ALIGN, "codes")])
    for call in (fp4, pack):
        _refused(call, [(dict(p=None), NULL, "packed"), (dict(p=_p(1, 8)), ALIGN, "packed")])
    _refused(pack, [(dict(p=_p(1)), ALIAS, "packed overlaps codes"), (dict(p=_p(2, -1072)), ALIAS, "packed overlaps scales"),
                    (dict(p=_p(2, -2160), gated=1), ALIAS, "packed overlaps scales")])
    _refused(quantize, [(dict(W=None), NULL, "W"), (dict(ld=8), SHAPE, "ld of W"), (dict(c=_p(0, 16)), ALIAS, "codes overlaps W"),
                        (dict(s=_p(1, 16)), ALIAS, "codes overlaps scales")])
    _refused(fp4, [(dict(M=-1), SHAPE, "M outside"), (dict(M=(1 << 23) + 1), SHAPE, "M outside"), (dict(kind=3), SHAPE, "x_kind"),
                   (dict(act=5), SHAPE, "act"), (dict(yt=2), SHAPE, "y_type"), (dict(X=None), NULL, "X"), (dict(Y=None), NULL, "Y"),
                   (dict(kind=1), NULL, "x_scales"), (dict(xs=_p(4)), SHAPE, "x_scales"), (dict(X=_p(0, 2)), ALIGN, "X"),
                   (dict(lx=68), ALIGN, "X"), (dict(lx=(1 << 31) + 8), SHAPE, "ld of X"), (dict(kind=1, xs=_p(4, 2)), ALIGN, "x_scales"),
                   (dict(lx=56), SHAPE, "ld of X"), (dict(Y=_p(0)), ALIAS, "Y overlaps X"), (dict(Y=_p(1)), ALIAS, "Y overlaps packed"),
                   (dict(kind=1, xs=_p(3)), ALIAS, "Y overlaps x_scales"), (dict(ly=8), SHAPE, "ld of Y")])


# --- the binding ----------------------------------------------------------------------------------------
def test_binding_refuses():
    torch = pytest.importorskip("torch")
    from tensor_transformer_mlp_03_amd import gated
    from tensor_transformer_mlp_03_amd.block import Edge
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="A has shape"):
        gated.GatedMLP(z(64, 80), z(48, 64))
    for act in ("none", "tanh"):
        with pytest.raises(ValueError, match="no gate"):
            gated.GatedMLP(z(64, 80), z(40, 64), act=act)
    m = gated.GatedMLP(z(64, 80), z(40, 64))
    with pytest.raises(ValueError, match="Z has shape"):
        m.forward(z(5, 64), z(4, 64))
    with pytest.raises(ValueError, match="P_save has shape"):
        m.forward(z(5, 64), z(5, 64), z(5, 40))
    with pytest.raises(TypeError, match="X must be bf16"):
        m.forward(z(5, 64, dtype=f32), z(5, 64))
    with pytest.raises(ValueError, match="X must be contiguous"):
        m.forward(z(5, 128)[:, ::2], z(5, 64))
    with pytest.raises(TypeError, match="dB must be bf16"):
        m.backward(z(5, 64), z(5, 64), None, z(5, 64), z(64, 80), z(40, 64, dtype=f32))
    with pytest.raises(TypeError, match="float32 or hold bf16"):
        m.forward(z(5, 64), z(5, 64, dtype=torch.float16))
    state = torch.zeros(2, dtype=torch.int64)
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError, match="p must"):
            gated.Dropout(p, state)
    with pytest.raises(TypeError, match="state"):
        gated.Dropout(0.1, torch.zeros(2)).forward(z(5, 64), None, z(5, 64))
    with pytest.raises(ValueError, match="site"):
        gated.Dropout(0.1, state, site=1 << 32).forward(z(5, 64), None, z(5, 64))
    with pytest.raises(TypeError, match="r must be bf16"):
        gated.Dropout(0.1, state).forward(z(5, 64), z(5, 64, dtype=f32), z(5, 64))
    with pytest.raises(ValueError, match="bias holds"):
        gated.Dropout(0.1, state, bias=z(63)).forward(z(5, 64), None, z(5, 64))
    with pytest.raises(ValueError, match="4-bit weight"):
        gated.Fp4Linear(z(9, 24, dtype=u8), z(9, 1, dtype=u8))
    with pytest.raises(ValueError, match="scales has shape"):
        gated.Fp4Linear(z(9, 32, dtype=u8), z(9, 1, dtype=u8))
    with pytest.raises(ValueError, match="4-bit weight"):
        gated.Fp4Linear(z(9, 32, dtype=u8), z(9, 2, dtype=u8), gated=True)
    with pytest.raises(ValueError, match="blocks of 32"):
        gated.Fp4Linear.from_weight(z(40, 9))
    with pytest.raises(ValueError, match="packed holds"):
        L.tpmlp_fp4_pack(z(9, 32, dtype=u8), z(9, 2, dtype=u8), z(1087, dtype=u8))
    q = object.__new__(gated.Fp4Linear)  # without the packing, which needs a GPU
    q.K, q.N, q.act, q.gated, q.packed, q._ws = 64, 9, "none", False, z(1088, dtype=u8), gated._Workspace()
    q._sizes = {}
    with pytest.raises(ValueError, match="do not fit"):
        q.forward(z(5, 32), z(5, 9))
    with pytest.raises(ValueError, match="needs x_scales"):
        q.forward(z(5, 64, dtype=u8), z(5, 9))
    with pytest.raises(ValueError, match="bf16 X"):
        q.forward(z(5, 64), z(5, 9), torch.zeros(5))
    with pytest.raises(ValueError, match="x_scales holds"):
        q.forward(z(5, 64, dtype=u8), z(5, 9), torch.zeros(4))
    with pytest.raises(TypeError, match="one-byte"):
        q.forward(z(5, 64, dtype=u8), z(5, 9), torch.zeros(5, 2, dtype=bf))
    with pytest.raises(ValueError, match="packed holds"):
        L.tpmlp_fp4_fwd(z(5, 64), None, z(1087, dtype=u8), z(5, 9))
    e = Edge(64, pre="rms", w_pre=z(64))
    with pytest.raises(TypeError, match="codes must hold one-byte"):
        e.forward_fp8(None, z(5, 64), None, z(5, 64), torch.zeros(5))
    with pytest.raises(ValueError, match="scales has shape"):
        e.forward_fp8(None, z(5, 64), None, z(5, 64, dtype=u8), z(5, 1, dtype=u8))
