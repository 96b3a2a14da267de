"""Argument checks of the block operators: every refusal happens on the host, before any
HIP call, and names its argument.  Runs where no GPU is visible, so that even a check that
failed could not send a made-up address to a kernel."""
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


def _p(i, off=0):
    return (1 << 40) + i * (1 << 34) + off


def _err():
    return L.lib().tpmlp_last_error().decode()


# --- edge -------------------------------------------------------------------------------------------------------
def _desc(**kw):
    a = dict(M=16, H=64, post=1, pre=1, y_type=0, r_type=0, param_type=1, alpha=1.0, eps=1e-5, w_post=_p(10),
             b_post=None, w_pre=_p(11), b_pre=None, gate=None, gate_rows=0, ld_gate=0)
    a.update(kw)
    return L.EdgeDesc(**a)


def _fwd(d=None, **kw):
    a = dict(y=_p(0), ly=0, r=_p(1), lr=0, ro=_p(2), lo=0, x=_p(3), lx=0)
    a.update(kw)
    d = _desc() if d is None else d
    st = L.lib().tpmlp_edge_fwd(ctypes.byref(d), a["y"], a["ly"], a["r"], a["lr"], a["ro"], a["lo"], a["x"], a["lx"], None)
    return st, _err()


def _bwd(d=None, **kw):
    a = dict(y=_p(0), ly=0, r=_p(1), lr=0, do=_p(2), lo=0, dx=_p(3), t=0, lx=0, dr=_p(4), ld=0, dy=_p(5), lg=0,
             dwp=_p(6), dbp=None, dwn=_p(7), dbn=None, dg=None, ws=_p(8), n=1 << 30)
    a.update(kw)
    d = _desc() if d is None else d
    st = L.lib().tpmlp_edge_bwd(ctypes.byref(d), *a.values(), None)
    return st, _err()


def test_edge_accepts():
    assert _fwd()[0] in PASSED and _bwd()[0] in PASSED
    assert _fwd(ro=_p(1))[0] in PASSED                                   # the stream in place
    assert _fwd(ro=None)[0] in PASSED                                    # only x wanted
    assert _fwd(_desc(post=0, w_post=None), y=None, ro=None)[0] in PASSED  # the first block's entry
    assert _fwd(_desc(pre=0, w_pre=None), x=None)[0] in PASSED
    assert _fwd(_desc(H=65), ly=67, y=_p(0, 4))[0] in PASSED             # odd sizes, strides and addresses
    assert _bwd(dr=_p(2))[0] in PASSED                                   # dr over dr_out
    assert _bwd(do=None)[0] in PASSED
    assert _bwd(dwp=None, dwn=None, ws=None, n=0)[0] in PASSED
    assert _fwd(_desc(M=0), y=None, r=None, ro=None, x=None)[0] == OK    # no tokens
    # column blocks of one buffer
    assert _fwd(y=_p(0), ly=512, x=_p(0, 64 * 4), lx=1024)[0] in PASSED


def test_edge_refuses():
    assert L.lib().tpmlp_edge_fwd(None, *[None, 0] * 4, None) == NULL
    for kw, text in ((dict(M=-1), "M outside"), (dict(M=(1 << 23) + 1), "M outside"),
                     (dict(M=1 << 23, gate=_p(13), gate_rows=3), "2^21 rows"), (dict(H=7), "H outside"), (dict(H=32769), "H outside"),
                     (dict(post=3), "tpmlp_norm"), (dict(r_type=2), "tpmlp_dtype"), (dict(param_type=-1), "tpmlp_dtype"),
                     (dict(alpha=float("nan")), "alpha"), (dict(eps=-1.0), "eps"), (dict(eps=float("inf")), "eps"),
                     (dict(post=0), "w_post"), (dict(b_post=_p(12)), "b_post"), (dict(b_pre=_p(12)), "b_pre"),
                     (dict(gate=_p(13), gate_rows=0), "gate_rows"),
                     (dict(gate=_p(13), gate_rows=4, ld_gate=63), "gate")):
        for call in (_fwd, _bwd):
            st, msg = call(_desc(**kw))
            assert st == SHAPE and text in msg, (kw, st, msg)
    for kw, text in ((dict(w_post=None), "w_post"), (dict(w_pre=None), "w_pre")):
        st, msg = _fwd(_desc(**kw))
        assert st == NULL and text in msg
    assert _fwd(_desc(w_pre=_p(11, 1)))[0] == ALIGN
    for kw, text in ((dict(r=None), "r is"), (dict(x=None), "x"), (dict(y=None), "y")):
        st, msg = _fwd(**kw)
        assert st == NULL and text in msg, (kw, msg)
    assert _fwd(_desc(pre=0, w_pre=None))[0] == SHAPE                     # x without a norm
    assert _fwd(_desc(pre=0, w_pre=None), x=None, ro=None)[0] == NULL    # nothing to write
    assert _fwd(ly=63)[0] == SHAPE
    assert _fwd(y=_p(0, 2))[0] == ALIGN and _fwd(x=_p(3, 1))[0] == ALIGN
    for kw in (dict(x=_p(1)), dict(ro=_p(0)), dict(ro=_p(1, 4)), dict(ro=_p(1), lo=128), dict(x=_p(2, 512)),
               dict(x=_p(10)), dict(y=_p(0), ly=512, x=_p(0, 64 * 4 - 2), lx=1024)):
        st, msg = _fwd(**kw)
        assert st == ALIAS, (kw, st, msg)


def test_edge_backward_refuses():
    for kw, text in ((dict(dx=None), "dx"), (dict(r=None), "r_out"), (dict(dr=None), "dr"), (dict(dy=None), "dy"),
                     (dict(ws=None), "ws")):
        st, msg = _bwd(**kw)
        assert st == NULL and text in msg, (kw, st, msg)
    assert _bwd(t=2)[0] == SHAPE
    for kw in (dict(dbp=_p(9)), dict(dbn=_p(9)), dict(dg=_p(9))):
        assert _bwd(**kw)[0] == SHAPE                                     # a gradient without its parameter
    plain = dict(pre=0, w_pre=None)
    assert _bwd(_desc(**plain), dwn=None)[0] == SHAPE                      # dx without a norm
    assert _bwd(_desc(**plain), dwn=None, dx=None, r=None, do=None)[0] == NULL
    assert _bwd(_desc(**plain), dwn=None, dx=None, r=None)[0] in PASSED
    assert _bwd(_desc(post=0, w_post=None), y=None, dwp=None)[0] == SHAPE  # dy without y
    d = _desc()
    need = L.lib().tpmlp_edge_bwd_workspace_bytes(ctypes.byref(d))
    assert need > 0 and _bwd(n=need)[0] in PASSED and _bwd(n=need - 1)[0] == WS
    assert _bwd(ws=_p(8, 8))[0] == ALIGN and _bwd(dwp=_p(6, 2))[0] == ALIGN
    for kw in (dict(dr=_p(1)), dict(dr=_p(2, 4)), dict(dy=_p(0)), dict(dwp=_p(7)), dict(dwp=_p(3)), dict(ws=_p(4)),
               dict(dwn=_p(11))):
        assert _bwd(**kw)[0] == ALIAS, kw


def test_edge_workspace_query():
    q = lambda **kw: L.lib().tpmlp_edge_bwd_workspace_bytes(ctypes.byref(_desc(**kw)))  # noqa: E731
    assert q(M=0) == 0 and q(H=4) == 0 and q(gate=_p(1), gate_rows=0) == 0
    assert q(M=4096, H=1024) >= 2 * 1024 * 4
    assert q(M=4096, H=1024, post=2) == 2 * q(M=4096, H=1024)            # a LayerNorm keeps twice the sums
    assert q(M=64, gate=_p(1), gate_rows=1) >= 64 * 64 * 4               # a slice a gate row


# --- route ------------------------------------------------------------------------------------------------------
def test_route_rows():
    rows = lambda *a: L.lib().tpmlp_route_rows(*a)  # noqa: E731
    assert rows(16, 2, 8, 8, 0) == 32 + 8 * 7
    assert rows(1, 1, 8, 8, 0) == 8 and rows(0, 1, 8, 8, 0) == 0
    assert rows(5, 3, 4, 1, 0) == 15 and rows(5, 3, 4, 8, 24) == 96
    for bad in (((1 << 23) + 1, 1, 8, 8, 0), (-1, 1, 8, 8, 0), (4, 0, 8, 8, 0), (4, 65, 8, 8, 0), (4, 1, 0, 8, 0), (4, 1, 513, 8, 0), (4, 1, 8, 0, 0),
                (4, 1, 8, 8, 12), (4, 1, 8, 8, -8), (1 << 31, 1, 8, 8, 0), (1 << 30, 2, 8, 8, 0),
                (4, 1, 512, 8, 1 << 23)):
        assert rows(*bad) == -1, bad


def _sort(**kw):
    a = dict(ids=_p(0), bits=32, T=4096, K=4, E=16, align=8, capacity=0, counts=_p(1), offsets=_p(2), row_of=_p(3),
             src_of=_p(4), ws=_p(5), n=1 << 24)
    a.update(kw)
    return L.lib().tpmlp_route_sort(*a.values(), None), _err()


def test_route_sort_arguments():
    assert _sort()[0] in PASSED and _sort(bits=64)[0] in PASSED
    assert _sort(T=8, ws=None, n=0)[0] in PASSED                          # one workgroup needs no workspace
    assert _sort(T=0, ids=None, row_of=None, src_of=None, ws=None, n=0)[0] in PASSED
    for kw in (dict(bits=16), dict(K=0), dict(E=0), dict(E=513), dict(align=0), dict(capacity=4), dict(T=-1)):
        assert _sort(**kw)[0] == SHAPE, kw
    for k in ("ids", "counts", "offsets", "row_of", "src_of", "ws"):
        assert _sort(**{k: None})[0] == NULL, k
    need = L.lib().tpmlp_route_workspace_bytes(4096, 4, 16)
    assert need > 0 and _sort(n=need)[0] in PASSED and _sort(n=need - 1)[0] == WS
    assert _sort(ids=_p(0, 2))[0] == ALIGN and _sort(bits=64, ids=_p(0, 4))[0] == ALIGN
    for kw in (dict(row_of=_p(0)), dict(counts=_p(2)), dict(ws=_p(4)), dict(ws=_p(0))):
        assert _sort(**kw)[0] == ALIAS, kw


def _dispatch(**kw):
    a = dict(X=_p(0), lx=0, row_of=_p(1), src_of=_p(2), T=16, K=2, H=64, rows=64, Xs=_p(3), ls=0)
    a.update(kw)
    return L.lib().tpmlp_route_dispatch(*a.values(), None), _err()


def _combine(**kw):
    a = dict(Zs=_p(0), zt=0, lz=0, row_of=_p(1), w=_p(2), T=16, K=2, H=64, rows=64, Y=_p(3), yt=0, ly=0)
    a.update(kw)
    return L.lib().tpmlp_route_combine(*a.values(), None), _err()


def _combine_bwd(**kw):
    a = dict(dY=_p(0), dt=0, ld=0, Zs=_p(1), zt=0, lz=0, row_of=_p(2), src_of=_p(3), w=_p(4), T=16, K=2, H=64, rows=64,
             dZs=_p(5), lo=0, dw=_p(6))
    a.update(kw)
    return L.lib().tpmlp_route_combine_bwd(*a.values(), None), _err()


def test_route_moves_arguments():
    for call, outs in ((_dispatch, ("Xs",)), (_combine, ("Y",)), (_combine_bwd, ("dZs", "dw"))):
        assert call()[0] in PASSED
        for kw in (dict(H=7), dict(H=(1 << 23) + 1), dict(K=0), dict(K=65), dict(T=-1), dict(rows=-1), dict(rows=1 << 31)):
            assert call(**kw)[0] == SHAPE, (call, kw)
        for o in outs:
            assert call(**{o: _p(1 if call is not _combine_bwd else 2)})[0] == ALIAS  # on row_of
            assert call(**{o: _p(9, 1)})[0] == ALIGN
        assert call(row_of=None)[0] == NULL
    assert _dispatch(X=None)[0] == NULL and _dispatch(src_of=None)[0] == NULL and _dispatch(Xs=None)[0] == NULL
    assert _dispatch(lx=63)[0] == SHAPE and _dispatch(rows=0, src_of=None, Xs=None)[0] == OK
    assert _combine(w=None)[0] in PASSED and _combine(zt=2)[0] == SHAPE and _combine(yt=-1)[0] == SHAPE
    assert _combine(T=0, row_of=None, w=None, Y=None)[0] == OK
    assert _combine_bwd(w=None)[0] in PASSED and _combine_bwd(dt=3)[0] == SHAPE
    assert _combine_bwd(dw=None, Zs=None)[0] in PASSED and _combine_bwd(dZs=None, src_of=None)[0] in PASSED
    for kw in (dict(dw=None), dict(Zs=None), dict(dZs=None), dict(src_of=None),
               dict(dw=None, Zs=None, dZs=None, src_of=None)):
        assert _combine_bwd(**kw)[0] == NULL, kw


# --- clipping ---------------------------------------------------------------------------------------------------
def _arrays(ptrs, outs, sizes, types):
    n = len(ptrs)
    v, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    return ((v * n)(*ptrs), None if outs is None else (v * n)(*outs), (i64 * n)(*sizes), (i32 * n)(*types), n)


def _clip(ptrs=(_p(0), _p(1, 2)), outs=None, sizes=(100, 7), types=(0, 1), scale=1.0, max_norm=1.0, norm=_p(2), ws=_p(3),
          n_ws=1 << 20):
    g, o, s, t, n = _arrays(ptrs, outs, sizes, types)
    return L.lib().tpmlp_clip_grad_norm(g, o, s, t, n, scale, max_norm, norm, ws, n_ws, None), _err()


def test_clip_arguments():
    assert _clip()[0] in PASSED and _clip(norm=None)[0] in PASSED
    assert _clip(outs=(_p(4), _p(1, 2)))[0] in PASSED
    assert _clip(ptrs=(None, _p(1)), sizes=(0, 7))[0] in PASSED            # a tensor without elements
    assert _clip(max_norm=float("inf"))[0] in PASSED
    for kw in (dict(sizes=(-1, 7)), dict(sizes=(1 << 60, 7)), dict(types=(0, 2)), dict(scale=float("inf")),
               dict(max_norm=0.0), dict(max_norm=float("nan"))):
        assert _clip(**kw)[0] == SHAPE, kw
    assert _clip(ptrs=(None, _p(1)))[0] == NULL and _clip(outs=(None, _p(1)))[0] == NULL and _clip(ws=None)[0] == NULL
    assert _clip(ptrs=(_p(0, 2), _p(1)))[0] == ALIGN and _clip(norm=_p(2, 1))[0] == ALIGN and _clip(ws=_p(3, 8))[0] == ALIGN
    for kw in (dict(outs=(_p(0, 4), _p(5))), dict(outs=(_p(1), _p(5))), dict(outs=(_p(5), _p(5, 64))),
               dict(outs=(_p(1, 4), _p(0))), dict(outs=(_p(5), _p(0, 398))), dict(ptrs=(_p(0), _p(0))), dict(ptrs=(_p(0), _p(0, 396))),
               dict(ptrs=(_p(0, 4), _p(0)))):
        assert _clip(**kw)[0] == ALIAS, kw
    assert _clip(ptrs=(_p(0), _p(0)), outs=(_p(4), _p(5)))[0] in PASSED    # read twice, written apart
    assert _clip(ptrs=(_p(0), _p(0, 400)))[0] in PASSED                    # slices of one buffer
    g, _, s, t, n = _arrays((_p(0), _p(1)), None, (100, 7), (0, 1))
    need = L.lib().tpmlp_grad_workspace_bytes(s, n)
    assert _clip(n_ws=need)[0] in PASSED and _clip(n_ws=need - 1)[0] == WS
    lib = L.lib()
    assert lib.tpmlp_grad_sumsq(g, s, t, n, None, _p(3), need, None) == NULL
    assert lib.tpmlp_grad_sumsq(g, s, t, n, _p(4, 4), _p(3), need, None) == ALIGN
    assert lib.tpmlp_grad_clip(g, None, s, t, n, None, 1.0, 1.0, None, None) == NULL
    assert lib.tpmlp_grad_clip(g, None, s, t, -1, _p(4), 1.0, 1.0, None, None) == SHAPE
    assert lib.tpmlp_grad_clip(None, None, s, t, n, _p(4), 1.0, 1.0, None, None) == NULL
    assert lib.tpmlp_clip_grad_norm(None, None, None, None, 0, 1.0, 1.0, _p(2), _p(3), 1 << 20, None) in PASSED


def test_clip_overlaps_against_every_pair():
    """The merged walk over the addresses refuses exactly what comparing every pair refuses."""
    import random
    rng = random.Random(0)
    for _ in range(4000):
        n = rng.randint(1, 4)
        sizes = [rng.randint(0, 5) for _ in range(n)]
        at = lambda: _p(0, 4 * rng.randint(0, 24))  # noqa: E731
        grads = [at() for _ in range(n)]
        outs = [g if rng.random() < 0.4 else at() for g in grads]

        def meet(a, i, b, j):
            return sizes[i] and sizes[j] and a[i] < b[j] + 4 * sizes[j] and b[j] < a[i] + 4 * sizes[i]

        want = any(meet(outs, i, outs, j) for i in range(n) for j in range(i)) or \
            any(meet(outs, i, grads, j) and not (i == j and outs[i] == grads[i]) for i in range(n) for j in range(n))
        st = _clip(ptrs=grads, outs=outs, sizes=sizes, types=[0] * n)[0]
        assert (st == ALIAS) == bool(want), (grads, outs, sizes, st)


def test_python_checks():
    """The binding refuses tensors of the wrong type, shape or layout before it calls the
    library (CPU tensors; nothing reaches a kernel)."""
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    w = torch.ones(16)
    d = L.edge_desc(16, pre="rms", w_pre=w)
    r, x = torch.zeros(4, 16), torch.zeros(4, 16, dtype=bf)
    with pytest.raises(TypeError, match="one type"):
        L.edge_desc(16, post="rms", pre="rms", w_post=w, w_pre=w.to(bf))
    with pytest.raises(ValueError, match="expected 16"):
        L.edge_desc(16, pre="rms", w_pre=torch.ones(15))
    with pytest.raises(TypeError, match="x must be bf16"):
        L.tpmlp_edge_fwd(d, None, r, None, torch.zeros(4, 16), stream=0)
    with pytest.raises(TypeError, match="r_out must be float32"):
        L.tpmlp_edge_fwd(d, None, r, x, x, stream=0)
    with pytest.raises(ValueError, match="contiguous columns"):
        L.tpmlp_edge_fwd(d, None, torch.zeros(16, 4).t(), None, x, stream=0)
    with pytest.raises(ValueError, match="shape"):
        L.tpmlp_edge_fwd(d, torch.zeros(4, 8), r, None, x, stream=0)
    with pytest.raises(TypeError, match="y must be float32 or"):
        L.tpmlp_edge_fwd(d, torch.zeros(4, 16, dtype=torch.float16), r, None, x, stream=0)
    with pytest.raises(TypeError, match="ids"):
        L.tpmlp_route_sort(torch.zeros(4, 2), 4, 8, 0, None, None, None, None, stream=0)
    with pytest.raises(ValueError, match="outs"):
        L.GradTable([w], [])
    with pytest.raises(ValueError, match="type or size"):
        L.GradTable([w], [w.to(bf)])
    with pytest.raises(ValueError, match="contiguous"):
        L.GradTable([torch.zeros(4, 4).t()])
    with pytest.raises(TypeError, match="float32 or hold"):
        L.GradTable([torch.zeros(4, dtype=torch.float64)])


def test_rows_that_share_memory():
    """A broadcast tensor's rows lie on one another: its stride of 0 is not the 0 that stands for dense rows."""
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    d = L.edge_desc(16, pre="rms", w_pre=torch.ones(16))
    r, x = torch.zeros(4, 16), torch.zeros(4, 16, dtype=bf)
    wide, none = torch.zeros(1, 16).expand(4, 16), torch.zeros(0, 16)
    with pytest.raises(ValueError, match="rows of r .*stride"):
        L.tpmlp_edge_fwd(d, None, wide, None, x, stream=0)
    with pytest.raises(ValueError, match="rows of dr_out .*stride"):
        L.tpmlp_edge_bwd(d, None, r, wide, x, r.clone(), None, stream=0)
    with pytest.raises(ValueError, match="rows of dx .*stride"):
        L.tpmlp_edge_bwd(d, None, r, None, wide, r.clone(), None, stream=0)
    with pytest.raises(ValueError, match="rows of gate .*stride"):
        L.edge_desc(16, gate=wide, gate_rows=2)
    with pytest.raises(ValueError, match="rows of y .*stride"):
        L.tpmlp_edge_fwd(d, torch.zeros(40).as_strided((4, 16), (8, 1)), r, None, x, stream=0)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="rows of X .*stride"):
        L.tpmlp_route_dispatch(wide.to(bf)[:1].expand(4, 16), idx, torch.zeros(8, dtype=torch.int32), torch.zeros(8, 16, dtype=bf),
                               stream=0)
    with pytest.raises(ValueError, match="rows of dY .*stride"):
        L.tpmlp_route_combine_bwd(wide, torch.zeros(8, 16), idx, None, None, None, torch.zeros(4, 2), stream=0)
    assert L._rows(none, (0, 16), "r")[1] == 0 and L._rows(wide[:1], (1, 16), "r")[1] == 0  # no second row: any stride


def test_gate_rows_for_every_token():
    """A gate's rows times gate_rows cover the call's tokens, in both directions; and rows beyond the
    one that stands for all tokens need a gate_rows."""
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    gate = torch.ones(3, 16)
    for M, rows in ((13, 4), (4, 1), (7, 2)):
        d = L.edge_desc(16, gate=gate, gate_rows=rows)
        y, r = torch.zeros(M, 16), torch.zeros(M, 16)
        with pytest.raises(ValueError, match="gate has 3 rows"):
            L.tpmlp_edge_fwd(d, y, r, r, None, stream=0)
        with pytest.raises(ValueError, match="gate has 3 rows"):
            L.tpmlp_edge_bwd(d, y, None, r, None, r, torch.zeros(M, 16, dtype=bf), stream=0)
        y, r = y[:3 * rows], r[:3 * rows]  # as many as it covers
        with pytest.raises(L.TpmlpError, match="HIP|UNSUPPORTED"):  # every check passed
            L.tpmlp_edge_fwd(d, y, r, r, None, stream=0)
    d = L.edge_desc(16, gate=gate[0], gate_rows=2)
    with pytest.raises(ValueError, match="gate has 1 rows"):
        L.tpmlp_edge_fwd(d, torch.zeros(3, 16), torch.zeros(3, 16), torch.zeros(3, 16), None, stream=0)
    d = L.edge_desc(16, gate=gate[0])  # one row for all
    with pytest.raises(L.TpmlpError, match="HIP|UNSUPPORTED"):
        L.tpmlp_edge_fwd(d, torch.zeros(30, 16), torch.zeros(30, 16), torch.zeros(30, 16), None, stream=0)
    with pytest.raises(ValueError, match="gate_rows"):
        L.edge_desc(16, gate=gate)
    with pytest.raises(ValueError, match="gate_rows"):
        L.edge_desc(16, gate=gate, gate_rows=-1)


def test_clip_own_buffers_apart():
    """norm, sumsq and the workspace are disjoint from the gradients, the outputs and one another."""
    lib = L.lib()
    norm, ws = _p(2), _p(3)
    need = lib.tpmlp_grad_workspace_bytes(_arrays((0, 0), None, (100, 7), (0, 1))[2], 2)
    apart = dict(outs=(_p(4), _p(5)), norm=norm, ws=ws, n_ws=need)
    assert _clip(**apart)[0] in PASSED
    for kw in (dict(norm=_p(0, 396)), dict(norm=_p(1)), dict(norm=_p(4)), dict(norm=_p(5, 12)), dict(norm=ws), dict(norm=_p(3, need - 4)),
               dict(ws=_p(0, 384)), dict(ws=_p(1)), dict(ws=_p(4, 16)), dict(ws=_p(5)), dict(ws=norm)):
        st, text = _clip(**{**apart, **kw})
        assert st == ALIAS and "overlaps" in text, (kw, st, text)
    for kw in (dict(norm=_p(0, 400)), dict(norm=_p(4, -4)), dict(norm=_p(3, need)), dict(ws=_p(0, 400)), dict(n_ws=1 << 40),
               dict(norm=None)):
        assert _clip(**{**apart, **kw})[0] in PASSED, kw
    g, o, s, t, n = _arrays((_p(0), _p(1)), (_p(4), _p(5)), (100, 7), (0, 1))
    for sumsq, w in ((_p(0, 392), ws), (_p(1, 8), ws), (_p(3, 0), ws), (_p(6), _p(0)), (_p(3, need - 8), ws)):
        assert lib.tpmlp_grad_sumsq(g, s, t, n, sumsq, w, need, None) == ALIAS, (hex(sumsq), hex(w))
    assert lib.tpmlp_grad_sumsq(g, s, t, n, _p(3, need), ws, need, None) in PASSED
    for sumsq, nm in ((_p(6), _p(6)), (_p(6), _p(6, 4)), (_p(4, 8), norm), (_p(5, 8), None), (_p(6), _p(0)), (_p(6), _p(5))):
        assert lib.tpmlp_grad_clip(g, o, s, t, n, sumsq, 1.0, 1.0, nm, None) == ALIAS, (hex(sumsq), nm)
    assert lib.tpmlp_grad_clip(g, o, s, t, n, _p(6), 1.0, 1.0, _p(6, 8), None) in PASSED
    assert lib.tpmlp_grad_clip(g, o, s, t, n, _p(0), 1.0, 1.0, norm, None) in PASSED  # only read, as the gradient is
    assert lib.tpmlp_grad_clip(g, None, s, t, n, _p(0), 1.0, 1.0, norm, None) == ALIAS


def test_edge_keeps_what_a_graph_writes_to(monkeypatch):
    """Another M replaces the gate's gradient and the workspace; those that a captured backward
    writes to stay allocated, others do not."""
    torch = pytest.importorskip("torch")
    import weakref
    from tensor_transformer_mlp_03_amd import block
    bf, used = torch.bfloat16, []
    monkeypatch.setattr(L, "tpmlp_edge_bwd", lambda d, *a, **k: used.append([weakref.ref(t) for t in (k["ws"], k["dgate"])]))
    for capturing in (False, True):
        monkeypatch.setattr(block, "_capturing", lambda: capturing, raising=False)
        edge = block.Edge(16, post="rms", w_post=torch.ones(16), gate=torch.ones(500, 16), gate_rows=2)
        for M in (8, 1000, 6):
            r = torch.zeros(M, 16)
            g = edge.backward(r, None, r, None, r, torch.zeros(M, 16, dtype=bf))
            first = g if M == 8 else first
        assert first["gate"].shape == (4, 16) and g["gate"].shape == (3, 16)  # a caller's dict stays that call's
        del first, g
        alive = [[t() is not None for t in refs] for refs in used]
        used.clear()
        # The largest workspace and the last gradient are the object's own.
        assert alive == ([[True, True]] * 3 if capturing else [[False, False], [True, False], [True, True]]), (capturing, alive)


def test_edge_call_keeps_its_own_sizes(monkeypatch):
    """The library is entered without the interpreter's lock: another thread's call through the same description,
    at any point of this one, changes neither its M nor its types."""
    torch = pytest.importorskip("torch")
    bf, seen, d = torch.bfloat16, [], L.edge_desc(16, pre="rms", w_pre=torch.ones(16), gate=torch.ones(16))

    def fwd(M, dtype):
        r = torch.zeros(M, 16, dtype=dtype)
        L.tpmlp_edge_fwd(d, r.clone(), r, r.clone(), torch.zeros(M, 16, dtype=bf), stream=0)

    def bwd(M, dtype):
        r = torch.zeros(M, 16, dtype=dtype)
        L.tpmlp_edge_bwd(d, r.clone(), r, r, r, r.clone(), torch.zeros(M, 16, dtype=bf), stream=0)

    def query(M, dtype):
        assert L.tpmlp_edge_bwd_workspace_bytes(d, M) == 0

    class Library:
        other, depth = None, 0

        def enter(self, ref, *_):
            Library.depth += 1
            if Library.depth == 1:  # the other thread's turn
                Library.other(4096, bf)
            e = ref._obj
            seen.append((e.M, e.r_type, e.y_type, e.H, e.gate))
            Library.depth -= 1
            return 0

        tpmlp_edge_fwd = tpmlp_edge_bwd = tpmlp_edge_bwd_workspace_bytes = enter

    monkeypatch.setattr(L, "lib", lambda: Library())
    for call in (fwd, bwd, query):
        for Library.other in (fwd, bwd, query):
            seen.clear()
            call(8, torch.float32)
            (M, r, y, H, gate), outer = seen
            assert M == 4096 and outer[0] == 8 and outer[3:] == (H, gate) == (16, d.gate), (seen, call)
            if call is not query:
                assert outer[1:3] == (L.F32, L.F32), (seen, call)


def test_edge_places_buffers_on_the_stream_of_the_call(monkeypatch):
    """What a backward allocates and lets go belongs to the stream that its kernels run on, and that stream is the
    one asked whether it is being captured."""
    torch = pytest.importorskip("torch")
    from tensor_transformer_mlp_03_amd import block
    current, asked, made = ["current"], [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    def capturing():
        asked.append(current[-1])
        return current[-1] == 77

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(current[-1]) or empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(block, "_capturing", capturing)
    monkeypatch.setattr(L, "tpmlp_edge_bwd", lambda *a, **k: None)
    for stream, name in ((77, 77), (0, "default"), (None, "current")):
        edge = block.Edge(16, post="rms", w_post=torch.ones(16), gate=torch.ones(500, 16), gate_rows=2)
        for M in (8, 1000):
            r = torch.zeros(M, 16)
            made.clear(), asked.clear()
            edge.backward(r, None, r, None, r, torch.zeros(M, 16, dtype=torch.bfloat16), stream=stream)
            assert set(made) == {name} and asked == [name], (stream, made, asked)
        assert bool(edge._captured) == (stream == 77)


def test_edge_keeps_captured_buffers_once(monkeypatch):
    """Captures over the same buffers hold them, not a note of each capture."""
    torch = pytest.importorskip("torch")
    from tensor_transformer_mlp_03_amd import block
    monkeypatch.setattr(block, "_capturing", lambda: True)
    monkeypatch.setattr(L, "tpmlp_edge_bwd", lambda *a, **k: None)
    edge = block.Edge(16, post="rms", w_post=torch.ones(16))
    for M in (1000, 8, 1000, 8, 8):
        r = torch.zeros(M, 16)
        edge.backward(r, None, r, None, r, torch.zeros(M, 16, dtype=torch.bfloat16))
    assert len(edge._captured) == 2  # w_post's gradient and the larger workspace


def test_host_tensors_are_refused(monkeypatch):
    """Where there is a GPU, a tensor in host memory is refused by name: its address would fault in a kernel."""
    torch = pytest.importorskip("torch")
    i32, bf, called = torch.int32, torch.bfloat16, []

    class Library:
        def __getattr__(self, name):
            if name == "tpmlp_route_rows":
                return lambda *a: 8
            return lambda *a: called.append(name) or 0

    class OnGpu(torch.Tensor):  # a host tensor that says it is not
        is_cuda = True

    def gpu(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)

    monkeypatch.setattr(L, "lib", lambda: Library())
    monkeypatch.setattr(L, "_gpu_here", lambda: True, raising=False)
    d = L.edge_desc(16, post="rms", pre="rms", w_post=gpu(16), w_pre=gpu(16), gate=gpu(1, 16))

    def each(call, **tensors):
        call(**tensors)
        assert called.pop() and not called
        for name, t in tensors.items():
            host = [t[0].as_subclass(torch.Tensor)] if isinstance(t, list) else t.as_subclass(torch.Tensor)
            with pytest.raises(ValueError, match="not on the GPU"):
                call(**{**tensors, name: host})
            assert not called, (call, name)

    s = dict(stream=0)
    each(lambda **k: L.edge_desc(16, post="layer", **k) and called.append(1), w_post=gpu(16), b_post=gpu(16), gate=gpu(1, 16))
    each(lambda **k: L.tpmlp_edge_fwd(d, **k, **s), y=gpu(4, 16), r=gpu(4, 16), r_out=gpu(4, 16), x=gpu(4, 16, dtype=bf))
    each(lambda **k: L.tpmlp_edge_bwd(d, **k, **s), y=gpu(4, 16), r_out=gpu(4, 16), dr_out=gpu(4, 16), dx=gpu(4, 16), dr=gpu(4, 16),
         dy=gpu(4, 16, dtype=bf), dw_post=gpu(16), dw_pre=gpu(16), dgate=gpu(1, 16), ws=gpu(64))
    ids, rows = gpu(4, 2, dtype=i32), gpu(8, dtype=i32)
    each(lambda **k: L.tpmlp_route_sort(E=4, align=1, capacity=0, **k, **s), ids=ids, counts=gpu(4, dtype=i32),
         offsets=gpu(5, dtype=i32), row_of=ids, src_of=rows, ws=gpu(64))
    each(lambda **k: L.tpmlp_route_dispatch(**k, **s), X=gpu(4, 16, dtype=bf), row_of=ids, src_of=rows, Xs=gpu(8, 16, dtype=bf))
    each(lambda **k: L.tpmlp_route_combine(**k, **s), Zs=gpu(8, 16), row_of=ids, w=gpu(4, 2), Y=gpu(4, 16))
    each(lambda **k: L.tpmlp_route_combine_bwd(**k, **s), dY=gpu(4, 16), Zs=gpu(8, 16), row_of=ids, src_of=rows, w=gpu(4, 2),
         dZs=gpu(8, 16, dtype=bf), dw=gpu(4, 2))
    each(lambda **k: L.GradTable(**k) and called.append(1), grads=[gpu(5)], outs=[gpu(5)])
    table, one = L.GradTable([gpu(5)]), gpu(1, dtype=torch.float64)
    each(lambda **k: L.tpmlp_grad_sumsq(table, **k, **s), sumsq=one, ws=gpu(64))
    each(lambda **k: L.tpmlp_grad_clip(table, max_norm=1.0, **k, **s), sumsq=one, norm=gpu(1))
    each(lambda **k: L.tpmlp_clip_grad_norm(table, 1.0, **k, **s), norm=gpu(1), ws=gpu(64))
