"""The block operators' kernels against the float64 oracle (oracle/block.py).

Tolerances.  An output's error is its last rounding, half a step of its type relative to the
value, plus what float32 evaluation loses: at most a number of roundings, counted below, times
2^-24 times the output's magnitude (the same expression with every term positive).

* A row's sum of squares: at most 32 elements in a lane one after another, 4 part sums, 6
  levels over the wave and 16 waves, under 64 roundings; half of that in 1 / deviation, 64 in
  a mean, and under 16 element-wise: r' within 100, and x, whose row is r', within 200.
* Backward: d within 200 and dy, which goes through the second norm, within 400.  A column
  sum adds at most M rows: within 450 + M.
* combine: K products and K sums, 2 K.  dw: H / 1024 steps of 4 in a lane, then 8 levels: H / 256 + 16.
* clip: the norm in float64, rounded once; a factor rounded once and a product: 2 and 4.
"""
import sys

import numpy as np
import pytest

from oracle import block as OB

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16
U = OB.U


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tensor_transformer_mlp_03_amd import _lib as L
    L.lib()


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"[case] {request.node.name}", flush=True)
    sys.stdout.flush()


def f64(t):
    return t.detach().cpu().double().numpy()


def close(name, got, want, mag, roundings, rows=None):
    """|got - want| <= half a step of got's type at want + roundings * 2^-24 * mag."""
    half = torch.finfo(got.dtype).eps / 2
    g = f64(got)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    tol = half * np.abs(want) + (1 + half) * roundings * U * np.abs(mag) + 1e-37
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / tol, 0)), g.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {g.size} off; at {i}: {g[i]!r} want {want[i]!r} tol {tol[i]!r}")


class Strided:
    """A [M,H] view with row stride ld at an element offset, in a buffer whose other elements
    hold a NaN that no call may change."""

    def __init__(self, M, H, dtype, ld=None, offset=0, fill=None):
        ld = H if ld is None else ld
        self.flat = torch.full((offset + M * ld + 64,), float("nan"), dtype=dtype, device="cuda")
        self.view = self.flat.as_strided((M, H), (ld, 1), offset)
        if fill is not None:
            self.view.copy_(fill)

    def untouched(self):
        rest = self.flat.clone()
        M, H = self.view.shape
        rest.as_strided((M, H), self.view.stride(), self.view.storage_offset()).fill_(float("nan"))
        return bool(torch.isnan(rest).all())


def normal(gen, *shape, dtype=F32, scale=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * scale + mean).to(dtype)


def edge_case(seed, M, H, post, pre, y, r, p, rows, **over):
    gen = torch.Generator().manual_seed(seed)
    c = dict(post=post, pre=pre, alpha=0.75, eps=1e-5)
    c.update(over)
    params = {}
    for side in ("post", "pre"):
        if c[side] != "none":
            params["w_" + side] = normal(gen, H, dtype=p, scale=0.2, mean=1.0)
        if c[side] == "layer":
            params["b_" + side] = normal(gen, H, dtype=p, scale=0.2)
    if rows:
        params["gate"] = normal(gen, max(1, -(-M // rows)), H, dtype=p, scale=0.3, mean=0.5)
    t = dict(y=normal(gen, M, H, dtype=y, mean=0.3) if y else None, r=normal(gen, M, H, dtype=r, scale=2.0, mean=-0.5),
             dr=normal(gen, M, H, dtype=r), dx=normal(gen, M, H, dtype=F32 if seed % 2 else BF16))
    return c, params, t


def make_edge(c, params, H, rows):
    from tensor_transformer_mlp_03_amd.block import Edge
    return Edge(H, **c, **{k: v.cuda() for k, v in params.items()}, gate_rows=rows)


def run_edge(seed, M, H, post, pre, y, r, p, rows, pad=0, offset=0, **over):
    c, params, t = edge_case(seed, M, H, post, pre, y, r, p, rows, **over)
    e = make_edge(c, params, H, rows)
    P = {k: f64(v) for k, v in params.items()}
    kw = dict(c, rows=rows or M, **P)
    n64 = lambda v: None if v is None else f64(v)  # noqa: E731
    ld = H + pad

    def put(v):
        return None if v is None else Strided(M, H, v.dtype, ld, offset, v).view

    want = OB.edge_forward(n64(t["y"]), n64(t["r"]), **kw)
    yd, rd = put(t["y"]), put(t["r"])
    ro, x = Strided(M, H, r, ld, offset), Strided(M, H, BF16, ld, offset)
    e.forward(yd, rd, ro.view, x.view if pre != "none" else None)
    torch.cuda.synchronize()
    close("r'", ro.view, want["r"], want["r_mag"], 100)
    if pre != "none":
        close("x", x.view, want["x"], want["x_mag"], 200)
        assert x.untouched()
    assert ro.untouched()

    # backward, from the stream as it was stored
    has_x = pre != "none"
    back = OB.edge_backward(n64(t["y"]), f64(ro.view), n64(t["dr"]), n64(t["dx"]) if has_x else None, **kw)
    dr, dy = Strided(M, H, r, ld, offset), Strided(M, H, BF16, ld, offset)
    g = e.backward(yd, ro.view if has_x else None, put(t["dr"]), put(t["dx"]) if has_x else None, dr.view,
                   dy.view if y else None)
    torch.cuda.synchronize()
    close("dr", dr.view, back["dr"], back["dr_mag"], 200)
    if y:
        close("dy", dy.view, back["dy"], back["dy_mag"], 400)
    assert dr.untouched() and dy.untouched()
    assert set(g) == set(params)
    for k in params:
        close("d" + k, g[k], back[k], back[k + "_mag"], 450 + M)


SIZES = [(1, 8), (3, 9), (5, 13), (4, 64), (9, 255), (6, 256), (7, 257), (5, 260), (33, 511), (2, 512), (6, 513), (130, 1000), (9, 1024), (5, 1025),
         (3, 2048), (4, 2050), (21, 3584), (3, 4096), (3, 4100), (2, 8192), (3, 8200), (3, 8196), (2, 8195), (2, 16384), (2, 16392), (3, 20480),
         (2, 20483), (2, 32768)]


@pytest.mark.parametrize("M,H", SIZES)
def test_edge_sizes(M, H):
    """Every row form of the kernels, whole and ragged, RMSNorm and LayerNorm."""
    run_edge(1 + H, M, H, "rms", "rms", F32, BF16, BF16, M)
    run_edge(2 + H, M, H, "layer", "layer", BF16, F32, F32, 2)


KINDS = [("none", "rms"), ("none", "layer"), ("rms", "none"), ("layer", "none"), ("none", "none"), ("rms", "layer"),
         ("layer", "rms")]


@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("rows", [0, 1, 3, 1000])
def test_edge_norms_and_gates(post, pre, rows):
    """Every pair of norms with no gate, one per token, per 3 tokens (the last group short), and one for all."""
    run_edge(5, 10, 200, post, pre, F32, F32, BF16, rows)
    run_edge(8, 10, 1400, post, pre, BF16, BF16, F32, rows)


@pytest.mark.parametrize("y", [None, F32, BF16])
@pytest.mark.parametrize("r", [F32, BF16])
@pytest.mark.parametrize("p", [F32, BF16])
def test_edge_types_and_strides(y, r, p):
    """Every type, with odd strides and addresses that only their elements are aligned to."""
    post = "rms" if y else "none"
    run_edge(3, 6, 331, post, "rms", y, r, p, 2 if y else 0, pad=5, offset=1)
    run_edge(4, 5, 1336, "layer" if y else "none", "layer", y, r, p, 0, pad=24, offset=8)


@pytest.mark.parametrize("rows", [64, 100, 7])
def test_edge_many_rows(rows):
    """More rows than workgroups hold at once, many gate groups and uneven chunks."""
    run_edge(6, 1500, 96, "rms", "rms", F32, F32, F32, rows)
    run_edge(7, 700, 1100, "layer", "layer", F32, BF16, BF16, rows)


def test_edge_no_tokens():
    c, params, _ = edge_case(1, 0, 64, "layer", "rms", F32, F32, F32, 4)
    e = make_edge(c, params, 64, 4)
    z = lambda d: torch.empty(0, 64, dtype=d, device="cuda")  # noqa: E731
    e.forward(z(F32), z(F32), z(F32), z(BF16))
    g = e.backward(z(F32), z(F32), z(F32), z(F32), z(F32), z(BF16))
    torch.cuda.synchronize()
    assert g["gate"].shape == (0, 64)
    for k in ("w_post", "b_post", "w_pre"):
        assert float(g[k].abs().max()) == 0.0, k


def test_edge_in_place():
    """r_out over r and dr over dr_out give the bits of separate buffers."""
    for H in (96, 2056):
        c, params, t = edge_case(2, 9, H, "rms", "layer", F32, F32, F32, 9)
        e = make_edge(c, params, H, 9)
        y, r = t["y"].cuda(), t["r"].cuda()
        ro, x, x2 = torch.empty_like(r), torch.empty(9, H, dtype=BF16, device="cuda"), torch.empty(9, H, dtype=BF16, device="cuda")
        e.forward(y, r, ro, x)
        e.forward(y, r, r, x2)
        assert torch.equal(r, ro) and torch.equal(x, x2)
        d, dx = t["dr"].cuda(), t["dx"].cuda()
        dr, dy, dy2 = torch.empty_like(d), torch.empty_like(x), torch.empty_like(x)
        g = {k: v.clone() for k, v in e.backward(y, ro, d, dx, dr, dy).items()}
        g2 = e.backward(y, ro, d, dx, d, dy2)
        assert torch.equal(d, dr) and torch.equal(dy, dy2)
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_edge_only_x_and_no_later_gradient():
    """r_out is not wanted; dr_out None stands for zeros."""
    c, params, t = edge_case(4, 6, 520, "rms", "rms", F32, BF16, BF16, 6)
    e = make_edge(c, params, 520, 6)
    y, r = t["y"].cuda(), t["r"].cuda()
    ro, x, x2 = torch.empty_like(r), torch.empty(6, 520, dtype=BF16, device="cuda"), torch.empty(6, 520, dtype=BF16, device="cuda")
    e.forward(y, r, ro, x)
    e.forward(y, r, None, x2)
    assert torch.equal(x, x2)
    outs = [(torch.empty_like(r), torch.empty_like(x)) for _ in range(2)]
    e.backward(y, ro, None, t["dx"].cuda(), *outs[0])
    e.backward(y, ro, torch.zeros_like(r), t["dx"].cuda(), *outs[1])
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_edge_bad_rows_stay_alone():
    """A row of NaN, of infinities or of zeros changes no other row."""
    for H in (200, 2050):
        c, params, t = edge_case(3, 8, H, "rms", "layer", F32, F32, F32, 0)
        e = make_edge(c, params, H, 0)
        y, r = t["y"].cuda(), t["r"].cuda()
        ro, x = torch.empty_like(r), torch.empty(8, H, dtype=BF16, device="cuda")
        e.forward(y, r, ro, x)
        y2, r2 = y.clone(), r.clone()
        y2[1], y2[3], y2[5], r2[5], r2[6, 7] = float("nan"), float("inf"), 0.0, 0.0, float("inf")
        ro2, x2 = torch.empty_like(ro), torch.empty_like(x)
        e.forward(y2, r2, ro2, x2)
        keep = [0, 2, 4, 7]
        assert torch.equal(ro[keep], ro2[keep]) and torch.equal(x[keep], x2[keep])
        assert bool(torch.isfinite(x2[5]).all()) and bool(torch.isnan(x2[1]).all())


def test_edge_infinite_y_without_a_norm():
    """dy = gate * d has no part of y where no norm follows the block."""
    for H in (64, 1000, 20480, 20001):
        c, params, t = edge_case(5, 3, H, "none", "rms", F32, F32, F32, 3)
        e = make_edge(c, params, H, 3)
        y = t["y"].cuda()
        ro, x = torch.empty(3, H, device="cuda"), torch.empty(3, H, dtype=BF16, device="cuda")
        e.forward(y, t["r"].cuda(), ro, x)
        outs = []
        for bad in (False, True):
            if bad:
                y[1, 5], y[2, 6] = float("inf"), float("nan")
            dr, dy = torch.empty_like(ro), torch.empty_like(x)
            e.backward(y, ro, t["dr"].cuda(), t["dx"].cuda(), dr, dy)
            outs.append((dr, dy))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1]), H


def test_edge_more_rows_than_one_launch():
    """2^21 rows go into one launch."""
    M, H = (1 << 21) + 3, 8
    c, params, _ = edge_case(5, 1, H, "rms", "rms", BF16, BF16, F32, 0)
    e = make_edge(c, params, H, 0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    y, r = (torch.randn(M, H, generator=gen, device="cuda").to(BF16) for _ in range(2))
    ro, x = torch.empty_like(r), torch.empty_like(r)
    e.forward(y, r, ro, x)
    part_r, part_x = torch.empty(5, H, dtype=BF16, device="cuda"), torch.empty(5, H, dtype=BF16, device="cuda")
    for at in (0, (1 << 21) - 2):
        e.forward(y[at:at + 5], r[at:at + 5], part_r, part_x)
        assert torch.equal(ro[at:at + 5], part_r) and torch.equal(x[at:at + 5], part_x)
    assert bool(torch.isfinite(x).all())


def test_edge_large_values():
    """A LayerNorm of values far from zero keeps its variance."""
    H = 1000
    c, params, t = edge_case(9, 4, H, "none", "layer", F32, F32, F32, 0)
    e = make_edge(c, params, H, 0)
    r = t["r"] + 3000.0
    want = OB.edge_forward(f64(t["y"]), f64(r), **c, rows=4, **{k: f64(v) for k, v in params.items()})
    ro, x = torch.empty(4, H, device="cuda"), torch.empty(4, H, dtype=BF16, device="cuda")
    e.forward(t["y"].cuda(), r.cuda(), ro, x)
    close("x", x, want["x"], want["x_mag"], 200)


def test_edge_gradient_is_a_difference():
    """<dr', r'> + <dx, x> moves along a direction of y as <dy, direction> says: central
    differences of the kernel's own forward in float32.  x is bf16, so its part is left out
    (no norm before the next block); the step's error is the float32 rounding of r', at most
    100 roundings of its magnitude, over the step, and the third-order term, of the order of
    the step squared."""
    M, H, h = 4, 256, 2.0 ** -6
    c, params, t = edge_case(12, M, H, "layer", "none", F32, F32, F32, 2, alpha=0.0)
    e = make_edge(c, params, H, 2)
    gen = torch.Generator().manual_seed(1)
    u = normal(gen, M, H).cuda()
    y, r, d = t["y"].cuda(), t["r"].cuda(), t["dr"].cuda()
    f = []
    for s in (h, -h):
        ro = torch.empty_like(r)
        e.forward(y + s * u, r, ro, None)
        f.append(float((ro.double() * d.double()).sum()))
    dr, dy = torch.empty_like(d), torch.empty(M, H, dtype=BF16, device="cuda")
    e.backward(y, None, d, None, dr, dy)
    got = float((dy.double() * u.double()).sum())
    mag = float((d.double().abs() * 2).sum())
    tol = 100 * U * mag / h + 2.0 ** -8 * float((dy.double() * u.double()).abs().sum()) + 8 * h * h * mag / np.sqrt(M * H)
    assert abs(got - (f[0] - f[1]) / (2 * h)) <= tol


def test_edge_offsets_past_32_bits():
    """Rows 2^31 elements apart."""
    H, ld = 136, 1 << 31
    c, params, t = edge_case(5, 3, H, "none", "rms", F32, BF16, F32, 0)
    flat = torch.empty(2 * ld + H, dtype=BF16, device="cuda")
    r = flat.as_strided((3, H), (ld, 1))
    r.copy_(t["r"])
    e = make_edge(c, params, H, 0)
    y = t["y"].cuda()
    x, x2 = torch.empty(3, H, dtype=BF16, device="cuda"), torch.empty(3, H, dtype=BF16, device="cuda")
    ro = torch.empty(3, H, dtype=BF16, device="cuda")
    e.forward(y, t["r"].cuda(), ro, x)
    e.forward(y, r, r, x2)
    assert torch.equal(x, x2) and torch.equal(r.clone(), ro)
    d, dx = t["dr"].cuda(), t["dx"].cuda()
    a, b = [(torch.empty_like(d), torch.empty_like(x)) for _ in range(2)]
    e.backward(y, ro, d, dx, *a)
    e.backward(y, r, d, dx, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# --- route -----------------------------------------------------------------------------------------------------
def route_ids(seed, T, K, E, drop=0.0, bad=False):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, K), generator=gen)
    off = torch.rand(T, K, generator=gen) < drop
    ids[off] = -1
    if bad and T:
        ids[0, 0], ids[-1, -1] = E, -(1 << 30)
    return ids


def check_sort(ids, E, align, capacity, dtype):
    from tensor_transformer_mlp_03_amd.block import Route
    T, K = ids.shape
    want = OB.route_sort(ids.numpy(), E, align, capacity)
    h = Route(T, K, E, align, capacity)
    assert h.rows == OB.route_rows(T, K, E, align, capacity)
    for t in (h.counts, h.offsets, h.row_of, h.src_of):
        t.fill_(-77)
    h.sort(ids.to(dtype).cuda())
    torch.cuda.synchronize()
    for name, w in zip(("counts", "offsets", "row_of", "src_of"), want):
        got = getattr(h, name).cpu().numpy()
        assert np.array_equal(got, w), (name, np.argwhere(got != w)[:5].tolist())
    return h


@pytest.mark.parametrize("T,K", [(0, 1), (1, 1), (1, 8), (7, 3), (63, 1), (64, 2), (65, 5), (1000, 4), (4096, 1),
                                 (4097, 1), (2500, 7), (70000, 2)])
@pytest.mark.parametrize("E", [1, 3, 8, 64, 65, 512])
def test_route_sort(T, K, E):
    check_sort(route_ids(T + E, T, K, E, 0.1, bad=T > 4), E, 8, 0, torch.int32)
    check_sort(route_ids(T + E, T, K, E), E, 1, 0, torch.int64)
    cap = -(-T * K // (2 * E)) // 8 * 8 + 8
    check_sort(route_ids(T + E, T, K, E, 0.1), E, 8, cap, torch.int64)


def test_route_sort_many_pairs():
    """More pairs than 256 workgroups of 2048: every expert's rows hold its pairs, in their order."""
    from tensor_transformer_mlp_03_amd.block import Route
    T, K, E = 300007, 2, 60
    ids = route_ids(4, T, K, E, 0.1).cuda()
    h = Route(T, K, E)
    h.sort(ids)
    flat = ids.reshape(-1)
    on = flat >= 0
    assert torch.equal(h.counts.long(), torch.bincount(flat[on], minlength=E))
    rows = h.row_of.reshape(-1).long()
    assert bool(((rows >= 0) == on).all())
    pairs = torch.arange(T * K, device="cuda")
    assert torch.equal(h.src_of.long()[rows[on]], pairs[on])
    assert int((h.src_of >= 0).sum()) == int(on.sum())
    order = torch.sort(torch.where(on, flat, E), stable=True).indices[:int(on.sum())]
    assert torch.equal(h.src_of[h.src_of >= 0].long(), order)


def test_route_sort_one_sided():
    """Every pair to one expert, no pair to any, and the smallest and the largest expert only."""
    for T in (100, 9000):
        for v in (0, 5, 31, -1, 32):
            check_sort(torch.full((T, 2), v), 32, 16, 0, torch.int32)
            check_sort(torch.full((T, 2), v), 32, 16, 48, torch.int32)


def put(v, pad=0, offset=0):
    return Strided(v.shape[0], v.shape[1], v.dtype, v.shape[1] + pad, offset, v).view


@pytest.mark.parametrize("T,K,E,H,capacity", [(1, 1, 4, 8, 0), (5, 2, 8, 9, 0), (33, 3, 7, 331, 0), (8, 2, 8, 4096, 0),
                                              (200, 8, 16, 512, 64), (77, 9, 60, 2049, 0), (300, 1, 1, 1032, 0),
                                              (50, 20, 64, 136, 8), (10, 4, 512, 5000, 0),
                                              (40, 5, 8, 72, 0), (40, 12, 8, 255, 0), (33, 2, 4, 256, 16),
                                              (90, 3, 4, 8, 0), (2100, 2, 4, 264, 0), (60, 64, 32, 16, 0)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_route_moves(T, K, E, H, capacity, pad, offset):
    """There and back, both gradients; dropped pairs and padding rows hold NaN where they are read."""
    gen = torch.Generator().manual_seed(T * 7 + H)
    h = check_sort(route_ids(T, T, K, E, 0.15), E, 8, capacity, torch.int32)
    row_of, src_of = h.row_of.cpu().numpy(), h.src_of.cpu().numpy()
    X = normal(gen, T, H, dtype=BF16)
    Xs = Strided(h.rows, H, BF16, H + pad, offset)
    h.dispatch(put(X, pad, offset), Xs.view)
    assert np.array_equal(f64(Xs.view), OB.route_dispatch(f64(X), row_of, h.rows)) and Xs.untouched()
    w = torch.rand(T, K, generator=gen)
    w[torch.from_numpy(row_of) < 0] = float("nan")  # of a pair that takes no part
    w64 = np.where(row_of >= 0, f64(w), 0.0)
    for zt in (F32, BF16):
        for yt in (F32, BF16):
            Z = normal(gen, h.rows, H, dtype=zt)
            Z64 = f64(Z)
            Z[torch.from_numpy(src_of) < 0] = float("nan")
            for ww, w_ in ((w, w64), (None, None)):
                Y = Strided(T, H, yt, H + pad, offset)
                h.combine(put(Z, pad, offset), None if ww is None else ww.cuda(), Y.view)
                want, mag = OB.route_combine(Z64, row_of, w_)
                close("Y", Y.view, want, mag, 2 * K)
                assert Y.untouched()
            dY = normal(gen, T, H, dtype=yt)
            dZs, dw = Strided(h.rows, H, BF16, H + pad, offset), torch.full((T, K), float("nan"), device="cuda")
            h.combine_backward(put(dY, pad, offset), put(Z, pad, offset), w.cuda(), dZs.view, dw)
            wz, ww_, mag = OB.route_combine_backward(f64(dY), Z64, row_of, w64, h.rows)
            close("dZs", dZs.view, wz, np.abs(wz), 1)
            close("dw", dw, ww_, mag, H / 256 + 16)
            assert dZs.untouched()
            # one of the two alone
            a, b = torch.empty(h.rows, H, dtype=BF16, device="cuda"), torch.empty(T, K, device="cuda")
            h.combine_backward(dY.cuda(), None, w.cuda(), a, None)
            from tensor_transformer_mlp_03_amd import _lib as L
            L.tpmlp_route_combine_bwd(dY.cuda(), Z.cuda(), h.row_of, None, w.cuda(), None, b)
            assert torch.equal(a, dZs.view) and torch.equal(b, dw)
    dXs = normal(gen, h.rows, H)
    dX = Strided(T, H, F32, H + pad, offset)
    h.dispatch_backward(put(dXs, pad, offset), dX.view)
    want, mag = OB.route_combine(f64(dXs), row_of, None)
    close("dX", dX.view, want, mag, 2 * K)


def test_route_no_tokens_and_all_dropped():
    from tensor_transformer_mlp_03_amd.block import Route
    h = Route(0, 2, 4, capacity=8)
    h.sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    Xs = torch.full((32, 64), 3.0, dtype=BF16, device="cuda")
    h.dispatch(torch.empty(0, 64, dtype=BF16, device="cuda"), Xs)
    assert float(Xs.abs().max()) == 0.0
    h = Route(6, 2, 4)
    h.sort(torch.full((6, 2), -1, dtype=torch.int64, device="cuda"))
    Z, Y = torch.full((h.rows, 64), float("nan"), device="cuda"), torch.full((6, 64), 5.0, device="cuda")
    h.combine(Z, torch.ones(6, 2, device="cuda"), Y)
    assert float(Y.abs().max()) == 0.0
    dZs, dw = torch.full((h.rows, 64), 2.0, dtype=BF16, device="cuda"), torch.full((6, 2), 2.0, device="cuda")
    h.combine_backward(Y + 1, Z, torch.ones(6, 2, device="cuda"), dZs, dw)
    assert float(dZs.abs().max()) == 0.0 and float(dw.abs().max()) == 0.0


def test_route_rows_out_of_range_are_dropped():
    """row_of entries outside the sorted buffer (not the sort's) are treated as dropped: no
    access, zeros in their place."""
    from tensor_transformer_mlp_03_amd import _lib as L
    row_of = torch.tensor([[0, 99], [-5, 1], [2 ** 31 - 1, -(2 ** 31)]], dtype=torch.int32, device="cuda")
    src_of = torch.tensor([0, 3, -1, -1], dtype=torch.int32, device="cuda")
    X = torch.arange(3 * 64, device="cuda").reshape(3, 64).to(BF16)
    Xs = torch.full((4, 64), 7.0, dtype=BF16, device="cuda")
    L.tpmlp_route_dispatch(X, row_of, src_of, Xs)
    assert torch.equal(Xs[0], X[0]) and torch.equal(Xs[1], X[1]) and float(Xs[2:].abs().max()) == 0.0
    Y = torch.empty(3, 64, device="cuda")
    L.tpmlp_route_combine(Xs, row_of, None, Y)
    assert torch.equal(Y[:2], X[:2].float()) and float(Y[2].abs().max()) == 0.0


def test_route_offsets_past_32_bits():
    from tensor_transformer_mlp_03_amd.block import Route
    H, ld = 72, 1 << 30
    h = Route(3, 1, 1, align=1)
    h.sort(torch.zeros(3, 1, dtype=torch.int32, device="cuda"))
    Xs = torch.empty(2 * ld + H, dtype=BF16, device="cuda").as_strided((3, H), (ld, 1))
    X = normal(torch.Generator().manual_seed(1), 3, H, dtype=BF16).cuda()
    h.dispatch(X, Xs)
    assert torch.equal(Xs.clone(), X)
    Y = torch.empty(3, H, dtype=BF16, device="cuda")
    h.combine(Xs, None, Y)
    assert torch.equal(Y, X)


# --- clipping ----------------------------------------------------------------------------------------------------
def grads_of(seed, sizes, kinds, offset=0, scale=0.1):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for n, k in zip(sizes, kinds):
        flat = torch.full((n + offset + 8,), float("nan"), dtype=k, device="cuda")
        flat[offset:offset + n] = normal(gen, n, dtype=k, scale=scale).cuda()
        out.append(flat)
    return out, [f[offset:offset + n] for f, n in zip(out, sizes)]


SIZE_SETS = {
    "one": [1], "odd": [1, 2, 3, 5, 1023, 1025, 4097], "chunks": [16383, 16384, 16385, 32768, 40000],
    "empty": [0, 7, 0, 0, 16384, 0], "many": [(37 * i) % 501 for i in range(300)], "long": [3000001, 17],
    "table": [5] * 128, "table1": [5] * 129,
}


@pytest.mark.parametrize("sizes", SIZE_SETS)
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("factor", [0.3, 4.0])
def test_clip(sizes, offset, factor):
    from tensor_transformer_mlp_03_amd.block import GradClip
    n = SIZE_SETS[sizes]
    kinds = [BF16 if i % 3 == 1 else F32 for i in range(len(n))]
    flats, g = grads_of(7, n, kinds, offset)
    g64 = [f64(t) for t in g]
    for scale in (1.0, -0.5):
        plain, _ = OB.clip(g64, np.inf, scale)
        max_norm = float(np.float32(factor * plain))
        norm, want = OB.clip(g64, max_norm, scale)
        outs = [torch.full_like(t, 9.0) for t in g]
        before = [f.clone() for f in flats]
        got = GradClip(g, outs).clip(max_norm, scale)
        close("norm", got, np.float64(norm), norm, 2)
        for o, w in zip(outs, want):
            close("out", o, w, w, 4)
        assert all(torch.equal(torch.nan_to_num(a, 5.0), torch.nan_to_num(b, 5.0)) for a, b in zip(before, flats))
        # in place, and through the two calls that ranks use
        h = GradClip(g)
        total = h.sumsq().clone()
        assert abs(float(total) - sum((v ** 2).sum() for v in g64)) <= 1e-12 * float(total)
        h.scale(max_norm, scale)
        for t, o in zip(g, outs):
            assert torch.equal(t, o)
        for f, b, t in zip(flats, before, g):
            f2, b2 = f.clone(), b.clone()
            f2[offset:offset + t.numel()] = b2[offset:offset + t.numel()] = 0
            assert torch.equal(torch.nan_to_num(f2, 5.0), torch.nan_to_num(b2, 5.0))
            f.copy_(b)


def test_clip_nothing():
    from tensor_transformer_mlp_03_amd.block import GradClip
    assert float(GradClip([]).clip(1.0)) == 0.0
    z = torch.zeros(100, device="cuda")
    assert float(GradClip([z]).clip(1.0)) == 0.0 and float(z.abs().max()) == 0.0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_clip_not_finite(bad):
    """The norm says so and the gradients keep their values."""
    from tensor_transformer_mlp_03_amd.block import GradClip
    g = [torch.ones(5000, device="cuda"), torch.ones(9, dtype=BF16, device="cuda")]
    g[0][4321] = bad
    keep = [t.clone() for t in g]
    norm = float(GradClip(g).clip(1.0))
    assert np.isnan(norm) if np.isnan(bad) else np.isposinf(norm)
    for t, k in zip(g, keep):
        assert torch.equal(torch.nan_to_num(t, 3.0), torch.nan_to_num(k, 3.0))
    h = GradClip(g)
    h.clip(1.0, scale=0.5)
    assert float(g[1][0]) == 0.5


def test_clip_squares_past_float32():
    from tensor_transformer_mlp_03_amd.block import GradClip
    g = torch.full((1 << 16,), 2.0 ** 100, device="cuda")
    h = GradClip([g])
    assert float(h.clip(1.0)) == 2.0 ** 108
    assert float(g[0]) == 2.0 ** -8
    tiny = torch.full((1 << 16,), 2.0 ** -100, device="cuda")
    assert float(GradClip([tiny]).clip(1.0)) == 2.0 ** -92 and float(tiny[0]) == 2.0 ** -100


def test_clip_past_32_bits():
    """A gradient of more than 2^31 elements."""
    from tensor_transformer_mlp_03_amd.block import GradClip
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    assert float(GradClip([g]).clip(6.5)) == 13.0
    assert float(g[-1]) == 1.5 and float(g[0]) == 2.0 and float(g[1 << 31]) == 6.0


# --- streams and graphs ------------------------------------------------------------------------------------------
def test_on_another_stream():
    """Every call runs on the stream it is given."""
    from tensor_transformer_mlp_03_amd.block import GradClip, Route
    c, params, t = edge_case(2, 40, 520, "rms", "rms", F32, F32, F32, 40)
    e = make_edge(c, params, 520, 40)
    y, r = t["y"].cuda(), t["r"].cuda()
    want_r, want_x = torch.empty_like(r), torch.empty(40, 520, dtype=BF16, device="cuda")
    e.forward(y, r, want_r, want_x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ro, x = torch.empty_like(want_r), torch.empty_like(want_x)
    ids = route_ids(3, 40, 2, 8).to(torch.int32).cuda()
    h = Route(40, 2, 8)
    Xs, Y = torch.empty(h.rows, 520, dtype=BF16, device="cuda"), torch.empty(40, 520, device="cuda")
    clip = GradClip([Y])
    torch.cuda.synchronize()
    e.forward(y, r, ro, x, stream=s)
    h.sort(ids, stream=s)
    h.dispatch(x, Xs, stream=s)
    h.combine(Xs, None, Y, stream=s)
    norm = clip.clip(1.0, stream=s)
    s.synchronize()
    assert torch.equal(ro, want_r) and torch.equal(x, want_x)
    both = 2 * want_x.float()
    assert abs(float(norm) - float(both.double().norm())) <= 1e-6 * float(norm)
    close("clipped", Y, f64(both) / float(both.double().norm()), f64(both) / float(norm), 4)


def test_in_a_graph():
    """A whole step captured once, replayed on new inputs with eager work between the replays."""
    from tensor_transformer_mlp_03_amd.block import GradClip, Route
    M, H, E, K = 70, 264, 6, 3
    c, params, t = edge_case(7, M, H, "layer", "rms", F32, F32, F32, 20)
    e = make_edge(c, params, H, 20)
    gen = torch.Generator().manual_seed(0)
    y, r, ids, w = t["y"].cuda(), t["r"].cuda(), route_ids(1, M, K, E, 0.1).cuda(), torch.rand(M, K, generator=gen).cuda()
    h = Route(M, K, E)
    new = lambda *s, d=F32: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    b = dict(ro=new(M, H), x=new(M, H, d=BF16), Xs=new(h.rows, H, d=BF16), Y=new(M, H), dZs=new(h.rows, H, d=BF16),
             dw=new(M, K), dX=new(M, H), dr=new(M, H), dy=new(M, H, d=BF16))
    e._place(M, r.device)
    outs = [torch.empty_like(g) for g in e.grads.values()]
    clip = GradClip(list(e.grads.values()), outs)

    def step():
        e.forward(y, r, b["ro"], b["x"])
        h.sort(ids)
        h.dispatch(b["x"], b["Xs"])
        h.combine(b["Xs"], w, b["Y"])
        h.combine_backward(b["Y"], b["Xs"], w, b["dZs"], b["dw"])
        h.dispatch_backward(b["dZs"], b["dX"])
        e.backward(y, b["ro"], b["Y"], b["dX"], b["dr"], b["dy"])
        clip.clip(0.5)

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for n in range(4):
        y.copy_(normal(gen, M, H))
        ids.copy_(route_ids(50 + n, M, K, E, 0.2))
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in (*b.values(), *outs, clip.norm, h.counts, h.row_of)]
        for v in (*b.values(), *outs):
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [*b.values(), *outs, clip.norm, h.counts, h.row_of]
        assert all(torch.equal(a, g) for a, g in zip(want, got)), n


def test_the_same_bits_twice():
    """No result depends on timing."""
    from tensor_transformer_mlp_03_amd.block import GradClip
    c, params, t = edge_case(3, 3000, 640, "layer", "layer", F32, BF16, BF16, 700)
    e = make_edge(c, params, 640, 700)
    y, r, d, dx = (t[k].cuda() for k in ("y", "r", "dr", "dx"))
    runs = []
    for _ in range(3):
        dr, dy = torch.empty_like(d), torch.empty(3000, 640, dtype=BF16, device="cuda")
        g = e.backward(y, r, d, dx, dr, dy)
        norm = GradClip([v.clone() for v in g.values()]).clip(1e-3)
        runs.append([dr, dy, norm.clone(), *(v.clone() for v in g.values())])
    assert all(torch.equal(a, b) for other in runs[1:] for a, b in zip(runs[0], other))


def test_graph_of_a_backward_outlives_other_sizes():
    """A captured backward's gradients and workspace stay its own while the object runs other sizes."""
    H, rows = 512, 4
    c, params, t = edge_case(6, 2000, H, "rms", "layer", F32, F32, BF16, rows)
    e = make_edge(c, params, H, rows)
    y, r, d, dx = (t[k].cuda() for k in ("y", "r", "dr", "dx"))

    def backward(M):
        dr, dy = torch.empty(M, H, device="cuda"), torch.empty(M, H, device="cuda", dtype=BF16)
        return e.backward(y[:M], r[:M], d[:M], dx[:M], dr, dy), dr, dy

    want = {k: v.clone() for k, v in backward(40)[0].items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got, dr, dy = backward(40)
    torch.cuda.current_stream().wait_stream(side)
    for M in (2000, 3, 801):
        other = {k: v.clone() for k, v in backward(M)[0].items()}
        junk = [torch.full((n,), 7.0, device="cuda") for n in (10 * H, 500 * H, 1 << 22)]  # takes what was freed
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want), M
        assert all(bool((j == 7.0).all()) for j in junk), M
        assert all(torch.equal(v, other[k]) for k, v in backward(M)[0].items()), M


@pytest.mark.parametrize("T,K,E,cap", [(0, 2, 5, 1000), (1, 1, 512, 40), (8, 2, 8, 3000), (512, 8, 256, 512), (700, 6, 3, 4104),
                                       (1100, 8, 512, 64), (70000, 2, 64, 9000)])
def test_route_sort_mostly_padding(T, K, E, cap):
    """A capacity far above what the pairs fill: workgroups that place nothing mark the padding."""
    check_sort(route_ids(T + E, T, K, E, 0.2, bad=T > 4), E, 8, cap, torch.int32)
    check_sort(torch.full((T, K), E - 1), E, 8, cap, torch.int64)


@pytest.mark.parametrize("T,H,K,z,y", [(2048, 4096, 8, F32, F32), (9001, 1032, 6, F32, BF16), (601, 20480, 8, BF16, F32)])
def test_route_large_moves_equal_their_parts(T, H, K, z, y):
    """Launches past the size from which accesses are non-temporal give the bits of small ones."""
    from tensor_transformer_mlp_03_amd import _lib as L
    h = check_sort(route_ids(T, T, K, 24, 0.1), 24, 8, 0, torch.int32)
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s, dtype: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    Zs, w, dY = rnd(h.rows, H, dtype=z), rnd(T, K, dtype=F32), rnd(T, H, dtype=y)
    assert Zs.numel() * Zs.element_size() + dY.numel() * dY.element_size() > 1 << 27
    Y, dZs, dw = torch.empty_like(dY), torch.empty(h.rows, H, dtype=BF16, device="cuda"), torch.empty_like(w)
    h.combine(Zs, w, Y)
    h.combine_backward(dY, Zs, w, dZs, dw)
    for t0 in range(0, T, 300):
        t = slice(t0, min(t0 + 300, T))
        keep, rows = torch.unique(h.row_of[t][h.row_of[t] >= 0].long(), return_inverse=True)
        sub = torch.full_like(h.row_of[t], -1)
        sub[h.row_of[t] >= 0] = rows.int()
        Zp, Yp, dwp = Zs[keep].contiguous(), torch.empty_like(Y[t]), torch.empty_like(dw[t])
        L.tpmlp_route_combine(Zp, sub, w[t], Yp)
        L.tpmlp_route_combine_bwd(dY[t], Zp, sub, None, w[t], None, dwp)
        assert torch.equal(Yp, Y[t]) and torch.equal(dwp, dw[t]), t0
        pair = h.src_of[keep].long()
        assert torch.equal(dZs[keep], (dY.float()[pair // K] * w.view(-1)[pair, None]).to(BF16)), t0
    assert not bool(dZs[h.src_of < 0].any())


@pytest.mark.parametrize("T,K,H,pad", [(5, 2, 64, 0), (9, 5, 331, 3), (6, 9, 1024, 0), (5, 3, 1032, 0), (7, 12, 2050, 1)])
def test_route_dropped_pair_of_a_bad_row(T, K, H, pad):
    """A dropped pair's dw is 0 whatever its token's dY holds; the token's other pairs see it."""
    h = check_sort(route_ids(T, T, K, 4, 0.4), 4, 8, 0, torch.int32)
    gen = torch.Generator().manual_seed(H)
    dY, Z, w = normal(gen, T, H), normal(gen, h.rows, H), torch.rand(T, K, generator=gen)
    dY[0, 3], dY[2, H - 1], dY[4] = float("inf"), float("nan"), float("-inf")
    kept, bad = h.row_of.cpu() >= 0, ~torch.isfinite(dY).all(1)
    assert bool((~kept[bad]).any()) and bool(kept[bad].any())
    dZs, dw = torch.empty(h.rows, H, dtype=BF16, device="cuda"), torch.full((T, K), 5.0, device="cuda")
    h.combine_backward(put(dY, pad), put(Z, pad), w.cuda(), dZs, dw)
    dw = dw.cpu()
    assert bool((dw[~kept] == 0.0).all()) and not bool(torch.isfinite(dw[kept & bad[:, None]]).any())
    want, mag = OB.route_combine_backward(f64(dY[~bad]), f64(Z), h.row_of.cpu().numpy()[~bad.numpy()], f64(w[~bad]), h.rows)[1:]
    close("dw", dw[~bad], want, mag, H / 256 + 16)


def test_edge_backward_on_given_streams():
    """While a backward runs on the stream that it was given, what another size has replaced is not handed out to
    other streams, neither if the object keeps to one stream nor if it goes from one to another."""
    H, rows = 512, 4
    c, params, t = edge_case(6, 2000, H, "rms", "layer", F32, F32, BF16, rows)
    y, r, d, dx = (t[k].cuda() for k in ("y", "r", "dr", "dx"))

    def backward(e, M, stream):
        dr, dy = torch.empty(M, H, device="cuda"), torch.empty(M, H, device="cuda", dtype=BF16)
        torch.cuda.current_stream().synchronize()
        return [dr, dy, *e.backward(y[:M], r[:M], d[:M], dx[:M], dr, dy, stream=stream).values()]

    want = {}
    for M in (40, 2000):
        want[M] = [v.clone() for v in backward(make_edge(c, params, H, rows), M, None)]
    torch.cuda.synchronize()
    for streams in ([1, 1], [1, 2], [None, 1]):
        s = {1: torch.cuda.Stream(), 2: torch.cuda.Stream(), None: torch.cuda.current_stream()}
        e = make_edge(c, params, H, rows)
        backward(e, 40, s[1] if streams[0] else None)
        torch.cuda.synchronize()
        last = s[streams[1]]
        with torch.cuda.stream(last):
            torch.cuda._sleep(100_000_000)
        small = backward(e, 40, last)
        old = [(v.data_ptr(), v.numel(), v.dtype) for v in (e._ws, e.grads["gate"])]
        large = backward(e, 2000, last)
        assert e._ws.data_ptr() != old[0][0] and e.grads["gate"].data_ptr() != old[1][0]
        del small[2:]  # the gate's gradient, which nothing holds now, and those that the second call overwrote
        junk = []
        for own in (torch.cuda.current_stream(), s[streams[0]]):
            if own != last:
                with torch.cuda.stream(own):
                    junk += [torch.full((n,), 7, dtype=k, device="cuda") for _, n, k in old for _ in range(3)]
        if not last.query():  # still at work
            assert not {j.data_ptr() for j in junk} & {a for a, _, _ in old}, streams
        torch.cuda.synchronize()
        assert all(bool((j == 7).all()) for j in junk)
        assert all(torch.equal(a, b) for a, b in zip(want[40], small)), streams
        assert all(torch.equal(a, b) for a, b in zip(want[2000], large)), streams
        handle = backward(make_edge(c, params, H, rows), 40, s[1].cuda_stream)
        s[1].synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[40], handle))
        zero = backward(make_edge(c, params, H, rows), 40, 0)  # the default stream's handle
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[40], zero))


def test_pinned_host_memory():
    """Host memory that the GPU reaches is taken like its own: ids that the host made, a norm that it reads."""
    from tensor_transformer_mlp_03_amd import _lib as L
    from tensor_transformer_mlp_03_amd.block import Route
    ids = route_ids(3, 50, 2, 8, 0.1).to(torch.int32)
    want, h = check_sort(ids, 8, 8, 0, torch.int32), Route(50, 2, 8)
    h.sort(ids.pin_memory())
    assert torch.equal(h.row_of, want.row_of) and torch.equal(h.src_of, want.src_of)
    g, norm = torch.full((4,), 2.0, device="cuda"), torch.zeros(1, pin_memory=True)
    table = L.GradTable([g])
    L.tpmlp_clip_grad_norm(table, 1.0, norm, torch.empty(L.tpmlp_grad_workspace_bytes(table), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert float(norm) == 4.0 and bool((g == 0.5).all())
    with pytest.raises(ValueError, match="not on the GPU"):
        h.sort(ids)
    with pytest.raises(ValueError, match="not on the GPU"):
        L.GradTable([torch.ones(3)])


# Each row form of the backward with three to nine rows a workgroup (a wave, up to 512 elements); the whole ones past
# 128 MB, from where their accesses are non-temporal.
LOOPS = [(24003, 256), (12003, 512), (6203, 1000), (3003, 2048), (2050, 3000), (1030, 6000), (1030, 8200),
         (12003, 255), (9301, 511), (2500, 1001), (2050, 2050), (1030, 4101)]


@pytest.mark.parametrize("M,H", LOOPS)
@pytest.mark.parametrize("kind,groups", [("rms", 1), ("layer", 3)])
def test_edge_backward_of_several_rows(M, H, kind, groups):
    from tensor_transformer_mlp_03_amd import _lib as L
    rows = -(-M // groups)
    c, params, _ = edge_case(1, 1, H, kind, kind, F32, F32, BF16, 1)
    e = make_edge(c, {**params, "gate": torch.ones(groups, H, dtype=BF16)}, H, rows)
    n = L.tpmlp_edge_bwd_workspace_bytes(e.desc, M) - (32 * M if H > 4096 else 0)
    at_once = n // (H * (8 if kind == "rms" else 16)) * (4 if H <= 512 else 1)
    assert 3 <= M / at_once <= 9
    assert H % 4 or 22 * M * H > 1 << 27
    run_edge(2 * H + 1, M, H, kind, kind, F32, F32, BF16, rows)


@pytest.mark.parametrize("H", [256, 512, 1000, 2048, 3000, 6000, 12000, 20000, 32768])
@pytest.mark.parametrize("kind,p", [("rms", F32), ("layer", BF16)])
def test_edge_forward_past_the_caches_equals_its_parts(H, kind, p):
    """Launches past 128 MB, in each row form, give the bits of small ones."""
    M = (1 << 27) // (14 * H) + 300
    c, params, _ = edge_case(3, 1, H, kind, kind, F32, F32, p, 0)
    params["gate"] = normal(torch.Generator().manual_seed(H), 1, H, dtype=p)
    e = make_edge(c, params, H, 0)
    gen = torch.Generator(device="cuda").manual_seed(H)
    y, r = (torch.randn(M, H, generator=gen, device="cuda") for _ in range(2))
    ro, x = torch.empty_like(r), torch.empty(M, H, dtype=BF16, device="cuda")
    e.forward(y, r, ro, x)
    step = (1 << 25) // (14 * H)
    assert step < M and bool(torch.isfinite(x).all())
    part_r, part_x = torch.empty(step, H, device="cuda"), torch.empty(step, H, dtype=BF16, device="cuda")
    for at in range(0, M, step):
        n = min(step, M - at)
        e.forward(y[at:at + n], r[at:at + n], part_r[:n], part_x[:n])
        assert torch.equal(ro[at:at + n], part_r[:n]) and torch.equal(x[at:at + n], part_x[:n]), at


@pytest.mark.parametrize("T,H,K,E,capacity", [(5003, 2048, 7, 24, 0), (5003, 2056, 7, 24, 1600), (160, 33000, 20, 8, 0)])
def test_route_dispatch_past_the_caches(T, H, K, E, capacity):
    """A dispatch past 128 MB: every row is its token's, padding rows are zeros."""
    h = check_sort(route_ids(T, T, K, E, 0.1), E, 8, capacity, torch.int32)
    assert 2 * H * (T + h.rows) > 1 << 27
    X = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").to(BF16)
    Xs = torch.full((h.rows, H), float("nan"), dtype=BF16, device="cuda")
    h.dispatch(X, Xs)
    on = h.src_of >= 0
    assert torch.equal(Xs[on], X[h.src_of[on].long() // K]) and not bool(Xs[~on].any())


def test_clip_many_tables():
    """More than one launch's 128 tensors and more than 2048 partial sums, which are then added up beforehand."""
    from tensor_transformer_mlp_03_amd.block import GradClip
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = [(torch.randn(163840 - 3 * i, generator=gen, device="cuda") * 0.1).to(BF16 if i % 3 == 1 else F32) for i in range(260)]
    total = sum(float(t.double().square().sum()) for t in g)
    norm = np.sqrt(total)
    for scale in (1.0, -0.5):
        max_norm = float(np.float32(0.3 * norm))
        outs = [torch.full_like(t, 9.0) for t in g]
        close("norm", GradClip(g, outs).clip(max_norm, scale), np.float64(norm * abs(scale)), norm * abs(scale), 2)
        factor = scale * min(1.0, max_norm / (norm * abs(scale)))
        for o, t in zip(outs, g):
            want = t.double() * factor
            half = torch.finfo(o.dtype).eps / 2
            assert bool(((o.double() - want).abs() <= (half + 4 * (1 + half) * U) * want.abs() + 1e-37).all())
    h = GradClip(g)
    assert abs(float(h.sumsq()) - total) <= 1e-12 * total
    h.scale(max_norm, scale)
    assert all(torch.equal(a, b) for a, b in zip(g, outs))
