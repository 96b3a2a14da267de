"""The gated block's kernels against the float64 oracle (oracle/gated.py).

Tolerances.  An output's error is its last rounding, half a step of its type relative to the value,
plus what comes before it:

* the gated MLP: the oracle's own tolerance, which carries the roundings to bf16 between the products
  and float32 sums of n terms (n 2^-24 of their magnitudes) through to the output;
* dropout: a sum, a product and a sum in float32, 4 roundings; the bias's gradient adds M rows: M + 8;
* the edge in 8 bits: x before its rounding within 200 roundings (as the edge's bf16 x), and one more
  for the product with the reciprocal of the scale; then half a step of E4M3, 2^-4 of the value or
  2^-10 of the scale below its normal range;
* 4-bit products: the oracle's own tolerance, exact products and a float32 sum of K terms.
"""
import sys

import numpy as np
import pytest

from oracle import block as OB
from oracle import gated as OG

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
NAMES = {"f32": F32, "bf16": BF16}
U = OG.U


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


def within(name, got, want, tol):
    """|got - want| <= half a step of got's type at want + tol."""
    half = torch.finfo(got.dtype).eps / 2
    g = f64(got)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    t = half * np.abs(want) + (1 + half) * tol + 1e-37
    bad = ~(np.abs(g - want) <= t)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / t, 0)), g.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {g.size} off; at {i}: {g[i]!r} want {want[i]!r} tol {t[i]!r}")


class Strided:
    """A [M,H] view with row stride ld at an element offset, in a buffer whose other elements hold a
    value that no call may change."""

    def __init__(self, M, H, dtype, ld=None, offset=0, fill=None):
        ld = H if ld is None else ld
        self.mark = 0x5A if dtype == U8 else 12345.0
        self.flat = torch.full((offset + M * ld + 64,), self.mark, dtype=dtype, device="cuda")
        self.view = self.flat.as_strided((M, H), (ld, 1), offset)
        if fill is not None:
            self.view.copy_(fill)

    def untouched(self):
        rest = self.flat.clone()
        v = self.view
        rest.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(self.mark)
        return bool((rest == torch.full_like(rest, self.mark)).all())


def normal(gen, *shape, dtype=F32, scale=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * scale + mean).to(dtype)


def guarded(t, rows=64):
    """A copy on the GPU between margins of NaN, and whether they are as they were."""
    n = t.numel()
    flat = torch.full((n + 2 * rows * 16,), float("nan"), dtype=t.dtype, device="cuda")
    v = flat[rows * 16:rows * 16 + n].view(t.shape)
    v.copy_(t)
    return v, lambda: bool(torch.isnan(flat[:rows * 16]).all() and torch.isnan(flat[rows * 16 + n:]).all())


# --- the gated MLP ----------------------------------------------------------------------------------
def glu_case(M, H, F, seed=0):
    gen = torch.Generator().manual_seed(seed * 1000 + M + H + F)
    return dict(X=normal(gen, M, H, dtype=BF16), A=normal(gen, H, 2 * F, dtype=BF16, scale=H ** -0.5),
                B=normal(gen, F, H, dtype=BF16, scale=F ** -0.5), dZ=normal(gen, M, H, dtype=BF16, scale=0.1),
                P=normal(gen, M, 2 * F, dtype=BF16))


def check_glu(M, H, F, act, z=BF16, x=BF16, w=F32, keep=True):
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    c = glu_case(M, H, F)
    n = {k: f64(v) for k, v in c.items()}
    X, dZ = c["X"].cuda(), c["dZ"].cuda()
    mlp = GatedMLP(c["A"].cuda(), c["B"].cuda(), act)
    want = OG.glu_forward(n["X"], n["A"], n["B"], act)
    Z, z_ok = guarded(torch.zeros(M, H, dtype=z))
    P, p_ok = guarded(torch.zeros(M, 2 * F, dtype=BF16))
    mlp.forward(X, Z, P if keep else None)
    torch.cuda.synchronize()
    within("Z", Z, want["Z"], want["Z_tol"])
    if keep:
        within("P", P, want["P"], want["P_tol"])
    assert z_ok() and p_ok()
    want = OG.glu_backward(n["dZ"], n["X"], n["A"], n["B"], n["P"] if keep else None, act)
    dX, x_ok = guarded(torch.zeros(M, H, dtype=x))
    dA, a_ok = guarded(torch.zeros(H, 2 * F, dtype=w))
    dB, b_ok = guarded(torch.zeros(F, H, dtype=w))
    mlp.backward(dZ, X, c["P"].cuda() if keep else None, dX, dA, dB)
    torch.cuda.synchronize()
    for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        within(name, got, want[name], want[name + "_tol"])
    assert x_ok() and a_ok() and b_ok()


@pytest.mark.parametrize("M", [1, 2, 3, 5, 7, 8, 9, 16, 17, 33, 64, 65, 127, 128, 129, 255, 257])
def test_glu_tokens(M):
    check_glu(M, 136, 72, "silu", keep=M % 2 == 0)


@pytest.mark.parametrize("H,F", [(8, 8), (8, 64), (64, 8), (24, 40), (64, 32), (72, 136), (256, 64), (264, 200), (520, 264),
                                 (1032, 24), (40, 1368)])
@pytest.mark.parametrize("M", [3, 70])
def test_glu_sizes(M, H, F):
    check_glu(M, H, F, "silu", z=F32, keep=M == 70)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "sigmoid"])
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("M", [5, 131])
def test_glu_activations(act, keep, M):
    check_glu(M, 96, 168, act, keep=keep)


@pytest.mark.parametrize("z", ["f32", "bf16"])
@pytest.mark.parametrize("w", ["f32", "bf16"])
def test_glu_types(z, w):
    check_glu(65, 80, 104, "gelu", z=NAMES[z], x=NAMES[z], w=NAMES[w])


@pytest.mark.parametrize("M,H,F", [(300, 1096, 520), (513, 520, 1032), (1001, 264, 264)])
def test_glu_several_tiles(M, H, F):
    check_glu(M, H, F, "silu", z=F32, x=F32, w=BF16, keep=M != 513)


@pytest.mark.parametrize("M,H,F", [(2100, 72, 40), (3000, 136, 24), (4305, 64, 408), (1999, 24, 1032)])
@pytest.mark.parametrize("x,w", [("f32", "bf16"), ("bf16", "f32")])
def test_glu_many_tokens(M, H, F, x, w):
    """Small weights: their gradients' products are split along the tokens, the tokens' along F or not."""
    check_glu(M, H, F, "silu", x=NAMES[x], w=NAMES[w], keep=x == "f32")


@pytest.mark.parametrize("M,H,F", [(1001, 1000, 1368), (40, 4096, 2048), (2, 4104, 2056), (9, 8200, 520), (2056, 1032, 2048),
                                   (6400, 264, 520)])
def test_glu_large(M, H, F):
    """Every plan (split along K, the larger tiles, transposed weights) in the norm.  On the way to an output lie
    at most three roundings to bf16 (P, and h or dP, and the output's), each off by at most 2^-8 of the value, and act' and
    act'' below 1.2: within 4 * 2^-8 of the magnitude that float32 products of the same operands have."""
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    c = {k: v.cuda() for k, v in glu_case(M, H, F, 1).items()}
    mlp = GatedMLP(c["A"], c["B"], "silu")
    e = lambda *s: torch.full(s, float("nan"), dtype=BF16, device="cuda")  # noqa: E731
    Z, P, dX, dA, dB = e(M, H), e(M, 2 * F), e(M, H), e(H, 2 * F), e(F, H)
    mlp.forward(c["X"], Z, P)
    mlp.backward(c["dZ"], c["X"], P, dX, dA, dB)
    d = {k: v.double() for k, v in c.items()}
    Pd = (d["X"] @ d["A"]).requires_grad_()
    h = torch.nn.functional.silu(Pd[:, :F]) * Pd[:, F:]
    want = {"P": Pd.detach(), "Z": (h @ d["B"]).detach(), "dB": (h.t() @ d["dZ"]).detach()}
    h.backward(d["dZ"] @ d["B"].t())
    want["dA"], want["dX"] = d["X"].t() @ Pd.grad, Pd.grad @ d["A"].t()
    for name, got in (("P", P), ("Z", Z), ("dX", dX), ("dA", dA), ("dB", dB)):
        off = float((got.double() - want[name]).norm() / want[name].norm())
        assert off <= 4 * 2.0 ** -8, (name, off)
        big = float(((got.double() - want[name]).abs() / (want[name].abs() + want[name].square().mean().sqrt())).max())
        assert big <= 0.1, (name, big)  # no element is wrong, whatever the norm says


def test_glu_offsets_past_32_bits():
    """P and dP of more than 2^32 bytes.  P of the first and last rows has the bits that the rows alone get
    (one K step); Z and dX are float32 sums of F and 2 F terms in another order, dA and dB the sums of two halves'."""
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    M, H, F = 70000, 64, 16384
    gen = torch.Generator("cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    X, dZ = n(M, H).bfloat16(), n(M, H).bfloat16()
    mlp = GatedMLP((n(H, 2 * F) / 8).bfloat16(), (n(F, H) / 128).bfloat16())
    e = lambda *s, dtype=F32: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731

    def run(lo, hi):
        Z, P, dX, dA, dB = e(hi - lo, H), e(hi - lo, 2 * F, dtype=BF16), e(hi - lo, H), e(H, 2 * F), e(F, H)
        mlp.forward(X[lo:hi], Z, P)
        mlp.backward(dZ[lo:hi], X[lo:hi], P, dX, dA, dB)
        return Z, P, dX, dA, dB

    Z, P, dX, dA, dB = run(0, M)
    for lo, hi in ((0, 128), (M - 200, M)):
        z, p, dx, _, _ = run(lo, hi)
        assert torch.equal(p, P[lo:hi])
        g, u = p[:, :F].float(), p[:, F:].float()
        h, dh = torch.nn.functional.silu(g) * u, dZ[lo:hi].float() @ mlp.B.float().t()
        s = torch.sigmoid(g)
        dp = torch.cat((dh * u * s * (1 + g * (1 - s)), dh * g * s), 1)
        assert ((z - Z[lo:hi]).abs() <= 2.1 * F * U * (h.abs() @ mlp.B.float().abs())).all()
        assert ((dx - dX[lo:hi]).abs() <= 2.1 * 2 * F * U * (dp.abs() @ mlp.A.float().abs().t())).all()
    del P
    halves = [run(0, M // 2)[3:], run(M // 2, M)[3:]]
    # Of M additions each is off by at most 2^-24 of a partial sum, whose norm over the elements grows with its
    # terms (random ones): on either side at most M 2^-24 of the sums' norm.
    for i, got in enumerate((dA, dB)):
        want = halves[0][i].double() + halves[1][i].double()
        assert float((got - want).norm() / want.norm()) <= 2 * M * U, i


def test_glu_gradient_is_a_difference():
    """<dZ, Z(x + h d) - Z(x - h d)> / 2h against <gradient, d> with float32 outputs.  The step moves values by
    1/8 of themselves, so that the difference stands out of the bf16 roundings in Z: these are off by at most 2^-8 of h's
    magnitude, at random over 96 x 64 elements, and the third derivative's term is measured by halving the step."""
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    M, H, F = 96, 64, 64
    c = glu_case(M, H, F, 3)
    X, A, B, dZ = (c[k].cuda() for k in ("X", "A", "B", "dZ"))
    g = [torch.empty(M, H, device="cuda"), torch.empty(H, 2 * F, device="cuda"), torch.empty(F, H, device="cuda")]
    GatedMLP(A, B, "gelu").backward(dZ, X, None, *g)

    def loss(x, a, b):
        Z = torch.empty(M, H, device="cuda")
        GatedMLP(a, b, "gelu").forward(x, Z)
        return float((Z.double() * dZ.double()).sum())

    gen = torch.Generator().manual_seed(9)
    for i, t in enumerate((X, A, B)):
        # a direction of the gradient's signs: the difference is as large as it can be
        d = (torch.sign(g[i]) * t.abs().float().mean() / 16).cuda()
        up, down = (t.float() + d).bfloat16(), (t.float() - d).bfloat16()
        real = (up.double() - down.double()) / 2
        args = [[X, A, B], [X, A, B]]
        args[0][i], args[1][i] = up, down
        diff = (loss(*args[0]) - loss(*args[1])) / 2
        want = float((g[i].double() * real).sum())
        assert abs(diff - want) <= 0.02 * abs(want), (i, diff, want)


def test_glu_no_tokens():
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    c = glu_case(1, 64, 40)
    mlp = GatedMLP(c["A"].cuda(), c["B"].cuda())
    e = lambda *s: torch.full(s, float("nan"), dtype=F32, device="cuda")  # noqa: E731
    none = torch.empty(0, 64, dtype=BF16, device="cuda")
    mlp.forward(none, e(0, 64), torch.empty(0, 80, dtype=BF16, device="cuda"))
    dA, dB = e(64, 80), e(40, 64)
    mlp.backward(none, none, None, e(0, 64), dA, dB)
    assert (dA == 0).all() and (dB == 0).all()


@pytest.mark.parametrize("M", [6, 70, 300])
def test_glu_bad_token_stays_alone(M):
    """A token of NaN or infinities spoils its own rows of Z, P and dX only; other rows keep their bits."""
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    H, F = 136, 72
    c = {k: v.cuda() for k, v in glu_case(M, H, F).items()}
    mlp = GatedMLP(c["A"], c["B"])

    def run(X, dZ):
        Z, P, dX = (torch.empty(M, n, dtype=BF16, device="cuda") for n in (H, 2 * F, H))
        dA, dB = torch.empty(H, 2 * F, device="cuda"), torch.empty(F, H, device="cuda")
        mlp.forward(X, Z, P)
        mlp.backward(dZ, X, P, dX, dA, dB)
        return Z, P, dX

    good = run(c["X"], c["dZ"])
    X, dZ = c["X"].clone(), c["dZ"].clone()
    X[2], dZ[2], X[M - 1, 5] = float("nan"), float("inf"), float("inf")
    bad = run(X, dZ)
    for g, b in zip(good, bad):
        keep = [i for i in range(M) if i not in (2, M - 1)]
        assert torch.equal(g[keep].view(torch.int16), b[keep].view(torch.int16))
        assert not torch.isfinite(b[2]).any()


def test_glu_large_pre_activations():
    """Gates far out: the sigmoid's exp overflows on one side and vanishes on the other."""
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    M, H, F = 4, 8, 8
    X = torch.zeros(M, H, dtype=BF16)
    X[:, 0] = torch.tensor([1e4, -1e4, 200.0, -200.0])
    A = torch.zeros(H, 2 * F, dtype=BF16)
    A[0, :F], A[0, F:] = 1.0, 2.0 ** -10
    B = torch.eye(F, H).bfloat16()
    for act in ("silu", "gelu", "relu", "sigmoid"):
        want = OG.glu_forward(f64(X), f64(A), f64(B), act)
        Z, P = torch.empty(M, H, device="cuda"), torch.empty(M, 2 * F, dtype=BF16, device="cuda")
        mlp = GatedMLP(A.cuda(), B.cuda(), act)
        mlp.forward(X.cuda(), Z, P)
        within(act, Z, want["Z"], want["Z_tol"])
        dX, dA, dB = torch.empty(M, H, device="cuda"), torch.empty(H, 2 * F, device="cuda"), torch.empty(F, H, device="cuda")
        mlp.backward(torch.ones(M, H, dtype=BF16, device="cuda"), X.cuda(), P, dX, dA, dB)
        back = OG.glu_backward(np.ones((M, H)), f64(X), f64(A), f64(B), f64(P), act)
        for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
            within(f"{act} {name}", got, back[name], back[name + "_tol"])


# --- dropout ------------------------------------------------------------------------------------------
def state_of(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def check_dropout(M, H, y, r, bias, p, pad=0, offset=0, site=3, first_row=0, seed=0x123456789ABCDEF, step=(5 << 32) + 77):
    from tensor_transformer_mlp_03_amd.gated import Dropout
    gen = torch.Generator().manual_seed(M * 131 + H)
    ld = H + pad
    Y = Strided(M, H, y, ld, offset, normal(gen, M, H, dtype=y))
    R = Strided(M, H, r, ld, offset, normal(gen, M, H, dtype=r, scale=2.0))
    b = normal(gen, H, dtype=bias).cuda() if bias else None
    out, dy = Strided(M, H, r, ld, offset), Strided(M, H, y, ld, offset)
    d = Dropout(p, state_of(seed, step), site, b)
    mask = OG.dropout_mask(M, H, p, seed, step, site, first_row)
    d.forward(Y.view, R.view, out.view, first_row)
    yb = f64(Y.view) + (f64(b) if bias else 0)
    mag = np.abs(f64(R.view)) + mask * (np.abs(f64(Y.view)) + (np.abs(f64(b)) if bias else 0))
    within("out", out.view, f64(R.view) + mask * yb, 4 * U * mag)
    db = torch.full((H,), float("nan"), device="cuda") if bias else None
    d.backward(R.view, dy.view, db, first_row)
    g = f64(R.view) * mask
    within("dy", dy.view, g, 2 * U * np.abs(g))
    if bias:
        within("db", db, g.sum(0), (M + 8) * U * np.abs(g).sum(0))
    assert out.untouched() and dy.untouched()


@pytest.mark.parametrize("M,H", [(1, 1), (1, 7), (3, 8), (2, 9), (5, 16), (17, 63), (4, 64), (33, 100), (100, 65), (7, 512), (65, 520),
                                 (16, 1000), (300, 1032), (2, 4104), (3, 20480), (40, 2047), (1000, 8), (4099, 24)])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout_sizes(M, H, p):
    check_dropout(M, H, F32 if M % 2 else BF16, BF16 if H % 2 else F32, BF16 if M % 3 else None, p)


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("r", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [None, "f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
def test_dropout_types_and_strides(y, r, bias, pad, offset):
    check_dropout(19, 136, NAMES[y], NAMES[r], NAMES.get(bias), 0.25, pad, offset)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 2.0 ** -16, 0.9999, 1.0])
def test_dropout_probabilities(p):
    check_dropout(9, 100, F32, F32, F32, p)


@pytest.mark.parametrize("seed,step,site,first", [(0, 0, 0, 0), (-1, -1, (1 << 32) - 1, 0), (1 << 62, 1 << 40, 1, (1 << 32) - 50)])
def test_dropout_states(seed, step, site, first):
    check_dropout(50, 72, BF16, BF16, BF16, 0.3, site=site, first_row=first, seed=seed, step=step)


def test_dropout_row_slices_agree():
    """Ranks that hold row slices drop what one that holds all rows does."""
    from tensor_transformer_mlp_03_amd.gated import Dropout
    d = Dropout(0.4, state_of(9, 2))
    y = torch.ones(64, 104, device="cuda")
    whole = torch.empty_like(y)
    d.forward(y, None, whole)
    for r in range(4):
        part = torch.empty(16, 104, device="cuda")
        d.forward(y[:16], None, part, first_row=16 * r)
        assert torch.equal(part, whole[16 * r:16 * r + 16])
    kept = whole != 0
    assert 0.5 < float(kept.float().mean()) < 0.7


def test_dropout_without_residual_and_in_place():
    from tensor_transformer_mlp_03_amd.gated import Dropout
    gen = torch.Generator().manual_seed(4)
    y, r = normal(gen, 33, 200).cuda(), normal(gen, 33, 200).cuda()
    d = Dropout(0.2, state_of(1, 1), 5)
    plain, added = torch.empty_like(y), torch.empty_like(y)
    d.forward(y, None, plain)
    d.forward(y, r, added)
    mask = OG.dropout_mask(33, 200, 0.2, 1, 1, 5)
    within("plain", plain, f64(y) * mask, 2 * U * np.abs(f64(y) * mask))
    a, b = r.clone(), y.clone()
    d.forward(y, a, a)        # over r
    assert torch.equal(a, added)
    d.forward(b, r, b)        # over y
    assert torch.equal(b, added)
    g = r.clone()
    dy = torch.empty_like(g)
    db, db2 = torch.empty(200, device="cuda"), torch.empty(200, device="cuda")
    d.backward(g, dy, db)
    d.backward(g, g, db2)     # over dout
    assert torch.equal(g, dy) and torch.equal(db, db2)


def test_dropout_dropped_values_reach_nothing():
    from tensor_transformer_mlp_03_amd.gated import Dropout
    mask = torch.from_numpy(OG.dropout_mask(40, 96, 0.5, 7, 0, 0)).cuda()
    d = Dropout(0.5, state_of(7, 0))
    for bad in (float("nan"), float("inf")):
        y = torch.where(mask == 0, bad, 1.0).float()
        out, dy, db = torch.empty_like(y), torch.empty_like(y), torch.empty(96, device="cuda")
        d.forward(y, None, out)
        assert torch.equal(out, mask.float())
        d.backward(y, dy, db)
        assert torch.equal(dy, mask.float()) and torch.equal(db, mask.float().sum(0))


def test_dropout_no_rows():
    from tensor_transformer_mlp_03_amd.gated import Dropout
    d = Dropout(0.5, state_of(7, 0))
    none, db = torch.empty(0, 40, device="cuda"), torch.full((40,), float("nan"), device="cuda")
    d.forward(none, none, torch.empty(0, 40, device="cuda"))
    d.backward(none, torch.empty(0, 40, device="cuda"), db)
    assert (db == 0).all()


def test_dropout_past_32_bits():
    """More than 2^32 bytes and 2^31 elements: the last rows equal a call on them alone."""
    from tensor_transformer_mlp_03_amd.gated import Dropout
    M, H = 131080, 16392
    d = Dropout(0.1, state_of(11, 3), bias=torch.ones(H, dtype=BF16, device="cuda"))
    y = torch.ones(M, H, dtype=BF16, device="cuda")
    out = torch.empty_like(y)
    d.forward(y, None, out)
    for at in (0, 65536, M - 24):
        part = torch.empty(24, H, dtype=BF16, device="cuda")
        d.forward(y[at:at + 24], None, part, first_row=at)
        assert torch.equal(part, out[at:at + 24]), at
    dy, db = out, torch.empty(H, device="cuda")
    d.backward(y, dy, db)
    part = torch.empty(24, H, dtype=BF16, device="cuda")
    d.backward(y[M - 24:], part, first_row=M - 24)
    assert torch.equal(part, dy[M - 24:])
    kept = db.double() / (65536 / (65536 - 6554)) / M
    assert float((kept - 0.9).abs().max()) < 0.01


# --- the edge in 8 bits -----------------------------------------------------------------------------------
def check_edge8(M, H, post, pre, y, r, p, kind, rows=0, pad=0, offset=0, scale_pad=0, seed=0):
    from tensor_transformer_mlp_03_amd.block import Edge
    gen = torch.Generator().manual_seed(seed + M * 7 + H)
    params = {}
    for side, k in (("post", post), ("pre", pre)):
        if k != "none":
            params["w_" + side] = normal(gen, H, dtype=p, scale=0.2, mean=1.0)
        if k == "layer":
            params["b_" + side] = normal(gen, H, dtype=p, scale=0.2)
    if rows:
        params["gate"] = normal(gen, -(-M // rows), H, dtype=p, scale=0.3, mean=0.5)
    Y = normal(gen, M, H, dtype=y, mean=0.3) if y else None
    R = normal(gen, M, H, dtype=r, scale=2.0, mean=-0.5)
    e = Edge(H, post=post, pre=pre, alpha=0.75, gate_rows=rows, **{k: v.cuda() for k, v in params.items()})
    want = OB.edge_forward(f64(Y) if y else None, f64(R), post, pre, rows=rows or M, alpha=0.75,
                           **{k: f64(v) for k, v in params.items()})
    ld = H + pad
    ro = Strided(M, H, r, ld, offset)
    codes = Strided(M, H, U8, ld, offset)
    if kind == "row":
        flat = torch.full((M + 4,), 12345.0, device="cuda")
        scales = flat[2:2 + M]
    else:
        S = Strided(M, H // 32, U8, H // 32 + scale_pad, offset)
        scales = S.view
    yv = Strided(M, H, y, ld, offset, Y).view if y else None
    e.forward_fp8(yv, Strided(M, H, r, ld, offset, R).view, ro.view, codes.view, scales)
    torch.cuda.synchronize()
    within("r", ro.view, want["r"], 100 * U * want["r_mag"])
    x, ex = want["x"], 200 * U * want["x_mag"]
    assert ro.untouched() and codes.untouched()
    if kind == "row":
        assert bool((flat[:2] == 12345.0).all() and (flat[2 + M:] == 12345.0).all())
        s = f64(scales)[:, None]
        amax = np.abs(x).max(1, keepdims=True)
        assert (np.abs(s * 448 - amax) <= ex.max(1, keepdims=True) + 4 * U * amax).all()
        per = np.broadcast_to(s, x.shape)
    else:
        assert S.untouched()
        got = scales.cpu().numpy().astype(np.int64)
        g, eg = np.abs(x).reshape(M, -1, 32), ex.reshape(M, -1, 32)
        lo, hi = (g - eg).max(2).clip(0), (g + eg).max(2)
        assert (OG.mx_exponent(lo, 448.0) <= got).all() and (got <= OG.mx_exponent(hi, 448.0)).all()
        per = OG.mx_values(got)
    v = OG.e4m3_values(codes.view.cpu().numpy()) * per
    tol = 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * per + 1.07 * (ex + 2 * U * np.abs(x))
    bad = ~(np.abs(v - x) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], v[bad][:3], x[bad][:3])


@pytest.mark.parametrize("H", [8, 9, 64, 100, 256, 257, 512, 1000, 1024, 1032, 2048, 4096, 4101, 8192, 12288, 20480, 32768])
def test_edge8_row_sizes(H):
    check_edge8(5, H, "none", "rms", F32, BF16, BF16, "row")


@pytest.mark.parametrize("H", [32, 64, 96, 256, 544, 1024, 1056, 2080, 4096, 4128, 8224, 12288, 20480, 32768])
def test_edge8_mx_sizes(H):
    check_edge8(5, H, "rms", "rms", F32, BF16, BF16, "mx")


@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "layer"), ("layer", "layer")])
@pytest.mark.parametrize("rows", [0, 3])
@pytest.mark.parametrize("kind", ["row", "mx"])
def test_edge8_norms(post, pre, rows, kind):
    check_edge8(7, 160, post, pre, BF16, F32, F32, kind, rows)


@pytest.mark.parametrize("y", [None, "f32", "bf16"])
@pytest.mark.parametrize("r", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset,scale_pad", [(0, 0, 0), (4, 4, 3), (3, 1, 1)])
@pytest.mark.parametrize("kind", ["row", "mx"])
def test_edge8_types_and_strides(y, r, pad, offset, scale_pad, kind):
    check_edge8(6, 288, "none" if y is None else "rms", "rms", NAMES.get(y), NAMES[r], BF16, kind, 0, pad, offset, scale_pad)


def test_edge8_of_many_rows():
    check_edge8(3000, 96, "none", "rms", BF16, F32, F32, "mx")
    check_edge8(3000, 100, "none", "rms", BF16, F32, F32, "row")


def test_edge8_past_the_caches_equals_its_parts():
    """A launch past 128 MB (non-temporal accesses) against the same rows in parts below it."""
    from tensor_transformer_mlp_03_amd.block import Edge
    M, H = 4096, 8192
    r = torch.randn(M, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    e = Edge(H, pre="rms", w_pre=torch.ones(H, device="cuda"))
    for scales in (lambda m: torch.empty(m, device="cuda"), lambda m: torch.empty(m, H // 32, dtype=U8, device="cuda")):
        whole, ws, wr = torch.empty(M, H, dtype=U8, device="cuda"), scales(M), torch.empty_like(r)
        e.forward_fp8(None, r, wr, whole, ws)
        for at in range(0, M, 1024):
            part, ps, pr = torch.empty(1024, H, dtype=U8, device="cuda"), scales(1024), torch.empty(1024, H, device="cuda")
            e.forward_fp8(None, r[at:at + 1024], pr, part, ps)
            assert torch.equal(part, whole[at:at + 1024]) and torch.equal(ps, ws[at:at + 1024]) and torch.equal(pr, wr[at:at + 1024])


@pytest.mark.parametrize("H", [64, 4096])
def test_edge8_rows_of_zeros_nan_and_extremes(H):
    from tensor_transformer_mlp_03_amd.block import Edge
    r = torch.zeros(6, H)
    r[1] = float("nan")
    r[2, :40] = 1.0
    r[3] = torch.linspace(-1, 1, H) * 1e-18   # its square is below the eps
    r[4, 0], r[5, 33] = float("inf"), float("nan")
    e = Edge(H, pre="rms", w_pre=torch.ones(H, device="cuda"), eps=1e-5)
    codes, row, mx = (torch.empty(6, n, dtype=d, device="cuda") for n, d in ((H, U8), (1, F32), (H // 32, U8)))
    for scales in (row.view(6), mx):
        e.forward_fp8(None, r.cuda(), None, codes, scales)
        v = OG.e4m3_values(codes.cpu().numpy())
        assert (v[0] == 0).all() and (v[2, 40:] == 0).all() and np.isfinite(v[2]).all() and np.isfinite(v[3]).all()
        assert np.isnan(v[1]).all() and np.isnan(v[5]).all() and np.isnan(v[4, 0]) and (v[4, 1:] == 0).all()
        per = f64(scales)[:, None] if scales is not mx else OG.mx_values(mx.cpu().numpy())
        x = f64(r[3]) / np.sqrt((f64(r[3]) ** 2).mean() + 1e-5)
        assert (np.abs(v[3] * per[3] - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * per[3] + 200 * U * np.abs(x)).all()
    assert row[0, 0] == 1 and row[1, 0] == 1 and (mx[:2] == 127).all() and (mx[2, 2:] == 127).all()


def test_edge8_tiny_and_huge_rows():
    """Without an eps a row's x does not depend on its size; weights carry it to the ends of float32."""
    from tensor_transformer_mlp_03_amd.block import Edge
    H = 64
    for w in (2.0 ** -149, 1e-40, 1e-38, 1e-30, 1e30, 2.0 ** 120):
        e = Edge(H, pre="rms", w_pre=torch.full((H,), w, device="cuda"), eps=0.0)
        r = torch.linspace(0.5, 1.5, H).view(1, H)
        x = f64(r) / np.sqrt((f64(r) ** 2).mean()) * float(np.float32(w))
        codes = torch.empty(1, H, dtype=U8, device="cuda")
        for scales in (torch.empty(1, device="cuda"), torch.empty(1, 2, dtype=U8, device="cuda")):
            e.forward_fp8(None, r.cuda(), None, codes, scales)
            per = f64(scales)[:, None] if scales.dtype == F32 else OG.mx_values(scales.cpu().numpy())
            v = OG.e4m3_values(codes.cpu().numpy()) * per
            # x in float32 is off by 2^-150 where it is subnormal
            tol = 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * per + 200 * U * np.abs(x) + 2.0 ** -149
            assert (np.abs(v - x) <= tol).all(), (w, v, x)


# --- 4-bit products ---------------------------------------------------------------------------------------
def fp4_weight(gen, N, K):
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.int64).to(U8)
    scales = torch.randint(118, 130, (N, K // 32), generator=gen, dtype=torch.int64).to(U8)
    return codes, scales


def fp4_x(gen, M, K, kind):
    """X and its scales, and the values that it stands for."""
    if kind == "bf16":
        x = normal(gen, M, K, dtype=BF16)
        return x, None, f64(x)
    codes = torch.randint(0, 254, (M, K), generator=gen, dtype=torch.int64)
    codes = torch.where(codes >= 127, codes + 1, codes).to(U8)  # no NaN
    if kind == "row":
        s = torch.rand(M, generator=gen) * 0.01 + 1e-3
        return codes, s, OG.e4m3_values(codes.numpy()) * f64(s)[:, None]
    s = torch.randint(115, 125, (M, K // 32), generator=gen, dtype=torch.int64).to(U8)
    return codes, s, OG.e4m3_values(codes.numpy()) * OG.mx_values(s.numpy())


def check_fp4(M, N, K, x="bf16", act="none", gated=False, y=F32, pad=0, offset=0, x_pad=0):
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    gen = torch.Generator().manual_seed(M * 10007 + N * 31 + K)
    codes, scales = fp4_weight(gen, 2 * N if gated else N, K)
    X, xs, values = fp4_x(gen, M, K, x)
    want, tol = OG.fp4_product(values, codes.numpy(), scales.numpy(), act, gated)
    Xv = Strided(M, K, X.dtype, K + x_pad, 0, X).view
    Y = Strided(M, N, y, N + pad, offset)
    Fp4Linear(codes.cuda(), scales.cuda(), act, gated).forward(Xv, Y.view, None if xs is None else xs.cuda())
    torch.cuda.synchronize()
    within("Y", Y.view, want, tol)
    assert Y.untouched()


@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 130])
@pytest.mark.parametrize("x", ["bf16", "row", "mx"])
def test_fp4_tokens(M, x):
    check_fp4(M, 40, 256, x)


@pytest.mark.parametrize("N", [1, 3, 15, 16, 17, 31, 33, 64, 65, 100, 257, 1367])
@pytest.mark.parametrize("x", ["bf16", "mx"])
@pytest.mark.parametrize("gated", [False, True])
def test_fp4_columns(N, x, gated):
    check_fp4(5, N, 160, x, "silu" if gated else "none", gated)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 256, 288, 992, 1024, 1056, 2080, 4096, 10240])
@pytest.mark.parametrize("x", ["bf16", "row", "mx"])
@pytest.mark.parametrize("M", [1, 20, 50])
def test_fp4_inner_sizes(K, x, M):
    check_fp4(M, 33, K, x)


@pytest.mark.parametrize("M", [4, 5, 16, 17, 33, 49, 64, 65])
@pytest.mark.parametrize("N,gated", [(17, False), (100, True), (20, True)])
@pytest.mark.parametrize("x", ["bf16", "row", "mx"])
def test_fp4_long_rows(M, N, gated, x):
    """A K of many blocks for each wave, and not a whole number of them."""
    check_fp4(M, N, 5408, x, "silu" if gated else "none", gated, BF16, x_pad=16)


@pytest.mark.parametrize("M,N,gated", [(16, 20480, True), (3, 12291, False), (40, 20490, False), (64, 4100, True), (20, 6160, True)])
def test_fp4_tiles_a_workgroup(M, N, gated):
    """Numbers of rows that ask for each of the tiles a workgroup, the last one short."""
    check_fp4(M, N, 96, "mx" if M % 2 else "bf16", "gelu", gated, BF16)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_fp4_activations(act, gated, y):
    check_fp4(9, 48, 128, "bf16", act, gated, NAMES[y])


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset,x_pad", [(4, 4, 16), (1, 0, 32), (3, 1, 16)])
@pytest.mark.parametrize("x", ["bf16", "row", "mx"])
@pytest.mark.parametrize("N", [44, 45])
def test_fp4_strides(y, pad, offset, x_pad, x, N):
    check_fp4(21, N, 96, x, y=NAMES[y], pad=pad, offset=offset, x_pad=x_pad)


def test_fp4_every_code_and_scale():
    """One product with 1: the weights' 16 values times every scale, exactly."""
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    N = 16 * 256
    codes = torch.zeros(N, 16, dtype=U8)
    codes[:, 0] = torch.arange(N) % 16
    scales = (torch.arange(N) // 16).to(U8).view(N, 1)
    want = OG.e2m1_values(codes.numpy())[:, 0] * OG.mx_values(scales.numpy())[:, 0]
    lin = Fp4Linear(codes.cuda(), scales.cuda())
    for X, xs in ((torch.zeros(1, 32, dtype=BF16), None), (torch.zeros(1, 32, dtype=U8), torch.ones(1)),
                  (torch.zeros(1, 32, dtype=U8), torch.full((1, 1), 127, dtype=U8))):
        X[0, 0] = 1 if X.dtype == BF16 else 0x38  # E4M3's 1
        Y = torch.empty(1, N, device="cuda")
        lin.forward(X.cuda(), Y, None if xs is None else xs.cuda())
        got = f64(Y)[0]
        nan = np.isnan(want)
        assert np.isnan(got[nan]).all()
        fine = ~nan & (np.abs(want) < 2.0 ** 128) & (np.abs(want) >= 2.0 ** -126)  # float32's normal range
        assert (got[fine] == want[fine]).all()
        assert (np.abs(got[~nan & (np.abs(want) < 2.0 ** -126)]) <= 2.0 ** -126).all()


@pytest.mark.parametrize("x", ["bf16", "row", "mx"])
@pytest.mark.parametrize("M", [7, 40])
def test_fp4_bad_token_stays_alone(x, M):
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    gen = torch.Generator().manual_seed(3)
    codes, scales = fp4_weight(gen, 72, 160)
    X, xs, _ = fp4_x(gen, M, 160, x)
    lin = Fp4Linear(codes.cuda(), scales.cuda())
    run = lambda t: (lambda Y: (lin.forward(t.cuda(), Y, None if xs is None else xs.cuda()), Y)[1])(  # noqa: E731
        torch.empty(M, 72, device="cuda"))
    good = run(X)
    bad_x = X.clone()
    bad_x[3, 100] = float("nan") if x == "bf16" else 0x7F
    bad = run(bad_x)
    keep = [i for i in range(M) if i != 3]
    assert torch.equal(good[keep], bad[keep]) and torch.isnan(bad[3]).all()


@pytest.mark.parametrize("K", [32, 96, 160, 480])
@pytest.mark.parametrize("M", [1, 20, 50])
def test_fp4_infinity_in_the_last_block(K, M):
    """An infinite value of X times weights that are not zero is infinite, whatever fills the last
    block of 128 k."""
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    codes = torch.full((40, K // 2), 0x22, dtype=U8)  # ones
    codes[1::2, K // 2 - 1] = 0xA2                    # the last one negative
    X = torch.ones(M, K, dtype=BF16)
    X[M // 2, K - 1] = float("inf")
    Y = torch.empty(M, 40, device="cuda")
    Fp4Linear(codes.cuda(), torch.full((40, K // 32), 127, dtype=U8).cuda()).forward(X.cuda(), Y)
    want = torch.tensor([float(K), float(K - 2)]).repeat(M, 20)
    want[M // 2] = torch.tensor([float("inf"), -float("inf")]).repeat(20)
    assert torch.equal(Y.cpu(), want)


@pytest.mark.parametrize("K,N,pad", [(32, 1, 0), (64, 9, 0), (96, 300, 5), (1056, 77, 0), (2048, 264, 8)])
def test_fp4_quantize(K, N, pad):
    from tensor_transformer_mlp_03_amd import _lib as L
    gen = torch.Generator().manual_seed(K + N)
    W = normal(gen, K, N, dtype=BF16) * torch.exp(2 * normal(gen, 1, N)).bfloat16()
    W[:32, 0] = 0
    if N > 4:
        W[0, 1], W[1, 2], W[2, 3] = float("nan"), float("inf"), 2.0 ** -130
        W[:7, 4] = torch.tensor([6.0, 0.25, 0.75, 1.25, 2.5, 3.5, -5.0])
        W[7:32, 4] = 0
        W[:32, 5] = torch.cat((torch.tensor([3.3e38]), torch.linspace(-1e38, 3e38, 31))).bfloat16()
    Wv = Strided(K, N, BF16, N + pad, pad, W).view
    codes, scales = torch.empty(N, K // 2, dtype=U8, device="cuda"), torch.empty(N, K // 32, dtype=U8, device="cuda")
    L.tpmlp_fp4_quantize(Wv, codes, scales)
    want_c, want_s = OG.e2m1_quantize(f64(W).T.copy())
    assert (scales.cpu().numpy() == want_s).all()
    fine = np.repeat(want_s != 255, 16, 1)
    got = codes.cpu().numpy()
    diff = fine & (got != want_c)
    if diff.any():  # zeros of either sign are one value
        assert (OG.e2m1_values(got)[np.repeat(diff, 2, 1)] == OG.e2m1_values(want_c)[np.repeat(diff, 2, 1)]).all()


@pytest.mark.parametrize("x", ["bf16", "row", "mx"])
@pytest.mark.parametrize("K", [64, 160])
def test_fp4_more_tokens_than_a_launch_takes(x, K):
    """The first and last rows equal those of the rows alone, across the launches' border too."""
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    gen = torch.Generator().manual_seed(K)
    M, N = 16 * 4096 + 37, 24
    codes, scales = fp4_weight(gen, N, K)
    X, xs, _ = fp4_x(gen, M, K, x)
    X, xs = X.cuda(), None if xs is None else xs.cuda()
    lin = Fp4Linear(codes.cuda(), scales.cuda(), "gelu")
    Y = torch.full((M, N), float("nan"), device="cuda")
    lin.forward(X, Y, xs)
    assert torch.isfinite(Y).all()
    for lo, hi in ((0, 50), (16 * 4096 - 20, 16 * 4096 + 20), (M - 30, M)):
        part = torch.empty(hi - lo, N, device="cuda")
        lin.forward(X[lo:hi], part, None if xs is None else xs[lo:hi])
        assert torch.equal(part, Y[lo:hi]), lo


def test_fp4_offsets_past_32_bits():
    """Codes of more than 2^31 bytes: the last rows' products equal those of the rows alone."""
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    N, K = 270336, 16384
    codes = torch.randint(0, 256, (N, K // 2), dtype=U8, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    scales = torch.full((N, K // 32), 120, dtype=U8, device="cuda")
    X = torch.randn(3, K, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    Y = torch.empty(3, N, device="cuda")
    Fp4Linear(codes, scales).forward(X, Y)
    for at in (0, N // 2 - 16, N - 64):
        part = torch.empty(3, 64, device="cuda")
        Fp4Linear(codes[at:at + 64], scales[at:at + 64]).forward(X, part)
        assert torch.equal(part, Y[:, at:at + 64]), at
    gated = torch.empty(3, N // 2, device="cuda")
    Fp4Linear(codes, scales, "relu", gated=True).forward(X, gated)
    assert torch.equal(gated, torch.relu(Y[:, :N // 2]) * Y[:, N // 2:])


# --- streams, graphs, repeated calls -----------------------------------------------------------------------
class Everything:
    """Every call of the gated block once, on its own buffers."""

    def __init__(self, M=37, H=96, F=136):
        from tensor_transformer_mlp_03_amd.block import Edge
        from tensor_transformer_mlp_03_amd.gated import Dropout, Fp4Linear, GatedMLP
        c = {k: v.cuda() for k, v in glu_case(M, H, F).items()}
        e = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.c, self.state = c, state_of(21, 0)
        self.mlp = GatedMLP(c["A"], c["B"])
        self.drop = Dropout(0.2, self.state, 4, torch.full((H,), 0.5, dtype=BF16, device="cuda"))
        self.edge = Edge(H, pre="rms", w_pre=torch.ones(H, device="cuda"))
        self.up, self.down = Fp4Linear.from_weight(c["A"][:H // 32 * 32], "silu", True), Fp4Linear.from_weight(c["B"][:128])
        self.r = torch.randn(M, H, device="cuda", generator=torch.Generator("cuda").manual_seed(8))
        self.out = dict(Z=e(M, H), P=e(M, 2 * F, dtype=BF16), dX=e(M, H), dA=e(H, 2 * F), dB=e(F, H), s=e(M, H), dy=e(M, H, dtype=BF16),
                        db=e(H), codes=e(M, H, dtype=U8), scales=e(M), mx=e(M, H // 32, dtype=U8), codes2=e(M, H, dtype=U8),
                        h=e(M, F, dtype=BF16), h2=e(M, F, dtype=BF16), z=e(M, H))

    def run(self, stream=None):
        o, c, kw = self.out, self.c, dict(stream=stream)
        self.mlp.forward(c["X"], o["Z"], o["P"], **kw)
        self.mlp.backward(c["dZ"], c["X"], o["P"], o["dX"], o["dA"], o["dB"], **kw)
        self.drop.forward(o["Z"], self.r, o["s"], **kw)
        self.drop.backward(o["s"], o["dy"], o["db"], **kw)
        self.edge.forward_fp8(None, o["s"], None, o["codes"], o["scales"], **kw)
        self.edge.forward_fp8(None, o["s"], None, o["codes2"], o["mx"], **kw)
        self.up.forward(o["codes"], o["h"], o["scales"], **kw)
        self.up.forward(o["codes2"], o["h2"], o["mx"], **kw)
        self.down.forward(o["h"][:, :128], o["z"], **kw)

    def take(self):
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in self.out.items()}
        for v in self.out.values():
            v.zero_()
        return got


def same(a, b):
    assert all(torch.equal(a[k], b[k]) for k in a), [k for k in a if not torch.equal(a[k], b[k])]


def test_the_same_bits_twice_and_on_another_stream():
    e = Everything()
    e.run()
    first = e.take()
    assert all(bool(v.float().abs().sum() > 0) for v in first.values())
    e.run()
    same(first, e.take())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        e.run()
    same(first, e.take())
    s.wait_stream(torch.cuda.current_stream())
    e.run(stream=s)
    same(first, e.take())
    e.run(stream=s.cuda_stream)
    same(first, e.take())


def test_in_a_graph():
    """Captured once, replayed with new inputs, the step advanced in the graph, eager work in between."""
    e = Everything()
    e.run()
    e.take()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.run()
        e.state[1].add_(1)
    eager = Everything()
    for i in range(4):
        e.c["X"].copy_(torch.randn(37, 96, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).bfloat16())
        eager.c["X"].copy_(e.c["X"])
        assert int(e.state[1]) == i
        eager.state[1] = i
        eager.run()
        g.replay()
        same(eager.take(), e.take())


def test_graph_outlives_other_sizes():
    """A workspace that a graph writes to stays where it is when a larger call takes another."""
    from tensor_transformer_mlp_03_amd.gated import GatedMLP
    c = {k: v.cuda() for k, v in glu_case(24, 96, 136).items()}
    mlp = GatedMLP(c["A"], c["B"])
    e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    small = [e(24, 96), e(96, 272), e(136, 96)]
    mlp.backward(c["dZ"], c["X"], None, *small)
    want = [t.clone() for t in small]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mlp.backward(c["dZ"], c["X"], None, *small)
    big = {k: v.cuda() for k, v in glu_case(999, 96, 136).items()}
    large = [e(999, 96), e(96, 272), e(136, 96)]
    for _ in range(3):
        mlp.backward(big["dZ"], big["X"], None, *large)
        fill = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]  # would land in a freed workspace
        for t in small:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        del fill
        assert all(torch.equal(a, b) for a, b in zip(small, want))
