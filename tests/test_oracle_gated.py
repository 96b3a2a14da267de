"""The float64 oracle of the gated block's operators: its gradients against differences, its random
numbers against the generator's published answers, its formats against their definitions.  CPU only."""
import numpy as np
import pytest

from oracle import gated as OG


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu", "sigmoid"])
def test_glu_gradients_are_differences(kind):
    rng = np.random.default_rng(5)
    M, H, F, h = 5, 6, 7, 1e-6
    t = {"X": rng.normal(0, 1, (M, H)), "A": rng.normal(0, 1, (H, 2 * F)), "B": rng.normal(0, 1, (F, H))}
    dZ = rng.normal(0, 1, (M, H))
    g = OG.glu_backward(dZ, t["X"], t["A"], t["B"], None, kind)
    for name, grad in (("X", "dX"), ("A", "dA"), ("B", "dB")):
        d = rng.normal(0, 1, t[name].shape)
        loss = [float((OG.glu_forward(*(v + s * h * d if k == name else v for k, v in t.items()), kind)["Z"] * dZ).sum())
                for s in (1, -1)]
        assert abs((loss[0] - loss[1]) / (2 * h) - float((g[grad] * d).sum())) <= 1e-6 * (1 + abs(float((g[grad] * d).sum())))


def test_glu_tolerances_hold_a_bf16_evaluation():
    """Rounding to bf16 between the products stays within the tolerances."""
    torch = pytest.importorskip("torch")
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
    X, A, B, dZ = r(9, 32), r(32, 48) * 0.2, r(24, 32) * 0.2, r(9, 32)
    X, A, B, dZ = (t.bfloat16() for t in (X, A, B, dZ))
    n = lambda t: t.double().numpy()  # noqa: E731
    f = OG.glu_forward(n(X), n(A), n(B), "silu")
    P = X.float() @ A.float()
    h = (torch.nn.functional.silu(P[:, :24]) * P[:, 24:]).bfloat16().float()
    assert (np.abs(n(h @ B.float()) - f["Z"]) <= f["Z_tol"]).all()
    Pb = P.bfloat16().float().requires_grad_()
    hb = torch.nn.functional.silu(Pb[:, :24]) * Pb[:, 24:]
    hb.backward(dZ.float() @ B.float().t())
    dP = Pb.grad.bfloat16().float()
    g = OG.glu_backward(n(dZ), n(X), n(A), n(B), None, "silu")
    for name, got in (("dX", dP @ A.float().t()), ("dA", X.float().t() @ dP), ("dB", hb.detach().bfloat16().float().t() @ dZ.float())):
        assert (np.abs(n(got) - g[name]) <= g[name + "_tol"]).all(), name


def test_philox_answers():
    """The generator's published answers for ten rounds: all zeros and all ones."""
    z = np.zeros(1, dtype=np.uint64)
    assert [int(v[0]) for v in OG.philox([z] * 4, [z] * 2)] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    o = z + np.uint64(0xFFFFFFFF)
    assert [int(v[0]) for v in OG.philox([o] * 4, [o] * 2)] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_numbers_are_uniform_and_apart():
    n = OG.numbers(256, 256, 12345, 1, 0)
    assert abs(n.mean() / 65536 - 0.5) < 0.01 and abs((n < 6554).mean() - 0.1) < 0.01
    for other in (OG.numbers(256, 256, 12346, 1, 0), OG.numbers(256, 256, 12345, 2, 0), OG.numbers(256, 256, 12345, 1, 1)):
        assert (n == other).mean() < 0.001
    assert (OG.numbers(16, 256, 12345, 1, 0, first_row=100) == n[100:116]).all()  # a rank's rows
    assert (OG.dropout_mask(4, 9, 0.0, 1, 1, 1) == 1).all() and (OG.dropout_mask(4, 9, 1.0, 1, 1, 1) == 0).all()


def test_formats():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = OG.e4m3_values(codes.numpy())
    assert ((got == want) | (np.isnan(got) & np.isnan(want))).all()
    assert OG.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert OG.mx_exponent(np.array([0.0, 448.0, 449.0, 224.0, 1e-45]), 448.0).tolist() == [127, 127, 128, 126, 0]


def test_e2m1_quantize():
    rng = np.random.default_rng(1)
    W = rng.normal(0, 1, (7, 96)) * np.exp(rng.normal(0, 3, (7, 1)))
    codes, scales = OG.e2m1_quantize(W)
    s = OG.mx_values(scales)
    v = OG.e2m1_values(codes) * s
    amax = np.abs(W.reshape(7, 3, 32)).max(2).repeat(32, 1)
    assert (amax <= 6 * s).all() and (amax > 3 * s).all()
    step = np.where(np.abs(W) / s < 2, 0.5, np.where(np.abs(W) / s < 4, 1, 2)) * s
    assert (np.abs(v - W) <= step / 2).all()
    ties = np.zeros((1, 32))
    ties[0, :9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, 6.0]
    got = OG.e2m1_values(OG.e2m1_quantize(ties)[0])[0, :9]
    assert got.tolist() == [0, 1, 1, 2, 2, 4, 4, 0, 6]
