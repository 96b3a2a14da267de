"""The float64 oracle of the block operators: its gradients against differences of its
forward, its sort against the definition, and simple exact cases.  CPU only."""
import numpy as np
import pytest

from oracle import block as OB


def _edge(rng, M, H, post, pre, gate_rows):
    p = {}
    for side, kind in (("post", post), ("pre", pre)):
        p["w_" + side] = rng.normal(1, 0.3, H) if kind != "none" else None
        p["b_" + side] = rng.normal(0, 0.3, H) if kind == "layer" else None
    p["gate"] = rng.normal(0.5, 0.3, (-(-M // gate_rows), H)) if gate_rows else None
    return p


@pytest.mark.parametrize("post,pre,rows", [("none", "rms", 0), ("rms", "rms", 5), ("layer", "layer", 2),
                                           ("none", "layer", 1), ("layer", "rms", 3), ("rms", "none", 0)])
def test_edge_gradients_are_differences(post, pre, rows):
    """Central differences of L = <dr', r'> + <dx, x> along a random direction of every input."""
    rng = np.random.default_rng(11)
    M, H, h = 5, 7, 1e-5
    p = _edge(rng, M, H, post, pre, rows)
    kw = dict(post=post, pre=pre, rows=rows, alpha=0.7, eps=1e-3)
    y, r = rng.normal(0, 1, (M, H)), rng.normal(0, 2, (M, H))
    dr, dx = rng.normal(0, 1, (M, H)), rng.normal(0, 1, (M, H))

    def loss(y, r, p):
        f = OB.edge_forward(y, r, **p, **kw)
        return (dr * f["r"]).sum() + ((dx * f["x"]).sum() if f["x"] is not None else 0.0)

    f = OB.edge_forward(y, r, **p, **kw)
    g = OB.edge_backward(y, f["r"], dr, dx if pre != "none" else None, **p, **kw)
    leaves = {"y": (y, g["dy"]), "r": (r, g["dr"]), **{k: (v, g[k]) for k, v in p.items() if v is not None}}
    for name, (v, grad) in leaves.items():
        t = rng.normal(0, 1, v.shape)

        def at(s):
            q = dict(p)
            if name in q:
                q[name] = v + s * t
            return loss(v + s * t if name == "y" else y, v + s * t if name == "r" else r, q)

        want = (at(h) - at(-h)) / (2 * h)
        got = (grad * t).sum()
        assert abs(got - want) <= 1e-7 * (np.abs(grad * t).sum() + 1), (name, got, want)


def test_edge_magnitudes_bound_the_values():
    rng = np.random.default_rng(5)
    M, H = 6, 33
    p = _edge(rng, M, H, "layer", "layer", 4)
    kw = dict(post="layer", pre="layer", rows=4, alpha=-0.5)
    y, r = rng.normal(3, 1, (M, H)), rng.normal(-2, 2, (M, H))
    f = OB.edge_forward(y, r, **p, **kw)
    b = OB.edge_backward(y, f["r"], rng.normal(0, 1, (M, H)), rng.normal(0, 1, (M, H)), **p, **kw)
    for res in (f, b):
        for k in [k for k in res if k + "_mag" in res]:
            assert np.all(np.abs(res[k]) <= res[k + "_mag"] * (1 + 1e-12)), k


def test_sort_small_case():
    ids = np.array([[1, 0], [1, 2], [-1, 1], [3, 0]])  # 3 names no expert
    counts, offsets, row_of, src_of = OB.route_sort(ids, 3, 4, 0)
    assert counts.tolist() == [2, 3, 1] and offsets.tolist() == [0, 4, 8, 12]
    assert row_of.tolist() == [[4, 0], [5, 8], [-1, 6], [-1, 1]]
    assert src_of.tolist()[:12] == [1, 7, -1, -1, 0, 2, 5, -1, 3, -1, -1, -1]
    counts, offsets, row_of, _ = OB.route_sort(ids, 3, 1, 2)
    assert counts.tolist() == [2, 2, 1] and offsets.tolist() == [0, 2, 4, 6]
    assert row_of.tolist() == [[2, 0], [3, 4], [-1, -1], [-1, 1]]


def test_route_gradients_are_transposes():
    """<dY, combine(Zs)> is linear in Zs and in w: its gradients give it back."""
    rng = np.random.default_rng(2)
    T, K, E, H = 9, 3, 4, 5
    ids = rng.integers(-1, E, (T, K))
    _, _, row_of, src_of = OB.route_sort(ids, E, 2, 0)
    rows = src_of.size
    Zs, w, dY = rng.normal(size=(rows, H)), rng.normal(size=(T, K)), rng.normal(size=(T, H))
    Y, _ = OB.route_combine(Zs, row_of, w)
    dZs, dw, _ = OB.route_combine_backward(dY, Zs, row_of, w, rows)
    np.testing.assert_allclose((dY * Y).sum(), (dZs * Zs).sum(), rtol=1e-12)
    np.testing.assert_allclose((dY * Y).sum(), (dw * w).sum(), rtol=1e-12)
    X = rng.normal(size=(T, H))
    dX, _ = OB.route_combine(dZs, row_of, None)
    np.testing.assert_allclose((OB.route_dispatch(X, row_of, rows) * dZs).sum(), (X * dX).sum(), rtol=1e-12)


def test_clip_cases():
    g = [np.array([3.0]), np.array([4.0, 0.0])]
    n, out = OB.clip(g, 10.0)
    assert n == 5.0 and out[0][0] == 3.0
    n, out = OB.clip(g, 1.0, scale=-2.0)
    assert n == 10.0 and np.isclose(out[1][0], -0.8)
    n, out = OB.clip([np.array([np.inf, 1.0])], 1.0)
    assert np.isinf(n) and out[0][1] == 1.0
