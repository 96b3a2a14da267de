"""Float64 oracle of the block operators, on the CPU with numpy: the edge between two
blocks, the route of tokens to experts and back, and the clipping of gradients.

Written from the definitions in include/tpmlp.h.  Next to each value stands a
*magnitude*: the same expression with every term taken positive, so that the rounding
error of any float32 evaluation in any order is at most a small multiple of
2^-24 times it, however much the terms cancel.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of float32, relative


def norm(v, kind, w, b, eps):
    """(N(v), normalised v, its magnitude, 1 / deviation) along the last axis."""
    if kind == "none":
        return v, v, np.abs(v), None
    mean = v.mean(-1, keepdims=True) if kind == "layer" else 0.0
    c = v - mean
    rstd = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    hat = c * rstd
    # the mean is itself a rounded sum of H terms, each as large as |v| is on average
    size = (np.abs(v) + (np.abs(v).mean(-1, keepdims=True) if kind == "layer" else 0.0)) * rstd
    n = hat * w
    return (n + b if b is not None else n), hat, size, rstd


def gate_rows(gate, rows, M):
    """The gate's row of each token [M,H]."""
    return np.repeat(gate, rows, 0)[:M] if gate.shape[0] > 1 or rows < M else np.broadcast_to(gate, (M, gate.shape[1]))


def _abs(v):
    return 0.0 if v is None else np.abs(v)


def edge_forward(y, r, post="none", pre="none", w_post=None, b_post=None, w_pre=None, b_pre=None, gate=None, rows=0,
                 alpha=1.0, eps=1e-5):
    """{"r": r', "x": x, "r_mag", "x_mag"} (x None without a norm before the next block)."""
    out, mag = alpha * r, np.abs(alpha * r)
    if y is not None:
        n, _, size, _ = norm(y, post, w_post, b_post, eps)
        m = size * (1.0 if w_post is None else np.abs(w_post)) + _abs(b_post)
        g = 1.0 if gate is None else gate_rows(gate, rows, r.shape[0])
        out, mag = out + g * n, mag + np.abs(g) * m
    res = {"r": out, "r_mag": mag, "x": None, "x_mag": None}
    if pre != "none":
        x, hat, size, rstd = norm(out, pre, w_pre, b_pre, eps)
        # r' carries an error of up to mag: through the row's statistics and directly
        err = mag + mag.mean(-1, keepdims=True) + np.abs(hat) * (np.abs(hat) * mag).mean(-1, keepdims=True)
        res["x"], res["x_mag"] = x, (size + rstd * err) * np.abs(w_pre) + _abs(b_pre)
    return res


def edge_backward(y, r_out, dr_out, dx, post="none", pre="none", w_post=None, b_post=None, w_pre=None, b_pre=None,
                  gate=None, rows=0, alpha=1.0, eps=1e-5):
    """Gradients {"dr", "dy", "w_post", "b_post", "w_pre", "b_pre", "gate"} of those that exist, and
    their magnitudes under "<name>_mag"."""
    some = next(t for t in (dr_out, dx) if t is not None)
    M, H = some.shape
    d = np.zeros((M, H)) if dr_out is None else dr_out.astype(np.float64)
    mag = np.abs(d)
    res = {}

    def back(u, um, hat, size, rstd, kind):
        mean = u.mean(-1, keepdims=True) if kind == "layer" else 0.0
        mean_m = um.mean(-1, keepdims=True) if kind == "layer" else 0.0
        g = rstd * (u - mean - hat * (u * hat).mean(-1, keepdims=True))
        return g, rstd * (um + mean_m + size * (um * size).mean(-1, keepdims=True))

    if pre != "none":
        _, hat, size, rstd = norm(r_out, pre, w_pre, b_pre, eps)
        g, gm = back(dx * w_pre, np.abs(dx * w_pre), hat, size, rstd, pre)
        d, mag = d + g, mag + gm
        res["w_pre"], res["w_pre_mag"] = (dx * hat).sum(0), (np.abs(dx) * size).sum(0)
        if b_pre is not None:
            res["b_pre"], res["b_pre_mag"] = dx.sum(0), np.abs(dx).sum(0)
    res["dr"], res["dr_mag"] = alpha * d, np.abs(alpha) * mag
    if y is None:
        return res
    n, hat, size, rstd = norm(y, post, w_post, b_post, eps)
    g = np.ones((M, H)) if gate is None else gate_rows(gate, rows, M)
    dn, dnm = g * d, np.abs(g) * mag
    if post == "none":
        res["dy"], res["dy_mag"] = dn, dnm
        nm = np.abs(y)
    else:
        res["dy"], res["dy_mag"] = back(dn * w_post, dnm * np.abs(w_post), hat, size, rstd, post)
        res["w_post"], res["w_post_mag"] = (dn * hat).sum(0), (dnm * size).sum(0)
        nm = size * np.abs(w_post) + _abs(b_post)
        if b_post is not None:
            res["b_post"], res["b_post_mag"] = dn.sum(0), dnm.sum(0)
    if gate is not None:
        cut = np.arange(0, M, rows)
        res["gate"] = np.add.reduceat(d * n, cut, 0)
        res["gate_mag"] = np.add.reduceat(mag * nm, cut, 0)
    return res


def route_rows(T, K, E, align, capacity):
    if capacity:
        return E * capacity
    return (T * K + min(E, T * K) * (align - 1)) // align * align


def route_sort(ids, E, align, capacity):
    """(counts, offsets, row_of, src_of) by walking the pairs in order."""
    T, K = ids.shape
    rows = route_rows(T, K, E, align, capacity)
    held = [[] for _ in range(E)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E and not (capacity and len(held[e]) >= capacity):
            held[e].append(p)
    offsets, row_of, src_of = [0], np.full(T * K, -1, np.int32), np.full(rows, -1, np.int32)
    for e in range(E):
        for i, p in enumerate(held[e]):
            row_of[p] = offsets[e] + i
            src_of[offsets[e] + i] = p
        offsets.append(offsets[e] + (capacity or -(-len(held[e]) // align) * align))
    return (np.array([len(h) for h in held], np.int32), np.array(offsets, np.int32), row_of.reshape(T, K), src_of)


def route_dispatch(X, row_of, rows):
    Xs = np.zeros((rows, X.shape[1]))
    for k in range(row_of.shape[1]):
        on = row_of[:, k] >= 0
        Xs[row_of[on, k]] = X[on]
    return Xs


def route_combine(Zs, row_of, w):
    """(Y, magnitude); w None: ones."""
    T, K = row_of.shape
    Y, mag = np.zeros((T, Zs.shape[1])), np.zeros((T, Zs.shape[1]))
    for k in range(K):
        on = row_of[:, k] >= 0
        term = Zs[row_of[on, k]] * (1.0 if w is None else w[on, k:k + 1])
        Y[on] += term
        mag[on] += np.abs(term)
    return Y, mag


def route_combine_backward(dY, Zs, row_of, w, rows):
    """(dZs, dw, magnitude of dw)."""
    T, K = row_of.shape
    dZs, dw, mag = np.zeros((rows, dY.shape[1])), np.zeros((T, K)), np.zeros((T, K))
    for k in range(K):
        on = row_of[:, k] >= 0
        dZs[row_of[on, k]] = dY[on] * (1.0 if w is None else w[on, k:k + 1])
        dw[on, k] = (dY[on] * Zs[row_of[on, k]]).sum(1)
        mag[on, k] = np.abs(dY[on] * Zs[row_of[on, k]]).sum(1)
    return dZs, dw, mag


def clip(grads, max_norm, scale=1.0):
    """(norm, scaled gradients)."""
    total = abs(scale) * np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    c = max_norm / total if np.isfinite(total) and total > max_norm else 1.0
    return total, [g.astype(np.float64) * (scale * c) for g in grads]
