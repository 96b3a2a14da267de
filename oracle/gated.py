"""Float64 oracle of the gated block's operators, on the CPU with numpy: the gated MLP, dropout,
E4M3 and E2M1 values with their scales, and products with 4-bit weights.

Written from the definitions in include/tpmlp.h.  Next to each value of the gated MLP stands a
tolerance: its rounding to bf16 (half a step, 2^-8 of the value, wherever the operator rounds
between its products) and float32 sums of n terms in any order (n 2^-24 of the terms' magnitudes),
carried through the products that follow.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24      # half a step of float32, relative
BF = 2.0 ** -8      # half a step of bf16
# The activations' float32 evaluation: GeLU's fit of Phi is within 1.5e-7 (2^-22.6), the others are a
# few operations of an ulp each; relative to |x| + |act(x)|.
ACT = 2.0 ** -20
SLOPE = 1.2         # |act'| and |act''| are below, but for ReLU's step

_erf = np.vectorize(math.erf)


def act(x, kind):
    """(act(x), act'(x))"""
    if kind == "none":
        return x, np.ones_like(x)
    if kind == "relu":
        return np.where(x < 0, 0.0, x), (x > 0).astype(np.float64)
    if kind == "gelu":
        cdf = 0.5 * (1 + _erf(x / math.sqrt(2))) if x.size else x
        return x * cdf, cdf + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-x))
    return (s, s * (1 - s)) if kind == "sigmoid" else (x * s, s * (1 + x * (1 - s)))


def glu_forward(X, A, B, kind):
    """{"P", "Z"} and their tolerances "P_tol", "Z_tol" before the last rounding."""
    H, F = X.shape[1], B.shape[0]
    P, eP = X @ A, (H + 4) * U * (np.abs(X) @ np.abs(A))
    g, u = P[:, :F], P[:, F:]
    a, _ = act(g, kind)
    h = a * u
    eh = np.abs(u) * (SLOPE * eP[:, :F] + ACT * (np.abs(a) + np.abs(g))) + np.abs(a) * eP[:, F:]
    eh = 1.01 * eh + BF * np.abs(h)
    Z = h @ B
    return {"P": P, "P_tol": eP, "Z": Z, "Z_tol": eh @ np.abs(B) + (F + 4) * U * ((np.abs(h) + eh) @ np.abs(B))}


def glu_backward(dZ, X, A, B, P, kind, again=BF):
    """{"dX", "dA", "dB"} and tolerances; P None: made again, and rounded by half a step of `again`."""
    (M, H), F = X.shape, B.shape[0]
    if P is None:
        P = X @ A
        eP = again * np.abs(P) + 1.01 * (H + 4) * U * (np.abs(X) @ np.abs(A))
    else:
        eP = np.zeros_like(P)
    g, u, eg, eu = P[:, :F], P[:, F:], eP[:, :F], eP[:, F:]
    a, da = act(g, kind)
    dh, edh = dZ @ B.T, (H + 4) * U * (np.abs(dZ) @ np.abs(B).T)
    ea = SLOPE * eg + ACT * (np.abs(a) + np.abs(g))
    eda = (np.abs(g) <= eg) * 1.0 if kind == "relu" else SLOPE * eg + ACT * (1 + np.abs(g))
    h, dg, du = a * u, dh * u * da, dh * a
    eh = 1.01 * (np.abs(u) * ea + np.abs(a) * eu) + BF * np.abs(h)
    edg = 1.02 * (np.abs(u * da) * edh + np.abs(dh * da) * eu + np.abs(dh * u) * eda) + BF * np.abs(dg)
    edu = 1.02 * (np.abs(a) * edh + np.abs(dh) * ea) + BF * np.abs(du)
    dP, edP = np.concatenate((dg, du), 1), np.concatenate((edg, edu), 1)

    def product(l, el, r, er, n):
        al, ar = np.abs(l) + el, np.abs(r) + er
        return l @ r, el @ ar + al @ er + (n + 4) * U * (al @ ar)

    zero = np.zeros_like
    out = {}
    out["dB"], out["dB_tol"] = product(h.T, eh.T, dZ, zero(dZ), M)
    out["dA"], out["dA_tol"] = product(X.T, zero(X.T), dP, edP, M)
    out["dX"], out["dX_tol"] = product(dP, edP, A.T, zero(A.T), 2 * F)
    return out


# --- dropout ------------------------------------------------------------------------------------
def philox(counter, key, rounds=10):
    """Philox 4x32 (J. Salmon et al., Parallel random numbers: as easy as 1, 2, 3, 2011): counter four
    and key two arrays of 32-bit values as uint64; four such arrays."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> half) ^ c[1] ^ k[0], p1 & low, (p0 >> half) ^ c[3] ^ k[1], p0 & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return c


def numbers(M, H, seed, step, site, first_row=0):
    """The 16-bit numbers of [M, H] elements."""
    w = lambda v: np.uint64(v & 0xFFFFFFFF)  # noqa: E731
    g, row = np.meshgrid(np.arange(-(-H // 8), dtype=np.uint64), np.arange(M, dtype=np.uint64) + np.uint64(first_row))
    words = philox([g, row, np.full_like(g, w(site)), np.full_like(g, w(step))], [w(seed), w(seed >> 32)])
    n = np.stack([x for v in words for x in (v & np.uint64(0xFFFF), v >> np.uint64(16))], -1)
    return n.reshape(M, -1)[:, :H].astype(np.int64)


def dropout_mask(M, H, p, seed, step, site, first_row=0):
    """0 where the element is dropped, 65536 / (65536 - d) elsewhere."""
    d = int(math.floor(p * 65536 + 0.5))
    return (numbers(M, H, seed, step, site, first_row) >= d) * (65536.0 / (65536 - d) if d < 65536 else 0.0)


# --- E4M3, E2M1 and their scales ------------------------------------------------------------------
def _table(exponent_bits, mantissa_bits, bias):
    """The values of the codes without a sign bit."""
    n, out = 1 << (exponent_bits + mantissa_bits), []
    for c in range(n):
        e, m = c >> mantissa_bits, (c & ((1 << mantissa_bits) - 1)) / (1 << mantissa_bits)
        out.append(math.ldexp(1 + m, e - bias) if e else math.ldexp(m, 1 - bias))
    return np.array(out)


E4M3 = _table(4, 3, 7)
E4M3[127] = np.nan
E2M1 = _table(2, 1, 1)


def e4m3_values(codes):
    codes = np.asarray(codes, dtype=np.int64)
    return np.where(codes >= 128, -1.0, 1.0) * E4M3[codes & 127]


def e2m1_values(codes):
    """[N, K / 2] bytes to [N, K] values, the lower k in the low half."""
    codes = np.asarray(codes, dtype=np.int64)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    return np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]


def mx_exponent(amax, top):
    """The smallest e with amax <= top 2^e (0 where amax is 0), as the byte e + 127."""
    out = np.full(amax.shape, 127, dtype=np.int64)
    m, e = np.frexp(amax)  # amax = m 2^e, m from 0.5 on
    mt, et = math.frexp(top)
    on = amax > 0
    out[on] = np.clip((e - et + (m > mt))[on] + 127, 0, 254)
    return out


def e2m1_quantize(W):
    """Codes [N, K / 2] and scale bytes [N, K / 32] of W[N, K], to nearest, ties to the even code; a block
    with a value that is not finite has scale 255."""
    N, K = W.shape
    g = W.reshape(N, K // 32, 32)
    fine = np.isfinite(g).all(2)
    g = np.where(np.isfinite(g), g, 0.0)
    scale = mx_exponent(np.abs(g).max(2), 6.0)
    v = np.ldexp(g, (127 - scale)[:, :, None])
    d = np.abs(np.abs(v)[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    near = d == best  # one, or two on a tie: the even one
    code = np.where(near.sum(-1) == 1, near.argmax(-1), np.where(near.argmax(-1) % 2 == 0, near.argmax(-1), near.argmax(-1) + 1))
    code = (code + 8 * np.signbit(v)).reshape(N, K // 2, 2)
    return code[:, :, 0] | code[:, :, 1] << 4, np.where(fine, scale, 255)


def mx_values(scales, block=32):
    """Scale bytes [N, B] to factors [N, B * block]; 255 is not a number."""
    s = np.asarray(scales, dtype=np.int64)
    return np.repeat(np.where(s == 255, np.nan, np.ldexp(1.0, s - 127)), block, 1)


def fp4_product(x, codes, scales, kind="none", gated=False):
    """(Y, its tolerance before the last rounding) from x [M, K], the values that X stands for."""
    w = e2m1_values(codes) * mx_values(scales)
    p, ep = x @ w.T, (x.shape[1] + 8) * U * (np.abs(x) @ np.abs(w).T)
    if not gated:
        a, _ = act(p, kind)
        return a, SLOPE * ep + ACT * (np.abs(a) + np.abs(p)) if kind != "none" else ep
    N = p.shape[1] // 2
    g, u = p[:, :N], p[:, N:]
    a, _ = act(g, kind)
    ea = SLOPE * ep[:, :N] + ACT * (np.abs(a) + np.abs(g))
    return a * u, 1.01 * (np.abs(u) * ea + np.abs(a) * ep[:, N:]) + U * np.abs(a * u)
