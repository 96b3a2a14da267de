"""Which kernels a call of the gated MLP takes: the library's planner (plan_gemm in csrc/tpmlp.hip, plan_glu_fwd and
plan_glu_bwd in csrc/glu.hip) written again, so that a test can say which of its paths a size is meant for.
test_glu_plans.py holds it against the workspaces that the library asks for."""
from collections import namedtuple

CU, BK, ALIGN = 256, 64, 256
RATE = {(256, 256): 4.3e12, (256, 128): 3.8e12, (128, 128): 3.3e12}
SPLIT_BW, LAUNCH = 4.0e12, 5e-6

Gemm = namedtuple("Gemm", "tile splits k_split n_full seconds")


def ceil(a, b):
    return -(-a // b)


def up(n, to=ALIGN):
    return ceil(n, to) * to


def gemm(M, N, K, hybrid=True, min_slice=512):
    best, least = None, 1e30
    for (bm, bn), rate in RATE.items():
        tiles = ceil(M, bm) * ceil(N, bn)
        for s in range(1, 17):
            k = up(ceil(K, s), BK)
            if ceil(K, k) != s:
                continue
            if s > 1 and k < min_slice:
                break
            t = float(ceil(tiles * s, CU)) * float(bm * bn * 2 * k) / rate
            if s > 1:
                t += float(s) * M * N * 4 * 2 / SPLIT_BW + LAUNCH
            if t < least * (1 - 1e-9):
                best, least = Gemm((bm, bn), s, k, 0, t), t
    tm, tn = ceil(M, 256), ceil(N, 256)
    c = tn - 1
    while c > 0 and tm * c % CU:
        c -= 1
    if hybrid and tm * tn > CU and c > 0:
        nt = N - 256 * c
        full = float(tm * c // CU) * float(256 * 256 * 2 * up(K, BK)) / 4.3e12
        for s in range(2, 17):
            k = up(ceil(K, s), BK)
            if ceil(K, k) != s:
                continue
            if k < 512:
                break
            t = full + float(ceil(tm * (tn - c) * s, CU)) * float(256 * 256 * 2 * k) / 4.3e12
            t += float(s) * M * nt * 4 * 2 / SPLIT_BW + 2 * LAUNCH
            if t < least * (1 - 1e-9):
                best, least = Gemm((256, 256), s, k, 256 * c, t), t
    return best


def part(p, M, N):
    return p.splits * M * (N - p.n_full) * 4 if p.splits > 1 else 0


def transposed(M, H, F, products, elements):
    """Whether transposing `elements` of bf16 first pays for this many products of 2 M H F."""
    return products * 2.0 * float(M) * H * F * (1 / 1.14e15 - 1 / 1.2e15) > 1.5 * (4.0 * float(elements) / 5.5e12)


def tokens(M, N, K):
    """(rows of a wave, slices) of a few tokens' product."""
    mt = M if M < 3 else 4
    groups, most = ceil(N, 128), 8192 // mt // 8 // 32 * 32

    def rows_for(blocks):
        return min(most, up(ceil(K, ceil(blocks, groups) * 8), 32))

    rows = max(rows_for(4 * CU), min(64, rows_for(CU)))
    return rows, ceil(K, rows * 8)


def forward(M, H, F):
    """{"tokens": ...} or {"h", "Z": Gemm, "wt"}, and "bytes"."""
    if M <= 2 or (M <= 4 and H * F <= 1 << 24):
        a, b = tokens(M, 2 * F, H), tokens(M, H, F)
        return dict(tokens=(a, b), bytes=up(a[1] * M * F * 8) + up(b[1] * M * H * 4))
    h, z = gemm(M, 2 * F, H, False, 256), gemm(M, H, F, True, 256)
    wt = transposed(M, H, F, 2, H * F)
    n = up(M * F * 2) + (up(H * F * 4) + up(H * F * 2) if wt else 0)
    return dict(tokens=None, h=h, Z=z, wt=wt, bytes=n + up(max(part(h, M, 2 * F), part(z, M, H))))


def makespan(n0, k0, n1, k1):
    """Steps until workgroups handed to free CUs in their order are done: n0 of k0, then n1 of k1."""
    q, r = divmod(n0, CU)
    t0 = q * k0
    t1 = t0 + k0 if r else t0
    if n1 == 0:
        return float(t1)
    lo, hi = t0, t1 + ceil(n1, CU) * k1
    while lo < hi:
        mid = (lo + hi) // 2
        done = (CU - r) * max(0, (mid - t0) // k1 if mid >= t0 else 0) + r * max(0, (mid - t1) // k1 if mid >= t1 else 0)
        lo, hi = (mid + 1, hi) if done < n1 else (lo, mid)
    return float(max(lo, t1))


def group(M, H, F, seconds):
    """(slices of dX, of dB and dA) of the launch that makes all three, or None."""
    tm, th, tf, t2f = (ceil(n, 128) for n in (M, H, F, 2 * F))
    n0, n1, k0, k1 = tm * th, tf * th + th * t2f, ceil(2 * F, BK), ceil(M, BK)
    if n0 + n1 > 8 * CU:
        return None
    best, least = None, seconds + 2 * LAUNCH
    step = 128.0 * 128 * 2 * BK / 3.3e12
    for sx in (1, 2, 3, 4, 6, 8, 12, 16):
        kx = ceil(k0, sx)
        if (sx > 1 and kx < 8) or ceil(k0, kx) != sx:
            continue
        for sw in (1, 2, 4, 8, 16):
            kw = ceil(k1, sw)
            if (sw > 1 and kw < 8) or ceil(k1, kw) != sw:
                continue
            x, w = (n0 * sx, kx + 3), (n1 * sw, kw + 3)
            t = step * (makespan(*x, *w) if kx >= kw else makespan(*w, *x))
            if sx > 1 or sw > 1:
                t += ((float(sx) * M * H if sx > 1 else 0) + (float(sw) * 3 * H * F if sw > 1 else 0)) * 4 * 2 / SPLIT_BW + LAUNCH
            if t < least * (1 - 1e-9):
                best, least = (sx, sw), t
    return best


def backward(M, H, F, recompute):
    """The products P, dh, dB, dA, dX, the "group" (None: a launch each), the transposes "wt" (A for P), "tdp"
    (dP for dA), "tdz" (dZ for dB) and "beside" (X's with dh), and "bytes"."""
    M8 = up(M, 8)
    p = dict(P=gemm(M, 2 * F, H), dh=gemm(M, F, H, False), dB=gemm(F, H, M), dA=gemm(H, 2 * F, M), dX=gemm(M, H, 2 * F))
    p["group"] = g = group(M, H, F, p["dB"].seconds + p["dA"].seconds + p["dX"].seconds)
    large = float(M) * H * F * 4.4e-17 * 2 > LAUNCH
    p["wt"] = recompute and transposed(M, H, F, 2, H * F)
    p["tdp"] = not g and large and transposed(M, H, F, 1, M * F)
    p["tdz"] = not g and large and transposed(M, F, H, 1, M * H)
    tiles = ceil(M, 128) * ceil(F, 128) * p["dh"].splits
    p["beside"] = not p["tdz"] and p["dh"].tile == (128, 128) and tiles + ceil(M, 256) * ceil(H, 64) <= CU
    mh, mf, m2f = up(M8 * H * 2), up(M8 * F * 2), up(M8 * F * 4)
    n = mh * (2 if p["tdz"] else 1) + (up(H * F * 4) if p["wt"] else 0) + (2 * m2f if recompute else 0) + mf + m2f + (m2f if p["tdp"] else 0)
    slices = [part(p["P"], M, 2 * F) if recompute else 0, part(p["dh"], M, F)]
    if g:
        slices.append((g[0] * M * H * 4 if g[0] > 1 else 0) + (g[1] * 3 * H * F * 4 if g[1] > 1 else 0))
    else:
        slices += [part(p["dB"], F, H), part(p["dA"], H, 2 * F), part(p["dX"], M, H)]
    p["bytes"] = n + up(max(slices))
    return p


def kind(p):
    return "hybrid" if p.n_full else "split" if p.splits > 1 else "%dx%d" % p.tile


def taken(M, H, F):
    """The kernels that a forward and both backwards of this size take, with H long enough for several turns of the
    GEMM's ring of slots: (product, how it is tiled or split, layout of its second operand)."""
    out, f = set(), forward(M, H, F)
    if not f["tokens"]:
        lay = "KC" if f["wt"] else "MC"
        out |= {("h", kind(f["h"]), lay), ("Z", kind(f["Z"]), lay)}
    for recompute in (False, True):
        b = backward(M, H, F, recompute)
        if recompute:
            out.add(("P", kind(b["P"]), "KC" if b["wt"] else "MC"))
        out.add(("dh", ("beside " if b["beside"] else "") + kind(b["dh"]), "KC"))
        if not b["group"]:
            out |= {("dB", kind(b["dB"]), "KC" if b["tdz"] else "MC"), ("dA", kind(b["dA"]), "KC" if b["tdp"] else "MC"),
                    ("dX", kind(b["dX"]), "KC")}
            if recompute:
                out.add(("each product by itself", "P made again", ""))
    return out


TILED, ALSO_SPLIT = ("128x128", "256x128", "256x256"), ("split", "hybrid")
# Everything that `taken` can say but for the launch of three products, which small sizes take.
PLANS = ({(p, k, lay) for p in ("P", "Z", "dA", "dB") for k in TILED + ALSO_SPLIT for lay in ("KC", "MC")} |
         {("dX", k, "KC") for k in TILED + ALSO_SPLIT} | {("h", k, lay) for k in TILED + ("split",) for lay in ("KC", "MC")} |
         {("dh", k, "KC") for k in TILED + ("split", "beside 128x128", "beside split")} |
         {("each product by itself", "P made again", "")})
# Training sizes, then sizes found by search, with a number of tokens that is no multiple of 8 and H from 700 on,
# that reach the rest of PLANS.
LARGE = [(2048, 4096, 4096), (4096, 1024, 4096), (2041, 4096, 4096), (2048, 20480, 10240),
         (9, 1072, 13224), (23999, 1680, 8), (6607, 1168, 8), (16781, 808, 72), (5521, 2224, 344), (9, 968, 8), (6487, 816, 12440),
         (16153, 1072, 2056), (3191, 18400, 968), (1167, 3736, 13040), (2505, 1272, 17864), (6637, 12920, 664), (11055, 16696, 320),
         (5637, 16240, 656), (1303, 3096, 16320), (11061, 720, 12904)]
