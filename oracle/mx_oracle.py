"""Plain oracle of the scored router and of the MXFP4 operators (numpy, fp64).

It shares no code with the CUDA path.  MXFP4 is stated element by element:
the nearest of the eight magnitudes, of two equally near ones the one with
the even code; the scale from the exponent of the block's largest magnitude.
"""
import numpy as np

from . import moe_oracle as O

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


# ---- MXFP4 -------------------------------------------------------------------


def scale_bytes(v):
    """uint8 [..., K/32]: floor(log2 of the block's largest magnitude) - 2 + 127, clamped; 255 with an Inf or NaN."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        a = np.abs(b).max(axis=-1)
        bad = ~np.isfinite(b).all(axis=-1)
        e = np.frexp(np.where(bad, 1.0, a))[1] - 1          # floor(log2 a) of a > 0
    byte = np.clip(e - 2, -127, 127) + 127
    byte = np.where(a == 0, 0, byte)
    return np.where(bad, 255, byte).astype(np.uint8)


def encode(v, byte):
    """uint8 [..., K]: the codes of v under the given scale bytes."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    bad = (byte == 255)[..., None]
    with np.errstate(invalid="ignore", over="ignore"):
        m = np.abs(np.where(bad, 0.0, b)) / np.exp2(byte.astype(np.float64) - 127)[..., None]
    m = np.where(bad, 0.0, m)
    code = np.zeros(m.shape, dtype=np.int64)
    mids = (GRID[1:] + GRID[:-1]) / 2
    for n, mid in enumerate(mids):                          # past the midpoint, or on it with the even code above
        code += (m > mid) | ((m == mid) & (n % 2 == 1))
    code = code + 8 * (np.signbit(b) & ~bad)
    return code.reshape(v.shape).astype(np.uint8)


def quantize(v):
    byte = scale_bytes(v)
    return encode(v, byte), byte


def values(code, byte):
    """fp64 values of codes (one a byte) and scale bytes."""
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(*v.shape[:-1], -1, BLOCK) * s[..., None]).reshape(v.shape)


def rounded(v):
    return values(*quantize(v))


def pack_codes(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack_codes(packed):
    out = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), dtype=np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def scale_at(row, blk, K):
    """Byte of (row, 32-block) in a weight matrix's scale section."""
    tile = (row // 128) * (K // 128) + blk // 4
    return tile * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + blk % 4


def matrix(w):
    """uint8: an MXFP4 weight matrix [N][K]."""
    N, K = w.shape
    code, byte = quantize(w)
    sc = np.empty(N * K // 32, dtype=np.uint8)
    for r in range(N):
        for b in range(K // 32):
            sc[scale_at(r, b, K)] = byte[r, b]
    return np.concatenate([pack_codes(code).reshape(-1), sc])


def gate_up_rows(F):
    """Row of the gate-and-up matrix of gate feature f, and of up feature f."""
    f = np.arange(F)
    return f // 32 * 64 + f % 32, f // 32 * 64 + 32 + f % 32


def ffn_blob(w_gate, w_up, w_down):
    F, d = w_gate.shape
    gu = np.empty((2 * F, d), dtype=w_gate.dtype)
    g, u = gate_up_rows(F)
    gu[g], gu[u] = w_gate, w_up
    return np.concatenate([matrix(gu), matrix(w_down)])


# ---- products ------------------------------------------------------------------


def sum_error(absum, terms):
    """Bound of an fp32 sum of `terms` exact products, in any order and with
    any rounding of the partial sums to 24 bits (each at most 2^-23
    relative): terms 2^-23 times the sum of the magnitudes."""
    return absum * terms * 2.0 ** -23


def product(x, w):
    """(y, bound of its fp32 sum) for fp64 values x [n][K], w [N][K]."""
    return x @ w.T, sum_error(np.abs(x) @ np.abs(w).T, x.shape[1])


def ffn(x, wg, wu, wd):
    """(y, bound) of one expert's FFN on values x [n][d] (all fp64).  The
    bound covers the fp32 sums, the fp32 SwiGLU and what they can do to the
    MXFP4 rounding of h: an element whose possible values straddle a rounding
    point (or whose block's largest magnitude straddles a power of two) may
    land on either side."""
    g, dg = product(x, wg)
    u, du = product(x, wu)
    sg = g / (1 + np.exp(-g))
    h = sg * u
    # |silu'| <= 1.1; exp to (2 + 1.2 |g|) 2^-23 relative, then an addition, a division, a product
    eps = (1.1 * dg * (np.abs(u) + du) + np.abs(sg) * du + np.abs(h) * (6 + 1.2 * np.abs(g)) * 2.0 ** -23)
    q = rounded(h)
    lo, hi = q.copy(), q.copy()
    mag = np.abs(h)
    small = scale_bytes(np.maximum(mag - eps, 0))
    large = scale_bytes(mag + eps)
    for byte in (small, scale_bytes(h), large):
        for v in (h - eps, h + eps):
            c = values(encode(v, byte), byte)
            lo, hi = np.minimum(lo, c), np.maximum(hi, c)
    y, dy = product(np.maximum(np.abs(lo), np.abs(hi)), np.abs(wd))[1], None
    return q @ wd.T, y + (hi - lo) @ np.abs(wd).T


def exact_rows(rng, rows, K, log2_scale=0):
    """Values [rows][K] on the grid times 2^log2_scale, a 6 in every block:
    they are their own MXFP4 form, all scales equal, so that products of two
    such operands are multiples of a quarter of their scales and fp32 sums of
    up to 2^24 / (36 * 4) of them are exact in any order."""
    v = GRID[rng.integers(0, 8, (rows, K // BLOCK, BLOCK))] * rng.choice([-1.0, 1.0], (rows, K // BLOCK, BLOCK))
    at = rng.integers(0, BLOCK, (rows, K // BLOCK, 1))
    np.put_along_axis(v, at, 6.0 * rng.choice([-1.0, 1.0], at.shape), axis=2)
    return v.reshape(rows, K) * 2.0 ** log2_scale


def hidden(x, wg, wu):
    """(q, lo, hi): hq = MXFP4 of silu(x wg) (x wu) for operands whose fp32
    sums are exact, and the least and largest value of each element that the
    fp32 SwiGLU's rounding (as in ffn) can make of it; lo = hi where no
    rounding point is that near."""
    g, u = x @ wg.T, x @ wu.T
    h = g / (1 + np.exp(-g)) * u
    eps = np.abs(h) * (6 + 1.2 * np.abs(g)) * 2.0 ** -23
    q = rounded(h)
    lo, hi = q.copy(), q.copy()
    for byte in (scale_bytes(np.maximum(np.abs(h) - eps, 0)), scale_bytes(np.abs(h) + eps)):
        for v in (h - eps, h + eps):
            c = values(encode(v, byte), byte)
            lo, hi = np.minimum(lo, c), np.maximum(hi, c)
    return q, lo, hi


def half_step(y, dtype_eps, tiny):
    """Half a step of a floating type: eps/2 relative, half the smallest subnormal near zero."""
    return np.abs(y) * dtype_eps / 2 + tiny / 2


# ---- scored router ---------------------------------------------------------------


def scores_of(l, scoring):
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1 / (1 + np.exp(-l))
        p = np.exp(l - l.max(axis=1, keepdims=True))
        return p / p.sum(axis=1, keepdims=True)


def route_scored(x, w_router, k, scoring="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renorm=True,
                 scale=1.0):
    """(idx int32 [T][k], weights fp64 [T][k], scores)."""
    l = O.router_logits(x, w_router)
    s = scores_of(l, scoring)
    with np.errstate(invalid="ignore"):
        c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    if bias is None and (group_top == 1 or topk_groups == n_groups):
        # c rises strictly with l: compare the logits, which neither underflow nor saturate.  (A softmax row with
        # a NaN or an infinite maximum is NaN throughout; a sigmoid of -inf is 0, above what counts as -inf.)
        if scoring == "softmax":
            c = np.where(np.isnan(s).all(axis=1, keepdims=True), -np.inf, l)
        else:
            c = np.where(l == -np.inf, -1.7e308, l)
    c = np.where(np.isnan(c), -np.inf, c)
    T, E = c.shape
    gs = E // n_groups
    idx = np.empty((T, k), dtype=np.int32)
    for t in range(T):
        allowed = np.arange(E)
        if topk_groups < n_groups:
            score = []
            for g in range(n_groups):
                top = np.sort(c[t, g * gs:(g + 1) * gs])[::-1][:group_top]
                score.append(top.sum())
            score = np.array(score)
            score = np.where(np.isnan(score), -np.inf, score)
            kept = np.sort(np.lexsort((np.arange(n_groups), -score))[:topk_groups])
            allowed = np.concatenate([np.arange(g * gs, (g + 1) * gs) for g in kept])
        order = np.lexsort((allowed, -c[t, allowed]))
        idx[t] = allowed[order[:k]]
    w = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if renorm:
        total = w.sum(axis=1, keepdims=True)
        with np.errstate(invalid="ignore", divide="ignore"):
            w = np.where(total == 0, 0.0, w / total)
    return idx, w * scale, s
