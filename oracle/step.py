"""The MoE step around the GEMMs: tokens to the experts' rows and back, the row
cast, the experts' forward product and AdamW with FP32 or 8-bit moments.

Test infrastructure only (see the package docstring).  Sums are in float64;
where the definition fixes FP32 steps (the row cast's scale and quotient, the
8-bit moments' new values, from which codes are decided) they are numpy
float32 operations in the defined order.
"""
import numpy as np

from .e4m3 import e4m3_decode, e4m3_encode
from .wgrad import FP32_REL

F = np.float32


def moe_sort(idx, G, align):
    """(counts, row_of_pair, pair_rows): one pair after the other in order."""
    idx = np.asarray(idx)
    T, topk = idx.shape
    flat = idx.reshape(-1)
    used = (flat >= 0) & (flat < G)
    n_e = np.bincount(flat[used], minlength=G)
    counts = -(-n_e // align) * align
    nxt = np.concatenate([[0], np.cumsum(counts)[:-1]])
    rows = np.full(T * topk, -1, np.int64)
    pairs = np.full(T * topk + G * (align - 1), -1, np.int64)
    for i in np.nonzero(used)[0]:
        rows[i] = nxt[flat[i]]
        pairs[rows[i]] = i
        nxt[flat[i]] += 1
    return counts, rows.reshape(T, topk), pairs


def moe_dispatch(x, rows, R):
    xs = np.zeros((R, x.shape[1]), np.asarray(x).dtype)
    for t, j in np.argwhere(rows >= 0):
        xs[rows[t, j]] = x[t]
    return xs


def moe_combine(ye, rows, w=None):
    """(y, S) with S = sum |w ye|, in float64."""
    ye = np.asarray(ye, np.float64)
    y = np.zeros((rows.shape[0], ye.shape[1]))
    S = np.zeros_like(y)
    for j in range(rows.shape[1]):
        t = np.nonzero(rows[:, j] >= 0)[0]
        v = ye[rows[t, j]] * (1.0 if w is None else np.asarray(w, np.float64)[t, j, None])
        y[t] += v
        S[t] += np.abs(v)
    return y, S


def moe_combine_backward(dy, ye, rows, w, R):
    """(dye, dw, Sw) with Sw = sum |dy ye|, in float64."""
    dy, ye, w = (np.asarray(v, np.float64) for v in (dy, ye, w))
    dye = np.zeros((R, dy.shape[1]))
    dw, Sw = np.zeros(rows.shape), np.zeros(rows.shape)
    for j in range(rows.shape[1]):
        t = np.nonzero(rows[:, j] >= 0)[0]
        dye[rows[t, j]] = w[t, j, None] * dy[t]
        prod = dy[t] * ye[rows[t, j]]
        dw[t, j], Sw[t, j] = prod.sum(1), np.abs(prod).sum(1)
    return dye, dw, Sw


ROW_FLOOR = F(2.0 ** -100) * (F(1) / F(448))


def quant_rows(x):
    """(codes [T, C], scales [T, ceil(C / 128)]) of the row cast."""
    x = np.asarray(x, F)
    T, C = x.shape
    nb = -(-C // 128)
    q, s = np.zeros((T, C), np.uint8), np.zeros((T, nb), F)
    for b in range(nb):
        v = x[:, b * 128:(b + 1) * 128]
        s[:, b] = np.maximum(np.abs(v).max(1), F(2.0 ** -100)) * (F(1) / F(448))
        q[:, b * 128:(b + 1) * 128] = e4m3_encode(v * (F(1) / s[:, b])[:, None])
    return q, s


def mgrouped_fp8_linear(x, sx, w, sw, ms):
    """(y, S) of the rows of every expert, in float64."""
    G, N, K = w.shape
    rep = lambda v, axis, n: np.take(np.repeat(np.asarray(v, np.float64), 128, axis),  # noqa: E731
                                     np.arange(n), axis)
    xd = e4m3_decode(x) * rep(sx, 1, K)
    y, S, at = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], N)), 0
    for e in range(G):
        if ms[e]:
            wd = e4m3_decode(w[e]) * rep(rep(sw[e], 0, N), 1, K)
            y[at:at + ms[e]] = xd[at:at + ms[e]] @ wd.T
            S[at:at + ms[e]] = np.abs(xd[at:at + ms[e]]) @ np.abs(wd).T
        at += ms[e]
    return y, S


def linear_bound(y, S):
    """Half a BF16 ulp, and the FP32 sums' share of S (block sums in the tensor
    core, as for the other products)."""
    return (2.0 ** -8) * 1.001 * np.abs(y) + FP32_REL * S


# ------------------------------------------------------------------ AdamW
def element_bits(n, seed, tensor, start=0):
    """32 bits of each element from its index, the seed and the tensor's place."""
    M = 0xFFFFFFFF
    key = (((seed ^ (seed >> 32)) & M) * 0x9E3779B9 + tensor * 0xBB67AE85) & M
    i = np.arange(start, start + n, dtype=np.uint64)
    h = ((i + np.uint64(key)) & np.uint64(M)) * np.uint64(0x9E3779B9) & np.uint64(M)
    h ^= (h >> np.uint64(16)) ^ np.uint64((key >> 16 | key << 16) & M)
    h = h * np.uint64(0x6A09E667) & np.uint64(M)
    return h ^ (h >> np.uint64(15))


def _blocks(v):
    n = -(-v.size // 128) * 128
    return np.concatenate([v, np.zeros(n - v.size, v.dtype)]).reshape(-1, 128)


def moment_decode(codes, scales):
    """float64 values of E4M3 codes with a UE8M0 scale per 128 elements."""
    v = e4m3_decode(_blocks(np.asarray(codes, np.uint8)))
    return (v * np.ldexp(1.0, np.asarray(scales, np.int64) - 127)[:, None]).reshape(-1)[:len(codes)]


def moment_encode(x, bits16, keep):
    """(codes, scales) of float32 moments: rounded up with probability of the
    part cut off, as bits16 / 2^16 decides; keep: above zero stays above zero.
    A code has its moment's sign, zeros included; what is not finite is 0x7F."""
    x = np.asarray(x, F)
    fin = np.isfinite(x)
    b = np.abs(_blocks(np.where(fin, x, F(0)))).astype(np.float64)
    amax = b.max(1)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(amax / 448))
        # log2 near a power of two: settle the smallest e with amax <= 448 * 2^e
        e = np.where(amax > 0, e, -127)
        e = np.where(amax > 448 * np.exp2(e), e + 1, e)
        e = np.where((amax > 0) & (amax <= 448 * np.exp2(e - 1)), e - 1, e)
    e = np.maximum(e, -127)
    y = b / np.exp2(e)[:, None]
    step = np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    # below 2^-6 the definition adds 2^-6 in FP32 first
    low = (y.astype(F) + F(2.0 ** -6)).astype(np.float64) - 2.0 ** -6
    y = np.where(y < 2.0 ** -6, low, y)
    u = _blocks(np.asarray(bits16).astype(np.int64)) / 65536
    q = np.floor(y / step + u) * step
    if keep:
        q = np.where((q == 0) & (b > 0), 2.0 ** -9, q)
    code = e4m3_encode(q).reshape(-1)[:x.size]
    code = np.where(np.signbit(x) & fin, code | 0x80, code)
    return np.where(fin, code, 0x7F).astype(np.uint8), (e + 127).astype(np.uint8)


def adamw(p, g, m, v, step, lr, b1, b2, eps, wd, gs=1.0):
    """FP32 (m', v', r') by the defined steps, and float64 (p', bound) where
    bound limits what FP32 may make of p'.  m, v: the held moments' values."""
    p64, g = np.asarray(p, np.float64), np.asarray(g, F) * F(gs)
    m0, v0 = np.asarray(m, F), np.asarray(v, F)
    m1 = F(b1) * m0 + F(1 - b1) * g
    v1 = F(b2) * v0 + F(1 - b2) * (g * g)
    c1, c2 = lr / (1 - b1 ** step), 1 / np.sqrt(1 - b2 ** step)
    g64, m64, v64 = g.astype(np.float64), m0.astype(np.float64), v0.astype(np.float64)
    den = np.sqrt(b2 * v64 + (1 - b2) * g64 ** 2) * c2 + eps
    big = c1 * (np.abs(b1 * m64) + np.abs((1 - b1) * g64)) / den
    new = p64 * (1 - lr * wd) - c1 * (b1 * m64 + (1 - b1) * g64) / den
    # three roundings of p; the update: its constants, three roundings of each
    # moment (half as much in r), the quotient's 2 ulp -- 16 half-ulps at most
    return m1, v1, np.sqrt(v1), new, 2.0 ** -22 * np.abs(p64) + 2.0 ** -20 * big + 1e-30
