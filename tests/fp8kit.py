"""E4M3 blocks of 128, products, experts and routing by scores in numpy, 64 bits, from the definitions: the plain forms the
GPU tests compare with."""
import numpy as np

TOP = 448.0
BLOCK = 128


def _table():
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = -mag if c & 128 else mag
    v[127] = v[255] = np.nan
    return v


VALUES = _table()          # of the 256 codes
GRID = VALUES[:127]        # the magnitudes, ascending


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def spread(scales, block_rows, rows, K):
    """A scale per element."""
    return np.repeat(np.repeat(scales, block_rows, axis=0)[:rows], BLOCK, axis=1)[:, :K]


def nearest(u):
    """Codes 0 .. 126 of magnitudes u: the nearest of the grid, ties to the even code, beyond 448 to 448."""
    i = np.searchsorted(GRID, u, side="right") - 1
    i = np.clip(i, 0, 126)
    j = np.minimum(i + 1, 126)
    low, high = u - GRID[i], GRID[j] - u
    up = (high < low) | ((high == low) & (i % 2 == 1))
    return np.where(up & (j > i), j, i)


def scale_of(top, rule):
    """Scales (float32) of blocks with largest magnitudes top."""
    out = np.empty(top.shape, np.float32)
    for at, t in np.ndenumerate(top):
        if not np.isfinite(t):
            out[at] = np.nan
        elif t == 0:
            out[at] = 1.0
        elif rule == "amax":
            out[at] = max(np.float32(np.float64(t) / TOP), np.float32(2.0 ** -126))
        else:
            e = int(np.frexp(t / TOP)[1])
            if 2.0 ** (e - 1) >= t / TOP:
                e -= 1
            out[at] = 2.0 ** max(e, -126)
    return out


def tops(x, block_rows):
    rows, K = x.shape
    R, C = -(-rows // block_rows), blocks(K)
    full = np.zeros((R * block_rows, C * BLOCK))
    full[:rows, :K] = np.abs(x)
    return full.reshape(R, block_rows, C, BLOCK).max(axis=(1, 3))  # a NaN stays


def quantise(x, block_rows=1, rule="amax"):
    """(codes uint8, scales float32) of x (float64 holding the input's values exactly)."""
    rows, K = x.shape
    t = tops(x, block_rows)
    s = scale_of(t, rule)
    per = spread(s.astype(np.float64), block_rows, rows, K)
    bad = np.isnan(per)
    with np.errstate(invalid="ignore"):
        u = np.where(bad, 0.0, np.abs(x) / np.where(bad, 1.0, per))
    codes = nearest(np.nan_to_num(u)) + 128 * np.signbit(x)
    return np.where(bad, 0, codes).astype(np.uint8), s


def values(codes, scales, block_rows):
    rows, K = codes.shape
    return VALUES[codes] * spread(scales.astype(np.float64), block_rows, rows, K)


def padded(scales):
    """Scale rows as the product takes them: a multiple of 16 bytes long, NaN behind the row."""
    out = np.full((scales.shape[0], (scales.shape[1] + 3) // 4 * 4), np.nan, np.float32)
    out[:, :scales.shape[1]] = scales
    return out


def cores_error(cores):
    """What the FP8 matrix cores' cutting adds, relative to the sum of the terms' magnitudes: of 8 products the seven others
    lose less than 2^-13 of the largest each."""
    return 7 * 2.0 ** -13 if cores else 0.0


def sum_error(K):
    """How far a product of K columns may be off, relative to the sum of its terms' magnitudes: per block of 128, each of
    up to 128 additions of exact products rounds or truncates one partial sum (2^-23); the product of the two scales and
    the fused add of each block round once (2^-24 each, as many as blocks), and joining up to 16 partial sums as often."""
    return (min(K, BLOCK) + (blocks(K) + 17) / 2) * 2.0 ** -23


# ------------------------------------------------------------------ experts
def slab(parts):
    """The bytes of a slab from [(codes, scales)] of W1, W3, W2."""
    b = np.concatenate([c.reshape(-1) for c, _ in parts] + [s.astype(np.float32).reshape(-1).view(np.uint8)
                                                            for _, s in parts])
    return np.concatenate([b, np.zeros(-len(b) % 16, np.uint8)])


def feed_forward(x, parts):
    """(y, how far it may be off) for rows x (already quantised values) of one expert.  The error is that of the sums and
    of the codes of h that such an error may move."""
    w1, w3, w2 = (values(c, s, 128) for c, s in parts)
    H, I = x.shape[1], w1.shape[0]
    g, u = x @ w1.T, x @ w3.T
    eg, eu = (np.abs(x) @ np.abs(w).T * sum_error(H) for w in (w1, w3))
    with np.errstate(over="ignore"):
        sg = g / (1 + np.exp(-g))
    h = sg * u
    # |silu'| <= 1.1; the exponential, the division and the products in fp32: 8 roundings
    eh = 1.1 * eg * np.abs(u) + np.abs(sg) * eu + 1.1 * eg * eu + 8 * 2.0 ** -24 * np.abs(h) + 1e-37
    s = scale_of(tops(h, 1), "amax").astype(np.float64)
    rel = spread(tops(eh, 1) / np.maximum(tops(h, 1), 1e-300), 1, *h.shape) + 2.0 ** -23  # of the scale
    per = spread(s, 1, *h.shape)
    low = np.sign(h) * GRID[nearest(np.maximum(np.abs(h) - eh, 0) / per * (1 - rel))]
    high = np.sign(h) * GRID[nearest((np.abs(h) + eh) / per * (1 + rel))]
    mid = np.sign(h) * GRID[nearest(np.abs(h) / per)]
    q = mid * per
    move = np.maximum(np.abs(high - mid), np.abs(low - mid)) * per + np.abs(q) * rel
    y = q @ w2.T
    return y, move @ np.abs(w2).T + (np.abs(q) + move) @ np.abs(w2).T * (sum_error(I) + cores_error(True))


# ------------------------------------------------------------------ routing
def logits(x, w, bias):
    """float32 logits [T, E] of x [T, H] and w [E, H] (float64 holding their values)."""
    v = x @ w.T
    return (v if bias is None else v + bias).astype(np.float32)


def route(l, balance, k, score, groups, top, rule, renorm, scale):
    """(idx [T,k], w [T,k] float64) from float32 logits."""
    l = l.astype(np.float64)
    T, E = l.shape
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            p = 1 / (1 + np.exp(-l))
        else:
            p = np.exp(l - l.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
    c = p if balance is None else p + balance.astype(np.float64)
    n = E // groups
    idx, w = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        left = list(range(E))
        if top < groups:
            worth = []
            for g in range(groups):
                best = sorted(c[t, g * n:g * n + n], reverse=True)
                worth.append(best[0] if rule == "max" else best[0] + best[1])
            keep = sorted(range(groups), key=lambda g: (-worth[g], g))[:top]
            left = [e for e in left if e // n in keep]
        idx[t] = sorted(left, key=lambda e: (-c[t, e], e))[:k]
        w[t] = p[t, idx[t]]
        if renorm:
            s = w[t].sum()
            w[t] = w[t] / s if s else 0.0
    return idx, scale * w
