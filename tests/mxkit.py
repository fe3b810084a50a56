"""MXFP4 rows in numpy, 64 bits, from the format's definition: the plain forms the GPU tests compare with.

A row of K columns is K/2 code bytes (byte b: column 2b in bits 0-3, 2b+1 in bits 4-7), K/32 E8M0 scale bytes and
zeros to a multiple of 16 bytes; a value is E2M1(code) * 2^(scale - 127).
"""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(K):
    return (K // 2 + K // 32 + 15) // 16 * 16


def quantise(x, rule):
    """(codes [R, K], scale bytes [R, K/32]) of x (float64 holding the input's values exactly)."""
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    codes = np.zeros(b.shape, np.int64)
    scales = np.zeros(b.shape[:2], np.int64)
    for i, j in np.ndindex(*b.shape[:2]):
        v = b[i, j]
        if not np.isfinite(v).all():
            scales[i, j] = 255
            continue
        top = np.abs(v).max()
        e = int(np.frexp(top)[1]) - 1 - 2 if top > 0 else -127
        if rule == "fit" and top > 6.0 * 2.0 ** e:
            e += 1
        e = max(e, -127)
        scales[i, j] = e + 127
        u = np.abs(v) * 2.0 ** -e
        off = np.abs(u[:, None] - MAGNITUDES[None, :])
        # nearest magnitude; of two equally near, the even code
        best = off.min(1, keepdims=True)
        even = np.where((off == best) & (np.arange(8) % 2 == 0), 0, 1)
        key = np.where(off == best, even, 2)
        codes[i, j] = key.argmin(1) + 8 * np.signbit(v)
    return codes.reshape(R, K), scales


def pack(codes, scales):
    R, K = codes.shape
    rows = np.zeros((R, row_bytes(K)), np.uint8)
    rows[:, :K // 2] = codes[:, 0::2] + 16 * codes[:, 1::2]
    rows[:, K // 2:K // 2 + K // 32] = scales
    return rows


def values(codes, scales):
    """[R, K] float64; a block of scale 255 is NaN."""
    v = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    with np.errstate(over="ignore"):
        s = np.where(scales == 255, np.nan, np.ldexp(1.0, (scales - 127).astype(np.int32)))
    return v * np.repeat(s, 32, axis=1)


def random_rows(rng, R, K, low, high):
    """(codes, scales) with scale bytes low .. high."""
    return rng.integers(0, 16, (R, K)), rng.integers(low, high + 1, (R, K // 32))


def block_norm(add, post, w_post, gate, scale, resid, eps):
    """The residual stream after a block, in 64 bits, before it is rounded; gate [H], [T, 1], [T, H] or None."""
    d = add.astype(np.float64)
    if post:
        d = d / np.sqrt((d * d).mean(1, keepdims=True) + eps)
        d = d if w_post is None else d * w_post
    if gate is not None:
        d = d * gate
    return resid + scale * d


def norm(resid, w_pre, eps):
    x = resid / np.sqrt((resid * resid).mean(1, keepdims=True) + eps)
    return x if w_pre is None else x * w_pre
