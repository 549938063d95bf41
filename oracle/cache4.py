"""Oracle of the cache in 4 bits: a block of 16 elements holds e2m1 codes and one e4m3 scale, a head
one float32 scale.  Every operation of the definition is a float32 operation, so codes and
scales have to be equal bit for bit.
"""
import numpy as np

from .target import to_e4m3

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def to_code(y):
    """e2m1 codes 0..15 (8: the sign) nearest to y, ties to the even code, past the largest the largest."""
    a = np.minimum(np.abs(np.asarray(y, np.float64)), 6.0)
    d = np.abs(a[..., None] - LEVELS)
    code = d.argmin(-1)                                   # of two equally near the lower
    up = np.minimum(code + 1, 7)
    tie = (np.take_along_axis(d, code[..., None], -1) == np.take_along_axis(d, up[..., None], -1))[..., 0] & (up > code)
    code = np.where(tie & (code % 2 == 1), up, code)
    return code + 8 * np.signbit(y)


def e4m3_byte(s):
    """The byte of a non-negative e4m3 value."""
    if np.isnan(s):
        return 0x7F
    if s < 2.0 ** -6:
        return int(round(s * 2 ** 9))
    e = int(np.floor(np.log2(s)))
    return (e + 7) * 8 + int(round((s / 2.0 ** e - 1) * 8))


def quantise(x, g):
    """Codes [..., D] and scale bytes [..., D / 16] of rows x [..., heads, D] (float32) with head scales g."""
    x, g = x.astype(np.float32), g.astype(np.float32)
    one = np.float32(1)
    with np.errstate(all="ignore"):
        blocks = x.reshape(*x.shape[:-1], -1, 16)
        r = one / (np.float32(6) * g)
        s = to_e4m3((np.abs(blocks).max(-1) * r[:, None]).astype(np.float32)).astype(np.float32)
        i = one / (s * g[:, None])
        i = np.where(np.isfinite(i), i, np.float32(0)).astype(np.float32)
        y = (blocks * i[..., None]).astype(np.float32)
    odd = np.isnan(s)
    codes = np.where(odd[..., None], 0, to_code(np.where(odd[..., None], 0, y)))
    return codes.reshape(x.shape).astype(np.uint8), np.vectorize(e4m3_byte, otypes=[np.uint8])(s)


def e4m3_value(b):
    b = np.asarray(b).astype(int)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, 2.0 ** (e - 7.0) * (1 + m / 8))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def values(codes, scale_bytes, g):
    """What codes [..., heads, D] and scales stand for, in float64 (block scale times head scale as in float32)."""
    x = np.where(codes & 8, -1.0, 1.0) * LEVELS[codes & 7]
    s = e4m3_value(scale_bytes).astype(np.float32) * g.astype(np.float32)[:, None]
    return x * np.repeat(s.astype(np.float64), 16, -1)


def layout(page, D):
    """Bytes of a row's codes, of its scales, and of the whole page."""
    code, scale = D // 2, -(-(D // 16) // 4) * 4
    return code, scale, -(-(page * (code + scale)) // 16) * 16


def put(cache, page, D, slot, head, codes, scale_bytes):
    """Stores one head's row in cache [blocks, heads, bytes]."""
    code, scale, _ = layout(page, D)
    block, r = slot // page, slot % page
    cache[block, head, r * code:(r + 1) * code] = codes[0::2] | (codes[1::2] << 4)
    at = page * code + r * scale
    cache[block, head, at:at + D // 16] = scale_bytes


def get(cache, page, D):
    """Codes [blocks, heads, page, D] and scale bytes [blocks, heads, page, D / 16] of a cache."""
    code, scale, _ = layout(page, D)
    n = page * code
    c = cache[..., :n].reshape(*cache.shape[:2], page, code)
    s = cache[..., n:n + page * scale].reshape(*cache.shape[:2], page, scale)[..., :D // 16]
    return np.stack([c & 15, c >> 4], -1).reshape(*cache.shape[:2], page, D), s
