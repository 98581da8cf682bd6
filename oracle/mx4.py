"""Oracle of the microscaled 4-bit floats, in 64 bits (numpy, CPU).

The format: blocks of 32 consecutive values of a row share a scale 2^(s - 127);
a value is a sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6.  The format's tables and
the generator's constants are published (OCP Microscaling Formats; Salmon et
al., 2011); everything here is worked out in float64 and integers, where each
operation on such values is exact.
"""

import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def philox(index, upper, seed, offset):
    """Four words of Philox4x32-10 for each index: key = seed, counter = the
    index (bit 63 set where upper), then offset."""
    m32 = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    index = np.asarray(index, np.uint64)
    c = [index & m32, index >> sh, np.full_like(index, offset & 0xFFFFFFFF),
         np.full_like(index, offset >> 32)]
    if upper:
        c[1] = c[1] | np.uint64(1 << 31)
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> sh) ^ c[1] ^ np.uint64(k[0]), q & m32,
             (p >> sh) ^ c[3] ^ np.uint64(k[1]), p & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1).astype(np.uint32)


def quantize(x, seed=None, offset=0, upper=False):
    """(codes 0..15 [rows, kb, 32], scales [rows, kb]) of a float32 matrix, blocks
    along its rows; nearest, or at random from (seed, offset).  For the blocks
    down a matrix's columns pass its transpose and upper=True."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    v = np.zeros((rows, kb * BLOCK), np.float32)
    v[:, :cols] = x
    v = v.reshape(rows, kb, BLOCK)
    finite = np.isfinite(v).all(-1)
    a = np.where(finite[..., None], np.abs(v), 0).astype(np.float64)
    top = a.max(-1)
    # the exponent field of binary32: subnormals and zero have 0
    e = np.where(top > 0, np.frexp(top)[1] - 1 + 127, 0).clip(min=0)
    s = e - 2
    if seed is not None:
        s = s + (top > 1.5 * 2.0 ** (e - 127.0))
    s = s.clip(min=0)
    y = a / (2.0 ** (s - 127.0))[..., None]
    if seed is None:
        d = np.abs(y[..., None] - GRID)
        near = d == d.min(-1, keepdims=True)
        # of two equally near codes the even one
        code = np.where(near[..., 0::2].any(-1), 2 * near[..., 0::2].argmax(-1),
                        2 * near[..., 1::2].argmax(-1) + 1)
    else:
        w = philox(np.arange(rows * kb * 4, dtype=np.uint64), upper, seed, offset)
        r = np.stack([w & 0xFFFF, w >> 16], -1).reshape(rows, kb, BLOCK).astype(np.float64)
        low = np.searchsorted(GRID, y, side="right") - 1  # the code at or below
        low = np.minimum(low, 7)
        step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
        cut = np.floor((y - GRID[low]) / step * 65536)  # 16 bits of the distance
        code = low + (cut + r >= 65536)
    code = code + 8 * np.signbit(v)
    code = np.where(finite[..., None], code, 0)
    return code.astype(np.uint8), np.where(finite, s, 255).astype(np.uint8)


def pack(code):
    """Bytes [rows, kb * 16] of codes [rows, kb, 32]."""
    c = code.reshape(code.shape[0], -1, 2)
    return (c[..., 0] | c[..., 1] << 4).astype(np.uint8)


def unpack(codes):
    b = np.asarray(codes, np.uint8)
    return np.stack([b & 15, b >> 4], -1).reshape(b.shape[0], -1, BLOCK)


def values(codes, scales, cols):
    """float64 values [rows, cols] of packed codes and scales."""
    c = unpack(codes)
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.asarray(scales, np.int64)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    return (v * f[..., None]).reshape(c.shape[0], -1)[:, :cols]


def reduce(peers, acc, scale):
    """fl((acc + S) * scale) in binary32, S the ascending sum of the peers'
    float32 values, one rounding an operation."""
    with np.errstate(all="ignore"):
        S = peers[0].astype(np.float32)
        for p in peers[1:]:
            S = S + p.astype(np.float32)
        if acc is not None:
            S = acc + S
        return (S * np.float32(scale)).astype(np.float32)
