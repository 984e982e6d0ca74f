"""4-bit E2M1 codes with E4M3 block scales for a KV cache (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

The pages name quantised KV caches as a backend feature ("Model execution",
section "Where it breaks") and fix no 4-bit format.  The reading taken: E2M1
codes - 1 sign bit, 2 exponent bits with bias 1, 1 mantissa bit, so the magnitudes
0, 0.5, 1, 1.5, 2, 3, 4, 6 - one E4M3 scale (``oracle.fp8``) for 16 consecutive
elements of a token's head row, and one fp32 scale per cache tensor.  An element
stands for t * scale * code.  A row's 16 elements x become y = x / t, the scale
E4M3(max|y| / 6), the codes E2M1(y / scale): every quotient rounded to fp32,
every code the nearest (ties to even), saturating at 448 and at 6; a scale of 0
has codes 0, and 16 elements with a NaN have the NaN scale and codes 0.

The page of one (block, KV head) is 16 rows of D / 2 code bytes (element 2 i in the
low nibble of byte i), then 16 rows of D / 16 scale bytes; a cache is
[num_blocks, Hkv, 9 D] bytes.
"""

from __future__ import annotations

import numpy as np

from . import fp8

BLOCK = 16
QUANT = 16
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode(codes) -> np.ndarray:
    """float64 value of each code (0..15)."""
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def encode(x) -> np.ndarray:
    """Nearest code of each value, ties to the even code, saturating at 6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 64.0)         # (beyond 6 all saturate)
    dist = np.abs(a[..., None] - MAGNITUDES)
    near = dist == dist.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return (pick + 8 * np.signbit(x)).astype(np.uint8)


def _div32(x, y):
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        return (np.asarray(x, dtype=np.float32) / np.asarray(y, dtype=np.float32)).astype(np.float32)


def quantize(x, t):
    """Rows [..., D] of float32 -> (codes [..., D], scale bytes [..., D / 16])."""
    y = _div32(x, np.float32(t))
    b = y.reshape(y.shape[:-1] + (-1, QUANT))
    nan = np.isnan(b).any(axis=-1)
    a = np.abs(np.where(np.isnan(b), np.float32(0), b)).max(axis=-1)
    scale = fp8.encode(_div32(a, np.float32(6)).astype(np.float64))
    scale = np.where(nan, np.uint8(fp8.NAN_CODE), scale)
    s = fp8.decode(scale).astype(np.float32)[..., None]
    live = ~nan & (scale != 0)
    z = _div32(np.where(live[..., None], b, np.float32(0)), np.where(live[..., None], s, np.float32(1)))
    codes = np.where(live[..., None], encode(z), np.uint8(0)).astype(np.uint8)
    return codes.reshape(y.shape), scale.astype(np.uint8)


def values(codes, scales, t) -> np.ndarray:
    """float64 values t * scale * code of rows [..., D]."""
    c = decode(codes).reshape(codes.shape[:-1] + (codes.shape[-1] // QUANT, QUANT))
    return (np.float64(np.float32(t)) * fp8.decode(scales)[..., None] * c).reshape(codes.shape)


def parts(cache, d):
    """Views of a cache: code bytes [blocks, Hkv, 16, D / 2] and scale bytes
    [blocks, Hkv, 16, D / 16]."""
    nb, hkv = cache.shape[:2]
    return (cache[:, :, :8 * d].reshape(nb, hkv, BLOCK, d // 2),
            cache[:, :, 8 * d:].reshape(nb, hkv, BLOCK, d // QUANT))


def write(cache, x, slots, t):
    """A copy of the cache with row i of x [N, Hkv, D] stored at slot slots[i]
    (negative slots, and slots past the cache, are skipped)."""
    out = cache.copy()
    nb, hkv = cache.shape[:2]
    d = x.shape[-1]
    codes, scales = quantize(x, t)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    for i, slot in enumerate(np.asarray(slots)):
        if not 0 <= slot < nb * BLOCK:
            continue
        blk, row = divmod(int(slot), BLOCK)
        out[blk, :, row * d // 2:(row + 1) * d // 2] = packed[i]
        at = 8 * d + row * d // QUANT
        out[blk, :, at:at + d // QUANT] = scales[i]
    return out


def rows(cache, slots, d, t) -> np.ndarray:
    """float64 values [N, Hkv, D] of the given slots."""
    codes, scales = parts(cache, d)
    s = np.asarray(slots, dtype=np.int64)
    packed = codes[s // BLOCK, :, s % BLOCK]
    c = np.stack([packed & 15, packed >> 4], axis=-1).reshape(packed.shape[:-1] + (d,))
    return values(c, scales[s // BLOCK, :, s % BLOCK], t)
