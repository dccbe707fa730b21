"""NVFP4 codec (microscaled 4-bit floating point), restated in float64 (oracle).

A row is cut into blocks of 16 elements.  Each element is an E2M1 code (sign, two exponent bits of
bias 1, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), each block has one E4M3 scale, each tensor one
float32 scale:

    value = code * block scale * tensor scale.

The write side, with t = float32(x) * float32(1 / tensor scale) (one float32 product, as the FP8 write
defines it):

    block scale = E4M3(max |t| / 6)          nearest-even, saturating
    code        = E2M1(t / block scale)      nearest-even, saturating; 0 where the block scale is 0

A NaN in a block makes its scale NaN (all codes 0); an infinity saturates.  Element 2b of a row is the
low nibble of byte b, element 2b + 1 the high nibble.
"""

from __future__ import annotations

import numpy as np

from . import fp8

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 16


def encode_e2m1(x) -> np.ndarray:
    """Nearest E2M1 code (0..15) of float64 values; halfway goes to the even code; saturates at 6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 8.0)  # everything above 5 is nearest to 6
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(axis=-1, keepdims=True)
    near = d == best
    first = near.argmax(axis=-1)
    last = len(MAGNITUDES) - 1 - near[..., ::-1].argmax(axis=-1)
    code = np.where(first % 2 == 0, first, last)  # of two neighbours one is even
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def decode_e2m1(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def pack(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed) -> np.ndarray:
    p = np.asarray(packed, dtype=np.uint8)
    return np.stack([p & 15, p >> 4], axis=-1).reshape(*p.shape[:-1], 2 * p.shape[-1])


def quantize(x_fp32, scale: float):
    """float32 rows [..., D] -> (packed codes [..., D/2], block-scale codes [..., D/16]), uint8."""
    inv = np.float32(1.0) / np.float32(scale)
    with np.errstate(over="ignore", invalid="ignore"):
        t = (np.asarray(x_fp32, dtype=np.float32) * inv).astype(np.float32).astype(np.float64)
        t = t.reshape(*t.shape[:-1], -1, BLOCK)
        nan = np.isnan(t).any(axis=-1)
        sf = fp8.encode(np.where(nan, np.nan, np.abs(t).max(axis=-1) / 6.0))
        s = np.where(nan, 0.0, fp8.decode(sf))[..., None]
        r = np.where(s > 0, t / np.where(s > 0, s, 1.0), 0.0)
        codes = np.where(s > 0, encode_e2m1(r), 0)
    return pack(codes.reshape(*codes.shape[:-2], -1).astype(np.uint8)), sf


def dequantize(packed, sf, scale: float) -> np.ndarray:
    """Stored codes and block scales -> float64 values."""
    c = decode_e2m1(unpack(packed))
    s = np.repeat(fp8.decode(sf), BLOCK, axis=-1)
    return c * s * np.float64(np.float32(scale))
