"""CPU oracle for the microscaled 4-bit path -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may use it; it shares no code with the HIP library.  Format and
rounding are those of the OCP Microscaling Formats specification v1.0 (MXFP4:
E2M1 elements, an E8M0 scale for each block of 32): blocks run along a row,
the scale exponent is floor(log2 amax) - 2 held in [-127, 127], elements are
rounded to nearest with ties to the even mantissa and saturate at 6.  Where
the specification leaves a choice: a block of zeros has scale byte 0 and keeps
its signed zeros; a block holding a NaN or an infinity has scale byte 255 (NaN)
and zero codes; codes past the end of a row are zero.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(t) -> np.ndarray:
    """Nearest E2M1 code (0..15) of each finite value."""
    t = np.asarray(t, np.float64)
    d = np.abs(np.minimum(np.abs(t), 6.0)[..., None] - VALUES)
    near = d.min(-1, keepdims=True)
    hit = d == near
    first = hit.argmax(-1)                       # a tie hits two neighbours: the even code is kept
    code = np.where((hit.sum(-1) == 2) & (first % 2 == 1), first + 1, first)
    return (code + 8 * np.signbit(t)).astype(np.uint8)


def quantize(x):
    """x (M x K float64) -> (packed codes M x 16 * blocks, scale bytes M x blocks)."""
    M, K = x.shape
    nb = -(-K // BLOCK)
    b = np.zeros((M, nb * BLOCK))
    b[:, :K] = x
    b = b.reshape(M, nb, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.full((M, nb), -127)
    np.maximum(e, np.frexp(top)[1] - 1 - 2, out=e, where=top > 0)
    codes = encode(np.ldexp(b, -e[..., None])).reshape(M, nb * BLOCK)
    codes[np.repeat(bad, BLOCK, 1)] = 0
    return codes[:, 0::2] | (codes[:, 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def decode(packed, scales, K) -> np.ndarray:
    """The float64 values (M x K) of packed codes and scale bytes."""
    packed, scales = np.asarray(packed), np.asarray(scales)
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1)
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (v.reshape(v.shape[0], -1, BLOCK) * s[..., None]).reshape(v.shape[0], -1)[:, :K]


def silu(x) -> np.ndarray:
    return x / (1.0 + np.exp(-x))
