"""MXFP4 (e2m1 elements, blocks of 32 with a power-of-two scale) in plain numpy: the codes by
comparison with every value of the format, nothing shared with the CUDA path.  Test
infrastructure only."""
from __future__ import annotations

import numpy as np

BLOCK = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(v):
    """v fp64 [..., n] -> uint8 [..., n/32]: max(floor(log2 amax) - 2, -127) + 127; 127 for a
    block of zeros; 255 for one with an infinity or a NaN."""
    b = np.abs(np.asarray(v, np.float64).reshape(*v.shape[:-1], -1, BLOCK))
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(np.isfinite(b), b, 0.0).max(-1)
    _, ex = np.frexp(np.where(amax > 0, amax, 1.0))   # amax = m 2^ex with m in [0.5, 1)
    byte = np.where(amax > 0, np.maximum(ex - 1 - 2, -127) + 127, 127)
    return np.where(bad, 255, byte).astype(np.uint8)


def quantize(v):
    """v fp64 [..., n] -> (codes uint8 [..., n/2], scale bytes uint8 [..., n/32])."""
    v = np.asarray(v, np.float64)
    s = scale_bytes(v)
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        a = np.abs(b) / np.exp2(s.astype(np.float64) - 127.0)[..., None]
    a = np.where((s == 255)[..., None], 0.0, a)
    dist = np.abs(a[..., None] - VALUES)
    # the nearest value; of two equally near ones the one with the even code
    best = dist.min(-1, keepdims=True)
    tie = dist == best
    even = tie & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), tie.argmax(-1))
    neg = np.signbit(b) & (s != 255)[..., None]
    code = (code + 8 * neg).astype(np.uint8).reshape(*v.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), s


def dequantize(codes, scales):
    codes = np.asarray(codes)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    val = np.where(nib & 8, -1.0, 1.0) * VALUES[nib & 7]
    s = np.asarray(scales).astype(np.float64)
    s = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return val * np.repeat(s, BLOCK, -1)
