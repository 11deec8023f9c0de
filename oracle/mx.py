"""Microscaled (OCP MX) formats in their plain definition.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

A block is 32 consecutive values along K with one scale 2^e (stored as e + 127) and 32 codes, E2M1
(4 bits) or E4M3 (8 bits, bias 7, largest 448, no infinities).  With b the block's largest magnitude,
e = clamp(floor(log2 b) - emax, -127, 127) (emax 2 or 8; -127 for b = 0) and a code is the nearest of
the format's numbers to v / 2^e, ties to the even code, at most the largest.
"""
from __future__ import annotations

import numpy as np

from .codecs import E2M1_MAGNITUDES, e2m1_decode

E4M3_MAGNITUDES = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                            for e in range(16) for m in range(8)][:127])   # code 127 is NaN
EMAX = {4: 2, 8: 8}


def grid(bits: int) -> np.ndarray:
    return E2M1_MAGNITUDES if bits == 4 else E4M3_MAGNITUDES


def encode(v: np.ndarray, bits: int) -> np.ndarray:
    """Nearest code of v (fp64), ties to the even one, saturating; the sign is kept."""
    g = grid(bits)
    a = np.minimum(np.abs(v), g[-1])
    hi = np.clip(np.searchsorted(g, a), 1, len(g) - 1)
    lo = hi - 1
    up, down = g[hi] - a, a - g[lo]
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (c | (np.signbit(v).astype(np.int64) << (bits - 1))).astype(np.uint8)


def decode(codes: np.ndarray, bits: int) -> np.ndarray:
    if bits == 4:
        return e2m1_decode(codes)
    c = np.asarray(codes).astype(np.int64)
    return E4M3_MAGNITUDES[np.minimum(c & 127, 126)] * np.where(c & 128, -1.0, 1.0)


def quantize(v: np.ndarray, bits: int):
    """v fp64 [.., K] -> (codes [.., K], one per byte; scale bytes [.., K/32])."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.clip(np.frexp(top)[1] - 1 - EMAX[bits], -127, 127), -127)
    return encode(np.ldexp(b, -e[..., None]), bits).reshape(v.shape), (e + 127).astype(np.uint8)


def dequantize(codes: np.ndarray, scales: np.ndarray, bits: int) -> np.ndarray:
    d = decode(codes, bits).reshape(*codes.shape[:-1], -1, 32)
    return np.ldexp(d, scales.astype(np.int64)[..., None] - 127).reshape(codes.shape)


# ------------------------------------------------------------------ the library's layouts
def pack_nibbles(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def packed_weights(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [N, K], scales [N, K/32] -> the packed bytes, written out index by index: block (n-tile,
    256-wide chunk) of 17408 bytes, codes at r*128 + c, scale of 32-block 4h + j at
    16384 + 512 h + 16 (r % 32) + 4 (r // 32) + j."""
    N, K = codes.shape
    out = np.zeros((N // 128, K // 256, 17408), dtype=np.uint8)
    nib = pack_nibbles(codes)
    for nt in range(N // 128):
        for kc in range(K // 256):
            for r in range(128):
                n = nt * 128 + r
                out[nt, kc, r * 128:(r + 1) * 128] = nib[n, kc * 128:(kc + 1) * 128]
                for b in range(8):
                    out[nt, kc, 16384 + (b // 4) * 512 + 16 * (r % 32) + 4 * (r // 32) + b % 4] = scales[n, kc * 8 + b]
    return out.reshape(-1)


def quad_scales(scales: np.ndarray) -> np.ndarray:
    """scales [R, K/32] -> [K/128, R, 4, 4]: entry (kb, r, c, j) the scale of block 4 kb + j of row
    r + 32 c, 0 past the last row."""
    R, nb = scales.shape
    out = np.zeros((nb // 4, R, 4, 4), dtype=np.uint8)
    for c in range(4):
        for r in range(max(R - 32 * c, 0)):
            out[:, r, c, :] = scales[r + 32 * c].reshape(nb // 4, 4)
    return out
