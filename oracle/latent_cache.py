"""Plain CPU oracle of the 4-bit latent cache (layout in include/hisa.h), in
float64 and Python integers, one group at a time.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

LATENT, ROPE, WIDTH, GROUP, RECORD = 512, 64, 576, 16, 416


def scale_of(code: int) -> float:
    return (1 + (code & 7) / 8) * 2.0 ** ((code >> 3) - 20)


SCALES = np.array([scale_of(c) for c in range(256)])


def quantise_group(x):
    """(scale code, codes) of 16 values: the smallest scale with 7 s >= max|x|, the
    largest one if none is; n = x / s to the nearest, ties to even, in -7..7; a
    NaN counts as 0."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    c = int(min(np.searchsorted(7 * SCALES, np.abs(x).max()), 255))
    if not np.abs(x).max() > 0:
        c = 0
    return c, np.clip(np.rint(np.clip(x / SCALES[c], -8, 8)), -7, 7).astype(int)


def encode(row, rope_bits) -> np.ndarray:
    """The 416-byte record of 512 latent values and the 64 bf16 bit patterns."""
    rec = np.zeros(RECORD, np.uint8)
    words = [0] * (LATENT // 8)
    for g in range(LATENT // GROUP):
        c, n = quantise_group(row[g * GROUP:(g + 1) * GROUP])
        rec[256 + g] = c
        for j in range(GROUP):
            f = g * GROUP + j
            words[f // 8] |= (int(n[j]) & 15) << (4 * ((f % 8) // 2) + 16 * (f % 2))
    rec[:256] = np.array(words, "<u4").view(np.uint8)
    rec[288:] = np.asarray(rope_bits, "<u2").view(np.uint8)
    return rec


def decode(rec) -> np.ndarray:
    """The 576 values (float64) a record stands for."""
    rec = np.asarray(rec, np.uint8)
    words = rec[:256].copy().view("<u4")
    out = np.empty(WIDTH)
    for f in range(LATENT):
        n = int(words[f // 8]) >> (4 * ((f % 8) // 2) + 16 * (f % 2)) & 15
        out[f] = (n - 16 if n > 7 else n) * SCALES[rec[256 + f // GROUP]]
    bits = rec[288:].copy().view("<u2").astype(np.uint32) << 16
    out[LATENT:] = bits.view(np.float32)
    return out


def decode_many(recs) -> np.ndarray:
    return np.stack([decode(r) for r in np.asarray(recs).reshape(-1, RECORD)])
