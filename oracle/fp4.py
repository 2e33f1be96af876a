"""4-bit KV-cache quantization, plain numpy (CPU oracle).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Blocks of 16 elements of a row share a scale. Elements are E2M1 codes (1 sign,
2 exponent bits with bias 1, 1 mantissa bit, subnormals; largest value 6), the
lower half of byte i holding element 2 i. Scales are bytes of 5 exponent bits
(bias 15) and 3 mantissa bits, subnormals, no sign. scale = the nearest one
(ties to the even byte) to the fp32 quotient amax / 6, at most 10240; code = the
nearest one (ties to the even code) to x / scale, at most 6 in magnitude, all 0
under scale 0.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# every scale with exponent below the all-ones one, ascending
E5M3 = np.array([math.ldexp(b if b < 8 else 8 + b % 8, max(b // 8, 1) - 18) for b in range(0xF8)])
MAX_SCALE = 10240.0


def nearest(x, table):
    """Index of the nearest value of an ascending table, ties to the even index."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(table, x, side="left"), 1, len(table) - 1)
    lo = hi - 1
    below, above = x - table[lo], table[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def quantize_blocks(x):
    """Blocks of the last axis of x (values of fp32 precision): (codes uint8
    [..., d / 2], scales uint8 [..., d / 16])."""
    x = np.asarray(x, np.float32)
    assert x.shape[-1] % BLOCK == 0
    b = x.reshape(x.shape[:-1] + (-1, BLOCK))
    amax = np.abs(b).max(-1)
    scale = nearest(np.minimum((amax / np.float32(6)).astype(np.float32), np.float32(MAX_SCALE)), E5M3).astype(np.uint8)
    s = E5M3[scale][..., None]
    mag = nearest(np.minimum(np.abs(b.astype(np.float64)) / np.where(s > 0, s, 1), 6.0), E2M1)
    code = np.where(s > 0, mag + 8 * np.signbit(b), 0).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def dequantize_blocks(codes, scales):
    """float64 values of quantized rows."""
    c = np.asarray(codes, np.uint8)
    x = np.empty(c.shape[:-1] + (c.shape[-1] * 2,))
    for half, part in ((0, c & 15), (1, c >> 4)):
        x[..., half::2] = np.where(part & 8, -1.0, 1.0) * E2M1[part & 7]
    s = E5M3[np.asarray(scales, np.uint8)]
    return (x.reshape(s.shape + (BLOCK,)) * s[..., None]).reshape(x.shape)


def append_kv_fp4(k_codes, k_scale, v_codes, v_scale, k_new, v_new, slots):
    """Quantize new rows ([T, Hkv, d]) and write them at their slots (pools
    [pages, Hkv, P, d / 2] and [pages, Hkv, P, d / 16])."""
    P = k_codes.shape[2]
    for codes, scales, new in ((k_codes, k_scale, k_new), (v_codes, v_scale, v_new)):
        c, s = quantize_blocks(new)
        for t, slot in enumerate(np.asarray(slots).tolist()):
            if slot >= 0:
                codes[slot // P, :, slot % P] = c[t]
                scales[slot // P, :, slot % P] = s[t]
