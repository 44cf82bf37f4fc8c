"""W8A8 layer (oracle, test infrastructure only): int8 codes with one scale per token and per
output channel.

  v     = f32(x) / f32(smooth_factor)  (activations) or f32(w) * f32(smooth_factor)  (weights)
          (activation quotients below 2^-110 in magnitude count as 0)
  v     = fwht_blocks(v, block)        (optional; ``oracle.hadamard``)
  amax  = max_k |v|, scale = f32(amax / 127), inv = f32(127 / amax)
  code  = the exact product v * inv rounded to the nearest integer, ties to even
  y     = round( (f32(sum q w) * ascale) * wscale + bias )

Rows with amax < 2^-100 get scale 0 and codes 0; rows whose amax is not finite scale NaN and
codes 0.  Every step that decides a code is float32, as in the kernels (the products v * inv are
exact in float64: 24 by 24 bits); the integer sum is exact; the steps after it are the kernels'
float32 operations in their order, so the layer is comparable bit for bit.

Pins (``tests/test_oracle_w8a8.py``): codes and scales against a pure-Python loop over Fractions,
the reconstruction bound |v - code * scale| <= (1/2 + 2^-15) scale, the special rows, and the
identity of a layer of integer weights and unit scales with the plain integer product.
"""

import numpy as np

from . import hadamard

TINY_ROW = np.float32(2.0 ** -100)
TINY_QUOTIENT = np.float32(2.0 ** -110)


def quantize_rows(v):
    """float32 rows -> (codes int8, scales f32)."""
    v = np.asarray(v, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(axis=1) if v.shape[1] else np.zeros(len(v), np.float32)
        bad = ~np.isfinite(v).all(axis=1)
        dead = ~bad & (amax < TINY_ROW)
        safe = np.where(bad | dead, np.float32(1), amax).astype(np.float32)
        scale = safe / np.float32(127)
        inv = np.float32(127) / safe
        codes = np.rint(v.astype(np.float64) * inv.astype(np.float64)[:, None])
    codes[bad | dead] = 0
    scale = np.where(bad, np.float32(np.nan), np.where(dead, np.float32(0), scale)).astype(np.float32)
    return codes.astype(np.int8), scale


def smooth_act(x, smooth, block):
    """float32 values that the activation quantizer rounds."""
    v = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if smooth is not None:
            v = v / np.asarray(smooth, np.float32)[None, :]
            v = np.where(np.abs(v) < TINY_QUOTIENT, np.float32(0), v)
        return hadamard.fwht_blocks(v, block) if block else v


def quantize_act(x, smooth=None, block=0):
    return quantize_rows(smooth_act(x, smooth, block))


def quantize_weight(w, smooth=None, block=0):
    v = np.asarray(w, np.float32)
    with np.errstate(all="ignore"):
        if smooth is not None:
            v = v * np.asarray(smooth, np.float32)[None, :]
        return quantize_rows(hadamard.fwht_blocks(v, block) if block else v)


def gemm_f32(qact, ascales, qweight, wscales, bias=None):
    """The layer's output before its last rounding (float32)."""
    # sums below 2^31 are exact in float64
    acc = np.asarray(qact).astype(np.float64) @ np.asarray(qweight).astype(np.float64).T
    with np.errstate(all="ignore"):
        y = acc.astype(np.float32) * np.asarray(ascales, np.float32)[:, None]
        y = y * np.asarray(wscales, np.float32)[None, :]
        if bias is not None:
            y = y + np.asarray(bias, np.float32)[None, :]
    return y


def linear_f32(x, qweight, wscales, smooth=None, bias=None, block=0):
    q, a = quantize_act(x, smooth, block)
    return gemm_f32(q, a, qweight, wscales, bias)
