"""W8A8 layer (oracle, test infrastructure only): int8 codes with one scale per token and per
output channel.

  v     = f32(x) / f32(smooth_factor)  (activations) or f32(w) * f32(smooth_factor)  (weights)
  u     = v, or the unnormalised butterflies of v per block (the order of ``oracle.hadamard``)
  amax  = max_k |u|, inv = f32(127 / amax), scale = f32(f32(amax * norm) / 127)
          (norm = f32(1/sqrt(B)), 1 without a rotation)
  code  = the exact product u * inv rounded to the nearest integer, ties to even
  y     = round( (f32(sum q w) * ascale) * wscale + bias )

Rows with amax * norm < 2^-100 get scale 0 and codes 0; rows whose amax is not finite scale NaN and
codes 0.  Every step that decides a code is float32, as in the kernels (the products u * inv are
exact in float64: 24 by 24 bits); the integer sum is exact; the steps after it are the kernels'
float32 operations in their order, so the layer is comparable bit for bit.

Pins (``tests/test_oracle_w8a8.py``): codes and scales against a pure-Python loop over Fractions,
the reconstruction bound |v - code * scale| <= (1/2 + 2^-15) scale, the special rows, and the
identity of a layer of integer weights and unit scales with the plain integer product.
"""

import numpy as np

from . import hadamard

TINY_ROW = np.float32(2.0 ** -100)


def butterflies(v, block):
    """float32 butterflies of every block, spans 1, 2, ..., block / 2, without the normalisation."""
    v = np.array(v, dtype=np.float32, copy=True)
    h = 1
    while h < block:
        p = v.reshape(v.shape[:-1] + (-1, 2, h))
        a, b = p[..., 0, :].copy(), p[..., 1, :].copy()
        p[..., 0, :], p[..., 1, :] = a + b, a - b
        h *= 2
    return v


def quantize_rows(u, norm=np.float32(1)):
    """float32 rows -> (codes int8, scales f32)."""
    u = np.asarray(u, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(u).max(axis=1) if u.shape[1] else np.zeros(len(u), np.float32)
        bad = ~np.isfinite(u).all(axis=1)
        dead = ~bad & (amax * norm < TINY_ROW)
        safe = np.where(bad | dead, np.float32(1), amax).astype(np.float32)
        scale = (safe * norm) / np.float32(127)
        inv = np.float32(127) / safe
        codes = np.rint(u.astype(np.float64) * inv.astype(np.float64)[:, None])
    codes[bad | dead] = 0
    scale = np.where(bad, np.float32(np.nan), np.where(dead, np.float32(0), scale)).astype(np.float32)
    return codes.astype(np.int8), scale


def _rotate_and_quantize(v, block):
    with np.errstate(all="ignore"):
        return quantize_rows(butterflies(v, block), hadamard.norm_const(block)) if block else quantize_rows(v)


def quantize_act(x, smooth=None, block=0):
    v = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        return _rotate_and_quantize(v if smooth is None else v / np.asarray(smooth, np.float32)[None, :], block)


def quantize_weight(w, smooth=None, block=0):
    v = np.asarray(w, np.float32)
    with np.errstate(all="ignore"):
        return _rotate_and_quantize(v if smooth is None else v * np.asarray(smooth, np.float32)[None, :], block)


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
