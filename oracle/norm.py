"""Residual addition, RMS norm, block Hadamard transform and quantization of
bf16 rows.

Test infrastructure only (see oracle/__init__.py).

[gist] §2.A puts the block Hadamard transform in front of the quantization of
a linear's input, and §4 fuses quantization into the kernel that produces
that input; in front of a block's first linear that producer is the norm.
The pages do not define it numerically; the reading here:

  r   = bf16_RNE(x + residual)      (x itself without a residual)
  inv = RN32(1 / sqrt(sum r^2 / K + eps))      (in fp64 up to the rounding)
  y   = RN32(RN32(r * inv) * weight)           (RN32(r * inv) without)

then the fp32 butterflies and the INT8 / BF16 / MX conversion of quant.py.
A row whose r holds a NaN or an infinity is marked as a whole: BF16 writes
NaNs, INT8 scale NaN with codes 0, MX scale byte 0xFF with codes 0.
"""
from __future__ import annotations

import math

import numpy as np

from .formats import bf16_to_f32, f32_to_bf16
from .hadamard import block_hadamard_f32
from .quant import MX_ELEM, int8_quantize, mx_quantize


def residual_sum(x_bits: np.ndarray, res_bits) -> np.ndarray:
    """bf16 bits of r."""
    if res_bits is None:
        return x_bits
    with np.errstate(over="ignore", invalid="ignore"):
        s = (bf16_to_f32(x_bits) + bf16_to_f32(res_bits)).astype(np.float32)
        bad = ~np.isfinite(s)
        b = f32_to_bf16(np.where(bad, np.float32(0), s))
    nan = np.where(np.isnan(s), np.uint16(0x7FC0), np.where(s > 0, np.uint16(0x7F80), np.uint16(0xFF80)))
    return np.where(bad, nan, b).astype(np.uint16)


def rmsnorm_f32(r_bits: np.ndarray, weight, eps: float) -> np.ndarray:
    """fp32 y before the transform (rows of finite r)."""
    r = bf16_to_f32(r_bits).astype(np.float32)
    M, K = r.shape
    ss = np.array([math.fsum(float(v) * float(v) for v in row) for row in r])
    inv = (1.0 / np.sqrt(ss / K + float(np.float32(eps)))).astype(np.float32)
    y = (r * inv[:, None]).astype(np.float32)
    if weight is not None:
        y = (y * np.asarray(weight, np.float32)[None, :]).astype(np.float32)
    return y


def rmsnorm_quantize(x_bits: np.ndarray, res_bits, weight, eps: float, had_block: int, fmt: str):
    """Returns a dict: r (bf16 bits), y (fp32, transformed), q and scales."""
    r = residual_sum(x_bits, res_bits)
    fin = np.isfinite(bf16_to_f32(r)).all(1)
    y = block_hadamard_f32(rmsnorm_f32(np.where(fin[:, None], r, np.uint16(0)), weight, eps), had_block)
    out = {"r": r, "y": y, "finite": fin}
    if fmt == "int8":
        q, s = int8_quantize(y)
        q[~fin] = 0
        s[~fin] = np.nan
        out.update(q=q, scales=s)
    elif fmt == "bf16":
        out.update(q=np.where(fin[:, None], f32_to_bf16(y), np.uint16(0x7FC0)))
    elif fmt in MX_ELEM:
        q, s = mx_quantize(y, MX_ELEM[fmt])
        q[~fin] = 0
        s[~fin] = 0xFF
        out.update(q=q, scales=s)
    else:
        raise ValueError(fmt)
    return out
