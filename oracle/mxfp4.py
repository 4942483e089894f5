"""MXFP4 variant of the layer (oracle; test infrastructure only, see ``oracle/__init__``).

The format is the microscaled 4-bit float of the OCP "Microscaling Formats (MX)" specification v1.0:
E2M1 elements, one power-of-two scale (E8M0: code c stands for 2^(c - 127), 255 for NaN) per 32
consecutive elements along K. Readings:

  * shared exponent e = floor(log2(amax)) - 2 (2 is E2M1's largest exponent), at least -127; an
    all-zero block takes -127; q = E2M1(v * 2^-e), nearest, ties to the even code, saturating at 6,
    the sign kept when the magnitude rounds to 0;
  * a block with an infinity or a NaN takes scale code 255 and zero codes;
  * K need not fill the last block: missing elements count as zero;
  * the layer keeps its SVDQuant structure: activations are quantized from fp32(x * inv_lambda) and
    y = Xq . Wq^T + (X L1s) L2 + bias, then SwiGLU.
"""
from __future__ import annotations

import numpy as np

from . import nvfp4
from .svdquant import apply_swiglu, smooth_activations

BLOCK = 32


def _blocks(v):
    rows, K = v.shape
    pad = -K % BLOCK
    return np.pad(v, ((0, 0), (0, pad))).reshape(rows, (K + pad) // BLOCK, BLOCK)


def quantize(v32: np.ndarray):
    """fp32 values [rows, K] -> (codes uint8 [rows, K], one per element, scale codes uint8
    [rows, ceil(K / 32)])."""
    v = np.asarray(v32, dtype=np.float64)
    rows, K = v.shape
    b = _blocks(v)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(axis=2)
    bad = ~np.isfinite(amax)
    m, e = np.frexp(np.where(bad | (amax == 0), 1.0, amax))     # amax = m 2^e, m in [1/2, 1)
    e = np.where(amax == 0, -127, np.maximum(e - 1 - 2, -127))
    scaled = np.ldexp(np.where(bad[:, :, None], 0.0, b), -e[:, :, None])
    codes = nvfp4.e2m1_encode(scaled)
    codes[bad] = 0
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(rows, -1)[:, :K], scales


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The fp64 value of every element (NaN in a block of scale code 255)."""
    rows, K = codes.shape
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (_blocks(nvfp4.e2m1_decode(codes)) * s[:, :, None]).reshape(rows, -1)[:, :K]


def quantize_activations(X: np.ndarray, inv_lambda: np.ndarray):
    return quantize(smooth_activations(X, inv_lambda))


def layer_forward(X, prep, weight_q, bias=None, swiglu=False) -> np.ndarray:
    """y = Xq . Wq^T + (X L1s) L2 + bias, then SwiGLU if asked; fp64 [M, N or N/2]."""
    y = dequantize(*quantize_activations(X, prep["inv_lambda"])) @ dequantize(*weight_q).T
    if prep["r"] > 0:
        y = y + (X @ prep["L1s"]) @ prep["L2"]
    if bias is not None:
        y = y + bias[None, :]
    return apply_swiglu(y) if swiglu else y
