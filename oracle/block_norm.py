"""Block norms in fp64 (oracle; test infrastructure only, see ``oracle/__init__``).

    x' = skip x + res gate_s . P(y)           h = Norm(x') . (1 + scale_s) + shift_s

P and Norm are RMS ("rms") or LayerNorm ("layer") over the row, or nothing; s is the row's sample.
These are the normalisations in front of and behind a diffusion transformer's blocks; the
conditioning vector supplies gate, scale and shift per sample.
"""
from __future__ import annotations

import numpy as np


def normalise(v, kind, weight=None, bias=None, eps=1e-6):
    v = np.asarray(v, dtype=np.float64)
    if kind == "layer":
        v = v - v.mean(axis=-1, keepdims=True)
    elif kind != "rms":
        raise ValueError(kind)
    n = v / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)
    if weight is not None:
        n = n * weight
    return n if bias is None else n + bias


def sample_rows(offsets, M):
    """Sample of every row of M (-1 outside every sample) of packed samples [offsets[s], offsets[s + 1])."""
    at = np.full(M, -1)
    for s in range(len(offsets) - 1):
        at[offsets[s]:offsets[s + 1]] = s
    return at


def residual(x, y, at, gate=None, post=None, skip=1.0, res=1.0):
    """x' [M, D]; post: None or (kind, weight, bias, eps); at: sample of each row."""
    p = np.asarray(y, dtype=np.float64) if post is None else normalise(y, *post)
    if gate is not None:
        p = gate[at] * p
    return skip * np.asarray(x, dtype=np.float64) + res * p


def modulated(x, at, norm, scale=None, shift=None):
    h = normalise(x, *norm)
    if scale is not None:
        h = h * (1.0 + scale[at])
    return h if shift is None else h + shift[at]
