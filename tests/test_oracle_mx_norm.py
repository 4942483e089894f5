"""Pins of the MXFP4 and block-norm oracles: properties their definitions fix, checked apart from the
oracle's own arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block_norm, mxfp4, nvfp4, svdquant


def _rows(seed, rows=24, K=96):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, K))
    v[:, ::17] *= 40.0
    return nvfp4.f32(v)


def test_requantizing_the_values_gives_the_values():
    v = _rows(1)
    q, s = mxfp4.quantize(v)
    d = mxfp4.dequantize(q, s)
    assert np.array_equal(mxfp4.dequantize(*mxfp4.quantize(d)), d)


@pytest.mark.parametrize("k", [-60, -1, 5, 60])
def test_power_of_two_invariance(k):
    v = _rows(2)
    q, s = mxfp4.quantize(v)
    q2, s2 = mxfp4.quantize(v * 2.0 ** k)
    assert np.array_equal(q, q2) and np.array_equal(s2.astype(int), s.astype(int) + k)


def test_largest_element_of_a_block_scales_into_4_to_8():
    v = _rows(3)
    _, s = mxfp4.quantize(v)
    top = np.abs(v.reshape(24, 3, 32)).max(axis=2) / 2.0 ** (s.astype(int) - 127)
    assert np.all((top >= 4.0) & (top < 8.0))


def test_error_is_half_a_step_or_the_saturation():
    v = _rows(4)
    q, s = mxfp4.quantize(v)
    scale = np.repeat(2.0 ** (s.astype(int) - 127), 32, axis=1)
    a, d = np.abs(v) / scale, np.abs(mxfp4.dequantize(q, s)) / scale
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert np.all(np.abs(np.minimum(a, 6.0) - d) <= step / 2)
    assert np.all(np.signbit(v) == ((q & 8) != 0))


def test_zero_subnormal_and_non_finite_blocks():
    v = np.zeros((1, 160))
    v[0, 33] = 2.0 ** -149          # the smallest fp32: far below 2^-127 / 4, so code 0 at the floor scale
    v[0, 64] = 1.5 * 2.0 ** -126
    v[0, 96] = np.inf
    v[0, 130] = np.nan
    v[0, 131] = 3.0
    q, s = mxfp4.quantize(v)
    assert s.tolist() == [[0, 0, 0, 255, 255]]
    assert q[0, 64] == 5 and np.count_nonzero(q) == 1          # 1.5 2^-126 = 3 * 2^-127
    d = mxfp4.dequantize(q, s)
    assert np.isnan(d[0, 96:]).all() and np.isfinite(d[0, :96]).all()


def test_a_partial_last_block_is_a_zero_filled_one():
    v = _rows(5, K=72)
    q, s = mxfp4.quantize(v)
    full = np.zeros((24, 96))
    full[:, :72] = v
    q2, s2 = mxfp4.quantize(full)
    assert q.shape == (24, 72) and np.array_equal(q, q2[:, :72]) and np.array_equal(s, s2)


@pytest.mark.parametrize("r,bias", [(0, False), (4, True)])
def test_layer_exact_rational(r, bias):
    rng = np.random.default_rng(6)
    M, K, N = 3, 40, 5
    X = svdquant.bf16_round(rng.standard_normal((M, K)) * np.where(np.arange(K) < 2, 30.0, 1.0))
    W = svdquant.bf16_round(rng.standard_normal((N, K)) / 6)
    b = svdquant.bf16_round(rng.standard_normal(N) * 0.1) if bias else None
    prep = svdquant.prepare_layer(X, W, r)
    wq = mxfp4.quantize(prep["R"])
    y = mxfp4.layer_forward(X, prep, wq, b)
    F = np.vectorize(Fraction)
    Xq, Wq = F(mxfp4.dequantize(*mxfp4.quantize_activations(X, prep["inv_lambda"]))), F(mxfp4.dequantize(*wq))
    for m in range(M):
        for n in range(N):
            v = sum(Xq[m, k] * Wq[n, k] for k in range(K))
            for j in range(r):
                v += sum(Fraction(X[m, k]) * Fraction(prep["L1s"][k, j]) for k in range(K)) * Fraction(prep["L2"][j, n])
            v += Fraction(b[n]) if bias else 0
            assert abs(float(v) - y[m, n]) <= 1e-12 * np.abs(y).max()


def test_norm_moments_and_invariances():
    rng = np.random.default_rng(7)
    v = rng.standard_normal((6, 77)) * 3 + 5
    n = block_norm.normalise(v, "layer", eps=0.0)
    assert np.abs(n.mean(axis=1)).max() < 1e-13 and np.abs((n * n).mean(axis=1) - 1).max() < 1e-13
    assert np.allclose(block_norm.normalise(2.5 * v + 11, "layer", eps=0.0), n, rtol=0, atol=1e-12)
    r = block_norm.normalise(v, "rms", eps=0.0)
    assert np.abs((r * r).mean(axis=1) - 1).max() < 1e-13
    assert np.allclose(block_norm.normalise(-4 * v, "rms", eps=0.0), -r, rtol=0, atol=1e-13)


def test_layer_norm_is_torchs():
    rng = np.random.default_rng(8)
    v, w, b = rng.standard_normal((5, 33)), rng.standard_normal(33), rng.standard_normal(33)
    t = torch.nn.functional.layer_norm(torch.from_numpy(v), (33,), torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    assert np.allclose(block_norm.normalise(v, "layer", w, b, 1e-5), t.numpy(), rtol=0, atol=1e-13)


def test_residual_and_samples():
    at = block_norm.sample_rows([0, 2, 2, 5], 7)
    assert at.tolist() == [0, 0, 2, 2, 2, -1, -1]
    x, y = np.ones((3, 4)), np.full((3, 4), 2.0)
    gate = np.array([[0.0] * 4, [3.0] * 4])
    out = block_norm.residual(x, y, np.array([0, 1, 1]), gate, None, skip=0.5, res=2.0)
    assert np.array_equal(out, np.array([[0.5] * 4, [12.5] * 4, [12.5] * 4]))
    h = block_norm.modulated(x, np.array([0, 1, 1]), ("rms", None, None, 0.0), scale=gate, shift=gate)
    assert np.array_equal(h, np.array([[1.0] * 4, [7.0] * 4, [7.0] * 4]))
