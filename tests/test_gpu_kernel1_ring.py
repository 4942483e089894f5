"""Kernel 1 (quantizer + down-projection) where a CTA's share of K has more stages of 64 columns than its ring of 8, so that
slots are used again and their barriers' phases turn: every format and rank, alone and with K split over clusters, whose
exchange of U at r = 64 takes the ring's memory over. Codes and scales bit for bit, outputs and U within derived bounds."""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_svdquant_b200 as svdq
from oracle import fp8b, svdquant

import test_gpu_fp8b
import test_gpu_mx
import test_gpu_parity_fp8r as fp8r_tests
from _parity import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r", [16, 32, 64])
@pytest.mark.parametrize("M,K,N", [
    (400, 3080, 136),     # four row tiles, clusters of four: 14, 14, 14 and 8 stages, the last block of 8 columns
    (520, 4616, 136),     # five row tiles: 20 stages, two turns of the ring, and 14
    (9300, 1160, 136)])   # 73 row tiles: one CTA each, 20 stages
def test_fp8b(cuda_device, M, K, N, r):
    test_gpu_fp8b._check(*test_gpu_fp8b._layer(M, K, N, r, M + K + r, True), False, cuda_device)


@pytest.mark.parametrize("r", [16, 32, 64])
@pytest.mark.parametrize("M,K,N", [(400, 3080, 136), (520, 4616, 136), (9300, 1160, 136)])
def test_mx(cuda_device, M, K, N, r):
    test_gpu_mx._check(*test_gpu_mx._layer(M, K, N, r, M + K + r, True), False, cuda_device)


@pytest.mark.parametrize("r", [16, 32, 64])
@pytest.mark.parametrize("M,K", [(400, 3072), (520, 4608)])
def test_fp8r(cuda_device, M, K, r):
    X, W, b = fp8r_tests._rand_layer(M, K, 256, r, M + r)
    prep, w, act = fp8r_tests._run(X, W, b, r, False, cuda_device)
    wq = fp8r_tests._check_codes(X, prep, w, act)
    fp8r_tests._check_outputs(X, prep, wq, b, False, w, act, cuda_device)
    assert svdq.device_status() == 0


@pytest.mark.parametrize("r", [16, 32, 64])
@pytest.mark.parametrize("cluster,K", [("1", 1280), ("2", 3072), ("3", 3072), ("4", 3072), ("4", 4608)])
def test_nvfp4(cuda_device, monkeypatch, cluster, K, r):
    """1280 on one CTA: 20 stages; 3072 on two to four: 24, 16 and 12; 4608 on four: 18.

    U is kept as u / alpha in two bf16 halves: 2^-16 of its value (half a step of 8 + 8 bits), 2^-22 for the division and
    the products with alpha. u itself is a sum of K products (exact: 8 x 8 bits) in K / 16 MMAs of 16 terms and up to 4
    partial sums, each addition off by 2^-23 of the sum of magnitudes at most."""
    rng = np.random.default_rng(K + r)
    X = rng.standard_normal((300, K))
    X[:, ::97] *= 50.0
    X = svdquant.bf16_round(X)
    W = svdquant.bf16_round(rng.standard_normal((256, K)) / K ** 0.5)
    monkeypatch.setenv("SVDQ_K1_CLUSTER", cluster)
    c = Case(X, W, None, r, False, cuda_device)
    c.check_scales()
    c.check_act_codes()
    c.check_outputs()
    hi, lo = c.act.U().double().cpu().numpy()
    u, want = (hi + lo)[:300] * float(c.act.alpha().item()), X @ c.prep["L1s"]
    tol = (2.0 ** -16 + 2.0 ** -22) * np.abs(want) + 2.0 ** -23 * (K / 16 + 16 + 4) * (np.abs(X) @ np.abs(c.prep["L1s"]))
    assert np.all(np.abs(u - want) <= tol), np.max(np.abs(u - want) / tol)


def test_codes_of_the_2048_layer(cuda_device):
    """The FP8 activations of the 2048^2 QKV layer: codes and scales of sampled rows, 48 stages a CTA."""
    M, K, r = 16896, 3072, 32
    g = torch.Generator(device=cuda_device).manual_seed(2)
    X = torch.randn(M, K, generator=g, device=cuda_device)
    X[:, ::100] *= 50
    X = X.to(torch.bfloat16)
    _, prep, _ = test_gpu_fp8b._layer(1, K, 128, r, 43)
    act = svdq.quantize_act_fp8b(X, test_gpu_fp8b._weight(prep, cuda_device), svdq.Fp8bAct(M, K, r, cuda_device))
    codes, scales = svdq.export_act_fp8b(act)
    rows = torch.cat([torch.arange(0, M, 61), torch.tensor([63, 64, 127, 128, M - 129, M - 1])]).to(cuda_device)
    want = fp8b.quantize_activations(X[rows].cpu().double().numpy(), prep["inv_lambda"])
    test_gpu_fp8b._codes_equal((codes[rows], scales[rows]), want)
    assert svdq.device_status() == 0
