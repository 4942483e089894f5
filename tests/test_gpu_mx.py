"""GPU parity of the MXFP4 layer with ``oracle/mxfp4.py``: codes, scales and decoded values bit for bit;
fp32 outputs within the bound ``_bound`` derives from the kernels' arithmetic; bf16 outputs equal to the
bf16 rounding of the fp32 outputs."""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_svdquant_b200 as svdq
from oracle import mxfp4, nvfp4, svdquant

from _parity import to_dev_bf16, to_dev_f32

pytestmark = pytest.mark.gpu


def _layer(M, K, N, r, seed, bias=False):
    rng = np.random.default_rng(seed)
    X = rng.standard_normal((M, K))
    X[:, ::61] *= 50.0
    bf = svdquant.bf16_round
    prep = {"inv_lambda": nvfp4.f32(np.exp(rng.uniform(-1, 1, K))), "R": nvfp4.f32(rng.standard_normal((N, K)) / K ** 0.5),
            "L1s": bf(rng.standard_normal((K, r)) / K ** 0.5), "L2": bf(rng.standard_normal((r, N)) * 0.3), "r": r}
    return bf(X), prep, bf(rng.standard_normal(N)) if bias else None


def _weight(prep, dev, swiglu=False):
    r = prep["r"]
    return svdq.MxWeight(to_dev_f32(prep["R"], dev), to_dev_bf16(prep["L1s"], dev) if r else None,
                         to_dev_bf16(prep["L2"], dev) if r else None, to_dev_f32(prep["inv_lambda"], dev), swiglu)


def _bound(X, prep, xq, wq, bias, swiglu):
    """Elementwise bound on the fp32 output's error. Products of E2M1 values and powers of two are exact;
    the tensor core's fp32 sums may round or truncate, at most 2^-23 of the sum of magnitudes per added
    group: K/64 + r/8 accumulating MMAs, and up to 64 terms aligned within one. U is a sum of K products
    of the same kind (K/16 MMAs) stored as a bf16 pair (2^-16 relative: half a step of 8 + 8 bits), times
    L2. SwiGLU: silu has slope at most 1.1 and tanh.approx's 2^-11 makes an error of 2.5e-4 |z|."""
    K = X.shape[1]
    S = np.abs(mxfp4.dequantize(*xq)) @ np.abs(mxfp4.dequantize(*wq)).T
    U = np.abs(X) @ np.abs(prep["L1s"])
    S = S + U @ np.abs(prep["L2"]) + (0 if bias is None else np.abs(bias))
    e = 2.0 ** -23 * (K / 64 + prep["r"] / 8 + 66) * S
    e = e + (2.0 ** -16 + 2.0 ** -23 * (K / 16 + 16)) * (U @ np.abs(prep["L2"]))
    if swiglu:
        z = mxfp4.dequantize(*xq) @ mxfp4.dequantize(*wq).T + (X @ prep["L1s"]) @ prep["L2"]
        z = np.abs(z if bias is None else z + bias)
        h = z.shape[1] // 2
        zg, zu, eg, eu = z[:, :h], z[:, h:], e[:, :h], e[:, h:]
        e = (1.1 * eg + 2.5e-4 * (zg + eg)) * (zu + eu) + zg * eu + 2.0 ** -22 * zg * zu
    return e


def _codes_equal(got, want):
    c, s = (t.cpu().numpy() for t in got)
    assert np.array_equal(s, want[1]), f"scales differ at {np.argwhere(s != want[1])[:5]}"
    c = nvfp4.unpack_nibbles(c)
    assert np.array_equal(c, want[0]), f"codes differ at {np.argwhere(c != want[0])[:5]}"


def _check(X, prep, bias, swiglu, dev):
    w = _weight(prep, dev, swiglu)
    Xd = to_dev_bf16(X, dev)
    act = svdq.quantize_act_mx(Xd, w, svdq.MxAct(X.shape[0], X.shape[1], prep["r"], dev))
    xq, wq = mxfp4.quantize_activations(X, prep["inv_lambda"]), mxfp4.quantize(prep["R"])
    _codes_equal(svdq.export_weight_mx(w), wq)
    _codes_equal(svdq.export_act_mx(act), xq)
    assert np.array_equal(svdq.dequantize_act_mx(act, out_dtype=torch.float32).cpu().double().numpy(),
                          mxfp4.dequantize(*xq))
    b = None if bias is None else to_dev_bf16(bias, dev)
    y32 = svdq.gemm_mx(act, w, b, out_dtype=torch.float32)
    y16 = svdq.linear_mx(Xd, w, b)
    torch.cuda.synchronize()
    assert svdq.device_status() == 0
    assert torch.equal(y16, y32.to(torch.bfloat16))
    err = np.abs(y32.cpu().double().numpy() - mxfp4.layer_forward(X, prep, wq, bias, swiglu))
    bound = _bound(X, prep, xq, wq, bias, swiglu)
    assert np.all(err <= bound), f"{np.count_nonzero(err > bound)} outputs off, worst {np.max(err / bound):.2f} bounds"


CASES = [
    # M, K, N, r, bias, swiglu
    (1, 8, 8, 0, False, False),          # the least of everything: one partial block, one 16-byte row
    (1, 512, 384, 32, True, False),      # one token
    (7, 40, 1000, 16, True, False),      # a partial second block, N short of its tile
    (16, 256, 144, 0, False, False),
    (17, 1608, 2344, 64, True, False),   # 128-wide tiles, r = 64
    (33, 768, 1296, 32, True, True),     # SwiGLU whose halves (648) fill no tile
    (64, 512, 16, 16, False, True),
    (129, 264, 768, 16, True, False),    # a second row block of one row; 384-wide tiles
    (300, 1024, 512, 32, False, False),  # 256-wide tiles, an odd number of row blocks
    (513, 512, 768, 0, True, True),
    (200, 2048, 376, 64, False, False),
]


@pytest.mark.parametrize("M,K,N,r,bias,swiglu", CASES)
def test_layer(cuda_device, M, K, N, r, bias, swiglu):
    _check(*_layer(M, K, N, r, M + K + N, bias), swiglu, cuda_device)


@pytest.mark.parametrize("M,K,N,r,swiglu", [(2048, 256, 9216, 32, False), (1024, 256, 6144, 16, True),
                                            (1300, 320, 4736, 64, False)])
def test_more_tiles_than_resident_pairs(cuda_device, M, K, N, r, swiglu):
    _check(*_layer(M, K, N, r, M + N, True), swiglu, cuda_device)


def test_code_edges(cuda_device):
    """Ties of the element grid, both signs, exact powers of two at a block's top, scales at both ends of
    E8M0, zero and subnormal blocks."""
    rng = np.random.default_rng(3)
    K = 288
    X = np.zeros((12, K))
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 6.0, 7.75, 4.0, 0.0])
    for m in range(9):
        X[m, 0], X[m, 1:13], X[m, 13:25] = 4.0 if m % 2 else 7.0, ties, -ties
        X[m, :32] *= 2.0 ** (40 * (m - 4)) if abs(40 * (m - 4)) < 120 else 2.0 ** (112 * np.sign(m - 4))
    X[9, 64:96] = rng.standard_normal(32) * 2.0 ** -112
    X[10, 96:128] = 2.0 ** -126
    X[11] = -0.0
    X = svdquant.bf16_round(X)
    prep = {"inv_lambda": np.ones(K), "R": nvfp4.f32(rng.standard_normal((128, K))), "r": 0,
            "L1s": np.zeros((K, 0)), "L2": np.zeros((0, 128))}
    prep["inv_lambda"][64:128] = 2.0 ** -20          # products at and below the end of the normal range
    w = _weight(prep, cuda_device)
    act = svdq.quantize_act_mx(to_dev_bf16(X, cuda_device), w, svdq.MxAct(12, K, 0, cuda_device))
    xq = mxfp4.quantize_activations(X, prep["inv_lambda"])
    assert xq[1].min() == 0 and xq[1].max() > 230
    _codes_equal(svdq.export_act_mx(act), xq)
    want = mxfp4.dequantize(*xq)
    assert np.array_equal(svdq.dequantize_act_mx(act, out_dtype=torch.float32).cpu().double().numpy(), want)


@pytest.mark.parametrize("M", [40, 400, 1100])
def test_non_finite_blocks_poison_their_rows_only(cuda_device, M):
    X, prep, _ = _layer(M, 320, 256, 0, 11)
    Xd = to_dev_bf16(X, cuda_device)
    Xd[3, 100], Xd[17, 319], Xd[20, 0] = float("nan"), float("inf"), float("-inf")
    w = _weight(prep, cuda_device)
    act = svdq.quantize_act_mx(Xd, w, svdq.MxAct(M, 320, 0, cuda_device))
    _, s = svdq.export_act_mx(act)
    bad = {(3, 3), (17, 9), (20, 0)}
    assert {tuple(i) for i in torch.nonzero(s == 255).tolist()} == bad
    assert torch.isnan(svdq.dequantize_act_mx(act)[17, 288:]).all()
    y = svdq.gemm_mx(act, w)
    clean = torch.ones(M, dtype=torch.bool)
    clean[[3, 17, 20]] = False
    assert torch.isnan(y[~clean.to(y.device)]).all() and torch.isfinite(y[clean.to(y.device)]).all()


def test_strided_rows_in_and_out(cuda_device):
    """X and Y as column slices of wider tensors: the neighbours of Y's slice stay as they were."""
    M, K, N = 150, 328, 136
    X, prep, bias = _layer(M, K, N, 16, 5, True)
    w, b = _weight(prep, cuda_device), to_dev_bf16(bias, cuda_device)
    wide = torch.full((M, K + 64), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    wide[:, 16:16 + K] = to_dev_bf16(X, cuda_device)
    for dtype, pad in ((torch.bfloat16, 24), (torch.float32, 12)):
        out = torch.full((M, N + 2 * pad), 7.0, dtype=dtype, device=cuda_device)
        got = svdq.linear_mx(wide[:, 16:16 + K], w, b, out=out[:, pad:pad + N], out_dtype=dtype)
        assert got.data_ptr() == out[:, pad:].data_ptr()
        assert torch.equal(got, svdq.linear_mx(to_dev_bf16(X, cuda_device), w, b, out_dtype=dtype))
        assert (out[:, :pad] == 7.0).all() and (out[:, pad + N:] == 7.0).all()
    vals = torch.full((M, K + 16), 7.0, dtype=torch.bfloat16, device=cuda_device)
    act = svdq.quantize_act_mx(wide[:, 16:16 + K], w, svdq.MxAct(M, K, 16, cuda_device))
    svdq.dequantize_act_mx(act, out=vals[:, 8:8 + K])
    assert torch.equal(vals[:, 8:8 + K], svdq.dequantize_act_mx(act)) and (vals[:, 8 + K:] == 7.0).all()


def test_a_row_stride_past_32_bits(cuda_device):
    X, prep, _ = _layer(3, 64, 128, 16, 9)
    w = _weight(prep, cuda_device)
    far = torch.empty(2 * (1 << 30) + 64, dtype=torch.bfloat16, device=cuda_device)
    view = torch.as_strided(far, (3, 64), (1 << 30, 1))
    view.copy_(to_dev_bf16(X, cuda_device))
    assert torch.equal(svdq.linear_mx(view, w), svdq.linear_mx(to_dev_bf16(X, cuda_device), w))


def test_checkpoint_round_trip(cuda_device):
    X, prep, bias = _layer(70, 200, 1296, 32, 21, True)
    w, Xd, b = _weight(prep, cuda_device, True), to_dev_bf16(X, cuda_device), to_dev_bf16(bias, cuda_device)
    w2 = svdq.MxWeight.from_state(w.state_dict(), cuda_device)
    assert torch.equal(svdq.linear_mx(Xd, w, b), svdq.linear_mx(Xd, w2, b))


def test_graph_replay_and_streams(cuda_device):
    """The layer captured once and replayed on new input in the same buffers, and two layers running
    on two streams at once, each with its own activation buffer."""
    X, prep, _ = _layer(260, 512, 768, 32, 31)
    w, Xd = _weight(prep, cuda_device), to_dev_bf16(X, cuda_device)
    Xs, act = Xd.clone(), svdq.MxAct(260, 512, 32, cuda_device)
    out = torch.empty(260, 768, dtype=torch.bfloat16, device=cuda_device)
    svdq.linear_mx(Xs, w, act=act, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svdq.linear_mx(Xs, w, act=act, out=out)
    X2 = Xd.flip(0).contiguous()
    Xs.copy_(X2)
    g.replay()
    want1, want2 = svdq.linear_mx(Xd, w), svdq.linear_mx(X2, w)
    assert torch.equal(out, want2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        y1 = [svdq.linear_mx(Xd, w) for _ in range(10)]
    with torch.cuda.stream(s2):
        y2 = [svdq.linear_mx(X2, w) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want1) for y in y1) and all(torch.equal(y, want2) for y in y2)
    assert svdq.device_status() == 0


@pytest.mark.slow
def test_headline_layer_sampled(cuda_device):
    """The 2048^2 QKV layer: all codes' values by sampled rows, outputs of sampled rows."""
    M, K, N, r = 16896, 3072, 9216, 32
    g = torch.Generator(device=cuda_device).manual_seed(1)
    Xd = torch.randn(M, K, generator=g, device=cuda_device)
    Xd[:, ::100] *= 50
    Xd = Xd.to(torch.bfloat16)
    _, prep, bias = _layer(1, K, N, r, 41, True)
    w = _weight(prep, cuda_device)
    y = svdq.linear_mx(Xd, w, to_dev_bf16(bias, cuda_device), out_dtype=torch.float32)
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 5000, M - 129, M - 1])
    X = Xd[rows.to(cuda_device)].cpu().double().numpy()
    wq, xq = mxfp4.quantize(prep["R"]), mxfp4.quantize_activations(X, prep["inv_lambda"])
    err = np.abs(y[rows.to(cuda_device)].cpu().double().numpy() - mxfp4.layer_forward(X, prep, wq, bias))
    assert np.all(err <= _bound(X, prep, xq, wq, bias, False))
    assert svdq.device_status() == 0


@pytest.mark.parametrize("M", [1, 2, 5, 16, 19, 37, 48, 49, 73, 96, 128])
@pytest.mark.parametrize("K,N,r,swiglu", [(3072, 640, 32, False), (1032, 768, 64, True), (4096, 1152, 16, False),
                                          (6144, 128, 0, False)])
def test_few_rows(cuda_device, M, K, N, r, swiglu):
    """Row counts on both sides of every split of the few-row kernels: rows per cluster, token columns, K
    shares of one to eight CTAs, 384-, 256- and 128-wide tiles, both halves of a SwiGLU tile."""
    _check(*_layer(M, K, N, r, M * 3 + K, M % 2 == 1), swiglu, cuda_device)


def test_few_rows_of_a_wide_layer(cuda_device):
    """More blocks of output columns than SMs, and a stage ring that wraps."""
    _check(*_layer(3, 6400, 19200, 32, 77, True), False, cuda_device)


@pytest.mark.parametrize("M,K,N,r", [(300, 512, 1536, 32), (513, 256, 2344, 64), (130, 1032, 392, 16), (700, 768, 640, 0)])
def test_128_wide_tiles_of_a_wider_packing(cuda_device, M, K, N, r):
    """Few enough blocks for 128-wide tiles, on weights packed 384 and 256 wide whose last tile is partly
    padding."""
    _check(*_layer(M, K, N, r, M + 5 * N, True), False, cuda_device)


def _product_kernel(act, w):
    """The name of the kernel that gemm_mx launches."""
    svdq.gemm_mx(act, w)
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA], acc_events=True) as p:
        svdq.gemm_mx(act, w)
        torch.cuda.synchronize()
    return [n for n in ("few_gemm_kernel", "pair_gemm_kernel") if any(n in e.key for e in p.key_averages())]


@pytest.mark.parametrize("K,N,swiglu,few", [
    # K split down to one step per CTA, no branch: few rows as far as the cluster shares the epilogue
    (256, 1024, False, 16), (512, 640, False, 16), (1024, 768, False, 32), (2048, 512, False, 64), (1800, 256, False, 64),
    (256, 2048, True, 16), (1024, 512, True, 32), (2048, 768, True, 64),
    # more than one step
    (1536, 256, False, 128), (2304, 256, False, 128), (1280, 512, True, 64)])
def test_single_step_products(cuda_device, K, N, swiglu, few):
    """Layers without a branch on both sides of the few-row product's rule, and which kernel took them."""
    X, prep, bias = _layer(few + 1, K, N, 0, K + N, True)
    w, Xd = _weight(prep, cuda_device, swiglu), to_dev_bf16(X, cuda_device)
    for M in sorted({1, 15, few, few + 1}):
        _check(X[:M], prep, bias, swiglu, cuda_device)
        act = svdq.quantize_act_mx(Xd[:M], w, svdq.MxAct(M, K, 0, cuda_device))
        assert _product_kernel(act, w) == ["few_gemm_kernel" if M <= few else "pair_gemm_kernel"], M


@pytest.mark.parametrize("M", [64, 65, 128])
@pytest.mark.parametrize("r", [0, 32])
def test_few_swiglu_rows_end_at_64(cuda_device, M, r):
    """Two accumulators of weight rows leave room for 64 tokens."""
    X, prep, bias = _layer(M, 3072, 512, r, M + r, True)
    _check(X, prep, bias, True, cuda_device)
    w = _weight(prep, cuda_device, True)
    act = svdq.quantize_act_mx(to_dev_bf16(X, cuda_device), w, svdq.MxAct(M, 3072, r, cuda_device))
    assert _product_kernel(act, w) == ["few_gemm_kernel" if M <= 64 else "pair_gemm_kernel"]
