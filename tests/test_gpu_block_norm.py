"""GPU parity of the block norms with ``oracle/block_norm.py`` within ``_bound``, and of the quantized
form with the unfused calls, bit for bit."""
import itertools

import numpy as np
import pytest
import torch

import bit_diffusion_transformer_svdquant_b200 as svdq
from oracle import block_norm as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24                       # half a step of fp32


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rand(g, *shape, dtype=BF16, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _norm(g, kind, D, affine, dtype=F32):
    if not affine:
        return svdq.Norm(kind, eps=1e-5)
    return svdq.Norm(kind, _rand(g, D, dtype=dtype, std=0.2, mean=1.0), _rand(g, D, dtype=dtype, std=0.2), eps=1e-5)


def _ref_norm(n):
    return None if n is None else (n.kind, _np(n.weight), _np(n.bias), n.eps)


def _norm_bound(v, e, n, D):
    """Error bound of Norm(v) computed in fp32 from values with error e. A sum of D terms loses at most c
    half-steps of its magnitudes: up to 64 terms in a thread, then 2 x 5 shuffle levels, each with the
    rounding of its terms: c = 80. The mean is off by c U mean|v| + max e, the root by (c + 4) U relative,
    and every element passes 4 more roundings."""
    kind, w, b, eps = n
    c = 80
    mean_err = (c * U * np.abs(v).mean(-1, keepdims=True) + e.max(-1, keepdims=True)) if kind == "layer" else 0.0
    d = np.abs(v - v.mean(-1, keepdims=True)) if kind == "layer" else np.abs(v)
    de = e + mean_err + U * d
    ms = (d * d).mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(ms + eps)
    # the root's relative error: half that of the mean square (2 de d, averaged), and its own roundings
    root = (de * (d + de)).mean(-1, keepdims=True) / (ms + eps) + (c + 4) * U
    wa = 1.0 if w is None else np.abs(w)
    out = (de * rstd + d * rstd * (root + 4 * U)) * wa
    return out if b is None else out + 2 * U * (d * rstd * wa + np.abs(b))


def _check(out, want, bound, dtype, what):
    got = _np(out)
    half = torch.finfo(dtype).eps / 2
    tol = bound + half * (np.abs(want) + bound) + 1e-40
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.nanmax(np.abs(got - want) / tol):.2f} bounds"


def _run(x, y, at, gate=None, post=None, skip=1.0, res=1.0, norm=None, scale=None, shift=None):
    """Oracle x' and h with their error bounds."""
    D = x.shape[-1]
    xv = _np(x).reshape(-1, D)
    if y is None:
        xo, e = xv, np.zeros_like(xv)
    else:
        yv = _np(y).reshape(-1, D)
        xo = ref.residual(xv, yv, at, _np(gate), _ref_norm(post), skip, res)
        pe = np.zeros_like(yv) if post is None else _norm_bound(yv, np.zeros_like(yv), _ref_norm(post), D)
        ga = 1.0 if gate is None else np.abs(_np(gate))[at]
        p = np.abs(yv if post is None else ref.normalise(yv, *_ref_norm(post)))
        e = abs(res) * ga * pe + 4 * U * (np.abs(skip * xv) + abs(res) * ga * (p + pe))
    if norm is None:
        return xo, e, None, None
    h = ref.modulated(xo, at, _ref_norm(norm), _np(scale), _np(shift))
    n = np.abs(ref.normalise(xo, *_ref_norm(norm)))
    he = _norm_bound(xo, e, _ref_norm(norm), D)
    if scale is not None:
        f = 1 + np.abs(_np(scale))[at]
        he = he * f + 2 * U * n * f
    if shift is not None:
        he = he + U * (np.abs(h) + np.abs(_np(shift))[at])
    return xo, e, h, he


SIZES = [(1, 1, 1), (1, 3, 7), (2, 5, 8), (1, 9, 40), (3, 17, 257), (2, 33, 256), (1, 130, 1000), (2, 65, 1544),
         (1, 40, 3072), (2, 7, 4096), (1, 5, 5003), (1, 21, 8192), (1, 3, 16384), (1, 3, 12288), (1, 2, 20001),
         (1, 2, 32768)]


@pytest.mark.parametrize("B,T,D", SIZES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_pre_norm(cuda_device, B, T, D, kind):
    g = torch.Generator(device="cuda").manual_seed(B * T + D)
    at = np.repeat(np.arange(B), T)
    for xt, mt, (affine, mod) in zip(itertools.cycle((BF16, F32)), (F32, BF16, BF16, F32),
                                     itertools.product((True, False), (True, False))):
        x = _rand(g, B, T, D, dtype=xt, mean=3.0 if affine else 0.0)
        norm = _norm(g, kind, D, affine, mt)
        m = _rand(g, B, 3 * D, dtype=mt, std=0.5)
        scale, shift = (m[:, D:2 * D], m[:, 2 * D:]) if mod else (None, None)
        _, _, h, he = _run(x, None, at, norm=norm, scale=scale, shift=shift)
        for ot in (BF16, F32):
            out = svdq.block_norm(x, norm, scale, shift, out_dtype=ot)
            assert out.shape == x.shape and out.dtype == ot
            _check(out.reshape(-1, D), h, he, ot, f"{kind} {xt} affine={affine} mod={mod}")


@pytest.mark.parametrize("B,T,D", SIZES)
@pytest.mark.parametrize("post,kind", [(None, None), ("rms", "layer"), ("layer", "rms"), (None, "layer")])
def test_gated_residual(cuda_device, B, T, D, post, kind):
    g = torch.Generator(device="cuda").manual_seed(7 * B * T + D)
    at = np.repeat(np.arange(B), T)
    for xt, yt, ht in ((BF16, BF16, BF16), (F32, BF16, BF16), (F32, F32, F32)):
        x, y = _rand(g, B, T, D, dtype=xt, std=4.0), _rand(g, B, T, D, dtype=yt, std=2.0, mean=0.5)
        gate, scale, shift = _rand(g, B, 3 * D, dtype=xt, std=0.5).split(D, dim=1)
        pn = _norm(g, post, D, True) if post else None
        nn = _norm(g, kind, D, xt == F32) if kind else None
        mods = dict(scale=scale, shift=shift) if kind else {}
        xo, e, h, he = _run(x, y, at, gate, pn, 0.75, 0.5, nn, **mods)
        out = svdq.gated_residual(x, y, gate=gate, post=pn, skip_scale=0.75, res_scale=0.5, norm=nn,
                                  h_dtype=ht if kind else None, **mods)
        got_x, got_h = out if kind else (out, None)
        _check(got_x.reshape(-1, D), xo, e, xt, f"x' {xt}")
        if kind:
            _check(got_h.reshape(-1, D), h, he, ht, f"h {xt}")


# rows enough for the factors of a sample to be shared: every chunk width, runs of several samples
MANY_ROWS = [(1, 400, 256), (3, 110, 512), (1, 310, 768), (2, 200, 1000), (1, 330, 1536), (3, 150, 1544), (2, 160, 3072),
             (1, 310, 8192), (1, 300, 16384), (1, 299, 32768)]


@pytest.mark.parametrize("B,T,D", MANY_ROWS)
def test_many_rows(cuda_device, B, T, D):
    g = torch.Generator(device="cuda").manual_seed(B + T + 3 * D)
    at = np.repeat(np.arange(B), T)
    for xt, yt, post, kind in ((BF16, BF16, "rms", "layer"), (F32, BF16, "layer", "rms")):
        x, y = _rand(g, B, T, D, dtype=xt, std=4.0), _rand(g, B, T, D, dtype=yt, std=2.0, mean=0.5)
        gate, scale, shift = _rand(g, B, 3 * D, std=0.5).split(D, dim=1)
        pn, nn = _norm(g, post, D, True), _norm(g, kind, D, False)
        xo, e, h, he = _run(x, y, at, gate, pn, 1.0, 0.5, nn, scale, shift)
        got_x, got_h = svdq.gated_residual(x, y, gate=gate, post=pn, res_scale=0.5, norm=nn, scale=scale, shift=shift)
        _check(got_x.reshape(-1, D), xo, e, xt, f"x' {xt}")
        _check(got_h.reshape(-1, D), h, he, BF16, f"h {xt}")
        _, _, h, he = _run(x, None, at, norm=nn, scale=scale, shift=shift)
        _check(svdq.block_norm(x, nn, scale, shift).reshape(-1, D), h, he, xt, f"norm {xt}")


@pytest.mark.parametrize("lengths", [[100, 0, 57, 1, 300], [31, 33, 350], [0, 460], [9] * 50])
def test_many_packed_rows(cuda_device, lengths):
    g = torch.Generator(device="cuda").manual_seed(len(lengths))
    lead, tail, D = 2, 7, 1544
    offsets = [lead + sum(lengths[:i]) for i in range(len(lengths) + 1)]
    M, B = offsets[-1] + tail, len(lengths)
    at = ref.sample_rows(offsets, M)
    x, y = _rand(g, M, D, dtype=F32), _rand(g, M, D)
    gate, scale, shift = _rand(g, B, 3 * D, std=0.5).split(D, dim=1)
    norm, inside = _norm(g, "layer", D, True), at >= 0
    out, h = torch.full_like(x, 7.0), torch.full_like(y, 7.0)
    packed = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    svdq.gated_residual(x, y, gate=gate, norm=norm, scale=scale, shift=shift, out=out, h=h, offsets=packed)
    xo, e, hw, he = _run(x[inside], y[inside], at[inside], gate, norm=norm, scale=scale, shift=shift)
    _check(out[inside], xo, e, F32, "x'")
    _check(h[inside], hw, he, BF16, "h")
    assert (out[~inside] == 7.0).all() and (h[~inside] == 7.0).all()


def test_plain_residual_in_place(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(1)
    for D in (96, 97):
        x, y = _rand(g, 50, D), _rand(g, 50, D)
        want = (x.float() + y.float()).to(BF16)
        got = svdq.gated_residual(x, y, out=x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(x, want)


@pytest.mark.parametrize("D", [128, 1544, 1001])
@pytest.mark.parametrize("lengths", [[5], [0, 3, 0, 0, 40, 1, 0], [0, 0], [64, 1, 63, 200]])
def test_packed_samples(cuda_device, D, lengths):
    """Samples of any length; rows before, behind and outside them keep what the outputs held."""
    g = torch.Generator(device="cuda").manual_seed(D + len(lengths))
    lead, tail = 3, 6
    offsets = [lead + sum(lengths[:i]) for i in range(len(lengths) + 1)]
    M, B = offsets[-1] + tail, len(lengths)
    at = ref.sample_rows(offsets, M)
    x, y = _rand(g, M, D, dtype=F32), _rand(g, M, D)
    x[:lead], y[-tail:] = float("nan"), float("inf")
    gate, scale, shift = _rand(g, B, 3 * D, std=0.5).split(D, dim=1)
    norm = _norm(g, "layer", D, True)
    out, h = torch.full_like(x, 7.0), torch.full_like(y, 7.0)
    svdq.gated_residual(x, y, gate=gate, norm=norm, scale=scale, shift=shift, out=out, h=h,
                        offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    inside = at >= 0
    if inside.any():
        xo, e, hw, he = _run(x[inside], y[inside], at[inside], gate, norm=norm, scale=scale, shift=shift)
        _check(out[inside], xo, e, F32, "x'")
        _check(h[inside], hw, he, BF16, "h")
    assert (out[~inside] == 7.0).all() and (h[~inside] == 7.0).all()


def test_offsets_of_any_content_stay_in_bounds(cuda_device):
    """Offsets that describe no packing (descending, negative, past M): rows may take any sample's
    vectors or none, but nothing outside the row range is written."""
    g = torch.Generator(device="cuda").manual_seed(4)
    M, D = 40, 64
    x = _rand(g, M, D)
    guard = torch.full((M + 20, D), 7.0, dtype=BF16, device="cuda")
    for offs in ([30, 10, 50], [-5, 7, 1000], [40, 0, 0], [2 ** 31 - 1, -2 ** 31, 12]):
        svdq.block_norm(x, svdq.Norm("rms"), scale=_rand(g, 2, D), offsets=torch.tensor(offs, dtype=torch.int32,
                                                                                         device="cuda"), out=guard[10:50])
        torch.cuda.synchronize()
        assert (guard[:10] == 7.0).all() and (guard[50:] == 7.0).all()


def test_strided_misaligned_and_far_rows(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(5)
    norm = _norm(g, "layer", 200, True)
    for left in (0, 3, 8):
        x = _rand(g, 3, 11, 230)[:, :, left:left + 200]
        out = torch.full((3, 11, 216), 7.0, dtype=BF16, device="cuda")
        svdq.block_norm(x, norm, out=out[:, :, 5:205])
        want = svdq.block_norm(x.contiguous(), norm)
        # the two paths add a row's squares in another order: half a step of bf16 either way
        d = (out[:, :, 5:205].float() - want.float()).abs()
        assert (d <= 2 * torch.finfo(BF16).eps / 2 * want.float().abs() + 1e-6).all()
        assert (out[:, :, :5] == 7.0).all() and (out[:, :, 205:] == 7.0).all()
    far = torch.empty(2 * (1 << 30) + 200, dtype=BF16, device="cuda")
    view = torch.as_strided(far, (3, 200), (1 << 30, 1))
    x = _rand(g, 3, 200)
    view.copy_(x)
    assert torch.equal(svdq.block_norm(view, norm), svdq.block_norm(x, norm))


def test_special_values(cuda_device):
    """A zero row stays finite through eps, a constant row normalises to its bias, a large mean does not
    cancel, and a NaN or infinity stays in its row."""
    D = 512
    x = torch.zeros(6, D, device="cuda")
    x[1], x[2] = 3.0, 1e6 + torch.arange(D, device="cuda") % 2
    x[3, 5], x[4, 6], x[5] = float("nan"), float("inf"), 1.0
    for kind in ("rms", "layer"):
        h = svdq.block_norm(x, svdq.Norm(kind))
        assert torch.isfinite(h[[0, 1, 2, 5]]).all() and torch.isnan(h[3]).all() and torch.isnan(h[4]).any()
        assert (h[0] == 0).all()
    h = svdq.block_norm(x, svdq.Norm("layer", eps=0.0))
    assert (h[2].abs() - 1.0).abs().max() <= 2.0 ** -20
    assert (svdq.block_norm(x, svdq.Norm("layer"))[1] == 0).all()


def test_empty_and_zero_eps(cuda_device):
    x = torch.empty(0, 64, device="cuda", dtype=BF16)
    assert svdq.block_norm(x, svdq.Norm("rms")).shape == (0, 64)
    out, h = svdq.gated_residual(x.view(0, 1, 64), x.view(0, 1, 64), norm=svdq.Norm("layer"))
    assert out.shape == h.shape == (0, 1, 64)


def test_refusals(cuda_device):
    x = torch.zeros(2, 3, 64, device="cuda", dtype=BF16)
    n = svdq.Norm("rms")
    bad = [
        lambda: svdq.block_norm(x.half(), n), lambda: svdq.block_norm(x[0, 0], n),
        lambda: svdq.block_norm(x, n, scale=torch.zeros(3, 64, device="cuda", dtype=BF16)),
        lambda: svdq.block_norm(x, n, scale=x[0, 0], shift=x[0, 0].float()),
        lambda: svdq.block_norm(x, svdq.Norm("rms", torch.ones(32, device="cuda"))),
        lambda: svdq.block_norm(x, n, out=torch.empty(3, 64, device="cuda", dtype=BF16)),
        lambda: svdq.block_norm(x.transpose(1, 2), n),
        lambda: svdq.block_norm(x[:1, :1].expand(2, 3, 64), n),
        lambda: svdq.block_norm(x, n, offsets=torch.tensor([0, 6], dtype=torch.int32, device="cuda")),
        lambda: svdq.block_norm(x[0], n, offsets=torch.tensor([0, 3], device="cuda")),
        lambda: svdq.gated_residual(x, x[:1]), lambda: svdq.gated_residual(x, x, out=x.float()),
        lambda: svdq.gated_residual(x, x, gate=x[0, 0].cpu()),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(svdq.SvdqError, match="overlap"):
        svdq.block_norm(x, n, out=x)
    with pytest.raises(svdq.SvdqError, match="at most"):
        svdq.block_norm(torch.zeros(1, 32776, device="cuda"), n)


# ---------------------------------------------------------------- quantized for the next layer

def _mx_weight(g, N, K):
    return svdq.MxWeight(_rand(g, N, K, dtype=F32, std=K ** -0.5), inv_lambda=_rand(g, K, dtype=F32, std=0.2, mean=1.0))


@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (2, 3, 40), (1, 130, 264), (3, 50, 1544), (1, 300, 3072), (2, 9, 8192),
                                   (1, 2, 32768), (1, 290, 1032), (1, 297, 1032), (2, 160, 264), (3, 110, 512),
                                   (1, 320, 8192)])
def test_quantized_is_the_unfused_chain(cuda_device, B, T, D):
    g = torch.Generator(device="cuda").manual_seed(B + T + D)
    x, y = _rand(g, B, T, D, std=3.0), _rand(g, B, T, D)
    gate, scale, shift = _rand(g, B, 3 * D, std=0.5).split(D, dim=1)
    norm, post, w = _norm(g, "layer", D, True), _norm(g, "rms", D, True), _mx_weight(g, 128, D)
    kw = dict(gate=gate, post=post, scale=scale, shift=shift)
    xo, h = svdq.gated_residual(x, y, norm=norm, **kw)
    want = svdq.quantize_act_mx(h.view(-1, D), w, svdq.MxAct(B * T, D, 0, "cuda"))
    got_x, act = svdq.gated_residual_quantize_mx(x, y, norm, w, svdq.MxAct(B * T, D, 0, "cuda"), **kw)
    assert torch.equal(got_x, xo)
    pre = svdq.norm_quantize_act_mx(x, norm, w, svdq.MxAct(B * T, D, 0, "cuda"), scale, shift)
    pre_want = svdq.quantize_act_mx(svdq.block_norm(x, norm, scale, shift).view(-1, D), w,
                                    svdq.MxAct(B * T, D, 0, "cuda"))
    for a, b in ((act, want), (pre, pre_want)):
        for u, v in zip(svdq.export_act_mx(a), svdq.export_act_mx(b)):
            assert torch.equal(u, v)
        # the padding past K too: the product reads whole K steps
        assert torch.equal(svdq.gemm_mx(a, w), svdq.gemm_mx(b, w))
        n = a.M * a.desc.K_pad // 2
        assert torch.equal(a.buf[:n], b.buf[:n])


def test_quantized_packed_rows(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(2)
    M, D = 40, 256
    x, w = _rand(g, M, D), _mx_weight(g, 128, D)
    offsets = torch.tensor([2, 12, 30], dtype=torch.int32, device="cuda")
    scale = _rand(g, 2, D)
    act = svdq.MxAct(M, D, 0, "cuda")
    act.buf.fill_(0xA5)
    svdq.norm_quantize_act_mx(x, svdq.Norm("rms"), w, act, scale=scale, offsets=offsets)
    h = torch.zeros_like(x)
    svdq.block_norm(x, svdq.Norm("rms"), scale=scale, offsets=offsets, out=h)
    want = svdq.quantize_act_mx(h, w, svdq.MxAct(M, D, 0, "cuda"))
    for u, v in zip(svdq.export_act_mx(act), svdq.export_act_mx(want)):
        assert torch.equal(u, v)


def test_block_as_it_is_used(cuda_device):
    """An MLP block as a diffusion transformer runs it, from the kernels to fp64: modulated norm quantized
    for the gate/up layer, SwiGLU, down layer, gate and residual in place -- eagerly and replayed from a
    graph on another input, on a stream of its own."""
    from oracle import mxfp4
    g = torch.Generator(device="cuda").manual_seed(6)
    B, T, D, F = 2, 37, 384, 640
    x = _rand(g, B, T, D)
    mods = _rand(g, B, 3 * D, std=0.5)
    gate, scale, shift = mods.split(D, dim=1)
    norm, post = _norm(g, "layer", D, False), _norm(g, "rms", D, True)
    up = svdq.MxWeight(_rand(g, 2 * F, D, dtype=F32, std=D ** -0.5), swiglu=True)
    L1, L2 = _rand(g, F, 16, std=F ** -0.5), _rand(g, 16, D, std=0.1)
    R_down = _rand(g, D, F, dtype=F32, std=F ** -0.5)
    down = svdq.MxWeight(R_down, L1, L2)
    a_up, a_down = svdq.MxAct(B * T, D, 0, "cuda"), svdq.MxAct(B * T, F, 16, "cuda")

    def block(x):
        h = svdq.gemm_mx(svdq.norm_quantize_act_mx(x, norm, up, a_up, scale, shift), up)
        y = svdq.linear_mx(h, down, act=a_down)
        return svdq.gated_residual(x, y.view(B, T, D), gate=gate, post=post, out=x), h, y

    first = x.clone()
    out, h, y = block(first.clone())
    # each step against fp64 on the step's own input
    at = np.repeat(np.arange(B), T)
    hv = _np(h)
    want_y = mxfp4.dequantize(*mxfp4.quantize(hv)) @ mxfp4.dequantize(*mxfp4.quantize(_np(R_down))).T \
        + (hv @ _np(L1)) @ _np(L2)
    assert np.abs(_np(y) - want_y).max() <= 2.0 ** -8 * np.abs(want_y).max() + 1e-4
    xo, e, _, _ = _run(first, y.view(B, T, D), at, gate, post)
    _check(out.reshape(-1, D), xo, e, BF16, "x'")
    buf = first.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        block(buf)
    second = _rand(g, B, T, D)
    want = block(second.clone())[0]
    buf.copy_(second)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, want) and svdq.device_status() == 0


@pytest.mark.parametrize("r", [0, 16])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("packed", [False, True])
def test_mlp_block_is_its_steps(cuda_device, r, xt, packed):
    """mlp_mx with a norm: bit for bit the calls it stands for, with and without a branch, samples in a
    batch or packed (rows behind the last sample stay as they were)."""
    g = torch.Generator(device="cuda").manual_seed(r + 2)
    B, T, D, F = 3, 50, 256, 384
    rows = B * T + (5 if packed else 0)
    x = _rand(g, rows, D, dtype=xt)
    x = x if packed else x.view(B, T, D)
    offsets = torch.tensor([0, 30, 30, B * T], dtype=torch.int32, device="cuda") if packed else None
    gate, scale, shift = _rand(g, B, 3 * D, std=0.5).split(D, dim=1)
    norm, post = _norm(g, "layer", D, False), _norm(g, "rms", D, True)

    def weight(N, K, swiglu):
        return svdq.MxWeight(_rand(g, N, K, dtype=F32, std=K ** -0.5), _rand(g, K, r, std=K ** -0.5) if r else None,
                             _rand(g, r, N, std=0.1) if r else None, swiglu=swiglu)
    up, down, b_up, b_down = weight(2 * F, D, True), weight(D, F, False), _rand(g, 2 * F), _rand(g, D)
    out = torch.full_like(x, 7.0)
    got = svdq.mlp_mx(x, up, down, b_up, b_down, norm, scale, shift, post, gate, 0.5, offsets=offsets, out=out)
    h = torch.zeros(x.shape, dtype=BF16, device="cuda")
    svdq.block_norm(x, norm, scale, shift, offsets, out=h)
    y = svdq.mlp_mx(h.view(rows, D), up, down, b_up, b_down)
    assert torch.equal(y, svdq.linear_mx(svdq.linear_mx(h.view(rows, D), up, b_up), down, b_down))
    want = torch.full_like(x, 7.0)
    svdq.gated_residual(x, y.view(x.shape), gate=gate, post=post, res_scale=0.5, offsets=offsets, out=want)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
    if packed:
        assert (got[B * T:] == 7.0).all()
    assert svdq.mlp_mx(x[:0], up, down, norm=norm).shape == x[:0].shape
    with pytest.raises(ValueError, match="block form"):
        svdq.mlp_mx(h.view(rows, D), up, down, gate=gate)
    with pytest.raises(ValueError, match="swiglu"):
        svdq.mlp_mx(x, down, up, norm=norm)


def test_slices_of_a_joint_stream(cuda_device):
    """Text and image tokens as slices of one [B, T, D] stream, columns as slices of a wider one: read,
    normalised and updated where they lie, on the 16-byte and the element-wise path."""
    g = torch.Generator(device="cuda").manual_seed(12)
    for D in (256, 250):
        norm = _norm(g, "layer", D, True)
        gate, scale, shift = _rand(g, 3, 3 * D, std=0.5).split(D, dim=1)
        both = _rand(g, 3, 40, D)
        y = _rand(g, 3, 28, D)
        text, image = both[:, :12], both[:, 12:]
        want_x, want_h = svdq.gated_residual(image.contiguous(), y, gate=gate, norm=norm, scale=scale, shift=shift)
        keep = text.clone()
        h = torch.full((3, 30, 2 * D), 7.0, device="cuda", dtype=BF16)
        got_x, got_h = svdq.gated_residual(image, y, gate=gate, norm=norm, scale=scale, shift=shift, out=image,
                                           h=h[:, 1:29, D:])
        assert torch.equal(both[:, 12:], want_x) and torch.equal(h[:, 1:29, D:], want_h)
        assert torch.equal(text, keep) and (h[:, :, :D] == 7.0).all() and (h[:, [0, 29]] == 7.0).all()
        # outputs beside inputs in the same memory
        wide = _rand(g, 3, 28, 2 * D)
        want = svdq.block_norm(wide[..., :D].contiguous(), norm, scale, shift)
        assert torch.equal(svdq.block_norm(wide[..., :D], norm, scale, shift, out=wide[..., D:]), want)
        want = svdq.block_norm(both[:, :12].contiguous(), norm, scale, shift)
        assert torch.equal(svdq.block_norm(both[:, :12], norm, scale, shift, out=both[:, 20:32]), want)
        with pytest.raises(svdq.SvdqError, match="overlap"):
            svdq.block_norm(both[:, :12], norm, out=both[:, 11:23])
        with pytest.raises(svdq.SvdqError, match="overlap"):
            svdq.block_norm(wide[..., :D], norm, out=wide[..., D - 1:-1])
    w = _mx_weight(g, 128, 256)
    both = _rand(g, 3, 40, 256)
    a = svdq.norm_quantize_act_mx(both[:, 5:25], svdq.Norm("rms"), w, svdq.MxAct(60, 256, 0, "cuda"))
    b = svdq.norm_quantize_act_mx(both[:, 5:25].contiguous(), svdq.Norm("rms"), w, svdq.MxAct(60, 256, 0, "cuda"))
    for u, v in zip(svdq.export_act_mx(a), svdq.export_act_mx(b)):
        assert torch.equal(u, v)
    # samples in another order than memory's are refused, not misread
    with pytest.raises(ValueError, match="overlap"):
        svdq.block_norm(both.transpose(0, 1), svdq.Norm("rms"))


def test_quantized_offsets_past_the_rows(cuda_device):
    """Offsets that reach behind the last row: the rows of padding of a quantized output are zero, not read
    from behind x, and x' ends with its rows. Tensors lie inside larger ones."""
    g = torch.Generator(device="cuda").manual_seed(8)
    M, D = 40, 256
    whole_x, whole_y = _rand(g, 400, D, dtype=F32), _rand(g, 400, D)
    x, y, w = whole_x[:M], whole_y[:M], _mx_weight(g, 128, D)
    norm = svdq.Norm("rms")
    for last in (M, M + 20, 128, 1 << 30, 2 ** 31 - 1):
        offsets = torch.tensor([0, 12, last], dtype=torch.int32, device="cuda")
        out, act = torch.full_like(whole_x, 7.0), svdq.MxAct(M, D, 0, "cuda")
        act.buf.fill_(0xA5)
        svdq.gated_residual_quantize_mx(x, y, norm, w, act, offsets=offsets, out=out[:M])
        want = svdq.gated_residual(x, y, norm=norm, offsets=torch.tensor([0, 12, M], dtype=torch.int32, device="cuda"))
        assert torch.equal(out[:M], want[0]) and (out[M:] == 7.0).all()
        codes = act.buf[:act.desc.M_pad * act.desc.K_pad // 2].view(act.desc.M_pad, -1)
        assert (codes[M:] == 0).all()
        ref_act = svdq.quantize_act_mx(want[1], w, svdq.MxAct(M, D, 0, "cuda"))
        for u, v in zip(svdq.export_act_mx(act), svdq.export_act_mx(ref_act)):
            assert torch.equal(u, v)


@pytest.mark.parametrize("D,xt,yt", [(8200, BF16, BF16), (12288, BF16, BF16), (12296, BF16, None), (16384, F32, None),
                                     (16384, BF16, None), (12288, F32, BF16)])
def test_quantized_wide_rows_are_the_unfused_chain(cuda_device, D, xt, yt):
    """Many rows so wide that shared factors leave no room for the smoothing reciprocals: the sums of both
    forms run in the same order, so that codes and scales are those of the stored h."""
    g = torch.Generator(device="cuda").manual_seed(D)
    T = 310
    x, w = _rand(g, T, D, dtype=xt, std=3.0), _mx_weight(g, 128, D)
    gate, scale, shift = _rand(g, 3, D, std=0.5)
    norm, act = _norm(g, "layer", D, True), svdq.MxAct(T, D, 0, "cuda")
    if yt is None:
        h = svdq.block_norm(x, norm, scale, shift, out_dtype=BF16)
        svdq.norm_quantize_act_mx(x, norm, w, act, scale, shift)
    else:
        y, post = _rand(g, T, D, dtype=yt), _norm(g, "rms", D, True)
        kw = dict(gate=gate, post=post, scale=scale, shift=shift)
        xo, h = svdq.gated_residual(x, y, norm=norm, h_dtype=BF16, **kw)
        got, _ = svdq.gated_residual_quantize_mx(x, y, norm, w, act, **kw)
        assert torch.equal(got, xo)
    want = svdq.quantize_act_mx(h, w, svdq.MxAct(T, D, 0, "cuda"))
    for u, v in zip(svdq.export_act_mx(act), svdq.export_act_mx(want)):
        assert torch.equal(u, v), (u != v).sum()


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("D,xt,yt", [(3072, F32, F32), (8192, F32, F32), (8200, F32, F32), (12288, F32, F32), (24576, F32, F32),
                                     (8200, F32, BF16), (32768, F32, BF16), (264, BF16, F32), (32768, BF16, F32)])
def test_quantized_fp32_rows_are_the_unfused_chain(cuda_device, D, xt, yt, T):
    """fp32 streams and block outputs at every width that the quantized form takes."""
    g = torch.Generator(device="cuda").manual_seed(D + T)
    x, y, w = _rand(g, T, D, dtype=xt, std=3.0), _rand(g, T, D, dtype=yt), _mx_weight(g, 128, D)
    gate, scale, shift = _rand(g, 3, D, std=0.5)
    kw = dict(gate=gate, post=_norm(g, "layer", D, True), scale=scale, shift=shift, res_scale=0.5)
    norm, act = _norm(g, "rms", D, True), svdq.MxAct(T, D, 0, "cuda")
    xo, h = svdq.gated_residual(x, y, norm=norm, h_dtype=BF16, **kw)
    got, _ = svdq.gated_residual_quantize_mx(x, y, norm, w, act, **kw)
    assert torch.equal(got, xo)
    want = svdq.quantize_act_mx(h, w, svdq.MxAct(T, D, 0, "cuda"))
    for u, v in zip(svdq.export_act_mx(act), svdq.export_act_mx(want)):
        assert torch.equal(u, v), (u != v).sum()


@pytest.mark.parametrize("left", ["x", "mods"])
def test_mlp_block_of_misaligned_slices(cuda_device, left):
    """A layer without a branch takes slices that do not start on 16 bytes, as one with a branch does."""
    g = torch.Generator(device="cuda").manual_seed(9)
    B, T, D, F = 2, 30, 256, 384
    at_x, at_m = (3, 0) if left == "x" else (0, 5)
    x = _rand(g, B, T, D + 8)[..., at_x:at_x + D]
    scale, shift = (_rand(g, B, D + 16, std=0.5)[:, at_m:at_m + D] for _ in range(2))
    norm = _norm(g, "layer", D, False)
    up = svdq.MxWeight(_rand(g, 2 * F, D, dtype=F32, std=D ** -0.5), swiglu=True)
    down = svdq.MxWeight(_rand(g, D, F, dtype=F32, std=F ** -0.5))
    got = svdq.mlp_mx(x, up, down, norm=norm, scale=scale, shift=shift)
    h = svdq.block_norm(x, norm, scale, shift, out_dtype=BF16)
    y = svdq.mlp_mx(h.view(-1, D), up, down)
    assert torch.equal(got, svdq.gated_residual(x, y.view(B, T, D)))
    with pytest.raises(svdq.SvdqError, match="16-byte"):            # the pass itself still refuses them
        svdq.norm_quantize_act_mx(x, norm, up, svdq.MxAct(B * T, D, 0, "cuda"), scale, shift)
    with pytest.raises(svdq.SvdqError, match="do not match"):       # other refusals stay refusals
        svdq.mlp_mx(x, up, down, norm=norm, acts=(svdq.MxAct(7, D, 0, "cuda"), svdq.MxAct(7, F, 0, "cuda")))


@pytest.mark.parametrize("B,T,D", [(2, 5, 96), (1, 9, 1001), (2, 160, 3072), (1, 310, 1544), (1, 4, 12288)])
def test_fp32_block_output_on_a_bf16_stream(cuda_device, B, T, D):
    g = torch.Generator(device="cuda").manual_seed(D + 1)
    at = np.repeat(np.arange(B), T)
    x, y = _rand(g, B, T, D, std=4.0), _rand(g, B, T, D, dtype=F32, std=2.0, mean=0.5)
    gate, scale, shift = _rand(g, B, 3 * D, std=0.5).split(D, dim=1)
    post, norm = _norm(g, "layer", D, True), _norm(g, "rms", D, False)
    xo, e, h, he = _run(x, y, at, gate, post, 1.0, 0.5, norm, scale, shift)
    got_x, got_h = svdq.gated_residual(x, y, gate=gate, post=post, res_scale=0.5, norm=norm, scale=scale, shift=shift)
    assert got_x.dtype == BF16 and got_h.dtype == F32
    _check(got_x.reshape(-1, D), xo, e, BF16, "x'")
    _check(got_h.reshape(-1, D), h, he, F32, "h")


@pytest.mark.parametrize("T", [20, 330])
@pytest.mark.parametrize("D,ht", [(264, BF16), (3072, F32), (8200, BF16)])
def test_h_stored_beside_its_codes(cuda_device, D, ht, T):
    """The C call's form with both outputs: h as the unquantized call stores it, and its codes."""
    g = torch.Generator(device="cuda").manual_seed(D + T)
    x, y, w = _rand(g, T, D, std=3.0), _rand(g, T, D), _mx_weight(g, 128, D)
    scale, shift = _rand(g, 2, D, std=0.5)
    norm = _norm(g, "layer", D, True)
    for out in (None, torch.empty_like(x)):
        h, act = torch.full((T, D + 8), 7.0, dtype=ht, device="cuda"), svdq.MxAct(T, D, 0, "cuda")
        args = svdq._lib._norm_args(x, None if out is None else y, None, None, 1.0, 1.0, norm, scale, shift, None, out,
                                    h[:, :D])
        svdq._lib._run_norm_quantize(args, x, w, act)
        if out is None:
            want = svdq.block_norm(x, norm, scale, shift, out_dtype=ht)
        else:
            xo, want = svdq.gated_residual(x, y, norm=norm, scale=scale, shift=shift, h_dtype=ht)
            assert torch.equal(out, xo)
        assert torch.equal(h[:, :D], want) and (h[:, D:] == 7.0).all()
        codes = svdq.quantize_act_mx(want.to(BF16), w, svdq.MxAct(T, D, 0, "cuda"))
        for u, v in zip(svdq.export_act_mx(act), svdq.export_act_mx(codes)):
            assert torch.equal(u, v)
