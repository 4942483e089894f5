"""Host logic of the MXFP4 layer and the block norms: size queries, layouts, argument checks before any
CUDA call, and the binding's refusals. No compute call is made."""
import ctypes

import pytest
import torch

import bit_diffusion_transformer_svdquant_b200 as svdq
from bit_diffusion_transformer_svdquant_b200 import _lib, build

BASE = 1 << 40
P = ctypes.c_void_p(1 << 41)


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def _up(x, to=256):
    return (x + to - 1) // to * to


def _weight_bytes(N_pad, K_pad, r):
    return (_up(N_pad * K_pad // 2) + _up(N_pad * K_pad // 32) + _up(4 * K_pad) + _up(2 * r * K_pad)
            + _up(2 * r * N_pad))


@pytest.mark.parametrize("N,K,r,swiglu,N_pad,K_pad", [
    (9216, 3072, 32, 0, 9216, 3072), (24576, 3072, 32, 1, 24576, 3072), (8, 8, 0, 0, 256, 256),
    (1000, 1608, 16, 0, 1024, 1792), (2344, 64, 64, 0, 2560, 256), (16, 256, 0, 1, 256, 256), (1536, 256, 0, 0, 1536, 256),
    (1296, 256, 16, 1, 1536, 256), (376, 256, 0, 0, 384, 256)])
def test_weight_sizes(L, N, K, r, swiglu, N_pad, K_pad):
    assert L.svdq_mx_weight_bytes(N, K, r, swiglu) == _weight_bytes(N_pad, K_pad, r)


def test_sizes_refused(L):
    assert L.svdq_mx_weight_bytes(9217, 256, 0, 0) == 0        # N % 8
    assert L.svdq_mx_weight_bytes(24, 256, 0, 1) == 0          # SwiGLU N % 16
    assert L.svdq_mx_weight_bytes(128, 252, 0, 0) == 0         # K % 8
    assert L.svdq_mx_weight_bytes(128, 256, 8, 0) == 0         # rank
    assert L.svdq_mx_weight_bytes(0, 256, 0, 0) == 0 and L.svdq_mx_weight_bytes(128, -8, 0, 0) == 0
    assert L.svdq_mx_act_bytes(0, 256, 0) == 0 and L.svdq_mx_act_bytes(1 << 24, 256, 0) == 0
    assert L.svdq_mx_act_bytes(4, 12, 0) == 0


def _pair(L, M=300, K=520, N=1000, r=16, swiglu=0):
    a = _lib.SvdqMxAct()
    nb = L.svdq_mx_act_bytes(M, K, r)
    assert L.svdq_mx_act_bind(M, K, r, ctypes.c_void_p(BASE), nb, ctypes.byref(a)) == 0
    w = _lib.SvdqMxWeight(N=N, K=K, r=r, swiglu_interleaved=swiglu, n_tile=256, N_pad=1024, K_pad=768)
    for i, f in enumerate(("codes", "scales", "inv_lambda", "L1s_t", "L2_t")):
        setattr(w, f, BASE + ((i + 8) << 24))
    return a, w


def test_act_bind_layout(L):
    a, _ = _pair(L)
    assert (a.M_pad, a.K_pad, a.codes) == (384, 768, BASE)
    assert a.scales - a.codes == 384 * 384 and a.U - a.scales == 384 * 24
    nb = L.svdq_mx_act_bytes(300, 520, 16)
    assert nb == 384 * 384 + 384 * 24 + _up(384 * 16 * 4)
    assert L.svdq_mx_act_bind(300, 520, 16, ctypes.c_void_p(BASE), nb - 1, ctypes.byref(a)) == 1
    assert L.svdq_mx_act_bind(300, 520, 16, ctypes.c_void_p(BASE + 16), nb, ctypes.byref(a)) == 2
    assert L.svdq_mx_act_bind(300, 524, 16, ctypes.c_void_p(BASE), nb, ctypes.byref(a)) == 2
    assert L.svdq_mx_act_bind(300, 520, 16, None, nb, ctypes.byref(a)) == 1


def _calls(L, a, w):
    yield L.svdq_mx_quantize_act(P, 520, ctypes.byref(w), ctypes.byref(a), None)
    yield L.svdq_mx_gemm(ctypes.byref(a), ctypes.byref(w), None, 0, P, 1000, 0, None)
    yield L.svdq_mx_linear(P, 520, ctypes.byref(w), ctypes.byref(a), None, 0, P, 1000, 0, None)


@pytest.mark.parametrize("field,value", [("n_tile", 384), ("N_pad", 1000), ("K_pad", 520), ("N", 1001), ("r", 8),
                                         ("codes", None), ("scales", None), ("inv_lambda", None), ("L1s_t", None),
                                         ("L2_t", None), ("swiglu_interleaved", 2)])
def test_weight_descriptors_refused(L, field, value):
    a, w = _pair(L)
    setattr(w, field, value)
    if field == "r":
        a.r = value
    assert list(_calls(L, a, w)) == [1, 1, 1]
    assert L.svdq_mx_export_weight(ctypes.byref(w), P, P, None) == 1
    assert b"descriptor" in L.svdq_last_error()


@pytest.mark.parametrize("field,value", [("M", 0), ("M", 400), ("M_pad", 300), ("K_pad", 520), ("codes", None),
                                         ("scales", None), ("U", None)])
def test_act_descriptors_refused(L, field, value):
    a, w = _pair(L)
    setattr(a, field, value)
    assert list(_calls(L, a, w)) == [1, 1, 1]
    assert L.svdq_mx_export_act(ctypes.byref(a), P, P, None) == 1
    assert L.svdq_mx_dequantize_act(ctypes.byref(a), P, 520, 0, None) == 1


def test_call_arguments_refused(L):
    a, w = _pair(L)
    A, W = ctypes.byref(a), ctypes.byref(w)
    odd = ctypes.c_void_p((1 << 41) + 8)
    assert L.svdq_mx_quantize_act(None, 520, W, A, None) == 1
    assert L.svdq_mx_quantize_act(odd, 520, W, A, None) == 2
    assert L.svdq_mx_quantize_act(P, 516, W, A, None) == 2          # ldx < K
    assert L.svdq_mx_quantize_act(P, 524, W, A, None) == 2          # ldx % 8
    assert L.svdq_mx_gemm(A, W, None, 1, P, 1000, 0, None) == 1     # bias missing
    assert L.svdq_mx_gemm(A, W, None, 2, P, 1000, 0, None) == 1     # not packed for SwiGLU
    assert L.svdq_mx_gemm(A, W, None, 4, P, 1000, 0, None) == 1
    assert L.svdq_mx_gemm(A, W, None, 0, P, 1000, 2, None) == 1     # out type
    assert L.svdq_mx_gemm(A, W, None, 0, P, 992, 0, None) == 2      # ldy < N
    assert L.svdq_mx_gemm(A, W, None, 0, P, 1004, 0, None) == 2     # rows of bf16 off 16 bytes
    assert L.svdq_mx_gemm(A, W, None, 0, odd, 1000, 0, None) == 2
    assert L.svdq_mx_gemm(A, W, odd, 1, P, 1000, 0, None) == 2
    # the whole layer refuses what either part refuses
    assert L.svdq_mx_linear(None, 520, W, A, None, 0, P, 1000, 0, None) == 1
    assert L.svdq_mx_linear(P, 524, W, A, None, 0, P, 1000, 0, None) == 2
    assert L.svdq_mx_linear(P, 520, W, A, None, 1, P, 1000, 0, None) == 1
    assert L.svdq_mx_linear(P, 520, W, A, None, 0, P, 1004, 0, None) == 2
    assert L.svdq_mx_dequantize_act(A, odd, 520, 0, None) == 2
    assert L.svdq_mx_dequantize_act(A, P, 512, 0, None) == 2
    assert L.svdq_mx_dequantize_act(A, P, 520, 7, None) == 1
    assert L.svdq_mx_export_act(A, ctypes.c_void_p((1 << 41) + 2), P, None) == 2
    a2, _ = _pair(L, r=32)
    assert L.svdq_mx_gemm(ctypes.byref(a2), W, None, 0, P, 1000, 0, None) == 1
    if not torch.cuda.is_available():                               # well-formed: stops at the device
        assert list(_calls(L, a, w)) == [3, 3, 3]


def test_pack_and_bind_arguments_refused(L):
    w = _lib.SvdqMxWeight()
    W, nb = ctypes.byref(w), L.svdq_mx_weight_bytes(1000, 520, 16, 0)
    dst = ctypes.c_void_p(BASE)
    assert L.svdq_mx_pack_weight(None, P, P, P, 1000, 520, 16, 0, dst, nb, W, None) == 1
    assert L.svdq_mx_pack_weight(P, None, P, P, 1000, 520, 16, 0, dst, nb, W, None) == 1
    assert L.svdq_mx_pack_weight(P, P, P, P, 1001, 520, 16, 0, dst, nb, W, None) == 2
    assert L.svdq_mx_pack_weight(P, P, P, P, 1000, 520, 16, 0, dst, nb - 1, W, None) == 1
    assert L.svdq_mx_pack_weight(P, P, P, P, 1000, 520, 16, 0, ctypes.c_void_p(BASE + 16), nb, W, None) == 2
    assert L.svdq_mx_pack_weight(ctypes.c_void_p((1 << 41) + 4), P, P, P, 1000, 520, 16, 0, dst, nb, W, None) == 2
    assert L.svdq_mx_weight_bind(1000, 520, 16, 0, None, nb, W) == 1
    assert L.svdq_mx_weight_bind(1000, 520, 16, 0, dst, nb - 1, W) == 1
    assert L.svdq_mx_weight_bind(1000, 523, 16, 0, dst, nb, W) == 2
    if not torch.cuda.is_available():
        assert L.svdq_mx_pack_weight(P, P, P, None, 1000, 520, 16, 0, dst, nb, W, None) == 3
        assert L.svdq_mx_weight_bind(1000, 520, 16, 0, dst, nb, W) == 3


def _norm_args(**kw):
    """A well-formed gated residual + norm over 12 rows of 40 at fake, disjoint addresses."""
    a = _lib.SvdqBlockNormArgs(M=12, D=40, samples=2, rows_per_sample=6, x=BASE, ldx=40, y=BASE + (1 << 20), ldy=48,
                               x_out=BASE + (2 << 20), ld_out=40, h=BASE + (3 << 20), ldh=40, gate=BASE + (4 << 20),
                               ld_gate=120, skip_scale=1.0, res_scale=1.0)
    a.norm = _lib.SvdqNorm(kind=2, eps=1e-6)
    for k, v in kw.items():
        obj = a
        *path, last = k.split("__")
        for p in path:
            obj = getattr(obj, p)
        setattr(obj, last, v)
    return a


NORM_BAD = [
    (dict(x=None), 1), (dict(M=-1), 1), (dict(D=0), 1), (dict(D=32769, ldx=32769, ldy=32769, ld_out=32769, ldh=32769), 2),
    (dict(x_f32=2), 1), (dict(mod_f32=-1), 1), (dict(samples=0), 1), (dict(rows_per_sample=0), 1),
    (dict(rows_per_sample=5), 1),                                       # 12 rows, 2 samples of 5
    (dict(norm__kind=3), 1), (dict(norm__eps=-1.0), 1), (dict(norm__eps=float("nan")), 1), (dict(post__kind=-1), 1),
    (dict(norm__kind=0), 1),                                            # h without a norm
    (dict(h=None), 1),                                                  # a norm without h
    (dict(h=None, norm__kind=0, scale=BASE), 1), (dict(y=None), 1), (dict(y=None, x_out=None), 1),
    (dict(x_out=None, h=None, norm__kind=0), 1),                        # nothing to write
    (dict(ldx=39), 1), (dict(ldy=0), 1), (dict(ldh=-40), 1), (dict(ld_gate=-1), 1),
    (dict(x=BASE + 1), 2), (dict(gate=BASE + (4 << 20) + 2, mod_f32=1), 2), (dict(norm__weight=BASE + (5 << 20) + 1), 2),
    (dict(x_out=BASE + 80), 1),                                         # shifted over x
    (dict(sx=239), 1), (dict(sh=-1), 1), (dict(s_out=1 << 38), 1),        # sample strides
    (dict(sx=400, x_out=BASE), 1),                                      # in place with other strides
    (dict(x_out=BASE, ld_out=48), 1), (dict(x_out=BASE + (1 << 20)), 1),
    (dict(h=BASE), 1), (dict(h=BASE + (1 << 20) + 64), 1), (dict(h=BASE + (2 << 20)), 1),
]


@pytest.mark.parametrize("change,status", NORM_BAD)
def test_block_norm_refusals(L, change, status):
    assert L.svdq_block_norm(ctypes.byref(_norm_args(**change)), None) == status, L.svdq_last_error()


@pytest.mark.parametrize("change", [{}, dict(x_out=BASE), dict(h=None, norm__kind=0), dict(x_out=None),
                                    dict(y=None, x_out=None, gate=None), dict(ldx=41, x=BASE + 2),
                                    dict(ldx=80, ldh=80, h=BASE + 80), dict(sx=480, sh=480, h=BASE + 480)])
def test_block_norm_well_formed(L, change):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: CPU only")
    assert L.svdq_block_norm(ctypes.byref(_norm_args(**change)), None) == 3, L.svdq_last_error()


# Samples whose stride is exactly the bytes they span, (rows - 1) ld + D: the columns of the next sample lie D further
# on, so that what is beside x in one sample is x itself in the next.
CLOSE = dict(sx=5 * 80 + 40, ldx=80, y=None, gate=None)


@pytest.mark.parametrize("change", [
    dict(CLOSE, x_out=None, h=BASE + 80, ldh=80, sh=440),
    dict(CLOSE, x_out=None, h=BASE + 80, ldh=80),                       # an even output beside it
    dict(CLOSE, x_out=None, h=BASE + 80, ldh=80, sh=480),
    dict(x_out=BASE + 80, s_out=440, ld_out=80, sx=440, ldx=80),
    dict(samples=12, rows_per_sample=1, sx=40, ldx=80, x_out=BASE + 80, s_out=40, ld_out=80),
    dict(y=BASE + 80, sy=440, ldy=80, x_out=BASE, s_out=440, ld_out=80),
])
def test_samples_that_touch_are_not_beside_each_other(L, change):
    assert L.svdq_block_norm(ctypes.byref(_norm_args(**change)), None) == 1, L.svdq_last_error()
    assert b"overlaps" in L.svdq_last_error()


@pytest.mark.parametrize("change", [dict(sx=480, ldx=80, sh=480, ldh=80, h=BASE + 80), dict(ldx=80, ldh=80, h=BASE + 80),
                                    dict(sx=440, ldx=80), dict(sx=440, ldx=80, s_out=440, ld_out=80, x_out=BASE)])
def test_samples_apart_or_in_place_are_taken(L, change):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: CPU only")
    assert L.svdq_block_norm(ctypes.byref(_norm_args(**change)), None) == 3, L.svdq_last_error()


def _quant_pair(L, r=0):
    act, w = _pair(L, M=12, K=40, N=1000, r=r)
    w.K_pad = 256
    return act, w


def test_block_norm_quantize_refusals(L):
    act, w = _quant_pair(L)

    def call(args, act=act, w=w):
        return L.svdq_block_norm_quantize_mx(ctypes.byref(args), ctypes.byref(w), ctypes.byref(act), None)
    ok = dict(h=None)
    if not torch.cuda.is_available():
        assert call(_norm_args(**ok)) == 3, L.svdq_last_error()
    assert call(_norm_args(**ok, norm__kind=0)) == 1
    assert call(_norm_args(**ok, M=11)) == 1
    assert call(_norm_args(**ok, x=BASE + 8)) == 2                      # 16-byte rows
    assert call(_norm_args(**ok, ldy=44)) == 2
    assert call(_norm_args(**ok, ld_gate=121)) == 2
    r16 = _quant_pair(L, 16)
    assert call(_norm_args(**ok), *r16) == 2                            # a branch
    w.K, w.K_pad = 48, 256
    assert call(_norm_args(**ok)) == 1
    assert L.svdq_block_norm_quantize_mx(None, ctypes.byref(w), ctypes.byref(act), None) == 1


def test_quantized_rows_up_to_the_stated_width(L):
    """Every width up to 32768 in whole groups of 8 is taken, but 24576 at most where x and y are both fp32."""
    def call(D, x_f32, y_f32, **kw):
        act, w = _pair(L, M=12, K=D, N=1000, r=0)
        w.K_pad = act.K_pad
        args = _norm_args(D=D, ldx=D, ldy=D, ld_out=D, ld_gate=D, x_f32=x_f32, y_f32=y_f32, h=None, x=BASE, y=BASE + (8 << 20),
                          x_out=BASE + (16 << 20), gate=BASE + (24 << 20), **kw)
        return L.svdq_block_norm_quantize_mx(ctypes.byref(args), ctypes.byref(w), ctypes.byref(act), None)
    assert call(24584, 1, 1) == 2 and b"24576" in L.svdq_last_error()
    assert call(32768, 1, 1) == 2
    if not torch.cuda.is_available():                               # well-formed: stops at the device
        for D, x_f32, y_f32 in ((8200, 1, 1), (12288, 1, 1), (24576, 1, 1), (32768, 1, 0), (32768, 0, 1), (32768, 0, 0)):
            assert call(D, x_f32, y_f32) == 3, L.svdq_last_error()


def test_binding_refuses_before_the_library(L):
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.MxWeight(torch.zeros(128, 256))
    with pytest.raises(ValueError, match="CUDA"):
        svdq.block_norm(cpu, svdq.Norm("rms"))
    with pytest.raises(ValueError, match="CUDA"):
        svdq.gated_residual(cpu, cpu)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.Norm("rms", weight=torch.ones(64))
    with pytest.raises(ValueError, match="kind"):
        svdq.Norm("batch")
    with pytest.raises(ValueError, match="eps"):
        svdq.Norm("rms", eps=-1e-6)
    with pytest.raises(ValueError, match="h without a norm"):
        svdq.gated_residual(cpu, cpu, h=cpu)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.MxAct(4, 64, 0, "cpu")
    with pytest.raises(svdq.SvdqError, match="unsupported shape"):
        svdq.MxAct(4, 63, 0, "cpu")
    state = {"abi": L.svdq_abi_version(), "format": "mxfp4", "N": 128, "K": 256, "r": 0, "swiglu": False}
    for blob in (torch.zeros(8, dtype=torch.uint8), torch.zeros(_weight_bytes(128, 256, 0), dtype=torch.int8)):
        with pytest.raises(ValueError, match="checkpoint blob"):
            svdq.MxWeight.from_state({**state, "blob": blob}, "cpu")
    with pytest.raises(ValueError, match="format"):
        svdq.MxWeight.from_state({**state, "format": None, "blob": None}, "cpu")


class _AsIfOnDevice:
    """A CPU tensor's shape, strides and address, as the binding reads them of a device tensor."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(1, 6, 64).expand(3, 6, 64),                    # one sample standing for three
    lambda: torch.zeros(1, 1, 64).expand(3, 1, 64),
    lambda: torch.zeros(3, 1, 64).expand(3, 6, 64),
    lambda: torch.zeros(1, 64).expand(6, 64),
    lambda: torch.zeros(4096).as_strided((3, 6, 64), (320, 64, 1)),    # a sample's last row is the next one's first
    lambda: torch.zeros(4096).as_strided((6, 64), (32, 1)),
])
def test_rows_that_share_memory_are_refused(make):
    with pytest.raises(ValueError, match="overlap"):
        svdq._lib._norm_rows(_AsIfOnDevice(make()), "x")


@pytest.mark.parametrize("shape,strides,ld,sample", [
    ((3, 6, 64), (384, 64, 1), 64, 0), ((3, 6, 64), (768, 128, 1), 128, 0), ((3, 6, 64), (1000, 64, 1), 64, 1000),
    ((3, 1, 64), (100, 7, 1), 64, 100), ((1, 6, 64), (0, 80, 1), 80, 0), ((3, 1, 64), (64, 0, 1), 64, 0)])
def test_row_and_sample_strides(shape, strides, ld, sample):
    t = torch.zeros(4096).as_strided(shape, strides)
    assert svdq._lib._norm_rows(_AsIfOnDevice(t), "x") == (t.data_ptr(), ld, 1, sample)


def test_no_rows_to_quantize_are_refused():
    """An empty x leaves nothing to write into an activation of at least one row, whose codes of the call before
    would pass for its own."""
    class Act:
        M = 4
    x = _AsIfOnDevice(torch.empty(0, 64))
    with pytest.raises(ValueError, match="act holds 4 rows, x none"):
        svdq.norm_quantize_act_mx(x, svdq.Norm("rms"), None, Act)
    with pytest.raises(ValueError, match="act holds 4 rows, x none"):
        svdq.gated_residual_quantize_mx(x, x, svdq.Norm("rms"), None, Act, out=x)


@pytest.mark.parametrize("rows,stride,ld", [(1, 67, 64), (1, 0, 64), (1, 64, 64), (3, 72, 72), (3, 67, 67)])
def test_the_stride_of_a_single_row_is_not_used(rows, stride, ld):
    """One row of a wider or odder matrix is taken like a row of its own."""
    t = torch.zeros(1024, dtype=torch.bfloat16).as_strided((rows, 64), (stride, 1))
    assert svdq._lib._rows(_AsIfOnDevice(t), torch.bfloat16, "X", rows, 64) == ld


def test_a_residual_without_a_block_output_is_refused():
    """x' would be returned as it was allocated."""
    class Act:
        M = 4
    x, norm = _AsIfOnDevice(torch.ones(4, 64)), svdq.Norm("rms")
    for call in (lambda: svdq.gated_residual(x, None, out=x), lambda: svdq.gated_residual(x, None, norm=norm, out=x, h=x),
                 lambda: svdq.gated_residual(x, None, norm=norm, out=x, h=x, h_dtype=torch.float32),
                 lambda: svdq.gated_residual_quantize_mx(x, None, norm, None, Act, out=x)):
        with pytest.raises(ValueError, match="^y: "):
            call()


def test_half_a_branch_is_refused():
    R, L1s, L2 = _AsIfOnDevice(torch.ones(16, 64)), torch.ones(64, 16), torch.ones(16, 16)
    for pair in ((L1s, None), (None, L2)):
        with pytest.raises(ValueError, match="a branch has both"):
            svdq.MxWeight(R, *pair)


def test_a_norm_follows_its_vectors():
    def vector(*shape, dtype=torch.float32):
        return _AsIfOnDevice(torch.ones(*shape, dtype=dtype))
    n = svdq.Norm("layer", vector(64), vector(64))
    device = n.weight.device
    assert n.fields("norm", 64, device)[2:] == (1, 0, n.weight.data_ptr(), n.bias.data_ptr())
    n.weight, n.bias = vector(128, dtype=torch.bfloat16), None              # other vectors
    assert n.fields("norm", 128, device)[2:] == (0, 0, n.weight.data_ptr(), 0)
    n.weight.t.data = torch.ones(128, dtype=torch.bfloat16)                 # the same tensor, other memory
    assert n.fields("norm", 128, device)[4] == n.weight.t.data_ptr()
    n.weight.t.data = torch.ones(32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="vectors of 32"):
        n.fields("norm", 128, device)
    n.bias = vector(16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="of one type"):
        n.fields("norm", 32, device)


C_PROGRAM = r"""
#include <stddef.h>
#include <stdio.h>
#include "svdq.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu\n", sizeof(svdq_mx_weight), sizeof(svdq_mx_act), sizeof(svdq_norm),
         sizeof(svdq_block_norm_args), offsetof(svdq_mx_weight, tmap), offsetof(svdq_block_norm_args, post),
         offsetof(svdq_block_norm_args, shift));
  return 0;
}
"""


def test_struct_layouts_match_c(tmp_path):
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text(C_PROGRAM)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.dirname(_lib.HEADER), str(src),
                    "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    B = _lib.SvdqBlockNormArgs
    assert got == [ctypes.sizeof(_lib.SvdqMxWeight), ctypes.sizeof(_lib.SvdqMxAct), ctypes.sizeof(_lib.SvdqNorm),
                   ctypes.sizeof(B), _lib.SvdqMxWeight.tmap.offset, B.post.offset, B.shift.offset]


def test_packed_norm_arguments_are_the_structure():
    """The binding packs svdq_block_norm_args as bytes: every field lands where the structure has it."""
    B = _lib.SvdqBlockNormArgs
    flat = []
    for name, ctype in B._fields_:
        flat += [f"{name}.{n}" for n, _ in ctype._fields_] if ctype is _lib.SvdqNorm else [name]
    packed = _lib._PACK_NORM_ARGS(*range(1, len(flat) + 1))
    assert len(packed) == ctypes.sizeof(B)
    a = B.from_buffer_copy(packed)
    for value, name in enumerate(flat, 1):
        obj = a
        for part in name.split("."):
            obj = getattr(obj, part)
        assert obj == value, name
