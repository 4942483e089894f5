"""ctypes binding of libsvdq.so (include/svdq.h). Argument marshalling only: every step of the layer
runs in the library's CUDA kernels; torch provides device memory and the current stream.

There is no fallback: if the library is missing or the device is not sm_100a, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from ctypes import POINTER, byref, c_char_p, c_float, c_int, c_longlong, c_size_t, c_ulonglong, c_void_p

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsvdq.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "svdq.h")

EPI_NONE, EPI_BIAS, EPI_SWIGLU, EPI_BIAS_SWIGLU = 0, 1, 2, 3
OUT_BF16, OUT_F32 = 0, 1
STATUS_NAMES = {0: "SVDQ_OK", 1: "SVDQ_ERR_INVALID_ARG", 2: "SVDQ_ERR_UNSUPPORTED", 3: "SVDQ_ERR_CUDA",
                4: "SVDQ_ERR_TIMEOUT"}
ERR_UNSUPPORTED = 2


class SvdqWeight(ctypes.Structure):
    _fields_ = [("N", c_int), ("K", c_int), ("r", c_int), ("swiglu_interleaved", c_int), ("n_tile", c_int),
                ("reserved0", c_int), ("codes", c_void_p), ("scales", c_void_p), ("g_w", c_void_p),
                ("inv_lambda", c_void_p), ("L1s_t", c_void_p), ("L2_t", c_void_p), ("tmap", c_ulonglong * 32)]


class SvdqAct(ctypes.Structure):
    _fields_ = [("M", c_int), ("K", c_int), ("r", c_int), ("M_pad", c_int), ("codes", c_void_p),
                ("scales", c_void_p), ("U", c_void_p), ("alpha", c_void_p)]


class SvdqFp8rWeight(ctypes.Structure):
    _fields_ = [("N", c_int), ("K", c_int), ("r", c_int), ("swiglu_interleaved", c_int), ("n_tile", c_int),
                ("reserved0", c_int), ("codes", c_void_p), ("row_scale", c_void_p), ("inv_lambda", c_void_p),
                ("L1s_t", c_void_p), ("L2_t", c_void_p), ("tmap", c_ulonglong * 32)]


class SvdqFp8rAct(ctypes.Structure):
    _fields_ = [("M", c_int), ("K", c_int), ("r", c_int), ("M_pad", c_int), ("codes", c_void_p),
                ("row_scale", c_void_p), ("row_rscale", c_void_p), ("U", c_void_p)]


class SvdqMxWeight(ctypes.Structure):
    _fields_ = [("N", c_int), ("K", c_int), ("r", c_int), ("swiglu_interleaved", c_int), ("n_tile", c_int),
                ("N_pad", c_int), ("K_pad", c_int), ("reserved0", c_int), ("codes", c_void_p), ("scales", c_void_p),
                ("inv_lambda", c_void_p), ("L1s_t", c_void_p), ("L2_t", c_void_p), ("tmap", c_ulonglong * 80)]


class SvdqMxAct(ctypes.Structure):
    _fields_ = [("M", c_int), ("K", c_int), ("r", c_int), ("M_pad", c_int), ("K_pad", c_int), ("reserved0", c_int),
                ("codes", c_void_p), ("scales", c_void_p), ("U", c_void_p)]


class SvdqNorm(ctypes.Structure):
    _fields_ = [("kind", c_int), ("eps", c_float), ("f32", c_int), ("reserved0", c_int), ("weight", c_void_p),
                ("bias", c_void_p)]


class SvdqBlockNormArgs(ctypes.Structure):
    _fields_ = [("M", c_int), ("D", c_int), ("samples", c_int), ("rows_per_sample", c_int), ("offsets", c_void_p),
                ("x", c_void_p), ("ldx", c_longlong), ("x_f32", c_int), ("y_f32", c_int), ("y", c_void_p),
                ("ldy", c_longlong), ("x_out", c_void_p), ("ld_out", c_longlong), ("h", c_void_p),
                ("ldh", c_longlong), ("h_f32", c_int), ("mod_f32", c_int), ("gate", c_void_p),
                ("ld_gate", c_longlong), ("scale", c_void_p), ("ld_scale", c_longlong), ("shift", c_void_p),
                ("ld_shift", c_longlong), ("skip_scale", c_float), ("res_scale", c_float), ("post", SvdqNorm),
                ("norm", SvdqNorm), ("sx", c_longlong), ("sy", c_longlong), ("s_out", c_longlong), ("sh", c_longlong)]


class SvdqError(RuntimeError):
    def __init__(self, func: str, status: int, message: str):
        super().__init__(f"{func}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def _declare(lib):
    W, A = POINTER(SvdqWeight), POINTER(SvdqAct)
    FW, FA = POINTER(SvdqFp8rWeight), POINTER(SvdqFp8rAct)
    MW, MA = POINTER(SvdqMxWeight), POINTER(SvdqMxAct)
    sig = {
        "svdq_fp8r_weight_bytes": (c_size_t, [c_int, c_int, c_int]),
        "svdq_fp8r_act_bytes": (c_size_t, [c_int, c_int, c_int]),
        "svdq_fp8r_pack_weight": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                          c_void_p, c_size_t, FW, c_void_p]),
        "svdq_fp8r_act_bind": (c_int, [c_int, c_int, c_int, c_void_p, c_size_t, FA]),
        "svdq_fp8r_quantize_act": (c_int, [c_void_p, FW, FA, c_void_p]),
        "svdq_fp8r_gemm": (c_int, [FA, FW, c_void_p, c_int, c_void_p, c_int, c_void_p]),
        "svdq_fp8r_export_weight": (c_int, [FW, c_void_p, c_void_p, c_void_p]),
        "svdq_fp8r_export_act": (c_int, [FA, c_void_p, c_void_p, c_void_p]),
        "svdq_mx_weight_bytes": (c_size_t, [c_int, c_int, c_int, c_int]),
        "svdq_mx_act_bytes": (c_size_t, [c_int, c_int, c_int]),
        "svdq_mx_pack_weight": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                        c_void_p, c_size_t, MW, c_void_p]),
        "svdq_mx_weight_bind": (c_int, [c_int, c_int, c_int, c_int, c_void_p, c_size_t, MW]),
        "svdq_mx_act_bind": (c_int, [c_int, c_int, c_int, c_void_p, c_size_t, MA]),
        "svdq_mx_quantize_act": (c_int, [c_void_p, c_longlong, MW, MA, c_void_p]),
        "svdq_mx_gemm": (c_int, [MA, MW, c_void_p, c_int, c_void_p, c_longlong, c_int, c_void_p]),
        "svdq_mx_linear": (c_int, [c_void_p, c_longlong, MW, MA, c_void_p, c_int, c_void_p, c_longlong, c_int, c_void_p]),
        "svdq_mx_export_weight": (c_int, [MW, c_void_p, c_void_p, c_void_p]),
        "svdq_mx_export_act": (c_int, [MA, c_void_p, c_void_p, c_void_p]),
        "svdq_mx_dequantize_act": (c_int, [MA, c_void_p, c_longlong, c_int, c_void_p]),
        "svdq_block_norm": (c_int, [c_void_p, c_void_p]),
        "svdq_block_norm_quantize_mx": (c_int, [c_void_p, MW, MA, c_void_p]),
        "svdq_mlp_scratch_bytes": (c_size_t, [c_int, c_int]),
        "svdq_gemm_swiglu_quant": (c_int, [A, W, c_void_p, W, c_void_p, A, c_void_p, c_size_t, c_void_p, c_void_p]),
        "svdq_gemm_swiglu_quant_noscratch": (c_int, [A, W, c_void_p, W, c_void_p, A, c_void_p, c_void_p]),
        "svdq_weight_bytes": (c_size_t, [c_int, c_int, c_int]),
        "svdq_act_bytes": (c_size_t, [c_int, c_int, c_int]),
        "svdq_weight_bytes_tiled": (c_size_t, [c_int, c_int, c_int, c_int]),
        "svdq_pack_weight": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_void_p,
                                     c_size_t, W, c_void_p]),
        "svdq_act_bind": (c_int, [c_int, c_int, c_int, c_void_p, c_size_t, A]),
        "svdq_weight_bind": (c_int, [c_int, c_int, c_int, c_int, c_int, c_void_p, c_size_t, W]),
        "svdq_calibrate_act": (c_int, [c_void_p, c_int, W, c_void_p, c_void_p]),
        "svdq_quantize_act": (c_int, [c_void_p, W, c_void_p, A, c_void_p]),
        "svdq_gemm": (c_int, [A, W, c_void_p, c_int, c_void_p, c_int, c_void_p]),
        "svdq_export_weight": (c_int, [W, c_void_p, c_void_p, c_void_p]),
        "svdq_export_act": (c_int, [A, c_void_p, c_void_p, c_void_p]),
        "svdq_device_status": (c_int, [c_int]),
        "svdq_watchdog_selftest": (c_int, [c_ulonglong, c_void_p]),
        "svdq_set_wait_limit_ns": (c_int, [c_ulonglong]),
        "svdq_status_str": (c_char_p, [c_int]),
        "svdq_last_error": (c_char_p, []),
        "svdq_abi_version": (c_int, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args


def lib():
    """The loaded library. Raises if libsvdq.so has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                               "g.build()'` (nvcc, sm_100a)")
        l = ctypes.CDLL(LIB_PATH)
        _declare(l)
        _lib = l
    return _lib


def header_functions() -> list[str]:
    """Names of the entry points include/svdq.h declares."""
    with open(HEADER) as f:
        return sorted(set(re.findall(r"^SVDQ_API\s+[\w\s\*]+?\b(svdq_\w+)\s*\(", f.read(), re.M)))


def _check(func: str, status: int):
    if status != 0:
        raise SvdqError(func, status, lib().svdq_last_error().decode())


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _need(t, dtype, name, ndim=None):
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor, got {t.dtype} on {t.device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {tuple(t.shape)}")


class PackedWeight:
    """One layer's packed weight (device buffer + svdq_weight descriptor)."""

    def __init__(self, R: torch.Tensor, L1s: torch.Tensor | None, L2: torch.Tensor | None,
                 inv_lambda: torch.Tensor, swiglu: bool = False):
        _need(R, torch.float32, "R", 2)
        _need(inv_lambda, torch.float32, "inv_lambda", 1)
        N, K = R.shape
        r = 0 if L1s is None else L1s.shape[1]
        if r:
            _need(L1s, torch.bfloat16, "L1s", 2)
            _need(L2, torch.bfloat16, "L2", 2)
            if tuple(L1s.shape) != (K, r) or tuple(L2.shape) != (r, N):
                raise ValueError("L1s must be [K, r] and L2 [r, N]")
        nbytes = lib().svdq_weight_bytes(N, K, r)
        if nbytes == 0:
            raise SvdqError("svdq_weight_bytes", 2, f"unsupported shape N={N} K={K} r={r}")
        self.device = R.device
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=R.device)
        self.desc = SvdqWeight()
        with torch.cuda.device(R.device):
            _check("svdq_pack_weight", lib().svdq_pack_weight(
                _ptr(R), _ptr(L1s) if r else None, _ptr(L2) if r else None, _ptr(inv_lambda), N, K, r,
                1 if swiglu else 0, _ptr(self.buf), nbytes, byref(self.desc), _stream(R.device)))
        self.N, self.K, self.r, self.swiglu = N, K, r, swiglu

    @property
    def n_tile(self) -> int:
        return self.desc.n_tile

    def state_dict(self) -> dict:
        """The packed blob (on the host) and the shape fields needed to re-bind it: a checkpoint of
        the quantized weight that does not need R, the branch factors or the pack kernels again."""
        return {"abi": lib().svdq_abi_version(), "N": self.N, "K": self.K, "r": self.r, "swiglu": self.swiglu,
                "n_tile": self.n_tile, "blob": self.buf.cpu()}

    @classmethod
    def from_state(cls, state: dict, device) -> "PackedWeight":
        """A packed weight from state_dict() output, copied to `device` and re-bound (its TMA
        descriptors re-encoded for the new address)."""
        if state["abi"] != lib().svdq_abi_version():
            raise ValueError(f"checkpoint ABI {state['abi']} != library ABI {lib().svdq_abi_version()}")
        blob = state["blob"]
        if not isinstance(blob, torch.Tensor) or blob.dtype != torch.uint8 or blob.dim() != 1 \
                or not blob.is_contiguous():
            raise ValueError("checkpoint blob: expected a contiguous one-dimensional uint8 tensor")
        need = lib().svdq_weight_bytes_tiled(state["N"], state["K"], state["r"], state["n_tile"])
        if need == 0 or blob.numel() != need:
            raise ValueError(f"checkpoint blob holds {blob.numel()} bytes; a weight packed with N={state['N']} "
                             f"K={state['K']} r={state['r']} n_tile={state['n_tile']} holds {need}")
        self = cls.__new__(cls)
        self.device = torch.device(device)
        self.buf = blob.to(self.device)
        self.desc = SvdqWeight()
        self.N, self.K, self.r, self.swiglu = state["N"], state["K"], state["r"], state["swiglu"]
        with torch.cuda.device(self.device):
            _check("svdq_weight_bind", lib().svdq_weight_bind(self.N, self.K, self.r, 1 if self.swiglu else 0,
                                                              state["n_tile"], _ptr(self.buf), self.buf.numel(),
                                                              byref(self.desc)))
        return self

    def g_w(self) -> torch.Tensor:
        off = self.desc.g_w - self.buf.data_ptr()
        return self.buf[off:off + 4].view(torch.float32)


class QuantizedAct:
    """A quantized activation buffer for M rows (codes, scales, U, alpha)."""

    def __init__(self, M: int, K: int, r: int, device):
        nbytes = lib().svdq_act_bytes(M, K, r)
        if nbytes == 0:
            raise SvdqError("svdq_act_bytes", 2, f"unsupported shape M={M} K={K} r={r}")
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.desc = SvdqAct()
        _check("svdq_act_bind", lib().svdq_act_bind(M, K, r, _ptr(self.buf), nbytes, byref(self.desc)))
        self.M, self.K, self.r, self.device = M, K, r, self.buf.device

    def _view(self, ptr, nbytes):
        off = ptr - self.buf.data_ptr()
        return self.buf[off:off + nbytes]

    def U(self) -> torch.Tensor:
        """[2, M_pad, r] bf16: the hi and lo halves of X L1s / alpha."""
        n = self.desc.M_pad * self.r
        return self._view(self.desc.U, 2 * n * 2).view(torch.bfloat16).view(2, self.desc.M_pad, self.r)

    def alpha(self) -> torch.Tensor:
        return self._view(self.desc.alpha, 4).view(torch.float32)


def calibrate_act(X: torch.Tensor, w: PackedWeight, out: torch.Tensor | None = None) -> torch.Tensor:
    """Static activation scale g_x (device fp32 [1]) from calibration data X [M, K] bf16."""
    _need(X, torch.bfloat16, "X", 2)
    out = torch.empty(1, dtype=torch.float32, device=X.device) if out is None else out
    with torch.cuda.device(X.device):
        _check("svdq_calibrate_act", lib().svdq_calibrate_act(_ptr(X), X.shape[0], byref(w.desc), _ptr(out),
                                                              _stream(X.device)))
    return out


def quantize_act(X: torch.Tensor, w: PackedWeight, g_x: torch.Tensor, act: QuantizedAct) -> QuantizedAct:
    """Kernel 1: smoothing + NVFP4 quantization + low-rank down-projection."""
    _need(X, torch.bfloat16, "X", 2)
    _need(g_x, torch.float32, "g_x")
    if X.shape[0] != act.M or X.shape[1] != w.K:
        raise ValueError("X shape does not match the act buffer / weight")
    with torch.cuda.device(X.device):
        _check("svdq_quantize_act", lib().svdq_quantize_act(_ptr(X), byref(w.desc), _ptr(g_x), byref(act.desc),
                                                            _stream(X.device)))
    return act


def gemm(act: QuantizedAct, w: PackedWeight, bias: torch.Tensor | None = None, epilogue: int | None = None,
         out_dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Kernel 2: NVFP4 GEMM + low-rank up-projection + bias / SwiGLU epilogue."""
    if epilogue is None:
        epilogue = (EPI_BIAS if bias is not None else EPI_NONE) | (EPI_SWIGLU if w.swiglu else 0)
    n_out = w.N // 2 if epilogue & EPI_SWIGLU else w.N
    if out is None:
        out = torch.empty(act.M, n_out, dtype=out_dtype, device=act.device)
    _need(out, out_dtype, "out", 2)
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", 1)
    code = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    with torch.cuda.device(act.device):
        _check("svdq_gemm", lib().svdq_gemm(byref(act.desc), byref(w.desc), _ptr(bias), epilogue, _ptr(out), code,
                                            _stream(act.device)))
    return out


def linear(X, w, g_x=None, bias=None, act=None, out=None, out_dtype=torch.bfloat16):
    """The whole layer: kernel 1 then kernel 2 on the current stream. With g_x None the activation
    scale is computed from this X first (the dynamic mode: one extra amax pass over X)."""
    if g_x is None:
        g_x = calibrate_act(X, w)
    act = QuantizedAct(X.shape[0], w.K, w.r, X.device) if act is None else act
    quantize_act(X, w, g_x, act)
    return gemm(act, w, bias, out=out, out_dtype=out_dtype)


def export_weight(w: PackedWeight):
    codes = torch.empty(w.N, w.K // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(w.N, w.K // 16, dtype=torch.uint8, device=w.device)
    with torch.cuda.device(w.device):
        _check("svdq_export_weight", lib().svdq_export_weight(byref(w.desc), _ptr(codes), _ptr(scales),
                                                              _stream(w.device)))
    return codes, scales


def export_act(act: QuantizedAct):
    codes = torch.empty(act.M, act.K // 2, dtype=torch.uint8, device=act.device)
    scales = torch.empty(act.M, act.K // 16, dtype=torch.uint8, device=act.device)
    with torch.cuda.device(act.device):
        _check("svdq_export_act", lib().svdq_export_act(byref(act.desc), _ptr(codes), _ptr(scales),
                                                        _stream(act.device)))
    return codes, scales


# ---------------------------------------------------------------- MLP chain with the down layer's
# kernel 1 fused into the gate/up GEMM's SwiGLU epilogue

def gemm_swiglu_quant(act: QuantizedAct, w: PackedWeight, bias, w_next: PackedWeight, g_x_next: torch.Tensor,
                      act_next: QuantizedAct, scratch: torch.Tensor | None = None,
                      h_out: torch.Tensor | None = None) -> QuantizedAct:
    """The gate/up GEMM with SwiGLU whose epilogue also quantizes h for the next layer (act_next);
    h itself is stored only into h_out (bf16 [M, N/2]) if given."""
    if not w.swiglu:
        raise ValueError("the gate/up weight must be packed with swiglu=True")
    _need(g_x_next, torch.float32, "g_x_next")
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", 1)
    if h_out is not None:
        _need(h_out, torch.bfloat16, "h_out", 2)
    need = lib().svdq_mlp_scratch_bytes(act.M, w_next.r)
    if need == 0:
        raise SvdqError("svdq_mlp_scratch_bytes", 2, f"unsupported M={act.M} r_next={w_next.r}")
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device=act.device)
    with torch.cuda.device(act.device):
        _check("svdq_gemm_swiglu_quant", lib().svdq_gemm_swiglu_quant(
            byref(act.desc), byref(w.desc), _ptr(bias), byref(w_next.desc), _ptr(g_x_next), byref(act_next.desc),
            _ptr(scratch), scratch.numel(), _ptr(h_out), _stream(act.device)))
    return act_next


def gemm_swiglu_quant_noscratch(act: QuantizedAct, w: PackedWeight, bias, w_next: PackedWeight,
                                g_x_next: torch.Tensor, act_next: QuantizedAct,
                                h_out: torch.Tensor | None = None) -> QuantizedAct:
    """gemm_swiglu_quant for callers that cannot allocate: the partial sums of U' go to the
    library's built-in 8 MiB device buffer instead of a scratch tensor (nothing is allocated here or
    in the library). Calls on one device share that buffer: keep them ordered on one stream."""
    if not w.swiglu:
        raise ValueError("the gate/up weight must be packed with swiglu=True")
    _need(g_x_next, torch.float32, "g_x_next")
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", 1)
    if h_out is not None:
        _need(h_out, torch.bfloat16, "h_out", 2)
    with torch.cuda.device(act.device):
        _check("svdq_gemm_swiglu_quant_noscratch", lib().svdq_gemm_swiglu_quant_noscratch(
            byref(act.desc), byref(w.desc), _ptr(bias), byref(w_next.desc), _ptr(g_x_next), byref(act_next.desc),
            _ptr(h_out), _stream(act.device)))
    return act_next


def mlp(X, w_up: PackedWeight, g_x_up, w_down: PackedWeight, g_x_down, bias_up=None, bias_down=None,
        out=None, out_dtype=torch.bfloat16):
    """The MLP chain X -> SwiGLU(X W_up^T + b_up) -> (.) W_down^T + b_down with the down layer's
    activation quantization done in the gate/up GEMM's epilogue (two GEMM launches, h stays on chip)."""
    act_up = quantize_act(X, w_up, g_x_up, QuantizedAct(X.shape[0], w_up.K, w_up.r, X.device))
    act_down = QuantizedAct(X.shape[0], w_down.K, w_down.r, X.device)
    gemm_swiglu_quant(act_up, w_up, bias_up, w_down, g_x_down, act_down)
    return gemm(act_down, w_down, bias_down, out=out, out_dtype=out_dtype)


# ---------------------------------------------------------------- row-wise FP8 (W8A8) variant

class Fp8rWeight:
    """One layer's weight packed for the row-wise FP8 path (E4M3 codes, one fp32 scale per row)."""

    def __init__(self, R: torch.Tensor, L1s: torch.Tensor | None, L2: torch.Tensor | None,
                 inv_lambda: torch.Tensor, swiglu: bool = False):
        _need(R, torch.float32, "R", 2)
        _need(inv_lambda, torch.float32, "inv_lambda", 1)
        N, K = R.shape
        r = 0 if L1s is None else L1s.shape[1]
        if r:
            _need(L1s, torch.bfloat16, "L1s", 2)
            _need(L2, torch.bfloat16, "L2", 2)
            if tuple(L1s.shape) != (K, r) or tuple(L2.shape) != (r, N):
                raise ValueError("L1s must be [K, r] and L2 [r, N]")
        nbytes = lib().svdq_fp8r_weight_bytes(N, K, r)
        if nbytes == 0:
            raise SvdqError("svdq_fp8r_weight_bytes", 2, f"unsupported shape N={N} K={K} r={r}")
        self.device = R.device
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=R.device)
        self.desc = SvdqFp8rWeight()
        with torch.cuda.device(R.device):
            _check("svdq_fp8r_pack_weight", lib().svdq_fp8r_pack_weight(
                _ptr(R), _ptr(L1s) if r else None, _ptr(L2) if r else None, _ptr(inv_lambda), N, K, r,
                1 if swiglu else 0, _ptr(self.buf), nbytes, byref(self.desc), _stream(R.device)))
        self.N, self.K, self.r, self.swiglu = N, K, r, swiglu


class Fp8rAct:
    """A row-wise FP8 activation buffer for M rows (codes, row scales, U)."""

    def __init__(self, M: int, K: int, r: int, device):
        nbytes = lib().svdq_fp8r_act_bytes(M, K, r)
        if nbytes == 0:
            raise SvdqError("svdq_fp8r_act_bytes", 2, f"unsupported shape M={M} K={K} r={r}")
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.desc = SvdqFp8rAct()
        _check("svdq_fp8r_act_bind", lib().svdq_fp8r_act_bind(M, K, r, _ptr(self.buf), nbytes, byref(self.desc)))
        self.M, self.K, self.r, self.device = M, K, r, self.buf.device


def quantize_act_fp8r(X: torch.Tensor, w: Fp8rWeight, act: Fp8rAct) -> Fp8rAct:
    """Row scales, then smoothing + E4M3 quantization + low-rank down-projection."""
    _need(X, torch.bfloat16, "X", 2)
    if X.shape[0] != act.M or X.shape[1] != w.K:
        raise ValueError("X shape does not match the act buffer / weight")
    with torch.cuda.device(X.device):
        _check("svdq_fp8r_quantize_act", lib().svdq_fp8r_quantize_act(_ptr(X), byref(w.desc), byref(act.desc),
                                                                      _stream(X.device)))
    return act


def gemm_fp8r(act: Fp8rAct, w: Fp8rWeight, bias: torch.Tensor | None = None, epilogue: int | None = None,
              out_dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """FP8 GEMM + low-rank up-projection + bias / SwiGLU epilogue."""
    if epilogue is None:
        epilogue = (EPI_BIAS if bias is not None else EPI_NONE) | (EPI_SWIGLU if w.swiglu else 0)
    n_out = w.N // 2 if epilogue & EPI_SWIGLU else w.N
    if out is None:
        out = torch.empty(act.M, n_out, dtype=out_dtype, device=act.device)
    _need(out, out_dtype, "out", 2)
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", 1)
    code = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    with torch.cuda.device(act.device):
        _check("svdq_fp8r_gemm", lib().svdq_fp8r_gemm(byref(act.desc), byref(w.desc), _ptr(bias), epilogue,
                                                      _ptr(out), code, _stream(act.device)))
    return out


def linear_fp8r(X, w: Fp8rWeight, bias=None, act=None, out=None, out_dtype=torch.bfloat16):
    """The whole row-wise FP8 layer on the current stream (the activation row scales always come
    from this X)."""
    act = Fp8rAct(X.shape[0], w.K, w.r, X.device) if act is None else act
    quantize_act_fp8r(X, w, act)
    return gemm_fp8r(act, w, bias, out=out, out_dtype=out_dtype)


def export_weight_fp8r(w: Fp8rWeight):
    codes = torch.empty(w.N, w.K, dtype=torch.uint8, device=w.device)
    scales = torch.empty(w.N, dtype=torch.float32, device=w.device)
    with torch.cuda.device(w.device):
        _check("svdq_fp8r_export_weight", lib().svdq_fp8r_export_weight(byref(w.desc), _ptr(codes), _ptr(scales),
                                                                        _stream(w.device)))
    return codes, scales


def export_act_fp8r(act: Fp8rAct):
    codes = torch.empty(act.M, act.K, dtype=torch.uint8, device=act.device)
    scales = torch.empty(act.M, dtype=torch.float32, device=act.device)
    with torch.cuda.device(act.device):
        _check("svdq_fp8r_export_act", lib().svdq_fp8r_export_act(byref(act.desc), _ptr(codes), _ptr(scales),
                                                                  _stream(act.device)))
    return codes, scales


# ---------------------------------------------------------------- MXFP4 variant
# The calls of this part and the next are small enough for host time to show (a norm of a few rows takes
# the GPU 4 us), so their checks touch each tensor few times and the device guard is entered only
# where the tensors' device is not the current one.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _enqueue(device, call):
    """A call (entry point, its arguments before the stream) on the device's current stream."""
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _enqueue(device, call)
    name, *args = call
    status = getattr(_lib or lib(), name)(*args, _raw_stream(index))
    if status:
        _check(name, status)


def _rows(t, dtype, name, rows, dim, device=None):
    """Row stride of a CUDA [rows, dim] matrix whose rows are contiguous."""
    if t.dtype is not dtype or not t.is_cuda or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a two-dimensional CUDA {dtype} tensor with contiguous rows, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    if t.shape != (rows, dim):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({rows}, {dim})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.stride(0) if rows > 1 else dim  # a single row's stride says nothing


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


class MxWeight:
    """One layer's weight packed as MXFP4 (E2M1 codes, one E8M0 scale per 32 elements along K) with its
    16-bit branch. inv_lambda None: no smoothing. N and K need only be multiples of 8."""

    def __init__(self, R: torch.Tensor, L1s: torch.Tensor | None = None, L2: torch.Tensor | None = None,
                 inv_lambda: torch.Tensor | None = None, swiglu: bool = False):
        _need(R, torch.float32, "R", 2)
        N, K = R.shape
        if inv_lambda is not None:
            _need(inv_lambda, torch.float32, "inv_lambda", 1)
            if inv_lambda.shape[0] != K:
                raise ValueError("inv_lambda must be [K]")
        if (L1s is None) != (L2 is None):
            raise ValueError("L1s and L2: a branch has both")
        r = 0 if L1s is None else L1s.shape[1]
        if r:
            _need(L1s, torch.bfloat16, "L1s", 2)
            _need(L2, torch.bfloat16, "L2", 2)
            if tuple(L1s.shape) != (K, r) or tuple(L2.shape) != (r, N):
                raise ValueError("L1s must be [K, r] and L2 [r, N]")
        _same_device(R.device, L1s=L1s, L2=L2, inv_lambda=inv_lambda)
        self._allocate(N, K, r, swiglu, R.device)
        with torch.cuda.device(self.device):
            _check("svdq_mx_pack_weight", lib().svdq_mx_pack_weight(
                _ptr(R), _ptr(L1s) if r else None, _ptr(L2) if r else None, _ptr(inv_lambda), N, K, r,
                1 if swiglu else 0, _ptr(self.buf), self.buf.numel(), byref(self.desc), _stream(self.device)))

    def _allocate(self, N, K, r, swiglu, device):
        nbytes = lib().svdq_mx_weight_bytes(N, K, r, 1 if swiglu else 0)
        if nbytes == 0:
            raise SvdqError("svdq_mx_weight_bytes", 2, f"unsupported shape N={N} K={K} r={r} swiglu={swiglu}")
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.buf.device
        self.desc = SvdqMxWeight()
        self.N, self.K, self.r, self.swiglu = N, K, r, bool(swiglu)

    @property
    def n_tile(self) -> int:
        return self.desc.n_tile

    def state_dict(self) -> dict:
        """The packed blob (on the host) and what re-binds it, as PackedWeight.state_dict."""
        return {"abi": lib().svdq_abi_version(), "format": "mxfp4", "N": self.N, "K": self.K, "r": self.r,
                "swiglu": self.swiglu, "blob": self.buf.cpu()}

    @classmethod
    def from_state(cls, state: dict, device) -> "MxWeight":
        if state["abi"] != lib().svdq_abi_version() or state.get("format") != "mxfp4":
            raise ValueError(f"checkpoint ABI {state['abi']} format {state.get('format')}: expected ABI "
                             f"{lib().svdq_abi_version()} format mxfp4")
        blob = state["blob"]
        need = lib().svdq_mx_weight_bytes(state["N"], state["K"], state["r"], 1 if state["swiglu"] else 0)
        if not isinstance(blob, torch.Tensor) or blob.dtype != torch.uint8 or blob.dim() != 1 \
                or not blob.is_contiguous() or need == 0 or blob.numel() != need:
            raise ValueError(f"checkpoint blob: expected a contiguous one-dimensional uint8 tensor of {need} bytes")
        self = cls.__new__(cls)
        self._allocate(state["N"], state["K"], state["r"], state["swiglu"], device)
        self.buf.copy_(blob)
        with torch.cuda.device(self.device):
            _check("svdq_mx_weight_bind", lib().svdq_mx_weight_bind(
                self.N, self.K, self.r, 1 if self.swiglu else 0, _ptr(self.buf), self.buf.numel(), byref(self.desc)))
        return self


class MxAct:
    """An MXFP4 activation buffer for M rows (codes, scales, U)."""

    def __init__(self, M: int, K: int, r: int, device):
        nbytes = lib().svdq_mx_act_bytes(M, K, r)
        if nbytes == 0:
            raise SvdqError("svdq_mx_act_bytes", 2, f"unsupported shape M={M} K={K} r={r}")
        if torch.device(device).type != "cuda":
            raise ValueError(f"device {device}: expected a CUDA device")
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.desc = SvdqMxAct()
        _check("svdq_mx_act_bind", lib().svdq_mx_act_bind(M, K, r, _ptr(self.buf), nbytes, byref(self.desc)))
        self.M, self.K, self.r, self.device = M, K, r, self.buf.device

    def U(self) -> torch.Tensor:
        """[2, M_pad, r] bf16: the hi and lo halves of X L1s."""
        n, off = self.desc.M_pad * self.r, self.desc.U - self.buf.data_ptr()
        return self.buf[off:off + 4 * n].view(torch.bfloat16).view(2, self.desc.M_pad, self.r)


def _check_quantize_mx(X, w, act):
    if act.K != w.K or act.r != w.r:
        raise ValueError(f"act (K={act.K} r={act.r}) does not match the weight (K={w.K} r={w.r})")
    ldx = _rows(X, torch.bfloat16, "X", act.M, w.K, act.device)
    if w.device != act.device:
        raise ValueError(f"weight is on {w.device}, expected {act.device}")
    return ("svdq_mx_quantize_act", X.data_ptr(), ldx, byref(w.desc), byref(act.desc))


def quantize_act_mx(X: torch.Tensor, w: MxWeight, act: MxAct) -> MxAct:
    """Smoothing + MXFP4 quantization + low-rank down-projection in one pass over X [M, K] (rows of
    any 16-byte stride)."""
    _enqueue(act.device, _check_quantize_mx(X, w, act))
    return act


def _check_gemm_mx(act, w, bias, epilogue, out_dtype, out):
    if epilogue is None:
        epilogue = (EPI_BIAS if bias is not None else EPI_NONE) | (EPI_SWIGLU if w.swiglu else 0)
    n_out = w.N // 2 if epilogue & EPI_SWIGLU else w.N
    if out_dtype not in _OUT_CODES:
        raise ValueError(f"out_dtype {out_dtype}: expected bfloat16 or float32")
    device = act.device
    if out is None:
        out, ldy = act.buf.new_empty((act.M, n_out), dtype=out_dtype), n_out
    else:
        ldy = _rows(out, out_dtype, "out", act.M, n_out, device)
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", 1)
        if bias.shape[0] != w.N or bias.device != device:
            raise ValueError(f"bias: [{bias.shape[0]}] on {bias.device}, expected [{w.N}] on {device}")
    if w.device != device:
        raise ValueError(f"weight is on {w.device}, expected {device}")
    return out, ("svdq_mx_gemm", byref(act.desc), byref(w.desc), None if bias is None else bias.data_ptr(), epilogue,
                 out.data_ptr(), ldy, _OUT_CODES[out_dtype])


_OUT_CODES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}


def gemm_mx(act: MxAct, w: MxWeight, bias: torch.Tensor | None = None, epilogue: int | None = None,
            out_dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The MXFP4 GEMM + low-rank up-projection + bias / SwiGLU epilogue. `out` may have any row stride
    of whole 16-byte units."""
    out, call = _check_gemm_mx(act, w, bias, epilogue, out_dtype, out)
    _enqueue(act.device, call)
    return out


def linear_mx(X, w: MxWeight, bias=None, act: MxAct | None = None, out=None, out_dtype=torch.bfloat16):
    """The whole MXFP4 layer on the current stream (the format has no tensor scale to calibrate)."""
    act = MxAct(X.shape[0], w.K, w.r, X.device) if act is None else act
    _, *x_args, _, _ = _check_quantize_mx(X, w, act)
    out, (_, act_ref, w_ref, *gemm_args) = _check_gemm_mx(act, w, bias, None, out_dtype, out)
    _enqueue(act.device, ("svdq_mx_linear", *x_args, w_ref, act_ref, *gemm_args))
    return out


def _export_mx(fn, obj, rows):
    codes = torch.empty(rows, obj.K // 2, dtype=torch.uint8, device=obj.device)
    scales = torch.empty(rows, (obj.K + 31) // 32, dtype=torch.uint8, device=obj.device)
    with torch.cuda.device(obj.device):
        _check(fn, getattr(lib(), fn)(byref(obj.desc), _ptr(codes), _ptr(scales), _stream(obj.device)))
    return codes, scales


def export_weight_mx(w: MxWeight):
    return _export_mx("svdq_mx_export_weight", w, w.N)


def export_act_mx(act: MxAct):
    return _export_mx("svdq_mx_export_act", act, act.M)


def dequantize_act_mx(act: MxAct, out: torch.Tensor | None = None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """The values the quantized (smoothed) activation stands for, [M, K]."""
    if out_dtype not in _OUT_CODES:
        raise ValueError(f"out_dtype {out_dtype}: expected bfloat16 or float32")
    if out is None:
        out, ld = act.buf.new_empty((act.M, act.K), dtype=out_dtype), act.K
    else:
        ld = _rows(out, out_dtype, "out", act.M, act.K, act.device)
    _enqueue(act.device, ("svdq_mx_dequantize_act", byref(act.desc), out.data_ptr(), ld, _OUT_CODES[out_dtype]))
    return out


# ---------------------------------------------------------------- block norms

NORM_KINDS = {"rms": 1, "layer": 2}


class Norm:
    """One normalisation of rows of D: "rms" (v / sqrt(mean(v^2) + eps)) or "layer" (mean removed), times
    weight, plus bias (each optional, [D], bf16 or fp32, both of one type)."""

    def __init__(self, kind: str, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                 eps: float = 1e-6):
        if kind not in NORM_KINDS:
            raise ValueError(f"norm kind {kind!r}: expected one of {sorted(NORM_KINDS)}")
        if not eps >= 0.0:
            raise ValueError(f"eps {eps}: expected a non-negative number")
        self.kind, self.eps, self.weight, self.bias = kind, float(eps), weight, bias
        self._check()

    def _check(self):
        weight, bias = self.weight, self.bias
        self.D = self.device = None
        given = [v for v in (weight, bias) if v is not None]
        for v in given:
            if v.dtype not in (torch.bfloat16, torch.float32) or not v.is_cuda or v.dim() != 1 \
                    or not v.is_contiguous() or v.dtype != given[0].dtype or v.shape != given[0].shape:
                raise ValueError("weight and bias: expected contiguous CUDA [D] tensors of one type, bf16 or fp32")
        if given:
            self.D, self.device = given[0].shape[0], given[0].device
            _same_device(self.device, weight=weight, bias=bias)
        self._f32 = int(bool(given) and given[0].dtype == torch.float32)
        self._checked, self._pointers = (weight, bias), self._addresses()

    def _addresses(self):
        return (0 if self.weight is None else self.weight.data_ptr(), 0 if self.bias is None else self.bias.data_ptr())

    def fields(self, name, D, device):
        """The fields of svdq_norm for rows of D on `device`; vectors that were exchanged are checked again."""
        if self._checked[0] is not self.weight or self._checked[1] is not self.bias \
                or self._pointers != self._addresses():
            self._check()
        if self.D is not None and (self.D != D or self.device != device):
            raise ValueError(f"{name}: vectors of {self.D} on {self.device}, expected {D} on {device}")
        return (NORM_KINDS[self.kind], self.eps, self._f32, 0, *self._pointers)


_F32 = {torch.bfloat16: 0, torch.float32: 1}


def _norm_rows(t, name, shape=None, device=None):
    """(pointer, row stride, fp32 flag, sample stride or 0) of a [M, D] or [B, T, D] activation."""
    f32, sh = _F32.get(t.dtype), t.shape
    if f32 is None or not t.is_cuda or len(sh) not in (2, 3):
        raise ValueError(f"{name}: expected a CUDA bf16 or fp32 tensor [rows, D] or [samples, rows, D], got {t.dtype} "
                         f"{tuple(sh)} on {t.device}")
    if shape is not None and (sh != shape or t.device != device):
        raise ValueError(f"{name}: shape {tuple(sh)} on {t.device}, expected {tuple(shape)} on {device}")
    D = sh[-1]
    if t.is_contiguous():
        return t.data_ptr(), D, f32, 0
    st, T = t.stride(), sh[-2]
    if D > 1 and st[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous, got strides {st}")
    ld = st[-2] if T > 1 else D
    many = len(sh) == 3 and sh[0] > 1
    if ld < D or (many and st[0] < (T - 1) * ld + D):
        raise ValueError(f"{name}: rows overlap (strides {st})")
    return t.data_ptr(), ld, f32, st[0] if many and st[0] != T * ld else 0


def _mod(m, name, D, samples, device, f32):
    """(pointer, sample stride) of a gate, scale or shift [D] or [samples, D]."""
    if m is None:
        return 0, 0
    if _F32.get(m.dtype) != f32 or m.device != device:
        raise ValueError("gate, scale and shift: expected tensors of one type, bf16 or fp32, on x's device")
    sh = m.shape
    if (sh != (D,) and sh != (samples, D) and sh != (1, D)) or (D > 1 and m.stride(-1) != 1):
        raise ValueError(f"{name}: shape {tuple(sh)}, expected [D] or [samples, D] = [{samples}, {D}] with contiguous "
                         "rows")
    return m.data_ptr(), m.stride(0) if len(sh) == 2 and sh[0] > 1 else 0


_NO_NORM = (0, 0.0, 0, 0, 0, 0)
# svdq_block_norm_args field by field, as SvdqBlockNormArgs: packing takes a fifth of filling that structure
_PACK_NORM_ARGS = struct.Struct("@4iPPqiiPqPqPqiiPqPqPqff" + 2 * "ifiiPP" + "4q").pack


def _norm_args(x, y, gate, post, res_scale, skip_scale, norm, scale, shift, offsets, out, h):
    device, shape = x.device, x.shape
    px, ldx, x_f32, sx = _norm_rows(x, "x")
    D = shape[-1]
    if offsets is not None:
        if len(shape) != 2:
            raise ValueError("x: expected [rows, D] with offsets")
        if offsets.dtype != torch.int32 or offsets.device != device or offsets.dim() != 1 or offsets.shape[0] < 2 \
                or not offsets.is_contiguous():
            raise ValueError("offsets: expected a contiguous int32 [samples + 1] tensor on x's device")
        M, samples, T, p_off = shape[0], offsets.shape[0] - 1, 0, offsets.data_ptr()
    else:
        samples, T = (shape[0], shape[1]) if len(shape) == 3 else (1, shape[0])
        M, samples, T, p_off = samples * T, samples or 1, T or 1, 0
    first = gate if gate is not None else scale if scale is not None else shift
    mod_f32 = 0 if first is None else _F32.get(first.dtype, -1)
    p_gate, ld_gate = _mod(gate, "gate", D, samples, device, mod_f32)
    p_scale, ld_scale = _mod(scale, "scale", D, samples, device, mod_f32)
    p_shift, ld_shift = _mod(shift, "shift", D, samples, device, mod_f32)
    post_fields = _NO_NORM if post is None else post.fields("post", D, device)
    norm_fields = _NO_NORM if norm is None else norm.fields("norm", D, device)
    py, ldy, y_f32, sy, po, ldo, so = 0, 0, 0, 0, 0, 0, 0
    if y is None:
        if out is not None:
            raise ValueError("y: expected a tensor of x's shape, got None")
    else:
        py, ldy, y_f32, sy = _norm_rows(y, "y", shape, device)
        po, ldo, o_f32, so = _norm_rows(out, "out", shape, device)
        if o_f32 != x_f32:
            raise ValueError(f"out: {out.dtype}, expected x's {x.dtype}")
    ph, ldh, h_f32, sh = (0, 0, 0, 0) if h is None else _norm_rows(h, "h", shape, device)
    if M == 0:
        return None  # no row: empty tensors have no address to pass
    return _PACK_NORM_ARGS(M, D, samples, T, p_off, px, ldx, x_f32, y_f32, py, ldy, po, ldo, ph, ldh, h_f32, mod_f32,
                           p_gate, ld_gate, p_scale, ld_scale, p_shift, ld_shift, skip_scale, res_scale,
                           *post_fields, *norm_fields, sx, sy, so, sh)


def _run_norm(a, device):
    if a is not None:
        _enqueue(device, ("svdq_block_norm", a))


def _run_norm_quantize(a, x, w, act):
    if a is None:  # an activation has a row at least: it would keep what it held
        raise ValueError(f"act holds {act.M} rows, x none")
    _same_device(x.device, weight=w, act=act)
    _enqueue(x.device, ("svdq_block_norm_quantize_mx", a, byref(w.desc), byref(act.desc)))


def _like(x, dtype):
    """A contiguous tensor of x's shape."""
    if dtype is None or dtype is x.dtype:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def block_norm(x, norm: Norm, scale=None, shift=None, offsets=None, out=None, out_dtype=None):
    """h = norm(x) (1 + scale) + shift over the last axis of x [rows, D] or [samples, rows, D]; scale and
    shift [D] or one row per sample. `offsets` (int32 [samples + 1]) gives packed samples of x [rows, D];
    rows outside them are left as they are in `out`. out_dtype defaults to x's (or out's) type."""
    if out is None:
        out = _like(x, out_dtype)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out: {out.dtype}, expected {out_dtype}")
    _run_norm(_norm_args(x, None, None, None, 1.0, 1.0, norm, scale, shift, offsets, None, out), x.device)
    return out


def gated_residual(x, y, gate=None, post: Norm | None = None, res_scale: float = 1.0, skip_scale: float = 1.0,
                   norm: Norm | None = None, scale=None, shift=None, offsets=None, out=None, h=None, h_dtype=None):
    """A block's end, x' = skip_scale x + res_scale gate post(y), and (with `norm`) the next block's
    norm h = norm(x') (1 + scale) + shift, in one pass. Returns x', or (x', h). `out` may be x itself
    (the residual stream updated in place). h_dtype defaults to y's type."""
    out = _like(x, None) if out is None else out
    if norm is None and (h is not None or h_dtype is not None):
        raise ValueError("h without a norm")
    if norm is not None and h is None:
        h = _like(x, h_dtype or (y if y is not None else x).dtype)
    elif h is not None and h_dtype is not None and h.dtype != h_dtype:
        raise ValueError(f"h: {h.dtype}, expected {h_dtype}")
    _run_norm(_norm_args(x, y, gate, post, res_scale, skip_scale, norm, scale, shift, offsets, out, h), x.device)
    return out if norm is None else (out, h)


def norm_quantize_act_mx(x, norm: Norm, w: MxWeight, act: MxAct, scale=None, shift=None, offsets=None) -> MxAct:
    """block_norm whose bf16 result is quantized for the next layer instead of stored: the codes and
    scales quantize_act_mx makes of it. For weights without a branch."""
    _run_norm_quantize(_norm_args(x, None, None, None, 1.0, 1.0, norm, scale, shift, offsets, None, None), x, w, act)
    return act


def gated_residual_quantize_mx(x, y, norm: Norm, w: MxWeight, act: MxAct, gate=None, post: Norm | None = None,
                               res_scale: float = 1.0, skip_scale: float = 1.0, scale=None, shift=None, offsets=None,
                               out=None):
    """gated_residual with norm whose bf16 h is quantized for the next layer instead of stored. Returns
    (x', act). For weights without a branch."""
    out = _like(x, None) if out is None else out
    _run_norm_quantize(_norm_args(x, y, gate, post, res_scale, skip_scale, norm, scale, shift, offsets, out, None), x, w,
                       act)
    return out, act


def _norm_into_act_mx(x, norm, w, act, scale, shift, offsets):
    """The quantized norm of x in one pass, or by way of a stored h: for a branch, which projects h, and for rows
    that the pass refuses (off 16 bytes, say)."""
    if w.r == 0:
        try:
            return norm_quantize_act_mx(x, norm, w, act, scale, shift, offsets)
        except SvdqError as e:
            if e.status != ERR_UNSUPPORTED:
                raise
    h = block_norm(x, norm, scale, shift, offsets, out_dtype=torch.bfloat16)
    return quantize_act_mx(h.view(-1, w.K), w, act)


def mlp_mx(x, w_up: MxWeight, w_down: MxWeight, bias_up=None, bias_down=None, norm: Norm | None = None, scale=None,
           shift=None, post: Norm | None = None, gate=None, res_scale: float = 1.0, skip_scale: float = 1.0, offsets=None,
           acts: tuple[MxAct, MxAct] | None = None, out=None):
    """The MXFP4 MLP chain, x -> SwiGLU(x W_up^T + b_up) -> (.) W_down^T + b_down (x [rows, K] bf16; result
    bf16). With `norm` it is a transformer's whole MLP block on the residual stream x ([rows, K] or
    [samples, rows, K], bf16 or fp32):
        skip_scale x + res_scale gate post(mlp(norm(x) (1 + scale) + shift))
    in x's type, with samples, `offsets` and `out` as in gated_residual. The norm's result is quantized
    where it is computed if w_up has no branch and x's rows and the vectors lie on 16 bytes. acts: the activation buffers of the two layers, for
    callers that keep them."""
    if not w_up.swiglu or w_down.K != w_up.N // 2:
        raise ValueError(f"w_up must be packed with swiglu=True and w_down take its {w_up.N // 2} outputs, not {w_down.K}")
    if norm is None:
        if any(v is not None for v in (scale, shift, post, gate, offsets)):
            raise ValueError("scale, shift, post, gate and offsets belong to the block form: give its norm")
    elif w_down.N != x.shape[-1]:
        raise ValueError(f"w_down returns {w_down.N} values to a residual stream of {x.shape[-1]}")
    rows = x.shape[:-1].numel()
    if rows == 0:
        return out if out is not None else _like(x, None) if norm is not None else x.new_empty((0, w_down.N))
    act_up, act_down = acts or (MxAct(rows, w_up.K, w_up.r, x.device), MxAct(rows, w_down.K, w_down.r, x.device))
    if norm is None:
        quantize_act_mx(x, w_up, act_up)
    else:
        _norm_into_act_mx(x, norm, w_up, act_up, scale, shift, offsets)
    y = linear_mx(gemm_mx(act_up, w_up, bias_up), w_down, bias_down, act_down, out=out if norm is None else None)
    if norm is None:
        return y
    return gated_residual(x, y.view(x.shape), gate=gate, post=post, res_scale=res_scale, skip_scale=skip_scale,
                          offsets=offsets, out=out)


def device_status(reset: bool = True) -> int:
    """Synchronizes; returns 0, or the SVDQ_ERR_TIMEOUT status if a bounded device wait ran out."""
    return lib().svdq_device_status(1 if reset else 0)


def watchdog_selftest(limit_ns: int, device=None):
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(device):
        _check("svdq_watchdog_selftest", lib().svdq_watchdog_selftest(limit_ns, _stream(device)))


def set_wait_limit_ns(ns: int):
    _check("svdq_set_wait_limit_ns", lib().svdq_set_wait_limit_ns(ns))


def last_error() -> str:
    return lib().svdq_last_error().decode()
