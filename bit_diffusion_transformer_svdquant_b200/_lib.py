"""ctypes binding of libsvdq.so (include/svdq.h). Argument marshalling only: every step of the layer
runs in the library's CUDA kernels; torch provides device memory and the current stream.

There is no fallback: if the library is missing or the device is not sm_100a, the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import struct
from ctypes import POINTER, byref, c_char_p, c_float, c_int, c_longlong, c_size_t, c_ulonglong, c_void_p
from fractions import Fraction

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


class SvdqFp8bWeight(ctypes.Structure):
    _fields_ = SvdqMxWeight._fields_


class SvdqFp8bAct(ctypes.Structure):
    _fields_ = SvdqMxAct._fields_


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


class SvdqRope(ctypes.Structure):
    _fields_ = [("dim", c_int), ("half", c_int), ("inverse", c_int), ("axes", c_int), ("axis_pairs", c_int * 4),
                ("amplitude", c_float), ("positions_i64", c_int), ("turns", c_void_p), ("positions", c_void_p),
                ("pb", c_longlong), ("pt", c_longlong)]


class SvdqHeads(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("sb", c_longlong), ("st", c_longlong), ("sh", c_longlong), ("out", c_void_p),
                ("ob", c_longlong), ("ot", c_longlong), ("oh", c_longlong), ("heads", c_int), ("reserved0", c_int),
                ("norm", SvdqNorm)]


class SvdqHeadsArgs(ctypes.Structure):
    _fields_ = [("samples", c_int), ("rows_per_sample", c_int), ("D", c_int), ("x_f32", c_int), ("out_f32", c_int),
                ("reserved0", c_int), ("q", SvdqHeads), ("k", SvdqHeads), ("v", SvdqHeads), ("rope", SvdqRope)]


class SvdqKvCache(ctypes.Structure):
    _fields_ = [("pages", c_int), ("page_size", c_int), ("heads", c_int), ("D", c_int), ("format", c_int),
                ("reserved0", c_int), ("codes", c_void_p * 2), ("scales", c_void_p * 2)]


class SvdqError(RuntimeError):
    def __init__(self, func: str, status: int, message: str):
        super().__init__(f"{func}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def _declare(lib):
    W, A = POINTER(SvdqWeight), POINTER(SvdqAct)
    FW, FA = POINTER(SvdqFp8rWeight), POINTER(SvdqFp8rAct)
    MW, MA = POINTER(SvdqMxWeight), POINTER(SvdqMxAct)
    BW, BA = POINTER(SvdqFp8bWeight), POINTER(SvdqFp8bAct)
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
        "svdq_rotary": (c_int, [c_void_p, c_void_p]),
        "svdq_kv_code_bytes": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
        "svdq_kv_scale_bytes": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
        "svdq_kv_write": (c_int, [POINTER(SvdqKvCache), c_void_p, c_void_p, c_int, c_void_p]),
        "svdq_kv_read": (c_int, [POINTER(SvdqKvCache), c_void_p, c_longlong, c_int, c_void_p, c_int, c_int, c_void_p,
                                 c_longlong, c_longlong, c_void_p, c_longlong, c_longlong, c_int, c_void_p]),
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
    for name in [n for n in sig if n.startswith("svdq_mx_")]:  # the block-scaled FP8 calls take the same arguments
        res, args = sig[name]
        sig[name.replace("svdq_mx_", "svdq_fp8b_")] = (res, [BW if a is MW else BA if a is MA else a for a in args])
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


class _ScaledWeight:
    """A weight packed with block scales, in the format of the subclass (entry points svdq_<format>_*)."""
    _prefix = _format = _desc_type = None

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
        self._call("pack_weight", _ptr(R), _ptr(L1s) if r else None, _ptr(L2) if r else None, _ptr(inv_lambda), N, K, r,
                   1 if swiglu else 0, _ptr(self.buf), self.buf.numel(), byref(self.desc), _stream(self.device))

    def _call(self, what, *args):
        name = f"{self._prefix}_{what}"
        with torch.cuda.device(self.device):
            _check(name, getattr(lib(), name)(*args))

    @classmethod
    def _bytes(cls, N, K, r, swiglu):
        return getattr(lib(), cls._prefix + "_weight_bytes")(N, K, r, 1 if swiglu else 0)

    def _allocate(self, N, K, r, swiglu, device):
        nbytes = self._bytes(N, K, r, swiglu)
        if nbytes == 0:
            raise SvdqError(self._prefix + "_weight_bytes", 2, f"unsupported shape N={N} K={K} r={r} swiglu={swiglu}")
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.buf.device
        self.desc = self._desc_type()
        self.N, self.K, self.r, self.swiglu = N, K, r, bool(swiglu)

    @property
    def n_tile(self) -> int:
        return self.desc.n_tile

    def state_dict(self) -> dict:
        """The packed blob (on the host) and what re-binds it, as PackedWeight.state_dict."""
        return {"abi": lib().svdq_abi_version(), "format": self._format, "N": self.N, "K": self.K, "r": self.r,
                "swiglu": self.swiglu, "blob": self.buf.cpu()}

    @classmethod
    def from_state(cls, state: dict, device):
        if state["abi"] != lib().svdq_abi_version() or state.get("format") != cls._format:
            raise ValueError(f"checkpoint ABI {state['abi']} format {state.get('format')}: expected ABI "
                             f"{lib().svdq_abi_version()} format {cls._format}")
        blob = state["blob"]
        need = cls._bytes(state["N"], state["K"], state["r"], state["swiglu"])
        if not isinstance(blob, torch.Tensor) or blob.dtype != torch.uint8 or blob.dim() != 1 \
                or not blob.is_contiguous() or need == 0 or blob.numel() != need:
            raise ValueError(f"checkpoint blob: expected a contiguous one-dimensional uint8 tensor of {need} bytes")
        self = cls.__new__(cls)
        self._allocate(state["N"], state["K"], state["r"], state["swiglu"], device)
        self.buf.copy_(blob)
        self._call("weight_bind", self.N, self.K, self.r, 1 if self.swiglu else 0, _ptr(self.buf), self.buf.numel(),
                   byref(self.desc))
        return self


class _ScaledAct:
    """An activation buffer for M rows (codes, scales, U), in the format of the subclass."""
    _prefix = _desc_type = None

    def __init__(self, M: int, K: int, r: int, device):
        nbytes = getattr(lib(), self._prefix + "_act_bytes")(M, K, r)
        if nbytes == 0:
            raise SvdqError(self._prefix + "_act_bytes", 2, f"unsupported shape M={M} K={K} r={r}")
        if torch.device(device).type != "cuda":
            raise ValueError(f"device {device}: expected a CUDA device")
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.desc = self._desc_type()
        name = self._prefix + "_act_bind"
        _check(name, getattr(lib(), name)(M, K, r, _ptr(self.buf), nbytes, byref(self.desc)))
        self.M, self.K, self.r, self.device = M, K, r, self.buf.device

    def U(self) -> torch.Tensor:
        """[2, M_pad, r] bf16: the hi and lo halves of X L1s."""
        n, off = self.desc.M_pad * self.r, self.desc.U - self.buf.data_ptr()
        return self.buf[off:off + 4 * n].view(torch.bfloat16).view(2, self.desc.M_pad, self.r)


class MxWeight(_ScaledWeight):
    """One layer's weight packed as MXFP4 (E2M1 codes, one E8M0 scale per 32 elements along K) with its
    16-bit branch. inv_lambda None: no smoothing. N and K need only be multiples of 8."""
    _prefix, _format, _desc_type = "svdq_mx", "mxfp4", SvdqMxWeight


class MxAct(_ScaledAct):
    """An MXFP4 activation buffer for M rows (codes, scales, U)."""
    _prefix, _desc_type = "svdq_mx", SvdqMxAct


def _check_quantize(X, w, act):
    if act.K != w.K or act.r != w.r:
        raise ValueError(f"act (K={act.K} r={act.r}) does not match the weight (K={w.K} r={w.r})")
    ldx = _rows(X, torch.bfloat16, "X", act.M, w.K, act.device)
    if w.device != act.device:
        raise ValueError(f"weight is on {w.device}, expected {act.device}")
    return (act._prefix + "_quantize_act", X.data_ptr(), ldx, byref(w.desc), byref(act.desc))


def quantize_act_mx(X: torch.Tensor, w: MxWeight, act: MxAct) -> MxAct:
    """Smoothing + MXFP4 quantization + low-rank down-projection in one pass over X [M, K] (rows of
    any 16-byte stride)."""
    _enqueue(act.device, _check_quantize(X, w, act))
    return act


def _check_gemm(act, w, bias, epilogue, out_dtype, out):
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
    return out, (act._prefix + "_gemm", byref(act.desc), byref(w.desc), None if bias is None else bias.data_ptr(),
                 epilogue, out.data_ptr(), ldy, _OUT_CODES[out_dtype])


_OUT_CODES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}


def gemm_mx(act: MxAct, w: MxWeight, bias: torch.Tensor | None = None, epilogue: int | None = None,
            out_dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The MXFP4 GEMM + low-rank up-projection + bias / SwiGLU epilogue. `out` may have any row stride
    of whole 16-byte units."""
    out, call = _check_gemm(act, w, bias, epilogue, out_dtype, out)
    _enqueue(act.device, call)
    return out


def _linear(X, w, bias, act, out, out_dtype):
    _, *x_args, _, _ = _check_quantize(X, w, act)
    out, (_, act_ref, w_ref, *gemm_args) = _check_gemm(act, w, bias, None, out_dtype, out)
    _enqueue(act.device, (act._prefix + "_linear", *x_args, w_ref, act_ref, *gemm_args))
    return out


def linear_mx(X, w: MxWeight, bias=None, act: MxAct | None = None, out=None, out_dtype=torch.bfloat16):
    """The whole MXFP4 layer on the current stream (the format has no tensor scale to calibrate)."""
    act = MxAct(X.shape[0], w.K, w.r, X.device) if act is None else act
    return _linear(X, w, bias, act, out, out_dtype)


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


def _dequantize(act, out, out_dtype):
    if out_dtype not in _OUT_CODES:
        raise ValueError(f"out_dtype {out_dtype}: expected bfloat16 or float32")
    if out is None:
        out, ld = act.buf.new_empty((act.M, act.K), dtype=out_dtype), act.K
    else:
        ld = _rows(out, out_dtype, "out", act.M, act.K, act.device)
    _enqueue(act.device, (act._prefix + "_dequantize_act", byref(act.desc), out.data_ptr(), ld, _OUT_CODES[out_dtype]))
    return out


def dequantize_act_mx(act: MxAct, out: torch.Tensor | None = None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """The values the quantized (smoothed) activation stands for, [M, K]."""
    return _dequantize(act, out, out_dtype)


# ---------------------------------------------------------------- block-scaled FP8 variant

class Fp8bWeight(_ScaledWeight):
    """One layer's weight packed as E4M3 codes with one E8M0 scale per block of 128 x 128 (rows of R in their
    original order), with its 16-bit branch. inv_lambda None: no smoothing. N and K need only be multiples of 8."""
    _prefix, _format, _desc_type = "svdq_fp8b", "fp8b", SvdqFp8bWeight


class Fp8bAct(_ScaledAct):
    """A block-scaled FP8 activation buffer for M rows: codes, one scale per row and 128 of K, U."""
    _prefix, _desc_type = "svdq_fp8b", SvdqFp8bAct


def quantize_act_fp8b(X: torch.Tensor, w: Fp8bWeight, act: Fp8bAct) -> Fp8bAct:
    """Smoothing + FP8 quantization in blocks of 128 + low-rank down-projection of X [M, K] (rows of any 16-byte
    stride)."""
    _enqueue(act.device, _check_quantize(X, w, act))
    return act


def gemm_fp8b(act: Fp8bAct, w: Fp8bWeight, bias: torch.Tensor | None = None, epilogue: int | None = None,
              out_dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The block-scaled FP8 GEMM + low-rank up-projection + bias / SwiGLU epilogue. `out` may have any row
    stride of whole 16-byte units."""
    out, call = _check_gemm(act, w, bias, epilogue, out_dtype, out)
    _enqueue(act.device, call)
    return out


def linear_fp8b(X, w: Fp8bWeight, bias=None, act: Fp8bAct | None = None, out=None, out_dtype=torch.bfloat16):
    """The whole block-scaled FP8 layer on the current stream (no tensor scale to calibrate)."""
    act = Fp8bAct(X.shape[0], w.K, w.r, X.device) if act is None else act
    return _linear(X, w, bias, act, out, out_dtype)


def _export_fp8b(fn, obj, rows, scale_rows):
    codes = torch.empty(rows, obj.K, dtype=torch.uint8, device=obj.device)
    scales = torch.empty(scale_rows, (obj.K + 127) // 128, dtype=torch.uint8, device=obj.device)
    with torch.cuda.device(obj.device):
        _check(fn, getattr(lib(), fn)(byref(obj.desc), _ptr(codes), _ptr(scales), _stream(obj.device)))
    return codes, scales


def export_weight_fp8b(w: Fp8bWeight):
    """Codes [N, K] and scale codes [ceil(N / 128), ceil(K / 128)]."""
    return _export_fp8b("svdq_fp8b_export_weight", w, w.N, (w.N + 127) // 128)


def export_act_fp8b(act: Fp8bAct):
    """Codes [M, K] and scale codes [M, ceil(K / 128)]."""
    return _export_fp8b("svdq_fp8b_export_act", act, act.M, act.M)


def dequantize_act_fp8b(act: Fp8bAct, out: torch.Tensor | None = None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """The values the quantized (smoothed) activation stands for, [M, K]."""
    return _dequantize(act, out, out_dtype)


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


# ---------------------------------------------------------------- rotary positions, key/value cache

# 2 pi to 2^-190. Frequencies are doubles; those that are exact, such as every axis's first (1 rad per position without
# scaling), would be off by 10^-7 rad at a position of 2^31 with a double's 2 pi. Others are off by as much themselves.
_TWO_PI = Fraction(628318530717958647692528676655900576839433879875021164194989, 10 ** 59)


class Rotary:
    """Rotary positions of the first `dim` values of a head, on one axis or on several (`axes`: rotated values of
    each, `dim` together). Pair i of an axis of d values turns by position * theta^(-2 i / d). layout: "interleaved"
    rotates (x[2p], x[2p + 1]), "half" (x[p], x[p + dim / 2]). scaling stretches the frequencies f for contexts longer
    than those trained on, by `factor` s:
        {"kind": "linear", "factor": s}     f / s
        {"kind": "ntk", "factor": s}        theta s^(d / (d - 2)) in place of theta
        {"kind": "yarn", "factor": s, "length": L, "beta_fast": 32, "beta_slow": 1, "amplitude": None}
            f (g + (1 - g) / s) with g = (L f / 2 pi - slow) / (fast - slow) within [0, 1], a ramp over the pair's turns
            (not over pair indices rounded at its ends, as some models' code has it): pairs that turn more than `fast` times over the trained length L keep their frequency, those below `slow` are stretched; the
            rotated values are multiplied by `amplitude` (None: 0.1 ln s + 1)."""

    def __init__(self, dim: int, axes=None, layout: str = "interleaved", theta: float = 10000.0,
                 scaling: dict | None = None, device="cuda"):
        axes = [dim] if axes is None else [int(d) for d in axes]
        if dim < 2 or dim % 2 or any(d < 2 or d % 2 for d in axes) or sum(axes) != dim or len(axes) > 4:
            raise ValueError(f"dim {dim}, axes {axes}: expected up to 4 axes of even sizes, dim together")
        if layout not in ("interleaved", "half"):
            raise ValueError(f"layout {layout!r}: expected 'interleaved' or 'half'")
        if not (theta > 0.0 and math.isfinite(theta)):
            raise ValueError(f"theta {theta}: expected a positive number")
        if torch.device(device).type != "cuda":
            raise ValueError(f"device {device}: expected a CUDA device")
        self.dim, self.axes, self.layout, self.theta = dim, axes, layout, float(theta)
        self.scaling = dict(scaling) if scaling else None
        self.frequencies, self.amplitude = self._scaled()
        turns = [round(Fraction(f) / _TWO_PI * (1 << 64)) % (1 << 64) for f in self.frequencies]
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.device = self.turns.device
        pairs = [d // 2 for d in axes]
        self._fields = (dim, int(layout == "half")), (len(axes), *pairs, *[0] * (4 - len(pairs)), self.amplitude)

    def _scaled(self):
        """(radians per position of every pair, amplitude)"""
        given = dict(self.scaling or {"kind": "linear", "factor": 1.0})
        kind, s = given.pop("kind", None), given.pop("factor", None)
        if kind not in ("linear", "ntk", "yarn") or not isinstance(s, (int, float)) or not (s > 0 and math.isfinite(s)):
            raise ValueError(f"scaling {self.scaling}: expected a kind ('linear', 'ntk' or 'yarn') and a positive factor")
        amplitude = 1.0
        if kind == "yarn":
            length, fast, slow = given.pop("length", None), given.pop("beta_fast", 32.0), given.pop("beta_slow", 1.0)
            amplitude = given.pop("amplitude", None)
            amplitude = 0.1 * math.log(s) + 1.0 if amplitude is None else float(amplitude)
            if not length or not length > 0 or not fast > slow or not math.isfinite(amplitude):
                raise ValueError(f"scaling {self.scaling}: expected a trained length and beta_fast > beta_slow")
        if given:
            raise ValueError(f"scaling {self.scaling}: {kind!r} takes no {sorted(given)}")
        out = []
        for d in self.axes:
            if kind == "ntk" and d == 2:
                raise ValueError("ntk scaling: an axis of 2 values has one frequency, 1")
            theta = self.theta * s ** (d / (d - 2)) if kind == "ntk" else self.theta
            for i in range(d // 2):
                f = theta ** (-2.0 * i / d)
                if kind == "linear":
                    f /= s
                elif kind == "yarn":
                    g = min(1.0, max(0.0, (length * f / (2.0 * math.pi) - slow) / (fast - slow)))
                    f = f * g + f / s * (1.0 - g)
                out.append(f)
        return out, amplitude

    def fields(self, positions, samples, T, device, inverse):
        """The fields of svdq_rope for `samples` x T rows on `device`."""
        if self.device != device:
            raise ValueError(f"rope is on {self.device}, expected {device}")
        n = len(self.axes)
        if positions is None or positions.dtype not in _INDEX or positions.device != device:
            raise ValueError(f"positions: expected an int32 or int64 tensor on {device}")
        sh, st = positions.shape, positions.stride()
        if n > 1:  # the last dimension is the axes'
            if len(sh) < 2 or sh[-1] != n or st[-1] != 1:
                raise ValueError(f"positions: shape {tuple(sh)} strides {st}, expected [rows, {n}] or [samples, rows, {n}] "
                                 "with contiguous axes")
            sh, st = sh[:-1], st[:-1]
        if sh != (T,) and sh != (samples, T):
            raise ValueError(f"positions: shape {tuple(positions.shape)} for {samples} x {T} rows and {n} axes")
        pb = st[0] if len(sh) == 2 and samples > 1 else 0
        pt = st[-1] if T > 1 else 0
        (dim, half), rest = self._fields
        return (dim, half, int(inverse), *rest, _INDEX[positions.dtype], self.turns.data_ptr(), positions.data_ptr(), pb, pt)


_INDEX = {torch.int32: 0, torch.int64: 1}
_NO_ROPE = (0, 0, 0, 0, 0, 0, 0, 0, 1.0, 0, 0, 0, 0, 0)
_NO_HEADS = (0,) * 10 + _NO_NORM
# svdq_heads_args field by field, as SvdqHeadsArgs
_PACK_HEADS_ARGS = struct.Struct("@6i" + 3 * "PqqqPqqqiiifiiPP" + "4i4ifiPPqq").pack


def _heads_like(x, name):
    """What q, k and v of one call share: (dtype, device, dimensions, samples, rows, D), from one of them."""
    sh, dtype, device = x.shape, x.dtype, x.device
    n = len(sh)
    if dtype not in _F32 or device.type != "cuda" or n not in (3, 4):
        raise ValueError(f"{name}: expected a CUDA bf16 or fp32 tensor [rows, heads, D] or [samples, rows, heads, D], got "
                         f"{dtype} {tuple(sh)} on {device}")
    return dtype, device, n, sh[0] if n == 4 else 1, sh[-3], sh[-1]


def _head_strides(t, name, dtype, like, heads=None):
    """(pointer, sample, row and head stride, heads) of a tensor that goes with `like`."""
    _, device, n, samples, T, D = like
    sh, st = t.shape, t.stride()
    if t.dtype is not dtype or t.device != device or len(sh) != n or sh[-1] != D or sh[-3] != T \
            or (n == 4 and sh[0] != samples) or (heads is not None and sh[-2] != heads):
        raise ValueError(f"{name}: {t.dtype} {tuple(sh)} on {t.device}, expected {dtype} "
                         f"{(samples,) * (n - 3) + (T, 'heads' if heads is None else heads, D)} on {device}")
    if D > 1 and st[-1] != 1:
        raise ValueError(f"{name}: the values of a head must be contiguous, got strides {st}")
    H = sh[-2]
    return t.data_ptr(), st[0] if samples > 1 else 0, st[-3] if T > 1 else 0, st[-2] if H > 1 else 0, H


def _heads_fields(x, name, norm, like, out=None, out_dtype=None):
    """The fields of svdq_heads of one tensor and, with out_dtype, its output: `out`, or a new one."""
    px, sb, st, sh, H = _head_strides(x, name, like[0], like)
    norm_fields = _NO_NORM if norm is None else norm.fields(name + "'s norm", like[5], like[1])
    if out_dtype is None:
        return None, (px, sb, st, sh, 0, 0, 0, 0, H, 0, *norm_fields)
    if out is None:
        out = _like(x, out_dtype)
        D = like[5]
        return out, (px, sb, st, sh, out.data_ptr(), like[4] * H * D, H * D, D, H, 0, *norm_fields)
    return out, (px, sb, st, sh, *_head_strides(out, name + "'s output", out_dtype, like, H), 0, *norm_fields)


def _out_dtype(x, out, out_dtype):
    """The type of an output that is given, asked for, or x's."""
    if out is None:
        dtype = out_dtype or x.dtype
    else:
        dtype = out.dtype
        if out_dtype is not None and dtype != out_dtype:
            raise ValueError(f"out: {dtype}, expected {out_dtype}")
    if dtype not in _F32:
        raise ValueError(f"out: {dtype}, expected bfloat16 or float32")
    return dtype


def rotary(x, rope: Rotary, positions, norm: Norm | None = None, k=None, k_norm: Norm | None = None, out=None, k_out=None,
           out_dtype=None, inverse: bool = False):
    """Rotary positions, after an optional norm over each head, of x and (in the same pass) of k: [rows, heads, D] or
    [samples, rows, heads, D], any strides with contiguous values, such as slices of a fused QKV output. positions:
    int32 or int64 [rows], [samples, rows], with several axes one more dimension. `out` may be x itself. inverse: by
    the negative angles, which undoes the rotation where its amplitude is 1. Returns out, or (out, k_out)."""
    like = _heads_like(x, "x")
    if k is None and (k_norm is not None or k_out is not None):
        raise ValueError("k_norm and k_out without k")
    dtype = _out_dtype(x, out, out_dtype)
    out, q_fields = _heads_fields(x, "x", norm, like, out, dtype)
    k_fields = _NO_HEADS
    if k is not None:
        k_out, k_fields = _heads_fields(k, "k", k_norm, like, k_out, dtype)
    x_dtype, device, _, samples, T, D = like
    rope_fields = rope.fields(positions, samples, T, device, inverse)
    if samples and T:
        _enqueue(device, ("svdq_rotary", _PACK_HEADS_ARGS(samples, T, D, _F32[x_dtype], _F32[dtype], 0, *q_fields,
                                                          *k_fields, *_NO_HEADS, *rope_fields)))
    return out if k is None else (out, k_out)


KV_FORMATS = {"fp8": 0, "mxfp4": 1}


class KvCache:
    """A paged key/value cache of quantized tokens: `pages` pages of `page_size` slots, each holding a token's key and
    value heads as E4M3 codes with one power-of-two scale per head ("fp8"), or as MXFP4 ("mxfp4", one per 32 values).
    `codes` [2, pages, page_size, heads, bytes] and `scales` [2, pages, page_size, heads, blocks] are its buffers (plane
    0 keys, 1 values), zero at first. D is a multiple of 8, at most 256."""

    def __init__(self, pages: int, page_size: int, heads: int, D: int, format: str = "fp8", device="cuda"):
        if format not in KV_FORMATS:
            raise ValueError(f"format {format!r}: expected one of {sorted(KV_FORMATS)}")
        sizes = (pages, page_size, heads, D, KV_FORMATS[format])
        if lib().svdq_kv_code_bytes(*sizes) == 0:
            raise SvdqError("svdq_kv_code_bytes", 2, f"unsupported cache pages={pages} page_size={page_size} heads={heads} "
                                                     f"D={D}")
        if torch.device(device).type != "cuda":
            raise ValueError(f"device {device}: expected a CUDA device")
        self.pages, self.page_size, self.heads, self.D, self.format = pages, page_size, heads, D, format
        self.codes, self.scales = (self._planes(n, device) for n in (lib().svdq_kv_code_bytes(*sizes),
                                                                     lib().svdq_kv_scale_bytes(*sizes)))
        self.device = self.codes.device
        self.desc = SvdqKvCache(*sizes, 0)
        for i in range(2):
            self.desc.codes[i], self.desc.scales[i] = self.codes[i].data_ptr(), self.scales[i].data_ptr()

    def _planes(self, nbytes, device):
        """Two planes of nbytes, zero, each on 256 bytes."""
        shape = (self.pages, self.page_size, self.heads)
        buf = torch.zeros(2, (nbytes + 255) // 256 * 256, dtype=torch.uint8, device=device)
        return buf[:, :nbytes].view(2, *shape, nbytes // math.prod(shape))


def kv_write(cache: KvCache, k, v, slots, rope: Rotary | None = None, positions=None, k_norm: Norm | None = None, q=None,
             q_norm: Norm | None = None, q_out=None):
    """Keys and values [rows, heads, D] (or [samples, rows, heads, D]) quantized into slots page * page_size + offset of
    the cache; slots int32 or int64, one per row, all different; rows whose slot is none of the cache's (-1: padding) are
    not written. Keys take k_norm and rope first, as in rotary. With q, its norm and rotation in the same pass;
    returns q_out then."""
    like = _heads_like(k, "k")
    dtype, device, _, samples, T, D = like
    _, k_fields = _heads_fields(k, "k", k_norm, like)
    _, v_fields = _heads_fields(v, "v", None, like)
    if device != cache.device or D != cache.D or k_fields[8] != cache.heads or v_fields[8] != cache.heads:
        raise ValueError(f"k: {k_fields[8]} heads and v: {v_fields[8]} of {D} on {device}, expected {cache.heads} of "
                         f"{cache.D} on {cache.device}")
    if slots.dtype not in _INDEX or slots.device != device or not slots.is_contiguous() \
            or slots.shape not in ((samples * T,), k.shape[:-2]):
        raise ValueError(f"slots: {slots.dtype} {tuple(slots.shape)} on {slots.device}, expected contiguous int32 or int64 "
                         f"{tuple(k.shape[:-2])} on {device}")
    if (rope is None) != (positions is None):
        raise ValueError("rope and positions go together")
    if q is None and (q_norm is not None or q_out is not None):
        raise ValueError("q_norm and q_out without q")
    q_fields, out_f32 = _NO_HEADS, 0
    if q is not None:
        q_dtype = _out_dtype(q, q_out, None)
        q_out, q_fields = _heads_fields(q, "q", q_norm, like, q_out, q_dtype)
        out_f32 = _F32[q_dtype]
    rope_fields = _NO_ROPE if rope is None else rope.fields(positions, samples, T, device, False)
    if samples and T:
        _enqueue(device, ("svdq_kv_write", byref(cache.desc), _PACK_HEADS_ARGS(
            samples, T, D, _F32[dtype], out_f32, 0, *q_fields, *k_fields, *v_fields, *rope_fields), slots.data_ptr(),
            _INDEX[slots.dtype]))
    return q_out


def kv_read(cache: KvCache, table, offsets, rows: int | None = None, out=None, out_dtype=torch.bfloat16):
    """The values of whole sequences, packed: (keys, values), each [rows, heads, D]; row i, offsets[s] <= i <
    offsets[s + 1], is token i - offsets[s] of sequence s, on page table[s, token // page_size]. table: int32
    [samples, columns]; offsets: int32 [samples + 1]. Rows outside every sequence are left as they are in `out` (a pair
    of tensors); without `out` give `rows`. Tokens on a page that is none of the cache's read as zeros."""
    device = cache.device
    if offsets.dtype != torch.int32 or offsets.device != device or offsets.dim() != 1 or offsets.shape[0] < 2 \
            or not offsets.is_contiguous():
        raise ValueError(f"offsets: expected a contiguous int32 [samples + 1] tensor on {device}")
    samples = offsets.shape[0] - 1
    if table.dtype != torch.int32 or table.device != device or table.dim() != 2 or table.shape[0] != samples \
            or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table: {table.dtype} {tuple(table.shape)} on {table.device}, expected int32 [{samples}, columns] "
                         f"with contiguous rows on {device}")
    if out is None:
        if rows is None:
            raise ValueError("rows or out: the number of rows is not known")
        if out_dtype not in _OUT_CODES:
            raise ValueError(f"out_dtype {out_dtype}: expected bfloat16 or float32")
        out = tuple(cache.codes.new_empty((rows, cache.heads, cache.D), dtype=out_dtype) for _ in range(2))
    k_out, v_out = out
    if k_out.dtype not in _OUT_CODES:
        raise ValueError(f"out: {k_out.dtype}, expected bfloat16 or float32")
    n = k_out.shape[0] if rows is None else rows
    like = (None, device, 3, 1, n, cache.D)
    pk, _, k_row, k_head, _ = _head_strides(k_out, "keys", k_out.dtype, like, cache.heads)
    pv, _, v_row, v_head, _ = _head_strides(v_out, "values", k_out.dtype, like, cache.heads)
    if n:
        _enqueue(device, ("svdq_kv_read", byref(cache.desc), table.data_ptr(), table.stride(0) if samples > 1 else
                          table.shape[1], table.shape[1], offsets.data_ptr(), samples, n, pk, k_row, k_head, pv, v_row,
                          v_head, _OUT_CODES[k_out.dtype]))
    return out


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
