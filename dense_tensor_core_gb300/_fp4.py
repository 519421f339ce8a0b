"""The 4-bit operators (include/dtc_fp4.h): their Python signatures, and the class of a matrix held in 4
bits. Checks, output allocation and calls are in the native module (csrc/fp4_binding.cpp), as for the
feed-forward operators; every arithmetic step runs in the library's kernels.

stream: None for the current stream; outputs and buffers belong to the stream of the call.
"""
import ctypes
import functools

import torch

from . import _ffn
from ._binding import _check
from ._ffn import _ACT, _KIND, _N, _code, _handle

_FORMAT = {"nvfp4": 0, "mxfp4": 1}
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_vp, _i64, _i32, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64


class fp4_matrix(ctypes.Structure):
    _fields_ = [("format", _i32), ("gated", _i32), ("matrices", _i64), ("rows", _i64), ("K", _i64),
                ("codes", _vp), ("scales", _vp), ("row_scale", _vp)]


class fp4_info(ctypes.Structure):
    _fields_ = [("code_bytes", _u64), ("scale_bytes", _u64), ("sets", _i64), ("groups", _i64)]


class gemm_fp4_options(ctypes.Structure):
    _fields_ = [("activation", _i32), ("bias", _vp), ("residual", _vp), ("ldc", _i64), ("ld_residual", _i64),
                ("workspace", _vp), ("workspace_bytes", _u64), ("tile_rows", _i32), ("split_k", _i32),
                ("timeout_ns", _u64), ("fault_inject", _i32)]


_lib = None


def _L():
    global _lib
    if _lib is None:
        L = _ffn._L()
        P = ctypes.POINTER

        def sig(name, *args):
            f = getattr(L, name)
            f.restype = _i32
            f.argtypes = list(args)

        m = P(fp4_matrix)
        sig("fp4_layout", m, P(fp4_info))
        sig("fp4_quantize", _i32, _vp, _i64, m, _vp)
        sig("fp4_dequantize", _i32, m, _vp, _vp)
        sig("fp4_pack_scales", _vp, m, _vp)
        sig("gemm_fp4", _i32, m, m, _vp, P(gemm_fp4_options), _vp)
        sig("gemm_fp4_workspace_size", _i64, _i64, _i64, _i32, P(_u64))
        sig("moe_experts_fp4", _i32, _vp, m, m, _vp, _vp, _vp, _i64, _i32, P(_ffn.moe_experts_options), _vp,
            _u64, _vp)
        sig("moe_experts_fp4_buffer_size", _i32, _i64, _i32, _i64, _i64, _i64, _i32, P(_u64))
        _lib = L
    return _lib


class Fp4:
    """A matrix [rows, K], or a stack [matrices, rows, K], held in 4 bits (quantize_fp4, pack_fp4):

    * codes [..., rows, K / 2] uint8: e2m1 codes, element k in the low nibble of byte k / 2 for even k;
    * scales uint8: the blocks' scales in the order in which the tensor cores take them;
    * row_scale [..., rows] fp32: the rows' factors (None: all 1);
    * shape; format "nvfp4" or "mxfp4"; gated: the scales are ordered for a gated product (gate rows first).
    """

    __slots__ = ("shape", "format", "gated", "_parts", "_views")

    def __init__(self, codes, scales, row_scale, format, gated=False):
        if codes.dim() not in (2, 3):
            raise ValueError("codes must be [rows, K / 2] or [matrices, rows, K / 2]")
        self.shape = (*codes.shape[:-1], 2 * codes.shape[-1])
        self.format, self.gated = format, bool(gated)
        self._views = (codes, scales, row_scale)
        self._parts = (codes, scales, row_scale, _code(_FORMAT, format, "format"), int(self.gated),
                       codes.shape[0] if codes.dim() == 3 else 1, codes.shape[-2], 2 * codes.shape[-1])

    def _look(self):
        if self._views is None:
            data, _, _, fmt, gated, matrices, rows, K = self._parts
            self._views = _N().fp4_views(data, fmt, gated, matrices, rows, K, len(self.shape) == 3)
        return self._views

    codes = property(lambda self: self._look()[0])
    scales = property(lambda self: self._look()[1])
    row_scale = property(lambda self: self._look()[2])

    def __repr__(self):
        return f"Fp4({list(self.shape)}, {self.format!r}{', gated' if self.gated else ''})"


def _held(q, name):
    if not isinstance(q, Fp4):
        raise TypeError(f"{name} must be an Fp4, got {type(q).__name__}")
    return q._parts


def quantize_fp4(x, format="nvfp4", gated=False, out=None, stream=None):
    """x [rows, K] (bf16 or fp16, may be rows of a larger array) or [matrices, rows, K] (dense) as an Fp4.
    K must be a multiple of 32. "nvfp4": e2m1 codes with a UE4M3 scale per 16 elements and a factor, a power of
    two, per row; "mxfp4": an E8M0 scale per 32. Ties go to even. A block with an infinity or NaN becomes NaN.
    gated: x is the weight of a gated product, gate rows first. out: an Fp4 of this shape, format and order
    whose buffers are written."""
    fmt, gated = _code(_FORMAT, format, "format"), bool(gated)
    data, matrices, rows, K = _N().quantize_fp4(x, fmt, int(gated), None if out is None else _held(out, "out"),
                                                _handle(stream))
    if out is not None:
        return out
    q = Fp4.__new__(Fp4)
    q.shape, q.format, q.gated, q._views = tuple(x.shape), format, gated, None
    q._parts = (data, None, None, fmt, int(gated), matrices, rows, K)
    return q


def dequantize_fp4(q, dtype=torch.bfloat16, out=None, stream=None):
    """The values that q stands for, in bf16, fp16 or fp32."""
    if dtype not in _DTYPE:
        raise TypeError(f"dtype must be bf16, fp16 or fp32, got {dtype}")
    parts = _held(q, "q")
    return _N().dequantize_fp4(parts, _DTYPE[dtype], out, len(q.shape) == 3, _handle(stream))


def pack_fp4(codes, scales, row_scale=None, format="nvfp4", gated=False, stream=None):
    """An Fp4 of codes [..., rows, K / 2], scales [..., rows, K / block] (row-major bytes, block 16 for "nvfp4"
    and 32 for "mxfp4", as gemm_nvfp4 takes them) and the rows' factors. codes and row_scale are kept as they
    are, the scales are put into the tensor cores' order."""
    if codes.dtype != torch.uint8:
        raise TypeError(f"codes must be uint8, got {codes.dtype}")
    if codes.dim() not in (2, 3):
        raise ValueError("codes must be [rows, K / 2] or [matrices, rows, K / 2]")
    block = 16 if format == "nvfp4" else 32
    want = (*codes.shape[:-1], 2 * codes.shape[-1] // block)
    if tuple(scales.shape) != want:
        raise ValueError(f"scales must be {want}, got {tuple(scales.shape)}")
    if row_scale is not None and tuple(row_scale.shape) != tuple(codes.shape[:-1]):
        raise ValueError(f"row_scale must be {tuple(codes.shape[:-1])}, got {tuple(row_scale.shape)}")
    packed = _N().pack_fp4(scales, codes.shape[0] if codes.dim() == 3 else 1, codes.shape[-2], 2 * codes.shape[-1],
                           _code(_FORMAT, format, "format"), int(bool(gated)), _handle(stream))
    return Fp4(codes, packed, row_scale, format, gated)


def gemm_fp4_workspace_size(M, N, K, activation="none"):
    """Bytes of workspace with which gemm_fp4 would split K over more SMs; 0 when it would not. A bound over both
    formats: NVFP4 products of up to 16 rows may take none of it."""
    out = _u64(0)
    _check(_L().gemm_fp4_workspace_size(M, N, K, _code(_ACT, activation, "activation"), ctypes.byref(out)))
    return out.value


def gemm_fp4(kind, A, B, C=None, bias=None, residual=None, activation="none", workspace=None, tile_rows=0,
             split_k=0, timeout_ns=0, fault_inject=0, stream=None):
    """C[M,N] = act(A . B^T + bias) + residual, C, bias and residual "bf16" or "f16", fp32 until the one rounding.
    A: an Fp4 [M, K]; B: an Fp4 [N, K] of the same format, for the gated activations (swiglu, geglu) [2N, K]
    with gated=True. C and residual may be rows of larger arrays, C may be the residual. workspace: a zero-filled
    CUDA tensor of gemm_fp4_workspace_size bytes, reusable like gemm_act's, also by its calls. tile_rows, split_k:
    0 for the plan's choice."""
    return _N().gemm_fp4(_code(_KIND, kind, "kind"), _code(_ACT, activation, "activation"), _held(A, "A"),
                         _held(B, "B"), C, bias, residual, workspace, tile_rows, split_k, timeout_ns, fault_inject,
                         _handle(stream))


@functools.lru_cache(maxsize=256)
def _buffer_size(device_index, fmt, T, k, E, H, F, act):
    out = _u64(0)
    with torch.cuda.device(device_index):
        _check(_L().moe_experts_fp4_buffer_size(fmt, T, k, E, H, F, act, ctypes.byref(out)))
    return out.value


def moe_experts_fp4(kind, x, w_in, w_out, weights, plan, activation="swiglu", residual=None, out=None,
                    timeout_ns=0, fault_inject=0, stream=None):
    """moe_experts with weights held in 4 bits: y[t] = residual[t] + sum_j weights[t,j] w_out[e] . q(h), h =
    act(w_in[e] . q(x[t])) rounded to 16 bits, q(v) the row v as quantize_fp4 makes it in the weights' format.
    x [T,H]; w_in an Fp4 [E, F, H] (gated: [E, 2F, H] with gated=True); w_out an Fp4 [E, H, F]; weights [T,k]
    bf16, fp16 or fp32; plan from moe_plan. H and F must be multiples of 32."""
    code, act = _code(_KIND, kind, "kind"), _code(_ACT, activation, "activation")
    wi, wo = _held(w_in, "w_in"), _held(w_out, "w_out")
    nbytes = 0
    if x.is_cuda:
        nbytes = _buffer_size(x.device.index, wo[3], plan.tokens, plan.top_k, wo[5], wo[6], wo[7], act)
    return _N().moe_experts_fp4(code, act, x, wi, wo, weights, plan.data, plan.tokens, plan.top_k, plan.experts,
                                residual, out, nbytes, timeout_ns, fault_inject, _handle(stream))
