"""The feed-forward operators (include/dtc_ffn.h): their Python signatures. The checks, the output
allocation and the calls are in the native module ``_ffn_native`` (csrc/ffn_binding.cpp), which
raises TypeError, ValueError or GemmError; sizes and layouts go through ctypes. Every arithmetic
step runs in the library's kernels.

stream: None for the current stream. A call allocates its outputs and buffers as under
``torch.cuda.stream(stream)``, so tensors it returns belong to that stream (``record_stream`` is for the
caller who uses them on another).
"""
import ctypes
import functools
import os

import torch

from . import _binding
from ._binding import GemmError, _check, _DTYPE, _layout_code

_ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5, "geglu": 6}
_KIND = {"bf16": 0, "f16": 1}
_LAYOUT = {"NT": 0, "NN": 1, "TN": 2, "TT": 3}
_SCORING = {"softmax": 0, "sigmoid": 1}

_vp, _i64, _i32, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64


class gemm_act_options(ctypes.Structure):
    _fields_ = [("activation", _i32), ("bias", _vp), ("residual", _vp), ("preact", _vp),
                ("lda", _i64), ("ldb", _i64), ("ldc", _i64), ("ld_residual", _i64),
                ("ld_preact", _i64), ("workspace", _vp), ("workspace_bytes", _u64),
                ("timeout_ns", _u64), ("fault_inject", _i32)]


class moe_route_options(ctypes.Structure):
    _fields_ = [("top_k", _i32), ("scoring", _i32), ("groups", _i32), ("top_groups", _i32),
                ("renormalize", _i32), ("scale", ctypes.c_float)]


class moe_plan_info(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("words", "offsets", "counts", "slots", "rows", "tiles",
                                    "scratch", "capacity", "max_tiles")]


class moe_experts_options(ctypes.Structure):
    _fields_ = [("activation", _i32), ("weights_dtype", _i32), ("residual", _vp),
                ("timeout_ns", _u64), ("fault_inject", _i32)]


class moe_experts_info(ctypes.Structure):
    _fields_ = [(n, _u64) for n in ("bytes", "x", "z", "h", "scale", "y", "split")]


_lib = None


def _L():
    global _lib
    if _lib is None:
        L = _binding.lib()
        P = ctypes.POINTER

        def sig(name, *args):
            f = getattr(L, name)
            f.restype = _i32
            f.argtypes = list(args)

        sig("gemm_act", _i32, _vp, _vp, _vp, _i64, _i64, _i64, _i32, P(gemm_act_options), _vp)
        sig("gemm_act_workspace_size", _i32, _i64, _i64, _i64, _i32, _i32, P(_u64))
        sig("gemm_act_backward", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32,
            P(gemm_act_options), _vp)
        sig("gemm_act_backward_workspace_size", _i32, _i64, _i64, _i64, _i32, _i32, P(_u64))
        sig("moe_route", _i32, _vp, _i64, _vp, _i64, _i64, P(moe_route_options), _vp, _vp, _vp)
        sig("moe_route_backward", _i32, _vp, _vp, _i64, _vp, _i64, _i64, P(moe_route_options), _vp,
            _vp)
        sig("moe_plan_layout", _i64, _i32, _i64, P(moe_plan_info))
        sig("moe_plan", _vp, _i64, _i32, _i64, _vp, _vp)
        sig("moe_experts_layout", _i32, _i64, _i32, _i64, _i64, _i64, _i32, _i32,
            P(moe_experts_info))
        sig("moe_experts", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i64, _i64, _i64,
            P(moe_experts_options), _i32, _vp, _vp)
        sig("moe_experts_backward_workspace_size", _i32, _i64, _i32, _i64, _i64, _i64, _i32, P(_u64))
        sig("moe_experts_backward", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
            _i32, _i64, _i64, _i64, P(moe_experts_options), _vp, _u64, _vp)
        _lib = L
    return _lib


_native = None


def _N():
    """The native module (raises if it has not been built)."""
    global _native
    if _native is None:
        if not os.path.exists(os.path.join(_binding.HERE, "_ffn_native.so")):
            raise RuntimeError("_ffn_native.so is missing: build it with "
                               "dense_tensor_core_gb300.build.build()")
        _L()  # the library it is linked against
        from . import _ffn_native

        _ffn_native.set_error(GemmError)
        _native = _ffn_native
    return _native


def _code(table, key, what):
    code = table.get(key)
    if code is None:
        raise ValueError(f"unknown {what} {key!r}: one of {', '.join(table)}")
    return code


def _layout(layout):
    code = _LAYOUT.get(layout)
    return _layout_code(layout) if code is None else code


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def gemm_act_workspace_size(kind, M, N, K, layout="NT", activation="none"):
    """Bytes of workspace with which gemm_act would split K over more SMs (few tiles, e.g. single
    tokens); 0 when it would not."""
    out = _u64(0)
    _check(_L().gemm_act_workspace_size(_DTYPE[kind], M, N, K, _layout_code(layout),
                                        _code(_ACT, activation, "activation"), ctypes.byref(out)))
    return out.value


def gemm_act(kind, A, B, C=None, layout="NT", bias=None, residual=None, activation="none",
             preact=None, workspace=None, timeout_ns=0, fault_inject=0, stream=None):
    """C[M,N] = act(Aop . Bop + bias) + residual, "bf16" or "f16", fp32 until the one rounding.
    Layouts as gemm_bf16's; A, B, C, residual and preact may be rows of larger row-major arrays.
    activation: none, relu, gelu, gelu_tanh, silu, or the gated swiglu / geglu (layout "NT", B
    [2N, K] with the gate rows first, bias [2N]). preact (optional, [M,N], gated [M,2N]) receives
    the sum before the activation, for gemm_act_backward. workspace: a zero-filled CUDA tensor of
    gemm_act_workspace_size bytes, reusable by later calls of the same stream, of other sizes too.
    C may be the residual."""
    return _N().gemm_act(_code(_KIND, kind, "kind"), _code(_ACT, activation, "activation"),
                         _layout(layout), A, B, C, bias, residual, preact, workspace, timeout_ns,
                         fault_inject, _handle(stream))


def gemm_act_backward_workspace_size(kind, M, N, K, layout="NT", activation="none"):
    """Bytes of workspace gemm_act_backward needs."""
    out = _u64(0)
    _check(_L().gemm_act_backward_workspace_size(_DTYPE[kind], M, N, K, _layout_code(layout),
                                                 _code(_ACT, activation, "activation"), ctypes.byref(out)))
    return out.value


def gemm_act_backward(kind, dC, A, B, preact=None, layout="NT", activation="none",
                      need=(True, True, True), workspace=None, timeout_ns=0, stream=None):
    """(dA, dB, dbias) of gemm_act from dC [M,N] and the preact it kept (not needed for "none"):
    dA and dB stored as A and B are, dbias fp32. need: which of the three to compute (the others
    are None). The gradient of a residual is dC. workspace: a zero-filled CUDA tensor of
    gemm_act_backward_workspace_size bytes, reusable like gemm_act's, also by calls of gemm_act;
    allocated here when not given."""
    act, code = _code(_ACT, activation, "activation"), _layout(layout)
    if workspace is None and dC.is_cuda and A.dim() == 2 and B.dim() == 2:
        K = A.shape[1 - code // 2]
        Nb = B.shape[0 if code in (0, 3) else 1]
        # the fill is ordered before the kernels, and the memory not reused before them, only on their
        # own stream
        with torch.cuda.device(dC.device), torch.cuda.stream(stream):
            n = gemm_act_backward_workspace_size(kind, dC.shape[0], Nb // 2 if act >= 5 else Nb, K,
                                                 layout, activation)
            workspace = torch.zeros(max(n, 16), dtype=torch.uint8, device=dC.device)
    return _N().gemm_act_backward(_code(_KIND, kind, "kind"), act, code, dC, A, B, preact,
                                  bool(need[0]), bool(need[1]), bool(need[2]), workspace, timeout_ns,
                                  _handle(stream))


# ------------------------------------------------------------------------------------------------
# routing
# ------------------------------------------------------------------------------------------------
def moe_route(logits, top_k, bias=None, scoring="softmax", groups=1, top_groups=1,
              renormalize=True, scale=1.0, weights=None, indices=None, stream=None):
    """Routes tokens to experts: logits [T,E] (bf16, fp16 or fp32, rows may be strided) to (weights
    [T,k] fp32, indices [T,k] int32). Experts are chosen by the logit (softmax) or its sigmoid plus
    `bias` [E] fp32, from the best `top_groups` of `groups` equal groups, in falling order, ties to
    the lowest index; weights come from the logits alone, over the choices (renormalize) or over all
    experts, times scale. Logits of -infinity or NaN are masked; where fewer than k experts can be
    chosen the rest are index -1 with weight 0."""
    return _N().moe_route(logits, top_k, bias, _code(_SCORING, scoring, "scoring"), groups, top_groups,
                          renormalize, scale, weights, indices, _handle(stream))


def moe_route_backward(dweights, logits, indices, scoring="softmax", renormalize=True, scale=1.0,
                       stream=None):
    """The gradient of moe_route's weights with respect to the logits: dlogits [T,E] in the logits'
    type, from dweights [T,k] fp32 and the chosen indices."""
    return _N().moe_route_backward(dweights, logits, indices, _code(_SCORING, scoring, "scoring"),
                                   renormalize, scale, _handle(stream))


@functools.lru_cache(maxsize=256)
def _plan_layout(T, k, E):
    i = moe_plan_info()
    _check(_L().moe_plan_layout(T, k, E, ctypes.byref(i)))
    return i.words, i.offsets, i.counts, i.slots, i.rows, i.capacity


class MoePlan:
    """The choices of a batch in expert order (moe_plan). `data` is the device buffer; the arrays
    below are views of it:

    * offsets [E + 1]: first row of each expert (a multiple of 16), then the end;
    * counts [E]: rows of each expert that hold a choice;
    * slots [T,k]: the row of each choice, -1 where it has none;
    * rows [capacity]: the choice t * k + j in each row, -1 in gap rows (past offsets[E]: unset).
    """

    def __init__(self, arrays, tokens, top_k, experts):
        self.data, self.offsets, self.counts, self.slots, self.rows = arrays
        self.tokens, self.top_k, self.experts = tokens, top_k, experts
        self.capacity = self.rows.shape[0]


def moe_plan(indices, experts, stream=None):
    """Puts the choices [T,k] int32 (outside 0 .. experts-1: no choice) in expert order, stable in
    the order of the tokens: a MoePlan."""
    if indices.dim() != 2:
        raise ValueError("indices must be [T, k]")
    T, k = indices.shape
    return MoePlan(_N().moe_plan(indices, experts, *_plan_layout(T, k, experts), _handle(stream)), T, k,
                   experts)


# ------------------------------------------------------------------------------------------------
# the experts
# ------------------------------------------------------------------------------------------------
@functools.lru_cache(maxsize=256)
def _experts_layout(device_index, dtype, T, k, E, H, F, act, train):
    info = moe_experts_info()
    back = _u64(0)
    with torch.cuda.device(device_index):
        _check(_L().moe_experts_layout(dtype, T, k, E, H, F, act, train, ctypes.byref(info)))
        if train:
            _check(_L().moe_experts_backward_workspace_size(dtype, T, k, E, H, F, act,
                                                            ctypes.byref(back)))
    return info.bytes, back.value


def _buffer_sizes(x, w_out, plan, code, act, train):
    """Bytes of the buffer in expert order and of the backward pass's scratch (0, 0 where the shapes
    are not those of a call: the native module says what is wrong)."""
    if not x.is_cuda or w_out.dim() != 3:
        return 0, 0
    E, H, F = w_out.shape
    return _experts_layout(x.device.index, code, plan.tokens, plan.top_k, E, H, F, act, train)


def moe_experts(kind, x, w_in, w_out, weights, plan, activation="swiglu", residual=None, out=None,
                save=False, timeout_ns=0, fault_inject=0, stream=None):
    """y[t] = residual[t] + sum_j weights[t,j] w_out[e] . act(w_in[e] . x[t]), e the j-th choice of
    token t in `plan` (moe_plan). x [T,H]; w_in [E, F, H] (gated: [E, 2F, H], gate rows first);
    w_out [E, H, F]; weights [T,k] bf16, fp16 or fp32. Experts without tokens cost nothing. With
    save, returns (y, saved) where saved is what moe_experts_backward needs."""
    code, act = _code(_KIND, kind, "kind"), _code(_ACT, activation, "activation")
    save = bool(save)
    nbytes, _ = _buffer_sizes(x, w_out, plan, code, act, save)
    return _N().moe_experts(code, act, x, w_in, w_out, weights, plan.data, plan.tokens, plan.top_k,
                            plan.experts, residual, out, save, nbytes, timeout_ns, fault_inject,
                            _handle(stream))


def moe_experts_backward(kind, dy, w_in, w_out, weights, plan, saved, activation="swiglu",
                         need_weights=True, need_x=True, timeout_ns=0, stream=None):
    """(dx, dw_in, dw_out, dweights) of moe_experts from dy [T,H] and what it saved; dw_in and
    dw_out are None without need_weights, dx without need_x. The gradient of a residual is dy."""
    code, act = _code(_KIND, kind, "kind"), _code(_ACT, activation, "activation")
    nbytes, scratch = _buffer_sizes(dy, w_out, plan, code, act, True)
    return _N().moe_experts_backward(code, act, dy, w_in, w_out, weights, plan.data, plan.tokens,
                                     plan.top_k, plan.experts, saved, nbytes, scratch, bool(need_x),
                                     bool(need_weights), timeout_ns, _handle(stream))
