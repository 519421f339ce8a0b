"""ctypes binding of the feed-forward operators (include/dtc_ffn.h): argument marshalling only, in
the manner of ``_binding``. Every arithmetic step runs in the library's kernels.
"""
import ctypes
import functools

import torch

from . import _binding
from ._binding import _check, _check_tensor, _DTYPE, _layout_code, _layout_name, _ld

_ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5, "geglu": 6}
_GATED = ("swiglu", "geglu")
_KIND = {"bf16": torch.bfloat16, "f16": torch.float16}
_FLOAT_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
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


# The current stream's handle without building a Stream object (several microseconds).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(dev, stream, f, *args):
    """The C call on `dev` (made current where it is not) and the given or current stream, which
    is the last argument of every entry point that enqueues work."""
    index = dev.index
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index:
        status = f(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = f(*args, handle)
    if status:
        _check(status)


def _mat(t, dt, name, dev):
    """Checks a 2-D operand that may be rows of a larger row-major array; its leading dimension (0:
    dense)."""
    if t.dtype is not dt or t.device != dev or not t.is_contiguous() or not t.is_cuda:
        _check_tensor(t, dt, name, True)
        if t.device != dev:
            raise ValueError(f"all tensors must be on one CUDA device, got {name} on {t.device} "
                             f"and others on {dev}")
        return _ld(t)
    return 0


def _dense(t, dt, name, dev):
    if t.dtype is not dt or t.device != dev or not t.is_contiguous() or not t.is_cuda:
        _check_tensor(t, dt, name)
        raise ValueError(f"all tensors must be on one CUDA device, got {name} on {t.device} and "
                         f"others on {dev}")


def _act_code(activation):
    if activation not in _ACT:
        raise ValueError(f"unknown activation {activation!r}: one of {', '.join(_ACT)}")
    return _ACT[activation]


def _kind_dtype(kind):
    if kind not in _KIND:
        raise ValueError(f"unknown kind {kind!r}: bf16 or f16")
    return _KIND[kind]


def _shape(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


# layout: (code, A stored [K,M], B stored [N,K])
_LAYOUT = {"NT": (0, False, True), "NN": (1, False, False), "TN": (2, True, False),
           "TT": (3, True, True)}


def _act_shapes(A, B, layout, gated):
    """(layout code, M, N, K, stored columns of Bop) of a gemm_act call."""
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    found = _LAYOUT.get(layout)
    if found is None:
        found = _LAYOUT[_layout_name(layout)]
    code, a_t, b_t = found
    M, K = A.shape
    if a_t:
        M, K = K, M
    Nb, Kb = B.shape
    if not b_t:
        Nb, Kb = Kb, Nb
    if Kb != K:
        raise ValueError(f"inner sizes differ: A is {tuple(A.shape)}, B is {tuple(B.shape)} ({layout})")
    if gated and Nb % 2:
        raise ValueError(f"a gated activation needs an even number of columns, got {Nb}")
    return code, M, Nb // 2 if gated else Nb, K, Nb


def _ws(workspace, dev):
    if workspace is None:
        return None, 0
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor of the operands' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _addr(t):
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def gemm_act_workspace_size(kind, M, N, K, layout="NT", activation="none"):
    """Bytes of workspace with which gemm_act would split K over more SMs (few tiles, e.g. single
    tokens); 0 when it would not."""
    out = _u64(0)
    _check(_L().gemm_act_workspace_size(_DTYPE[kind], M, N, K, _layout_code(layout),
                                        _act_code(activation), ctypes.byref(out)))
    return out.value


def gemm_act(kind, A, B, C=None, layout="NT", bias=None, residual=None, activation="none",
             preact=None, workspace=None, timeout_ns=0, fault_inject=0, stream=None):
    """C[M,N] = act(Aop . Bop + bias) + residual, "bf16" or "f16", fp32 until the one rounding.
    Layouts as gemm_bf16's; A, B, C, residual and preact may be rows of larger row-major arrays.
    activation: none, relu, gelu, gelu_tanh, silu, or the gated swiglu / geglu (layout "NT", B
    [2N, K] with the gate rows first, bias [2N]). preact (optional, [M,N], gated [M,2N]) receives
    the sum before the activation, for gemm_act_backward. workspace: a zero-filled CUDA tensor of
    gemm_act_workspace_size bytes, reusable by later calls of the same stream. C may be the
    residual."""
    dt = _kind_dtype(kind)
    act = _act_code(activation)
    dev = A.device
    lda, ldb = _mat(A, dt, "A", dev), _mat(B, dt, "B", dev)
    code, M, N, K, Nb = _act_shapes(A, B, layout, activation in _GATED)
    ldc = ldr = ldz = 0
    bias_p = res_p = pre_p = None
    if C is None:
        C = torch.empty((M, N), dtype=dt, device=dev)
    else:
        ldc = _mat(C, dt, "C", dev)
        _shape(C, (M, N), "C")
    if bias is not None:
        _dense(bias, dt, "bias", dev)
        _shape(bias, (Nb,), "bias")
        bias_p = _addr(bias)
    if residual is not None:
        ldr = _mat(residual, dt, "residual", dev)
        _shape(residual, (M, N), "residual")
        res_p = _addr(residual)
    if preact is not None:
        ldz = _mat(preact, dt, "preact", dev)
        _shape(preact, (M, Nb), "preact")
        pre_p = _addr(preact)
    ws, ws_bytes = _ws(workspace, dev)
    o = gemm_act_options(act, bias_p, res_p, pre_p, lda, ldb, ldc, ldr, ldz, ws, ws_bytes,
                         timeout_ns, fault_inject)
    _call(dev, stream, _L().gemm_act, _DTYPE[kind], _addr(A), _addr(B), _addr(C), M, N, K, code,
          ctypes.byref(o))
    return C


def gemm_act_backward_workspace_size(kind, M, N, K, layout="NT", activation="none"):
    """Bytes of workspace gemm_act_backward needs."""
    out = _u64(0)
    _check(_L().gemm_act_backward_workspace_size(_DTYPE[kind], M, N, K, _layout_code(layout),
                                                 _act_code(activation), ctypes.byref(out)))
    return out.value


def gemm_act_backward(kind, dC, A, B, preact=None, layout="NT", activation="none",
                      need=(True, True, True), workspace=None, timeout_ns=0, stream=None):
    """(dA, dB, dbias) of gemm_act from dC [M,N] and the preact it kept (not needed for "none"):
    dA and dB stored as A and B are, dbias fp32. need: which of the three to compute (the others
    are None). The gradient of a residual is dC. workspace: a zero-filled CUDA tensor of
    gemm_act_backward_workspace_size bytes; allocated here when not given."""
    dt = _kind_dtype(kind)
    act = _act_code(activation)
    dev = dC.device
    ldc, lda, ldb = (_mat(t, dt, name, dev) for t, name in ((dC, "dC"), (A, "A"), (B, "B")))
    code, M, N, K, Nb = _act_shapes(A, B, layout, activation in _GATED)
    _shape(dC, (M, N), "dC")
    pre_p, ldz = None, 0
    if act:
        if preact is None:
            raise ValueError(f"the gradient of {activation} needs preact")
        ldz = _mat(preact, dt, "preact", dev)
        _shape(preact, (M, Nb), "preact")
        pre_p = _addr(preact)
    if workspace is None:
        with torch.cuda.device(dev):
            n = gemm_act_backward_workspace_size(kind, M, N, K, layout, activation)
        workspace = torch.zeros(max(n, 16), dtype=torch.uint8, device=dev)
    ws, ws_bytes = _ws(workspace, dev)
    dA = torch.empty(A.shape, dtype=dt, device=dev) if need[0] else None
    dB = torch.empty(B.shape, dtype=dt, device=dev) if need[1] else None
    db = torch.empty((Nb,), dtype=torch.float32, device=dev) if need[2] else None
    o = gemm_act_options(act, None, None, pre_p, lda, ldb, ldc, 0, ldz, ws, ws_bytes, timeout_ns, 0)
    _call(dev, stream, _L().gemm_act_backward, _DTYPE[kind], _addr(dC), _addr(A), _addr(B),
          _addr(dA), _addr(dB), _addr(db), M, N, K, code, ctypes.byref(o))
    return dA, dB, db


# ------------------------------------------------------------------------------------------------
# routing
# ------------------------------------------------------------------------------------------------
def _route_args(logits, top_k, scoring, groups, top_groups, renormalize, scale):
    code = _FLOAT_CODE.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be bf16, fp16 or fp32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if scoring not in _SCORING:
        raise ValueError(f"unknown scoring {scoring!r}: softmax or sigmoid")
    return code, _mat(logits, logits.dtype, "logits", logits.device), moe_route_options(
        top_k, _SCORING[scoring], groups, top_groups, 1 if renormalize else 0, scale)


def moe_route(logits, top_k, bias=None, scoring="softmax", groups=1, top_groups=1,
              renormalize=True, scale=1.0, weights=None, indices=None, stream=None):
    """Routes tokens to experts: logits [T,E] (bf16, fp16 or fp32, rows may be strided) to (weights
    [T,k] fp32, indices [T,k] int32). Experts are chosen by the logit (softmax) or its sigmoid plus
    `bias` [E] fp32, from the best `top_groups` of `groups` equal groups, in falling order, ties to
    the lowest index; weights come from the logits alone, over the choices (renormalize) or over all
    experts, times scale. Logits of -infinity or NaN are masked; where fewer than k experts can be
    chosen the rest are index -1 with weight 0."""
    code, ld, o = _route_args(logits, top_k, scoring, groups, top_groups, renormalize, scale)
    T, E = logits.shape
    dev = logits.device
    if bias is not None:
        _dense(bias, torch.float32, "bias", dev)
        _shape(bias, (E,), "bias")
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    else:
        _dense(weights, torch.float32, "weights", dev)
        _shape(weights, (T, top_k), "weights")
    if indices is None:
        indices = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    else:
        _dense(indices, torch.int32, "indices", dev)
        _shape(indices, (T, top_k), "indices")
    _call(dev, stream, _L().moe_route, code, _addr(logits), ld, _addr(bias), T, E, ctypes.byref(o),
          _addr(weights), _addr(indices))
    return weights, indices


def moe_route_backward(dweights, logits, indices, scoring="softmax", renormalize=True, scale=1.0,
                       stream=None):
    """The gradient of moe_route's weights with respect to the logits: dlogits [T,E] in the logits'
    type, from dweights [T,k] fp32 and the chosen indices."""
    if indices.dim() != 2:
        raise ValueError("indices must be [T, k]")
    k = indices.shape[1]
    code, ld, o = _route_args(logits, k, scoring, 1, 1, renormalize, scale)
    T, E = logits.shape
    dev = logits.device
    _dense(indices, torch.int32, "indices", dev)
    _dense(dweights, torch.float32, "dweights", dev)
    _shape(indices, (T, k), "indices")
    _shape(dweights, (T, k), "dweights")
    out = torch.empty((T, E), dtype=logits.dtype, device=dev)
    _call(dev, stream, _L().moe_route_backward, code, _addr(dweights), _addr(logits), ld,
          _addr(indices), T, E, ctypes.byref(o), _addr(out))
    return out


@functools.lru_cache(maxsize=256)
def _plan_layout(T, k, E):
    info = moe_plan_info()
    _check(_L().moe_plan_layout(T, k, E, ctypes.byref(info)))
    return info


class MoePlan:
    """The choices of a batch in expert order (moe_plan). `data` is the device buffer; the arrays
    below are views of it:

    * offsets [E + 1]: first row of each expert (a multiple of 16), then the end;
    * counts [E]: rows of each expert that hold a choice;
    * slots [T,k]: the row of each choice, -1 where it has none;
    * rows [capacity]: the choice t * k + j in each row, -1 in gap rows (past offsets[E]: unset).
    """

    def __init__(self, data, layout, tokens, top_k, experts):
        self.data, self._layout = data, layout
        self.tokens, self.top_k, self.experts = tokens, top_k, experts
        self.capacity = layout.capacity

    def _view(self, at, n):
        return self.data[at:at + n]

    @property
    def offsets(self):
        return self._view(self._layout.offsets, self.experts + 1)

    @property
    def counts(self):
        return self._view(self._layout.counts, self.experts)

    @property
    def slots(self):
        return self._view(self._layout.slots, self.tokens * self.top_k).view(self.tokens, self.top_k)

    @property
    def rows(self):
        return self._view(self._layout.rows, self.capacity)


def moe_plan(indices, experts, stream=None):
    """Puts the choices [T,k] int32 (outside 0 .. experts-1: no choice) in expert order, stable in
    the order of the tokens: a MoePlan."""
    dev = indices.device
    _dense(indices, torch.int32, "indices", dev)
    if indices.dim() != 2:
        raise ValueError("indices must be [T, k]")
    T, k = indices.shape
    layout = _plan_layout(T, k, experts)
    data = torch.empty(layout.words, dtype=torch.int32, device=dev)
    _call(dev, stream, _L().moe_plan, _addr(indices), T, k, experts, data.data_ptr())
    return MoePlan(data, layout, T, k, experts)


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


def _experts_args(kind, x, w_in, w_out, weights, plan, activation, name):
    dt = _kind_dtype(kind)
    act = _act_code(activation)
    dev = x.device
    _dense(x, dt, name, dev)
    _dense(w_in, dt, "w_in", dev)
    _dense(w_out, dt, "w_out", dev)
    if x.dim() != 2 or w_in.dim() != 3 or w_out.dim() != 3:
        raise ValueError(f"{name} must be [T, H], w_in [E, F, H] (gated [E, 2F, H]), w_out [E, H, F]")
    T, H = x.shape
    E, _, F = w_out.shape
    _shape(w_out, (E, H, F), "w_out")
    _shape(w_in, (E, 2 * F if activation in _GATED else F, H), "w_in")
    if plan.tokens != T or plan.experts != E:
        raise ValueError(f"the plan is for {plan.tokens} tokens and {plan.experts} experts, not "
                         f"{T} and {E}")
    wcode = _FLOAT_CODE.get(weights.dtype)
    if wcode is None:
        raise TypeError(f"weights must be bf16, fp16 or fp32, got {weights.dtype}")
    _dense(weights, weights.dtype, "weights", dev)
    _shape(weights, (T, plan.top_k), "weights")
    if plan.data.device != dev:
        raise ValueError(f"the plan is on {plan.data.device}, the tensors on {dev}")
    return dt, dev, act, wcode, T, E, H, F


def moe_experts(kind, x, w_in, w_out, weights, plan, activation="swiglu", residual=None, out=None,
                save=False, timeout_ns=0, fault_inject=0, stream=None):
    """y[t] = residual[t] + sum_j weights[t,j] w_out[e] . act(w_in[e] . x[t]), e the j-th choice of
    token t in `plan` (moe_plan). x [T,H]; w_in [E, F, H] (gated: [E, 2F, H], gate rows first);
    w_out [E, H, F]; weights [T,k] bf16, fp16 or fp32. Experts without tokens cost nothing. With
    save, returns (y, saved) where saved is what moe_experts_backward needs."""
    dt, dev, act, wcode, T, E, H, F = _experts_args(kind, x, w_in, w_out, weights, plan, activation,
                                                    "x")
    if residual is not None:
        _dense(residual, dt, "residual", dev)
        _shape(residual, (T, H), "residual")
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=dev)
    else:
        _dense(out, dt, "out", dev)
        _shape(out, (T, H), "out")
    nbytes, _ = _experts_layout(dev.index, _DTYPE[kind], T, plan.top_k, E, H, F, act, int(save))
    buffer = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    o = moe_experts_options(act, wcode, _addr(residual), timeout_ns, fault_inject)
    _call(dev, stream, _L().moe_experts, _DTYPE[kind], _addr(x), _addr(w_in), _addr(w_out),
          _addr(weights), plan.data.data_ptr(), _addr(out), T, plan.top_k, E, H, F, ctypes.byref(o), int(save),
          buffer.data_ptr())
    return (out, buffer) if save else out


def moe_experts_backward(kind, dy, w_in, w_out, weights, plan, saved, activation="swiglu",
                         need_weights=True, need_x=True, timeout_ns=0, stream=None):
    """(dx, dw_in, dw_out, dweights) of moe_experts from dy [T,H] and what it saved; dw_in and
    dw_out are None without need_weights, dx without need_x. The gradient of a residual is dy."""
    dt, dev, act, wcode, T, E, H, F = _experts_args(kind, dy, w_in, w_out, weights, plan, activation,
                                                    "dy")
    nbytes, back = _experts_layout(dev.index, _DTYPE[kind], T, plan.top_k, E, H, F, act, 1)
    if saved.dtype != torch.uint8 or saved.numel() != nbytes or saved.device != dev:
        raise ValueError("saved is not what moe_experts returned for these sizes with save=True")
    ws = torch.empty(back, dtype=torch.uint8, device=dev)
    dx = torch.empty((T, H), dtype=dt, device=dev) if need_x else None
    dwi = torch.empty(w_in.shape, dtype=dt, device=dev) if need_weights else None
    dwo = torch.empty(w_out.shape, dtype=dt, device=dev) if need_weights else None
    dw = torch.empty(weights.shape, dtype=weights.dtype, device=dev)
    o = moe_experts_options(act, wcode, None, timeout_ns, 0)
    _call(dev, stream, _L().moe_experts_backward, _DTYPE[kind], _addr(dy), _addr(w_in), _addr(w_out),
          _addr(weights), plan.data.data_ptr(), _addr(saved), _addr(dx), _addr(dwi), _addr(dwo),
          _addr(dw), T, plan.top_k, E, H, F, ctypes.byref(o), ws.data_ptr(), back)
    return dx, dwi, dwo, dw
