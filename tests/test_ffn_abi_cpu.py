"""The feed-forward operators' C ABI and binding without a GPU: bad arguments are rejected before any
CUDA call, sizes and layouts are computed."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    from dense_tensor_core_gb300 import _ffn, build

    build.build()
    return _ffn._L()


def _act(L, dtype=0, A=0x1000, B=0x2000, C=0x3000, M=16, N=16, K=16, layout=0, back=False, **o):
    from dense_tensor_core_gb300._ffn import gemm_act_options

    opts = gemm_act_options()
    for k, v in o.items():
        setattr(opts, k, v)
    vp = ctypes.c_void_p
    if back:
        return L.gemm_act_backward(dtype, vp(C), vp(A), vp(B), vp(0x5000), vp(0x6000), None, M, N, K,
                                   layout, ctypes.byref(opts), None)
    return L.gemm_act(dtype, vp(A), vp(B), vp(C), M, N, K, layout, ctypes.byref(opts), None)


BAD_ACT = [dict(dtype=2), dict(dtype=-1), dict(layout=4), dict(activation=7), dict(activation=-1),
           dict(M=-1), dict(K=2 ** 31), dict(N=2 ** 30, activation=5), dict(A=0), dict(B=0), dict(C=0),
           dict(A=0x1008), dict(C=0x3002), dict(N=12), dict(lda=8), dict(lda=20), dict(ldb=-8),
           dict(ldc=2 ** 31), dict(workspace=0x1004)]


@pytest.mark.parametrize("kw", BAD_ACT + [dict(residual=0x4008), dict(preact=0x4004), dict(bias=0x4002),
                                          dict(residual=0x4000, ld_residual=8),
                                          dict(preact=0x4000, ld_preact=20), dict(K=12)])
def test_gemm_act_rejects(L, kw):
    assert _act(L, **kw) == INVALID
    assert L.gemm_last_error()


@pytest.mark.parametrize("kw", BAD_ACT + [dict(activation=1, preact=0), dict(K=12),
                                          dict(activation=1, preact=0x4000, ld_preact=12)])
def test_gemm_act_backward_rejects(L, kw):
    assert _act(L, back=True, **kw) == INVALID


@pytest.mark.parametrize("layout", [1, 2, 3])
@pytest.mark.parametrize("back", [False, True])
def test_gated_takes_nt_only(L, layout, back):
    assert _act(L, layout=layout, activation=5, preact=0x4000, back=back) == UNSUPPORTED


@pytest.mark.parametrize("M,N", [(16, 0), (0, 16), (0, 0)])
@pytest.mark.parametrize("act", [0, 1, 5])
def test_empty_gradient_needs_no_workspace(L, M, N, act):
    out = ctypes.c_uint64(7)
    assert L.gemm_act_backward_workspace_size(0, M, N, 64, 0, act, ctypes.byref(out)) == 0
    assert out.value == 0


def test_empty_results_are_no_ops(L):
    assert _act(L, A=0, B=0, C=0, M=0) == 0
    assert _act(L, A=0, B=0, C=0, N=0) == 0


def _route(L, dtype=2, logits=0x1000, ld=0, T=4, E=64, weights=0x2000, indices=0x3000, none=False, **o):
    from dense_tensor_core_gb300._ffn import moe_route_options

    opts = moe_route_options(8, 0, 1, 1, 1, 1.0)
    for k, v in o.items():
        setattr(opts, k, v)
    vp = ctypes.c_void_p
    return L.moe_route(dtype, vp(logits), ld, None, T, E, None if none else ctypes.byref(opts),
                       vp(weights), vp(indices), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(none=True), dict(T=-1), dict(E=0), dict(E=1025), dict(scoring=2),
    dict(groups=0), dict(groups=33), dict(groups=3), dict(groups=4, top_groups=5), dict(top_groups=0),
    dict(top_k=0), dict(top_k=33), dict(E=4), dict(groups=8, top_groups=1, top_k=9), dict(ld=32),
    dict(logits=0), dict(weights=0), dict(indices=0), dict(logits=0x1002), dict(indices=0x3002)])
def test_route_rejects(L, kw):
    assert _route(L, **kw) == INVALID
    assert L.gemm_last_error()


def test_route_of_no_tokens(L):
    assert _route(L, T=0, logits=0, weights=0, indices=0) == 0


def test_plan_layout(L):
    from dense_tensor_core_gb300._ffn import moe_plan_info

    i = moe_plan_info()
    for T, k, E in [(0, 1, 1), (1, 8, 64), (100, 6, 60), (5000, 8, 256)]:
        assert L.moe_plan_layout(T, k, E, ctypes.byref(i)) == 0
        n = T * k
        assert i.capacity % 16 == 0 and i.capacity >= n + 15 * min(E, n)
        assert i.max_tiles >= min(E, n) + n // 256
        spans = [(0, 1), (i.tiles, 4 * i.max_tiles), (i.offsets, E + 1), (i.counts, E), (i.slots, n),
                 (i.rows, i.capacity)]
        ends = sorted((a, a + b) for a, b in spans)
        assert all(x[1] <= y[0] for x, y in zip(ends, ends[1:])) and ends[-1][1] <= i.words
        assert i.tiles % 4 == 0  # 16-byte records


@pytest.mark.parametrize("T,k,E", [(-1, 1, 8), (1, 0, 8), (1, 33, 64), (1, 1, 0), (1, 1, 1025),
                                   (2 ** 31, 1, 8), (2 ** 30, 2, 8)])
def test_plan_layout_rejects(L, T, k, E):
    from dense_tensor_core_gb300._ffn import moe_plan_info

    assert L.moe_plan_layout(T, k, E, ctypes.byref(moe_plan_info())) == INVALID
    assert L.moe_plan_layout(1, 1, 8, None) == INVALID


def _experts(L, dtype=0, x=0x1000, w_in=0x2000, w_out=0x3000, weights=0x4000, plan=0x5000, y=0x6000, T=4,
             k=2, E=8, H=64, F=64, buffer=0x7000, back=False, **o):
    from dense_tensor_core_gb300._ffn import moe_experts_options

    opts = moe_experts_options(5, 2, None, 0, 0)
    for n, v in o.items():
        setattr(opts, n, v)
    vp = ctypes.c_void_p
    if back:
        return L.moe_experts_backward(dtype, vp(x), vp(w_in), vp(w_out), vp(weights), vp(plan), vp(buffer),
                                      vp(y), vp(0x8000), vp(0x9000), vp(0xA000), T, k, E, H, F,
                                      ctypes.byref(opts), vp(0xB000), 1 << 40, None)
    return L.moe_experts(dtype, vp(x), vp(w_in), vp(w_out), vp(weights), vp(plan), vp(y), T, k, E, H, F,
                         ctypes.byref(opts), 0, vp(buffer), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(activation=9), dict(weights_dtype=3), dict(k=0), dict(E=0), dict(T=-1), dict(H=0),
    dict(H=12), dict(F=4), dict(F=20), dict(E=1024, H=2 ** 24), dict(x=0), dict(w_in=0), dict(w_out=0),
    dict(weights=0), dict(plan=0), dict(buffer=0), dict(x=0x1008), dict(w_in=0x2004), dict(plan=0x5004),
    dict(weights=0x4002)])
def test_experts_rejects(L, kw, back):
    assert _experts(L, back=back, **kw) == INVALID
    assert L.gemm_last_error()


def test_experts_of_no_tokens(L):
    assert _experts(L, T=0, x=0, y=0, buffer=0, plan=0, weights=0) == 0


def test_binding_refuses_before_the_library():
    import dense_tensor_core_gb300 as dtc

    a = torch.zeros((8, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not CUDA tensors
        dtc.gemm_act("bf16", a, a)
    with pytest.raises(TypeError):
        dtc.gemm_act("f16", a, a)
    with pytest.raises(ValueError):
        dtc.gemm_act("bf16", a, a, activation="tanh")
    with pytest.raises(ValueError):
        dtc.gemm_act("mxfp8", a, a)
    with pytest.raises(TypeError):
        dtc.moe_route(torch.zeros((4, 8), dtype=torch.float64), 2)
    with pytest.raises(ValueError):
        dtc.moe_route(torch.zeros((4, 8)), 2)
    with pytest.raises(ValueError):
        dtc.moe_route(torch.zeros((4, 8)), 2, scoring="relu")
    with pytest.raises(TypeError):
        dtc.moe_plan(torch.zeros((4, 2), dtype=torch.int64), 8)
