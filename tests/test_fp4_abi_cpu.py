"""The 4-bit operators' C ABI and binding without a GPU: bad arguments are rejected before any CUDA call, sizes
are computed, and the reference's own steps hold."""
import ctypes

import pytest
import torch

import fp4_ref as Q

INVALID = 1
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from dense_tensor_core_gb300 import _fp4, build

    build.build()
    return _fp4._L()


def held(fmt=0, gated=0, matrices=1, rows=16, K=64, codes=0x1000, scales=0x2000, row_scale=0x3000):
    from dense_tensor_core_gb300._fp4 import fp4_matrix

    return fp4_matrix(fmt, gated, matrices, rows, K, codes, scales, row_scale)


@pytest.mark.parametrize("fmt,gated,E,rows,K,sets,groups", [
    (0, 0, 1, 1, 32, 1, 1), (0, 0, 1, 128, 64, 1, 1), (0, 0, 3, 129, 96, 2, 2), (1, 0, 1, 300, 128, 1, 3),
    (1, 0, 2, 128, 160, 2, 1), (0, 1, 2, 16, 64, 1, 1), (1, 1, 1, 272, 2080, 17, 3), (0, 0, 0, 8, 32, 1, 1),
    (0, 0, 1, 0, 64, 1, 0), (1, 0, 1, 4, 0, 0, 1)])
def test_layout(L, fmt, gated, E, rows, K, sets, groups):
    from dense_tensor_core_gb300._fp4 import fp4_info

    i = fp4_info()
    assert L.fp4_layout(ctypes.byref(held(fmt, gated, E, rows, K)), ctypes.byref(i)) == 0
    assert (i.code_bytes, i.scale_bytes, i.sets, i.groups) == (E * rows * K // 2, E * groups * sets * 512, sets, groups)


BAD_LAYOUT = [dict(fmt=2), dict(fmt=-1), dict(matrices=-1), dict(rows=-1), dict(K=-32), dict(K=48), dict(K=2 ** 24 + 32),
              dict(gated=1, rows=24), dict(rows=2 ** 31), dict(matrices=2 ** 20, rows=2 ** 20),
              dict(matrices=2 ** 24, rows=1, K=2 ** 16)]


@pytest.mark.parametrize("kw", BAD_LAYOUT)
def test_layout_rejects(L, kw):
    from dense_tensor_core_gb300._fp4 import fp4_info

    i = fp4_info()
    assert L.fp4_layout(ctypes.byref(held(**kw)), ctypes.byref(i)) == INVALID
    assert L.gemm_last_error()
    assert L.fp4_layout(None, ctypes.byref(i)) == INVALID
    assert L.fp4_layout(ctypes.byref(held()), None) == INVALID


@pytest.mark.parametrize("kw,x,ld,dtype", [(k, 0x5000, 0, 0) for k in BAD_LAYOUT] + [
    ({}, 0, 0, 0), ({}, 0x5002, 0, 0), ({}, 0x5000, 56, 0), ({}, 0x5000, 68, 0), ({}, 0x5000, -64, 0),
    ({}, 0x5000, 2 ** 31, 0), ({}, 0x5000, 0, 2), ({}, 0x5000, 0, -1), (dict(codes=0), 0x5000, 0, 0),
    (dict(scales=0), 0x5000, 0, 1), (dict(codes=0x1008), 0x5000, 0, 0), (dict(row_scale=0), 0x5000, 0, 0),
    (dict(row_scale=0x3002), 0x5000, 0, 0)])
def test_quantize_rejects(L, kw, x, ld, dtype):
    assert L.fp4_quantize(dtype, vp(x), ld, ctypes.byref(held(**kw)), None) == INVALID
    assert L.gemm_last_error()


def test_quantize_and_back_of_nothing(L):
    for kw in (dict(rows=0), dict(K=0), dict(matrices=0)):
        q = held(codes=0, scales=0, row_scale=0, **kw)
        assert L.fp4_quantize(0, None, 0, ctypes.byref(q), None) == 0
        assert L.fp4_dequantize(0, ctypes.byref(q), None, None) == 0
        assert L.fp4_pack_scales(None, ctypes.byref(q), None) == 0
    assert L.fp4_quantize(0, vp(0x5000), 0, None, None) == INVALID
    assert L.fp4_dequantize(0, None, vp(0x5000), None) == INVALID
    assert L.fp4_dequantize(3, ctypes.byref(held()), vp(0x5000), None) == INVALID
    assert L.fp4_dequantize(0, ctypes.byref(held()), vp(0x5004), None) == INVALID
    assert L.fp4_pack_scales(None, ctypes.byref(held()), None) == INVALID


def gemm(L, A=None, B=None, dtype=0, C=0x7000, **o):
    from dense_tensor_core_gb300._fp4 import gemm_fp4_options

    opts = gemm_fp4_options()
    for k, v in o.items():
        setattr(opts, k, v)
    return L.gemm_fp4(dtype, ctypes.byref(A or held()), ctypes.byref(B or held(rows=32)), vp(C), ctypes.byref(opts), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=-1), dict(C=0), dict(C=0x7002), dict(activation=7), dict(activation=-1), dict(ldc=24),
    dict(ldc=36), dict(A=held(fmt=1, row_scale=0)), dict(A=held(K=96)), dict(A=held(matrices=2)),
    dict(B=held(matrices=2, rows=32)), dict(A=held(gated=1)), dict(B=held(rows=32, gated=1)), dict(activation=5),
    dict(A=held(codes=0)), dict(B=held(scales=0)), dict(A=held(codes=0x1004)), dict(B=held(rows=12)),
    dict(bias=0x4004), dict(residual=0x4008), dict(residual=0x4000, ld_residual=8), dict(workspace=0x4004),
    dict(tile_rows=-32), dict(tile_rows=288), dict(tile_rows=48), dict(A=held(rows=100), tile_rows=96),
    dict(A=held(rows=300), tile_rows=224), dict(split_k=-1), dict(B=held(K=64, rows=2 ** 31))])
def test_gemm_rejects(L, kw):
    assert gemm(L, **kw) == INVALID
    assert L.gemm_last_error()


def test_empty_products(L):
    assert gemm(L, A=held(rows=0, codes=0, scales=0), C=0) == 0
    assert gemm(L, B=held(rows=0, codes=0, scales=0), C=0) == 0
    n = ctypes.c_uint64(7)
    assert L.gemm_fp4_workspace_size(0, 64, 64, 0, ctypes.byref(n)) == 0 and n.value == 0
    for bad in ((-1, 64, 64, 0), (1, 2 ** 31, 64, 0), (1, 64, 2 ** 25, 0), (1, 64, 64, 9)):
        assert L.gemm_fp4_workspace_size(*bad, ctypes.byref(n)) == INVALID
    assert L.gemm_fp4_workspace_size(1, 64, 64, 0, None) == INVALID


def experts(L, dtype=0, x=0x5000, weights=0x6000, plan=0x7000, y=0x8000, buffer=0x9000, T=4, k=2, E=8, H=64, F=32,
            fmt=0, w_in=None, w_out=None, **o):
    from dense_tensor_core_gb300._ffn import moe_experts_options

    opts = moe_experts_options(5, 2, None, 0, 0)
    for n, v in o.items():
        setattr(opts, n, v)
    gated = opts.activation >= 5
    wi = w_in or held(fmt, int(gated), E, 2 * F if gated else F, H)
    wo = w_out or held(fmt, 0, E, H, F)
    return L.moe_experts_fp4(dtype, vp(x), ctypes.byref(wi), ctypes.byref(wo), vp(weights), vp(plan), vp(y), T, k,
                             ctypes.byref(opts), vp(buffer), 1 << 40, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(activation=9), dict(weights_dtype=3), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(T=-1),
    dict(H=0), dict(F=0), dict(x=0), dict(weights=0), dict(plan=0), dict(y=0), dict(buffer=0), dict(x=0x5008),
    dict(plan=0x7004), dict(weights=0x6002), dict(residual=0x4008), dict(w_in=held(0, 0, 8, 64, 64)),
    dict(w_in=held(0, 1, 8, 32, 64)), dict(w_in=held(1, 1, 8, 64, 64)), dict(w_in=held(0, 1, 4, 64, 64)),
    dict(w_out=held(0, 1, 8, 64, 32)), dict(w_out=held(0, 0, 8, 96, 32)), dict(w_out=held(0, 0, 8, 64, 32, codes=0)),
    dict(fmt=2)])
def test_experts_rejects(L, kw):
    assert experts(L, **kw) == INVALID
    assert L.gemm_last_error()


def test_experts_of_no_tokens(L):
    assert experts(L, T=0, x=0, y=0, buffer=0, plan=0, weights=0) == 0


def test_binding_refuses_before_the_library():
    import dense_tensor_core_gb300 as dtc

    x = torch.zeros((8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not a CUDA tensor
        dtc.quantize_fp4(x)
    with pytest.raises(TypeError):
        dtc.quantize_fp4(x.float())
    with pytest.raises(ValueError):
        dtc.quantize_fp4(x, format="fp4")
    with pytest.raises(TypeError):
        dtc.dequantize_fp4(x)
    codes, scales = torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 4), dtype=torch.uint8)
    for bad in ((codes.int(), scales), (codes[0], scales), (codes, scales[:, :2]), (codes, scales[:4])):
        with pytest.raises((TypeError, ValueError)):
            dtc.pack_fp4(*bad)
    with pytest.raises(ValueError):
        dtc.pack_fp4(codes, scales, torch.ones(4))
    with pytest.raises(ValueError):  # not CUDA tensors
        dtc.pack_fp4(codes, scales)
    q = dtc.Fp4(codes, torch.zeros(512, dtype=torch.uint8), None, "nvfp4")
    assert q.shape == (8, 64) and "nvfp4" in repr(q)
    with pytest.raises(ValueError):
        dtc.gemm_fp4("bf16", q, q)
    with pytest.raises(TypeError):
        dtc.gemm_fp4("bf16", codes, q)
    with pytest.raises(ValueError):
        dtc.gemm_fp4("f32", q, q)
    with pytest.raises(ValueError):
        dtc.gemm_fp4("bf16", q, q, activation="tanh")


# ------------------------------------------------------------------------------------------------
# the reference's own steps
# ------------------------------------------------------------------------------------------------
def test_reference_rounds_to_the_nearest_code_ties_to_even():
    x = torch.zeros((1, 32), dtype=torch.bfloat16)
    x[0, :16] = torch.tensor([6, .25, .26, .75, .74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.48, 5, 5.03, -5, -.25])
    want = [6, 0, .5, 1, .5, 1, 1.5, 2, 2, 3, 4, 3, 4, 6, -4, 0]
    v = Q.rounded(x, "mxfp4")  # (the largest is 6: the scale is 1)
    assert v[0, :16].tolist() == want
    y = x.clone()
    y[0, 16] = 2688  # a factor of 1, and a scale of 1 for the first block
    codes, scales, g = Q.quantize(y, "nvfp4")
    assert g.tolist() == [1] and scales.tolist() == [[0x38, 0x7E]]
    assert Q.values(codes, scales, g, "nvfp4")[0, :16].tolist() == want


def test_reference_factors():
    for top, e in ((2688.0, 0), (2704.0, 1), (1344.0, -1), (1352.0, 0), (1.0, -11), (2.0 ** -120, -100), (0.0, 0)):
        x = torch.zeros((1, 32), dtype=torch.bfloat16)
        x[0, 5] = top
        assert Q.quantize(x, "nvfp4")[2].tolist() == [2.0 ** e]


def test_reference_chunks():
    s = torch.arange(130 * 6, dtype=torch.int32).remainder(251).to(torch.uint8).reshape(130, 6)
    c = Q.chunks(s, "nvfp4")
    assert c.numel() == 2 * 2 * 512
    for row, block in ((0, 0), (1, 0), (31, 3), (32, 1), (127, 5), (128, 0), (129, 4)):
        group, r, set_ = row // 128, row % 128, block // 4
        assert c[(group * 2 + set_) * 512 + 16 * (r % 32) + 4 * (r // 32) + block % 4] == s[row, block]
    g = torch.arange(16 * 2, dtype=torch.uint8).reshape(16, 2) + 1
    d = Q.chunks(g, "mxfp4", gated=True)
    for place, row in ((0, 0), (7, 7), (8, 8), (15, 15)):  # 8 gate rows, then the up rows
        assert d[16 * place] == g[row, 0]
