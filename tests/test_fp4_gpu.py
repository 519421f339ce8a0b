"""The 4-bit operators on the GPU against 64-bit references: quantisation code by code, the product and its
epilogue, routed experts, and runs of them together."""
import math

import pytest
import torch

import ffn_ref as R
import fp4_ref as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(M, K, kind, seed, spread=1.0):
    g = gen(seed)
    x = torch.randn((M, K), generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn((M, 1), generator=g, device="cuda"))
    x *= torch.exp(spread * torch.randn((M, K), generator=g, device="cuda"))
    return x.to(R.DT[kind])


def same_bits(q, x, fmt, gated=False):
    codes, scales, g = Q.quantize(x, fmt)
    got = Q.unpack(q.codes)  # (a zero's sign is left open)
    assert torch.equal(torch.where(got == 8, 0, got), torch.where(codes == 8, 0, codes))
    if fmt == "nvfp4":
        assert torch.equal(q.row_scale, g)
    else:
        assert q.row_scale is None
    want = Q.chunks(scales, fmt, gated)
    got = q.scales.cpu()
    assert got.shape == want.shape
    # places past the rows hold anything
    live = Q.chunks(torch.ones_like(scales), fmt, gated) != 0
    assert torch.equal(got[live], want[live])
    # and places past K in rows that exist hold 0
    E = scales.shape[0] if scales.dim() == 3 else 1
    blocks = scales.shape[-1]
    if blocks % 4 and not gated:
        chunk = got.reshape(E, -1, (blocks + 3) // 4, 32, 4, 4)
        assert int(chunk[:, 0, -1, 0, 0, blocks % 4:].sum()) == 0


# ------------------------------------------------------------------------------------------------
# quantisation
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 8192), (3, 96), (130, 64), (33, 992), (7, 1056), (300, 2080), (5, 4128),
                                 (4, 8224), (2, 16384), (3, 16416), (2, 40000), (9, 1536), (9, 1568), (5, 6144), (5, 6176),
                                 (2, 12288), (2, 12320)])
def test_quantize(fmt, kind, M, K):
    import dense_tensor_core_gb300 as dtc
    x = rows(M, K, kind, M + K)
    if M > 2:
        x[1] = 0
        x[2, :32] = 0
        x[2, 40] = -0.0
    q = dtc.quantize_fp4(x, format=fmt)
    assert q.shape == (M, K) and q.format == fmt
    same_bits(q, x, fmt)
    want = Q.rounded(x, fmt)
    for dtype in (torch.bfloat16, torch.float32):  # exact
        v = dtc.dequantize_fp4(q, dtype=dtype)
        assert v.dtype == dtype and torch.equal(v.double(), want)
    v = dtc.dequantize_fp4(q, dtype=torch.float16).double()
    assert bool((torch.isinf(v) | ((v - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25)).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_every_value_against_every_scale(fmt, kind):
    """Rows that hold every finite number of the type beside a block maximum of each significand: the codes
    of all ratios of a value to a scale, ties among them."""
    import dense_tensor_core_gb300 as dtc
    dt = R.DT[kind]
    bits = torch.arange(0x8000, device="cuda", dtype=torch.int32).to(torch.int16).view(dt)
    vals = bits[torch.isfinite(bits)]
    step = 4 if kind == "f16" else 1  # significands of the largest element
    for i in range(0, 2 ** (10 if kind == "f16" else 7), step):
        top = torch.tensor([(1 + i / 2 ** (10 if kind == "f16" else 7))], device="cuda").to(dt)
        v = vals[(vals <= top) & (vals > top.float() / 4096)]  # smaller ones are zeros: see below
        v = torch.cat([v, v.new_zeros(-v.numel() % 15)]).reshape(-1, 15)
        b = torch.cat([top.expand(v.shape[0], 1), v], 1)  # a block of 16 each, the maximum first
        if fmt == "mxfp4":
            b = torch.cat([b, -b], 1)
        x = b.reshape(1, -1)
        x = torch.cat([x, x.new_zeros((1, -x.shape[1] % 32))], 1)
        same_bits(dtc.quantize_fp4(x, format=fmt), x, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_largest_and_smallest_rows(fmt):
    import dense_tensor_core_gb300 as dtc
    x = torch.zeros((12, 64), device="cuda")
    x[0, 3], x[1, 3], x[2, 3], x[3, 3] = 2.0 ** -133, 2.0 ** -126, 2.0 ** -100, 1.5 * 2.0 ** -127
    x[4], x[5, 7], x[5, 40] = 2.0 ** 127, 2.0 ** 127, 2.0 ** 90
    x[6, 0], x[6, 20] = 2688.0, 6.0
    x[7, 0] = 2704.0
    x[8, 0], x[8, 16], x[8, 32], x[8, 48] = 2688.0, 6 * 2.0 ** -9, 3 * 2.0 ** -9, 3.03125 * 2.0 ** -9
    x[9, 0], x[9, 1], x[9, 33] = 7.5, 8.0, 7.0
    x[10], x[11, :3] = -2.0 ** -60, torch.tensor([-1.0, -0.0, 1e-30])
    x = x.bfloat16()
    q = dtc.quantize_fp4(x, format=fmt)
    same_bits(q, x, fmt)
    assert torch.equal(dtc.dequantize_fp4(q, dtype=torch.float32).double(), Q.rounded(x, fmt))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_infinities_and_nan_stay_in_their_block(fmt, kind):
    import dense_tensor_core_gb300 as dtc
    x = rows(5, 160, kind, 3, 0.3)
    x[0, 5], x[1, 40], x[2, 159] = float("inf"), float("nan"), float("-inf")
    x[3] = float("nan")
    q = dtc.quantize_fp4(x, format=fmt)
    same_bits(q, x, fmt)
    v = dtc.dequantize_fp4(q)
    n = Q.BLOCK[fmt]
    bad = (~torch.isfinite(x)).unflatten(-1, (-1, n)).any(-1)[..., None].expand(-1, -1, n).flatten(-2)
    assert torch.equal(torch.isnan(v), bad)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("E,M,K,gated", [(3, 40, 96, False), (2, 130, 64, False), (3, 48, 160, True), (1, 16, 32, True),
                                         (2, 144, 1056, True)])
def test_stacks_and_gated_order(fmt, E, M, K, gated):
    import dense_tensor_core_gb300 as dtc
    x = rows(E * M, K, "bf16", 9).reshape(E, M, K)
    q = dtc.quantize_fp4(x, format=fmt, gated=gated)
    assert q.shape == (E, M, K)
    same_bits(q, x, fmt, gated)
    assert torch.equal(dtc.dequantize_fp4(q).double(), Q.rounded(x, fmt))
    # the same from codes and scales in rows
    codes, scales, g = Q.quantize(x, fmt)
    p = dtc.pack_fp4(Q.pack(codes), scales, g, format=fmt, gated=gated)
    assert torch.equal(p.scales.cpu(), Q.chunks(scales, fmt, gated))
    assert torch.equal(dtc.dequantize_fp4(p).double(), Q.rounded(x, fmt))


def test_strided_rows_given_outputs_and_no_rows():
    import dense_tensor_core_gb300 as dtc
    big = rows(40, 512, "f16", 4)
    x = big[::2, 64:352]
    q = dtc.quantize_fp4(x)
    same_bits(q, x, "nvfp4")
    out = dtc.quantize_fp4(torch.ones_like(x))
    assert dtc.quantize_fp4(x, out=out) is out and torch.equal(out.codes, q.codes)
    same_bits(out, x, "nvfp4")
    v = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    assert dtc.dequantize_fp4(q, dtype=torch.float32, out=v) is v
    assert torch.equal(v.double(), Q.rounded(x, "nvfp4"))
    for shape in ((0, 64), (4, 0), (0, 16, 64)):
        e = dtc.quantize_fp4(torch.empty(shape, dtype=torch.float16, device="cuda"))
        assert e.shape == shape and dtc.dequantize_fp4(e).shape == shape


# ------------------------------------------------------------------------------------------------
# the product
# ------------------------------------------------------------------------------------------------
def operands(kind, fmt, M, N, K, act, seed=0):
    Nb = 2 * N if act in R.GATED else N
    g = gen(seed)
    a = rows(M, K, kind, seed + 1, 0.4)
    b = (torch.randn((Nb, K), generator=g, device="cuda") * K ** -0.5).to(R.DT[kind])
    return a, b, Nb


def rand(shape, kind, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(R.DT[kind])


def run(kind, fmt, M, N, K, act="none", bias=False, res=False, ws=True, seed=0, **kw):
    import dense_tensor_core_gb300 as dtc
    a, b, Nb = operands(kind, fmt, M, N, K, act, seed)
    bi = rand((Nb,), kind, seed + 2, 0.2) if bias else None
    re = rand((M, N), kind, seed + 3) if res else None
    qa, qb = dtc.quantize_fp4(a, format=fmt), dtc.quantize_fp4(b, format=fmt, gated=act in R.GATED)
    w = None
    if ws:
        n = 1 << 26 if kw.get("split_k") else dtc.gemm_fp4_workspace_size(M, N, K, activation=act)
        w = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    y = dtc.gemm_fp4(kind, qa, qb, bias=bi, residual=re, activation=act, workspace=w, **kw)
    dtc.gemm_stream_status()
    want, bound = Q.product(kind, Q.rounded(a, fmt), Q.rounded(b, fmt), bi, re, act)
    R.check(y, want, bound, f"{kind} {fmt} {M}x{N}x{K} {act} {kw}")
    return y


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (128, 256, 256), (32, 8, 64), (1, 256, 256), (5, 72, 96), (33, 136, 160),
                                   (64, 264, 1056), (100, 520, 992), (257, 504, 544), (300, 1032, 2080),
                                   (1, 2048, 4096), (17, 640, 8192), (600, 256, 320)])
def test_gemm_shapes(fmt, kind, M, N, K):
    run(kind, fmt, M, N, K, bias=M % 2 == 1, res=N % 16 == 8)


@pytest.mark.parametrize("M,N,K,act", [(1, 5000, 288, "none"), (8, 9000, 96, "silu"), (3, 2600, 160, "swiglu"),
                                       (2, 4400, 1056, "geglu"), (16, 4000, 64, "none"), (9, 5000, 128, "gelu"),
                                       (1, 10000, 64, "none"), (4, 5136, 8192, "none")])
def test_gemm_few_rows_many_features(M, N, K, act):
    for kind in ("bf16", "f16"):
        run(kind, "nvfp4", M, N, K, act, bias=True, res=M % 2 == 0)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 64, 96), (70, 200, 288), (260, 136, 512)])
def test_gemm_activations(fmt, act, M, N, K):
    run("bf16", fmt, M, N, K, act, bias=True, res=M != 70)
    run("f16", fmt, M, N, K, act, bias=False, res=M == 70)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tile", [32, 64, 96, 128, 160, 192, 224, 256])
def test_gemm_tiles(fmt, tile):
    """Every tile height: one tile that holds all rows, and (multiples of 64) several."""
    run("bf16", fmt, tile - 3, 392, 1120, tile_rows=tile)
    if tile % 64 == 0:
        run("bf16", fmt, 3 * tile + 5, 264, 608, bias=True, tile_rows=tile)
        run("f16", fmt, 2 * tile, 136, 352, "swiglu", tile_rows=tile)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K,split,tile", [(1, 256, 2048, 4, 32), (40, 264, 4128, 3, 64), (200, 136, 1568, 2, 224),
                                              (1, 8, 8192, 16, 32), (300, 256, 1024, 2, 128)])
def test_gemm_splits(fmt, M, N, K, split, tile):
    a = run("bf16", fmt, M, N, K, bias=True, res=True, split_k=split, tile_rows=tile)
    b = run("bf16", fmt, M, N, K, bias=True, res=True, split_k=split, tile_rows=tile)
    assert torch.equal(a, b)
    run("f16", fmt, M, N, K, "geglu", split_k=split, tile_rows=tile)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(1500, 4096, 512), (4000, 2056, 1024), (2048, 4104, 288)])
def test_gemm_many_tiles(fmt, M, N, K):
    """More tiles than pairs: accumulators by turns, scale columns reused, tiles beyond whole waves split."""
    run("bf16", fmt, M, N, K, "gelu", bias=True, res=True)
    run("f16", fmt, M, N // 2 // 8 * 8, K, "swiglu", bias=True)
    run("bf16", fmt, M, N, K, tile_rows=64)


def test_each_element_and_scale_is_its_own():
    """One-hot operands: every place of K and of the scale blocks, and every row and column, is read where it
    belongs (a wrong scale order or place changes a value)."""
    import dense_tensor_core_gb300 as dtc
    for fmt in ("nvfp4", "mxfp4"):
        n, K, M, N = Q.BLOCK[fmt], 544, 256, 272
        g = gen(8)
        codes = torch.randint(0, 16, (M, K), generator=g, device="cuda", dtype=torch.uint8)
        lo, hi = (0x28, 0x48) if fmt == "nvfp4" else (120, 134)
        scales = torch.randint(lo, hi, (M, K // n), generator=g, device="cuda", dtype=torch.uint8)
        f = torch.rand(M, generator=g, device="cuda") + 0.5
        a = dtc.pack_fp4(Q.pack(codes), scales, f, format=fmt)
        va = Q.values(codes, scales, None, fmt) * f.double()[:, None]
        for k0 in (0, N):
            one = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
            s1 = torch.randint(lo, hi, (N, K // n), generator=g, device="cuda", dtype=torch.uint8)
            i = torch.arange(N, device="cuda")
            one[i, k0 + i] = 2  # 1.0
            b = dtc.pack_fp4(Q.pack(one), s1, None, format=fmt)
            y = dtc.gemm_fp4("f16", a, b).double()
            want = va @ Q.values(one, s1, None, fmt).t()
            assert bool(((y - want).abs() <= 2.0 ** -10 * want.abs() + 2.0 ** -24).all())


def test_nan_scales_reach_their_rows_only():
    import dense_tensor_core_gb300 as dtc
    a, b, _ = operands("bf16", "nvfp4", 70, 72, 256, "none")
    a[5, 17] = float("nan")
    b[9, 200] = float("inf")
    for fmt in ("nvfp4", "mxfp4"):
        y = dtc.gemm_fp4("bf16", dtc.quantize_fp4(a, format=fmt), dtc.quantize_fp4(b, format=fmt))
        want = torch.zeros((70, 72), dtype=torch.bool, device="cuda")
        want[5] = True
        want[:, 9] = True
        assert torch.equal(torch.isnan(y), want)


def test_strided_results_and_in_place_residual():
    import dense_tensor_core_gb300 as dtc
    kind, fmt, M, N, K = "bf16", "nvfp4", 150, 200, 320
    a, b, _ = operands(kind, fmt, M, N, K, "none")
    qa, qb = dtc.quantize_fp4(a), dtc.quantize_fp4(b)
    res = rand((M, N), kind, 6)
    want = dtc.gemm_fp4(kind, qa, qb, residual=res)
    big = torch.full((M + 2, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    view = big[1:M + 1, 8:8 + N]
    view.copy_(res)
    assert dtc.gemm_fp4(kind, qa, qb, C=view, residual=view) is view and torch.equal(view, want)
    big[1:M + 1, 8:8 + N] = 7.0
    assert bool((big == 7.0).all())


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
def test_degenerate_sizes(act):
    import dense_tensor_core_gb300 as dtc
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    gated = act in R.GATED
    q = lambda r, k, g=False: dtc.quantize_fp4(z(r, k), gated=g)  # noqa: E731
    assert dtc.gemm_fp4("bf16", q(0, 64), q(32, 64, gated), activation=act).shape == (0, 16 if gated else 32)
    bias, res = rand((32,), "bf16", 1), rand((5, 16 if gated else 32), "bf16", 2)
    y = dtc.gemm_fp4("bf16", q(5, 0), q(32, 0, gated), bias=bias, residual=res, activation=act)
    want = R.act(bias.double(), act) + res.double()
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17).all())


def test_workspace_is_shared_with_gemm_act():
    import dense_tensor_core_gb300 as dtc
    n = max(dtc.gemm_fp4_workspace_size(1, 4096, 8192), dtc.gemm_act_workspace_size("bf16", 24, 512, 8192))
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    a, b, _ = operands("bf16", "nvfp4", 1, 4096, 8192, "none")
    qa, qb = dtc.quantize_fp4(a), dtc.quantize_fp4(b)
    c, d = rand((24, 8192), "bf16", 1), rand((512, 8192), "bf16", 2)
    want = dtc.gemm_fp4("bf16", qa, qb, workspace=ws), dtc.gemm_act("bf16", c, d, workspace=ws)
    for _ in range(3):
        got = dtc.gemm_fp4("bf16", qa, qb, workspace=ws), dtc.gemm_act("bf16", c, d, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------------------------
# the experts
# ------------------------------------------------------------------------------------------------
def experts_case(kind, fmt, T, E, k, H, F, act, seed=0, masked=True):
    g = gen(seed)
    x = rows(T, H, kind, seed + 1, 0.4)
    Fz = 2 * F if act in R.GATED else F
    wi, wo = rand((E, Fz, H), kind, seed + 2, H ** -0.5), rand((E, H, F), kind, seed + 3, F ** -0.5)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]) if T else \
        torch.zeros((0, k), device="cuda", dtype=torch.int64)
    idx = idx.to(torch.int32)
    if masked and T > 2:
        idx[1] = -1  # a token without an expert
        idx[2, k - 1] = -1
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    return x, wi, wo, idx, w


def experts_reference(kind, fmt, x, wi, wo, idx, w, res, act):
    xq = Q.rounded(x, fmt)
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda") if res is None else res.double()
    for e in range(wi.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            h = R.act(xq[t] @ Q.rounded(wi[e], fmt).t(), act).to(R.DT[kind])
            y.index_add_(0, t, w[t, j, None].double() * (Q.rounded(h, fmt) @ Q.rounded(wo[e], fmt).t()))
    return y


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F,act", [
    (1, 8, 2, 128, 64, "swiglu"), (1, 64, 8, 512, 256, "swiglu"), (5, 8, 8, 96, 32, "gelu"), (40, 8, 2, 288, 160, "silu"),
    (300, 4, 2, 512, 96, "geglu"), (700, 3, 1, 256, 224, "none"), (1000, 2, 2, 160, 544, "relu"), (77, 48, 6, 544, 352, "swiglu"),
    (900, 1, 1, 128, 64, "gelu_tanh")])
def test_experts(fmt, T, E, k, H, F, act):
    """In 64 bits h is as close as can be, but a value next to a rounding border of its 16-bit type or of its
    codes may fall on the other side: one step of h's code there (at most 1/3 of the value with its block's scale
    the same), on few of F values. The norm of the difference is held to 2 roundings of the result's type and
    those: 1 in 100 of the values with a 16-bit neighbour, of which 1 in 16 changes a code."""
    import dense_tensor_core_gb300 as dtc
    for kind in ("bf16", "f16"):
        x, wi, wo, idx, w = experts_case(kind, fmt, T, E, k, H, F, act)
        res = rand((T, H), kind, 7) if T % 2 else None
        plan = dtc.moe_plan(idx, E)
        y = dtc.moe_experts_fp4(kind, x, dtc.quantize_fp4(wi, format=fmt, gated=act in R.GATED),
                                dtc.quantize_fp4(wo, format=fmt), w, plan, activation=act, residual=res)
        dtc.gemm_stream_status()
        R.close(y, experts_reference(kind, fmt, x, wi, wo, idx, w, res, act),
                2 * R.U[kind] + (1 / 3) * (1 / 1600) ** 0.5, f"{kind} {fmt}")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F", [(9, 4, 2, 2080, 64), (5, 3, 2, 4128, 96), (6, 2, 1, 8224, 64), (300, 2, 1, 8224, 64),
                                       (6, 2, 2, 64, 2080), (6, 2, 2, 96, 8224), (60, 1024, 4, 96, 64), (40, 33, 32, 64, 32)])
def test_experts_of_wide_rows_many_experts_and_many_choices(fmt, T, E, k, H, F):
    test_experts(fmt, T, E, k, H, F, "swiglu")


@pytest.mark.parametrize("T", [3, 60])
def test_experts_chosen_twice_and_weights_of_any_sign(T):
    """A token may choose an expert twice; weights may be 0 or negative. Tolerance as in test_experts."""
    import dense_tensor_core_gb300 as dtc
    kind, fmt, act, E, k, H, F = "bf16", "nvfp4", "swiglu", 5, 4, 256, 96
    x, wi, wo, idx, w = experts_case(kind, fmt, T, E, k, H, F, act, masked=False)
    idx[:, 1] = idx[:, 0]
    idx[0] = 2
    w[:, 2], w[:, 3] = 0, -w[:, 3]
    y = dtc.moe_experts_fp4(kind, x, dtc.quantize_fp4(wi, gated=True), dtc.quantize_fp4(wo), w, dtc.moe_plan(idx, E),
                            activation=act)
    R.close(y, experts_reference(kind, fmt, x, wi, wo, idx, w, None, act), 2 * R.U[kind] + (1 / 3) * (1 / 1600) ** 0.5,
            "twice")


def test_experts_equal_their_parts():
    """The call against the same steps through the other operators, expert by expert: equal but for the order of
    fp32 sums."""
    import dense_tensor_core_gb300 as dtc
    kind, act, T, E, k, H, F = "bf16", "swiglu", 90, 4, 2, 256, 128
    x, wi, wo, idx, w = experts_case(kind, "nvfp4", T, E, k, H, F, act)
    y = dtc.moe_experts_fp4(kind, x, dtc.quantize_fp4(wi, gated=True), dtc.quantize_fp4(wo), w, dtc.moe_plan(idx, E),
                            activation=act)
    want = torch.zeros((T, H), device="cuda", dtype=torch.float64)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        h = dtc.gemm_fp4(kind, dtc.quantize_fp4(x[t]), dtc.quantize_fp4(wi[e], gated=True), activation=act)
        o = dtc.dequantize_fp4(dtc.quantize_fp4(h)).double() @ dtc.dequantize_fp4(dtc.quantize_fp4(wo[e])).double().t()
        want.index_add_(0, t, w[t, j, None].double() * o)
    R.check(y, want, 2.0 ** -8 * want.abs() + 2.0 ** -14 * want.abs().amax(), "experts")


def test_experts_weight_types_and_no_tokens():
    import dense_tensor_core_gb300 as dtc
    kind, act, T, E, k, H, F = "f16", "silu", 50, 8, 3, 192, 96
    x, wi, wo, idx, w = experts_case(kind, "mxfp4", T, E, k, H, F, act)
    wi4, wo4 = dtc.quantize_fp4(wi, format="mxfp4"), dtc.quantize_fp4(wo, format="mxfp4")
    plan = dtc.moe_plan(idx, E)
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        wt = w.to(dt)
        a = dtc.moe_experts_fp4(kind, x, wi4, wo4, wt, plan, activation=act)
        b = dtc.moe_experts_fp4(kind, x, wi4, wo4, wt.float(), plan, activation=act)
        assert torch.equal(a, b)
    none = torch.full_like(idx, -1)
    res = rand((T, H), kind, 3)
    y = dtc.moe_experts_fp4(kind, x, wi4, wo4, w, dtc.moe_plan(none, E), activation=act, residual=res)
    assert torch.equal(y, res)
    e = dtc.moe_experts_fp4(kind, x[:0], wi4, wo4, w[:0], dtc.moe_plan(idx[:0], E), activation=act)
    assert e.shape == (0, H)


def test_same_bits_every_time():
    import dense_tensor_core_gb300 as dtc
    x, wi, wo, idx, w = experts_case("bf16", "nvfp4", 333, 16, 4, 512, 256, "swiglu")
    wi4, wo4, plan = dtc.quantize_fp4(wi, gated=True), dtc.quantize_fp4(wo), dtc.moe_plan(idx, 16)
    a = dtc.moe_experts_fp4("bf16", x, wi4, wo4, w, plan)
    for _ in range(3):
        assert torch.equal(a, dtc.moe_experts_fp4("bf16", x, wi4, wo4, w, plan))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("act", R.ACTS)
def test_activations_of_extreme_sums(act, kind):
    """Sums that are the bias alone, from the type's smallest numbers to its largest, infinities and NaN, each beside
    ordinary ones: every value is its own sum's and no other's."""
    import dense_tensor_core_gb300 as dtc
    gated = act in R.GATED
    dt, big = R.DT[kind], torch.finfo(R.DT[kind]).max
    inf, nan = float("inf"), float("nan")
    gates = [0.0, 1e-7, -1e-7, 1.0, -1.0, 3.0, -3.0, -5.5, 8.0, -9.5, 14.5, -13.0, 30.0, -30.0, -41.0, -60.0, 75.0,
             -86.0, 90.0, -104.0, 1000.0, -1000.0, big, -big, inf, 0.5, -inf, -0.5, nan, 0.25, 2.0, nan]
    N, M, K = 64, 37, 64
    g = torch.tensor(gates + gates[::-1], device="cuda", dtype=torch.float64).to(dt)
    bias = torch.cat([g, torch.full_like(g, 0.5)]) if gated else g
    a = torch.zeros((M, K), device="cuda", dtype=dt)
    b = rand((2 * N if gated else N, K), kind, 5)
    y = dtc.gemm_fp4(kind, dtc.quantize_fp4(a), dtc.quantize_fp4(b, gated=gated), bias=bias, activation=act)
    z = bias.double().expand(M, -1)
    if act == "gelu_tanh":  # (without R.act's 1 + tanh, which cancels)
        want = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    else:
        want = R.act(z, act)
    # the limits: relu, gelu and silu of -infinity are 0, which 0 times infinity in the formula is not
    if act != "none":
        want = torch.where(z[:, :N] == -inf, 0.0, want)
    # z is exact. The exponential's argument, at most 88, is off by at most 5 roundings of it (gelu_tanh), 88 x 5 x 2^-24,
    # and the rest by less than 2^-18: 2^-14 of the value. Exponentials below 2^-126 are 0. Then one rounding to the
    # type (below its smallest normal number: half a subnormal step).
    top = torch.finfo(dt)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    over = want.abs() > big  # (finite ones beyond the type become infinite or its largest number)
    ok = ~torch.isnan(want) & ~over
    err = (y.double() - want).abs()[ok]
    tol = (top.eps / 2 + 2.0 ** -14) * want.abs()[ok] + top.tiny * top.eps
    tol += 2.0 ** -126 * z[:, :N].abs().clamp(max=200)[ok]
    assert (err <= tol).all(), (act, kind, y.double()[ok][err > tol], want[ok][err > tol])
    assert (y.double()[over].abs() >= big).all()
    assert torch.equal(y.nan_to_num(), y[:1].nan_to_num().expand(M, -1))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M", [1, 40])
def test_factors_whose_product_leaves_the_range(fmt, M):
    """Rows from 2^-60 to 2^100 and features from 2^-60 to 2^76, so that products of two factors reach from below fp32's range to above
    it: a result that fits is right, one of no common elements 0, one above the range infinite."""
    import dense_tensor_core_gb300 as dtc
    K, N = 128, 48
    exps = [-60, -50, -30, -8, 0, 9, 40, 64, 76, 100]
    a = rows(M, K, "bf16", 11).double()
    b = rows(N, K, "bf16", 12).double()
    ea = torch.tensor([exps[(i + 7) % 10] for i in range(M)], device="cuda")
    eb = torch.tensor([exps[i % 9] for i in range(N)], device="cuda")
    a, b = a * Q.pow2(ea)[:, None], b * Q.pow2(eb)[:, None]
    a[:, :64] = 0  # a feature with nothing behind has no elements in common with any row
    b[1::3, 64:] = 0
    a, b = a.bfloat16(), b.bfloat16()
    y = dtc.gemm_fp4("bf16", dtc.quantize_fp4(a, format=fmt), dtc.quantize_fp4(b, format=fmt))
    want = Q.rounded(a, fmt) @ Q.rounded(b, fmt).t()
    size = Q.rounded(a, fmt).abs() @ Q.rounded(b, fmt).abs().t()
    big = torch.finfo(torch.bfloat16).max
    fits = size < big * (1 - 2.0 ** -8)  # (MXFP4's scales are inside the sum)
    assert fits.any() and (want == 0).any()
    # (a bf16 value has 8 bits: half a step is up to 2^-8 of it)
    err = (y.double() - want).abs()[fits]
    tol = (2.0 ** -8 * want.abs() + (K + 2) * 2.0 ** -23 * size + 2.0 ** -133)[fits]
    assert (err <= tol).all(), (fmt, y.double()[fits][~(err <= tol)], want[fits][~(err <= tol)])
    over = want.abs() > big * (1 + 2.0 ** -8)
    assert over.any()
    assert torch.isinf(y[over]).all()


@pytest.mark.parametrize("M", [5, 33])
def test_packed_signed_scales_are_nan(M):
    """A UE4M3 byte with the sign bit set makes its row NaN, in the values and in the product, as 0x7F does."""
    import dense_tensor_core_gb300 as dtc
    K, N = 96, 40
    codes = torch.randint(0, 256, (M, K // 2), generator=gen(1), device="cuda", dtype=torch.uint8)
    scales = torch.randint(1, 0x7E, (M, K // 16), generator=gen(2), device="cuda", dtype=torch.uint8)
    scales[0, 1], scales[1, 5], scales[3, 0] = 0x80, 0xB8, 0x7F
    q = dtc.pack_fp4(codes, scales)
    bad = torch.zeros((M, K // 16), device="cuda", dtype=torch.bool)
    bad[0, 1] = bad[1, 5] = bad[3, 0] = True
    assert torch.equal(torch.isnan(dtc.dequantize_fp4(q)), bad.repeat_interleave(16, 1))
    y = dtc.gemm_fp4("bf16", q, dtc.quantize_fp4(rand((N, K), "bf16", 3)))
    assert torch.equal(torch.isnan(y), bad.any(1)[:, None].expand(M, N))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_offsets_past_32_bits(fmt):
    """Rows and results of more than 2^31 elements: the last ones against the same rows by themselves."""
    import dense_tensor_core_gb300 as dtc
    M, K, tail = 66000, 32800, 300
    x = torch.empty((M, K), device="cuda", dtype=torch.bfloat16).normal_(generator=gen(1))
    q = dtc.quantize_fp4(x, format=fmt)
    last = dtc.quantize_fp4(x[-tail:].contiguous(), format=fmt)
    assert torch.equal(q.codes[-tail:], last.codes)
    back = dtc.dequantize_fp4(q)
    assert torch.equal(back[-tail:], dtc.dequantize_fp4(last))
    del x, back
    b = dtc.quantize_fp4(rand((264, K), "bf16", 2, K ** -0.5), format=fmt)
    # (the same tiles of rows, so the same order of sums)
    y = dtc.gemm_fp4("bf16", q, b, tile_rows=256, split_k=1)
    assert torch.equal(y[-tail:], dtc.gemm_fp4("bf16", last, b, tile_rows=256, split_k=1))
    del q, y
    a, w = dtc.quantize_fp4(rand((M, 64), "bf16", 3), format=fmt), rand((K, 64), "bf16", 4)
    res = torch.empty((M, K), device="cuda", dtype=torch.bfloat16).normal_(generator=gen(5))
    y = dtc.gemm_fp4("bf16", a, dtc.quantize_fp4(w, format=fmt), residual=res)
    want = Q.rounded(rand((M, 64), "bf16", 3)[-tail:], fmt) @ Q.rounded(w, fmt).t() + res[-tail:].double()
    # one rounding, and the fp32 sum of 64 products
    size = Q.rounded(rand((M, 64), "bf16", 3)[-tail:], fmt).abs() @ Q.rounded(w, fmt).abs().t() + res[-tail:].abs()
    assert ((y[-tail:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 66 * 2.0 ** -23 * size).all()
