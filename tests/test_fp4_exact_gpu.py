"""The 4-bit operators element by element: scales' padding, and experts whose sums are exact."""
import pytest
import torch

import ffn_ref as R
import fp4_ref as Q
from test_fp4_gpu import gen, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# ------------------------------------------------------------------------------------------------
# scales' padding
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("E,M,K,gated", [(1, 1, 32, False), (1, 130, 96, False), (3, 40, 160, False), (1, 300, 2080, False),
                                         (1, 5, 8224, False), (2, 3, 16416, False), (1, 2, 40032, False), (2, 144, 1056, True),
                                         (3, 48, 96, True)])
def test_places_past_k_are_zero_in_every_row(fmt, kind, E, M, K, gated):
    """The product multiplies the scales of a row's last set by codes of 0: none of them may be the NaN that stood in
    the buffer before."""
    import dense_tensor_core_gb300 as dtc
    x = rand((E, M, K), kind, K + M)
    out = dtc.quantize_fp4(torch.ones_like(x), format=fmt, gated=gated)
    out.scales.fill_(0xFF)
    dtc.quantize_fp4(x, format=fmt, gated=gated, out=out)
    blocks = K // Q.BLOCK[fmt]
    sets = (blocks + 3) // 4
    places = torch.zeros((E, M, 4 * sets), dtype=torch.uint8)
    places[:, :, :blocks], places[:, :, blocks:] = 1, 2
    places = Q.chunks(places, fmt, gated)
    got = out.scales.cpu()
    assert got.shape == places.shape
    assert torch.equal(got[places == 1], Q.chunks(Q.quantize(x, fmt)[1], fmt, gated)[places == 1])
    assert int((places == 2).sum()) == E * M * (4 * sets - blocks)
    assert not got[places == 2].any()
    assert bool((got[places == 0] == 0xFF).all())  # (of no row: left as they were)


# ------------------------------------------------------------------------------------------------
# the experts
# ------------------------------------------------------------------------------------------------
def exact_rows(shape, kind, seed, size=1.0):
    """Rows that 4 bits hold exactly: code values times `size`, a power of two, the largest code in every block."""
    g = gen(seed)
    t = torch.tensor(Q.E2M1 + [-v for v in Q.E2M1], device="cuda")
    x = t[torch.randint(0, 16, shape, generator=g, device="cuda")]
    x[..., ::16] = 6.0 * torch.sign(x[..., 1::16] + 0.25)
    return (x * size).to(R.DT[kind])


EXPERTS = [(1, 8, 2, 1056, 96), (5, 6, 3, 2080, 416), (90, 4, 2, 288, 224), (300, 2, 1, 96, 2080), (700, 3, 2, 288, 544),
           (1300, 2, 2, 544, 96), (2100, 5, 3, 1312, 352), (257, 1, 1, 160, 160)]


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F", EXPERTS)
def test_each_element_of_the_experts(fmt, kind, act, T, E, k, H, F):
    """x and w_in are rows of code values, so each of the first product's sums is a multiple of 1/4 (times a power of
    two) below 2^17: exact in any order. h is then one number whatever the tiles, and quantises to one row. What is left
    per element: the second sum in fp32, F + 2 steps of 2^-23 of its terms' sizes, two factors, k terms of the join with
    their weights, and the result's rounding."""
    import dense_tensor_core_gb300 as dtc
    Fz = 2 * F if act in R.GATED else F
    x = exact_rows((T, H), kind, 1)
    wi = exact_rows((E, Fz, H), kind, 2, 2.0 ** -10)
    wo = rand((E, H, F), kind, 3, F ** -0.5)
    for w in (x, wi):
        assert torch.equal(Q.rounded(w, fmt), w.double())
    g = gen(4)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).to(torch.int32)
    if T > 2:
        idx[1], idx[2, k - 1] = -1, -1
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    wi4 = dtc.quantize_fp4(wi, format=fmt, gated=act in R.GATED)
    y = dtc.moe_experts_fp4(kind, x, wi4, dtc.quantize_fp4(wo, format=fmt), w, dtc.moe_plan(idx, E), activation=act)
    dtc.gemm_stream_status()
    want = torch.zeros((T, H), device="cuda", dtype=torch.float64)
    size = torch.zeros_like(want)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        if act == "none":
            h = (x[t].double() @ wi[e].double().t()).to(R.DT[kind])
        else:  # (the same exact sums through the product's epilogue, on tiles)
            h = dtc.gemm_fp4(kind, dtc.quantize_fp4(x[t], format=fmt), dtc.quantize_fp4(wi[e], format=fmt, gated=True),
                             activation=act, tile_rows=64, split_k=1)
        hq, oq, wt = Q.rounded(h, fmt), Q.rounded(wo[e], fmt), w[t, j, None].double()
        want.index_add_(0, t, wt * (hq @ oq.t()))
        size.index_add_(0, t, wt * (hq.abs() @ oq.abs().t()))
    u = R.U[kind]
    bound = (F + 2 + k + 4) * 2.0 ** -23 * size * (1 + u) + u * want.abs() + R.TINY[kind]
    R.check(y, want, bound, f"{fmt} {kind} {act} {T} {E} {k} {H} {F}")
