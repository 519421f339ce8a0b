"""Products and experts with a handful of rows, around the sizes where another kernel takes them, on
the GPU against the 64-bit reference."""
import pytest
import torch

import ffn_ref as R
from test_gemm_act_gpu import operands, rand, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# rows at and past 8 and 16; features off a block; K of less than a warp's piece, off 64 and 512, of
# several whole turns, and at both sides of what counts as short for few blocks
@pytest.mark.parametrize("M", [1, 7, 8, 9, 16, 17])
@pytest.mark.parametrize("N,K", [(8, 8), (24, 72), (40, 1544), (2440, 2056), (136, 4104), (136, 4112),
                                 (2440, 4616)])
@pytest.mark.parametrize("kind,name", [("bf16", "swiglu"), ("f16", "gelu")])
def test_forward(M, N, K, kind, name):
    import dense_tensor_core_gb300 as dtc
    A, B, Nb = operands(kind, "NT", M, N, K, name)
    bias, res = rand((Nb,), kind, 7, 0.3), rand((M, N), kind, 8)
    z = torch.full((M, Nb), float("nan"), dtype=R.DT[kind], device="cuda")
    y, ey, zr, ez = R.gemm_act(kind, A, B, "NT", bias, res, name)
    got = dtc.gemm_act(kind, A, B, bias=bias, residual=res, activation=name, preact=z,
                       workspace=workspace(kind, M, N, K, "NT", name))
    R.check(got, y, ey, "y")
    R.check(z, zr, ez, "z")


@pytest.mark.parametrize("M", [3, 12])
def test_strides_and_what_is_written(M):
    import dense_tensor_core_gb300 as dtc
    N, K = 200, 264
    A0, B0 = rand((M, K + 24), "bf16", 1), rand((N, K + 40), "bf16", 2, K ** -0.5)
    A0[:, K:] = float("nan")  # read by nobody
    B0[:, K:] = float("nan")
    out = torch.full((M + 1, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    y, ey, _, _ = R.gemm_act("bf16", A0[:, :K], B0[:, :K], "NT", None, None, "silu")
    dtc.gemm_act("bf16", A0[:, :K], B0[:, :K], out[:M, :N], activation="silu")
    R.check(out[:M, :N], y, ey, "y")
    assert bool((out[M:] == 7).all()) and bool((out[:, N:] == 7).all())


def test_a_bad_row_stays_in_its_row():
    import dense_tensor_core_gb300 as dtc
    A, B, _ = operands("bf16", "NT", 5, 72, 520, "none")
    clean = dtc.gemm_act("bf16", A, B)
    A[2] = float("nan")
    A[4, 3] = float("inf")
    got = dtc.gemm_act("bf16", A, B)
    keep = [0, 1, 3]
    assert torch.equal(got[keep], clean[keep]) and bool(got[2].isnan().all())
    B[71] = float("nan")  # the last feature, which blocks past it read too
    assert torch.equal(dtc.gemm_act("bf16", A, B)[keep, :71], clean[keep, :71])


# up to 8 tokens and past it; an expert that every choice names has more rows than one turn takes
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9])
@pytest.mark.parametrize("kind,H,F,name", [("bf16", 264, 136, "swiglu"), ("f16", 1032, 520, "gelu")])
@pytest.mark.parametrize("one", [False, True])
def test_experts(T, kind, H, F, name, one):
    import dense_tensor_core_gb300 as dtc
    E, k = 6, 3
    Fz = 2 * F if name in R.GATED else F
    x, res = rand((T, H), kind, 1), rand((T, H), kind, 2)
    wi, wo = rand((E, Fz, H), kind, 3, H ** -0.5), rand((E, H, F), kind, 4, F ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    if one:
        idx.fill_(4)
    if T > 1:
        idx[1] = -1  # a token without experts
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
    plan = dtc.moe_plan(idx, E)
    y, bound = R.experts_bound(kind, x.double(), wi.double(), wo.double(), w.double(), idx, name, res.double())
    got = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, residual=res)
    dtc.gemm_stream_status()
    R.check(got, y, bound, "y")
    assert torch.equal(dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, residual=res, save=True)[0], got)


# the number of tokens from which tiles take over, with experts of several turns of 8 rows
@pytest.mark.parametrize("T", [10, 15, 16, 17])
@pytest.mark.parametrize("kind,E,k,H,F,name", [("bf16", 3, 2, 520, 264, "geglu"), ("f16", 40, 8, 72, 136, "silu")])
def test_experts_around_the_change(T, kind, E, k, H, F, name):
    import dense_tensor_core_gb300 as dtc
    Fz = 2 * F if name in R.GATED else F
    x = rand((T, H), kind, 1)
    wi, wo = rand((E, Fz, H), kind, 3, H ** -0.5), rand((E, H, F), kind, 4, F ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(T)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
    plan = dtc.moe_plan(idx, E)
    y, bound = R.experts_bound(kind, x.double(), wi.double(), wo.double(), w.double(), idx, name)
    got = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name)
    dtc.gemm_stream_status()
    R.check(got, y, bound, "y")
    # kept rows of a training call give a gradient
    y2, saved = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, save=True)
    assert torch.equal(y2, got)
    dy = rand((T, H), kind, 9)
    grads = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, activation=name)
    leaf = [t.double().requires_grad_() for t in (x, wi, wo, w)]
    want = torch.autograd.grad(R.experts(*leaf, idx, name), leaf, dy.double())
    for a, r, n, what in zip(grads, want, (4, 3, 2, 2), ("dx", "dw_in", "dw_out", "dweights")):
        R.close(a, r, 1.1 * n * R.U[kind], what)


# few tokens with a reduction at and past the length from which few blocks no longer do
@pytest.mark.parametrize("H,F", [(64, 8192), (64, 8200), (8192, 72), (8200, 72), (16384, 1024)])
@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (3, 8, 2), (16, 8, 8)])
@pytest.mark.parametrize("kind,name", [("bf16", "swiglu"), ("f16", "gelu")])
def test_experts_with_a_long_reduction(kind, name, T, E, k, H, F):
    import dense_tensor_core_gb300 as dtc
    Fz = 2 * F if name in R.GATED else F
    x, wi, wo = rand((T, H), kind, 1), rand((E, Fz, H), kind, 2, H ** -0.5), rand((E, H, F), kind, 3, F ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(T + k)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
    y, bound = R.experts_bound(kind, x.double(), wi.double(), wo.double(), w.double(), idx, name)
    plan = dtc.moe_plan(idx, E)
    got = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name)
    dtc.gemm_stream_status()
    R.check(got, y, bound, "y")
    assert torch.equal(dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, save=True)[0], got)
