"""gemm_act and its gradient on the GPU against the 64-bit reference."""
import math

import pytest
import torch

import ffn_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def rand(shape, kind, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(R.DT[kind])


def operands(kind, layout, M, N, K, name, seed=1):
    Nb = 2 * N if name in R.GATED else N
    A = rand((M, K) if layout[0] == "N" else (K, M), kind, seed)
    B = rand((Nb, K) if layout[1] == "T" else (K, Nb), kind, seed + 1, max(K, 1) ** -0.5)
    return A, B, Nb


def workspace(kind, M, N, K, layout, name):
    import dense_tensor_core_gb300 as dtc
    n = dtc.gemm_act_workspace_size(kind, M, N, K, layout=layout, activation=name)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")


# sizes: one row and one past a tile's row steps; features off the 256 (gated 128) of a tile; K of
# less than a block, of whole blocks, off 64 (other tensor maps) and off 16 (half an MMA step)
SIZES = [(1, 8, 8), (1, 264, 128), (2, 4096, 512), (16, 256, 4104), (33, 520, 200), (255, 136, 192),
         (257, 1032, 1000), (700, 2056, 328)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind,name", [("bf16", "gelu"), ("f16", "silu"), ("bf16", "swiglu"),
                                       ("f16", "geglu"), ("bf16", "relu"), ("f16", "gelu_tanh"),
                                       ("bf16", "none")])
def test_forward_nt(M, N, K, kind, name):
    import dense_tensor_core_gb300 as dtc
    A, B, Nb = operands(kind, "NT", M, N, K, name)
    bias, res = rand((Nb,), kind, 7, 0.3), rand((M, N), kind, 8)
    z = torch.empty((M, Nb), dtype=R.DT[kind], device="cuda")
    y, ey, zr, ez = R.gemm_act(kind, A, B, "NT", bias, res, name)
    for ws in (None, workspace(kind, M, N, K, "NT", name)):
        got = dtc.gemm_act(kind, A, B, bias=bias, residual=res, activation=name, preact=z, workspace=ws)
        dtc.gemm_stream_status()
        R.check(got, y, ey, f"{name} y")
        R.check(z, zr, ez, f"{name} z")
        z.fill_(float("nan"))


@pytest.mark.parametrize("layout,M,N,K", [("NN", 77, 520, 136), ("NN", 300, 264, 1000),
                                          ("TN", 8, 264, 72), ("TN", 520, 520, 200),
                                          ("TT", 72, 136, 1032), ("TT", 512, 256, 256),
                                          ("TN", 256, 256, 384)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_layouts(layout, M, N, K, kind):
    import dense_tensor_core_gb300 as dtc
    A, B, Nb = operands(kind, layout, M, N, K, "gelu")
    bias = rand((Nb,), kind, 7, 0.3)
    y, ey, _, _ = R.gemm_act(kind, A, B, layout, bias, None, "gelu")
    got = dtc.gemm_act(kind, A, B, layout=layout, bias=bias, activation="gelu",
                       workspace=workspace(kind, M, N, K, layout, "gelu"))
    dtc.gemm_stream_status()
    R.check(got, y, ey, layout)


def test_large_tiles_and_many_waves():
    import dense_tensor_core_gb300 as dtc
    M, N, K = 3000, 2304, 320  # several tiles a pair: both accumulators and every ring phase
    A, B, _ = operands("bf16", "NT", M, N, K, "silu")
    y, ey, _, _ = R.gemm_act("bf16", A, B, "NT", None, None, "silu")
    R.check(dtc.gemm_act("bf16", A, B, activation="silu"), y, ey, "many waves")


@pytest.mark.parametrize("name", ["gelu", "swiglu"])
def test_rows_of_larger_arrays(name):
    import dense_tensor_core_gb300 as dtc
    kind, M, N, K = "bf16", 130, 264, 136
    Nb = 2 * N if name in R.GATED else N
    big = rand((M, K + 24), kind, 1)
    A, Bb = big[:, 8:8 + K], rand((Nb, K + 8), kind, 2, K ** -0.5)
    B = Bb[:, :K]
    Cb = torch.full((M, N + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    Zb = torch.full((M, Nb + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    Rb = rand((M, N + 8), kind, 3)
    y, ey, z, ez = R.gemm_act(kind, A, B, "NT", None, Rb[:, :N], name)
    dtc.gemm_act(kind, A, B, Cb[:, :N], residual=Rb[:, :N], activation=name, preact=Zb[:, :Nb])
    dtc.gemm_stream_status()
    R.check(Cb[:, :N], y, ey, "y")
    R.check(Zb[:, :Nb], z, ez, "z")
    assert bool((Cb[:, N:] == 5).all()) and bool((Zb[:, Nb:] == 5).all())  # outside untouched


def test_residual_in_place_and_repeat():
    import dense_tensor_core_gb300 as dtc
    kind, M, N, K = "bf16", 300, 520, 264
    A, B, _ = operands(kind, "NT", M, N, K, "gelu")
    res = rand((M, N), kind, 3)
    first = dtc.gemm_act(kind, A, B, residual=res, activation="gelu")
    assert torch.equal(dtc.gemm_act(kind, A, B, residual=res, activation="gelu"), first)
    dtc.gemm_act(kind, A, B, res, residual=res, activation="gelu")
    assert torch.equal(res, first)


def test_split_sums_repeat_bit_for_bit():
    import dense_tensor_core_gb300 as dtc
    kind, M, N, K = "bf16", 3, 1024, 8192
    A, B, _ = operands(kind, "NT", M, N, K, "none")
    ws = workspace(kind, M, N, K, "NT", "none")
    assert ws.numel() > 16  # these sizes split K
    first = dtc.gemm_act(kind, A, B, workspace=ws)
    for _ in range(20):
        assert torch.equal(dtc.gemm_act(kind, A, B, workspace=ws), first)
    y, ey, _, _ = R.gemm_act(kind, A, B, "NT", None, None, "none")
    R.check(first, y, ey, "split")


def test_degenerate_sizes():
    import dense_tensor_core_gb300 as dtc
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert dtc.gemm_act("bf16", e(0, 64), e(32, 64)).shape == (0, 32)
    assert dtc.gemm_act("bf16", e(8, 64), e(0, 64)).shape == (8, 0)
    bias, res = rand((32,), "bf16", 1), rand((5, 32), "bf16", 2)
    got = dtc.gemm_act("bf16", e(5, 0), e(32, 0), bias=bias, residual=res, activation="silu")
    y = R.act(bias.double(), "silu") + res.double()
    R.check(got, y.expand(5, 32), R.U["bf16"] * 1.01 * y.abs() + 2.0 ** -18, "K = 0")


@pytest.mark.parametrize("name", R.ACTS)
def test_infinities_and_nan(name):
    # a bias of +-infinity or NaN gives the activation's limits, and only in its own column
    import dense_tensor_core_gb300 as dtc
    M, N, K = 40, 64, 128
    A, B, Nb = operands("bf16", "NT", M, N, K, name)
    bias = torch.zeros(Nb, dtype=torch.bfloat16, device="cuda")
    bias[0], bias[1], bias[2] = math.inf, -math.inf, math.nan
    y = dtc.gemm_act("bf16", A, B, bias=bias, activation=name).float()
    assert bool(torch.isnan(y[:, 2]).all()) and bool(torch.isfinite(y[:, 3:]).all())
    if name not in R.GATED:
        assert bool((y[:, 0] == math.inf).all())
        want = -math.inf if name == "none" else 0.0
        assert bool((y[:, 1] == want).all())


def test_other_stream():
    import dense_tensor_core_gb300 as dtc
    M, N, K = 200, 512, 1024
    A, B, _ = operands("bf16", "NT", M, N, K, "gelu")
    want = dtc.gemm_act("bf16", A, B, activation="gelu")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    C = torch.empty_like(want)
    dtc.gemm_act("bf16", A, B, C, activation="gelu", stream=s)
    s.synchronize()
    assert torch.equal(C, want)
    with torch.cuda.stream(s):
        D = dtc.gemm_act("bf16", A, B, activation="gelu")
    s.synchronize()
    assert torch.equal(D, want)


def test_captured_in_a_graph():
    import dense_tensor_core_gb300 as dtc
    M, N, K = 64, 512, 2048
    A, B, _ = operands("bf16", "NT", M, N, K, "silu")
    ws = workspace("bf16", M, N, K, "NT", "silu")
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    dtc.gemm_act("bf16", A, B, C, activation="silu", workspace=ws)
    want = C.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            dtc.gemm_act("bf16", A, B, C, activation="silu", workspace=ws)
    C.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, want)


def test_timeout_reports_then_recovers():
    import dense_tensor_core_gb300 as dtc
    M, N, K = 512, 512, 1024
    A, B, _ = operands("bf16", "NT", M, N, K, "gelu")
    dtc.gemm_stream_status()
    dtc.gemm_act("bf16", A, B, activation="gelu", timeout_ns=20_000_000, fault_inject=1)
    with pytest.raises(dtc.GemmError) as e:
        dtc.gemm_stream_status()
    assert e.value.status == 4
    got = dtc.gemm_act("bf16", A, B, activation="gelu")
    dtc.gemm_stream_status()
    y, ey, _, _ = R.gemm_act("bf16", A, B, "NT", None, None, "gelu")
    R.check(got, y, ey, "after a timeout")


# ------------------------------------------------------------------------------------------------
# gradient
# ------------------------------------------------------------------------------------------------
def reference_gradient(kind, dC, A, B, z, layout, name):
    a, b = R.op_a(A, layout), R.op_b(B, layout)
    if name == "none":
        dz = dC.double()
    else:
        zz = z.double().requires_grad_()
        dz, = torch.autograd.grad(R.act(zz, name), zz, dC.double())
    dA, dB = dz @ b.t(), a.t() @ dz
    return (dA if layout[0] == "N" else dA.t(), dB.t() if layout[1] == "T" else dB, dz)


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (100, 136, 192), (777, 264, 200), (2050, 520, 136)])
def test_gradient_nt(M, N, K, name):
    kind = "bf16" if N % 16 else "f16"
    _gradient(kind, "NT", M, N, K, name)


@pytest.mark.parametrize("layout", ["NN", "TN", "TT"])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_gradient_layouts(layout, name):
    _gradient("bf16", layout, 200, 136, 264, name)


def _gradient(kind, layout, M, N, K, name):
    import dense_tensor_core_gb300 as dtc
    A, B, Nb = operands(kind, layout, M, N, K, name)
    dC, z = rand((M, N), kind, 5), rand((M, Nb), kind, 6, 1.5)
    dA, dB, db = dtc.gemm_act_backward(kind, dC, A, B, preact=z if name != "none" else None,
                                       layout=layout, activation=name)
    dtc.gemm_stream_status()
    ra, rb, dz = reference_gradient(kind, dC, A, B, z, layout, name)
    # dZ's rounding and the result's, each at most U of the norm (2 U leaves the sums' 2^-23 room)
    R.close(dA, ra, 2.1 * R.U[kind], "dA")
    R.close(dB, rb, 2.1 * R.U[kind], "dB")
    # fp32 sums of M unrounded fp32 values: the activation's error and the summation's
    e = 2.0 ** -17 * dz.abs().sum(0) * 2 + M * 2.0 ** -24 * dz.abs().sum(0) + 1e-30
    if name != "none":
        e = e + 2.0 ** -17 * (dC.double().abs().sum(0).repeat(Nb // N) * z.double().abs().max())
    R.check(db, dz.sum(0), e, "dbias")


def test_gradient_against_differences():
    import dense_tensor_core_gb300 as dtc
    kind, M, N, K, name = "f16", 64, 72, 80, "swiglu"
    A, B, Nb = operands(kind, "NT", M, N, K, name)
    bias, dC = rand((Nb,), kind, 3, 0.3), rand((M, N), kind, 5)
    z = torch.empty((M, Nb), dtype=torch.float16, device="cuda")
    dtc.gemm_act(kind, A, B, bias=bias, activation=name, preact=z)
    dA, dB, db = dtc.gemm_act_backward(kind, dC, A, B, preact=z, activation=name)

    def loss(a, b, c):
        return float((R.act(a @ b.t() + c, name) * dC.double()).sum())

    a, b, c, h = A.double(), B.double(), bias.double(), 1e-6
    for g, i in ((dA, 0), (dB, 1), (db, 2)):
        v = torch.randn(g.shape, dtype=torch.float64, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(i))
        at = [a, b, c]
        up, dn = list(at), list(at)
        up[i], dn[i] = at[i] + h * v, at[i] - h * v
        fd = (loss(*up) - loss(*dn)) / (2 * h)
        # three roundings (z, dZ, the result), each at most U of the gradient's norm along v
        assert abs(float((g.double() * v).sum()) - fd) <= 3 * R.U[kind] * float(g.double().norm() * v.norm())


def test_gradient_parts_strides_and_empty():
    import dense_tensor_core_gb300 as dtc
    kind, M, N, K = "bf16", 96, 128, 64
    A, B, _ = operands(kind, "NT", M, N, K, "gelu")
    dCb, zb = rand((M, N + 8), kind, 5), rand((M, N + 16), kind, 6)
    dC, z = dCb[:, :N], zb[:, :N]
    full = dtc.gemm_act_backward(kind, dC, A, B, preact=z, activation="gelu")
    dense = dtc.gemm_act_backward(kind, dC.contiguous(), A, B, preact=z.contiguous(), activation="gelu")
    for x, y in zip(full, dense):
        assert torch.equal(x, y)
    only = dtc.gemm_act_backward(kind, dC, A, B, preact=z, activation="gelu", need=(False, True, False))
    assert only[0] is None and only[2] is None and torch.equal(only[1], full[1])
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dA, dB, db = dtc.gemm_act_backward(kind, e(0, N), e(0, K), B, preact=e(0, N), activation="gelu")
    assert dA.shape == (0, K) and bool((dB == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("layout", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("name", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(40, 0, 64), (0, 24, 64), (40, 24, 0), (40, 0, 0), (0, 0, 64)])
def test_gradient_of_empty_operands(M, N, K, name, layout):
    import dense_tensor_core_gb300 as dtc
    if name in R.GATED and layout != "NT":
        pytest.skip("gated activations take NT")
    A, B, Nb = operands("bf16", layout, M, N, K, name)
    dC, z = rand((M, N), "bf16", 5), rand((M, Nb), "bf16", 6)
    dA, dB, db = dtc.gemm_act_backward("bf16", dC, A, B, preact=z, layout=layout, activation=name)
    dtc.gemm_stream_status()
    assert dA.shape == A.shape and dB.shape == B.shape and db.shape == (Nb,)
    assert bool((dA == 0).all()) and bool((dB == 0).all())  # sums over nothing
    if K:
        assert bool((db == 0).all())
    elif N:
        _, _, dz = reference_gradient("bf16", dC, A, B, z, layout, name)
        # at most 40 fp32 additions of terms within 2^-16
        R.check(db, dz.sum(0), (2.0 ** -16 + 40 * 2.0 ** -24) * 1.2 *
                (dC.double().abs().sum(0).repeat(Nb // N) * (1 + z.double().abs().max())), "dbias")
