"""The 4-bit operators on streams, in captured graphs, after waits that gave up, and with arguments that they
refuse."""
import time

import pytest
import torch

import ffn_ref as R
import fp4_ref as Q
from test_ffn_streams_gpu import DELAY, dirty, overwrite
from test_fp4_gpu import experts_case, operands, rand, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def chain(x, w, case, stream=None):
    """Rows to 4 bits, a product, the values back, and the routed experts: all of a call's outputs."""
    import dense_tensor_core_gb300 as dtc
    q = dtc.quantize_fp4(x, stream=stream)
    y = dtc.gemm_fp4("bf16", q, w, activation="gelu", stream=stream)
    v = dtc.dequantize_fp4(q, stream=stream)
    t, wi, wo, idx, g = case
    plan = dtc.moe_plan(idx, wi.shape[0], stream=stream)
    z = dtc.moe_experts_fp4("bf16", t, wi, wo, g, plan, stream=stream)
    return y, v, z


def make(T=200):
    import dense_tensor_core_gb300 as dtc
    x, b, _ = operands("bf16", "nvfp4", 300, 520, 1056, "none")
    t, wi, wo, idx, g = experts_case("bf16", "nvfp4", T, 8, 2, 512, 256, "swiglu")
    return x, dtc.quantize_fp4(b), (t, dtc.quantize_fp4(wi, gated=True), dtc.quantize_fp4(wo), idx, g)


@pytest.mark.parametrize("busy", ["current", "given"])
@pytest.mark.parametrize("T", [1, 200])
def test_memory_belongs_to_the_given_stream(busy, T):
    from dense_tensor_core_gb300 import _fp4
    args = make(T)
    want = chain(*args)
    sizes = [300 * 1056 // 2 + 3 * 17 * 512 + 256 * 3 + 1200, 300 * 520 * 2, 300 * 1056 * 2, T * 512 * 2,
             _fp4._buffer_size(0, 0, T, 2, 8, 512, 256, 5)]
    s = torch.cuda.Stream()
    dirty([torch.cuda.current_stream(), s], sizes)
    with torch.cuda.stream(s if busy == "given" else None):
        torch.cuda._sleep(DELAY)
    got = chain(*args, stream=s)
    keep = overwrite(sizes)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    del keep


def test_two_streams_at_once():
    import dense_tensor_core_gb300 as dtc
    args = make()
    want = chain(*args)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            got.append(chain(*args, stream=s))
    torch.cuda.synchronize()
    dtc.gemm_stream_status()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 200])
def test_captured_and_replayed_on_new_inputs(T):
    import dense_tensor_core_gb300 as dtc
    x, w, (t, wi, wo, idx, g) = make(T)
    n = dtc.gemm_fp4_workspace_size(1, 4096, 8192)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    a1, b1, _ = operands("bf16", "nvfp4", 1, 4096, 8192, "none")
    big = dtc.quantize_fp4(b1)

    def everything():
        one = dtc.gemm_fp4("bf16", dtc.quantize_fp4(a1), big, workspace=ws, split_k=4, tile_rows=32)
        return (*chain(x, w, (t, wi, wo, idx, g)), one)

    everything()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        everything()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            out = everything()
    for seed in (5, 6, 7):
        x.copy_(rows(*x.shape, "bf16", seed, 0.4))
        t.copy_(rows(*t.shape, "bf16", seed + 1, 0.4))
        a1.copy_(rows(*a1.shape, "bf16", seed + 2, 0.4))
        idx.copy_(idx.roll(1, 1) if T == 1 else idx.roll(3, 0))
        want = everything()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tile,split", [(64, 1), (256, 1), (32, 3)])
def test_wait_that_nothing_completes_reports_timeout_then_recovers(fmt, tile, split):
    import dense_tensor_core_gb300 as dtc
    M, N, K = (24 if split > 1 else 300), 520, 2080
    a, b, _ = operands("bf16", fmt, M, N, K, "none")
    qa, qb = dtc.quantize_fp4(a, format=fmt), dtc.quantize_fp4(b, format=fmt)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    dtc.gemm_stream_status()
    t0 = time.time()
    dtc.gemm_fp4("bf16", qa, qb, workspace=ws, tile_rows=tile, split_k=split, timeout_ns=20_000_000, fault_inject=1)
    with pytest.raises(dtc.GemmError) as e:
        dtc.gemm_stream_status()
    assert e.value.status == 4 and time.time() - t0 < 30
    dtc.gemm_stream_status()  # (cleared by the report)
    ws.zero_()
    y = dtc.gemm_fp4("bf16", qa, qb, workspace=ws, tile_rows=tile, split_k=split)
    dtc.gemm_stream_status()
    want, bound = Q.product("bf16", Q.rounded(a, fmt), Q.rounded(b, fmt), None, None, "none")
    R.check(y, want, bound, "after a timeout")


def test_experts_timeout_reports_and_recovers():
    import dense_tensor_core_gb300 as dtc
    _, _, (t, wi, wo, idx, g) = make(100)
    plan = dtc.moe_plan(idx, 8)
    want = dtc.moe_experts_fp4("bf16", t, wi, wo, g, plan)
    dtc.gemm_stream_status()
    dtc.moe_experts_fp4("bf16", t, wi, wo, g, plan, timeout_ns=20_000_000, fault_inject=1)
    with pytest.raises(dtc.GemmError) as e:
        dtc.gemm_stream_status()
    assert e.value.status == 4
    assert torch.equal(dtc.moe_experts_fp4("bf16", t, wi, wo, g, plan), want)
    dtc.gemm_stream_status()


def test_one_workspace_for_sizes_in_turn():
    """Splits of few and of many tiles through one workspace, gemm_act's among them, and results of NaNs before."""
    import dense_tensor_core_gb300 as dtc
    calls = [(1, 2048, 4096, "none", 32, 4), (40, 4096, 4096, "gelu", 64, 2), (24, 512, 8192, "swiglu", 32, 8),
             (1, 8192, 8192, "none", 32, 2), (130, 264, 4128, "silu", 64, 3)]
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    c, d = rand((32, 4096), "bf16", 1), rand((1024, 4096), "bf16", 2)
    want = dtc.gemm_act("bf16", c, d)
    for M, N, K, act, tile, split in calls + calls[::-1]:
        a, b, _ = operands("bf16", "nvfp4", M, N, K, act)
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        dtc.gemm_fp4("bf16", dtc.quantize_fp4(a), dtc.quantize_fp4(b, gated=act in R.GATED), C=y, activation=act,
                     workspace=ws, tile_rows=tile, split_k=split)
        ref, bound = Q.product("bf16", Q.rounded(a, "nvfp4"), Q.rounded(b, "nvfp4"), None, None, act)
        R.check(y, ref, bound, f"{M} x {N} x {K} {act}")
        # (sums of a split K are added in another order)
        R.close(dtc.gemm_act("bf16", c, d, workspace=ws), want.double(), 2.0 ** -8, "gemm_act")


# ------------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------------
def refused(call):
    import dense_tensor_core_gb300 as dtc
    with pytest.raises((ValueError, TypeError, dtc.GemmError)):
        call()


def test_rows_that_are_refused():
    import dense_tensor_core_gb300 as dtc
    x = rows(8, 128, "bf16", 1)
    for bad in (x[:, :80], x[:, 1:97], x.t(), x.float(), x.double(), x[0], x.reshape(2, 2, 2, 128), x.cpu(),
                torch.zeros((4, 100), dtype=torch.bfloat16, device="cuda")[:, :96]):
        refused(lambda: dtc.quantize_fp4(bad))
    refused(lambda: dtc.quantize_fp4(x, gated=True))  # 8 rows: not pairs of octets
    q = dtc.quantize_fp4(x)
    for out in (dtc.quantize_fp4(x, format="mxfp4"), dtc.quantize_fp4(x[:4]), x,
                dtc.quantize_fp4(torch.cat([x, x]), gated=True)):
        refused(lambda: dtc.quantize_fp4(x, out=out))
    refused(lambda: dtc.dequantize_fp4(q, dtype=torch.float64))
    refused(lambda: dtc.dequantize_fp4(q, out=torch.empty((8, 64), dtype=torch.bfloat16, device="cuda")))
    refused(lambda: dtc.dequantize_fp4(q, dtype=torch.float32, out=torch.empty((8, 128), dtype=torch.bfloat16, device="cuda")))


def test_held_matrices_that_are_refused():
    import dense_tensor_core_gb300 as dtc
    q = dtc.quantize_fp4(rows(8, 128, "bf16", 1))
    make_ = lambda **k: dtc.Fp4(k.get("codes", q.codes), k.get("scales", q.scales), k.get("g", q.row_scale),  # noqa: E731
                                k.get("fmt", "nvfp4"))
    assert dtc.gemm_fp4("bf16", make_(), q).shape == (8, 8)
    for bad in (make_(scales=q.scales[:512]), make_(scales=q.scales.cpu()), make_(g=q.row_scale[:4]),
                make_(g=q.row_scale.double()), make_(codes=q.codes.int()), make_(codes=q.codes[:, ::2]),
                make_(fmt="mxfp4"), make_(codes=q.codes[:, :40])):
        refused(lambda: dtc.gemm_fp4("bf16", bad, q))
        refused(lambda: dtc.dequantize_fp4(bad))


def test_products_that_are_refused():
    import dense_tensor_core_gb300 as dtc
    x = rows(40, 128, "bf16", 1)
    a, b = dtc.quantize_fp4(x), dtc.quantize_fp4(x[:32])
    g = dtc.quantize_fp4(x[:32], gated=True)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for call in (lambda: dtc.gemm_fp4("bf16", a, dtc.quantize_fp4(x[:32], format="mxfp4")),
                 lambda: dtc.gemm_fp4("bf16", a, dtc.quantize_fp4(x[:32, :64])), lambda: dtc.gemm_fp4("bf16", a, g),
                 lambda: dtc.gemm_fp4("bf16", a, b, activation="swiglu"), lambda: dtc.gemm_fp4("bf16", g, b),
                 lambda: dtc.gemm_fp4("bf16", a, dtc.quantize_fp4(x[:12])),  # N % 8
                 lambda: dtc.gemm_fp4("bf16", a, dtc.quantize_fp4(x[:32].reshape(2, 16, 128))),
                 lambda: dtc.gemm_fp4("bf16", a, b, bias=z(16)), lambda: dtc.gemm_fp4("f16", a, b, bias=z(32)),
                 lambda: dtc.gemm_fp4("bf16", a, b, residual=z(40, 16)), lambda: dtc.gemm_fp4("bf16", a, b, C=z(40, 40)),
                 lambda: dtc.gemm_fp4("bf16", a, b, C=z(32, 40).t()), lambda: dtc.gemm_fp4("bf16", a, b, tile_rows=40),
                 lambda: dtc.gemm_fp4("bf16", a, b, tile_rows=32), lambda: dtc.gemm_fp4("bf16", a, b, split_k=2),
                 lambda: dtc.gemm_fp4("bf16", a, b, timeout_ns=-1), lambda: dtc.gemm_fp4("bf16", a, b, split_k=2 ** 32),
                 lambda: dtc.gemm_fp4("bf16", a, b, workspace=torch.zeros(64, dtype=torch.uint8))):
        refused(call)
    assert dtc.gemm_fp4("bf16", a, b).shape == (40, 32)


def test_experts_that_are_refused():
    import dense_tensor_core_gb300 as dtc
    _, _, (t, wi, wo, idx, g) = make(20)
    plan = dtc.moe_plan(idx, 8)
    call = lambda **k: dtc.moe_experts_fp4("bf16", k.get("t", t), k.get("wi", wi), k.get("wo", wo), k.get("g", g),  # noqa: E731
                                           k.get("plan", plan), activation=k.get("act", "swiglu"),
                                           residual=k.get("res"), timeout_ns=k.get("ns", 0))
    assert call().shape == (20, 512)
    plain = dtc.quantize_fp4(rand((8, 512, 512), "bf16", 1))
    short = dtc.moe_plan(idx[:10], 8)
    spoiled = dtc.moe_plan(idx, 8)
    spoiled.data = spoiled.data[:-1]
    for k in (dict(t=t[:10]), dict(t=t.half()), dict(t=t[:, :256]), dict(wi=plain), dict(wo=wi), dict(act="silu"),
              dict(wi=dtc.quantize_fp4(rand((8, 512, 512), "bf16", 1), format="mxfp4", gated=True)),
              dict(g=g[:, :1]), dict(g=g.double()), dict(plan=short), dict(plan=spoiled), dict(res=t[:10]), dict(ns=-1),
              dict(plan=dtc.moe_plan(idx, 9))):
        refused(lambda: call(**k))
