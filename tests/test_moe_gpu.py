"""Routing, plan and routed experts on the GPU against plain references."""
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_logits(T, E, dtype, seed, masked=True):
    z = torch.randn((T, E), generator=gen(seed), device="cuda") * 1.5
    if masked:
        z[torch.rand((T, E), generator=gen(seed + 1), device="cuda") < 0.1] = -math.inf
        z[::7] = -math.inf  # rows that choose nothing
        if T > 3:
            z[3] = torch.finfo(dtype).min  # all alike and as low as they get: still a choice
            z[1, 0] = math.nan
    return z.to(dtype)


@pytest.mark.parametrize("T,E,k,groups,top", [
    (1, 8, 1, 1, 1), (5, 64, 8, 1, 1), (40, 256, 8, 8, 4), (30, 60, 7, 4, 3), (17, 60, 60 // 2, 1, 1),
    (20, 20, 5, 10, 4), (9, 1000, 32, 8, 8), (12, 1024, 16, 32, 5), (33, 32, 3, 4, 1), (8, 3, 3, 3, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, groups, top, scoring, renorm):
    import dense_tensor_core_gb300 as dtc
    dtype = (torch.float32, torch.bfloat16, torch.float16)[(T + k) % 3]
    z = make_logits(T, E, dtype, T + E)
    bias = torch.randn(E, generator=gen(5), device="cuda") * 0.2 if k % 2 == 0 else None
    w, i = dtc.moe_route(z, k, bias=bias, scoring=scoring, groups=groups, top_groups=top,
                         renormalize=renorm, scale=2.5)
    W, I = R.route(z, k, bias, scoring, groups, top, renorm, 2.5)
    assert torch.equal(i.cpu(), I)
    # a few fp32 operations on an exponential of a few ulp, and for the full softmax a sum of E terms
    assert bool(((w.cpu().double() - W).abs() <= (20 + E) * 2.0 ** -23 * W.abs() + 1e-37).all())


@pytest.mark.parametrize("E", [16, 64, 60, 512])
def test_ties_go_to_the_lowest_index(E):
    import dense_tensor_core_gb300 as dtc
    z = torch.zeros((6, E), device="cuda")  # every key alike: more ties than lanes
    z[1] = -0.0
    z[2, ::2] = -0.0
    z[3, E // 2:] = 1.0
    w, i = dtc.moe_route(z, 8, renormalize=True)
    first = torch.arange(8, dtype=torch.int32)
    for t in (0, 1, 2, 4):
        assert torch.equal(i[t].cpu(), first)
    assert torch.equal(i[3].cpu(), first + E // 2)
    assert torch.allclose(w, torch.full_like(w, 0.125), rtol=1e-6)
    _, g = dtc.moe_route(z[:1], 4, groups=4, top_groups=2, scoring="sigmoid")
    assert torch.equal(g[0].cpu(), first[:4])


def test_route_strided_rows_and_empty():
    import dense_tensor_core_gb300 as dtc
    big = make_logits(50, 130, torch.float32, 3, masked=False)
    for z in (big[:, :64], big[:, 1:65], big[::2, :128]):
        w, i = dtc.moe_route(z, 6)
        w2, i2 = dtc.moe_route(z.contiguous(), 6)
        assert torch.equal(i, i2) and torch.equal(w, w2)
    w, i = dtc.moe_route(torch.empty((0, 64), device="cuda"), 4)
    assert w.shape == (0, 4) and i.shape == (0, 4)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (40, 64, 8), (33, 60, 5), (10, 300, 32)])
def test_route_gradient(T, E, k, scoring, renorm):
    import dense_tensor_core_gb300 as dtc
    z = torch.randn((T, E), generator=gen(T), device="cuda")
    z[:, 2] = -math.inf
    dw = torch.randn((T, k), generator=gen(9), device="cuda")
    _, idx = dtc.moe_route(z, k, scoring=scoring, renormalize=renorm)
    idx[0, k - 1] = -1
    got = dtc.moe_route_backward(dw, z, idx, scoring=scoring, renormalize=renorm, scale=1.5)
    zz = z.double().requires_grad_()
    f = lambda x: (R.route_weights(x, idx, scoring, renorm, 1.5) * dw.double()).sum()  # noqa: E731
    want, = torch.autograd.grad(f(zz), zz)
    want = want.nan_to_num(0.0)
    # differences of fp32 terms of the size of scale |dw|: a few ulp of that
    tol = (40 + E) * 2.0 ** -24 * 1.5 * dw.double().abs().amax(1, keepdim=True)
    assert bool(((got.double() - want).abs() <= tol).all())
    assert bool((got[:, 2] == 0).all())
    v = torch.randn((T, E), dtype=torch.float64, device="cuda", generator=gen(4))
    h = 1e-6
    with torch.no_grad():
        fd = float(f(z.double() + h * v) - f(z.double() - h * v)) / (2 * h)
    assert abs(float((got.double() * v).sum()) - fd) <= float((tol * v.abs()).sum()) + 1e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_route_gradient_16_bit(dtype):
    import dense_tensor_core_gb300 as dtc
    z = torch.randn((100, 128), generator=gen(1), device="cuda").to(dtype)
    dw = torch.randn((100, 6), generator=gen(9), device="cuda")
    _, idx = dtc.moe_route(z, 6)
    got = dtc.moe_route_backward(dw, z, idx)
    want = dtc.moe_route_backward(dw, z.float(), idx)
    assert got.dtype == dtype and torch.equal(got, want.to(dtype))


# ------------------------------------------------------------------------------------------------
# plan
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E", [(0, 4, 8), (1, 1, 1), (1, 8, 64), (7, 3, 5), (64, 32, 1024), (1000, 6, 60),
                                   (1025, 8, 256), (2000, 8, 16), (9001, 4, 48), (50000, 3, 200)])
def test_plan(T, k, E):
    import dense_tensor_core_gb300 as dtc
    # uneven loads, an expert that gets nothing, choices that are none
    p = torch.rand((T, k, E), generator=gen(T + 1), device="cuda") if T * k * E < 4e6 else None
    if p is not None:
        idx = (p * torch.linspace(0.2, 1.0, E, device="cuda")).argmax(2) if T else \
            torch.empty((0, k), dtype=torch.long, device="cuda")
    else:
        idx = (torch.rand((T, k), generator=gen(T), device="cuda") ** 2 * E).long()
    idx = idx.to(torch.int32)
    if T > 5:
        idx[2] = -1
        idx[4, 0] = E  # out of range: no choice
        idx[idx == E // 2] = 0
    plan = dtc.moe_plan(idx, E)
    off, counts, slots = R.plan(idx.cpu(), E)
    assert plan.offsets.tolist() == off and plan.counts.tolist() == counts
    assert plan.slots.reshape(-1).tolist() == slots
    rows = plan.rows[:off[-1]].tolist()
    want = [-1] * off[-1]
    for i, s in enumerate(slots):
        if s >= 0:
            want[s] = i
    assert rows == want


# ------------------------------------------------------------------------------------------------
# experts
# ------------------------------------------------------------------------------------------------
def batch(kind, T, E, k, H, F, name, seed=1, wdtype=None):
    dt = R.DT[kind]
    r = lambda s, n, std=1.0: (torch.randn(s, generator=gen(seed + n), device="cuda") * std).to(dt)  # noqa: E731
    Fz = 2 * F if name in R.GATED else F
    x, wi, wo = r((T, H), 1), r((E, Fz, H), 2, H ** -0.5), r((E, H, F), 3, F ** -0.5)
    score = torch.rand((T, E), generator=gen(seed + 4), device="cuda") ** 2 * \
        torch.linspace(0.3, 1.0, E, device="cuda")
    idx = score.topk(k, 1).indices.to(torch.int32)
    if T > 4:
        idx[1] = -1           # a token without experts
        idx[3, k - 1] = -1
    w = torch.softmax(torch.randn((T, k), generator=gen(seed + 5), device="cuda"), 1).to(wdtype or dt)
    return x, wi, wo, idx, w


@pytest.mark.parametrize("kind,T,E,k,H,F,name", [
    ("bf16", 1, 4, 2, 64, 64, "swiglu"), ("f16", 1, 64, 8, 264, 136, "geglu"),
    ("bf16", 3, 8, 8, 1024, 2048, "silu"), ("bf16", 40, 16, 4, 200, 328, "gelu"),
    ("f16", 300, 8, 2, 520, 264, "swiglu"), ("bf16", 700, 3, 1, 128, 72, "relu"),
    ("f16", 513, 20, 5, 72, 520, "none"), ("bf16", 1100, 2, 2, 256, 256, "gelu_tanh"),
    ("bf16", 2000, 64, 6, 320, 192, "swiglu")])
def test_experts(kind, T, E, k, H, F, name):
    import dense_tensor_core_gb300 as dtc
    x, wi, wo, idx, w = batch(kind, T, E, k, H, F, name, wdtype=torch.float32 if T % 2 else None)
    res = x * 0.5
    plan = dtc.moe_plan(idx, E)
    y, bound = R.experts_bound(kind, x.double(), wi.double(), wo.double(), w.double(), idx, name, res.double())
    got = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, residual=res)
    dtc.gemm_stream_status()
    R.check(got, y, bound, "y")
    saved = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, residual=res, save=True)[0]
    assert torch.equal(saved, got)


@pytest.mark.parametrize("kind,T,E,k,H,F,name,wdtype", [
    ("bf16", 1, 8, 2, 64, 64, "swiglu", torch.float32), ("f16", 60, 16, 3, 264, 136, "gelu", None),
    ("bf16", 500, 8, 2, 256, 200, "swiglu", None), ("f16", 900, 5, 2, 136, 264, "geglu", torch.float32),
    ("bf16", 333, 12, 4, 128, 72, "none", torch.bfloat16), ("bf16", 333, 12, 4, 128, 264, "relu", None),
    ("f16", 333, 40, 6, 72, 128, "silu", None), ("bf16", 600, 4, 2, 520, 520, "gelu_tanh", None)])
def test_experts_gradient(kind, T, E, k, H, F, name, wdtype):
    import dense_tensor_core_gb300 as dtc
    x, wi, wo, idx, w = batch(kind, T, E, k, H, F, name, wdtype=wdtype)
    dy = torch.randn((T, H), generator=gen(77), device="cuda").to(R.DT[kind])
    plan = dtc.moe_plan(idx, E)
    y, saved = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, save=True)
    got = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, activation=name)
    dtc.gemm_stream_status()
    leaf = [t.double().requires_grad_() for t in (x, wi, wo, w)]
    out = R.experts(*leaf, idx, name)
    want = torch.autograd.grad(out, leaf, dy.double(), allow_unused=True)
    # roundings on the way (each at most U of the norm): dx: z, dz, its rows, the result; dw_in: z, dz,
    # the result; dw_out: h, the result; dweights: z, the result (none in fp32)
    for g, r, n, what in zip(got, want, (4, 3, 2, 2), ("dx", "dw_in", "dw_out", "dweights")):
        R.close(g, r, 1.1 * n * R.U[kind], what)
    dead = torch.ones(E, dtype=torch.bool, device="cuda")
    dead[idx[idx >= 0].long()] = False
    assert bool((got[1][dead] == 0).all()) and bool((got[2][dead] == 0).all())
    assert bool((got[3][idx < 0] == 0).all())
    if T > 4:
        assert bool((got[0][1] == 0).all())
    part = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, activation=name, need_weights=False)
    assert part[1] is None and torch.equal(part[0], got[0]) and torch.equal(part[3], got[3])
    part = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, activation=name, need_x=False)
    assert part[0] is None and torch.equal(part[1], got[1]) and torch.equal(part[3], got[3])


def test_experts_gradient_against_differences():
    import dense_tensor_core_gb300 as dtc
    kind, name = "f16", "swiglu"
    x, wi, wo, idx, w = batch(kind, 40, 6, 2, 64, 72, name, wdtype=torch.float32)
    dy = torch.randn(x.shape, generator=gen(7), device="cuda").to(torch.float16)
    plan = dtc.moe_plan(idx, 6)
    _, saved = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, save=True)
    got = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, activation=name)
    at = [t.double() for t in (x, wi, wo, w)]
    h = 1e-6
    for i, g in enumerate(got):
        v = torch.randn(g.shape, dtype=torch.float64, device="cuda", generator=gen(20 + i))
        f = [float((R.experts(*[t + s * h * v if j == i else t for j, t in enumerate(at)], idx, name)
                    * dy.double()).sum()) for s in (1, -1)]
        fd = (f[0] - f[1]) / (2 * h)
        assert abs(float((g.double() * v).sum()) - fd) <= 4.4 * R.U[kind] * float(g.double().norm() * v.norm())


def test_experts_edges():
    import dense_tensor_core_gb300 as dtc
    kind, E, k, H, F, name = "bf16", 4, 3, 128, 128, "swiglu"
    x, wi, wo, idx, w = batch(kind, 50, E, k, H, F, name)
    # every choice on one expert, the same expert three times a token: rows beyond the token count
    same = torch.full_like(idx, 2)
    plan = dtc.moe_plan(same, E)
    y, bound = R.experts_bound(kind, x.double(), wi.double(), wo.double(), w.double(), same, name)
    R.check(dtc.moe_experts(kind, x, wi, wo, w, plan), y, bound, "one expert")
    # nothing chosen: the residual, and no gradient
    none = torch.full_like(idx, -1)
    plan = dtc.moe_plan(none, E)
    y, saved = dtc.moe_experts(kind, x, wi, wo, w, plan, residual=x, save=True)
    assert torch.equal(y, x)
    for g in dtc.moe_experts_backward(kind, x, wi, wo, w, plan, saved):
        assert bool((g == 0).all())
    # no tokens
    e = dtc.moe_plan(idx[:0], E)
    y, saved = dtc.moe_experts(kind, x[:0], wi, wo, w[:0], e, save=True)
    assert y.shape == (0, H)
    _, dwi, dwo, _ = dtc.moe_experts_backward(kind, x[:0], wi, wo, w[:0], e, saved)
    assert bool((dwi == 0).all()) and bool((dwo == 0).all())


def test_experts_infinite_weights_of_others_do_not_leak():
    # an expert whose weights are NaN spoils its own tokens only, forward and backward
    import dense_tensor_core_gb300 as dtc
    kind, T, E, k, H, F, name = "bf16", 300, 4, 1, 136, 72, "swiglu"
    x, wi, wo, idx, w = batch(kind, T, E, k, H, F, name)
    wi[2], wo[2] = math.nan, math.inf
    dy = x
    plan = dtc.moe_plan(idx, E)
    y, saved = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, save=True)
    dx, dwi, dwo, _ = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, activation=name)
    clean = (idx != 2).all(1)
    assert bool(torch.isfinite(y[clean]).all()) and bool(torch.isfinite(dx[clean]).all())
    assert not bool(torch.isfinite(y[(idx == 2).any(1)]).any())
    for e in (0, 1, 3):
        assert bool(torch.isfinite(dwi[e]).all()) and bool(torch.isfinite(dwo[e]).all())


def test_experts_on_another_stream_and_in_a_graph():
    import dense_tensor_core_gb300 as dtc
    x, wi, wo, idx, w = batch("bf16", 100, 8, 2, 256, 128, "swiglu")
    want = dtc.moe_experts("bf16", x, wi, wo, w, dtc.moe_plan(idx, 8))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = dtc.moe_experts("bf16", x, wi, wo, w, dtc.moe_plan(idx, 8))
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dtc.moe_experts("bf16", x, wi, wo, w, dtc.moe_plan(idx, 8), out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_stale_plan_is_harmless():
    # a plan whose contents are not a plan at all: the kernels' own checks keep every access inside
    # the buffers (what comes out means nothing)
    import dense_tensor_core_gb300 as dtc
    x, wi, wo, idx, w = batch("bf16", 60, 8, 2, 128, 64, "swiglu")
    plan = dtc.moe_plan(idx, 8)
    want = dtc.moe_experts("bf16", x, wi, wo, w, plan)
    good = plan.data.clone()
    for fill in (-1, 0, 7, 2 ** 30):
        plan.data.fill_(fill)
        y, saved = dtc.moe_experts("bf16", x, wi, wo, w, plan, save=True)
        dtc.moe_experts_backward("bf16", x, wi, wo, w, plan, saved)
        torch.cuda.synchronize()
    plan.data.copy_(good)
    assert torch.equal(dtc.moe_experts("bf16", x, wi, wo, w, plan), want)


def test_rows_past_2_to_the_31_elements():
    import dense_tensor_core_gb300 as dtc
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB")
    T, E, k, H, F = 70000, 4, 16, 2048, 64  # 1.12 million rows of 2048: past 2^31 elements
    x = torch.randn((T, H), generator=gen(1), device="cuda").to(torch.bfloat16)
    wi = (torch.randn((E, F, H), generator=gen(2), device="cuda") * H ** -0.5).to(torch.bfloat16)
    wo = (torch.randn((E, H, F), generator=gen(3), device="cuda") * F ** -0.5).to(torch.bfloat16)
    idx = torch.randint(0, E, (T, k), generator=gen(4), device="cuda").to(torch.int32)
    w = torch.rand((T, k), generator=gen(5), device="cuda")
    y = dtc.moe_experts("bf16", x, wi, wo, w, dtc.moe_plan(idx, E), activation="gelu")
    for part in (slice(0, 50), slice(T - 50, T)):
        r, b = R.experts_bound("bf16", x[part].double(), wi.double(), wo.double(), w[part].double(), idx[part], "gelu")
        R.check(y[part], r, b, "rows")


def test_experts_timeout_reports_then_recovers():
    import dense_tensor_core_gb300 as dtc
    x, wi, wo, idx, w = batch("bf16", 300, 4, 2, 1024, 512, "swiglu")
    plan = dtc.moe_plan(idx, 4)
    dtc.gemm_stream_status()
    want = dtc.moe_experts("bf16", x, wi, wo, w, plan)
    dtc.moe_experts("bf16", x, wi, wo, w, plan, timeout_ns=20_000_000, fault_inject=1)
    with pytest.raises(dtc.GemmError) as e:
        dtc.gemm_stream_status()
    assert e.value.status == 4
    assert torch.equal(dtc.moe_experts("bf16", x, wi, wo, w, plan), want)
    dtc.gemm_stream_status()
