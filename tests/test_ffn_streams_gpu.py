"""The `stream` argument: what a call allocates and fills belongs to the stream its kernels run on, so
neither work still queued on the current stream nor what the current stream allocates next touches it."""
import pytest
import torch

import ffn_ref as R
from test_gemm_act_gpu import operands, rand

pytestmark = pytest.mark.gpu

DELAY = 100_000_000  # clock cycles, some 50 ms: far longer than the calls below


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dirty(streams, nbytes):
    """Leaves freed blocks of ones for the allocator to hand out again on these streams."""
    for s in streams:
        with torch.cuda.stream(s):
            for n in nbytes:
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()


def overwrite(nbytes):
    """Allocates and fills what the current stream gets for these sizes, a few times over."""
    keep = []
    for n in nbytes:
        for _ in range(4):
            keep.append(torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
    return keep


@pytest.mark.parametrize("busy", ["current", "given"])
def test_gradient_allocates_its_workspace_on_the_given_stream(busy):
    import dense_tensor_core_gb300 as dtc
    kind, M, N, K, name = "bf16", 777, 1544, 1032, "silu"
    A, B, Nb = operands(kind, "NT", M, N, K, name)
    dC, z = rand((M, N), kind, 5), rand((M, Nb), kind, 6)
    want = dtc.gemm_act_backward(kind, dC, A, B, preact=z, activation=name)
    n = dtc.gemm_act_backward_workspace_size(kind, M, N, K, activation=name)
    s = torch.cuda.Stream()
    dirty([torch.cuda.current_stream(), s], [n])
    with torch.cuda.stream(s if busy == "given" else None):
        torch.cuda._sleep(DELAY)
    got = dtc.gemm_act_backward(kind, dC, A, B, preact=z, activation=name, stream=s)
    keep = overwrite([n])
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    torch.cuda.synchronize()
    del keep


def experts_case(T=300, E=8, k=2, H=512, F=256, name="swiglu"):
    kind = "bf16"
    x, wi, wo = rand((T, H), kind, 1), rand((E, 2 * F, H), kind, 2, H ** -0.5), rand((E, H, F), kind, 3, F ** -0.5)
    logits = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    return kind, E, k, x, wi, wo, logits, rand((T, H), kind, 5)


def layer(case, stream=None):
    """All of the routed layer's calls; their outputs."""
    import dense_tensor_core_gb300 as dtc
    kind, E, k, x, wi, wo, logits, dy = case
    w, idx = dtc.moe_route(logits, k, stream=stream)
    plan = dtc.moe_plan(idx, E, stream=stream)
    y = dtc.moe_experts(kind, x, wi, wo, w, plan, stream=stream)
    y2, saved = dtc.moe_experts(kind, x, wi, wo, w, plan, save=True, stream=stream)
    dx, dwi, dwo, dw = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, stream=stream)
    dl = dtc.moe_route_backward(dw, logits, idx, stream=stream)
    return w, idx, y, y2, dx, dwi, dwo, dw, dl


def buffer_sizes(case):
    from dense_tensor_core_gb300 import _ffn
    kind, E, k, x, wi, wo, logits, dy = case
    sizes = [_ffn._experts_layout(0, 0, x.shape[0], k, E, x.shape[1], wo.shape[2], 5, train) for train in (False, True)]
    return [sizes[0][0], sizes[1][0], sizes[1][1]] + [t.numel() * t.element_size() for t in (x, wi, wo, logits)]


@pytest.mark.parametrize("T", [1, 12, 300])
@pytest.mark.parametrize("busy", ["current", "given"])
def test_experts_buffers_belong_to_the_given_stream(busy, T):
    case = experts_case(T)
    want = layer(case)
    sizes = buffer_sizes(case)
    s = torch.cuda.Stream()
    dirty([torch.cuda.current_stream(), s], sizes)
    with torch.cuda.stream(s if busy == "given" else None):
        torch.cuda._sleep(DELAY)
    got = layer(case, s)
    keep = overwrite(sizes)
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    torch.cuda.synchronize()
    del keep


@pytest.mark.parametrize("busy", ["current", "given"])
def test_outputs_belong_to_the_given_stream(busy):
    import dense_tensor_core_gb300 as dtc
    kind, M, N, K, name = "bf16", 300, 520, 264, "gelu"
    A, B, _ = operands(kind, "NT", M, N, K, name)
    want = dtc.gemm_act(kind, A, B, activation=name)
    s = torch.cuda.Stream()
    n = want.numel() * want.element_size()
    dirty([torch.cuda.current_stream(), s], [n])
    if busy == "current":  # the current stream still has to write into memory that it has freed
        torch.cuda._sleep(DELAY)
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    else:
        with torch.cuda.stream(s):
            torch.cuda._sleep(DELAY)
    got = dtc.gemm_act(kind, A, B, activation=name, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_the_current_stream_and_device_are_left_alone():
    import dense_tensor_core_gb300 as dtc
    A, B, _ = operands("bf16", "NT", 40, 64, 64, "none")
    s, before = torch.cuda.Stream(), torch.cuda.current_stream()
    dtc.gemm_act("bf16", A, B, stream=s)
    with pytest.raises(ValueError):
        dtc.gemm_act("bf16", A, B[:, :32], stream=s)
    assert torch.cuda.current_stream() == before
    dtc.gemm_act("bf16", A, B, stream=torch.cuda.default_stream())
    assert torch.cuda.current_stream() == before
