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
