"""The `stream` argument of the products that allocate a workspace: it belongs to the stream the kernels
run on."""
import pytest
import torch

from test_ffn_streams_gpu import DELAY, dirty, overwrite

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def sparse():
    import dense_tensor_core_gb300 as dtc
    M, N, K = 256, 320, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    vals, B = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((M, K // 2), (N, K)))
    meta = torch.full((M, K // 8), 0x44, dtype=torch.uint8, device="cuda")  # the first two of every four
    return M * K * 2, lambda stream: dtc.gemm_sp("bf16", vals, meta, B, stream=stream)


def nvfp4():
    import dense_tensor_core_gb300 as dtc
    from dense_tensor_core_gb300 import workloads
    M, N, K = 256, 256, 512
    args = [torch.from_numpy(x).cuda() for x in workloads.make_nvfp4(M, N, K, 12)]
    return dtc.gemm_nvfp4_workspace_size(M, N, K), lambda stream: dtc.gemm_nvfp4(*args, stream=stream)


def dense():
    import dense_tensor_core_gb300 as dtc
    g = torch.Generator(device="cuda").manual_seed(1)
    A, B = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((256, 512), (320, 512)))
    return 256 * 320 * 2, lambda stream: dtc.gemm_bf16(A, B, stream=stream)


@pytest.mark.parametrize("busy", ["current", "given"])
@pytest.mark.parametrize("make", [sparse, nvfp4, dense])
def test_memory_belongs_to_the_given_stream(make, busy):
    n, call = make()
    want = call(None)
    s = torch.cuda.Stream()
    dirty([torch.cuda.current_stream(), s], [n])
    if busy == "current":  # the current stream still has to write into memory that it has freed
        torch.cuda._sleep(DELAY)
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    else:
        with torch.cuda.stream(s):
            torch.cuda._sleep(DELAY)
    got = call(s)
    keep = overwrite([n]) if busy == "given" else None
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del keep
