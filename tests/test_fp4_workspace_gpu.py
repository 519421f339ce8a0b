"""The workspace of the 4-bit products: splits of the plan's own choice beside gemm_act's, and products that take none."""
import pytest
import torch

import ffn_ref as R
import fp4_ref as Q
from test_fp4_gpu import operands, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


HEAD = 1 << 16  # (the words that are zero between calls lie in front of this)


@pytest.mark.parametrize("fmt,M", [("mxfp4", 1), ("nvfp4", 24), ("mxfp4", 40), ("nvfp4", 64)])
def test_splits_of_the_plans_choice_beside_gemm_act(fmt, M):
    """One workspace of the size that both ask for: gemm_fp4 splits K in it (its pieces overwrite what was there), and
    both stay right, by the definition, however they take turns."""
    import dense_tensor_core_gb300 as dtc
    N, K = 4096, 8192
    n4 = dtc.gemm_fp4_workspace_size(M, N, K)
    n = max(n4, dtc.gemm_act_workspace_size("bf16", 24, 512, 8192))
    assert n4 > 2 * HEAD
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    a, b, _ = operands("bf16", fmt, M, N, K, "none")
    qa, qb = dtc.quantize_fp4(a, format=fmt), dtc.quantize_fp4(b, format=fmt)
    c, d = rand((24, 8192), "bf16", 1), rand((512, 8192), "bf16", 2, 8192 ** -0.5)
    want, bound = Q.product("bf16", Q.rounded(a, fmt), Q.rounded(b, fmt), None, None, "none")
    want2, bound2, _, _ = R.gemm_act("bf16", c, d, "NT", None, None, "none")
    first = None
    for _ in range(3):
        ws[HEAD:] = 0xFF  # NaNs, if a piece that was not written were read
        y = dtc.gemm_fp4("bf16", qa, qb, workspace=ws)
        assert int((ws[HEAD:n4] != 0xFF).sum()) > 0, "no piece was written"
        z = dtc.gemm_act("bf16", c, d, workspace=ws)
        dtc.gemm_stream_status()
        R.check(y, want, bound, f"{fmt} {M}")
        R.check(z, want2, bound2, "gemm_act")
        if first is not None:
            assert torch.equal(y, first[0]) and torch.equal(z, first[1])
        first = y, z


def test_a_few_rows_in_nvfp4_take_no_workspace():
    """Their kernel does not split K: it neither needs nor touches what gemm_fp4_workspace_size, a bound over both
    formats, asks for."""
    import dense_tensor_core_gb300 as dtc
    a, b, _ = operands("bf16", "nvfp4", 1, 4096, 8192, "none")
    qa, qb = dtc.quantize_fp4(a), dtc.quantize_fp4(b)
    ws = torch.full((dtc.gemm_fp4_workspace_size(1, 4096, 8192),), 0xAB, dtype=torch.uint8, device="cuda")
    y = dtc.gemm_fp4("bf16", qa, qb, workspace=ws)
    assert bool((ws == 0xAB).all())
    assert torch.equal(y, dtc.gemm_fp4("bf16", qa, qb))
