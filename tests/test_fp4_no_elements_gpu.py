"""Rows of no elements: what quantize_fp4 leaves in their factors."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("shape,gated", [((4, 0), False), ((2, 16, 0), True), ((300, 0), False)])
def test_factors_of_rows_without_elements_are_one(shape, gated):
    """As for a row of zeros."""
    import dense_tensor_core_gb300 as dtc
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    q = dtc.quantize_fp4(x, gated=gated)
    q.row_scale.fill_(7.0)
    assert dtc.quantize_fp4(x, gated=gated, out=q) is q
    assert q.row_scale.shape == shape[:-1] and bool((q.row_scale == 1).all())
