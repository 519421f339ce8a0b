"""Arguments that the binding refuses with tensors on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def experts():
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    idx = torch.zeros((20, 2), dtype=torch.int32, device="cuda")
    return idx, (e(20, 64), e(4, 64, 64), e(4, 64, 64), torch.zeros((20, 2), device="cuda"))


@pytest.mark.parametrize("spoil", [lambda d: d[:-1], lambda d: d[:16], lambda d: d[:0], lambda d: torch.cat([d, d]),
                                   lambda d: d[::2], lambda d: d.long(), lambda d: d.cpu()])
def test_plans_of_another_size(spoil):
    import dense_tensor_core_gb300 as dtc
    idx, args = experts()
    plan = dtc.moe_plan(idx, 4)
    _, saved = dtc.moe_experts("bf16", *args, plan, activation="silu", save=True)
    plan.data = spoil(plan.data)
    with pytest.raises((ValueError, TypeError)):
        dtc.moe_experts("bf16", *args, plan, activation="silu")
    with pytest.raises((ValueError, TypeError)):
        dtc.moe_experts_backward("bf16", *args, plan, saved, activation="silu")


@pytest.mark.parametrize("kw", [dict(top_k=2 ** 32 + 2), dict(top_k=-1), dict(top_k=2 ** 63 - 1), dict(groups=2 ** 32 + 1),
                                dict(top_groups=2 ** 32 + 1)])
def test_counts_past_32_bits(kw):
    import dense_tensor_core_gb300 as dtc
    args = dict(dict(top_k=2), **kw)
    with pytest.raises((ValueError, dtc.GemmError)):
        dtc.moe_route(torch.zeros((4, 8), device="cuda"), args.pop("top_k"), **args)


def test_negative_wait_limits():
    import dense_tensor_core_gb300 as dtc
    idx, args = experts()
    plan = dtc.moe_plan(idx, 4)
    x, w = args[0], args[1][0]
    _, saved = dtc.moe_experts("bf16", *args, plan, activation="silu", save=True)
    for call in (lambda: dtc.gemm_act("bf16", x, w, timeout_ns=-1),
                 lambda: dtc.gemm_act_backward("bf16", x, x, w, timeout_ns=-1),
                 lambda: dtc.moe_experts("bf16", *args, plan, activation="silu", timeout_ns=-1),
                 lambda: dtc.moe_experts_backward("bf16", *args, plan, saved, activation="silu", timeout_ns=-1)):
        with pytest.raises(ValueError):
            call()
