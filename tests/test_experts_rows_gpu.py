"""The join of a token's experts adds unrounded rows: with whole numbers that every product holds
exactly, the result is the exact sum, rounded once."""
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


def whole(shape, seed, high=31):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-high, high + 1, shape, generator=g, device="cuda").double()


def choices(T, E, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    if T > 4:
        idx[1] = -1
        idx[3, k - 1] = -1
    return idx


# H whole 256-column pieces of the join, below one and off them; T with and without tiles, split and not;
# sums stay below the largest fp16, and rows need more bits than 16-bit types have
@pytest.mark.parametrize("T", [1, 5, 16, 17, 60, 700])
@pytest.mark.parametrize("H,E,k", [(72, 4, 2), (64, 8, 4), (136, 3, 1)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_forward_and_gradient(kind, T, H, E, k):
    import dense_tensor_core_gb300 as dtc
    dt = R.DT[kind]
    idx = choices(T, E, k, T)
    got = idx >= 0
    at = idx.clamp(min=0).long()
    w = torch.ones((T, k), device="cuda")
    x, m, res = whole((T, H), 1), whole((E, H, H), 2), whole((T, H), 3, 200)
    eye = torch.eye(H, device="cuda").to(dt).expand(E, H, H).contiguous()
    plan = dtc.moe_plan(idx, E)
    rows = torch.einsum("tkij,tj->tki", m[at], x) * got[..., None]
    want = rows.sum(1)
    assert T < 5 or not torch.equal(rows.to(dt).double().sum(1), want)  # rounded rows would show
    for r in (None, res):
        exact = want if r is None else want + r
        for save in (False, True):
            y = dtc.moe_experts(kind, x.to(dt), eye, m.to(dt), w, plan, activation="none",
                                residual=None if r is None else r.to(dt), save=save)
            assert torch.equal(y[0] if save else y, exact.to(dt))
    # dx = the sum of the rows dz . W_in with dz = dy (W_out the identity)
    _, saved = dtc.moe_experts(kind, x.to(dt), m.to(dt), eye, w, plan, activation="none", save=True)
    dx = dtc.moe_experts_backward(kind, x.to(dt), m.to(dt), eye, w, plan, saved, activation="none")[0]
    exact = (torch.einsum("tkji,tj->tki", m[at], x) * got[..., None]).sum(1)
    assert torch.equal(dx, exact.to(dt))


def test_wide_rows():
    # several 256-column pieces a row and a last one that is part empty; one input column each, so that
    # the sums stay small
    import dense_tensor_core_gb300 as dtc
    T, H, F, E, k = 40, 1160, 64, 5, 3
    idx = choices(T, E, k, 9)
    w = torch.ones((T, k), device="cuda")
    x, wi, wo = whole((T, H), 1, 1), torch.zeros((E, F, H), device="cuda").double(), whole((E, H, F), 3)
    wi[:, torch.arange(F), torch.arange(F) * 18] = 1
    y = dtc.moe_experts("bf16", x.bfloat16(), wi.bfloat16(), wo.bfloat16(), w, dtc.moe_plan(idx, E), activation="none")
    exact = torch.einsum("tkij,tj->tki", wo[idx.clamp(min=0).long()], x[:, torch.arange(F) * 18])
    assert torch.equal(y, (exact * (idx >= 0)[..., None]).sum(1).bfloat16())
