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


# the gradient of a weight is taken at the unrounded first product: with fp32 weights nothing on the way
# to it is rounded to 16 bits
@pytest.mark.parametrize("T,F", [(1, 136), (12, 136), (40, 72), (300, 136)])
@pytest.mark.parametrize("kind,name", [("bf16", "swiglu"), ("bf16", "silu"), ("f16", "geglu"), ("bf16", "gelu")])
def test_gradient_at_the_unrounded_product(kind, name, T, F):
    import dense_tensor_core_gb300 as dtc
    dt, H, E, k = R.DT[kind], 64, 8, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda std, *s: (torch.randn(s, generator=g, device="cuda") * std).to(dt)  # noqa: E731
    x, dy = r(1, T, H), r(1, T, H)
    wi, wo = r(H ** -0.5, E, 2 * F if name in R.GATED else F, H), r(F ** -0.5, E, H, F)
    idx, w = choices(T, E, k, T), torch.rand((T, k), generator=g, device="cuda")
    plan = dtc.moe_plan(idx, E)
    _, saved = dtc.moe_experts(kind, x, wi, wo, w, plan, activation=name, save=True)
    dw = dtc.moe_experts_backward(kind, dy, wi, wo, w, plan, saved, activation=name)[3]
    got, at = idx >= 0, idx.clamp(min=0).long()
    xd, dyd, wi, wo = x.double(), dy.double(), wi.double()[at], wo.double()[at]
    z = torch.einsum("tkfh,th->tkf", wi, xd)
    ez = (H + 2) * 2.0 ** -23 * torch.einsum("tkfh,th->tkf", wi.abs(), xd.abs())
    dh = torch.einsum("tkhf,th->tkf", wo, dyd)
    edh = (H + 2) * 2.0 ** -23 * torch.einsum("tkhf,th->tkf", wo.abs(), dyd.abs())
    h, eh = R.act(z, name), R.act_bound(z, ez, name)
    want = (dh * h).sum(2) * got
    bound = (edh * (h.abs() + eh) + dh.abs() * eh).sum(2) + (F + 2) * 2.0 ** -23 * (dh * h).abs().sum(2)
    R.check(dw, want, bound * got, "dweights")
    if T > 5 and kind == "bf16":  # a rounded product would show
        off = ((dh * R.act(z.to(dt).double(), name)).sum(2) * got - want).abs() > bound
        assert bool(off.any())
