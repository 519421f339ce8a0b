"""The activations and their derivatives where they are small: relative bounds over the negative tail,
from sums that are exact (K = 0, so that Z is the bias; one row, so that dbias is dZ, in fp32)."""
import math

import pytest
import torch

import ffn_ref as R

pytestmark = pytest.mark.gpu

# how far down each tail goes before its result leaves the normal numbers of fp32 (tanh's and the
# logistic's are cut off there)
LOWEST = {"gelu": -12.5, "gelu_tanh": -9.5, "silu": -85.0}


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def tail(kind, name):
    z = torch.linspace(LOWEST[name], 6.0, 4096, dtype=torch.float64, device="cuda")
    return z.to(R.DT[kind])


def parts(z, name):
    """f(z), f'(z) and the size of the terms of f'(z), without cancellation, and the relative error of
    fp32: the argument of the exponential (of erfc, which falls as one) is off by a few roundings of its
    size, which is that of the result's relative error; the rest by a few ulp."""
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        q = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * p, p + z * q, p + (z * q).abs(), (z * z + 16) * 2.0 ** -22
    if name == "silu":
        v, dv = z, torch.ones_like(z)
    else:
        c = math.sqrt(2 / math.pi)
        v, dv = 2 * c * (z + 0.044715 * z ** 3), 2 * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(v)
    t = s * torch.sigmoid(-v)
    return z * s, s + z * t * dv, s + (z * t * dv).abs(), (2 * v.abs() + 16) * 2.0 ** -22


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu", "geglu", "swiglu"])
@pytest.mark.parametrize("rows", [1, 40])  # without tiles and with
def test_forward(kind, name, rows):
    import dense_tensor_core_gb300 as dtc
    inner = {"geglu": "gelu", "swiglu": "silu"}.get(name, name)
    z = tail(kind, inner)
    N, K = z.numel(), 0 if rows > 1 else 8
    gated = name in R.GATED
    bias = torch.cat([z, torch.ones_like(z)]) if gated else z
    e = lambda *s: torch.zeros(s, dtype=z.dtype, device="cuda")  # noqa: E731
    y = dtc.gemm_act(kind, e(rows, K), e(bias.numel(), K), bias=bias, activation=name)
    f, _, _, rel = parts(z.double(), inner)
    bound = (R.U[kind] * (1 + rel) + rel) * f.abs() + R.TINY[kind]
    R.check(y, f.expand(rows, N), bound.expand(rows, N), name)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_derivative(kind, name):
    import dense_tensor_core_gb300 as dtc
    z = tail(kind, name)
    N = z.numel()
    ones = torch.ones((1, N), dtype=z.dtype, device="cuda")
    A, B = torch.zeros((1, 8), dtype=z.dtype, device="cuda"), torch.zeros((N, 8), dtype=z.dtype, device="cuda")
    _, _, db = dtc.gemm_act_backward(kind, ones, A, B, preact=z[None], activation=name, need=(False, False, True))
    _, d, size, rel = parts(z.double(), name)
    R.check(db, d, rel * size, name)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_experts_gradient(kind):
    # one expert and one choice a token with weight 1: the gradient of the weight is dy . W_out f(z), in
    # fp32 here, and W_out the identity, so that each token shows one value of f
    import dense_tensor_core_gb300 as dtc
    T, H = 512, 512
    z = torch.linspace(LOWEST["gelu"], 6.0, T, dtype=torch.float64, device="cuda").to(R.DT[kind])
    eye = torch.eye(H, dtype=z.dtype, device="cuda")
    x = torch.diag(z)  # token t: z[t] in column t
    idx, w = torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda")
    plan = dtc.moe_plan(idx, 1)
    _, saved = dtc.moe_experts(kind, x, eye[None], eye[None], w, plan, activation="gelu", save=True)
    _, _, _, dw = dtc.moe_experts_backward(kind, eye, eye[None], eye[None], w, plan, saved, activation="gelu")
    f, _, _, rel = parts(z.double(), "gelu")
    R.check(dw[:, 0], f, rel * f.abs(), "dweights")
