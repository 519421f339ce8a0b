"""The feed-forward example learns, and a token alone gets what it gets in a batch."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_feed_forward_example():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_tensor_core_gb300.examples import feed_forward

    losses, diff, top = feed_forward.run(steps=12)
    assert losses[-1] < losses[0]
    # roundings to bf16 (2^-8 each) of h, y, the logits, h of the experts, their rows and the result
    # may fall the other way when the sums run in another order
    assert diff <= 6 * 2.0 ** -8 * top


def test_gradients_of_the_whole_layer():
    import ffn_ref as R
    from dense_tensor_core_gb300.examples.feed_forward import Layer

    layer = Layer(256, 128, 16, 4, 1)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((500, 256), generator=g, device="cuda").bfloat16()
    dy = torch.randn((500, 256), generator=g, device="cuda").bfloat16()
    _, saved = layer.forward(x, train=True)
    got = layer.backward(dy, saved)
    p = {n: w.double().requires_grad_() for n, w in layer.half.items()}
    X, chosen = x.double(), saved[5]
    base = X + R.act(X @ p["up"].t(), "swiglu") @ p["down"].t()
    w = torch.softmax(torch.gather(X @ p["router"].t(), 1, chosen.long()), 1)
    y = R.experts(X, p["experts_in"], p["experts_out"], w, chosen, "swiglu", base)
    want = torch.autograd.grad(y, list(p.values()), dy.double())
    # at most 6 roundings to bf16 on the way to any of them, each at most 2^-8 of the norm
    for n, r in zip(p, want):
        R.close(got[n], r, 6 * R.U["bf16"], n)
