"""A mixture-of-experts feed-forward layer, trained and then run a token at a time:

    y = x + shared(x) + sum_j w_j expert_j(x)

with a gated layer that every token passes (gemm_act), a router (gemm_act, moe_route) and the experts
it chooses (moe_plan, moe_experts), and the gradient of all of it by the operators' own backward
forms. Weights are kept in fp32 and used in bf16; torch does the loss and the update. Run:

    python -m dense_tensor_core_gb300.examples.feed_forward
"""
import argparse

import torch

import dense_tensor_core_gb300 as dtc

KIND, ACT = "bf16", "swiglu"


class Layer:
    def __init__(self, hidden, inner, experts, top_k, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=device) * s[-1] ** -0.5  # noqa: E731
        self.top_k, self.experts = top_k, experts
        self.w = {"router": r(experts, hidden), "up": r(2 * inner, hidden), "down": r(hidden, inner),
                  "experts_in": r(experts, 2 * inner, hidden), "experts_out": r(experts, hidden, inner)}
        self.half = {n: w.bfloat16() for n, w in self.w.items()}

    def forward(self, x, train=False):
        p = self.half
        z = x.new_empty((x.shape[0], p["up"].shape[0])) if train else None
        h = dtc.gemm_act(KIND, x, p["up"], activation=ACT, preact=z)
        y = dtc.gemm_act(KIND, h, p["down"], residual=x)
        logits = dtc.gemm_act(KIND, x, p["router"])
        weights, chosen = dtc.moe_route(logits, self.top_k)
        plan = dtc.moe_plan(chosen, self.experts)
        if not train:
            return dtc.moe_experts(KIND, x, p["experts_in"], p["experts_out"], weights, plan, activation=ACT,
                                   residual=y)
        y, rows = dtc.moe_experts(KIND, x, p["experts_in"], p["experts_out"], weights, plan, activation=ACT,
                                  residual=y, save=True)
        return y, (x, z, h, logits, weights, chosen, plan, rows)

    def backward(self, dy, saved):
        """Gradients of the weights (those of x are not needed by one layer)."""
        p, g = self.half, {}
        x, z, h, logits, weights, chosen, plan, rows = saved
        _, g["experts_in"], g["experts_out"], dweights = dtc.moe_experts_backward(
            KIND, dy, p["experts_in"], p["experts_out"], weights, plan, rows, activation=ACT, need_x=False)
        dlogits = dtc.moe_route_backward(dweights, logits, chosen)
        only = (False, True, False)
        _, g["router"], _ = dtc.gemm_act_backward(KIND, dlogits, x, p["router"], need=only)
        dh, g["down"], _ = dtc.gemm_act_backward(KIND, dy, h, p["down"], need=(True, True, False))
        _, g["up"], _ = dtc.gemm_act_backward(KIND, dh, x, p["up"], z, activation=ACT, need=only)
        return g

    def update(self, grads, rate):
        for n, g in grads.items():
            self.w[n].add_(g.float(), alpha=-rate)
            self.half[n].copy_(self.w[n])


def run(tokens=512, hidden=256, inner=128, experts=16, top_k=4, steps=20, rate=0.1):
    """(losses of the steps, largest difference between a batch's rows and the same rows alone, the
    largest value of the batch's result)."""
    layer, goal = Layer(hidden, inner, experts, top_k, 1), Layer(hidden, inner, experts, top_k, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    want = goal.forward(x).float()
    losses = []
    for _ in range(steps):
        y, saved = layer.forward(x, train=True)
        off = y.float() - want
        losses.append(off.square().sum(1).mean())
        layer.update(layer.backward((off * (2 / tokens)).bfloat16(), saved), rate)
    y = layer.forward(x)
    alone = torch.cat([layer.forward(x[i:i + 1]) for i in range(4)])
    dtc.gemm_stream_status()
    diff, top = (alone.float() - y[:4].float()).abs().max(), y[:4].float().abs().max()
    return [float(v) for v in losses], float(diff), float(top)


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 512), ("hidden", 256), ("inner", 128), ("experts", 16), ("top-k", 4),
                        ("steps", 20)):
        a.add_argument("--" + name, type=int, default=value)
    a.add_argument("--rate", type=float, default=0.1)
    o = a.parse_args()
    losses, diff, top = run(o.tokens, o.hidden, o.inner, o.experts, o.top_k, o.steps, o.rate)
    print(f"loss {losses[0]:.4g} -> {losses[-1]:.4g} in {len(losses)} steps; four tokens one at a time "
          f"differ from the batch by {diff:.3g} of {top:.3g}")


if __name__ == "__main__":
    main()
