"""Plain 64-bit references of the feed-forward operators, and the bounds their 16-bit results are
held to. Nothing here uses the library.

Rounding to the 16-bit type changes a value by at most U of its size (half an ulp: 2^-8 for bf16,
whose significand has 8 bits, 2^-11 for fp16, whose has 11), plus half the smallest subnormal of fp16. A sum of K products of 16-bit numbers
accumulated in fp32 (with truncation at worst) is off by at most (K + 2) 2^-23 times the sum of the
products' sizes. The activations in fp32 are off by at most 2^-18 of their size (an exponential of an
argument below 2^7 with a few ulp, a division, a handful of operations), and their slopes are at most
1.13."""
import math

import torch

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
GATED = ("swiglu", "geglu")
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "geglu")


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    g, u = z.chunk(2, -1)
    return act(g, {"swiglu": "silu", "geglu": "gelu"}[name]) * u


def act_bound(z, ez, name):
    """Bound of the error of act(z) in fp32 when z is off by ez."""
    if name in GATED:
        g, u = z.chunk(2, -1)
        eg, eu = ez.chunk(2, -1)
        inner = {"swiglu": "silu", "geglu": "gelu"}[name]
        e1 = act_bound(g, eg, inner)
        return e1 * (u.abs() + eu) + act(g, inner).abs() * eu + 2.0 ** -22 * act(z, name).abs()
    return 1.13 * ez + 2.0 ** -18 * z.abs()


def op_a(A, layout):
    return A.double() if layout[0] == "N" else A.double().t()


def op_b(B, layout):
    return B.double().t() if layout[1] == "T" else B.double()


def gemm_act(kind, A, B, layout, bias, residual, name):
    """(y, bound of y, z, bound of z)"""
    a, b = op_a(A, layout), op_b(B, layout)
    z, s = a @ b, a.abs() @ b.abs()
    if bias is not None:
        z, s = z + bias.double(), s + bias.double().abs()
    ez = (a.shape[1] + 2) * 2.0 ** -23 * s
    y, ey = act(z, name), act_bound(z, ez, name)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -23 * y.abs()
    u, t = U[kind], TINY[kind]
    return y, ey * (1 + u) + u * y.abs() + t, z, ez * (1 + u) + u * z.abs() + t


def check(got, ref, bound, what):
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst "
                                 f"{float((d / bound).nan_to_num(1e30).max()):.3g} of it")


def close(got, ref, tol, what):
    """The norm of the difference against the norm of the reference."""
    d, n = float((got.double() - ref).norm()), float(ref.norm())
    assert d <= tol * n or (n == 0 and d == 0), f"{what}: off by {d / max(n, 1e-300):.3g}, allowed {tol:.3g}"


# ------------------------------------------------------------------------------------------------
# routing, token by token
# ------------------------------------------------------------------------------------------------
def route(logits, k, bias, scoring, groups, top_groups, renorm, scale):
    """(weights as 64-bit numbers, indices), keys in fp32 as the operator defines them."""
    z32 = logits.float().cpu()
    T, E = z32.shape
    key = 1 / (1 + torch.exp(-z32)) if scoring == "sigmoid" else z32.clone()
    if bias is not None:
        key = key + bias.float().cpu()
    z = z32.double()
    W, I = torch.zeros(T, k, dtype=torch.float64), torch.full((T, k), -1, dtype=torch.int32)
    for t in range(T):
        live = [e for e in range(E) if z32[t, e] > -math.inf and key[t, e] > -math.inf]
        if groups > 1:
            per = E // groups
            score = {}
            for g in range(groups):
                ks = sorted((float(key[t, e]) for e in live if e // per == g), reverse=True)
                if ks:
                    two = scoring == "sigmoid" and len(ks) > 1
                    score[g] = float(torch.tensor(ks[0]) + torch.tensor(ks[1])) if two else ks[0]
            best = sorted(score, key=lambda g: (-score[g], g))[:top_groups]
            live = [e for e in live if e // per in best]
        chosen = sorted(live, key=lambda e: (-float(key[t, e]), e))[:k]
        if not chosen:
            continue
        zc = z[t, chosen]
        if scoring == "sigmoid":
            w = torch.sigmoid(zc)
            if renorm:
                w = w / w.sum() if w.sum() > 0 else w * 0
        elif renorm:
            w = torch.softmax(zc, 0)
        else:
            every = z[t][z32[t] > -math.inf]
            m = every.max()  # (taken out by hand: log of the count vanishes beside a logit of 3e38)
            w = torch.exp(zc - m) / torch.exp(every - m).sum()
        W[t, :len(chosen)] = w * scale
        I[t, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return W, I


def route_weights(z, idx, scoring, renorm, scale):
    """The weights of given choices as a differentiable function of 64-bit logits (no masked ones
    among the choices)."""
    got = idx >= 0
    zc = torch.gather(z, 1, idx.clamp(min=0).long())
    if scoring == "sigmoid":
        w = torch.where(got, torch.sigmoid(zc), 0.0)
        if renorm:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    elif renorm:
        w = torch.where(got, torch.exp(zc - zc.detach().max(1, keepdim=True).values), 0.0)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.where(got, torch.exp(zc - torch.logsumexp(z, 1, keepdim=True)), 0.0)
    return w * scale


def plan(idx, E):
    """(offsets, counts, slots) by a walk over the choices."""
    flat = idx.reshape(-1).tolist()
    counts = [0] * E
    for e in flat:
        if 0 <= e < E:
            counts[e] += 1
    off = [0]
    for c in counts:
        off.append(off[-1] + (c + 15) // 16 * 16)
    at, slots = list(off[:E]), []
    for e in flat:
        if 0 <= e < E:
            slots.append(at[e])
            at[e] += 1
        else:
            slots.append(-1)
    return off, counts, slots


def experts(x, w_in, w_out, w, idx, name, residual=None):
    """y as a differentiable function of 64-bit tensors."""
    T, k = idx.shape
    y = torch.zeros_like(x) if residual is None else residual
    for e in range(w_in.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            h = act(x[t] @ w_in[e].t(), name) * w[t, j, None]
            y = y.index_add(0, t, h @ w_out[e].t())
    return y


def experts_bound(kind, x, w_in, w_out, w, idx, name, residual=None):
    """Elementwise bound of the error of y: the first product's sum, the activation, the rounding of
    weight times activation, the second product's sum, the rounding of its rows, the join and the
    last rounding."""
    u, t16 = U[kind], TINY[kind]
    E, F = w_in.shape[0], w_out.shape[2]
    bound = torch.zeros_like(x)
    size = torch.zeros_like(x) if residual is None else residual.abs().clone()
    y = torch.zeros_like(x) if residual is None else residual.clone()
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        z = x[t] @ w_in[e].t()
        ez = (x.shape[1] + 2) * 2.0 ** -23 * (x[t].abs() @ w_in[e].t().abs())
        ww = w[t, j, None].abs()
        h = act(z, name) * w[t, j, None]
        eh = (act_bound(z, ez, name) * ww + 2.0 ** -22 * h.abs()) * (1 + u) + u * h.abs() + t16
        o = h @ w_out[e].t()
        eo = eh @ w_out[e].t().abs() + (F + 2) * 2.0 ** -23 * ((h.abs() + eh) @ w_out[e].t().abs())
        eo = eo * (1 + u) + u * o.abs() + t16
        bound.index_add_(0, t, eo)
        size.index_add_(0, t, o.abs())
        y.index_add_(0, t, o)
    bound = bound + (idx.shape[1] + 2) * 2.0 ** -23 * size
    return y, bound * (1 + u) + u * y.abs() + t16
