"""The feed-forward operators of a language model beside the dense product: what is measured.

* ``act``, ``act_bwd``: a product with bias, activation (plain or gated) and residual in its
  epilogue, and its gradient.
* ``route``, ``route_bwd``: routing of tokens to experts (scores, groups, top-k, weights, the rows'
  places in expert order), and the gradient of the weights with respect to the logits.
* ``experts``, ``experts_train``: the routed experts' two products with the weighted join, and a
  training step through them.

`run` computes a case with elementary torch operations in 32 bits, or, where `own` is true, with the
calls of dense_tensor_core_gb300. `exact` computes it from the definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GATED = ("swiglu", "geglu")
ALIGN = 16  # an expert's rows start at a multiple of this


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # the smallest product of the tests and the smoke run, with everything in its epilogue: latency
        dict(name="act_small", op="act", kind="bf16", layout="NT", M=256, N=256, K=512, act="gelu",
             bias=True, res=True, keep=False),
        # one new token through an 8192 x 8192 layer (the skinny benchmark product's B): serving
        dict(name="act_token", op="act", kind="bf16", layout="NT", M=1, N=8192, K=8192, act="none",
             bias=True, res=True, keep=False),
        # a ragged batch through a gated layer in training: odd M, N and K off every tile size
        dict(name="act_odd", op="act", kind="f16", layout="NT", M=1111, N=2056, K=2040, act="swiglu",
             bias=True, res=False, keep=True),
        # the headline product with its epilogue
        dict(name="act_large", op="act", kind="bf16", layout="NT", M=4096, N=4096, K=8192,
             act="gelu_tanh", bias=True, res=True, keep=True),
        # gradients of a ragged ungated layer, weights stored [K, N]
        dict(name="act_bwd_odd", op="act_bwd", kind="f16", layout="NN", M=777, N=1544, K=1032,
             act="silu"),
        # gradients of the headline product as a gated layer of the same work
        dict(name="act_bwd_large", op="act_bwd", kind="bf16", layout="NT", M=4096, N=2048, K=8192,
             act="swiglu"),
        # routing of a few new tokens: latency
        dict(name="route_small", op="route", logits="f32", T=4, E=64, k=8, scoring="softmax",
             bias=False, groups=1, top_groups=1, renorm=True),
        # routing of a long prompt over many experts in groups, with a balance bias
        dict(name="route_large", op="route", logits="f32", T=65536, E=256, k=8, scoring="sigmoid",
             bias=True, groups=8, top_groups=4, renorm=True),
        # a training step of a router with an odd number of experts and bf16 logits
        dict(name="route_bwd_odd", op="route_bwd", logits="bf16", T=16383, E=60, k=4,
             scoring="softmax", bias=True, groups=1, top_groups=1, renorm=False),
        # one new token through its experts: serving
        dict(name="experts_token", op="experts", kind="bf16", T=1, E=64, k=8, H=2048, F=1024,
             act="swiglu", res=True),
        # a prompt through its experts
        dict(name="experts_prompt", op="experts", kind="bf16", T=4096, E=64, k=8, H=2048, F=1024,
             act="swiglu", res=True),
        # a training step with ragged token counts and an odd inner size
        dict(name="experts_train", op="experts_train", kind="bf16", T=5000, E=48, k=6, H=2048,
             F=1000, act="swiglu", res=False),
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(round(v / mult)) * mult)


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 6e11 and w["bytes"] <= 1.5e9:
            return c


def _draw(rng):
    op = rng.choice(["act", "act", "act_bwd", "route", "route_bwd", "experts", "experts",
                     "experts_train"])
    kind = rng.choice(["bf16", "f16"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "geglu"])
    if op in ("act", "act_bwd"):
        layout = "NT" if act in GATED else rng.choice(["NT", "NN", "TN", "TT"])
        m_mult = 8 if layout[0] == "T" else 1
        c = dict(op=op, kind=kind, layout=layout,
                 M=_log(rng, 1 if op == "act" else 16, 8192, m_mult), N=_log(rng, 64, 8192, 8),
                 K=_log(rng, 64, 8192, 8), act=act)
        if op == "act":
            c.update(bias=rng.random() < 0.7, res=rng.random() < 0.5, keep=rng.random() < 0.4)
        return c
    E = rng.choice([8, 16, 20, 32, 60, 64, 96, 128, 160, 256])
    k = rng.randint(1, 8)
    if op in ("route", "route_bwd"):
        groups = rng.choice([g for g in (1, 4, 8) if E % g == 0 and E // g >= 2])
        top = rng.randint(1, groups)
        return dict(op=op, logits=rng.choice(["f32", "bf16", "f16"]),
                    T=_log(rng, 1 if op == "route" else 64, 65536), E=E,
                    k=min(k, top * (E // groups)), scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top,
                    renorm=rng.random() < 0.7)
    return dict(op=op, kind=kind, T=_log(rng, 1 if op == "experts" else 32, 8192), E=E, k=k,
                H=_log(rng, 128, 4096, 8), F=_log(rng, 64, 2048, 8), act=act,
                res=op == "experts" and rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _router_logits(g, T, E, dtype):
    """Logits with experts of uneven popularity; one token in 50 is padding (its whole row masked),
    one logit in 200 is masked."""
    z = torch.randn((T, E), generator=g, device="cuda") * 1.5
    z += torch.randn((1, E), generator=g, device="cuda") * 0.5
    z.masked_fill_(torch.rand((T, E), generator=g, device="cuda") < 0.005, -math.inf)
    if T > 1:
        z.masked_fill_(torch.rand((T, 1), generator=g, device="cuda") < 0.02, -math.inf)
    return z.to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("act", "act_bwd"):
        M, N, K, lay, dt = case["M"], case["N"], case["K"], case["layout"], DT[case["kind"]]
        Nb = 2 * N if case["act"] in GATED else N
        s["A"] = _normal(g, (M, K) if lay[0] == "N" else (K, M), 1.0, dt)
        s["B"] = _normal(g, (Nb, K) if lay[1] == "T" else (K, Nb), K ** -0.5, dt)
        if op == "act":
            s["bias"] = _normal(g, (Nb,), 0.2, dt) if case["bias"] else None
            s["res"] = _normal(g, (M, N), 1.0, dt) if case["res"] else None
        else:
            s["dC"] = _normal(g, (M, N), 1.0, dt)
            s["z"] = _normal(g, (M, Nb), 1.0, dt) if case["act"] != "none" else None
        if own:
            import dense_tensor_core_gb300 as dtc
            size = dtc.gemm_act_workspace_size if op == "act" else dtc.gemm_act_backward_workspace_size
            n = size(case["kind"], M, N, K, layout=lay, activation=case["act"])
            s["ws"] = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    elif op in ("route", "route_bwd"):
        s["logits"] = _router_logits(g, case["T"], case["E"], DT[case["logits"]])
        s["bias"] = _normal(g, (case["E"],), 0.1, torch.float32) if case["bias"] else None
        if op == "route_bwd":
            s["dw"] = _normal(g, (case["T"], case["k"]), 1.0, torch.float32)
    else:
        T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
        dt = DT[case["kind"]]
        Fz = 2 * F if case["act"] in GATED else F
        s["x"] = _normal(g, (T, H), 1.0, dt)
        s["w_in"] = _normal(g, (E, Fz, H), H ** -0.5, dt)
        s["w_out"] = _normal(g, (E, H, F), F ** -0.5, dt)
        z = _router_logits(g, T, E, torch.float32)
        v, i = torch.topk(z, k, dim=1)
        s["idx"] = torch.where(torch.isinf(v), -1, i).to(torch.int32)
        s["w"] = torch.nan_to_num(torch.softmax(v, 1)).to(dt)
        s["res"] = _normal(g, (T, H), 1.0, dt) if case["res"] else None
        if op == "experts_train":
            s["dy"] = _normal(g, (T, H), 1.0, dt)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_tensor_core_gb300 as dtc
    c = s["case"]
    op = c["op"]
    if op == "act":
        z = None
        if c["keep"]:
            z = torch.empty((c["M"], c["N"] * (2 if c["act"] in GATED else 1)), dtype=s["A"].dtype,
                            device="cuda")
        y = dtc.gemm_act(c["kind"], s["A"], s["B"], layout=c["layout"], bias=s["bias"],
                         residual=s["res"], activation=c["act"], preact=z, workspace=s["ws"])
        return {"y": y, "z": z} if c["keep"] else {"y": y}
    if op == "act_bwd":
        dA, dB, db = dtc.gemm_act_backward(c["kind"], s["dC"], s["A"], s["B"], preact=s["z"],
                                           layout=c["layout"], activation=c["act"],
                                           workspace=s["ws"])
        return {"dA": dA, "dB": dB, "db": db}
    if op in ("route", "route_bwd"):
        w, idx = dtc.moe_route(s["logits"], c["k"], bias=s["bias"], scoring=c["scoring"],
                               groups=c["groups"], top_groups=c["top_groups"],
                               renormalize=c["renorm"], scale=1.5)
        if op == "route":
            p = dtc.moe_plan(idx, c["E"])
            return {"w": w, "idx": idx, "offsets": p.offsets, "slots": p.slots}
        dl = dtc.moe_route_backward(s["dw"], s["logits"], idx, scoring=c["scoring"],
                                    renormalize=c["renorm"], scale=1.5)
        return {"w": w, "idx": idx, "dlogits": dl}
    plan = dtc.moe_plan(s["idx"], c["E"])
    if op == "experts":
        return {"y": dtc.moe_experts(c["kind"], s["x"], s["w_in"], s["w_out"], s["w"], plan,
                                     activation=c["act"], residual=s["res"])}
    y, saved = dtc.moe_experts(c["kind"], s["x"], s["w_in"], s["w_out"], s["w"], plan,
                               activation=c["act"], save=True)
    dx, dw_in, dw_out, dw = dtc.moe_experts_backward(c["kind"], s["dy"], s["w_in"], s["w_out"],
                                                     s["w"], plan, saved, activation=c["act"])
    return {"y": y, "dx": dx, "dw_in": dw_in, "dw_out": dw_out, "dw": dw}


# The plain forms: fp32, elementary operations.
def _f(z, name):
    """act(z) of an ungated name."""
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
    return 0.5 * z * (1 + torch.tanh(u))


def _df(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


_GATE = {"swiglu": "silu", "geglu": "gelu"}


def _act(z, name):
    if name in GATED:
        g, u = z.chunk(2, -1)
        return _f(g, _GATE[name]) * u
    return _f(z, name)


def _act_back(dh, z, name):
    if name in GATED:
        g, u = z.chunk(2, -1)
        return torch.cat([dh * u * _df(g, _GATE[name]), dh * _f(g, _GATE[name])], -1)
    return dh * _df(z, name)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "act":
        dt = s["A"].dtype
        a = s["A"].float() if c["layout"][0] == "N" else s["A"].float().t()
        b = s["B"].float().t() if c["layout"][1] == "T" else s["B"].float()
        z = a @ b
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(dt), "z": z.to(dt)} if c["keep"] else {"y": y.to(dt)}
    if op == "act_bwd":
        dt = s["A"].dtype
        a = s["A"].float() if c["layout"][0] == "N" else s["A"].float().t()
        b = s["B"].float().t() if c["layout"][1] == "T" else s["B"].float()
        dz = s["dC"].float()
        if s["z"] is not None:
            dz = _act_back(dz, s["z"].float(), c["act"])
        dA, dB = dz @ b.t(), a.t() @ dz
        return {"dA": (dA if c["layout"][0] == "N" else dA.t()).to(dt).contiguous(),
                "dB": (dB.t() if c["layout"][1] == "T" else dB).to(dt).contiguous(),
                "db": dz.sum(0)}
    if op in ("route", "route_bwd"):
        w, idx = _route(s["logits"], s["bias"], c)
        if op == "route":
            off, slots, _, _ = _places(idx, c["E"])
            return {"w": w, "idx": idx, "offsets": off, "slots": slots}
        return {"w": w, "idx": idx, "dlogits": _route_back(s["dw"], s["logits"], idx, c)}
    return _experts(s)


def _first(keys, k):
    """Values and places of the k largest, in falling order, ties to the lowest place."""
    v, i = torch.sort(keys, dim=-1, descending=True, stable=True)
    return v[..., :k], i[..., :k]


def _route(logits, bias, c):
    z = logits.float()
    T, E = z.shape
    live = z > -math.inf  # false for -inf and NaN
    key = 1 / (1 + torch.exp(-z)) if c["scoring"] == "sigmoid" else z
    if bias is not None:
        key = key + bias
    key = torch.where(live, key, -math.inf)
    if c["groups"] > 1:
        G = c["groups"]
        per = key.reshape(T, G, E // G)
        two = _first(per, 2)[0]
        score = two[..., 0]
        if c["scoring"] == "sigmoid":
            score = score + torch.where(two[..., 1] > -math.inf, two[..., 1], 0)
        _, best = _first(score, c["top_groups"])
        keep = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, best, True)
        key = torch.where(keep[..., None], per, -math.inf).reshape(T, E)
    v, i = _first(key, c["k"])
    got = v > -math.inf
    zi = torch.where(got, torch.gather(z, 1, i), -math.inf)
    if c["scoring"] == "sigmoid":
        w = torch.where(got, 1 / (1 + torch.exp(-zi)), 0)
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, 0)
    elif c["renorm"]:
        e = torch.exp(zi - zi.max(1, keepdim=True).values)
        w = torch.where(got, e / e.sum(1, keepdim=True), 0)
    else:
        zl = torch.where(live, z, -math.inf)
        m = zl.max(1, keepdim=True).values
        w = torch.where(got, torch.exp(zi - m) / torch.exp(zl - m).sum(1, keepdim=True), 0)
    return w * 1.5, torch.where(got, i, -1).to(torch.int32)


def _route_back(dw, logits, idx, c):
    z = logits.float()
    got = idx >= 0
    at = idx.clamp(min=0).long()
    zi = torch.where(got, torch.gather(z, 1, at), -math.inf)
    g = torch.where(got, dw * 1.5, 0)
    dl = torch.zeros_like(z)
    if c["scoring"] == "sigmoid":
        p = torch.where(got, 1 / (1 + torch.exp(-zi)), 0)
        if c["renorm"]:
            total = p.sum(1, keepdim=True)
            mean = torch.where(total > 0, (g * p).sum(1, keepdim=True) / total, 0)
            g = torch.where(total > 0, (g - mean) / total, 0)
        d = g * p * (1 - p)
    elif c["renorm"]:
        e = torch.exp(zi - zi.max(1, keepdim=True).values)
        p = torch.where(got, e / e.sum(1, keepdim=True), 0)
        d = p * (g - (g * p).sum(1, keepdim=True))
    else:
        zl = torch.where(z > -math.inf, z, -math.inf)
        e = torch.exp(zl - zl.max(1, keepdim=True).values)
        pa = torch.where(zl > -math.inf, e / e.sum(1, keepdim=True), 0)
        p = torch.where(got, torch.gather(pa, 1, at), 0)
        dl = -pa * (g * p).sum(1, keepdim=True)
        d = g * p
    return dl.scatter_add(1, at, torch.where(got, d, 0)).to(logits.dtype)


def _places(idx, E):
    """Offsets (multiples of 16) and each choice's row in expert order; also counts and the places
    within an expert."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, E)
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(E + 1, dtype=torch.long, device=idx.device).scatter_add_(
        0, key, torch.ones_like(key))
    start = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(key)
    rank[order] = torch.arange(key.numel(), device=idx.device) - start[key[order]]
    padded = (counts[:E] + ALIGN - 1) // ALIGN * ALIGN
    off = torch.cat([padded.new_zeros(1), torch.cumsum(padded, 0)])
    slots = torch.where(flat >= 0, off[key.clamp(max=E - 1)] + rank, -1)
    return off.to(torch.int32), slots.reshape(idx.shape).to(torch.int32), counts[:E], rank


def _experts(s):
    """Every expert's rows, padded to the fullest expert's count, in one batched product; for no more
    choices than experts, each choice's own weights instead."""
    c = s["case"]
    T, E, k, H = c["T"], c["E"], c["k"], c["H"]
    dt = s["x"].dtype
    idx = s["idx"].long()
    got = idx >= 0
    e = idx.clamp(min=0).reshape(-1)
    w = torch.where(got, s["w"].float(), 0)
    few = T * k <= E
    if few:
        win, wout = s["w_in"][e].float(), s["w_out"][e].float()
        B, cap, place = T * k, 1, torch.arange(T * k, device=e.device)
    else:
        _, _, counts, rank = _places(s["idx"], E)
        win, wout = s["w_in"].float(), s["w_out"].float()
        B, cap = E, max(1, int(counts.max()))
        place = e * cap + rank.clamp(max=cap - 1)
    live = got.reshape(-1, 1)
    rows = torch.arange(T, device=e.device).repeat_interleave(k)

    def spread(t):  # [T k, H] rows to [B, cap, H], zero where no choice goes
        out = torch.zeros((B * cap, t.shape[1]), device=t.device)
        return out.index_add_(0, place, torch.where(live, t, 0)).reshape(B, cap, -1)

    xs = spread(s["x"].float()[rows])
    z = xs @ win.transpose(1, 2)
    h = _act(z, c["act"])
    o = h @ wout.transpose(1, 2)
    each = torch.where(live, o.reshape(B * cap, H)[place], 0).reshape(T, k, H)
    y = (w[..., None] * each).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    if c["op"] == "experts":
        return {"y": y.to(dt)}
    dy = s["dy"].float()
    do = spread((w[..., None] * dy[:, None, :]).reshape(T * k, H))
    dw = torch.where(got, (dy[:, None, :] * each).sum(2), 0)
    dz = _act_back(do @ wout, z, c["act"])
    dxs = (dz @ win).reshape(B * cap, H)[place]
    dx = torch.where(live, dxs, 0).reshape(T, k, H).sum(1)
    dwin, dwout = dz.transpose(1, 2) @ xs, do.transpose(1, 2) @ h
    if few:
        dwin = torch.zeros(s["w_in"].shape, device=e.device).index_add_(0, e, dwin)
        dwout = torch.zeros(s["w_out"].shape, device=e.device).index_add_(0, e, dwout)
    return {"y": y.to(dt), "dx": dx.to(dt), "dw_in": dwin.to(dt), "dw_out": dwout.to(dt),
            "dw": dw.to(dt)}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("act", "act_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        gated = case["act"] in GATED
        Nb = 2 * N if gated else N
        if op == "act":
            b = 2 * (M * K + Nb * K + M * N)
            b += 2 * Nb * case["bias"] + 2 * M * N * case["res"] + 2 * M * Nb * case["keep"]
            return {"bytes": b, "flops": 2 * M * Nb * K}
        b = 2 * (2 * M * K + 2 * Nb * K + M * N + (M * Nb if case["act"] != "none" else 0)) + 4 * Nb
        return {"bytes": b, "flops": 4 * M * Nb * K}
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["logits"] == "f32" else 2
        b = T * E * size + 4 * E * case["bias"] + 8 * T * k
        b += 4 * T * k + 4 * (E + 1) if op == "route" else T * E * size + 4 * T * k
        return {"bytes": b, "flops": T * E * 4}
    T, E, k, H, F = case["T"], case["E"], case["k"], case["H"], case["F"]
    Fz = 2 * F if case["act"] in GATED else F
    touched = E * (1 - (1 - k / E) ** T) if k < E else E  # experts that some token chooses
    weights = 2 * touched * (Fz * H + F * H)
    flops = 2 * T * k * (Fz * H + F * H)
    io = 2 * T * H * (2 + case["res"]) + 6 * T * k
    if op == "experts":
        return {"bytes": weights + io, "flops": flops}
    return {"bytes": weights + 2 * E * (Fz * H + F * H) + io + 4 * T * H + 2 * T * k,
            "flops": 3 * flops}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {n: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for n, v in s.items()}
    if op in ("act", "act_bwd"):
        A = d["A"] if case["layout"][0] == "N" else d["A"].mT
        B = d["B"].mT if case["layout"][1] == "T" else d["B"]
        if op == "act":
            z = torch.matmul(A, B)
            if d["bias"] is not None:
                z += d["bias"]
            y = _x_act(z, case["act"])
            if d["res"] is not None:
                y = y + d["res"]
            return {"y": y, "z": z} if case["keep"] else {"y": y}
        dz = _x_back(d["dC"], d["z"], case["act"])
        dA, dB = torch.matmul(dz, B.mT), torch.matmul(A.mT, dz)
        return {"dA": dA if case["layout"][0] == "N" else dA.mT.contiguous(),
                "dB": dB.mT.contiguous() if case["layout"][1] == "T" else dB, "db": dz.sum(0)}
    if op in ("route", "route_bwd"):
        return _x_route(d, case)
    return _x_experts(d, case)


def _x_sigma(z):
    return torch.special.expit(z)


def _x_pair(z, name):
    """(act(z), act'(z))"""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.relu(), torch.heaviside(z, torch.zeros_like(z))
    if name == "silu":
        p = _x_sigma(z)
        return z * p, p + z * p * _x_sigma(-z)
    if name == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    v = math.sqrt(8 / math.pi) * (z + 0.044715 * z.pow(3))  # 0.5 (1 + tanh(v / 2)) = sigma(v)
    p = _x_sigma(v)
    return z * p, p + z * p * _x_sigma(-v) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z.square())


def _x_act(z, name):
    if name in GATED:
        n = z.shape[-1] // 2
        return _x_pair(z[..., :n], _GATE[name])[0] * z[..., n:]
    return _x_pair(z, name)[0]


def _x_back(dy, z, name):
    if name == "none":
        return dy
    if name in GATED:
        n = z.shape[-1] // 2
        f, df = _x_pair(z[..., :n], _GATE[name])
        return torch.cat([dy * z[..., n:] * df, dy * f], -1)
    return dy * _x_pair(z, name)[1]


def _x_route(d, c):
    """In numpy, token by token where groups or masks need it. None for the choices (whole numbers)."""
    import numpy as np
    z = d["logits"].cpu().numpy()
    T, E = z.shape
    k = c["k"]
    dead = ~(z > -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        key = 1 / (1 + np.exp(-z)) if c["scoring"] == "sigmoid" else z.copy()
    if d["bias"] is not None:
        key = key + d["bias"].cpu().numpy()
    key[dead] = -np.inf
    if c["groups"] > 1:
        per = key.reshape(T, c["groups"], -1)
        top = -np.sort(-per, axis=2)
        score = top[..., 0].copy()
        if c["scoring"] == "sigmoid":
            score += np.where(np.isfinite(top[..., 1]), top[..., 1], 0)
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where((rank < c["top_groups"])[..., None], per, -np.inf).reshape(T, E)
    i = np.argsort(-key, axis=1, kind="stable")[:, :k]
    got = np.take_along_axis(key, i, 1) > -np.inf
    chosen = np.zeros((T, E), bool)
    np.put_along_axis(chosen, i, got, 1)
    with np.errstate(all="ignore"):
        if c["scoring"] == "sigmoid":
            p = np.where(dead, 0.0, 1 / (1 + np.exp(-z)))
            inside = chosen
        else:
            inside = chosen if c["renorm"] else ~dead
            zz = np.where(inside, z, -np.inf)
            p = np.exp(zz - zz.max(1, keepdims=True))
            p = np.where(inside, p / p.sum(1, keepdims=True), 0.0)
        full = np.where(chosen, p, 0.0)
        total = np.ones((T, 1))
        if c["scoring"] == "sigmoid" and c["renorm"]:
            total = full.sum(1, keepdims=True)
            full = np.where(total > 0, full / total, 0.0)
    w = np.where(got, np.take_along_axis(full, i, 1), 0.0) * 1.5
    if c["op"] == "route":
        return {"w": torch.from_numpy(w), "idx": None, "offsets": None, "slots": None}
    g = np.zeros((T, E))
    np.put_along_axis(g, i, np.where(got, d["dw"].cpu().numpy() * 1.5, 0.0), 1)
    g = np.where(chosen, g, 0.0)
    if c["scoring"] == "sigmoid":
        if c["renorm"]:
            with np.errstate(all="ignore"):
                g = np.where(chosen & (total > 0), (g - (g * full).sum(1, keepdims=True)) / total, 0.0)
        dl = g * p * (1 - p)
    else:
        dl = p * (g - (g * p).sum(1, keepdims=True))
    return {"w": torch.from_numpy(w), "idx": None, "dlogits": torch.from_numpy(dl)}


def _x_experts(d, c):
    """Expert by expert."""
    T, E, k, H, F = (c[n] for n in ("T", "E", "k", "H", "F"))
    train = c["op"] == "experts_train"
    idx, w, x = d["idx"].long(), d["w"], d["x"]
    y = torch.zeros_like(x) if d["res"] is None else d["res"].clone()
    if train:
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        dwi, dwo = torch.zeros_like(d["w_in"]), torch.zeros_like(d["w_out"])
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        z = x[t] @ d["w_in"][e].mT
        h = _x_act(z, c["act"])
        o = h @ d["w_out"][e].mT
        y.index_add_(0, t, w[t, j, None] * o)
        if train:
            dy = d["dy"][t]
            dw[t, j] = (dy * o).sum(1)
            do = w[t, j, None] * dy
            dwo[e] = do.mT @ h
            dz = _x_back(do @ d["w_out"][e], z, c["act"])
            dwi[e] = dz.mT @ x[t]
            dx.index_add_(0, t, dz @ d["w_in"][e])
    if not train:
        return {"y": y}
    return {"y": y, "dx": dx, "dw_in": dwi, "dw_out": dwo, "dw": dw}
