"""4-bit operators beside the dense and the routed products: what is measured.

* ``quant``: microscaled 4-bit quantisation of rows, and the values that the result stands for.
* ``linear``: a product of 4-bit operands with bias, activation (plain or gated) and residual in its
  epilogue; its rows come in 4 bits already (``ready``) or in 16 and are quantised in the call.
* ``experts``: routed experts whose weights are held in 4 bits: rows quantised, two products over the
  experts' ragged rows with a quantisation between them, the weighted join.

Formats (row by row, e2m1 elements, ties to even, e2m1's largest value 6 where they go past it):

* nvfp4: a factor g = 2^e per row, e the lowest with max|row| <= 6 * 448 * g (0 for a row of zeros, -100
  at least); a UE4M3 scale s per 16 elements, max|block| / (6 g) rounded; elements x / (s g) rounded (0
  where s is 0).
* mxfp4: an E8M0 scale 2^(floor(log2 max|block|) - 2) per 32 elements (1 for a block of zeros, 2^-126 at
  least), elements x / scale rounded.

`run` computes a case with elementary torch operations in 32 bits, or, where `own` is true, with the
calls of dense_tensor_core_gb300. `exact` computes it from the definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
GATED = ("swiglu", "geglu")
BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # the row of one new token, as wide as the benchmark's layers: latency
        dict(name="quant_token", op="quant", fmt="nvfp4", kind="bf16", M=1, K=8192),
        # a ragged batch, rows that end inside the tiles
        dict(name="quant_odd", op="quant", fmt="mxfp4", kind="f16", M=1111, K=2080),
        # the weights of an 8192 x 8192 layer
        dict(name="quant_large", op="quant", fmt="nvfp4", kind="bf16", M=8192, K=8192),
        # the smallest product of the tests and the smoke run, quantisation included: latency
        dict(name="linear_small", op="linear", fmt="mxfp4", kind="bf16", M=256, N=256, K=512, act="gelu",
             bias=True, res=True, ready=False),
        # one new token through an 8192 x 8192 layer: serving
        dict(name="linear_token", op="linear", fmt="nvfp4", kind="bf16", M=1, N=8192, K=8192, act="none",
             bias=True, res=True, ready=False),
        # a ragged batch through a gated layer: odd M, N and K off every tile size
        dict(name="linear_odd", op="linear", fmt="nvfp4", kind="f16", M=1111, N=2056, K=2080, act="swiglu",
             bias=True, res=False, ready=False),
        # the headline product in 4 bits, with an epilogue
        dict(name="linear_large", op="linear", fmt="nvfp4", kind="bf16", M=4096, N=4096, K=8192,
             act="gelu_tanh", bias=True, res=True, ready=True),
        # the same sizes as a user has them from a 16-bit layer before, the other format
        dict(name="linear_large_mx", op="linear", fmt="mxfp4", kind="f16", M=4096, N=4096, K=8192,
             act="none", bias=False, res=False, ready=False),
        # one new token through its experts: serving
        dict(name="experts_token", op="experts", fmt="nvfp4", kind="bf16", T=1, E=64, k=8, H=2048, F=1024,
             act="swiglu", res=True),
        # a few sequences' new tokens, an odd inner size, the other format
        dict(name="experts_odd", op="experts", fmt="mxfp4", kind="f16", T=77, E=48, k=6, H=2048, F=992,
             act="silu", res=False),
        # a prompt through its experts
        dict(name="experts_prompt", op="experts", fmt="nvfp4", kind="bf16", T=4096, E=64, k=8, H=2048,
             F=1024, act="swiglu", res=True),
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(round(v / mult)) * mult)


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        held = c["E"] * c["H"] * c["F"] * (3 if c["act"] in GATED else 2) if c["op"] == "experts" else 0
        if w["flops"] <= 4.2e11 and w["bytes"] <= 2.9e8 and held <= 4.1e8:
            return c


def _draw(rng):
    op = rng.choice(["quant", "linear", "linear", "linear", "experts", "experts"])
    c = dict(op=op, fmt=rng.choice(["nvfp4", "nvfp4", "mxfp4"]), kind=rng.choice(["bf16", "f16"]))
    if op == "quant":
        return dict(c, M=_log(rng, 1, 8192), K=_log(rng, 64, 16384, 32))
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "geglu"])
    if op == "linear":
        return dict(c, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192, 8), K=_log(rng, 64, 8192, 32), act=act,
                    bias=rng.random() < 0.7, res=rng.random() < 0.5, ready=rng.random() < 0.4)
    return dict(c, T=_log(rng, 1, 8192), E=rng.choice([8, 16, 20, 32, 60, 64, 96, 128, 160, 256]),
                k=rng.randint(1, 8), H=_log(rng, 128, 4096, 32), F=_log(rng, 64, 2048, 32), act=act,
                res=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _rows(g, M, K, dtype):
    """Activations: rows of unlike size, a few columns much larger than the rest, one row in 50 zero
    (padding)."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x *= torch.exp(torch.randn((M, 1), generator=g, device="cuda") * 0.5)
    x *= 1 + 20 * (torch.rand((1, K), generator=g, device="cuda") < 0.004)
    if M > 1:
        x.masked_fill_(torch.rand((M, 1), generator=g, device="cuda") < 0.02, 0)
    return x.to(dtype)


def _routes(g, T, E, k, dtype):
    """Choices of a router with experts of uneven popularity and one token in 50 without an expert."""
    z = torch.randn((T, E), generator=g, device="cuda") * 1.5
    z += torch.randn((1, E), generator=g, device="cuda") * 0.5
    if T > 1:
        z.masked_fill_(torch.rand((T, 1), generator=g, device="cuda") < 0.02, -math.inf)
    v, i = torch.topk(z, k, dim=1)
    idx = torch.where(torch.isinf(v), -1, i).to(torch.int32)
    return idx, torch.nan_to_num(torch.softmax(v, 1))


def _held(w, fmt, gated=False):
    """Weights (or rows) as a program holds them: codes, scales and factors, row by row, and the
    framework's own layout of the same where it is asked for."""
    codes, scales, g = _quantize(w, fmt)
    packed = (codes[..., 0::2] | codes[..., 1::2] << 4).contiguous()
    held = dict(codes=packed, scales=scales, g=g, fmt=fmt)
    if own:
        import dense_tensor_core_gb300 as dtc
        held["q"] = dtc.pack_fp4(packed, scales, g, format=fmt, gated=gated)
    return held


def prepare(case, seed):
    g = _gen(seed)
    op, fmt, dt = case["op"], case["fmt"], DT[case["kind"]]
    s = dict(case=case)
    if op == "quant":
        s["x"] = _rows(g, case["M"], case["K"], dt)
        return s
    gated = case["act"] in GATED
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        Nb = 2 * N if gated else N
        x = _rows(g, M, K, dt)
        s["x"] = _held(x, fmt) if case["ready"] else x
        s["w"] = _held(_normal(g, (Nb, K), K ** -0.5, dt), fmt, gated)
        s["bias"] = _normal(g, (Nb,), 0.2, dt) if case["bias"] else None
        s["res"] = _normal(g, (M, N), 1.0, dt) if case["res"] else None
        if own:
            import dense_tensor_core_gb300 as dtc
            n = dtc.gemm_fp4_workspace_size(M, N, K, activation=case["act"])
            s["ws"] = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
        return s
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    s["x"] = _rows(g, T, H, dt)
    s["w_in"] = _held(_normal(g, (E, 2 * F if gated else F, H), H ** -0.5, dt), fmt, gated)
    s["w_out"] = _held(_normal(g, (E, H, F), F ** -0.5, dt), fmt)
    s["idx"], s["w"] = _routes(g, T, E, k, dt)
    s["res"] = _normal(g, (T, H), 1.0, dt) if case["res"] else None
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_tensor_core_gb300 as dtc
    c = s["case"]
    if c["op"] == "quant":
        return {"values": dtc.dequantize_fp4(dtc.quantize_fp4(s["x"], format=c["fmt"]))}
    if c["op"] == "linear":
        x = s["x"]["q"] if c["ready"] else dtc.quantize_fp4(s["x"], format=c["fmt"])
        return {"y": dtc.gemm_fp4(c["kind"], x, s["w"]["q"], bias=s["bias"], residual=s["res"],
                                  activation=c["act"], workspace=s["ws"])}
    plan = dtc.moe_plan(s["idx"], c["E"])
    return {"y": dtc.moe_experts_fp4(c["kind"], s["x"], s["w_in"]["q"], s["w_out"]["q"], s["w"], plan,
                                     activation=c["act"], residual=s["res"])}


# The plain forms: fp32, elementary operations.
def _pow2(e):
    """2^e in fp32 for whole numbers e in -126 .. 127, by its bits (powers and divisions by a number
    are not rounded correctly everywhere)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantize(x, fmt):
    """(codes, scales, row factors) of rows: 4-bit codes one to a byte, scale codes, fp32 or None."""
    x = x.float()
    b = x.unflatten(-1, (-1, BLOCK[fmt]))
    top = b.abs().amax(-1)
    if fmt == "nvfp4":
        m, e = torch.frexp(top.amax(-1))  # m in [0.5, 1); 6 * 448 = 0.65625 * 2^12
        e = torch.where(m > 0.65625, e - 11, e - 12).clamp(min=-100)
        g = _pow2(torch.where(m > 0, e, 0))
        s8 = (top / (6 * g[..., None])).to(torch.float8_e4m3fn)
        s, scales = s8.float() * g[..., None], s8.view(torch.uint8)
    else:
        m, e = torch.frexp(top)  # floor(log2 top) = e - 1
        e = torch.where(m > 0, (e - 3).clamp(-126, 127), 0)
        g, scales = None, (e + 127).to(torch.uint8)
        s = _pow2(e)
    t = torch.where(s[..., None] > 0, b / s[..., None], 0)
    a = t.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte())
    return (code | (b.signbit().byte() << 3)).flatten(-2), scales, g


def _decode(codes, scales, g, fmt):
    """The fp32 values of codes one to a byte."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    v = table[codes.int()].unflatten(-1, (-1, BLOCK[fmt]))
    if fmt == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).float() * g[..., None]
    else:
        s = _pow2(scales.int() - 127)
    return (v * s[..., None]).flatten(-2)


def _values(held, at=None):
    """The fp32 values of held weights; `at`: of these matrices only."""
    c, s, g = (held[n] if at is None or held[n] is None else held[n][at] for n in ("codes", "scales", "g"))
    return _decode(torch.stack([c & 15, c >> 4], -1).flatten(-2), s, g, held["fmt"])


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


_GATE = {"swiglu": "silu", "geglu": "gelu"}


def _act(z, name):
    if name in GATED:
        g, u = z.chunk(2, -1)
        return _f(g, _GATE[name]) * u
    return _f(z, name)


def _plain(s):
    c = s["case"]
    if c["op"] == "quant":
        return {"values": _decode(*_quantize(s["x"], c["fmt"]), c["fmt"]).to(torch.bfloat16)}
    if c["op"] == "linear":
        x = _values(s["x"]) if c["ready"] else _decode(*_quantize(s["x"], c["fmt"]), c["fmt"])
        z = x @ _values(s["w"]).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(DT[c["kind"]])}
    return _experts(s)


def _experts(s):
    """Every expert's rows, padded to the fullest expert's count, in one batched product; for no more
    choices than experts, each choice's own weights instead. The activation is rounded to 16 bits before
    it is quantised, as the operator has it."""
    c = s["case"]
    T, E, k, H, dt = c["T"], c["E"], c["k"], c["H"], DT[c["kind"]]
    flat = s["idx"].reshape(-1).long()
    live = (flat >= 0)[:, None]
    e = flat.clamp(min=0)
    xq = _decode(*_quantize(s["x"], c["fmt"]), c["fmt"])
    rows = xq[torch.arange(T, device=e.device).repeat_interleave(k)]
    if T * k <= E:
        win, wout = _values(s["w_in"], e), _values(s["w_out"], e)
        xs, place = rows[:, None, :], torch.arange(T * k, device=e.device)
    else:
        win, wout = _values(s["w_in"]), _values(s["w_out"])
        key = torch.where(live[:, 0], flat, E)
        order = torch.sort(key, stable=True)[1]
        counts = torch.zeros(E + 1, dtype=torch.long, device=e.device).scatter_add_(
            0, key, torch.ones_like(key))
        start = torch.cumsum(counts, 0) - counts
        rank = torch.empty_like(key)
        rank[order] = torch.arange(T * k, device=e.device) - start[key[order]]
        cap = max(1, int(counts[:E].max()))
        place = e * cap + rank.clamp(max=cap - 1)
        xs = torch.zeros((E * cap, H), device=e.device)
        xs = xs.index_add_(0, place, torch.where(live, rows, 0)).reshape(E, cap, H)
    h = _act(xs @ win.transpose(1, 2), c["act"]).to(dt)
    o = _decode(*_quantize(h, c["fmt"]), c["fmt"]) @ wout.transpose(1, 2)
    each = torch.where(live, o.reshape(-1, H)[place], 0).reshape(T, k, H)
    y = (s["w"][..., None] * each).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(dt)}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def _size(fmt, rows, K):
    """Bytes of rows held in 4 bits."""
    return rows * K / 2 + rows * K / BLOCK[fmt] + (4 * rows if fmt == "nvfp4" else 0)


def work(case):
    fmt = case["fmt"]
    if case["op"] == "quant":  # 16-bit values in, 16-bit values out, and the 4-bit form written and read
        M, K = case["M"], case["K"]
        return {"bytes": 4 * M * K + 2 * _size(fmt, M, K), "flops": 2 * M * K}
    Fz = 2 if case["act"] in GATED else 1
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        b = _size(fmt, M, K) if case["ready"] else 2 * M * K
        b += _size(fmt, Fz * N, K) + 2 * M * N * (1 + case["res"]) + 2 * Fz * N * case["bias"]
        return {"bytes": b, "flops": 2 * M * Fz * N * K}
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    touched = E * (1 - (1 - k / E) ** T) if k < E else E  # experts that some token chooses
    b = touched * (_size(fmt, Fz * F, H) + _size(fmt, H, F)) + 2 * T * H * (2 + case["res"]) + 8 * T * k
    return {"bytes": b, "flops": 2 * T * k * (Fz + 1) * F * H}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E4M3 = [(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127]


def _nearest(v, table):
    """Places in a rising table of the values nearest to v; of two as near, the even one."""
    t = torch.tensor(table, dtype=torch.float64, device=v.device)
    mid = (t[1:] + t[:-1]) / 2
    i, j = torch.searchsorted(mid, v), torch.searchsorted(mid, v, right=True)
    return torch.where(i % 2 == 0, i, j), t


def _x_pow2(e):
    """2^e for whole numbers e in -140 .. 140."""
    return torch.tensor([2.0 ** n for n in range(-140, 141)], dtype=torch.float64, device=e.device)[e.long() + 140]


def _x_round(x, fmt):
    """What the quantised rows stand for."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK[fmt])
    top = b.abs().max(-1).values
    if fmt == "nvfp4":
        row = top.max(-1, keepdim=True).values
        e = torch.ceil(torch.log2(row / 2688) - 1e-9).clamp(min=-100)
        g = _x_pow2(torch.where(row > 0, e, 0))
        i, t = _nearest((top / (6 * g)).contiguous(), _E4M3)
        s = t[i] * g
    else:
        e = (torch.floor(torch.log2(top) + 1e-9) - 2).clamp(-126, 127)
        s = _x_pow2(torch.where(top > 0, e, 0))
    s = s[..., None]
    q = (b.abs() / torch.where(s > 0, s, 1.0)).contiguous()
    i, t = _nearest(q, _E2M1)
    return torch.where(s > 0, t[i] * s * torch.sign(b), 0.0).reshape(x.shape)


def _x_values(held):
    """The values of held weights."""
    c = held["codes"].long()
    c = torch.stack([c % 16, c // 16], -1).reshape(*c.shape[:-1], -1)
    v = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=c.device)[c]
    v = v.reshape(*c.shape[:-1], -1, BLOCK[held["fmt"]])
    sc = held["scales"].long()
    if held["fmt"] == "nvfp4":
        s = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=c.device)[sc]
        s = s * held["g"].double()[..., None]
    else:
        s = _x_pow2(sc - 127)
    return (v * s[..., None]).reshape(c.shape)


def _x_act(z, name):
    if name in GATED:
        n = z.shape[-1] // 2
        return _x_act(z[..., :n], _GATE[name]) * z[..., n:]
    if name == "none":
        return z
    if name == "relu":
        return z.relu()
    if name == "silu":
        return z * torch.special.expit(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.special.expit(math.sqrt(8 / math.pi) * (z + 0.044715 * z.pow(3)))


def exact(case, seed):
    s = prepare(case, seed)
    fmt = case["fmt"]
    if case["op"] == "quant":
        return {"values": _x_round(s["x"].double(), fmt)}
    res = None if s["res"] is None else s["res"].double()
    if case["op"] == "linear":
        x = _x_values(s["x"]) if case["ready"] else _x_round(s["x"].double(), fmt)
        z = torch.matmul(x, _x_values(s["w"]).mT)
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _x_act(z, case["act"])
        return {"y": y if res is None else y + res}
    x, w, idx = _x_round(s["x"].double(), fmt), s["w"].double(), s["idx"].long()
    y = torch.zeros_like(x) if res is None else res
    for e in range(case["E"]):  # expert by expert
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            part = {n: {m: v[e] if torch.is_tensor(v) else v for m, v in s[n].items() if m != "q"}
                    for n in ("w_in", "w_out")}
            h = _x_act(x[t] @ _x_values(part["w_in"]).mT, case["act"]).to(DT[case["kind"]]).double()
            y.index_add_(0, t, w[t, j, None] * (_x_round(h, fmt) @ _x_values(part["w_out"]).mT))
    return {"y": y}
