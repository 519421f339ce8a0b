"""Plain 64-bit references of the 4-bit operators. Nothing here uses the library.

Codes, scales and factors are whole numbers of few bits, so their products are exact in 64 bits; a value
goes to the nearest of a table of code values, a tie to the even code, by comparison with the midpoints
(also exact). What the product's result may be off by: the sum of K exact products, accumulated in fp32
with truncation at worst, (K + 2) 2^-23 of the products' sizes; two roundings for the factors; then the
epilogue's bounds of ffn_ref."""
import torch

import ffn_ref as R

BLOCK = {"nvfp4": 16, "mxfp4": 32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127]


def nearest(v, table):
    """Index of the nearest table value (ties: the even index) of v >= 0."""
    t = torch.tensor(table, dtype=torch.float64, device=v.device)
    mid = (t[1:] + t[:-1]) / 2
    v = v.contiguous()
    below, upto = torch.searchsorted(mid, v), torch.searchsorted(mid, v, right=True)
    return torch.where(below % 2 == 0, below, upto)


def exponent(v):
    """floor(log2 v) of v > 0, by frexp."""
    return torch.frexp(v)[1] - 1


def pow2(e):
    return torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e.cpu().int()).to(e.device)


def quantize(x, fmt):
    """(codes one to a byte, scale bytes, factors or None) of [..., K]."""
    x = x.double()
    b = x.unflatten(-1, (-1, BLOCK[fmt]))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], 0.0, b)
    top = b.abs().amax(-1)
    if fmt == "nvfp4":
        row = top.amax(-1)
        e = exponent(torch.where(row > 0, row, 1.0) / 2688)
        e = torch.where(2688 * pow2(e) < row, e + 1, e).clamp(min=-100)
        e = torch.where(row > 0, e, 0)
        g = pow2(e)
        code = nearest(top / g[..., None] / 6, E4M3)  # (a tie is 6 x (8 + m + 1/2) 2^j: below 8 bits, exact)
        s = torch.tensor(E4M3, dtype=torch.float64, device=x.device)[code] * g[..., None]
        scales, factors = torch.where(bad, 0x7F, code), g.float()
    else:
        e = torch.where(top > 0, (exponent(torch.where(top > 0, top, 1.0)) - 2).clamp(min=-126), 0)
        s = pow2(e)
        scales, factors = torch.where(bad, 0xFF, e + 127), None
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    # |x| against the midpoints times the scale (exact: at most 11 + 7 bits)
    q = torch.zeros(b.shape, dtype=torch.uint8, device=x.device)
    for i, m in enumerate(mid):
        edge = m * s[..., None]
        q += ((b.abs() > edge) | ((b.abs() == edge) & (i % 2 == 1))).byte()
    q = torch.where(s[..., None] > 0, q, 0)
    sign = torch.where(bad[..., None], False, torch.signbit(x.unflatten(-1, (-1, BLOCK[fmt]))))
    return (q | (sign.byte() << 3)).flatten(-2), scales.to(torch.uint8), factors


def values(codes, scales, factors, fmt):
    """The 64-bit values of codes one to a byte."""
    t = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    v = t[codes.long()].unflatten(-1, (-1, BLOCK[fmt]))
    if fmt == "nvfp4":
        s = torch.tensor(E4M3 + [float("nan")] + [float("nan")] * 128, dtype=torch.float64,
                         device=codes.device)[scales.long()]
        if factors is not None:
            s = s * factors.double()[..., None]
    else:
        s = torch.where(scales == 255, float("nan"), pow2(scales.int() - 127))
    return (v * s[..., None]).flatten(-2)


def rounded(x, fmt):
    return values(*quantize(x, fmt), fmt)


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).contiguous()


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def chunks(scales, fmt, gated=False):
    """Row-major scale bytes [..., rows, blocks] in the storage order of include/dtc_fp4.h, place by place."""
    s = scales.cpu()
    s = s if s.dim() == 3 else s[None]
    E, rows, blocks = s.shape
    sets = (blocks + 3) // 4
    F = rows // 2
    groups = (F + 63) // 64 if gated else (rows + 127) // 128
    out = torch.zeros((E, groups, sets, 32, 4, 4), dtype=torch.uint8)
    for g in range(groups):
        for p in range(128):
            if gated:
                f = 64 * g + 8 * (p // 16) + p % 8
                r = f + F * (p % 16 // 8) if f < F else rows
            else:
                r = 128 * g + p
            if r < rows:
                row = torch.zeros((E, 4 * sets), dtype=torch.uint8)
                row[:, :blocks] = s[:, r]
                out[:, g, :, p % 32, p // 32] = row.reshape(E, sets, 4)
    return out.flatten()


def product(kind, a, b, bias, residual, act):
    """(y, bound) of a product of 64-bit values a [M,K], b [N,K]."""
    z, s = a @ b.t(), a.abs() @ b.abs().t()
    ez = ((a.shape[1] + 2) * 2.0 ** -23 + 2.0 ** -22) * s
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -23 * z.abs()
    y, ey = R.act(z, act), R.act_bound(z, ez, act)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -23 * y.abs()
    u = R.U[kind]
    return y, ey * (1 + u) + u * y.abs() + R.TINY[kind]


# Significand bits and lowest exponent of a normal number.
FLOAT = {torch.float32: (24, -126), torch.bfloat16: (8, -126), torch.float16: (11, -14)}


def nearest_float(v, dtype):
    """The number of a float type nearest to a 64-bit one, a tie to even, in one rounding (a conversion by torch
    goes through fp32)."""
    bits, low = FLOAT[dtype]
    v = v.cpu()
    e = torch.where(v != 0, torch.frexp(v)[1] - 1, low).clamp(min=low, max=127)
    step = pow2(e - bits + 1)  # (a normal number of 64 bits, so that dividing by it is exact)
    r = torch.round(v / step) * step
    return torch.where(r.abs() > torch.finfo(dtype).max, torch.copysign(torch.tensor(float("inf")).double(), v), r)
