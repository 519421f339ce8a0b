"""dequantize_fp4 of matrices whose factors are any fp32 numbers: code x scale x factor, rounded once."""
import pytest
import torch

import fp4_ref as Q

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def every_code_and_scale(fmt, rows):
    """Rows that hold every code beside every scale."""
    n, count = Q.BLOCK[fmt], 128 if fmt == "nvfp4" else 256
    scales = torch.arange(count, dtype=torch.uint8).clamp(max=count - 2)  # (the last is the NaN)
    codes = torch.arange(16, dtype=torch.uint8).repeat(count * n // 16)
    return codes.expand(rows, -1).contiguous().cuda(), scales.expand(rows, -1).contiguous().cuda()


def ordinary(rows):
    g = torch.Generator().manual_seed(7)
    f = (torch.rand(rows, generator=g) + 0.5) * torch.exp2(torch.randint(-20, 20, (rows,), generator=g).float())
    f[::3] *= -1
    return f


def at_the_ends():
    """Powers of two over fp32's range, its largest and smallest numbers, and ordinary significands beside the ends."""
    e = torch.cat([torch.arange(-149, 128, 6), torch.tensor([117, 118, 119, 120, 125, 126, 127])])
    p = torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e.int())
    odd = p * (1 + 0.7318255901336670 * (e > -126))  # (24 bits at most where the number is normal)
    return torch.cat([p, odd.clamp(max=3.4e38), torch.tensor([3.4028234663852886e38, 3 * 2.0 ** -149, 5 * 2.0 ** -140, 0.0])]).float()


def beside_ties():
    """Factors whose product with a value of 6 significant bits (45 = 3 x 15) or 2 (3) lies beside the middle of two
    neighbours of a 16-bit type, nearer than half a step of fp32: rounded to fp32 first it is that middle."""
    g = torch.Generator().manual_seed(3)
    out = []
    for p in (8, 11):
        for m, bits in ((45, 30), (3, 26)):
            n = torch.randint(2 ** (p - 1), 2 ** p, (400,), generator=g, dtype=torch.int64)
            t = (2 * n + 1) * 2 ** (bits - p - 1)
            for G in (t // m, t // m + 1):
                out.append(G[(G >= 2 ** 23) & (G < 2 ** 24)])
    f = torch.cat(out).double() * 2.0 ** -24
    return (f * torch.where(torch.arange(f.numel()) % 2 == 0, 1, -1)).float()


@pytest.mark.parametrize("factors", [ordinary, at_the_ends, beside_ties])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_any_factor_is_rounded_once(fmt, dtype, factors):
    import dense_tensor_core_gb300 as dtc
    f = factors(64).cuda() if factors is ordinary else factors().cuda()
    codes, scales = every_code_and_scale(fmt, f.numel())
    got = dtc.dequantize_fp4(dtc.pack_fp4(Q.pack(codes), scales, f, format=fmt), dtype=dtype).double().cpu()
    # (the definition: exact in 64 bits, 2 + 4 + 24 bits)
    want = Q.nearest_float(Q.values(codes, scales, None, fmt) * f.double()[:, None], dtype)
    bad = got != want
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_no_factors(fmt, dtype):
    import dense_tensor_core_gb300 as dtc
    codes, scales = every_code_and_scale(fmt, 3)
    got = dtc.dequantize_fp4(dtc.pack_fp4(Q.pack(codes), scales, None, format=fmt), dtype=dtype).double().cpu()
    assert torch.equal(got, Q.nearest_float(Q.values(codes, scales, None, fmt), dtype))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_zero_codes_beside_large_factors_are_zero(fmt):
    import dense_tensor_core_gb300 as dtc
    codes = torch.zeros((3, 64), dtype=torch.uint8, device="cuda")
    codes[:, 33] = 1
    scales = torch.full((3, 64 // Q.BLOCK[fmt]), 0x7E if fmt == "nvfp4" else 254, dtype=torch.uint8, device="cuda")
    f = torch.tensor([2.0 ** 120, 2.0 ** -30, -3e38], device="cuda")
    v = dtc.dequantize_fp4(dtc.pack_fp4(Q.pack(codes), scales, f, format=fmt), dtype=torch.float32)
    s = 448.0 if fmt == "nvfp4" else 2.0 ** 127
    want = [min(0.5 * s * float(x), float("inf")) if abs(0.5 * s * float(x)) < 3.5e38 else float("inf") * (1 if x > 0 else -1)
            for x in f.double()]
    assert v[:, 33].tolist() == want
    v[:, 33] = 0
    assert not v.any()  # (a NaN counts as true)
