"""The single rounding that dequantize_fp4 is held to, against numpy's and against neighbours."""
import numpy as np
import torch

import fp4_ref as Q


def test_nearest_float_of_fp16_and_fp32_is_numpys():
    g = torch.Generator().manual_seed(1)
    v = torch.randn(20000, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-30, 18, (20000,), generator=g).double())
    v = torch.cat([v, torch.tensor([0.0, 65504.0, 65519.99, 65520.0, -65520.0, 2.0 ** -25, 3 * 2.0 ** -25, 2.0 ** -24])])
    with np.errstate(over="ignore"):
        assert np.array_equal(Q.nearest_float(v, torch.float16).numpy(), v.numpy().astype(np.float16).astype(np.float64))
        w = v * 2.0 ** 120
        for x in (v, w, v * 2.0 ** -140):
            assert np.array_equal(Q.nearest_float(x, torch.float32).numpy(), x.numpy().astype(np.float32).astype(np.float64))


def test_nearest_float_of_bf16():
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    table = (bits << 16).view(torch.float32).double()  # every number from 0 up
    assert torch.equal(Q.nearest_float(table, torch.bfloat16), table)
    mid = (table[1:] + table[:-1]) / 2
    lower_is_even = bits[:-1] % 2 == 0
    assert torch.equal(Q.nearest_float(mid, torch.bfloat16), torch.where(lower_is_even, table[:-1], table[1:]))
    tiny = mid * 2.0 ** -40  # far below a step of fp32
    assert torch.equal(Q.nearest_float(mid + tiny, torch.bfloat16), table[1:])
    assert torch.equal(Q.nearest_float(tiny - mid, torch.bfloat16), -table[:-1])
    top = float(table[-1])
    assert Q.nearest_float(torch.tensor([top * (1 + 2.0 ** -9), -top * 2], dtype=torch.float64), torch.bfloat16).tolist() == [
        top, -float("inf")]
