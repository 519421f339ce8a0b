"""The size limits of a matrix in 4 bits, as include/dtc_fp4.h states them, at their borders. No GPU."""
import ctypes

import pytest

LIMIT = 2 ** 31 - 1 - 256


@pytest.fixture(scope="module")
def layout():
    from dense_tensor_core_gb300 import _fp4, build

    build.build()
    L = _fp4._L()

    def call(fmt, gated, matrices, rows, K):
        i = _fp4.fp4_info()
        q = _fp4.fp4_matrix(fmt, gated, matrices, rows, K, None, None, None)
        return L.fp4_layout(ctypes.byref(q), ctypes.byref(i)) == 0, i

    return call


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("matrices", [1, 7])
@pytest.mark.parametrize("K", [32, 4096, 65568, 1 << 24])
def test_scale_chunks(layout, fmt, gated, matrices, K):
    """Four times the chunks may be up to the limit, which rows of long K meet before their number does."""
    sets = -(-K // (128 if fmt else 64))
    groups = min(LIMIT // (4 * sets * matrices), LIMIT // matrices // 128)  # of 128 rows each
    ok, i = layout(fmt, gated, matrices, groups * 128, K)
    assert ok and i.groups == groups and i.sets == sets
    assert i.scale_bytes == matrices * groups * sets * 512
    assert i.code_bytes == matrices * groups * 128 * (K // 2)
    more = (groups + 1) * 128
    assert (4 * (groups + 1) * sets * matrices > LIMIT) or (matrices * more > LIMIT)
    assert not layout(fmt, gated, matrices, more, K)[0]


def test_rows(layout):
    assert layout(0, 0, 1, LIMIT, 32)[0] and not layout(0, 0, 1, LIMIT + 1, 32)[0]
    assert not layout(0, 0, 2, LIMIT // 2 + 1, 32)[0]
