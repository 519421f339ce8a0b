"""One workspace through calls of different sizes, pitches and alignments: what a call leaves behind
must not reach a later call that lays the workspace out in another way."""
import pytest
import torch

import ffn_ref as R
from test_gemm_act_gpu import operands, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_tensor_core_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def forward(ws, kind, M, N, K, name="none", layout="NT", shift=0):
    """A call into a C of NaNs, checked against the reference. shift: elements by which A's rows are
    moved off the 128-byte lines."""
    import dense_tensor_core_gb300 as dtc
    A, B, _ = operands(kind, layout, M, N, K, name)
    if shift:
        flat = torch.zeros(A.numel() + shift, dtype=A.dtype, device="cuda")
        flat[shift:] = A.reshape(-1)
        A = flat[shift:].view(A.shape)
    C = torch.full((M, N), float("nan"), dtype=A.dtype, device="cuda")
    y, ey, _, _ = R.gemm_act(kind, A, B, layout, None, None, name)
    dtc.gemm_act(kind, A, B, C, layout=layout, activation=name, workspace=ws)
    dtc.gemm_stream_status()
    R.check(C, y, ey, f"{M} x {N} x {K} {name} {layout}")


def size(kind, M, N, K, name="none", layout="NT"):
    import dense_tensor_core_gb300 as dtc
    return dtc.gemm_act_workspace_size(kind, M, N, K, layout=layout, activation=name)


# sizes that split few tiles before sizes that split many, and back
CALLS = [(32, 1024, 4096, "none"), (32, 4096, 4096, "none"), (64, 512, 2048, "silu"), (64, 4096, 4096, "gelu"),
         (33, 512, 4096, "swiglu"), (200, 2048, 4096, "geglu"), (32, 1024, 4096, "relu")]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_sizes_in_turn(kind):
    need = [size(kind, *c) for c in CALLS]
    assert all(n > 0 for n in need)  # all of them split K
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    for c in CALLS + CALLS[::-1]:
        forward(ws, kind, *c)


def test_layouts_in_turn():
    calls = [(64, 512, 2048, "none", lay) for lay in ("NT", "NN", "TN", "TT")] + \
            [(64, 4096, 4096, "none", lay) for lay in ("TT", "NN", "TN", "NT")]
    ws = torch.zeros(max(size("bf16", *c) for c in calls), dtype=torch.uint8, device="cuda")
    for c in calls:
        forward(ws, "bf16", *c)


@pytest.mark.parametrize("M,N,K", [(622, 6488, 5760), (64, 4096, 4096)])
def test_one_size_at_two_alignments(M, N, K):
    # the plan depends on whether rows start on 128-byte lines
    ws = torch.zeros(size("bf16", M, N, K) * 2, dtype=torch.uint8, device="cuda")
    for shift in (8, 0, 8, 0):
        forward(ws, "bf16", M, N, K, shift=shift)
