"""One workspace through calls of different sizes, pitches and alignments: what a call leaves behind
must not reach a later call that lays the workspace out in another way."""
import pytest
import torch

import ffn_ref as R
from test_gemm_act_gpu import operands, rand, reference_gradient

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


def back_size(kind, M, N, K, name, layout="NT"):
    import dense_tensor_core_gb300 as dtc
    return dtc.gemm_act_backward_workspace_size(kind, M, N, K, layout=layout, activation=name)


def backward(ws, kind, M, N, K, name, layout="NT"):
    """Against the same call with a workspace of its own, bit for bit; that one against the reference."""
    import dense_tensor_core_gb300 as dtc
    A, B, Nb = operands(kind, layout, M, N, K, name)
    dC, z = rand((M, N), kind, 5), rand((M, Nb), kind, 6, 1.5) if name != "none" else None
    own, got = (dtc.gemm_act_backward(kind, dC, A, B, preact=z, layout=layout, activation=name, workspace=w)
                for w in (torch.zeros(back_size(kind, M, N, K, name, layout), dtype=torch.uint8, device="cuda"), ws))
    dtc.gemm_stream_status()
    ra, rb, dz = reference_gradient(kind, dC, A, B, z, layout, name)
    R.close(own[0], ra, 2.1 * R.U[kind], "dA")  # (the rounding of dZ and of the result)
    R.close(own[1], rb, 2.1 * R.U[kind], "dB")
    # terms up to 1.13 |dC| (gated: times |u| or the gate's), activations within 2^-18, M fp32 additions
    size = dC.double().abs().sum(0).repeat(Nb // N) * (1.13 * (z.double().abs().max() if z is not None else 1.0) + 1.0)
    R.check(own[2], dz.sum(0), (2.0 ** -16 + M * 2.0 ** -24) * size, "dbias")
    for x, y, what in zip(got, own, ("dA", "dB", "dbias")):
        assert torch.equal(x, y), f"{what} of {M} x {N} x {K} {name}"


# products with and without stream-K pieces; column sums over few strips and many row blocks, over many
# strips, and over more strips than SMs (one row block each)
BACK = [(777, 1544, 1032, "silu"), (4096, 2048, 4096, "gelu"), (2050, 136, 264, "swiglu"),
        (40, 40960, 64, "none"), (100, 20480, 64, "geglu"), (4096, 4096, 2048, "none"), (64, 72, 64, "relu")]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_gradients_in_turn(kind):
    import dense_tensor_core_gb300 as dtc
    assert any(dtc.gemm_workspace_size(kind, M, K, N, layout="NN") for M, N, K, _ in BACK[:-1])  # stream-K
    assert not dtc.gemm_workspace_size(kind, 64, 64, 72, layout="NN")
    ws = torch.zeros(max(back_size(kind, *c) for c in BACK), dtype=torch.uint8, device="cuda")
    for c in BACK + BACK[::-1]:
        backward(ws, kind, *c)


def test_both_directions_in_turn():
    ws = torch.zeros(max([back_size("bf16", *c) for c in BACK] + [size("bf16", *c) for c in CALLS]),
                     dtype=torch.uint8, device="cuda")
    for c, b in zip(CALLS, BACK):
        forward(ws, "bf16", *c)
        backward(ws, "bf16", *b)
    for c, b in zip(CALLS, BACK[::-1]):
        backward(ws, "bf16", *b)
        forward(ws, "bf16", *c)
