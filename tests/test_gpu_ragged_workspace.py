"""The ragged products' workspace, as a call is planned (bounds as in test_gpu_ragged.py)."""
import pytest

import fp8_block_scaled_e4m3_amd as dg
from tests.gpu_support import require_gpu
from tests.test_gpu_ragged import close, exact, normal, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()
    dg.load_library()


@pytest.mark.parametrize("op", ["nn", "tn"])
def test_slices_with_a_given_workspace(op):
    """Few tiles and a long contraction: the planned call uses a workspace; the one it is given holds
    the sums, the bytes behind it stay; without one the call is right too."""
    import torch
    n, k, rows = (7168, 248, 13) if op == "nn" else (328, 264, 9000)
    a, off = normal((rows, n), 1, "bf16"), offsets_of([rows])
    b = normal((1, n, k) if op == "nn" else (rows, k), 2, "bf16")
    shape = (rows, k) if op == "nn" else (1, n, k)
    size = dg.dg_ragged_workspace_bytes(dg.DG_RAGGED_NN if op == "nn" else dg.DG_RAGGED_TN, rows, n, k, 1, 1, 1)
    assert size > 0
    call = dg.dg_m_grouped_gemm_ragged_nn if op == "nn" else dg.dg_k_grouped_gemm_ragged_tn
    ws = torch.full((size + 64,), 7, dtype=torch.uint8, device="cuda")
    want, mag = exact(op, [rows], 0, a, b)
    for given in (ws[:size], ws[:0], None):
        d = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        call(a, b, d, off, workspace=given)
        torch.cuda.synchronize()
        close(d, want, mag, n if op == "nn" else rows, "bf16", op)
    assert (ws[size:] == 7).all() and (ws[:size] != 7).any()


def test_many_tiles_want_no_workspace():
    assert dg.dg_ragged_workspace_bytes(dg.DG_RAGGED_NT, 32768, 4096, 7168, 8, 1, 1) == 0
    assert dg.dg_ragged_workspace_bytes(dg.DG_RAGGED_TN, 16384, 4096, 7168, 8, 1, 0) == 0


def test_workspace_on_another_stream():
    """A call on a stream of its own takes its workspace there: two such calls, one behind the other,
    with work of the current stream between, agree."""
    import torch
    a, off = normal((13, 7168), 1, "bf16"), offsets_of([13])
    b = normal((1, 7168, 248), 2, "bf16")
    want = torch.zeros((13, 248), dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_gemm_ragged_nn(a, b, want, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [torch.zeros_like(want) for _ in range(2)]
    torch.cuda.synchronize()
    for d in got:
        dg.dg_m_grouped_gemm_ragged_nn(a, b, d, off, stream=side)
        torch.full((1 << 20,), 3.0, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
