"""The ragged products where the last round of large tiles goes to smaller ones: the same result
whatever part of a round is left (bounds as in test_gpu_ragged.py)."""
import pytest
import torch

import fp8_block_scaled_e4m3_amd as dg
from tests.gpu_support import require_gpu, say
from tests.test_gpu_ragged import SENTINEL, close, exact, normal, offsets_of

pytestmark = pytest.mark.gpu

LONG, WIDTH = 2056, 1032           # contraction; columns of D: five tiles of 256, the last one of 8
ROWS = [[14080],                                        # 275 tiles
        [5003, 0, 1, 130, 8950, 255],                   # segments whose last tiles hold one half
        [257] * 27 + [0] + [127] * 5]                   # two row tiles of one row more than a tile, and short ones


@pytest.fixture(autouse=True)
def as_planned():
    require_gpu()
    dg.load_library()
    yield
    dg.dg_set_ragged_tile(0, 0)
    dg.dg_set_num_cus(0)


def call(op, a, b, off, rows, first, tile, cus=0):
    d = torch.full((rows + 2 * first, WIDTH + 8), SENTINEL, dtype=a.dtype, device="cuda")
    dg.dg_set_ragged_tile(*tile)
    dg.dg_set_num_cus(cus)
    getattr(dg, f"dg_m_grouped_gemm_ragged_{op}")(a, b, d[:, :WIDTH], off)
    torch.cuda.synchronize()
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", ROWS, ids=lambda c: f"{len(c)}groups")
@pytest.mark.parametrize("op", ["nt", "nn"])
def test_any_part_of_a_round(op, counts, dtype):
    """Grids from a few workgroups to the whole device leave another part of a round each; every
    result has the bits of the smaller tile alone, and those are within the bound."""
    rows, first = sum(counts), 3
    n, k = (WIDTH, LONG) if op == "nt" else (LONG, WIDTH)
    a = normal((rows + 2 * first, LONG), 5, dtype, 8)
    b, off = normal((len(counts), n, k), 6, dtype), offsets_of(counts, first)
    say(f"ragged {op} rounds {counts[:6]} {dtype}")
    want = call(op, a, b, off, rows, first, (128, 128))
    if dtype == "bf16":
        value, mag = exact(op, counts, first, a, b)
        close(want[first:first + rows, :WIDTH], value, mag, LONG, dtype, op)
    for cus in (0, 200, 131, 96, 64, 8, 5, 1):
        say(f"  {cus or 'all'} CUs")
        got = call(op, a, b, off, rows, first, (256, 256), cus)
        assert torch.equal(got, want), f"{cus} CUs"
    assert (want[:first] == SENTINEL).all() and (want[first + rows:] == SENTINEL).all()
    assert (want[:, WIDTH:] == SENTINEL).all()


@pytest.mark.parametrize("op", ["nt", "nn"])
def test_offsets_that_hold_fewer_rows(op):
    """The host plans for the rows that it is told of; the offsets may hold any part of them."""
    rows = 14080
    n, k = (WIDTH, LONG) if op == "nt" else (LONG, WIDTH)
    a, b = normal((rows, LONG), 7, "bf16"), normal((3, n, k), 8, "bf16")
    for counts in ([0, 0, 0], [0, 1, 0], [129, 0, 300], [6000, 0, 700]):
        say(f"ragged {op} fewer rows {counts}")
        off = offsets_of(counts)
        want, got = (call(op, a, b, off, rows, 0, (t, t)) for t in (128, 256))
        assert torch.equal(got, want) and (got[sum(counts):] == SENTINEL).all(), counts
        assert sum(counts) == 0 or (got[:sum(counts), :WIDTH] != SENTINEL).any()


@pytest.mark.parametrize("op", ["nt", "nn"])
def test_captured(op):
    """Both launches are captured, and replays agree with the eager call."""
    counts = ROWS[1]
    rows = sum(counts)
    n, k = (WIDTH, LONG) if op == "nt" else (LONG, WIDTH)
    a, b = normal((rows, LONG), 9, "bf16"), normal((len(counts), n, k), 10, "bf16")
    off, fn = offsets_of(counts), getattr(dg, f"dg_m_grouped_gemm_ragged_{op}")
    want, d = (torch.zeros((rows, WIDTH), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.dg_set_ragged_tile(256, 256)
    fn(a, b, want, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(a, b, d, off)
    for _ in range(3):
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want)
        fn(a, b, d, off)
