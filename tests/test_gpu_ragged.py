"""The products grouped by expert with ragged segments (forward, input gradient, weight
gradient) against the formula in 64 bits, and the gradients against differences.

Bound.  The products are exact in fp32 (two 8- or 11-bit significands), so the sum in fp32 is off by
at most E = (terms) 2^-24 S, S being the sum of the products' magnitudes (the matrix unit adds several
products per step, so the number of terms bounds its additions).  Rounding to D's type is monotonic:
the element lies between the roundings of exact - E and exact + E."""
import numpy as np
import pytest
import torch  # noqa: F401  (before the library is loaded, at collection: both then share torch's HIP runtime)

import fp8_block_scaled_e4m3_amd as dg
from tests.gpu_support import require_gpu, say

pytestmark = pytest.mark.gpu

SENTINEL = -77.0


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()
    dg.load_library()


TILES = [(0, 0, 0)] + [(*t, 0) for t in dg.dg_ragged_tile_info()] + [(128, 128, 3), (32, 128, 4), (128, 128, 32)]


@pytest.fixture(autouse=True, params=TILES, ids=lambda t: f"{t[0]}x{t[1]}by{t[2]}")
def tile(request):
    """Every test runs as planned, with each compiled tile, and with the contraction in slices."""
    dg.dg_set_ragged_tile(*request.param)
    yield request.param
    dg.dg_set_ragged_tile(0, 0)


def types():
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def offsets_of(counts, first=0):
    import torch
    return torch.tensor(np.cumsum([first] + list(counts)), dtype=torch.int32, device="cuda")


def normal(shape, seed, dtype, pad=0):
    """Seeded values; with ``pad`` the rows are a view of wider ones, whose rest is NaN."""
    import torch
    x = np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)
    t = torch.from_numpy(x).to(types()[dtype]).cuda()
    if not pad:
        return t
    wide = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :shape[1]] = t
    return wide[:, :shape[1]]


def exact(op, counts, first, a, b):
    """(result, sum of magnitudes) in 64 bits: [rows, width] or [groups, n, k]."""
    out, mag, at = [], [], first
    a, b = a.double().cpu(), b.double().cpu()
    for g, c in enumerate(counts):
        x = a[at:at + c]
        y = b[at:at + c] if op == "tn" else (b[g].T if op == "nt" else b[g])
        x = x.T if op == "tn" else x
        out.append(x @ y)
        mag.append(x.abs() @ y.abs())
        at += c
    import torch
    join = torch.stack if op == "tn" else torch.cat
    return join(out).numpy(), join(mag).numpy()


def close(got, want, mag, terms, dtype, where=""):
    import torch
    got = got.double().cpu().numpy()
    lo, hi = (torch.from_numpy(want + sign * terms * 2.0 ** -24 * mag).to(types()[dtype]).double().numpy()
              for sign in (-1, 1))
    bad = ~((lo <= got) & (got <= hi))
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def run_weights(op, counts, n, k, dtype="bf16", seed=0, first=0, last=0, pad=0):
    import torch
    rows = first + sum(counts) + last
    wa, wd = (k, n) if op == "nt" else (n, k)
    a = normal((rows, wa), seed, dtype, pad)
    b = normal((len(counts), n, k), seed + 1, dtype)
    d = torch.full((rows, wd + pad), SENTINEL, dtype=a.dtype, device="cuda")
    view = d[:, :wd]
    say(f"ragged {op} counts={list(counts)[:8]} n={n} k={k} {dtype} pad={pad}")
    getattr(dg, f"dg_m_grouped_gemm_ragged_{op}")(a, b, view, offsets_of(counts, first))
    torch.cuda.synchronize()
    end = first + sum(counts)
    want, mag = exact(op, counts, first, a, b)
    close(view[first:end], want, mag, wa, dtype, op)
    assert (view[:first] == SENTINEL).all() and (view[end:] == SENTINEL).all(), "rows outside the segments"
    assert (d[:, wd:] == SENTINEL).all(), "columns beyond the width"


COUNTS = [[1], [0, 1, 0], [3, 0, 130, 1, 257], [128, 256, 64], [17] * 9, [0, 0, 700, 0], [33, 65, 31, 129, 5]]


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("n,k", [(128, 128), (8, 8), (264, 72), (72, 456)])
def test_products_with_weights(op, counts, n, k):
    run_weights(op, counts, n, k, seed=n + k)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_strides_and_rows_outside_the_segments(op, dtype):
    run_weights(op, [40, 0, 129, 7], 200, 136, dtype=dtype, first=5, last=300, pad=24)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,n,k", [([2000, 5, 1100], 520, 648), ([300] * 8, 1024, 256), ([4, 2, 0, 1] * 16, 384, 1032),
                                        ([9000], 264, 72)])
def test_larger_products(op, dtype, counts, n, k):
    run_weights(op, counts, n, k, dtype=dtype, seed=3)


def run_tn(counts, n, k, dtype="bf16", out="same", add=False, seed=0, first=0, last=0, pad=0):
    import torch
    rows = first + sum(counts) + last
    kind = dtype if out == "same" else out
    a, b = normal((rows, n), seed, dtype, pad), normal((rows, k), seed + 1, dtype, pad)
    d = normal((len(counts), n, k), seed + 2, kind)
    before = d.double().cpu().numpy()
    say(f"ragged tn counts={list(counts)[:8]} n={n} k={k} {dtype} out={kind} add={add}")
    dg.dg_k_grouped_gemm_ragged_tn(a, b, d, offsets_of(counts, first), accumulate=add)
    torch.cuda.synchronize()
    want, mag = exact("tn", counts, first, a, b)
    if add:
        want, mag = want + before, mag + np.abs(before)
    close(d, want, mag, max(counts) + 1, kind, "tn")


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("n,k", [(128, 128), (8, 8), (264, 72), (72, 456)])
def test_weight_gradient(counts, n, k):
    run_tn(counts, n, k, seed=n + k)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("counts,n,k", [([40, 0, 129, 7], 200, 136), ([2500, 300], 264, 520)])
def test_weight_gradient_types(dtype, out, add, counts, n, k):
    run_tn(counts, n, k, dtype=dtype, out=out, add=add, seed=5, first=3, last=40, pad=8)


@pytest.mark.parametrize("add", [False, True])
def test_weight_gradient_without_rows(add):
    """No row at all: zeros replace what D held; accumulation leaves it."""
    import torch
    d = normal((3, 64, 72), 1, "bf16")
    before = d.clone()
    a, b = (torch.empty((0, w), dtype=torch.bfloat16, device="cuda") for w in (64, 72))
    dg.dg_k_grouped_gemm_ragged_tn(a, b, d, offsets_of([0, 0, 0]), accumulate=add)
    torch.cuda.synchronize()
    assert torch.equal(d, before if add else torch.zeros_like(d))


@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
def test_nan_and_infinity_stay_in_their_rows(op):
    """A row of NaN or infinity shows in its own row (or its group's gradient) alone, also where the
    next segment's rows lie in the same tile of rows."""
    import torch
    counts, n, k = [10, 20, 5], 136, 200
    a = normal((40, n if op != "nt" else k), 1, "bf16")
    a[9] = float("nan")         # last row of group 0
    a[30] = float("inf")        # first row of group 2
    a[35:] = float("nan")       # rows outside the segments
    if op == "tn":
        b = normal((40, k), 2, "bf16")
        d = torch.zeros((3, n, k), dtype=torch.bfloat16, device="cuda")
        dg.dg_k_grouped_gemm_ragged_tn(a, b, d, offsets_of(counts))
        assert d[0].isnan().all() and d[1].isfinite().all() and not d[2].isfinite().any()
    else:
        b = normal((3, n, k), 2, "bf16")
        d = torch.zeros((40, n if op == "nt" else k), dtype=torch.bfloat16, device="cuda")
        getattr(dg, f"dg_m_grouped_gemm_ragged_{op}")(a, b, d, offsets_of(counts))
        fine = d.isfinite().all(1).cpu()
        assert fine[[i for i in range(35) if i not in (9, 30)]].all() and not fine[9] and not fine[30]
        assert (d[35:] == 0).all()


@pytest.mark.parametrize("op", ["nt", "tn"])
def test_offsets_out_of_order_stay_inside(op):
    """Offsets below an earlier one count as that one, those past the rows as their number."""
    import torch
    n, k, rows = 72, 136, 50
    given, meant = [-4, 20, 12, 30, 1 << 30], [0, 20, 20, 30, 50]
    a, counts = normal((rows, n if op == "tn" else k), 1, "bf16"), np.diff(meant)
    off = torch.tensor(given, dtype=torch.int32, device="cuda")
    if op == "tn":
        b = normal((rows, k), 2, "bf16")
        d = torch.zeros((4, n, k), dtype=torch.bfloat16, device="cuda")
        dg.dg_k_grouped_gemm_ragged_tn(a, b, d, off)
    else:
        b = normal((4, n, k), 2, "bf16")
        d = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
        dg.dg_m_grouped_gemm_ragged_nt(a, b, d, off)
    want, mag = exact(op, counts, 0, a, b)
    close(d, want, mag, max(n, k, rows), "bf16", op)


def test_gradients_agree_with_differences():
    """The loss sum(r . forward(x, w)): its directional difference in x and in w equals the
    gradients' products with the direction.  The loss is linear in each, so a difference over a step
    of 1 in exactly representable numbers has no truncation error; small integers keep every sum
    exact (below 2^24, and below 2^8 in the BF16 outputs)."""
    import torch
    counts, n, k = [5, 0, 12, 1], 24, 16
    rng = np.random.default_rng(8)

    def ints(*shape, hi=2):
        return torch.from_numpy(rng.integers(-hi, hi + 1, shape).astype(np.float32)).to(torch.bfloat16).cuda()

    x, w, r = ints(18, k), ints(4, n, k), ints(18, n, hi=1)
    dx, dw = ints(18, k, hi=1), ints(4, n, k, hi=1)
    off = offsets_of(counts)

    def loss(x, w):
        y = torch.empty((18, n), dtype=torch.bfloat16, device="cuda")
        dg.dg_m_grouped_gemm_ragged_nt(x, w, y, off)
        return (y.double() * r.double()).sum()

    gx = torch.empty_like(x)
    gw = torch.empty((4, n, k), dtype=torch.float32, device="cuda")
    dg.dg_m_grouped_gemm_ragged_nn(r, w, gx, off)
    dg.dg_k_grouped_gemm_ragged_tn(r, x, gw, off)
    assert loss(x + dx, w) - loss(x, w) == (gx.double() * dx.double()).sum()
    assert loss(x, w + dw) - loss(x, w) == (gw.double() * dw.double()).sum()


def test_stream_and_cu_cap():
    """On another stream than the current one, and with fewer CUs: the same bits."""
    import torch
    counts, n, k = [300, 17, 0, 500], 520, 264
    a, b, off = normal((817, k), 1, "bf16"), normal((4, n, k), 2, "bf16"), offsets_of(counts)
    want = torch.empty((817, n), dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_gemm_ragged_nt(a, b, want, off)
    side = torch.cuda.Stream()
    got = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    dg.dg_set_num_cus(7)
    try:
        dg.dg_m_grouped_gemm_ragged_nt(a, b, got, off, stream=side)
    finally:
        dg.dg_set_num_cus(0)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
def test_graph_replays_follow_the_offsets(op):
    """A captured call reads the offsets at each replay; every replay equals the eager result."""
    import torch
    n, k, rows = 136, 264, 400
    a = normal((rows, k if op == "nt" else n), 1, "bf16")
    b = normal((rows, k) if op == "tn" else (4, n, k), 2, "bf16")
    shape = {"nt": (rows, n), "nn": (rows, k), "tn": (4, n, k)}[op]
    off = offsets_of([100, 100, 100, 100])
    call = dg.dg_k_grouped_gemm_ragged_tn if op == "tn" else getattr(dg, f"dg_m_grouped_gemm_ragged_{op}")
    d, want = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call(a, b, d, off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, b, d, off)
    for counts in ([100] * 4, [400, 0, 0, 0], [1, 2, 3, 394], [0, 0, 0, 10], [130, 140, 0, 130]):
        off.copy_(offsets_of(counts))
        d.zero_()
        want.zero_()
        graph.replay()
        torch.cuda.synchronize()
        call(a, b, want, off)
        torch.cuda.synchronize()
        assert torch.equal(d, want), counts
