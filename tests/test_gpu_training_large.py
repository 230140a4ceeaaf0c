"""The training operators where element numbers and byte offsets pass 32 bits.  Inputs are made on
the GPU; the parts checked are at the far end, against 64 bits with the bounds of
test_gpu_ragged.py and test_gpu_adamw.py."""
import pytest

import fp8_block_scaled_e4m3_amd as dg
from tests.gpu_support import require_gpu, say
from tests.test_gpu_ragged import close, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()
    dg.load_library()


@pytest.fixture(autouse=True)
def free():
    import torch
    yield
    torch.cuda.empty_cache()


def values(*shape):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.bfloat16)


ROWS, WIDE = 300000, 8192          # 4.9 GB of BF16
COUNTS = [200001, 0, 99000, 900]


def test_rows_past_32_bits_with_weights():
    import torch
    a, b = values(ROWS, WIDE), values(4, 16, WIDE)
    d = torch.zeros(ROWS, 16, dtype=torch.bfloat16, device="cuda")
    say("large nt")
    dg.dg_m_grouped_gemm_ragged_nt(a, b, d, offsets_of(COUNTS))
    for rows, g in ((slice(199990, 200001), 0), (slice(200001, 200030), 2), (slice(299080, ROWS - 99), 3)):
        x, w = a[rows].double().cpu(), b[g].double().cpu()
        close(d[rows], (x @ w.T).numpy(), (x.abs() @ w.T.abs()).numpy(), WIDE, "bf16", "nt")
    assert (d[ROWS - 99:] == 0).all()
    say("large nn: the wide matrix is the output")
    dy, w = values(ROWS, 16), b.contiguous()
    a.zero_()
    dg.dg_m_grouped_gemm_ragged_nn(dy, w, a, offsets_of(COUNTS))
    for rows, g in ((slice(200001, 200010), 2), (slice(ROWS - 110, ROWS - 99), 3)):
        x, v = dy[rows].double().cpu(), w[g].double().cpu()
        close(a[rows], (x @ v).numpy(), (x.abs() @ v.abs()).numpy(), 16, "bf16", "nn")
    assert (a[ROWS - 99:] == 0).all()


def test_weight_gradient_of_rows_past_32_bits():
    import torch
    a, b = values(ROWS, 16), values(ROWS, WIDE)
    d = torch.zeros(4, 16, WIDE, device="cuda")
    say("large tn")
    dg.dg_k_grouped_gemm_ragged_tn(a, b, d, offsets_of(COUNTS))
    assert (d[1] == 0).all()
    x, y = a[299001:ROWS - 99].double().cpu(), b[299001:ROWS - 99].double().cpu()
    close(d[3], (x.T @ y).numpy(), (x.T.abs() @ y.abs()).numpy(), 900, "f32", "tn")


def test_weights_past_32_bits():
    """40 groups of 8192 x 8192 weights: 2.7 G elements."""
    import torch
    b = torch.empty(40, WIDE, WIDE, dtype=torch.bfloat16, device="cuda")
    b[39] = values(WIDE, WIDE)
    b[38] = 1.0
    a = values(6, WIDE)
    d = torch.zeros(6, WIDE, dtype=torch.bfloat16, device="cuda")
    say("large weights")
    off = offsets_of([0] * 38 + [2, 4])
    x, w = a[2:].double().cpu(), b[39].double().cpu()
    dg.dg_m_grouped_gemm_ragged_nt(a, b, d, off)
    close(d[2:], (x @ w.T).numpy(), (x.abs() @ w.T.abs()).numpy(), WIDE, "bf16", "nt")
    dg.dg_m_grouped_gemm_ragged_nn(a, b, d, off)
    close(d[2:], (x @ w).numpy(), (x.abs() @ w.abs()).numpy(), WIDE, "bf16", "nn")
    say("large weight gradients")
    b[39] = 0
    dg.dg_k_grouped_gemm_ragged_tn(a, values(6, WIDE), b, off)
    y = values(6, WIDE)[2:].double().cpu()
    close(b[39][:64], (x[:, :64].T @ y).numpy(), (x[:, :64].T.abs() @ y.abs()).numpy(), 4, "bf16", "tn")


@pytest.mark.parametrize("fp8", [False, True], ids=["f32states", "fp8states"])
def test_adamw_elements_past_32_bits(fp8):
    """One tensor of 2^31 + 1000 elements (BF16): its last elements, and the element after an exact
    multiple of 2^31, move as a short tensor's with the same values."""
    import torch
    n, tail = 2 ** 31 + 1000, 1256            # (the tail begins with a block of 128)
    kind = torch.float8_e4m3fn if fp8 else torch.float32
    big = [torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
           torch.zeros(n, dtype=kind, device="cuda"), torch.zeros(n, dtype=kind, device="cuda")]
    big[0][-tail:], big[1][-tail:] = values(tail), values(tail) * 1e-3
    small = [x[-tail:].clone() for x in big]
    extra = [[torch.ones(-(-x.numel() // 128), device="cuda") for _ in range(2)] for x in (big[0], small[0])] if fp8 else None
    say("large adamw", fp8)
    for i, x in enumerate((big, small)):
        scales = [[s] for s in extra[i]] if fp8 else [None, None]
        plan = dg.dg_adamw_plan([x[0]], [x[1]], [x[2]], [x[3]], *scales)
        for step in (1, 2):
            dg.dg_adamw_step(plan, step, 1e-2, 0.9, 0.95, 1e-8, 0.1)
    torch.cuda.synchronize()
    for b, s in zip(big, small):
        assert torch.equal(b[-tail:].float(), s.float()) and not (s == 0).all()
    assert (big[0][:-tail] == 0).all()
