"""The AdamW step over many tensors against the formula in 64 bits, and, for the 8-bit states,
against the same fp32 operations one by one on the CPU, bit for bit.

Bounds.  With u = 2^-24 and every operation rounded once: m = m b1 + g (1 - b1), constants included,
is off by at most 5u(|m b1| + |g (1 - b1)|); v, where g enters squared, by 6u of itself (its terms have
one sign); its root by 3u + u.  The quotient m / (root r2 + eps) gains 3u more from its divisor and 1u from
the division, and the update 2u (the constant and the product), p's product 2u, the last difference u of the result."""
import math

import numpy as np
import pytest

import fp8_block_scaled_e4m3_amd as dg
from tests.gpu_support import require_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LR, B1, B2, EPS, WD = 1e-3, 0.9, 0.95, 1e-8, 0.1


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()
    dg.load_library()


def types():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def blocks(x):
    import torch
    return torch.cat([x, x.new_zeros(-x.numel() % 128)]).view(-1, 128)


def encode(x, root=False):
    """Codes and scales of fp32 values on the CPU, one correctly rounded operation at a time."""
    import torch
    b = blocks(x)
    amax = b.abs().amax(1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
    q = (b / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if root:
        q = torch.where((b > 0) & (q == 0), torch.ones_like(q), q)
    return q.reshape(-1)[:x.numel()].clone(), scale


def sqrt32(x):
    """The correctly rounded fp32 root (numpy's; torch's on the CPU can be one ulp off)."""
    import torch
    return torch.from_numpy(np.sqrt(x.numpy()))


def decode(q, scale):
    import torch
    return (blocks(q.view(torch.float8_e4m3fn).float()) * scale[:, None]).reshape(-1)[:q.numel()]


def make(sizes, param, grad, copy, fp8, seed):
    """CPU inputs: per tensor p, g, m, v (fp32 values; 8-bit states already coded and decoded)."""
    import torch
    rng = np.random.default_rng(seed)
    out = []
    for i, n in enumerate(sizes):
        def draw(scale):
            return torch.from_numpy(rng.standard_normal(n, dtype=np.float32) * np.float32(scale))
        t = {"p": draw(0.05).to(types()[param]), "g": draw(1e-3 * 2.0 ** -(i % 7)).to(types()[grad]),
             "m": draw(3e-4), "v": draw(1e-3) ** 2 + 1e-10}
        if n > 4:
            t["m"][1] = t["v"][1] = t["g"][1] = 0.0          # an element that never had a gradient
            t["v"][2] = 1e-16                                # a root far below its block's largest
        if fp8:
            t["m"], t["ms"] = encode(t["m"])
            t["v"], t["vs"] = encode(t["v"].sqrt(), root=True)
        out.append(t)
    return out


def on_gpu(tensors, copy):
    dev = [{k: x.cuda() for k, x in t.items()} for t in tensors]
    if copy != "none":
        for t in dev:
            t["c"] = t["p"].new_zeros(t["p"].shape, dtype=types()[copy])
    return dev


def plan_of(dev):
    get = lambda k: [t[k] for t in dev] if dev and k in dev[0] else None  # noqa: E731
    return dg.dg_adamw_plan(get("p"), get("g"), get("m"), get("v"), get("ms"), get("vs"), get("c"))


def formula64(t, step, lr=LR, b1=B1, b2=B2, eps=EPS, wd=WD, gs=1.0):
    p, g = t["p"].double(), t["g"].double() * gs
    m, v = (decode(t["m"], t["ms"]).double(), decode(t["v"], t["vs"]).double() ** 2) if "ms" in t else \
        (t["m"].double(), t["v"].double())
    mag = (m * b1).abs() + (g * (1 - b1)).abs()
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    upd = lr / (1 - b1 ** step) / ((v / (1 - b2 ** step)).sqrt() + eps)
    new = p * (1 - lr * wd) - upd * m
    tiny = 2.0 ** -126
    err_p = U * (2 * p.abs() + new.abs()) * 1.01 + upd * mag * 16 * U + tiny
    return {"p": (new, err_p), "m": (m, 5.05 * U * mag + tiny), "v": (v, 6.05 * U * v + tiny)}


def within(got, want, err, what, dtype=None):
    """The roundings (to ``dtype``) of want -/+ err enclose got."""
    got, lo, hi = got.double().cpu(), want - err, want + err
    if dtype is not None:
        lo, hi = lo.to(dtype).double(), hi.to(dtype).double()
    bad = ~((lo <= got) & (got <= hi))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {int(bad.nonzero()[0])}"


def check(tensors, dev, step, **kw):
    for i, (t, d) in enumerate(zip(tensors, dev)):
        w = formula64(t, step, **kw)
        within(d["p"], *w["p"], f"param {i}", d["p"].dtype)
        if "c" in d:
            within(d["c"], *w["p"], f"copy {i}", d["c"].dtype)
        if "ms" not in d:
            within(d["m"], *w["m"], f"exp_avg {i}")
            within(d["v"], *w["v"], f"exp_avg_sq {i}")


SIZES = [[1], [7, 128, 129], [2048, 2047, 2049, 0, 5], [100003], [64] * 40 + [4096, 33]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("param", ["f32", "bf16"])
@pytest.mark.parametrize("grad,copy", [("f32", "none"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("fp8", [False, True], ids=["f32states", "fp8states"])
def test_step_matches_the_formula(sizes, param, grad, copy, fp8):
    import torch
    say(f"adamw {len(sizes)} tensors up to {max(sizes)}, {param} {grad} {copy} fp8={fp8}")
    tensors = make(sizes, param, grad, copy, fp8, seed=len(sizes))
    dev = on_gpu(tensors, copy)
    dg.dg_adamw_step(plan_of(dev), 3, LR, B1, B2, EPS, WD)
    torch.cuda.synchronize()
    check(tensors, dev, 3)
    for t, d in zip(tensors, dev):
        assert torch.equal(d["g"].cpu(), t["g"])


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_fp8_states_bit_exact_over_steps(sizes):
    """Codes and scales of three steps equal the fp32 operations done one at a time."""
    import torch
    tensors = make(sizes, "f32", "bf16", "none", True, seed=11)
    dev = on_gpu(tensors, "none")
    plan = plan_of(dev)
    for step in (1, 2, 3):
        dg.dg_adamw_step(plan, step, LR, B1, B2, EPS, WD)
        torch.cuda.synchronize()
        for i, (t, d) in enumerate(zip(tensors, dev)):
            g = t["g"].float()
            m, r = decode(t["m"], t["ms"]), decode(t["v"], t["vs"])
            m = m * B1 + g * (1.0 - B1)
            v = (r * r) * B2 + (g * g) * (1.0 - B2)
            t["m"], t["ms"] = encode(m)
            t["v"], t["vs"] = encode(sqrt32(v), root=True)
            for key in ("m", "v", "ms", "vs"):
                assert torch.equal(d[key].cpu(), t[key]), f"step {step}, tensor {i}: {key}"


def test_a_small_root_never_becomes_zero():
    """One large root in a block: the others keep the smallest code, and their next update stays bounded
    by the learning rate's order instead of m / eps."""
    import torch
    t = make([128], "f32", "f32", "none", True, seed=2)
    t[0]["g"] = torch.full((128,), 1e-6)
    t[0]["g"][0] = 10.0
    t[0]["m"], t[0]["ms"] = encode(torch.zeros(128))
    t[0]["v"], t[0]["vs"] = encode(torch.zeros(128), root=True)
    dev = on_gpu(t, "none")
    plan = plan_of(dev)
    before = dev[0]["p"].clone()
    for step in (1, 2, 3):
        dg.dg_adamw_step(plan, step, LR, B1, B2, EPS, 0.0)
    torch.cuda.synchronize()
    assert (dev[0]["v"] != 0).all()
    assert ((dev[0]["p"] - before).abs() <= 3 * 1.5 * LR).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["f32states", "fp8states"])
def test_zero_state_zero_gradient(fp8):
    """Nothing moves but the decay: no 0 / 0 with eps > 0."""
    import torch
    t = make([300], "f32", "f32", "none", fp8, seed=4)
    zero = torch.zeros(300)
    t[0]["g"] = zero
    if fp8:
        (t[0]["m"], t[0]["ms"]), (t[0]["v"], t[0]["vs"]) = encode(zero), encode(zero, root=True)
    else:
        t[0]["m"], t[0]["v"] = zero, zero
    dev = on_gpu(t, "none")
    dg.dg_adamw_step(plan_of(dev), 1, LR, B1, B2, EPS, WD)
    torch.cuda.synchronize()
    assert torch.equal(dev[0]["p"].cpu(), t[0]["p"] * (1.0 - LR * WD))


def test_grad_scale_and_hyperparameters():
    import torch
    tensors = make([5000, 77], "f32", "bf16", "bf16", False, seed=6)
    dev = on_gpu(tensors, "bf16")
    # (a power of two: the scaled gradient is exact, as the bounds assume)
    scale = torch.tensor(0.125, device="cuda")
    dg.dg_adamw_step(plan_of(dev), 1000, 3e-5, 0.8, 0.999, 1e-6, 0.0, grad_scale=scale)
    torch.cuda.synchronize()
    check(tensors, dev, 1000, lr=3e-5, b1=0.8, b2=0.999, eps=1e-6, wd=0.0, gs=0.125)


@pytest.mark.parametrize("fp8", [False, True], ids=["f32states", "fp8states"])
def test_neighbours_are_left_alone(fp8):
    """Tensors as views of one buffer, with guard elements between them that stay as they are."""
    import torch
    tensors = make([1000, 130, 2050], "f32", "f32", "bf16", fp8, seed=9)
    dev, guards = [], []
    for t in tensors:
        d = {}
        for key, x in list(t.items()) + [("c", t["p"].to(torch.bfloat16))]:
            buf = torch.full((x.numel() + 64,), 3, dtype=x.dtype, device="cuda")
            d[key] = buf[32:32 + x.numel()]
            d[key].copy_(x)
            if key != "g":
                guards.append((buf, 32 + x.numel()))
        dev.append(d)
    dg.dg_adamw_step(plan_of(dev), 3, LR, B1, B2, EPS, WD)
    torch.cuda.synchronize()
    check(tensors, dev, 3)
    assert all((b[:32] == 3).all() and (b[end:] == 3).all() for b, end in guards)


def test_nan_spoils_its_element_alone_with_f32_states():
    import torch
    tensors = make([500], "f32", "f32", "none", False, seed=1)
    dev = on_gpu(tensors, "none")
    dev[0]["g"][100] = float("nan")
    dg.dg_adamw_step(plan_of(dev), 3, LR, B1, B2, EPS, WD)
    torch.cuda.synchronize()
    for key in ("p", "m", "v"):
        bad = dev[0][key].isnan().nonzero().flatten().tolist()
        assert bad == [100], key


def test_update_direction_agrees_with_differences():
    """Plain quadratic loss (p - q)^2 / 2 with the gradient taken by central differences of the loss:
    steps of AdamW bring every element nearer to q."""
    import torch
    rng = np.random.default_rng(5)
    p = torch.from_numpy(rng.standard_normal(1000, dtype=np.float32)).cuda()
    q = torch.from_numpy(rng.standard_normal(1000, dtype=np.float32)).cuda()
    g, m, v = torch.zeros_like(p), torch.zeros_like(p), torch.zeros_like(p)
    plan = dg.dg_adamw_plan([p], [g], [m], [v])
    loss = lambda x: (x.double() - q.double()) ** 2 / 2  # noqa: E731
    far = (p - q).abs() > 0.2
    first = loss(p)
    for step in range(1, 101):
        g.copy_((loss(p.double() + 1e-3) - loss(p.double() - 1e-3)) / 2e-3)
        dg.dg_adamw_step(plan, step, 1e-3, 0.9, 0.99, 1e-8, 0.0)
    assert (loss(p)[far] < first[far]).all()


def test_stream_and_graph():
    """On another stream, and replayed from a graph: the bits of eager steps with the same scalars."""
    import torch
    tensors = make([3000, 129], "f32", "bf16", "bf16", True, seed=21)
    eager, graphed = on_gpu(tensors, "bf16"), on_gpu(tensors, "bf16")
    pe, pg = plan_of(eager), plan_of(graphed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_adamw_step(pg, 5, LR, B1, B2, EPS, WD)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        dg.dg_adamw_step(pe, 5, LR, B1, B2, EPS, WD, stream=side)
        side.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, graphed):
            assert all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)
