"""The library's training operators as measured work: listed and drawn cases, their inputs, a plain
form in elementary torch operations and the library's own calls, and the results in 64 bits.

Two operators that a training step of a mixture of experts runs one after the other:

* matrix products grouped by expert with ragged segment lengths: forward ("nt"), input gradient
  ("nn") and weight gradient ("tn");
* an AdamW step over many tensors at once, with optimizer states in 32 bits or in 8 (E4M3 codes,
  one fp32 scale per 128 elements; the second moment is held as its root).

``own`` selects the library's calls in ``run``; otherwise ``run`` computes the plain form.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128            # elements that share one scale of an 8-bit state
FP8_MAX = 448.0        # largest finite E4M3 value
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
FIRST_STEP = 100       # the states are those of a run under way


# ---- cases ---------------------------------------------------------------------------------

def listed():
    def product(name, op, rows, groups, n, k, dtype="bf16", skew=1.1, out="same", add=False):
        return {"name": name, "op": op, "rows": rows, "groups": groups, "n": n, "k": k, "dtype": dtype,
                "skew": skew, "out": out, "add": add}

    def adamw(name, tensors, smallest, largest, states, grad, copy, param="f32"):
        return {"name": name, "op": "adamw", "tensors": tensors, "smallest": smallest, "largest": largest,
                "states": states, "grad": grad, "copy": copy, "param": param}

    return [
        # one token sent to its experts in a small model: the call's latency
        product("forward_one_token", "nt", 2, 8, 512, 1024, skew=0.0),
        # generation: a batch of tokens over the experts of a layer, bound by the weights' bytes
        product("forward_generation", "nt", 64, 16, 4096, 7168, skew=0.5),
        # many narrow experts with odd widths and ragged segments, FP16
        product("forward_narrow_f16", "nt", 5003, 32, 1416, 712, dtype="f16", skew=0.8),
        # training or prefill: the skewed split of a large batch over eight wide experts
        product("forward_training", "nt", 32768, 8, 4096, 7168),
        # input gradient of a small micro-batch over many narrow experts, some of them empty
        product("input_grad_small", "nn", 701, 48, 1408, 2048, skew=1.3),
        # input gradient of a large batch
        product("input_grad_training", "nn", 16384, 8, 4096, 7168),
        # weight gradient of a small micro-batch, kept in the operands' type
        product("weight_grad_small", "tn", 1001, 32, 768, 1032, skew=0.8),
        # weight gradient of a large batch, added to an fp32 buffer over micro-batches
        product("weight_grad_training", "tn", 16384, 8, 4096, 7168, out="f32", add=True),
        # the small tensors of a model (gains, biases, routers): latency and launch count
        adamw("adamw_small_tensors", 48, 64, 8192, "f32", "f32", copy="none"),
        # a model of many odd-sized tensors, BF16 gradients, 8-bit states
        adamw("adamw_odd_fp8", 96, 999, 1000003, "fp8", "bf16", copy="bf16"),
        # the experts' weights with 32-bit states, fp32 gradients and the BF16 copy the products read
        adamw("adamw_experts_f32", 8, 2048 * 7168, 2048 * 7168, "f32", "f32", copy="bf16"),
        # the same weights with 8-bit states and BF16 gradients
        adamw("adamw_experts_fp8", 8, 2048 * 7168, 2048 * 7168, "fp8", "bf16", copy="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """A layer width: one in common use, or an odd multiple of eight anywhere in the range."""
    if rng.random() < 0.5:
        return rng.choice([256, 512, 768, 1024, 1408, 2048, 2560, 4096, 5120, 7168])
    return 8 * (2 * _log_uniform(rng, 4, 440) + 1)


def draw(rng):
    if rng.random() < 0.3:
        states = rng.choice(["f32", "fp8"])
        smallest = _log_uniform(rng, 1, 200000)
        largest = smallest * _log_uniform(rng, 1, 64)
        most = max(1, min(200, 100000000 // largest))
        return {"op": "adamw", "tensors": _log_uniform(rng, 1, most), "smallest": smallest, "largest": largest,
                "states": states, "grad": rng.choice(["f32", "bf16"]), "copy": rng.choice(["none", "bf16", "f16"]),
                "param": rng.choice(["f32", "f32", "bf16"])}
    op = rng.choice(["nt", "nn", "tn"])
    while True:
        rows, groups, n, k = _log_uniform(rng, 1, 32768), _log_uniform(rng, 1, 64), _width(rng), _width(rng)
        # no more than the largest listed case, in products and in weights
        if rows * n * k <= 32768 * 4096 * 7168 // 2 and groups * n * k <= 16 * 4096 * 7168 // 2:
            break
    out = rng.choice(["same", "f32"]) if op == "tn" else "same"
    return {"op": op, "rows": rows, "groups": groups, "n": n, "k": k, "dtype": rng.choice(["bf16", "bf16", "f16"]),
            "skew": rng.choice([0.0, 0.5, 1.1, 1.5]), "out": out, "add": op == "tn" and rng.random() < 0.5}


# ---- inputs --------------------------------------------------------------------------------

def _counts(case):
    """Rows of each expert, largest first: the expected split of Zipf's law (remainders to the
    largest fractions), so the last of many experts stay empty where the rows are few."""
    g, rows = case["groups"], case["rows"]
    w = [(i + 1) ** -case["skew"] for i in range(g)]
    share = [rows * x / sum(w) for x in w]
    got = [math.floor(s) for s in share]
    for i in sorted(range(g), key=lambda i: (got[i] - share[i], i))[:rows - sum(got)]:
        got[i] += 1
    return got


def _sizes(case):
    """Tensor lengths spread evenly (over their logarithm) from the smallest to the largest."""
    t, lo, hi = case["tensors"], case["smallest"], case["largest"]
    return [int(round(lo * (hi / lo) ** (i / max(1, t - 1)))) for i in range(t)]


def _to_fp8(x):
    """Codes and scales of a flat fp32 tensor: per 128 elements, scale = amax / 448 (1 where amax is
    0), codes rounded to nearest even."""
    pad = -x.numel() % BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).view(-1, BLOCK)
    amax = b.abs().amax(1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, FP8_MAX))
    q = (b / scale[:, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q.view(-1)[:x.numel()], scale


def _root_to_fp8(r):
    """As _to_fp8 for roots of the second moment: one that is not zero gets at least the smallest code."""
    q, scale = _to_fp8(r)
    bits = q.contiguous().view(torch.uint8)
    bits = torch.where((r > 0) & (bits == 0), torch.ones_like(bits), bits)
    return bits.view(torch.float8_e4m3fn), scale


def _from_fp8(q, scale):
    pad = -q.numel() % BLOCK
    b = torch.nn.functional.pad(q.float(), (0, pad)).view(-1, BLOCK)
    return (b * scale[:, None]).view(-1)[:q.numel()]


def _flat(sizes, unit, dtype, values=None):
    """One buffer for all tensors of a kind, each starting at a multiple of `unit` elements, and the
    tensors as views of it (the padding between them is zero)."""
    starts, end = [], 0
    for s in sizes:
        starts.append(end)
        end += -(-s // unit) * unit
    buf = torch.zeros(end, dtype=dtype, device="cuda")
    views = [buf[a:a + s] for a, s in zip(starts, sizes)]
    for i in range(len(sizes)):
        if values is not None:
            views[i].copy_(values(i))
    return buf, views


def _adamw_inputs(case, gen):
    """What a training program holds of one parameter group, in flat buffers per kind: 32-bit or BF16
    weights, gradients, both moments, and the 16-bit copies that the products read."""
    sizes = _sizes(case)

    def normal(n, scale):
        return torch.randn(n, device="cuda", generator=gen) * scale

    def spread(i):
        return 2.0 ** -(i % 5)          # gradients' sizes differ from tensor to tensor

    def moment(i):                      # of a run under way: of the gradients' order, smaller
        return normal(sizes[i], 3e-4 * spread(i))

    def root(i):                        # root of the second moment, some elements near zero
        return (normal(sizes[i], 7e-4 * spread(i)).square() + (3e-5 * spread(i)) ** 2).sqrt()

    buf, view = {}, {}
    buf["params"], view["params"] = _flat(sizes, 16, DTYPES[case["param"]], lambda i: normal(sizes[i], 0.02))
    buf["grads"], view["grads"] = _flat(sizes, 16, DTYPES[case["grad"]], lambda i: normal(sizes[i], 1e-3 * spread(i)))
    if case["copy"] != "none":
        buf["copies"], view["copies"] = _flat(sizes, 16, DTYPES[case["copy"]], lambda i: view["params"][i])
    if case["states"] == "fp8":
        blocks = [-(-s // BLOCK) for s in sizes]
        for name, value, cast in (("m", moment, _to_fp8), ("v", root, _root_to_fp8)):
            buf[name], view[name] = _flat(sizes, 16, torch.float8_e4m3fn)
            buf[name + "_scale"], view[name + "_scale"] = _flat(blocks, 4, torch.float32)
            for i in range(len(sizes)):
                q, scale = cast(value(i))
                view[name][i].copy_(q)
                view[name + "_scale"][i].copy_(scale)
    else:
        buf["m"], view["m"] = _flat(sizes, 16, torch.float32, moment)
        buf["v"], view["v"] = _flat(sizes, 16, torch.float32, lambda i: root(i).square())
    return {"case": dict(case), "step": FIRST_STEP, "buf": buf, **view}


def _product_inputs(case, gen, seed):
    """The operands of a product grouped by expert: tokens sorted by expert, the segments' offsets
    (and their lengths, as a plain program would hold them), weights, and the output's buffer."""
    rows, g, n, k, t = case["rows"], case["groups"], case["n"], case["k"], DTYPES[case["dtype"]]
    counts = _counts(case)
    counts = [counts[i] for i in torch.randperm(g, generator=torch.Generator().manual_seed(seed)).tolist()]
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * scale

    state = {"case": dict(case), "counts": counts, "offsets": offsets}
    if case["op"] != "nn":              # activations of unit size with a few wide columns
        wide = 1.0 + 7.0 * (torch.rand(k, device="cuda", generator=gen) < 0.01)
        state["x"] = (normal(rows, k) * wide).to(t)
    if case["op"] != "nt":
        state["dy"] = normal(rows, n, scale=0.01).to(t)
    if case["op"] != "tn":
        state["w"] = torch.stack([normal(n, k, scale=k ** -0.5).to(t) for _ in range(g)])
        state["out"] = torch.zeros(rows, n if case["op"] == "nt" else k, dtype=t, device="cuda")
    else:
        kind = t if case["out"] == "same" else torch.float32
        state["out"] = torch.stack([normal(n, k, scale=0.01).to(kind) for _ in range(g)])
    return state


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return _adamw_inputs(case, gen) if case["op"] == "adamw" else _product_inputs(case, gen, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    if own and case["op"] == "adamw":   # the table of tensors, laid out once for a parameter group
        import fp8_block_scaled_e4m3_amd as dg
        state["plan"] = dg.dg_adamw_plan(state["params"], state["grads"], state["m"], state["v"],
                                         state.get("m_scale"), state.get("v_scale"), state.get("copies"))
    return state


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "adamw":
        state["step"] += 1
        _adamw_own(state) if own else _adamw_plain(state)
        return {key: x for key, x in state["buf"].items() if key != "grads"}
    _product_own(state) if own else _product_plain(state)
    return state["out"]


def _product_own(state):
    import fp8_block_scaled_e4m3_amd as dg
    op, out, offsets = state["case"]["op"], state["out"], state["offsets"]
    if op == "nt":
        dg.dg_m_grouped_gemm_ragged_nt(state["x"], state["w"], out, offsets)
    elif op == "nn":
        dg.dg_m_grouped_gemm_ragged_nn(state["dy"], state["w"], out, offsets)
    else:
        dg.dg_k_grouped_gemm_ragged_tn(state["dy"], state["x"], out, offsets, accumulate=state["case"]["add"])


def _product_plain(state):
    case, counts, out = state["case"], state["counts"], state["out"]
    if case["op"] == "nt":
        parts = [x.float() @ w.float().t() for x, w in zip(state["x"].split(counts), state["w"]) if len(x)]
        out.copy_(torch.cat(parts))
    elif case["op"] == "nn":
        parts = [y.float() @ w.float() for y, w in zip(state["dy"].split(counts), state["w"]) if len(y)]
        out.copy_(torch.cat(parts))
    else:
        parts = [y.float().t() @ x.float() for y, x in zip(state["dy"].split(counts), state["x"].split(counts))]
        out.copy_(torch.stack(parts) + out.float() if case["add"] else torch.stack(parts))


def _adamw_own(state):
    import fp8_block_scaled_e4m3_amd as dg
    dg.dg_adamw_step(state["plan"], state["step"], LR, BETA1, BETA2, EPS, DECAY)


def _adamw_plain(state):
    t = state["step"]
    root2 = 1.0 / math.sqrt(1.0 - BETA2 ** t)
    size = LR / (1.0 - BETA1 ** t)
    for i, p in enumerate(state["params"]):
        g = state["grads"][i].float()
        if "m_scale" in state:
            m = _from_fp8(state["m"][i], state["m_scale"][i])
            v = _from_fp8(state["v"][i], state["v_scale"][i])
            v = v * v
        else:
            m, v = state["m"][i], state["v"][i]
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + (g * g) * (1.0 - BETA2)
        r = v.sqrt()
        new = p.float() * (1.0 - LR * DECAY) - (m / (r * root2 + EPS)) * size
        p.copy_(new)
        if "copies" in state:
            state["copies"][i].copy_(new)
        if "m_scale" in state:
            m, state["m_scale"][i][:] = _to_fp8(m)
            v, state["v_scale"][i][:] = _root_to_fp8(r)
        state["m"][i].copy_(m)
        state["v"][i].copy_(v)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    if case["op"] == "adamw":
        elements = sum(_sizes(case))
        size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
        # weights read and written, gradient read, copy written, two states read and written
        each = 2 * size[case["param"]] + size[case["grad"]] + size[case["copy"]]
        each += 16 if case["states"] == "f32" else 4 + 16 / BLOCK
        return {"bytes": elements * each, "flops": elements * 16}
    rows, n, k = case["rows"], case["n"], case["k"]
    flops = 2.0 * rows * n * k
    if case["op"] == "tn":
        out = case["groups"] * n * k * (2 if case["out"] == "same" else 4)
        return {"bytes": rows * (n + k) * 2 + out * (2 if case["add"] else 1), "flops": flops}
    used = sum(c > 0 for c in _counts(case))
    return {"bytes": rows * (n + k) * 2 + used * n * k * 2, "flops": flops}


# ---- the results in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    state = _inputs(case, seed)
    return _exact_adamw(state) if case["op"] == "adamw" else _exact_product(state)


def _exact_product(state):
    case, out = state["case"], state["out"].double()
    at = 0
    for e, c in enumerate(state["counts"]):
        rows = slice(at, at + c)
        at += c
        if case["op"] == "nt":
            out[rows] = torch.matmul(state["x"][rows].double(), state["w"][e].double().T)
        elif case["op"] == "nn":
            out[rows] = torch.matmul(state["dy"][rows].double(), state["w"][e].double())
        else:
            if not case["add"]:
                out[e] = 0
            out[e] += torch.matmul(state["dy"][rows].double().T, state["x"][rows].double())
    return out


def _exact_adamw(state):
    """The definition, tensor by tensor; the codes of an 8-bit state as the unrounded quotients they
    stand for (their scales being the blocks' largest magnitudes over 448)."""
    t = FIRST_STEP + 1
    res = {key: b.double() for key, b in state["buf"].items() if key != "grads"}

    def place(key, i, value):
        start = state[key][i].storage_offset()
        res[key][start:start + value.numel()] = value

    def blocks(x):
        return torch.cat([x, x.new_zeros(-x.numel() % BLOCK)]).view(-1, BLOCK)

    def load(key, i):
        x = state[key][i].double()
        if "m_scale" not in state:
            return x
        x = (blocks(x) * state[key + "_scale"][i].double()[:, None]).reshape(-1)[:x.numel()]
        return x if key == "m" else x ** 2

    def store(key, i, x):
        if "m_scale" in state:
            b = blocks(x if key == "m" else x.sqrt())
            amax = b.abs().max(dim=1).values
            scale = torch.where(amax > 0, amax / FP8_MAX, 1.0)
            place(key + "_scale", i, scale)
            x = (b / scale[:, None]).reshape(-1)[:x.numel()]
        place(key, i, x)

    for i in range(len(state["params"])):
        g, m, v = state["grads"][i].double(), load("m", i), load("v", i)
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        mhat, vhat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        p = state["params"][i].double()
        p = p - LR * DECAY * p - LR * mhat / (vhat.sqrt() + EPS)
        place("params", i, p)
        if "copies" in state:
            place("copies", i, p)
        store("m", i, m)
        store("v", i, v)
    return res
