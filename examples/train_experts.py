"""Train the experts of a small mixture-of-experts layer with the library's training operators, then
serve the trained weights through its FP8 products.

The layer sends every token to one expert, y = W2[e] f(W1[e] x) with f(h) = max(h, 0)^2.  A step is

* forward: tokens sorted by expert, the two products at the segments that routing gives
  (dg_m_grouped_gemm_ragged_nt);
* backward: both input gradients (dg_m_grouped_gemm_ragged_nn) and both weight gradients, added up
  over micro-batches in fp32 (dg_k_grouped_gemm_ragged_tn);
* AdamW on fp32 weights with 8-bit or fp32 states, which also writes the BF16 copies that the next
  forward pass reads (dg_adamw_plan, dg_adamw_step).

The task is synthetic: the experts learn another, fixed set of experts.  Afterwards the weights are
cast to E4M3 with 128x128 scales and the layer runs on the contiguous grouped FP8 product.

    python examples/train_experts.py [--steps N] [--states e4m3|f32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_e4m3_amd as dg  # noqa: E402


def activation(h):
    return h.float().clamp(min=0).square().to(h.dtype)


def activation_gradient(h, dz):
    return (2 * h.float().clamp(min=0) * dz.float()).to(h.dtype)


class Experts:
    """Weights of the layer: fp32, with the BF16 copies the products read, gradients and states."""

    def __init__(self, experts, hidden, inner, states, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shapes = [(experts, inner, hidden), (experts, hidden, inner)]
        self.master = [torch.randn(s, device="cuda", generator=gen) * s[2] ** -0.5 for s in shapes]
        self.weights = [w.to(torch.bfloat16) for w in self.master]
        self.grads = [torch.zeros_like(w) for w in self.master]
        self.step_count = 0
        if states == "e4m3":
            kind, scales = torch.float8_e4m3fn, [torch.ones(-(-w.numel() // 128), device="cuda") for w in self.master]
            self.scales = [scales, [s.clone() for s in scales]]
        else:
            kind, self.scales = torch.float32, [None, None]
        self.moments = [[torch.zeros(w.shape, device="cuda").to(kind) for w in self.master] for _ in range(2)]
        self.plan = dg.dg_adamw_plan(self.master, self.grads, self.moments[0], self.moments[1], self.scales[0],
                                     self.scales[1], self.weights)

    def forward(self, x, offsets):
        w1, w2 = self.weights
        h = torch.empty(x.shape[0], w1.shape[1], dtype=x.dtype, device="cuda")
        dg.dg_m_grouped_gemm_ragged_nt(x, w1, h, offsets)
        z = activation(h)
        y = torch.empty_like(x)
        dg.dg_m_grouped_gemm_ragged_nt(z, w2, y, offsets)
        return h, z, y

    def backward(self, x, offsets, h, z, dy, first):
        """Adds the gradients of this micro-batch to the weights' (replaces them with the first's);
        returns the input's."""
        w1, w2 = self.weights
        dz, dx = torch.empty_like(z), torch.empty_like(x)
        dg.dg_k_grouped_gemm_ragged_tn(dy, z, self.grads[1], offsets, accumulate=not first)
        dg.dg_m_grouped_gemm_ragged_nn(dy, w2, dz, offsets)
        dh = activation_gradient(h, dz)
        dg.dg_k_grouped_gemm_ragged_tn(dh, x, self.grads[0], offsets, accumulate=not first)
        dg.dg_m_grouped_gemm_ragged_nn(dh, w1, dx, offsets)
        return dx

    def update(self, lr):
        self.step_count += 1
        dg.dg_adamw_step(self.plan, self.step_count, lr, beta1=0.9, beta2=0.95, weight_decay=0.0)


def route(tokens, experts, gen):
    """A skewed assignment of tokens to experts: the tokens sorted by expert, and the offsets."""
    share = 1.0 / torch.arange(1, experts + 1, device="cuda", dtype=torch.float32)
    chosen = torch.multinomial(share, tokens.shape[0], replacement=True, generator=gen)
    order = torch.argsort(chosen, stable=True)
    counts = torch.bincount(chosen, minlength=experts)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return tokens[order], offsets


def train(steps=60, states="e4m3", experts=8, hidden=256, inner=512, tokens=1000, micro_batches=2, lr=2e-3, seed=0,
          say=print):
    """The trained layer and the loss of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, student = Experts(experts, hidden, inner, states, 1), Experts(experts, hidden, inner, states, 2)
    losses = []
    for step in range(steps):
        total = 0.0
        for part in range(micro_batches):
            x, offsets = route(torch.randn(tokens, hidden, device="cuda", generator=gen).to(torch.bfloat16), experts, gen)
            want = teacher.forward(x, offsets)[2]
            h, z, y = student.forward(x, offsets)
            error = y.float() - want.float()
            total = total + error.square().mean() / micro_batches
            dy = (error * (2.0 / (error.numel() * micro_batches))).to(torch.bfloat16)
            student.backward(x, offsets, h, z, dy, first=part == 0)
        student.update(lr)
        losses.append(total)
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step}: loss {float(total):.5f}")
    return student, [float(x) for x in losses]


def to_fp8_rows(x):
    """Activations in E4M3 with 1x128 scales."""
    q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(x.shape[1] // 128, dg.dg_get_aligned_ld_sa(x.shape[0]), device="cuda")
    dg.dg_quantize_fp8_1x128(x, q, scales)
    return q, scales


def to_fp8_weights(w):
    """Weights [experts, N, K] in E4M3 with 128x128 scales."""
    q = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(w.shape[0], -(-w.shape[1] // 128), w.shape[2] // 128, device="cuda")
    for e in range(w.shape[0]):
        dg.dg_quantize_fp8_128x128(w[e], q[e], scales[e])
    return q, scales


def serve_fp8(layer, x, offsets):
    """The layer on the FP8 grouped product: segments padded to the library's alignment."""
    align = dg.dg_get_m_alignment()
    counts = offsets.diff().tolist()
    first = offsets.tolist()
    padded = [-(-c // align) * align for c in counts]
    rows = torch.zeros(sum(padded), x.shape[1], dtype=x.dtype, device="cuda")
    indices = torch.full((sum(padded),), -1, dtype=torch.int32, device="cuda")
    at, places = 0, []
    for e, (c, p) in enumerate(zip(counts, padded)):
        rows[at:at + c] = x[first[e]:first[e] + c]
        indices[at:at + c] = e
        places.append(torch.arange(at, at + c, device="cuda"))
        at += p
    z = rows
    for i, w in enumerate(layer.weights):
        (a, sa), (b, sb) = to_fp8_rows(z), to_fp8_weights(w)
        out = torch.zeros(rows.shape[0], w.shape[1], dtype=torch.bfloat16, device="cuda")
        dg.dg_m_grouped_gemm_fp8_contiguous(a, sa, b, sb, out, indices)
        z = activation(out) if i == 0 else out
    return z[torch.cat(places)]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--states", choices=["e4m3", "f32"], default="e4m3")
    args = ap.parse_args()
    layer, _ = train(args.steps, args.states)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, offsets = route(torch.randn(500, 256, device="cuda", generator=gen).to(torch.bfloat16), 8, gen)
    y, y8 = layer.forward(x, offsets)[2].float(), serve_fp8(layer, x, offsets).float()
    print(f"served in FP8: relative error {float((y8 - y).norm() / y.norm()):.3f} against the BF16 layer")


if __name__ == "__main__":
    main()
