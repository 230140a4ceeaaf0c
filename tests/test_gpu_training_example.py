"""The training operators together, as examples/train_experts.py uses them."""
import pytest

from tests.gpu_support import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


@pytest.mark.parametrize("states", ["e4m3", "f32"])
def test_training_lowers_the_loss_and_serves_in_fp8(states):
    """Forty steps at least halve the loss (the last five against the first five, which differ by
    their batches).  An E4M3 code is off by 2^-4 of its value at most, about 2^-5.3 in the mean
    square; a product's two operands make that 2^-4.8 of its size, two products in a row with the
    square between them (which doubles the first's) sqrt(4 + 1) 2^-4.8 = 0.08.  Twice that is
    allowed."""
    import torch

    from examples import train_experts as example
    layer, losses = example.train(steps=40, states=states, say=lambda *a: None)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5]), (losses[:5], losses[-5:])
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, offsets = example.route(torch.randn(500, 256, device="cuda", generator=gen).to(torch.bfloat16), 8, gen)
    y, y8 = layer.forward(x, offsets)[2].float(), example.serve_fp8(layer, x, offsets).float()
    assert float((y8 - y).norm() / y.norm()) < 0.16


def test_states_of_8_bits_follow_those_of_32():
    """The same run with either states: after twenty steps the losses differ by less than a tenth."""
    from examples import train_experts as example
    last = [example.train(steps=20, states=s, say=lambda *a: None)[1][-1] for s in ("e4m3", "f32")]
    assert abs(last[0] - last[1]) < 0.1 * last[1], last


def test_layer_gradients_agree_with_automatic_ones():
    """Input and weight gradients of the whole layer against torch's, in fp32 on the CPU from the same
    BF16 weights.  BF16 roundings of h, z, y, dz and dh (2^-9 in the mean square each, five in a
    row, the square's doubled) stay under 2^-6 of a gradient's norm."""
    import torch

    from examples import train_experts as example
    layer = example.Experts(3, 128, 256, "f32", 4)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, offsets = example.route(torch.randn(300, 128, device="cuda", generator=gen).to(torch.bfloat16), 3, gen)
    dy = torch.randn(300, 128, device="cuda", generator=gen).to(torch.bfloat16)
    h, z, _ = layer.forward(x, offsets)
    dx = layer.backward(x, offsets, h, z, dy, first=True)
    w = [v.float().cpu().requires_grad_() for v in layer.weights]
    xc = x.float().cpu().requires_grad_()
    at = offsets.tolist()
    y = torch.cat([(xc[a:b] @ w[0][e].T).clamp(min=0).square() @ w[1][e].T for e, (a, b) in enumerate(zip(at, at[1:]))])
    y.backward(dy.float().cpu())
    for got, want in ((dx, xc.grad), (layer.grads[0], w[0].grad), (layer.grads[1], w[1].grad)):
        assert float((got.float().cpu() - want).norm() / want.norm()) < 2.0 ** -6
