"""The 16-bit operators together, as a layer uses them: router, alignment, both products
with adapters of several requests, and a training step (the example's block), and adapters
beside the quantised product."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples", "expert_block_16bit.py")
    spec = importlib.util.spec_from_file_location("expert_block_16bit", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# Each bf16 rounding on the way is off by at most half a step, 2^-8 of its value, evenly
# spread and so 2^-8 / sqrt(3) in root mean square at most (of a value's upper end).  A
# forward rounds the gate/up sums (twice with adapters) and the activation; a gradient
# passes at most twice as many: dy, the activation's, the gate/up sums' and its own.  Errors
# of independent roundings add in squares; they pass SiLU, whose derivative is at most
# 1.1, and products that neither raise nor lower a relative rms: times 2 for both.
STEP = 2.0 ** -8 / 3 ** 0.5
FORWARD, GRADIENT = 2 * 3 ** 0.5 * STEP, 2 * 6 ** 0.5 * STEP


@pytest.mark.parametrize("tokens", [1, 7, 200, 700])
def test_block(example, tokens):
    plain, adapted, *grads = example.main(["--tokens", str(tokens)])
    assert plain < FORWARD and adapted < FORWARD
    assert all(g < GRADIENT for g in grads)


def test_gradients_against_differences(example):
    """The block's gradients along a direction of each leaf against central differences
    of the float64 block."""
    b = example.ExpertBlock(E=4, k=2, H=64, I=64)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(40, 64, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(40, 4, generator=g, device="cuda")
    target = torch.randn(40, 64, generator=g, device="cuda")
    got, _ = example.train(b, x, logits, target)
    leaves = [x.double(), b.w13.double(), b.w2.double()]

    def loss(x64, w13, w2):
        return ((b.reference(x64, logits, w13=w13, w2=w2) - target.double()).square().mean() * 1000).item()
    for i, grad in enumerate(got):
        d = grad.double() / grad.double().norm()      # (along the gradient itself: nothing cancels)
        h = 1e-4 * leaves[i].norm().item()
        up = loss(*[t + h * d if j == i else t for j, t in enumerate(leaves)])
        down = loss(*[t - h * d if j == i else t for j, t in enumerate(leaves)])
        want = (up - down) / (2 * h)
        assert abs(grad.double().norm().item() - want) < GRADIENT * abs(want) + 1e-6 * abs(up)


def test_adapters_beside_a_quantised_product():
    """A 4-bit dense product on 8-bit rows with float32 results, and the adapters of 16-bit
    rows added to it in place: one rounding at the end."""
    import weight_quantized_moe_gb300 as mq
    T, K, N, r, L = 33, 256, 200, 16, 4
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(N, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    a = (torch.randn(L, r, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    b = torch.randn(L, N, r, generator=g).to(torch.bfloat16).cuda()
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32).cuda()
    q, s = mq.moe_quantize_mx(x, bits=8)
    qw, sw = mq.moe_quantize_mx(w, bits=4)
    base = mq.moe_mx_product(q, s, qw, sw, out_dtype=torch.float32)
    got = mq.moe_lora_product(x, a, b, ids, base=base.clone())
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0
    want = base.double()
    for t in range(T):
        l = int(ids[t])
        if l >= 0:
            want[t] += b[l].double() @ (a[l].double() @ x[t].double())
    mag = (b.double().abs().amax(0) @ (a.double().abs().amax(0) @ x.double().abs().T)).T
    assert ((got.double() - want).abs() <= (K + r + 2) * 2.0 ** -23 * mag + 2.0 ** -23 * want.abs()).all()
    assert torch.equal(got[ids == -1], base[ids == -1])
