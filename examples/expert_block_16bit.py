"""An expert block with 16-bit weights: a training step, and serving with adapters of
several requests beside the same weights.

    router  ->  token-slots in expert order  ->  gate/up product (+ adapters)  ->
    SiLU and multiply  ->  down product (+ adapters)  ->  router-weighted sum

    python examples/expert_block_16bit.py [--tokens T]

Training goes through autograd (moe_grouped_product); serving adds each request's
adapters in place (moe_lora_product), here to both products.  The figures printed are the
block's differences from the same block in float64.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_quantized_moe_gb300 as mq  # noqa: E402


def silu_and_mul(h):
    gate, up = h.float().chunk(2, dim=-1)
    return torch.nn.functional.silu(gate) * up


class ExpertBlock:
    """Experts [E, 2I, H] and [E, H, I] in bf16, and L adapters of rank r for each product
    of each expert."""

    def __init__(self, E=8, k=2, H=256, I=384, L=3, r=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.E, self.k, self.H, self.I = E, k, H, I

        def weights(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)
        self.w13 = weights(E, 2 * I, H, scale=H ** -0.5)
        self.w2 = weights(E, H, I, scale=I ** -0.5)
        self.lora13 = (weights(L, E, r, H, scale=H ** -0.5), weights(L, E, 2 * I, r, scale=0.5 * r ** -0.5))
        self.lora2 = (weights(L, E, r, I, scale=I ** -0.5), weights(L, E, H, r, scale=0.5 * r ** -0.5))
        self.scaling = torch.full((L,), 0.5, device=device)

    def route(self, logits):
        """(slots in expert order, first slot of each expert, weights of the tokens' slots)."""
        topk_w, topk_ids = mq.moe_topk_route(logits, self.k, True)
        order, _, offsets, _ = mq.moe_align_block(topk_ids, self.E, 1)
        return order[:topk_ids.numel()].long(), offsets, topk_w

    def __call__(self, x, logits, adapter_ids=None):
        """x bf16 [T, H], logits float32 [T, E], adapter_ids int32 [T] or None."""
        order, offsets, topk_w = self.route(logits)
        token = order // self.k
        rows = x[token]                             # (its gradient sums a token's slots)
        h = mq.moe_grouped_product(rows, self.w13, offsets)
        if adapter_ids is not None:
            ids = adapter_ids[token]
            mq.moe_lora_product(rows, *self.lora13, ids, base=h, expert_offsets=offsets, scaling=self.scaling, out=h)
        act = silu_and_mul(h).to(x.dtype)
        y = mq.moe_grouped_product(act, self.w2, offsets, out_dtype=torch.float32)
        if adapter_ids is not None:
            mq.moe_lora_product(act, *self.lora2, ids, base=y, expert_offsets=offsets, scaling=self.scaling, out=y)
        weighted = y * topk_w.reshape(-1)[order, None]
        return torch.zeros(x.shape, device=x.device).index_add(0, token, weighted)

    def reference(self, x, logits, adapter_ids=None, w13=None, w2=None):
        """The same block in float64; x, w13 and w2 may be leaves."""
        d = lambda t: t.double()  # noqa: E731
        order, offsets, topk_w = self.route(logits)
        w13, w2 = d(self.w13) if w13 is None else w13, d(self.w2) if w2 is None else w2
        out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        at = offsets.tolist()

        def project(rows, w, adapters, e, l):
            y = rows @ w[e].T
            if l >= 0:
                y = y + float(self.scaling[l]) * (rows @ d(adapters[0][l, e]).T) @ d(adapters[1][l, e]).T
            return y
        for e in range(self.E):
            slots = order[at[e]:at[e + 1]]
            ids = torch.full_like(slots, -1) if adapter_ids is None else adapter_ids[slots // self.k].long()
            for l in ids.unique().tolist():
                some = slots[ids == l]
                h = project(d(x[some // self.k]), w13, self.lora13, e, l)
                act = torch.nn.functional.silu(h[:, :self.I]) * h[:, self.I:]
                y = project(act, w2, self.lora2, e, l)
                out = out.index_add(0, some // self.k, y * d(topk_w).reshape(-1)[some, None])
        return out


def difference(got, want):
    """Root mean square of the difference over that of what is wanted."""
    return ((got.double() - want).square().mean().sqrt() / want.square().mean().sqrt()).item()


def train(block, x, logits, target):
    """Gradients (of x, w13, w2) of the mean squared error of one step, and float64's."""
    found = []
    for leaves, run in (((x.clone(), block.w13, block.w2), block), ((x.double(), block.w13.double(), block.w2.double()), None)):
        a, w13, w2 = (t.detach().requires_grad_() for t in leaves)
        if run is None:
            out = block.reference(a, logits, w13=w13, w2=w2)
        else:
            kept = block.w13, block.w2
            block.w13, block.w2 = w13, w2
            out = block(a, logits)
            block.w13, block.w2 = kept
        loss = (out - target.to(out.dtype)).square().mean() * 1000
        found.append(torch.autograd.grad(loss, (a, w13, w2)))
    return found


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=200)
    args = p.parse_args(argv)
    block = ExpertBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(args.tokens, block.H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(args.tokens, block.E, generator=g, device="cuda")
    target = torch.randn(args.tokens, block.H, generator=g, device="cuda")
    # requests of 20 tokens each, on adapters 0, 1, 2 and none in turn
    ids = (torch.arange(args.tokens, device="cuda") // 20 % 4).to(torch.int32)
    ids[ids == 3] = -1
    with torch.no_grad():
        plain = difference(block(x, logits), block.reference(x, logits))
        adapted = difference(block(x, logits, ids), block.reference(x, logits, ids))
    got, want = train(block, x, logits, target)
    grads = [difference(a, b) for a, b in zip(got, want)]
    torch.cuda.synchronize()
    if mq.mq_device_status() != 0:
        raise RuntimeError("device status set")
    print(f"{args.tokens} tokens: difference from float64 {plain:.4f}, with adapters {adapted:.4f}; "
          "gradients of rows, gate/up and down weights " + " ".join(f"{v:.4f}" for v in grads))
    return [plain, adapted, *grads]


if __name__ == "__main__":
    main()
