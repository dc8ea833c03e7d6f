"""One expert block in microscaled formats, as a decoder layer would run it:

    residual + RMS norm  ->  router on the 16-bit rows  ->  4-bit experts on the
    8-bit rows  ->  the next layer's residual addition

    python examples/mx_moe_block.py [--tokens T] [--bits 4|8]

Weights are random; the block's output is compared with the same block in
float32 on the dequantised weights, so the figure printed is what the 8- or
4-bit rows cost.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_quantized_moe_gb300 as mq  # noqa: E402


class MxMoeBlock:
    """Norm weight, router and 4-bit experts of one block, with its workspace."""

    def __init__(self, E=8, k=2, H=2048, I=1408, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.E, self.k, self.H, self.I = E, k, H, I
        self.norm = torch.ones(H, dtype=torch.bfloat16, device=device)
        self.gate = torch.randn(E, H, generator=g, device=device, dtype=torch.bfloat16) * 0.05
        w13 = torch.randn(E, 2 * I, H, generator=g, device=device, dtype=torch.bfloat16) * 0.03
        w2 = torch.randn(E, H, I, generator=g, device=device, dtype=torch.bfloat16) * 0.03
        self.w13, self.s13 = mq.moe_quantize_mx(w13, bits=4)   # once, at load time
        self.w2, self.s2 = mq.moe_quantize_mx(w2, bits=4)
        self.workspace = None

    def __call__(self, x, residual, bits=8):
        """(x + residual, expert output) for bf16 rows [T, H]."""
        T = x.shape[0]
        need = mq.moe_mx_forward_workspace(T, self.H, self.I, self.E, self.k, bits)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        q, scale, residual, y = mq.moe_rmsnorm_mx(x, self.norm, residual=residual, bits=bits,
                                                  want_y=True)
        topk_w, topk_ids = mq.moe_topk_route((y @ self.gate.T).float(), self.k, True)
        out = mq.moe_mx_forward(q, scale, self.w13, self.s13, self.w2, self.s2, topk_w, topk_ids,
                                a_bits=bits, workspace=self.workspace)
        return residual, out

    def reference(self, x, residual):
        """The same block in float32 on the dequantised weights."""
        h = x.float() + residual.float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)
        topk_w, topk_ids = mq.moe_topk_route((y.to(torch.bfloat16) @ self.gate.T).float(), self.k, True)
        w13 = mq.moe_dequantize_mx(self.w13, self.s13, bits=4, dtype=torch.float32)
        w2 = mq.moe_dequantize_mx(self.w2, self.s2, bits=4, dtype=torch.float32)
        out = torch.zeros_like(h)
        for e in range(self.E):
            t, j = torch.nonzero(topk_ids == e, as_tuple=True)
            u = y[t] @ w13[e].T
            act = torch.nn.functional.silu(u[:, :self.I]) * u[:, self.I:]
            out.index_add_(0, t, (act @ w2[e].T) * topk_w[t, j, None])
        return out


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--bits", type=int, default=8, choices=(4, 8))
    args = p.parse_args(argv)
    block = MxMoeBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual = (torch.randn(args.tokens, block.H, generator=g, device="cuda").to(torch.bfloat16)
                   for _ in range(2))
    _, out = block(x, residual, bits=args.bits)
    ref = block.reference(x, residual)
    torch.cuda.synchronize()
    if mq.mq_device_status() != 0:
        raise RuntimeError("device status set")
    err = ((out.float() - ref).square().mean().sqrt() / ref.square().mean().sqrt()).item()
    print(f"{args.tokens} tokens, {args.bits}-bit rows: rms difference {err:.4f} of the float32 block's rms")
    return err


if __name__ == "__main__":
    main()
