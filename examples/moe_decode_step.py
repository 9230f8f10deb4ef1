"""The mixture-of-experts half of a decoder block, one decode step of a batch: residual addition and norm to e4m3
codes, the router's choice, and the chosen experts, with random weights.

    python examples/moe_decode_step.py [--tokens 1 8 64] [--experts 32] [--hidden 7168] [--width 2048] [--top-k 8]

prints the time of a step for each batch and how far its output is from the same step in 64 bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_sa_amd as dg  # noqa: E402


def quantize_128x128(w):
    """e4m3 codes and 128x128 scales (amax / 448) of weights [N, K]."""
    N, K = w.shape
    blocks = w.view(N // 128, 128, K // 128, 128)
    scales = blocks.abs().amax((1, 3)) / 448
    codes = (blocks / scales[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(N, K), scales


class MoeBlock:
    """Weights and workspace of one block; `step` is what a serving loop calls for each token batch."""

    def __init__(self, hidden, width, experts, top_k, max_tokens, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=g, device=device)  # noqa: E731
        self.top_k = top_k
        self.norm = (1 + 0.1 * normal(hidden)).to(torch.bfloat16)
        self.router = (normal(hidden, experts) * hidden ** -0.5).to(torch.bfloat16)

        def stack(n, k):
            parts = [quantize_128x128(normal(n, k) * k ** -0.5) for _ in range(experts)]
            return torch.stack([p[0].view(torch.uint8) for p in parts]), torch.stack([p[1] for p in parts])

        self.w13, self.s13 = stack(2 * width, hidden)     # gate rows, then up rows
        self.w2, self.s2 = stack(hidden, width)
        self.workspace = dg.workspace(dg.dg_fp8_moe_layer_workspace_bytes(max_tokens, top_k, hidden, width), device)

    def step(self, x, residual):
        """x [T, hidden] bf16: what the attention half adds to the residual stream [T, hidden] (updated in place).
        Returns what the next block adds to it."""
        q, s, _, y = dg.dg_fp8_rmsnorm_quantize_1x128(x, self.norm, 1e-6, residual=residual, residual_out=residual,
                                                      normed=True)
        ids, weights = dg.dg_moe_gate_topk(y @ self.router, self.top_k)
        return dg.dg_fp8_moe_layer(q, s, self.w13, self.s13, self.w2, self.s2, ids, weights, self.workspace)

    def reference(self, x, residual):
        """The step in 64 bits from the same codes of the activations and the same choice of experts."""
        q, s, _, y = dg.dg_fp8_rmsnorm_quantize_1x128(x, self.norm, 1e-6, residual=residual, normed=True)
        ids, weights = dg.dg_moe_gate_topk(y @ self.router, self.top_k)
        value = lambda codes, scales: (codes.view(torch.float8_e4m3fn).double()  # noqa: E731
                                       * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1))
        a = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)
        out = torch.zeros_like(a)
        for e in ids.unique().tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            g, u = (a[t] @ value(self.w13[e], self.s13[e]).t()).chunk(2, 1)
            h = g * torch.sigmoid(g) * u
            out.index_add_(0, t, weights[t, j, None].double() * (h @ value(self.w2[e], self.s2[e]).t()))
        return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 8, 64])
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--top-k", type=int, default=8)
    args = ap.parse_args()
    block = MoeBlock(args.hidden, args.width, args.experts, args.top_k, max(args.tokens))
    for T in args.tokens:
        x = torch.randn((T, args.hidden), device="cuda").to(torch.bfloat16)
        residual = torch.randn((T, args.hidden), device="cuda").to(torch.bfloat16)
        exact = block.reference(x, residual)
        out = block.step(x, residual.clone())
        off = float((out.double() - exact).norm() / exact.norm())
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for n in (10, 100):                # warm up, then time
            start.record()
            for _ in range(n):
                block.step(x, residual)
            end.record()
            end.synchronize()
        print("%3d tokens: %8.1f us a step, output %.4f from 64 bits" % (T, start.elapsed_time(end) * 10, off))


if __name__ == "__main__":
    main()
