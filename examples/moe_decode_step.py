"""A decoder block, one step of a batch, with random weights. Its attention half: residual addition and norm to e4m3
codes, the product that gives queries, keys and values, rotary positions and the paged cache's write, attention of the
new tokens over the cache, and the output's product. Its mixture-of-experts half: residual addition and norm, the
router's choice, and the chosen experts.

    python examples/moe_decode_step.py [--tokens 1 8 64] [--experts 32] [--hidden 7168] [--width 2048] [--top-k 8]
                                       [--heads 64] [--kv-heads 8] [--context 4096]

prints the time of each half for each batch (one new token a sequence) and how far its output is from the same half in
64 bits.
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


def value(codes, scales):
    """Codes [N, K] and 128x128 scales in 64 bits."""
    return codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


class AttentionBlock:
    """Weights, paged cache and workspace of one block's attention half. `step` takes the new tokens of a batch of
    sequences, one or many each: decoding, chunks of prompts, or both."""

    def __init__(self, hidden, heads, kv_heads, pages, page_size, max_tokens, max_batch, head_dim=128, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=g, device=device)  # noqa: E731
        self.heads, self.kv_heads, self.head_dim, self.page_size = heads, kv_heads, head_dim, page_size
        self.norm = (1 + 0.1 * normal(hidden)).to(torch.bfloat16)
        self.w_qkv, self.s_qkv = quantize_128x128(normal((heads + 2 * kv_heads) * head_dim, hidden) * hidden ** -0.5)
        self.w_out, self.s_out = quantize_128x128(normal(hidden, heads * head_dim) * (heads * head_dim) ** -0.5)
        self.freqs, self.factor = dg.dg_rope_frequencies(head_dim, device=device)
        # Keys and values are halves of each page.
        codes = torch.zeros((pages, 2, page_size, kv_heads, head_dim), dtype=torch.uint8, device=device)
        scales = torch.ones((pages, 2, page_size, kv_heads), device=device)
        self.cache = codes[:, 0], scales[:, 0], codes[:, 1], scales[:, 1]
        self.workspace = dg.workspace(dg.dg_fp8_paged_attention_workspace_bytes(max_tokens, max_batch, heads, kv_heads,
                                                                               head_dim, max_tokens), device)

    def attend(self, x, residual, slots, positions, table, kv_lens, q_starts, longest):
        """Up to the attention's output [T, heads, head_dim]; also the rotated queries."""
        q8, s, _, _ = dg.dg_fp8_rmsnorm_quantize_1x128(x, self.norm, 1e-6, residual=residual, residual_out=residual)
        qkv = dg.dg_fp8_gemm_nt(q8, s, self.w_qkv, self.s_qkv).view(len(x), -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        dg.dg_fp8_rope_cache_write(k, v, *self.cache, slots, positions, self.freqs, q=q, factor=self.factor, q_out=q)
        return dg.dg_fp8_paged_attention(q, *self.cache, table, kv_lens, q_starts, longest, self.workspace), q

    def step(self, x, residual, slots, positions, table, kv_lens, q_starts, longest):
        """x [T, hidden] bf16: what the block before adds to the residual stream [T, hidden] (updated in place); the
        tokens' slots and positions; the pages and lengths of the sequences, the new tokens among them. Returns what
        the mixture-of-experts half adds."""
        o, _ = self.attend(x, residual, slots, positions, table, kv_lens, q_starts, longest)
        return dg.dg_fp8_gemm_nt(*dg.dg_fp8_quantize_1x128(o.flatten(1)), self.w_out, self.s_out)

    def reference(self, q, table, kv_lens, q_starts):
        """Attention of the rotated queries over what the cache holds, in 64 bits, and the weighted sum of the values'
        magnitudes."""
        out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        size = torch.zeros_like(out)
        starts = q_starts.tolist()
        for b, n in enumerate(kv_lens.tolist()):
            rows = slice(starts[b], starts[b + 1])
            j = torch.arange(n, device=q.device)
            slots = table[b].long()[j // self.page_size] * self.page_size + j % self.page_size
            k, v = (dg.dg_fp8_cache_read(c, s, slots, dtype=torch.float32).double().transpose(0, 1).repeat_interleave(
                self.heads // self.kv_heads, 0) for c, s in (self.cache[:2], self.cache[2:]))
            x = q[rows].double().transpose(0, 1) @ k.transpose(1, 2).contiguous() * self.head_dim ** -0.5
            m = starts[b + 1] - starts[b]
            x = x.masked_fill(j > torch.arange(n - m, n, device=q.device)[:, None], float("-inf"))
            p = torch.softmax(x, 2)
            out[rows], size[rows] = (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1)
        return out, size

    def fill(self, table, lengths, seed=1):
        """Random keys and values for the first tokens of each sequence."""
        g = torch.Generator(device=table.device).manual_seed(seed)
        for b, n in enumerate(lengths):
            j = torch.arange(n, device=table.device)
            slots = table[b].long()[j // self.page_size] * self.page_size + j % self.page_size
            kv = torch.randn((2, n, self.kv_heads, self.head_dim), generator=g, device=table.device)
            dg.dg_fp8_rope_cache_write(kv[0], kv[1], *self.cache, slots, j.int(), self.freqs, factor=self.factor)


def batch_of(table, page_size, new, lengths):
    """What a step takes beside its rows, for sequences with so many new tokens of so many."""
    device = table.device
    positions = [torch.arange(n - m, n, device=device) for m, n in zip(new, lengths)]
    slots = torch.cat([table[b].long()[j // page_size] * page_size + j % page_size for b, j in enumerate(positions)])
    starts = torch.tensor([0, *new], device=device).cumsum(0).int()
    return dict(slots=slots, positions=torch.cat(positions).int(), table=table,
                kv_lens=torch.tensor(lengths, dtype=torch.int32, device=device), q_starts=starts, longest=max(new))


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
        a = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)
        out = torch.zeros_like(a)
        for e in ids.unique().tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            g, u = (a[t] @ value(self.w13[e], self.s13[e]).t()).chunk(2, 1)
            h = g * torch.sigmoid(g) * u
            out.index_add_(0, t, weights[t, j, None].double() * (h @ value(self.w2[e], self.s2[e]).t()))
        return out


def timed(step):
    """Microseconds of a step."""
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for n in (10, 100):                # warm up, then time
        start.record()
        for _ in range(n):
            step()
        end.record()
        end.synchronize()
    return start.elapsed_time(end) * 10


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 8, 64])
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--page-size", type=int, default=64)
    args = ap.parse_args()
    most, width = max(args.tokens), -(-args.context // args.page_size)
    block = MoeBlock(args.hidden, args.width, args.experts, args.top_k, most)
    attention = AttentionBlock(args.hidden, args.heads, args.kv_heads, most * width, args.page_size, most, most)
    table = torch.randperm(most * width, device="cuda").int().view(most, width)
    attention.fill(table, [args.context] * most)
    for T in args.tokens:
        x = torch.randn((T, args.hidden), device="cuda").to(torch.bfloat16)
        residual = torch.randn((T, args.hidden), device="cuda").to(torch.bfloat16)
        batch = batch_of(table[:T], args.page_size, [1] * T, [args.context] * T)
        o, q = attention.attend(x, residual.clone(), **batch)
        exact, _ = attention.reference(q, batch["table"], batch["kv_lens"], batch["q_starts"])
        off = float((o.double() - exact).norm() / exact.norm())
        print("%3d tokens: attention %8.1f us a step, %.4f from 64 bits" % (
            T, timed(lambda: attention.step(x, residual, **batch)), off))
        residual = torch.randn((T, args.hidden), device="cuda").to(torch.bfloat16)
        exact = block.reference(x, residual)
        off = float((block.step(x, residual.clone()).double() - exact).norm() / exact.norm())
        print("            experts   %8.1f us a step, %.4f from 64 bits" % (timed(lambda: block.step(x, residual)), off))


if __name__ == "__main__":
    main()
