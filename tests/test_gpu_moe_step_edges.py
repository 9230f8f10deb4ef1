"""The serving step's operators on the GPU at the borders of their ranges."""
import math

import numpy as np
import pytest
import torch

from fp8_block_scaled_sa_amd import ops
from tests.check import assert_close
from tests.gpu_util import bits
from tests.test_gpu_moe_step import (BF16, F8, check_norm, layer_reference, make_layer, normal, run_layer,
                                     to_bf16_bits)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- layer: the two parts of h at the end of bf16's range

# h = (0x1.FE + c 2^-8) 2^127: bf16's largest number for c = 0, from c = 1 on
# nearer to 2^128 than to it (or as near), past fp32's range for c = 4.
PARTS = [0.0, 0.5, 0.875, 1.0, 1.125, 1.875, 4.0]


def layer_at_the_border(T):
    """One expert, h_0 = +-(0x1.FE + c 2^-8) 2^127 and h_1 = -+0x1.FE 2^127, each a product of g = 2^64 (where
    silu(g) is g) and u; even rows of W2 take h_0, odd ones h_0 + h_1, all times 2^-100. Every sum is exact."""
    H, I = 384, 128  # noqa: E741
    c = torch.tensor(PARTS).repeat_interleave(2).repeat(T)[:T]
    sign = torch.tensor([1.0, -1.0]).repeat(T)[:T]
    x = torch.zeros((T, H))
    x[:, 0], x[:, 1], x[:, 129], x[:, 257] = 1, sign, sign, sign * c
    sx = torch.tensor([2.0 ** 32, 2.0 ** 28, 2.0 ** 24]).expand(T, 3).contiguous()
    w13 = torch.zeros((1, 2 * I, H))
    w13[0, :2, 0] = 1                                               # g
    w13[0, I, 1], w13[0, I, 129], w13[0, I, 257] = 1.875, 1.875, 1  # 1.875 (1 + 2^-4) = 0x1.FE
    w13[0, I + 1, 1], w13[0, I + 1, 129] = -1.875, -1.875
    s13 = torch.tensor([2.0 ** 32, 2.0 ** 31])[None, :, None].expand(1, 2, 3).contiguous()
    w2 = torch.zeros((1, H, I))
    w2[0, :, 0], w2[0, 1::2, 1] = 1, 1
    code = lambda v: v.to(F8).view(torch.uint8)  # noqa: E731
    a = [t.cuda() for t in (code(x), sx, code(w13), s13, code(w2), torch.full((1, 3, 1), 2.0 ** -100),
                            torch.zeros((T, 1), dtype=torch.int32), torch.ones((T, 1)))]
    # in fp64; bf16 of it is one rounding (the sums have at most 12 bits)
    h0 = torch.where(c >= 4, math.inf, (0x1FE / 256 + c.double() / 256) * 2.0 ** 127)
    even, odd = sign * h0 * 2.0 ** -100, sign * (h0 - 0x1FE / 256 * 2.0 ** 127) * 2.0 ** -100
    ref = torch.stack([even, odd], 1).repeat(1, H // 2).float().to(BF16)
    return a, ref


@pytest.mark.parametrize("T", [1, 8, 14, 33, 64])
def test_layer_h_at_the_end_of_bf16(gpu_device, T):
    a, ref = layer_at_the_border(T)
    got = bits(run_layer(a))
    # a zero's sign is that of the sum's order
    assert np.array_equal(np.where(got == 0x8000, 0, got), np.where(bits(ref) == 0x8000, 0, bits(ref)))


# ---------------------------------------------------------------- outputs on a stream that is not the current one

def step_calls(side):
    """Each operator on small inputs with new outputs on stream side, as functions."""
    a = make_layer(4, 2, 4, 512, 256, 7)
    x = torch.ones((4, 512), dtype=BF16, device="cuda")
    w = torch.ones(512, dtype=BF16, device="cuda")
    logits = torch.zeros((4, 8), device="cuda")
    ws = ops.workspace(ops.dg_fp8_moe_layer_workspace_bytes(4, 2, 512, 256))
    return [lambda: ops.dg_fp8_rmsnorm_quantize_1x128(x, w, residual=x, normed=True, stream=side),
            lambda: ops.dg_moe_gate_topk(logits, 2, stream=side),
            lambda: ops.dg_fp8_moe_layer(*a, ws, stream=side),
            lambda: ops.dg_fp8_quantize_1x128(x, stream=side)]


def blocks(out):
    """Size and address of each output."""
    return [(t.numel() * t.element_size(), t.data_ptr()) for t in (out if isinstance(out, tuple) else (out,))]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("raw", [False, True])
def test_outputs_dropped_while_their_stream_works(gpu_device, which, raw):
    """Outputs that are dropped before the kernel has run are not handed out to the current stream."""
    side = torch.cuda.Stream()
    call = step_calls(side.cuda_stream if raw else side)[which]
    side.wait_stream(torch.cuda.current_stream())
    call()                       # memory of both streams' pools is there
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    out = call()
    held = blocks(out)
    del out
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n, _ in held for _ in range(4)]
    assert not {t.data_ptr() for t in new} & {at for _, at in held}
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", range(4))
def test_outputs_dropped_while_the_current_stream_reads(gpu_device, which):
    """Nor are outputs that the current stream has still to read handed out to their own stream."""
    side = torch.cuda.Stream()
    call = step_calls(side)[which]
    side.wait_stream(torch.cuda.current_stream())
    call()
    torch.cuda.synchronize()
    out = call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    held = blocks(out)
    del out
    with torch.cuda.stream(side):
        new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n, _ in held for _ in range(4)]
    assert not {t.data_ptr() for t in new} & {at for _, at in held}
    torch.cuda.synchronize()


# ---------------------------------------------------------------- the largest launches

def test_norm_most_rows(gpu_device):
    M, K = 2 ** 26 - 4, 128
    x = torch.empty((M, K), dtype=BF16, device="cuda")
    ends = torch.cat([torch.arange(5), torch.arange(M - 5, M)]).cuda()
    x[ends] = normal((10, K), 7).to(BF16).cuda()
    w = torch.ones(K, dtype=BF16, device="cuda")
    q, s, _, _ = ops.dg_fp8_rmsnorm_quantize_1x128(x, w)
    q2, s2, _, _ = ops.dg_fp8_rmsnorm_quantize_1x128(x[ends], w)
    assert torch.equal(q[ends], q2) and torch.equal(s[ends], s2)


def test_gate_most_tokens(gpu_device):
    logits = torch.zeros((2 ** 28 - 16, 1), dtype=BF16, device="cuda")
    ids = torch.full((2 ** 28 - 16, 1), 7, dtype=torch.int32, device="cuda")
    ops.dg_moe_gate_topk(logits, 1, ids=ids)
    assert not ids.any()


# ---------------------------------------------------------------- layer: tiles by the number of tokens

@pytest.mark.parametrize("T,k,E,ids", [(8, 16, 24, "distinct"), (7, 16, 5, "repeated"), (8, 9, 3, "one"),
                                       (9, 7, 9, "one"), (16, 4, 40, "distinct"), (17, 3, 4, "one"),
                                       (32, 2, 2, "distinct"), (33, 1, 2, "one"), (64, 1, 100, "distinct")])
def test_layer_tiles(gpu_device, T, k, E, ids):
    a = make_layer(T, k, E, 256, 384, 300 + T + k, ids)
    assert_close(bits(run_layer(a)), to_bf16_bits(layer_reference(*a)), "layer")


# ---------------------------------------------------------------- norm: the ends of the range of its squares

@pytest.mark.parametrize("K", [128, 1152, 8320])
@pytest.mark.parametrize("exponent", [-62, -40, 40, 56])
def test_norm_small_and_large_rows(gpu_device, K, exponent):
    """Without an eps, the rows' size falls out of the norm: as exact at both ends of what the header names."""
    x = normal((5, K), K, False).clamp(-3, 3)
    x[:, 0] = 1                                      # the largest value is at least that
    x = x * 2.0 ** exponent
    w = 1 + 0.1 * normal((K,), 2, False)
    q, s, _, y = ops.dg_fp8_rmsnorm_quantize_1x128(x.cuda(), w.cuda(), 0.0, normed=True)
    check_norm(x, w, 0.0, None, q, s, None, y)


def test_norm_past_the_ends(gpu_device):
    x = torch.ones((3, 256))
    x[0] *= 2.0 ** 64                                # squares add up to more than fp32 holds
    x[1] *= 2.0 ** -80                               # and to nothing
    q, s, _, y = ops.dg_fp8_rmsnorm_quantize_1x128(x.cuda(), torch.ones(256, device="cuda"), 0.0, normed=True)
    assert not q[0].any() and bool((s[0] == 1).all()) and not y[0].any()
    assert bool((y[1] == math.inf).all()) and bool((y[2] == 1).all())


def test_layer_far_negative_gate(gpu_device):
    """g = -128: exp(-g) is infinite, silu(g) is -0, and so is every product with it: no NaN."""
    H, I = 128, 128  # noqa: E741
    code = lambda v, *s: torch.full(s, float(v)).to(F8).view(torch.uint8)  # noqa: E731
    w13 = torch.cat([code(-1, 1, I, H), code(1, 1, I, H)], 1)
    a = [t.cuda() for t in (code(1, 2, H), torch.ones((2, 1)), w13, torch.ones((1, 2, 1)), code(1, 1, H, I),
                            torch.ones((1, 1, 1)), torch.zeros((2, 1), dtype=torch.int32), torch.ones((2, 1)))]
    assert bool((run_layer(a) == 0).all())
