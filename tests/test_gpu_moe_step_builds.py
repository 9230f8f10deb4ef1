"""The serving step's operators: the release library against its -O1 -g build, and a hundred repeats, bit for bit
(a race on LDS, or a wait that holds for one instruction schedule only, shows up as a difference). Every result is
held to the 64-bit form too, and nothing beside the outputs is written."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_sa_amd import ops
from tests.check import assert_close
from tests.gpu_util import GUARD, bits, guards_intact, sentinel_bf16
from tests.test_gpu_debug_build import both, debug_lib  # noqa: F401
from tests.test_gpu_moe_step import BF16, F32, check_gate, check_norm, layer_reference, make_layer, normal, to_bf16_bits

gpu = pytest.mark.gpu

# Every tile of both layer kernels: passes of 1, 2 and 4 tiles of tokens (gate and up), of 1 to 4 of pairs (down),
# waves without a K block (H 128 to 384), whole and partial chunks of I, grids by pair and by expert.
LAYERS = [(1, 1, 1, 128, 128, "distinct"), (1, 8, 32, 1024, 512, "distinct"), (8, 16, 16, 384, 640, "distinct"),
          (16, 4, 4, 640, 384, "distinct"), (24, 2, 2, 256, 1152, "distinct"), (32, 2, 3, 512, 256, "one"),
          (45, 3, 4, 896, 128, "distinct"), (64, 2, 2, 512, 384, "distinct"), (64, 16, 24, 256, 256, "sparse"),
          (40, 5, 9, 256, 256, "repeated")]
NORMS = [(1, 128, BF16, BF16, BF16), (70, 1152, F32, F32, BF16), (9, 2048, BF16, F32, F32), (5, 4224, BF16, BF16, BF16),
         (33, 7168, BF16, BF16, BF16), (3, 8320, F32, None, F32), (2, 32896, BF16, BF16, F32), (1, 65536, F32, F32, F32)]
GATES = [(1, 16, 1, F32), (37, 33, 5, BF16), (64, 96, 6, F32), (19, 256, 8, BF16), (50, 300, 10, F32), (6, 1024, 16, F32)]


def layer_once(a, ws, out):
    """The layer into out from a workspace of NaN bytes: nothing in it may come from an earlier call."""
    ws.fill_(0xFF)
    ops.dg_fp8_moe_layer(*a, ws, out=out)


def layer_case(T, k, E, H, I, ids):  # noqa: E741
    a = make_layer(T, k, E, H, I, 500 + T + k, ids)
    return a, ops.workspace(ops.dg_fp8_moe_layer_workspace_bytes(T, k, H, I)), sentinel_bf16((T, H))


@gpu
@pytest.mark.parametrize("T,k,E,H,I,ids", LAYERS)
def test_layer_release_equals_O1(gpu_device, debug_lib, T, k, E, H, I, ids):  # noqa: F811,E741
    a, ws, out = layer_case(T, k, E, H, I, ids)

    def run():
        layer_once(a, ws, out)
        torch.cuda.synchronize()
        return bits(out)        # and looks at the bands around out
    rel, dbg = both(debug_lib, run)
    assert np.array_equal(rel, dbg), "-O1 build differs from the release build"
    assert_close(rel, to_bf16_bits(layer_reference(*a)), "layer")


@gpu
@pytest.mark.parametrize("T,k,E,H,I,ids", LAYERS)
def test_layer_repeats(gpu_device, T, k, E, H, I, ids):  # noqa: E741
    a, ws, out = layer_case(T, k, E, H, I, ids)
    layer_once(a, ws, out)
    first = out.clone()
    for r in range(100):
        layer_once(a, ws, out)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), "repeat %d differs" % r
    assert guards_intact(out)


def norm_case(M, K, xt, rt, wt):
    x, w = normal((M, K), M + K).to(xt), (1 + 0.3 * normal((K,), 2, False)).to(wt)
    return x, w, None if rt is None else (3 * normal((M, K), 3)).to(rt)


def same(a, b):
    return all((x is None and y is None) or torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


@gpu
@pytest.mark.parametrize("M,K,xt,rt,wt", NORMS)
def test_norm_release_equals_O1_and_repeats(gpu_device, debug_lib, M, K, xt, rt, wt):  # noqa: F811
    x, w, r = norm_case(M, K, xt, rt, wt)
    d = [x.cuda(), w.cuda(), None if r is None else r.cuda()]

    def run():
        return ops.dg_fp8_rmsnorm_quantize_1x128(d[0], d[1], 1e-5, residual=d[2], normed=True)
    rel, dbg = both(debug_lib, run)
    assert same(rel, dbg), "-O1 build differs from the release build"
    for i in range(100):
        assert same(rel, run()), "repeat %d differs" % i
    check_norm(x, w, 1e-5, r, *rel)


@gpu
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                               ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k,dtype", GATES)
def test_gate_release_equals_O1_and_repeats(gpu_device, debug_lib, T, E, k, dtype, score, renormalize):  # noqa: F811
    logits = (3 * normal((T, E), E + k, False)).to(dtype)
    logits[::5, ::3] = -float("inf")
    d = logits.cuda()

    def run():
        return ops.dg_moe_gate_topk(d, k, score=score, renormalize=renormalize)
    rel, dbg = both(debug_lib, run)
    assert same(rel, dbg), "-O1 build differs from the release build"
    for i in range(100):
        assert same(rel, run()), "repeat %d differs" % i
    check_gate(logits, k, score, renormalize)


# ---------------------------------------------------------------- the guard bands themselves, on the host

@pytest.mark.parametrize("at", [None, 0, GUARD - 1, GUARD, GUARD + 255, GUARD + 256, 2 * GUARD + 255])
def test_guard_bands_see_a_write(monkeypatch, at):
    """A value written into a band around an output of 256 elements is seen, one inside the output is not a fault."""
    full = torch.full
    monkeypatch.setattr(torch, "full", lambda *a, device=None, **kw: full(*a, **kw))
    out = sentinel_bf16((2, 128))
    whole = torch.empty(0, dtype=torch.int16).set_(out.untyped_storage())
    assert whole.numel() == 2 * GUARD + 256
    if at is not None:
        whole[at] = 0
    assert guards_intact(out) == (at is None or GUARD <= at < GUARD + 256)
