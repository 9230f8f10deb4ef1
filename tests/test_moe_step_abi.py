"""The serving step's operators (residual norm to codes, router top-k, expert
layer) reject bad arguments on the host, through the C ABI and through the
Python binding; none of these calls reaches a device."""
import ctypes
import os
import re
import sys

import pytest
import torch

from fp8_block_scaled_sa_amd import DGError, _lib, ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dg_fp8.h")

OK, NULL, SHAPE, MISALIGNED, STRIDE, UNSUPPORTED, HIP, ALIASING, SCRATCH = range(9)
GOT_TO_THE_DEVICE = (OK, UNSUPPORTED, HIP)

# Fake, never-dereferenced addresses that do not overlap.
X, R, RO, W, Y, Q, S, W2, S2, IDS, WTS, WS, OUT = (0x10000000 * (i + 1) for i in range(13))


def norm(**kw):
    args = dict(X=X, xt=1, ldx=512, R=R, rt=1, ldr=512, RO=RO, ldro=512, W=W, wt=1, eps=1e-6, Y=Y, ldy=512,
                Q=Q, ldq=512, S=S, s_m=1, s_kb=64, M=64, K=512, stream=None)
    args.update(kw)
    return _lib.load().dg_fp8_rmsnorm_quantize_1x128(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(K=500), SHAPE), (dict(K=0), SHAPE), (dict(M=-1), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE),
    (dict(xt=2), UNSUPPORTED), (dict(rt=-1), UNSUPPORTED), (dict(wt=7), UNSUPPORTED), (dict(M=2 ** 31), UNSUPPORTED),
    (dict(K=65664, ldx=65664, ldr=65664, ldro=65664, ldy=65664, ldq=65664), UNSUPPORTED),
    (dict(ldx=2 ** 28 + 16), UNSUPPORTED), (dict(M=2 ** 26), UNSUPPORTED),
    (dict(M=2 ** 24, K=1152, ldx=1152, ldr=1152, ldro=1152, ldy=1152, ldq=1152), UNSUPPORTED),
    (dict(M=2 ** 22, K=8320, ldx=8320, ldr=8320, ldro=8320, ldy=8320, ldq=8320), UNSUPPORTED),
    (dict(X=None), NULL), (dict(W=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL), (dict(RO=None), NULL),
    (dict(ldx=504), STRIDE), (dict(ldr=256), STRIDE), (dict(ldro=256), STRIDE), (dict(ldy=256), STRIDE),
    (dict(ldq=496), STRIDE), (dict(s_m=-1), STRIDE), (dict(s_m=0), STRIDE), (dict(s_m=1, s_kb=32), STRIDE),
    (dict(s_m=3, s_kb=1), STRIDE),
    (dict(X=X + 8), MISALIGNED), (dict(R=R + 2), MISALIGNED), (dict(RO=RO + 8), MISALIGNED),
    (dict(W=W + 4), MISALIGNED), (dict(Y=Y + 2), MISALIGNED), (dict(Q=Q + 8), MISALIGNED), (dict(S=S + 2), MISALIGNED),
    (dict(ldx=516), MISALIGNED), (dict(ldr=516), MISALIGNED), (dict(ldy=516), MISALIGNED), (dict(ldq=520), MISALIGNED),
    (dict(RO=X), ALIASING), (dict(RO=R, ldro=520), ALIASING), (dict(RO=R + 512), ALIASING), (dict(Y=X), ALIASING),
    (dict(Q=R), ALIASING), (dict(S=W), ALIASING), (dict(Y=RO), ALIASING), (dict(S=Q + 512), ALIASING),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def test_norm_accepted_and_empty():
    assert norm(M=0, X=None, W=None, Q=None, S=None) == OK
    for kw in (dict(), dict(R=None, RO=None, rt=0, ldr=0, ldro=0), dict(Y=None, ldy=0), dict(RO=R),
               dict(xt=0, rt=0, wt=0), dict(s_m=4, s_kb=1), dict(eps=0.0)):
        assert norm(**kw) in GOT_TO_THE_DEVICE


def gate(**kw):
    args = dict(logits=X, lt=0, ldl=256, score=0, renorm=1, factor=1.0, ids=IDS, weights=WTS, T=64, E=256, k=8,
                stream=None)
    args.update(kw)
    return _lib.load().dg_moe_gate_topk(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(k=9, E=8), SHAPE),
    (dict(E=1025, ldl=1025), UNSUPPORTED), (dict(k=17), UNSUPPORTED), (dict(lt=2), UNSUPPORTED),
    (dict(score=2), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED), (dict(ldl=2 ** 29), UNSUPPORTED),
    (dict(T=2 ** 28), UNSUPPORTED),
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL),
    (dict(ldl=255), STRIDE),
    (dict(logits=X + 2), MISALIGNED), (dict(ids=IDS + 2), MISALIGNED), (dict(weights=WTS + 1), MISALIGNED),
    (dict(ids=X + 1024), ALIASING), (dict(weights=X), ALIASING), (dict(weights=IDS), ALIASING),
])
def test_gate_refusals(kw, status):
    assert gate(**kw) == status


def test_gate_accepted_and_empty():
    assert gate(T=0, logits=None, ids=None, weights=None) == OK
    for kw in (dict(), dict(lt=1, logits=X + 2), dict(score=1, renorm=0), dict(E=1, k=1), dict(E=1024, ldl=1024, k=16)):
        assert gate(**kw) in GOT_TO_THE_DEVICE


def ws_bytes(T, k, H, I):  # noqa: E741
    return _lib.load().dg_fp8_moe_layer_workspace_bytes(T, k, H, I)


def layer(**kw):
    E, H, I = 4, 512, 256  # noqa: E741
    args = dict(X=X, ldx=H, sX=S, sx_m=1, sx_kb=8, W13=W, ld13=H, w13_e=2 * I * H, s13=Y, s13_e=16, s13_nb=4, s13_kb=1,
                W2=W2, ld2=I, w2_e=H * I, s2=S2, s2_e=8, s2_nb=2, s2_kb=1, ids=IDS, wts=WTS, out=OUT, ldo=H,
                T=8, k=2, E=E, H=H, I=I, ws=WS, ws_bytes=ws_bytes(8, 2, H, I), stream=None)
    args.update(kw)
    return _lib.load().dg_fp8_moe_layer(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(E=0), SHAPE), (dict(H=500), SHAPE), (dict(I=200), SHAPE),
    (dict(I=0), SHAPE),
    (dict(T=65), UNSUPPORTED), (dict(k=17), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
    (dict(H=2 ** 18 + 128, ldx=2 ** 21, ld13=2 ** 21, ldo=2 ** 21), UNSUPPORTED),
    (dict(ld13=2 ** 25 + 16, w13_e=2 ** 40), UNSUPPORTED), (dict(sx_m=2 ** 22 + 1), UNSUPPORTED),
    (dict(ldo=2 ** 25 + 8), UNSUPPORTED), (dict(w2_e=2 ** 51), UNSUPPORTED),
    (dict(sx_kb=2 ** 29), UNSUPPORTED), (dict(T=64, k=16, E=1024, I=2 ** 18), UNSUPPORTED),
] + [(dict([(n, None)]), NULL) for n in ("X", "sX", "W13", "s13", "W2", "s2", "ids", "wts", "out", "ws")] + [
    (dict(ldx=256), STRIDE), (dict(ld13=496), STRIDE), (dict(ld2=128), STRIDE), (dict(ldo=256), STRIDE),
    (dict(w13_e=512 * 512 - 16), STRIDE), (dict(w2_e=512 * 256 - 16), STRIDE), (dict(w2_e=0), STRIDE),
    (dict(sx_m=-1), STRIDE), (dict(s13_nb=-4), STRIDE), (dict(s2_e=-1), STRIDE),
    (dict(X=X + 8), MISALIGNED), (dict(W13=W + 1), MISALIGNED), (dict(W2=W2 + 8), MISALIGNED),
    (dict(out=OUT + 8), MISALIGNED), (dict(ws=WS + 8), MISALIGNED), (dict(sX=S + 2), MISALIGNED),
    (dict(ids=IDS + 2), MISALIGNED), (dict(wts=WTS + 2), MISALIGNED), (dict(ldx=520), MISALIGNED),
    (dict(ld13=520, w13_e=512 * 520), MISALIGNED), (dict(ldo=516), MISALIGNED), (dict(w2_e=512 * 256 + 8), MISALIGNED),
    (dict(ws_bytes=ws_bytes(8, 2, 512, 256) - 1), SCRATCH), (dict(ws_bytes=0), SCRATCH), (dict(ws_bytes=-1), SCRATCH),
    (dict(out=X), ALIASING), (dict(out=W + 4096), ALIASING), (dict(out=IDS), ALIASING), (dict(ws=OUT), ALIASING),
    (dict(ws=X), ALIASING), (dict(ws=WTS - 4096), ALIASING), (dict(out=S2), ALIASING),
])
def test_layer_refusals(kw, status):
    assert layer(**kw) == status


def test_layer_accepted_and_empty():
    assert layer(T=0, X=None, ids=None, ws=None) == OK
    for kw in (dict(), dict(E=1, w13_e=0, w2_e=0), dict(s13_e=0, s13_nb=0, s13_kb=0), dict(T=64, k=4, ws_bytes=1 << 20)):
        assert layer(**kw) in GOT_TO_THE_DEVICE


def test_layer_workspace_bytes():
    assert ops.dg_fp8_moe_layer_workspace_bytes(64, 8, 7168, 2048) >= 64 * 8 * (7168 + 2048) * 4
    assert ops.dg_fp8_moe_layer_workspace_bytes(0, 8, 7168, 2048) == 0
    for bad, status in (((65, 8, 7168, 2048), UNSUPPORTED), ((1, 8, 7168, 200), SHAPE), ((-1, 1, 128, 128), SHAPE)):
        with pytest.raises(DGError) as e:
            ops.dg_fp8_moe_layer_workspace_bytes(*bad)
        assert e.value.status == status


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        ops.dg_fp8_rmsnorm_quantize_1x128(x, w)
    with pytest.raises(TypeError):
        ops.dg_fp8_rmsnorm_quantize_1x128(x.half(), w)
    with pytest.raises(ValueError):
        ops.dg_fp8_rmsnorm_quantize_1x128(x, w[:128])
    with pytest.raises(ValueError):
        ops.dg_fp8_rmsnorm_quantize_1x128(x, w, residual=x[:3])
    with pytest.raises(TypeError):
        ops.dg_fp8_rmsnorm_quantize_1x128(x, w, residual=x, residual_out=x.float())
    with pytest.raises(ValueError):
        ops.dg_fp8_rmsnorm_quantize_1x128(x, w, residual_out=x)
    with pytest.raises(ValueError):
        ops.dg_fp8_rmsnorm_quantize_1x128(x.t(), w)

    logits = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="device"):
        ops.dg_moe_gate_topk(logits, 2)
    with pytest.raises(TypeError):
        ops.dg_moe_gate_topk(logits.double(), 2)
    with pytest.raises(ValueError):
        ops.dg_moe_gate_topk(logits, 2, score="tanh")
    with pytest.raises(ValueError):
        ops.dg_moe_gate_topk(logits, 2, ids=torch.zeros((4, 3), dtype=torch.int32))

    code = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    good = dict(x=code(4, 256), sx=torch.ones(4, 2), w13=code(3, 256, 256), s13=torch.ones(3, 2, 2),
                w2=code(3, 256, 128), s2=torch.ones(3, 2, 1), topk_ids=torch.zeros((4, 2), dtype=torch.int32),
                topk_weights=torch.ones(4, 2), workspace=None)
    for name, bad in (("x", code(4, 128)), ("w13", code(3, 384, 256)), ("w2", code(2, 256, 128)),
                      ("sx", torch.ones(4, 1)), ("s13", torch.ones(3, 1, 2)), ("s2", torch.ones(3, 2, 2)),
                      ("topk_ids", torch.zeros(8, dtype=torch.int32)), ("workspace", code(65536)), ("x", code(4, 256))):
        with pytest.raises(ValueError):
            ops.dg_fp8_moe_layer(**{**good, name: bad})
    for name in ("x", "w13", "sx"):
        with pytest.raises(TypeError):
            ops.dg_fp8_moe_layer(**{**good, name: good[name].double()})


def parameters(name):
    """Parameter names of an entry point, from the header."""
    text = re.search(r"^dg_status %s\((.*?)\);" % name, open(HEADER).read(), re.M | re.S).group(1)
    return [p.split()[-1].lstrip("*") for p in text.split(",")]


@pytest.fixture
def recorded(monkeypatch):
    """Calls of the binding on host tensors, as {parameter: argument} by the header's names."""
    calls = []
    kept = []

    def entry(name):
        names = parameters(name)
        res, types = _lib.SIGNATURES[name]
        assert len(names) == len(types)

        def call(*args):
            calls.append(dict(zip(names, args)))
            return OK
        kept.append(ctypes.CFUNCTYPE(res, *types)(call))
        return ctypes.cast(kept[-1], ctypes.c_void_p).value

    class Library:
        _addresses = {n: entry(n) for n in ("dg_fp8_rmsnorm_quantize_1x128", "dg_moe_gate_topk", "dg_fp8_moe_layer")}

    monkeypatch.setattr(_lib, "_lib", Library())
    ops._binding().any_device(True)
    yield calls
    ops._binding().any_device(False)


def test_norm_binding_passes_every_argument_by_its_name(recorded):
    M, K = 3, 512
    x = torch.zeros((M, K + 8), dtype=torch.bfloat16)[:, :K]
    r, w = torch.zeros((M, K + 4))[:, :K], torch.ones(K, dtype=torch.bfloat16)
    q, s, ro, y = ops.dg_fp8_rmsnorm_quantize_1x128(x, w, 0.25, residual=r, normed=True, stream=77)
    assert recorded.pop() == dict(
        X=x.data_ptr(), x_dtype=1, ldx=K + 8, R=r.data_ptr(), r_dtype=0, ldr=K + 4, R_out=ro.data_ptr(), ldro=K,
        W=w.data_ptr(), w_dtype=1, eps=0.25, Y=y.data_ptr(), ldy=K, Q=q.data_ptr(), ldq=K, S=s.data_ptr(),
        s_stride_m=1, s_stride_kb=M, M=M, K=K, stream=77)
    assert [(t.dtype, tuple(t.shape), t.stride()) for t in (q, s, ro, y)] == [
        (torch.uint8, (M, K), (K, 1)), (torch.float32, (M, 4), (1, M)), (torch.float32, (M, K), (K, 1)),
        (torch.bfloat16, (M, K), (K, 1))]
    given = dict(q=torch.zeros((M, K + 16), dtype=torch.uint8)[:, :K], s=torch.zeros((M, 6))[:, :4],
                 y=torch.zeros((M, K + 24), dtype=torch.bfloat16)[:, :K])
    out = ops.dg_fp8_rmsnorm_quantize_1x128(x, w, residual=r, residual_out=r, stream=1, **given)
    assert out[0] is given["q"] and out[1] is given["s"] and out[2] is r and out[3] is given["y"]
    c = recorded.pop()
    assert (c["ldq"], c["s_stride_m"], c["s_stride_kb"], c["ldy"], c["ldro"], c["R_out"]) == (
        K + 16, 6, 1, K + 24, K + 4, r.data_ptr())
    assert ops.dg_fp8_rmsnorm_quantize_1x128(x, w, stream=1)[2:] == (None, None)
    c = recorded.pop()
    assert c["R"] is None and c["R_out"] is None and c["Y"] is None
    # a single row's stride means nothing in torch
    ops.dg_fp8_rmsnorm_quantize_1x128(torch.zeros((K, 1), dtype=torch.bfloat16).t(), w, stream=1)
    assert recorded.pop()["ldx"] == K


def test_gate_binding_passes_every_argument_by_its_name(recorded):
    logits = torch.zeros((5, 40))[:, :32]
    ids, weights = ops.dg_moe_gate_topk(logits, 4, score="sigmoid", renormalize=False, factor=2.5, stream=3)
    assert recorded.pop() == dict(logits=logits.data_ptr(), l_dtype=0, ldl=40, score=1, renormalize=0, factor=2.5,
                                  ids=ids.data_ptr(), weights=weights.data_ptr(), T=5, E=32, top_k=4, stream=3)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    assert tuple(ids.shape) == tuple(weights.shape) == (5, 4) and ids.is_contiguous() and weights.is_contiguous()


def test_layer_binding_passes_every_argument_by_its_name(recorded):
    T, k, E, H, I = 3, 2, 4, 256, 384  # noqa: E741
    code = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x, sx = code(T, H + 16)[:, :H], torch.zeros((2, T)).t()
    w13, s13 = code(E, 2 * I + 1, H + 32)[:, :2 * I, :H], torch.zeros((E, 7, 2))[:, :6]
    w2, s2 = code(E, H + 2, I + 48)[:, :H, :I], torch.zeros((E, 3, 2)).transpose(1, 2)
    ids, weights, ws = torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, k)), code(100)
    out = ops.dg_fp8_moe_layer(x, sx, w13, s13, w2, s2, ids, weights, ws, stream=9)
    assert recorded.pop() == dict(
        X=x.data_ptr(), ldx=H + 16, sX=sx.data_ptr(), sx_stride_m=1, sx_stride_kb=T,
        W13=w13.data_ptr(), ld13=H + 32, w13_stride_e=(2 * I + 1) * (H + 32), s13=s13.data_ptr(), s13_stride_e=14,
        s13_stride_nb=2, s13_stride_kb=1, W2=w2.data_ptr(), ld2=I + 48, w2_stride_e=(H + 2) * (I + 48),
        s2=s2.data_ptr(), s2_stride_e=6, s2_stride_nb=1, s2_stride_kb=2, topk_ids=ids.data_ptr(),
        topk_weights=weights.data_ptr(), out=out.data_ptr(), ldo=H, T=T, top_k=k, E=E, H=H, I=I,
        workspace=ws.data_ptr(), workspace_bytes=100, stream=9)
    assert out.dtype == torch.bfloat16 and tuple(out.shape) == (T, H) and out.is_contiguous()
    wide = torch.zeros((T, H + 8), dtype=torch.bfloat16)[:, :H]
    assert ops.dg_fp8_moe_layer(x, sx, w13, s13, w2, s2, ids, weights, ws, out=wide, stream=9) is wide
    assert recorded.pop()["ldo"] == H + 8


def test_binding_raises_the_status(recorded, monkeypatch):
    """Through the real entry point: a host pointer never gets past the argument checks here (K % 128)."""
    monkeypatch.undo()
    ops._binding().any_device(True)
    with pytest.raises(DGError) as e:
        ops.dg_fp8_rmsnorm_quantize_1x128(torch.zeros((2, 200)), torch.ones(200), s=torch.zeros((2, 1)))
    assert e.value.status == SHAPE
    with pytest.raises(DGError) as e:
        ops.dg_moe_gate_topk(torch.zeros((2, 8)), 9)
    assert e.value.status == SHAPE
    with pytest.raises(DGError):
        ops.dg_moe_gate_topk(torch.zeros((2, 8)), -1)


class NoTruth:
    def __bool__(self):
        raise TypeError("neither")


def test_binding_refuses_what_is_no_tensor_or_number():
    x, w = torch.zeros((2, 256)), torch.ones(256)
    for call in (lambda: ops.dg_fp8_rmsnorm_quantize_1x128([1.0], w), lambda: ops.dg_moe_gate_topk(None, 2),
                 lambda: ops.dg_fp8_rmsnorm_quantize_1x128(x, w, eps="a"), lambda: ops.dg_moe_gate_topk(x, "2"),
                 lambda: ops.dg_moe_gate_topk(x, 2, renormalize=NoTruth()), lambda: ops.dg_fp8_moe_layer(*[None] * 9)):
        with pytest.raises(TypeError):
            call()


def test_outputs_are_not_leaked(recorded):
    """Reference counts of given and returned objects after many calls."""
    x, w = torch.zeros((2, 256)), torch.ones(256)
    q = torch.zeros((2, 256), dtype=torch.uint8)
    before = sys.getrefcount(q), sys.getrefcount(x), sys.getrefcount(w)
    for _ in range(50):
        out = ops.dg_fp8_rmsnorm_quantize_1x128(x, w, q=q, stream=1)
    count = sys.getrefcount(out[1])
    assert count == 2       # the tuple's, and the argument's
    del out
    assert (sys.getrefcount(q), sys.getrefcount(x), sys.getrefcount(w)) == before
