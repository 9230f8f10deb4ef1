"""The operators over a paged cache (rotary positions and the cache's write, its
read, attention of new tokens) reject bad arguments on the host, through the C
ABI and through the Python binding; none of these calls reaches a device. And
the frequencies of rotary positions."""
import ctypes
import math
import os
import re

import pytest
import torch

from fp8_block_scaled_sa_amd import DGError, _lib, ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dg_fp8.h")

OK, NULL, SHAPE, MISALIGNED, STRIDE, UNSUPPORTED, HIP, ALIASING, SCRATCH = range(9)
GOT_TO_THE_DEVICE = (OK, UNSUPPORTED, HIP)

# Fake, never-dereferenced addresses that do not overlap.
Q, QO, K, V, POS, FREQS, SLOTS, KC, KS, VC, VS, TABLE, LENS, STARTS, OUT, WS = (0x10000000 * (i + 1) for i in range(16))
PAGES, PAGE, HEADS, D = 8, 16, 2, 128


class Cache(ctypes.Structure):
    """dg_fp8_cache."""
    _fields_ = [(n, ctypes.c_void_p if n in ("codes", "scales") else ctypes.c_int64) for n in (
        "codes", "stride_page", "stride_token", "stride_head", "scales", "s_stride_page", "s_stride_token", "s_stride_head",
        "pages", "page_size", "heads", "head_dim")]


def cache(at, s_at, **kw):
    """A cache [PAGES, PAGE, HEADS, D] with tokens before heads, with what `kw` changes."""
    args = dict(codes=at, scales=s_at, stride_page=PAGE * HEADS * D, stride_token=HEADS * D, stride_head=D,
                s_stride_page=PAGE * HEADS, s_stride_token=HEADS, s_stride_head=1, pages=PAGES, page_size=PAGE,
                heads=HEADS, head_dim=D)
    args.update(kw)
    return Cache(**args)


def ref(c):
    return ctypes.byref(c) if c is not None else None


SIZES = [  # of a cache, in every call
    (dict(pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(heads=0), SHAPE), (dict(heads=-1), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(page_size=2 ** 20 + 1), UNSUPPORTED), (dict(pages=2 ** 27), UNSUPPORTED), (dict(heads=65537), UNSUPPORTED)]
MEMORY = [
    (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(stride_page=-16), STRIDE), (dict(stride_head=-16), STRIDE),
    (dict(s_stride_token=-1), STRIDE), (dict(stride_page=2 ** 40 + 16), UNSUPPORTED),
    (dict(s_stride_page=2 ** 40 + 1), UNSUPPORTED), (dict(stride_page=2 ** 36), UNSUPPORTED),
    (dict(stride_page=9 * 2 ** 30, stride_token=2 ** 29), UNSUPPORTED), (dict(codes=KC + 8), MISALIGNED),
    (dict(scales=KS + 2), MISALIGNED), (dict(stride_page=4096 + 8), MISALIGNED), (dict(stride_page=8192, stride_token=264), MISALIGNED),
    (dict(stride_page=8192, stride_token=272, stride_head=136), MISALIGNED)]
WRITTEN = [  # rows that overlap
    (dict(stride_page=0), STRIDE), (dict(stride_token=128), STRIDE), (dict(stride_head=112), STRIDE),
    (dict(stride_page=4080), STRIDE), (dict(s_stride_head=0), STRIDE), (dict(s_stride_page=31), STRIDE),
    (dict(s_stride_token=1), STRIDE)]


# ---------------------------------------------------------------- write

def write(kc=None, vc=None, **kw):
    q_heads = kw.get("q_heads", 4)
    args = dict(Q=Q, q_t=512, q_h=128, QO=QO, qo_t=512, qo_h=128, q_heads=q_heads, K=K, k_t=256, k_h=128, V=V, v_t=256,
                v_h=128, type=1, positions=POS, freqs=FREQS, rot=128, interleaved=0, factor=1.0, slots=SLOTS,
                kc=cache(KC, KS, **(kc or {})), vc=cache(VC, VS, **(vc or {})), T=64, stream=None)
    args.update(kw)
    args["kc"], args["vc"] = ref(args["kc"]), ref(args["vc"])
    return _lib.load().dg_fp8_rope_cache_write(*args.values())


@pytest.mark.parametrize("kw,status", SIZES + [(k, s) for k, s in MEMORY if s != NULL] + MEMORY + WRITTEN)
def test_write_refuses_caches(kw, status):
    both = {k: v for k, v in kw.items() if k in ("pages", "page_size", "heads", "head_dim")}
    assert write(kc=kw, vc=both) == status


@pytest.mark.parametrize("kw", [dict(pages=4), dict(page_size=8), dict(heads=1), dict(head_dim=64)])
def test_write_refuses_caches_that_differ(kw):
    assert write(vc=kw) == SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), NULL), (dict(vc=None), NULL),
])
def test_write_refuses_no_cache(kw, status):
    args = dict(kc=cache(KC, KS), vc=cache(VC, VS))
    args.update(kw)
    lib = _lib.load()
    assert lib.dg_fp8_rope_cache_write(Q, 512, 128, QO, 512, 128, 4, K, 256, 128, V, 256, 128, 1, POS, FREQS, 128, 0, 1.0,
                                       SLOTS, ref(args["kc"]), ref(args["vc"]), 64, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(rot=-16), SHAPE), (dict(rot=144), SHAPE), (dict(rot=8), SHAPE), (dict(rot=40), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(q_heads=-1), SHAPE), (dict(Q=None), SHAPE),
    (dict(type=2), UNSUPPORTED), (dict(type=-1), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED), (dict(T=2 ** 24), UNSUPPORTED),
    (dict(q_heads=65537), UNSUPPORTED), (dict(q_t=2 ** 28 + 8), UNSUPPORTED), (dict(k_t=2 ** 28 + 8), UNSUPPORTED),
    (dict(v_h=2 ** 28 + 8), UNSUPPORTED), (dict(qo_t=2 ** 28 + 8), UNSUPPORTED),
    (dict(K=None), NULL), (dict(V=None), NULL), (dict(slots=None), NULL), (dict(QO=None), NULL),
    (dict(positions=None), NULL), (dict(freqs=None), NULL),
    (dict(k_t=-256), STRIDE), (dict(v_h=-128), STRIDE), (dict(q_h=-128), STRIDE), (dict(qo_t=-512), STRIDE),
    (dict(qo_t=256), STRIDE), (dict(qo_h=64), STRIDE), (dict(qo_t=0), STRIDE), (dict(qo_t=504), STRIDE),
    (dict(K=K + 8), MISALIGNED), (dict(V=V + 2), MISALIGNED), (dict(Q=Q + 8), MISALIGNED), (dict(QO=QO + 4), MISALIGNED),
    (dict(slots=SLOTS + 4), MISALIGNED), (dict(positions=POS + 2), MISALIGNED), (dict(freqs=FREQS + 4), MISALIGNED),
    (dict(k_t=260), MISALIGNED), (dict(v_h=132), MISALIGNED), (dict(q_t=516), MISALIGNED), (dict(qo_t=516), MISALIGNED),
    (dict(type=0, k_t=258), MISALIGNED),
    (dict(QO=K), ALIASING), (dict(QO=V + 256), ALIASING), (dict(QO=SLOTS), ALIASING), (dict(QO=POS), ALIASING),
    (dict(QO=FREQS), ALIASING), (dict(QO=Q + 16), ALIASING), (dict(QO=Q, qo_t=1024), ALIASING),
    (dict(QO=Q, type=0), ALIASING), (dict(QO=KC), ALIASING), (dict(QO=VS), ALIASING), (dict(K=KC), ALIASING),
    (dict(Q=VC + 64), ALIASING), (dict(slots=KS), ALIASING), (dict(V=VS), ALIASING),
])
def test_write_refusals(kw, status):
    assert write(**kw) == status


@pytest.mark.parametrize("vc", [dict(codes=KC), dict(scales=KS), dict(scales=KC + 64), dict(codes=KS)])
def test_write_refuses_caches_in_one_place(vc):
    assert write(vc=vc) == ALIASING


def test_write_accepted_and_empty():
    assert write(T=0, K=None, V=None, slots=None, Q=None, q_heads=0) == OK
    halves = dict(stride_page=2 * PAGE * HEADS * D, s_stride_page=2 * PAGE * HEADS)
    heads_first = dict(stride_head=PAGE * D, stride_token=D, s_stride_head=PAGE, s_stride_token=1)
    for kw in (dict(), dict(type=0), dict(rot=0, positions=None, freqs=None), dict(rot=16, interleaved=1), dict(QO=Q),
               dict(Q=None, QO=None, q_heads=0), dict(kc=halves, vc=dict(codes=KC + PAGE * HEADS * D,
                                                                        scales=KS + 4 * PAGE * HEADS, **halves)),
               dict(kc=heads_first, vc=heads_first), dict(k_t=0, v_t=0, q_t=0), dict(T=1, qo_t=0),
               dict(QO=Q, q_t=1024, q_h=128, qo_t=1024, qo_h=128, K=Q + 1024, k_t=1024, V=Q + 1536, v_t=1024)):
        assert write(**kw) in GOT_TO_THE_DEVICE


# ---------------------------------------------------------------- read

def read(kc=None, **kw):
    args = dict(cache=cache(KC, KS, **(kc or {})), slots=SLOTS, out=OUT, type=1, o_t=256, o_h=128, T=64, stream=None)
    args.update(kw)
    args["cache"] = ref(args["cache"])
    return _lib.load().dg_fp8_cache_read(*args.values())


@pytest.mark.parametrize("kw,status", SIZES + MEMORY)
def test_read_refuses_caches(kw, status):
    assert read(kc=kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), NULL), (dict(T=-1), SHAPE), (dict(type=2), UNSUPPORTED), (dict(T=2 ** 30), UNSUPPORTED),
    (dict(T=2 ** 29), UNSUPPORTED), (dict(o_t=2 ** 28 + 8), UNSUPPORTED), (dict(slots=None), NULL), (dict(out=None), NULL),
    (dict(o_t=-256), STRIDE), (dict(o_t=128), STRIDE), (dict(o_h=0), STRIDE), (dict(o_t=252), MISALIGNED),
    (dict(o_h=132, o_t=264), MISALIGNED), (dict(out=OUT + 8), MISALIGNED), (dict(slots=SLOTS + 4), MISALIGNED),
    (dict(out=KC), ALIASING), (dict(out=KS), ALIASING), (dict(out=SLOTS), ALIASING), (dict(slots=OUT + 512), ALIASING),
])
def test_read_refusals(kw, status):
    assert read(**kw) == status


def test_read_accepted_and_empty():
    assert read(T=0, slots=None, out=None) == OK
    for kw in (dict(), dict(type=0), dict(o_t=128, o_h=64 * 128), dict(kc=dict(stride_page=0, s_stride_page=0)),
               dict(T=1, o_t=0)):
        assert read(**kw) in GOT_TO_THE_DEVICE


# ---------------------------------------------------------------- attention

def ws_bytes(T=64, B=3, q_heads=8, heads=HEADS, head_dim=D, longest=40):
    return _lib.load().dg_fp8_paged_attention_workspace_bytes(T, B, q_heads, heads, head_dim, longest)


def attend(kc=None, vc=None, **kw):
    args = dict(Q=Q, q_t=1024, q_h=128, q_heads=8, kc=cache(KC, KS, **(kc or {})), vc=cache(VC, VS, **(vc or {})),
                table=TABLE, table_stride=9, width=8, lens=LENS, starts=STARTS, B=3, T=64, longest=40, scale=0.1, window=0,
                out=OUT, o_t=1024, o_h=128, ws=WS, ws_bytes=ws_bytes(), stream=None)
    args.update(kw)
    args["kc"], args["vc"] = ref(args["kc"]), ref(args["vc"])
    return _lib.load().dg_fp8_paged_attention(*args.values())


@pytest.mark.parametrize("kw,status", SIZES + MEMORY)
def test_attention_refuses_caches(kw, status):
    if "codes" in kw and kw["codes"]:
        kw = dict(kw, codes=VC + kw["codes"] - KC)
    if "scales" in kw and kw["scales"]:
        kw = dict(kw, scales=VS + kw["scales"] - KS)
    both = {k: v for k, v in kw.items() if k in ("pages", "page_size", "heads", "head_dim")}
    if both.get("heads") == 65537:
        assert attend(kc=both, vc=kw, q_heads=65537) == status
    else:
        assert attend(kc=both, vc=kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(q_heads=0), SHAPE), (dict(q_heads=7), SHAPE), (dict(longest=0), SHAPE),
    (dict(longest=-3), SHAPE), (dict(width=-1), SHAPE), (dict(window=-1), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(scale=math.inf), SHAPE), (dict(scale=-math.inf), SHAPE),
    (dict(T=2 ** 31), UNSUPPORTED), (dict(T=2 ** 28, q_heads=8), UNSUPPORTED), (dict(B=2 ** 24), UNSUPPORTED),
    (dict(B=2 ** 23, q_heads=8, longest=1), UNSUPPORTED), (dict(width=2 ** 26 + 1), UNSUPPORTED),
    (dict(width=2 ** 26, table_stride=2 ** 26, B=200), UNSUPPORTED), (dict(q_heads=65538), UNSUPPORTED),
    (dict(q_t=2 ** 28 + 8), UNSUPPORTED), (dict(o_h=2 ** 28 + 8), UNSUPPORTED), (dict(table_stride=2 ** 28 + 1), UNSUPPORTED),
    (dict(Q=None), NULL), (dict(out=None), NULL), (dict(lens=None), NULL), (dict(starts=None), NULL),
    (dict(table=None), NULL), (dict(ws=None), NULL),
    (dict(q_t=-8), STRIDE), (dict(o_h=-8), STRIDE), (dict(o_t=512), STRIDE), (dict(o_h=64), STRIDE), (dict(o_t=0), STRIDE),
    (dict(table_stride=7), STRIDE), (dict(table_stride=-1), STRIDE),
    (dict(q_t=1028), MISALIGNED), (dict(o_t=1028), MISALIGNED), (dict(Q=Q + 8), MISALIGNED), (dict(out=OUT + 8), MISALIGNED),
    (dict(table=TABLE + 2), MISALIGNED), (dict(lens=LENS + 1), MISALIGNED), (dict(starts=STARTS + 2), MISALIGNED),
    (dict(ws=WS + 8), MISALIGNED),
    (dict(ws_bytes=0), SCRATCH), (dict(ws_bytes=-1), SCRATCH), (dict(ws_bytes=1000), SCRATCH),
    (dict(out=Q), ALIASING), (dict(out=KC), ALIASING), (dict(out=VS), ALIASING), (dict(out=TABLE), ALIASING),
    (dict(out=STARTS), ALIASING), (dict(ws=Q), ALIASING), (dict(ws=LENS), ALIASING), (dict(ws=VC), ALIASING),
    (dict(out=WS + 1024), ALIASING),
])
def test_attention_refusals(kw, status):
    if "kc" in kw or "vc" in kw:        # (None stands for the default in attend's own)
        lib, c = _lib.load(), [None if n in kw else ref(cache(KC, KS)) for n in ("kc", "vc")]
        assert lib.dg_fp8_paged_attention(Q, 1024, 128, 8, *c, TABLE, 9, 8, LENS, STARTS, 3, 64, 40, 0.1, 0, OUT, 1024, 128,
                                          WS, ws_bytes(), None) == status
    else:
        assert attend(**kw) == status


@pytest.mark.parametrize("kw", [dict(pages=4), dict(page_size=8), dict(heads=1), dict(head_dim=64)])
def test_attention_refuses_caches_that_differ(kw):
    assert attend(vc=kw) == SHAPE


def test_attention_accepted_and_empty():
    nothing = dict(Q=None, out=None, lens=None, starts=None, table=None, ws=None, ws_bytes=0)
    assert attend(T=0, **nothing) == OK
    assert attend(B=0, **nothing) == OK
    assert attend(T=0, B=2 ** 24 - 1, width=2 ** 26, **nothing) == OK
    for kw in (dict(), dict(window=5), dict(scale=-1.0), dict(scale=0.0), dict(width=0, table=None), dict(kc=None, vc=dict(
            codes=KC, scales=KS)), dict(o_t=128, o_h=64 * 128), dict(longest=1), dict(longest=10 ** 12),
            dict(B=1, table_stride=0, T=40)):
        kw = dict(kw)
        if "longest" in kw or "B" in kw:
            kw["ws_bytes"] = ws_bytes(T=kw.get("T", 64), B=kw.get("B", 3), longest=kw.get("longest", 40))
        assert attend(**kw) in GOT_TO_THE_DEVICE


def test_attention_workspace_bytes():
    assert ws_bytes(T=0) == 0 and ws_bytes(B=0) == 0
    # monotone in the tokens, the sequences and the longest one's
    for D_ in (64, 128):
        for heads, q_heads in ((1, 1), (2, 8), (8, 64), (1, 40)):
            sizes = [1, 2, 3, 4, 5, 8, 16, 17, 32, 33, 64, 100, 255, 256, 300, 1000, 4096, 100000]
            last = 0
            for T in sizes:
                now = ws_bytes(T, 4, q_heads, heads, D_, 10 ** 6)
                assert now >= last > -1 and now % 4 == 0
                last = now
            last = 0
            for longest in sizes:
                now = ws_bytes(5000, 4, q_heads, heads, D_, longest)
                assert now >= last
                last = now
            last = 0
            for B in sizes[:-1]:
                now = ws_bytes(5000, B, q_heads, heads, D_, 7)
                assert now >= last
                last = now
    assert ws_bytes() <= 2 ** 28
    for kw, status in ((dict(T=-1), SHAPE), (dict(q_heads=3), SHAPE), (dict(longest=0), SHAPE), (dict(head_dim=0), SHAPE),
                       (dict(head_dim=80), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED), (dict(B=2 ** 24), UNSUPPORTED)):
        assert ws_bytes(**kw) == -status
    with pytest.raises(DGError) as e:
        ops.dg_fp8_paged_attention_workspace_bytes(64, 3, 7, 2, 128, 40)
    assert e.value.status == SHAPE


# ---------------------------------------------------------------- the binding

def code(*s):
    return torch.zeros(s, dtype=torch.uint8)


def good():
    """Arguments of the three calls that fit each other."""
    T, Hq = 5, 4
    c = dict(k_cache=code(PAGES, PAGE, HEADS, D), k_scales=torch.ones(PAGES, PAGE, HEADS),
             v_cache=code(PAGES, PAGE, HEADS, D), v_scales=torch.ones(PAGES, PAGE, HEADS))
    w = dict(k=torch.zeros(T, HEADS, D), v=torch.zeros(T, HEADS, D), **c, slots=torch.arange(T),
             positions=torch.arange(T, dtype=torch.int32), freqs=torch.ones(D // 2, dtype=torch.float64),
             q=torch.zeros(T, Hq, D))
    r = dict(cache=c["k_cache"], scales=c["k_scales"], slots=torch.arange(T))
    a = dict(q=torch.zeros((T, Hq, D), dtype=torch.bfloat16), **c, block_table=torch.zeros((2, 4), dtype=torch.int32),
             kv_lens=torch.ones(2, dtype=torch.int32), q_starts=torch.zeros(3, dtype=torch.int32), max_q_len=3,
             workspace=code(1 << 20))
    return w, r, a


def test_binding_refuses_host_tensors():
    w, r, a = good()
    for call, args in ((ops.dg_fp8_rope_cache_write, w), (ops.dg_fp8_cache_read, r), (ops.dg_fp8_paged_attention, a)):
        with pytest.raises(ValueError, match="device"):
            call(**args)


@pytest.mark.parametrize("name,bad", [
    ("v", torch.zeros(5, 1, D)), ("v", torch.zeros(4, HEADS, D)), ("k", torch.zeros(5, HEADS * D)),
    ("k", torch.zeros(5, D, HEADS).transpose(1, 2)), ("k_cache", code(PAGES, PAGE, HEADS, 64)),
    ("v_cache", code(PAGES + 1, PAGE, HEADS, D)), ("k_cache", code(PAGES * PAGE, HEADS, D)),
    ("k_scales", torch.ones(PAGES, PAGE)), ("v_scales", torch.ones(PAGES, PAGE, HEADS + 1)),
    ("slots", torch.arange(6)), ("slots", torch.zeros((5, 1), dtype=torch.int64)), ("slots", torch.arange(10)[::2]),
    ("positions", None), ("positions", torch.zeros(4, dtype=torch.int32)), ("q", torch.zeros(5, 0, D)),
    ("q", torch.zeros(6, 4, D)), ("q", torch.zeros(5, 4, 64)), ("q_out", torch.zeros((5, 3, D), dtype=torch.bfloat16)),
    ("freqs", torch.ones((2, 32), dtype=torch.float64))])
def test_write_binding_refuses_shapes(name, bad):
    with pytest.raises(ValueError):
        ops.dg_fp8_rope_cache_write(**{**good()[0], name: bad})


@pytest.fixture
def any_device():
    """The binding takes host tensors, up to the library's own checks."""
    ops._binding().any_device(True)
    yield
    ops._binding().any_device(False)


@pytest.mark.parametrize("name,dtype", [
    ("k", torch.float16), ("v", torch.bfloat16), ("q", torch.bfloat16), ("k_cache", torch.float32), ("v_cache", torch.int8),
    ("k_scales", torch.float64), ("slots", torch.int32), ("positions", torch.int64), ("freqs", torch.float32)])
def test_write_binding_refuses_types(any_device, name, dtype):
    w = good()[0]
    with pytest.raises(TypeError):
        ops.dg_fp8_rope_cache_write(**{**w, name: w[name].to(dtype)})


def test_write_binding_refuses_an_output_without_queries(any_device):
    w = good()[0]
    with pytest.raises(ValueError):
        ops.dg_fp8_rope_cache_write(**{**w, "q": None, "q_out": torch.zeros((5, 4, D), dtype=torch.bfloat16)})
    with pytest.raises(TypeError):
        ops.dg_fp8_rope_cache_write(**{**w, "q_out": torch.zeros(5, 4, D)})


@pytest.mark.parametrize("kw,error", [
    (dict(slots=torch.zeros((2, 2), dtype=torch.int64)), ValueError), (dict(slots=torch.zeros(3)), TypeError),
    (dict(dtype=torch.float16), TypeError), (dict(out=torch.zeros(5, HEADS, 64)), ValueError),
    (dict(out=torch.zeros(4, HEADS, D)), ValueError), (dict(scales=torch.ones(PAGES, PAGE)), ValueError),
    (dict(cache=torch.zeros(PAGES, PAGE, HEADS, D)), TypeError), (dict(out=torch.zeros(5, HEADS, D).half()), (TypeError,
                                                                                                           ValueError))])
def test_read_binding_refusals(any_device, kw, error):
    with pytest.raises(error):
        ops.dg_fp8_cache_read(**{**good()[1], **kw})


@pytest.mark.parametrize("name,bad,error", [
    ("q", torch.zeros(5, 4, D), TypeError), ("q", torch.zeros((5, 4, 64), dtype=torch.bfloat16), ValueError),
    ("q", torch.zeros((5, 512), dtype=torch.bfloat16), ValueError), ("k_cache", code(PAGES, PAGE, HEADS, 64), ValueError),
    ("v_cache", code(PAGES, PAGE, 1, D), ValueError), ("v_scales", torch.ones(PAGES, HEADS, PAGE), ValueError),
    ("block_table", torch.zeros((2, 4), dtype=torch.int64), TypeError),
    ("block_table", torch.zeros((4, 2), dtype=torch.int32).t(), ValueError),
    ("block_table", torch.zeros(8, dtype=torch.int32), ValueError), ("kv_lens", torch.ones(3, dtype=torch.int32), ValueError),
    ("kv_lens", torch.ones(2), TypeError), ("q_starts", torch.zeros(2, dtype=torch.int32), ValueError),
    ("q_starts", torch.zeros(3, dtype=torch.int64), TypeError), ("out", torch.zeros(5, 4, D), TypeError),
    ("out", torch.zeros((5, 3, D), dtype=torch.bfloat16), ValueError), ("workspace", code(8, 8).t(), ValueError),
    ("max_q_len", "3", TypeError)])
def test_attention_binding_refusals(any_device, name, bad, error):
    if name == "workspace":
        bad = code(8, 9)[:, :8]
    with pytest.raises(error):
        ops.dg_fp8_paged_attention(**{**good()[2], name: bad})


def parameters(name):
    """Parameter names of an entry point, from the header."""
    text = re.search(r"^dg_status %s\((.*?)\);" % name, open(HEADER).read(), re.M | re.S).group(1)
    return [p.split()[-1].lstrip("*") for p in text.split(",")]


@pytest.fixture
def recorded(monkeypatch):
    """Calls of the binding on host tensors, as {parameter: argument} by the header's names, caches as dicts."""
    calls = []
    kept = []
    names = ("dg_fp8_rope_cache_write", "dg_fp8_cache_read", "dg_fp8_paged_attention")

    def entry(name):
        params = parameters(name)
        res, types = _lib.SIGNATURES[name]
        assert len(params) == len(types)

        def call(*args):
            named = dict(zip(params, args))
            for n in ("cache", "k_cache", "v_cache"):
                if n in named:
                    c = Cache.from_address(named[n])
                    named[n] = {f: getattr(c, f) for f, _ in Cache._fields_}
            calls.append(named)
            return OK
        kept.append(ctypes.CFUNCTYPE(res, *types)(call))
        return ctypes.cast(kept[-1], ctypes.c_void_p).value

    class Library:
        _addresses = {n: entry(n) for n in names}

    monkeypatch.setattr(_lib, "_lib", Library())
    ops._binding().any_device(True)
    yield calls
    ops._binding().any_device(False)


def fields(codes, s):
    return dict(codes=codes.data_ptr(), stride_page=codes.stride(0), stride_token=codes.stride(1),
                stride_head=codes.stride(2), scales=s.data_ptr(), s_stride_page=s.stride(0), s_stride_token=s.stride(1),
                s_stride_head=s.stride(2), pages=codes.shape[0], page_size=codes.shape[1], heads=codes.shape[2],
                head_dim=codes.shape[3])


def caches():
    kc, vc = code(PAGES, HEADS, PAGE, D).transpose(1, 2), code(PAGES + 1, PAGE, HEADS + 1, D)[1:, :, :HEADS]
    ks, vs = torch.ones(HEADS, PAGES, PAGE).permute(1, 2, 0), torch.ones(PAGES, PAGE, 2 * HEADS)[..., ::2]
    return kc, ks, vc, vs


def test_cache_fields_are_the_headers():
    text = re.search(r"typedef struct dg_fp8_cache \{(.*?)\} dg_fp8_cache;", open(HEADER).read(), re.S).group(1)
    names = [n.strip(" *") for line in text.strip().split(";")[:-1] for n in line.split(None, 1)[1].split(",")]
    assert [n.split()[-1].lstrip("*") for n in names] == [f for f, _ in Cache._fields_]


def test_write_binding_passes_every_argument_by_its_name(recorded):
    T, Hq = 3, 4
    kc, ks, vc, vs = caches()
    qkv = torch.zeros((T, Hq + 2 * HEADS + 1, D), dtype=torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + HEADS], qkv[:, Hq + HEADS:Hq + 2 * HEADS]
    slots, pos, freqs = torch.arange(T), torch.arange(T, dtype=torch.int32), torch.ones(16, dtype=torch.float64)
    wide = (Hq + 2 * HEADS + 1) * D
    out = ops.dg_fp8_rope_cache_write(k, v, kc, ks, vc, vs, slots, pos, freqs, q=q, interleaved=True, factor=0.5, stream=7)
    assert recorded.pop() == dict(
        Q=q.data_ptr(), q_stride_t=wide, q_stride_h=D, Q_out=out.data_ptr(), qo_stride_t=Hq * D, qo_stride_h=D, q_heads=Hq,
        K=k.data_ptr(), k_stride_t=wide, k_stride_h=D, V=v.data_ptr(), v_stride_t=wide, v_stride_h=D, x_dtype=1,
        positions=pos.data_ptr(), freqs=freqs.data_ptr(), rot=32, interleaved=1, factor=0.5, slots=slots.data_ptr(),
        k_cache=fields(kc, ks), v_cache=fields(vc, vs), T=T, stream=7)
    assert out.dtype == torch.bfloat16 and tuple(out.shape) == (T, Hq, D) and out.is_contiguous()
    assert ops.dg_fp8_rope_cache_write(k, v, kc, ks, vc, vs, slots, pos, freqs, q=q, q_out=q, stream=1) is q
    c = recorded.pop()
    assert (c["Q_out"], c["qo_stride_t"], c["qo_stride_h"], c["interleaved"], c["factor"]) == (q.data_ptr(), wide, D, 0, 1.0)
    assert ops.dg_fp8_rope_cache_write(k.float(), v.float(), kc, ks, vc, vs, slots, stream=1) is None
    c = recorded.pop()
    assert (c["Q"], c["Q_out"], c["q_heads"], c["positions"], c["freqs"], c["rot"], c["x_dtype"]) == (
        None, None, 0, None, None, 0, 0)


def test_read_binding_passes_every_argument_by_its_name(recorded):
    kc, ks, _, _ = caches()
    slots = torch.arange(5)
    out = ops.dg_fp8_cache_read(kc, ks, slots, stream=3)
    assert recorded.pop() == dict(cache=fields(kc, ks), slots=slots.data_ptr(), out=out.data_ptr(), out_dtype=1,
                                  out_stride_t=HEADS * D, out_stride_h=D, T=5, stream=3)
    assert out.dtype == torch.bfloat16 and tuple(out.shape) == (5, HEADS, D)
    given = torch.zeros((5, HEADS + 1, D + 4))[:, 1:, :D]
    assert ops.dg_fp8_cache_read(kc, ks, slots, out=given, stream=3) is given
    c = recorded.pop()
    assert (c["out_dtype"], c["out_stride_t"], c["out_stride_h"]) == (0, (HEADS + 1) * (D + 4), D + 4)
    assert ops.dg_fp8_cache_read(kc, ks, slots, dtype=torch.float32, stream=3).dtype == torch.float32


def test_attention_binding_passes_every_argument_by_its_name(recorded):
    T, Hq, B = 5, 6, 2
    kc, ks, vc, vs = caches()
    q = torch.zeros((T, Hq + 1, D), dtype=torch.bfloat16)[:, 1:]
    table = torch.zeros((B, 12), dtype=torch.int32)[:, :9]
    lens, starts, ws = torch.ones(B, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32), code(100)
    out = ops.dg_fp8_paged_attention(q, kc, ks, vc, vs, table, lens, starts, 4, ws, window=33, stream=5)
    c = recorded.pop()
    scale = c.pop("scale")
    assert abs(scale - D ** -0.5) <= 2 ** -24 * scale
    assert c == dict(
        Q=q.data_ptr(), q_stride_t=(Hq + 1) * D, q_stride_h=D, q_heads=Hq, k_cache=fields(kc, ks), v_cache=fields(vc, vs),
        block_table=table.data_ptr(), table_stride=12, table_width=9, kv_lens=lens.data_ptr(), q_starts=starts.data_ptr(),
        B=B, T=T, max_q_len=4, window=33, out=out.data_ptr(), out_stride_t=Hq * D, out_stride_h=D,
        workspace=ws.data_ptr(), workspace_bytes=100, stream=5)
    assert out.dtype == torch.bfloat16 and tuple(out.shape) == (T, Hq, D) and out.is_contiguous()
    given = torch.zeros((Hq, T, D + 8), dtype=torch.bfloat16)[..., :D].transpose(0, 1)
    assert ops.dg_fp8_paged_attention(q, kc, ks, vc, vs, table, lens, starts, 4, None, scale=0.25, out=given,
                                      stream=5) is given
    c = recorded.pop()
    assert (c["scale"], c["window"], c["out_stride_t"], c["out_stride_h"], c["workspace"], c["workspace_bytes"]) == (
        0.25, 0, D + 8, T * (D + 8), None, 0)


def test_binding_raises_the_status(any_device):
    """Through the real entry points: what only they refuse."""
    w, r, a = good()
    for call, args, kw, status in (
            (ops.dg_fp8_rope_cache_write, w, dict(freqs=torch.ones(5, dtype=torch.float64)), SHAPE),
            (ops.dg_fp8_rope_cache_write, w, dict(k_cache=code(2, 2, HEADS, 96), v_cache=code(2, 2, HEADS, 96),
                                                  k_scales=torch.ones(2, 2, HEADS), v_scales=torch.ones(2, 2, HEADS),
                                                  k=torch.zeros(5, HEADS, 96), v=torch.zeros(5, HEADS, 96),
                                                  q=torch.zeros(5, 4, 96)), UNSUPPORTED),
            (ops.dg_fp8_cache_read, r, dict(cache=code(2, 2, 2, 32), scales=torch.ones(2, 2, 2)), UNSUPPORTED),
            (ops.dg_fp8_paged_attention, a, dict(max_q_len=0), SHAPE),
            (ops.dg_fp8_paged_attention, a, dict(window=-1), SHAPE),
            (ops.dg_fp8_paged_attention, a, dict(scale=math.nan), SHAPE)):
        with pytest.raises(DGError) as e:
            call(**{**args, **kw})
        assert e.value.status == status


def test_binding_refuses_what_is_no_tensor_or_number():
    w, r, a = good()
    for call, args, name, bad in ((ops.dg_fp8_rope_cache_write, w, "k", [1.0]), (ops.dg_fp8_rope_cache_write, w, "slots", 3),
                                  (ops.dg_fp8_rope_cache_write, w, "factor", "a"), (ops.dg_fp8_cache_read, r, "slots", None),
                                  (ops.dg_fp8_paged_attention, a, "scale", "a"), (ops.dg_fp8_paged_attention, a, "kv_lens", 1)):
        with pytest.raises(TypeError):
            call(**{**args, name: bad})


# ---------------------------------------------------------------- frequencies

def test_rope_frequencies():
    freqs, factor = ops.dg_rope_frequencies(128, base=10000.0, device="cpu")
    assert freqs.dtype == torch.float64 and factor == 1.0
    want = [10000.0 ** (-2 * i / 128) for i in range(64)]
    assert torch.allclose(freqs, torch.tensor(want, dtype=torch.float64), rtol=1e-14, atol=0)
    assert ops.dg_rope_frequencies(2, device="cpu")[0].tolist() == [1.0]


def test_rope_frequencies_for_longer_contexts():
    plain, _ = ops.dg_rope_frequencies(64, device="cpu")
    linear, factor = ops.dg_rope_frequencies(64, scaling="linear", stretch=4.0, device="cpu")
    assert torch.allclose(linear, plain / 4, rtol=1e-15, atol=0) and factor == 1.0
    based, factor = ops.dg_rope_frequencies(64, scaling="base", stretch=4.0, device="cpu")
    assert based[0] == 1.0 and abs(float(based[-1] / plain[-1]) - 0.25) < 1e-13 and factor == 1.0
    assert bool((based[1:] < plain[1:]).all()) and bool((based >= plain / 4 * (1 - 1e-13)).all())
    parts, factor = ops.dg_rope_frequencies(64, scaling="parts", stretch=4.0, original=2048, fast=32.0, slow=1.0, device="cpu")
    assert abs(factor - (0.1 * math.log(4.0) + 1.0)) < 1e-15
    turns = 2048 * plain / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], plain[turns >= 32]) and bool((turns >= 32).any())
    assert torch.allclose(parts[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15, atol=0) and bool((turns <= 1).any())
    between = (turns > 1) & (turns < 32)
    share = (turns - 1) / 31
    assert torch.allclose(parts[between], (plain * (share + (1 - share) / 4))[between], rtol=1e-13, atol=0)
    for scaling in ("linear", "base", "parts"):
        same, factor = ops.dg_rope_frequencies(64, scaling=scaling, stretch=1.0, device="cpu")
        assert torch.allclose(same, plain, rtol=1e-14, atol=0) and factor == 1.0


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=-2), dict(rot=7), dict(scaling="other"), dict(stretch=0.5),
                                dict(stretch=math.nan), dict(scaling="parts", fast=1.0, slow=1.0)])
def test_rope_frequencies_refusals(kw):
    with pytest.raises(ValueError):
        ops.dg_rope_frequencies(**{"rot": 64, "device": "cpu", **kw})
