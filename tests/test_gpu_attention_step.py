"""The operators over a paged cache of e4m3 codes on the GPU against plain 64-bit forms: rotary positions and the
cache's write, its read, and attention of new tokens.

Tolerances. A value rounded once is off by half a step of its type (torch.finfo(t).eps / 2, relative); before it:
  write      cosine and sine of an fp32 angle in half turns: the angle's rounding moves them by pi 2^-24, the functions
             by 2 ulp, their product with factor by half one: together under 2^-21 of the factor; the two products and
             the sum add 2^-23: an element is within 2^-20 factor (|x| + |y|) of the formula's; scales likewise, and a
             code stands within half a step of what it should (2^-4 of the value, 2^-10 below the normal codes) plus that;
  read       the fp32 product's rounding (2^-24) and the type's;
  attention  x is a sum of D exact products in fp32: off by at most (D + 4) 2^-24 sum_d |q_d k_d| scale =: e. A weight
             exp(x) is then off by 2 e (relative, e < 1/2) plus 2^-20 of the exponential and the scales; a sum over n
             keys adds n 2^-24, numerator and denominator each. fp16 takes the weights, by 2^-11 off, in the numerator
             or (many rows) in both, which counts twice; there it also takes sV and sV V, 2^-11 each: 2^-9 in all. With
             A = sum p |v| / sum p an output is within (2^-9 + 4 e + 2^-19 + n 2^-23) A of the formula's before its
             rounding to bf16. fp16's numbers below 2^-14 are off by up to 2^-25 instead. Of the weights: the largest of
             a row is 2^7 or more, so this is 2^-32 of it, for n keys of values up to 448 M, M the largest |sV| (few
             rows: the weight times sV / M', M' < 2 M a power of two, twice that). Of sV V (many rows) in units of
             M' / 2^6: 2^-31 M'. Together below n 2^-31 448 M = n 2^-31 max |v|, which counts where scales lie apart.
"""
import math

import pytest
import torch

from fp8_block_scaled_sa_amd import ops
from tests.gpu_util import guards_intact, sentinel_bf16
from tests.test_gpu_debug_build import both, debug_lib  # noqa: F401

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def normal(shape, seed, outliers=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:
        x[torch.rand(shape, generator=g, device="cuda") < 1e-3] *= 20
    return x


def half(dtype):
    return torch.finfo(dtype).eps / 2


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- a cache

def quantized(x):
    """Codes (uint8) and scales of rows [..., D]. (Divided by a tensor: by a number, torch multiplies with its
    reciprocal on the device, which is off by an ulp.)"""
    amax = x.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448))
    return (x / s[..., None]).clamp(-448, 448).to(F8).view(torch.uint8), s


def make_cache(pages, page, heads, D, seed, layout="tokens"):
    """Codes [pages, page, heads, D] and scales [pages, page, heads] of normal rows; layout: the order in memory."""
    codes, s = quantized(normal((pages, page, heads, D), seed))
    if layout == "heads":               # [pages, heads, page, D]
        codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
        s = s.transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "padded":
        buf = torch.full((pages, page + 1, heads, D + 16), 0x7F, dtype=torch.uint8, device="cuda")
        buf[:, :page, :, :D] = codes
        codes = buf[:, :page, :, :D]
        sbuf = torch.full((heads, pages, page + 2), math.nan, device="cuda")
        sbuf[:, :, :page] = s.permute(2, 0, 1)
        s = sbuf[:, :, :page].permute(1, 2, 0)
    return codes, s


def values(codes, s):
    return codes.contiguous().view(F8).double() * s.double()[..., None]


# ---------------------------------------------------------------- write

def rotated(x, positions, freqs, factor, interleaved):
    """The formula in 64 bits, and the sum of magnitudes that the tolerance refers to."""
    y, size = x.double().clone(), x.double().abs()
    n = 0 if freqs is None else len(freqs)
    if n:
        a = positions.double()[:, None] * freqs
        co, si = (factor * a.cos())[:, None], (factor * a.sin())[:, None]
        first = slice(0, 2 * n, 2) if interleaved else slice(0, n)
        second = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
        u, v = x.double()[..., first], x.double()[..., second]
        y[..., first], y[..., second] = u * co - v * si, u * si + v * co
        size[..., first] = size[..., second] = factor * (u.abs() + v.abs())
    return y, size


def check_codes(codes, s, ref, size):
    """Codes [T, heads, D] and scales against rows ref, which an fp32 computation has within 2^-20 size."""
    off = 2.0 ** -20 * size
    amax = ref.abs().amax(-1)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert bool(((s.double() - want).abs() <= 2.0 ** -23 * want + off.amax(-1) / 448).all())
    t = ref / s.double()[..., None]
    got = codes.view(F8).double()
    slack = off / s.double()[..., None] + 2.0 ** -22 * t.abs()
    assert bool(((got - t).abs() <= torch.clamp((t.abs() + slack) * half(F8), min=2.0 ** -10) + slack).all())
    assert bool((got.abs().amax(-1) == torch.where(amax > 0, 448.0, 0.0)).all())


WRITES = [  # T, q_heads, heads, D, rot, page, dtype, interleaved
    (1, 32, 8, 128, 128, 64, BF16, False), (1, 1, 1, 64, 64, 1, BF16, True), (2, 3, 1, 128, 64, 16, F32, False),
    (61, 24, 4, 64, 32, 16, F32, True), (37, 5, 5, 128, 16, 7, BF16, False), (300, 8, 2, 64, 64, 48, BF16, False),
    (5, 70, 3, 128, 128, 5, BF16, True), (9, 0, 2, 128, 96, 32, F32, False), (33, 4, 1, 128, 0, 16, BF16, False),
    (1025, 8, 1, 128, 128, 128, F32, False), (700, 1, 1, 64, 48, 33, BF16, True)]


@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
@pytest.mark.parametrize("T,q_heads,heads,D,rot,page,dtype,interleaved", WRITES)
def test_write(gpu_device, T, q_heads, heads, D, rot, page, dtype, interleaved, layout):
    pages = T // page + 3
    g = torch.Generator(device="cuda").manual_seed(T + D)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    slots[::5] = -1
    if T > 3:
        slots[1], slots[2] = pages * page, -(1 << 40)
    qkv = normal((T, q_heads + 2 * heads, D), T + 1).to(dtype)
    q, k, v = qkv.split([q_heads, heads, heads], 1)
    positions = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    freqs, factor = ops.dg_rope_frequencies(rot, scaling="parts", stretch=4.0) if rot else (None, 1.0)
    kc, ks = make_cache(pages, page, heads, D, 5, layout)
    vc, vs = make_cache(pages, page, heads, D, 6, layout)
    before = [t.clone() for t in (kc, ks, vc, vs)]
    whole = [torch.empty(0, dtype=t.dtype, device="cuda").set_(t.untyped_storage()) for t in (kc, ks, vc, vs)]
    image = [t.clone() for t in whole]
    out = ops.dg_fp8_rope_cache_write(k, v, kc, ks, vc, vs, slots, positions=positions if rot else None, freqs=freqs,
                                      q=q if q_heads else None, interleaved=interleaved, factor=factor)
    torch.cuda.synchronize()
    if q_heads:
        ref, size = rotated(q, positions, freqs, factor, interleaved)
        assert out.dtype == BF16
        assert bool(((out.double() - ref).abs() <= half(BF16) * ref.abs() + 2.0 ** -19 * size).all())
    else:
        assert out is None
    kept = (slots >= 0) & (slots < pages * page)
    at = slots[kept]
    for codes, s, old, x, turns in ((kc, ks, before[:2], k, freqs), (vc, vs, before[2:], v, None)):
        ref, size = rotated(x, positions, turns, factor, interleaved)
        p, t = at // page, at % page
        check_codes(codes[p, t], s[p, t], ref[kept], size[kept])
        # the other slots, and what lies between the rows, are as they were
        codes[p, t], s[p, t] = old[0][p, t], old[1][p, t]
    assert all(same(a, b) for a, b in zip(whole, image))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_without_rotation_is_the_quantizer(gpu_device, dtype):
    """Rows of 128: the same codes and scales as dg_fp8_quantize_1x128, bit for bit, tiny and zero rows among them."""
    T, heads = 200, 3
    x = normal((T, heads, 128), 3)
    x[5] *= 1e-30
    x[6] *= 1e-38
    x[7] = 0
    x[8] *= 1e30
    x = x.to(dtype)
    kc, ks = make_cache(4, 64, heads, 128, 1)
    vc, vs = make_cache(4, 64, heads, 128, 2)
    slots = torch.arange(T, device="cuda")
    ops.dg_fp8_rope_cache_write(x, x.flip(0).contiguous(), kc, ks, vc, vs, slots)
    q, s = ops.dg_fp8_quantize_1x128(x.reshape(T, heads * 128))
    assert torch.equal(kc.view(-1, heads * 128)[:T], q) and torch.equal(ks.view(-1, heads)[:T], s)
    assert torch.equal(vc.view(-1, heads * 128)[:T], q.flip(0)) and torch.equal(vs.view(-1, heads)[:T], s.flip(0))


def test_write_far_positions(gpu_device):
    """Positions up to 2^31 - 1 and negative ones: the angle's whole turns cost nothing."""
    positions = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32, device="cuda")
    T = len(positions)
    freqs, _ = ops.dg_rope_frequencies(64)
    x = normal((T, 1, 64), 9)
    kc, ks = make_cache(1, 16, 1, 64, 1)
    vc, vs = make_cache(1, 16, 1, 64, 2)
    q = ops.dg_fp8_rope_cache_write(x, x, kc, ks, vc, vs, torch.arange(T, device="cuda"), positions, freqs, q=x)
    ref, size = rotated(x, positions, freqs, 1.0, False)
    # 2^31 radians in fp64 are off by 2^-22, on either side
    assert bool(((q.double() - ref).abs() <= half(BF16) * ref.abs() + (2.0 ** -19 + 2.0 ** -20) * size).all())


def test_write_in_place(gpu_device):
    """Queries turned in place in a fused tensor that keys and values are columns of."""
    T, Hq, H, D = 77, 12, 2, 128
    qkv = normal((T, Hq + 2 * H, D), 4).to(BF16)
    freqs, _ = ops.dg_rope_frequencies(D)
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")

    def go(qkv, in_place):
        q, k, v = qkv.split([Hq, H, H], 1)
        c = [*make_cache(5, 16, H, D, 1), *make_cache(5, 16, H, D, 2)]
        out = ops.dg_fp8_rope_cache_write(k, v, *c, slots, positions, freqs, q=q, q_out=q if in_place else None)
        return [out, *c]
    want = go(qkv, False)
    mine = qkv.clone()
    got = go(mine, True)
    assert all(same(a, b) for a, b in zip(want, got))
    assert torch.equal(mine[:, Hq:], qkv[:, Hq:])


def test_write_keys_and_values_of_one_tensor(gpu_device):
    """K and V as halves of each page of one tensor."""
    T, H, D = 40, 2, 64
    k, v = normal((T, H, D), 1), normal((T, H, D), 2)
    both = torch.zeros((4, 2, 16, H, D), dtype=torch.uint8, device="cuda")
    s = torch.zeros((4, 2, 16, H), device="cuda")
    slots = torch.randperm(64, device="cuda")[:T]
    ops.dg_fp8_rope_cache_write(k, v, both[:, 0], s[:, 0], both[:, 1], s[:, 1], slots)
    for i, x in ((0, k), (1, v)):
        want = quantized(x.cpu())
        assert torch.equal(both[:, i].reshape(64, H, D)[slots].cpu(), want[0])
        assert torch.equal(s[:, i].reshape(64, H)[slots].cpu(), want[1])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_write_of_what_is_not_finite(gpu_device, bad):
    """The row reads back as NaN, its codes are finite, its neighbours are untouched."""
    T, H, D = 9, 2, 128
    x = normal((T, H, D), 1)
    y = x.clone()
    y[4, 1, 77] = bad
    slots = torch.arange(T, device="cuda")
    freqs, _ = ops.dg_rope_frequencies(D)
    positions = slots.int()
    got = []
    for z in (x, y):
        c = [*make_cache(1, 16, H, D, 1), *make_cache(1, 16, H, D, 2)]
        ops.dg_fp8_rope_cache_write(z, z, *c, slots, positions, freqs)
        got.append([ops.dg_fp8_cache_read(c[0], c[1], slots, dtype=F32), ops.dg_fp8_cache_read(c[2], c[3], slots, dtype=F32)])
        assert not bool(((c[0] & 0x7F) == 0x7F).any()) and not bool(((c[2] & 0x7F) == 0x7F).any())
    for a, b in zip(*got):
        assert bool(b[4, 1].isnan().all())
        b[4, 1] = a[4, 1]
        assert torch.equal(a, b)


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
@pytest.mark.parametrize("T,heads,D,page", [(1, 1, 64, 1), (1, 8, 128, 64), (333, 4, 64, 16), (57, 3, 128, 5),
                                            (2000, 5, 128, 48)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_read(gpu_device, T, heads, D, page, dtype, layout):
    pages = max(2, T // page // 2)
    codes, s = make_cache(pages, page, heads, D, T, layout)
    g = torch.Generator(device="cuda").manual_seed(T)
    slots = torch.randint(0, pages * page, (T,), generator=g, device="cuda")     # repeats among them
    slots[::7] = torch.tensor([-1, pages * page, -(1 << 50), 1 << 50], device="cuda").repeat(T)[:len(slots[::7])]
    out = torch.full((T, heads + 1, D + 16), 7.0, dtype=dtype, device="cuda")
    got = ops.dg_fp8_cache_read(codes, s, slots, out=out[:, :heads, :D])
    there = (slots >= 0) & (slots < pages * page)
    ref = torch.zeros((T, heads, D), dtype=F64, device="cuda")
    at = slots[there]
    ref[there] = values(codes[at // page, at % page], s[at // page, at % page])
    assert bool(((got.double() - ref).abs() <= (half(dtype) + 2.0 ** -24) * ref.abs()).all())
    out[:, :heads, :D] = 7.0
    assert bool((out == 7.0).all())
    new = ops.dg_fp8_cache_read(codes, s, slots, dtype=dtype)
    assert new.dtype == dtype and tuple(new.shape) == (T, heads, D)
    assert bool(((new.double() - ref).abs() <= (half(dtype) + 2.0 ** -24) * ref.abs()).all())


# ---------------------------------------------------------------- attention

class Batch:
    """Sequences of (new tokens, tokens) on random pages, with everything that a call takes."""

    def __init__(self, lengths, heads, kv_heads, D, page, seed=0, layout="tokens", gap=0, spare=2, width=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lengths, self.page, self.D = lengths, page, D
        need = [-(-n // page) for _, n in lengths]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.width = max(need + [1]) if width is None else width
        self.table = torch.full((len(lengths), self.width), -1, dtype=torch.int32, device="cuda")
        used = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[used:used + n]
            used += n
        starts = [gap]
        for m, _ in lengths:
            starts.append(starts[-1] + m)
        self.starts = starts
        T = starts[-1] + gap
        self.q = 2 * torch.randn((T, heads, D), generator=g, device="cuda")
        self.q = self.q.to(BF16)
        self.k = make_cache(pages, page, kv_heads, D, seed + 1, layout)
        self.v = make_cache(pages, page, kv_heads, D, seed + 2, layout)
        self.kv_lens = torch.tensor([n for _, n in lengths], dtype=torch.int32, device="cuda")
        self.q_starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.longest = max([m for m, _ in lengths] + [1])
        self.ws = ops.workspace(ops.dg_fp8_paged_attention_workspace_bytes(T, len(lengths), heads, kv_heads, D, self.longest))
        self.ws.fill_(0xFF)

    def call(self, out=None, **kw):
        longest = kw.pop("longest", self.longest)
        ws = kw.pop("ws", self.ws)
        return ops.dg_fp8_paged_attention(self.q, *self.k, *self.v, self.table, self.kv_lens, self.q_starts, longest, ws,
                                          out=out, **kw)

    def reference(self, scale=None, window=0):
        """Outputs in 64 bits and how far they may be off, sequence by sequence: rows of no sequence are NaN."""
        q, D, page = self.q.double(), self.D, self.page
        scale = D ** -0.5 if scale is None else scale
        T, Hq, _ = q.shape
        H = self.k[0].shape[2]
        pages = self.k[0].shape[0]
        out = torch.full(q.shape, math.nan, dtype=F64, device="cuda")
        tol = torch.zeros_like(out)
        for b, (m, n) in enumerate(self.lengths):
            n = min(n, self.width * page)
            if m == 0:
                continue
            j = torch.arange(n, device="cuda")
            held = self.table[b].long()[j // page]
            there = (held >= 0) & (held < pages)
            held = torch.where(there, held, 0)
            k, v = (values(c[held, j % page], s[held, j % page]) for c, s in (self.k, self.v))   # [n, H, D]
            pos = torch.arange(n - m, n, device="cuda")[:, None]
            seen = (j <= pos) & there
            if window:
                seen &= j > pos - window
            for h in range(Hq):
                kh, vh = k[:, h // (Hq // H)], v[:, h // (Hq // H)]
                rows = slice(self.starts[b], self.starts[b] + m)
                # what is not seen holds anything, NaN too
                used = seen.any(0)[:, None]
                kh, vh = torch.where(used, kh, 0.0), torch.where(used, vh, 0.0)
                x = torch.where(seen, scale * (q[rows, h] @ kh.t()), -math.inf)
                e = (D + 4) * 2.0 ** -24 * abs(scale) * (q[rows, h].abs() @ kh.abs().t())
                top = torch.where(seen.any(1, keepdim=True), x.amax(1, keepdim=True) if n else x, 0.0)
                p = torch.exp(x - top)
                total = p.sum(1, keepdim=True)
                some = total > 0
                o = torch.where(some, p @ vh / torch.where(some, total, 1.0), 0.0)
                a = torch.where(some, p @ vh.abs() / torch.where(some, total, 1.0), 0.0)
                worst = torch.where(seen, e, 0.0).amax(1, keepdim=True) if n else torch.zeros_like(total)
                out[rows, h] = o
                tol[rows, h] = half(BF16) * o.abs() + (2.0 ** -9 + 4 * worst + 2.0 ** -19 + n * 2.0 ** -23) * a
                tol[rows, h] += n * 2.0 ** -31 * vh.abs().amax() if n else 0.0
        return out, tol

    def check(self, got, **kw):
        ref, tol = self.reference(**kw)
        rows = slice(self.starts[0], self.starts[-1])
        off = (got.double() - ref)[rows].abs()
        worst = (off - tol[rows]).amax() if off.numel() else torch.zeros(())
        assert bool((off <= tol[rows]).all()), "off by %.3g more than allowed" % float(worst)


SINGLES = [  # lengths, heads, kv_heads, D, page
    ([(1, 1)], 1, 1, 64, 1), ([(1, 1)], 8, 1, 128, 64), ([(1, 31)], 16, 1, 64, 16), ([(1, 32)], 32, 8, 128, 64),
    ([(1, 33)], 4, 4, 128, 16), ([(1, 127), (1, 128), (1, 129), (1, 255), (1, 5)], 8, 2, 128, 16),
    ([(1, 4000)], 32, 8, 128, 64), ([(1, 200 + 37 * i) for i in range(70)], 4, 2, 64, 48),
    ([(1, 1000), (1, 3), (1, 2777)], 28, 4, 128, 7), ([(1, 700), (1, 999)], 40, 1, 128, 32),
    ([(1, 3000)], 64, 1, 64, 16)]


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", SINGLES)
@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
def test_attention_of_single_tokens(gpu_device, lengths, heads, kv_heads, D, page, layout):
    b = Batch(lengths, heads, kv_heads, D, page, 3, layout)
    b.check(b.call())


FEW = [([(2, 2)], 8, 1, 128, 16), ([(4, 100), (4, 4), (4, 257)], 32, 8, 128, 32), ([(5, 1000), (1, 10), (3, 3)], 8, 2, 64, 48),
       ([(8, 300)], 64, 8, 128, 64), ([(16, 16), (16, 2000)], 4, 1, 128, 16), ([(64, 129), (0, 50), (1, 64)], 1, 1, 64, 16)]


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", FEW)
def test_attention_of_few_tokens(gpu_device, lengths, heads, kv_heads, D, page):
    b = Batch(lengths, heads, kv_heads, D, page, 4)
    b.check(b.call())


CHUNKS = [([(65, 65)], 1, 1, 64, 16), ([(128, 128)], 2, 1, 128, 64), ([(129, 1000)], 8, 8, 128, 48),
          ([(100, 100), (100, 777), (1, 500), (0, 9), (17, 64)], 28, 4, 128, 16), ([(512, 3000)], 8, 2, 128, 64),
          ([(1000, 1000), (1, 1)], 16, 2, 64, 32), ([(300, 5000)], 4, 1, 128, 7), ([(1, 400)] * 20 + [(200, 900)], 8, 1, 64, 16),
          ([(40, 90)], 96, 1, 128, 16)]


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", CHUNKS)
def test_attention_of_chunks(gpu_device, lengths, heads, kv_heads, D, page):
    b = Batch(lengths, heads, kv_heads, D, page, 5)
    b.check(b.call())


@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 1000, 5000])
@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", [
    ([(1, 1500), (1, 3), (1, 64)], 8, 2, 128, 16), ([(4, 300), (7, 7)], 8, 2, 64, 48),
    ([(200, 1500), (1, 77), (150, 150)], 8, 2, 128, 32)])
def test_attention_window(gpu_device, lengths, heads, kv_heads, D, page, window):
    """With the pages before every window given back, and NaN where they were."""
    b = Batch(lengths, heads, kv_heads, D, page, 6)
    for i, (m, n) in enumerate(lengths):
        gone = max(0, n - m + 1 - window) // page
        for c, s in (b.k, b.v):
            c[b.table[i, :gone].long()] = 0x7F
            s[b.table[i, :gone].long()] = math.nan
        b.table[i, :gone] = -1
    b.check(b.call(window=window), window=window)


# ---------------------------------------------------------------- attention where it can go wrong

EDGES = [  # (new tokens, tokens): none, more new tokens than tokens, none new
    [(1, 0), (1, 1), (1, 2)], [(5, 3), (4, 0), (0, 7), (2, 2)], [(0, 0), (0, 5)],
    [(300, 40), (70, 0), (0, 100), (257, 300)], [(70, 70), (1, 0), (40, 1)]]


@pytest.mark.parametrize("lengths", EDGES)
@pytest.mark.parametrize("D", [64, 128])
def test_attention_rows_that_see_nothing_are_zero(gpu_device, lengths, D):
    b = Batch(lengths, 8, 2, D, 16, 7, gap=1)
    got = b.call()
    b.check(got)
    for i, (m, n) in enumerate(lengths):
        rows = got[b.starts[i]:b.starts[i] + max(0, m - n)]
        assert bool((rows == 0).all())


def spoil(b, seed, bad_codes=True):
    """Whatever no row sees holds NaN codes and scales: spare pages, and the places behind each sequence's end."""
    pages, page = b.k[0].shape[:2]
    used = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
    for i, (_, n) in enumerate(b.lengths):
        j = torch.arange(min(n, b.width * page), device="cuda")
        held = b.table[i].long()[j // page]
        there = (held >= 0) & (held < pages)
        used[held[there], (j % page)[there]] = True
    for c, s in (b.k, b.v):
        if bad_codes:
            c[~used] = 0x7F
        s[~used] = torch.tensor([math.nan, math.inf, -math.inf], device="cuda")[seed % 3]


MIXES = [([(1, 700), (1, 33), (1, 128)], 8, 2, 128, 16), ([(4, 300), (2, 65)], 8, 1, 64, 48),
         ([(90, 90), (1, 200), (130, 1000)], 8, 2, 128, 33), ([(200, 333)], 4, 1, 64, 7), ([(40, 300), (33, 64)] * 3, 8, 4, 128, 16)]


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_attention_of_what_is_not_seen(gpu_device, lengths, heads, kv_heads, D, page, seed):
    """NaN and infinities behind the sequences' ends and in other pages; pages missing in the middle, by any number."""
    b = Batch(lengths, heads, kv_heads, D, page, 8 + seed)
    for i, (_, n) in enumerate(lengths):
        need = -(-n // page)
        gone = torch.arange(need, device="cuda")[seed::3]
        pages = b.k[0].shape[0]
        b.table[i, gone] = torch.tensor([-1, pages, 2 ** 31 - 1, -2 ** 31, -7, pages + 1], device="cuda",
                                        dtype=torch.int32).repeat(need)[:len(gone)]
    spoil(b, seed)
    b.check(b.call())
    b.check(b.call(window=50), window=50)


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_attention_with_values_not_finite_in_the_future(gpu_device, lengths, heads, kv_heads, D, page):
    """The last key's value row and scale: the rows before it do not count it, the last row becomes NaN."""
    b = Batch(lengths, heads, kv_heads, D, page, 9)
    clean, tol = b.call(), b.reference()[1]
    for what in range(3):
        for i, (m, n) in enumerate(lengths):
            at = int(b.table[i, (n - 1) // page]), (n - 1) % page
            if what == 0:
                b.v[0][at] = 0x7F
            elif what == 1:
                b.v[0][at] = 0
                b.v[1][at] = math.nan
            else:
                b.v[1][at] = math.inf
        got = b.call()
        for i, (m, n) in enumerate(lengths):
            rows, last = slice(b.starts[i], b.starts[i] + m - 1), b.starts[i] + m - 1
            assert bool(torch.isfinite(got[rows]).all())
            off = (got[rows].double() - clean[rows].double()).abs()
            assert bool((off <= 2 * tol[rows]).all())
            if what < 2:
                assert bool(got[last].isnan().all())
            else:
                assert not bool(torch.isfinite(got[last]).all())


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_attention_with_a_key_not_finite(gpu_device, lengths, heads, kv_heads, D, page):
    """A NaN in the first key that all rows see makes every row NaN, and no row of another sequence."""
    b = Batch(lengths, heads, kv_heads, D, page, 10)
    clean = b.call()
    b.k[0][int(b.table[0, 0]), 0, :, 5] = 0xFF
    got = b.call()
    m = lengths[0][0]
    assert bool(got[:m].isnan().all())
    assert torch.equal(got[m:], clean[m:])


# Scales of keys and values: equal, one of a few very large ones, tiny, of both signs, zero rows among them.
SCALES = ["one", "large", "tiny", "spread", "falling", "rising", "negative", "zeros"]


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", [
    ([(1, 20), (1, 1), (1, 600)], 8, 2, 128, 16), ([(40, 40), (33, 33), (70, 75)], 1, 1, 64, 16),
    ([(100, 128)], 4, 1, 128, 64), ([(40, 700), (64, 96)], 8, 2, 128, 16), ([(300, 2000)], 4, 1, 64, 48)])
def test_attention_over_scales(gpu_device, lengths, heads, kv_heads, D, page, kind):
    """V's scales from 2^-100 to 2^100, and up to 2^18 apart within a sequence."""
    b = Batch(lengths, heads, kv_heads, D, page, 11)
    s = b.v[1]
    shape = s.shape
    order = torch.zeros(shape[:2], dtype=F64, device="cuda")     # of a slot in its sequence
    for i, (_, n) in enumerate(lengths):
        j = torch.arange(n, device="cuda")
        order[b.table[i].long()[j // page], j % page] = j.double() / max(n, 1)
    order = order[..., None].expand(shape)
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.rand(shape, generator=g, device="cuda", dtype=F64)
    new = {"one": torch.ones_like(u), "large": 2.0 ** 100 * (1 + u), "tiny": 2.0 ** -100 * (1 + u),
           "spread": 2.0 ** (18 * u - 9), "falling": 2.0 ** (9 - 18 * order), "rising": 2.0 ** (18 * order - 9),
           "negative": torch.where(u < 0.5, -1.0, 1.0) * (1 + u), "zeros": torch.ones_like(u)}[kind]
    b.v = (b.v[0], new.float())
    if kind == "zeros":
        b.v[0][u < 0.3] = 0
    got = b.call()
    assert bool(torch.isfinite(got[b.starts[0]:b.starts[-1]]).all())
    b.check(got)


@pytest.mark.parametrize("scale", [0.0, -0.07, 1.0, 1e-30, 3.0])
def test_attention_scale(gpu_device, scale):
    b = Batch([(1, 300), (70, 130), (3, 3)], 4, 1, 64, 16, 12)
    b.q /= 8                             # weights that are not all on one key at the largest scale
    b.check(b.call(scale=scale), scale=scale)


def test_attention_of_large_scores(gpu_device):
    """Scores beyond the range of exp, of both signs, rising and falling along the keys."""
    for lengths in ([(1, 3000)], [(64, 64), (300, 2000)]):
        b = Batch(lengths, 8, 2, 128, 16, 13)
        order = torch.zeros(b.k[1].shape[:2], device="cuda")
        for i, (_, n) in enumerate(lengths):
            j = torch.arange(n, device="cuda")
            order[b.table[i].long()[j // 16], j % 16] = j.float()
        for sign in (1.0, -1.0):
            ks = b.k[1].clone()
            b.k[0][...] = torch.tensor([2.0], device="cuda").to(F8).view(torch.uint8)[0]
            b.q[...] = 1.0
            b.q[1::2] = -1.0
            b.k = (b.k[0], (sign * order / 8)[..., None].expand(ks.shape).contiguous())
            b.check(b.call())


def test_attention_strides_and_what_lies_between(gpu_device):
    """Q and out within wider tensors, heads before tokens too; rows of no sequence and of too long ones as they were."""
    for lengths, longest in (([(1, 200), (1, 33)], 1), ([(3, 90), (9, 40), (1, 5)], 4), ([(70, 300), (130, 130), (1, 9)], 100)):
        b = Batch(lengths, 8, 2, 128, 16, 14, gap=3)
        T = b.q.shape[0]
        want = b.call(out=torch.zeros_like(b.q))
        wide = torch.full((T, 11, 136), 0.5, dtype=BF16, device="cuda")
        wide[:, 2:10, :128] = b.q
        b.q = wide[:, 2:10, :128]
        for layout in ("tokens", "heads"):
            buf = sentinel_bf16((T, 10, 144) if layout == "tokens" else (10, T, 144))
            out = (buf if layout == "tokens" else buf.transpose(0, 1))[:, 1:9, 8:136]
            image = buf.clone()
            assert b.call(out=out, longest=longest) is out
            for i, (m, _) in enumerate(lengths):
                rows = slice(b.starts[i], b.starts[i] + m)
                if m <= longest:
                    assert torch.equal(out[rows], want[rows])
                    out[rows] = (image if layout == "tokens" else image.transpose(0, 1))[rows, 1:9, 8:136]
            assert same(buf, image)


def test_attention_cache_strides(gpu_device):
    """Keys and values as halves of each page, heads before tokens: the same results, bit for bit."""
    for lengths in ([(1, 500), (1, 3)], [(90, 200), (1, 70)]):
        b = Batch(lengths, 8, 2, 64, 16, 15)
        want = b.call()
        for dims in ((0, 1, 2, 3, 4), (0, 1, 3, 2, 4), (1, 0, 2, 3, 4), (3, 0, 1, 2, 4)):
            both, s = torch.stack([b.k[0], b.v[0]], 1), torch.stack([b.k[1], b.v[1]], 1)
            inverse = [dims.index(i) for i in range(5)]
            both = both.permute(dims).contiguous().permute(inverse)
            s = s.permute(dims[:4]).contiguous().permute(inverse[:4])
            k, v = (both[:, 0], s[:, 0]), (both[:, 1], s[:, 1])
            got = ops.dg_fp8_paged_attention(b.q, *k, *v, b.table, b.kv_lens, b.q_starts, b.longest, b.ws)
            assert torch.equal(got, want)


def test_attention_table_narrower_than_the_sequences_and_wider(gpu_device):
    for width in (1, 3, 200):
        b = Batch([(1, 100), (2, 31)], 4, 2, 64, 16, 16)
        wide = torch.full((2, max(width, b.width) + 5), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        wide[:, :b.width] = b.table
        b.table, b.width = wide[:, :width], width
        got = b.call()
        # the sequences end where the table does
        b.lengths = [(m, min(n, width * 16)) for m, n in b.lengths]
        b.check(got)


def test_attention_lengths_out_of_range_do_no_harm(gpu_device):
    """Whatever the lengths and starts hold: no fault, nothing beside out and workspace written."""
    for lengths in ([(1, 100), (1, 40), (1, 7)], [(70, 100), (1, 40), (90, 90)]):
        b = Batch(lengths, 8, 2, 128, 16, 17)
        T = b.q.shape[0]
        for lens in ([2 ** 31 - 1] * 3, [-1, -2 ** 31, 5], [1 << 20, 0, 33]):
            for starts in (b.starts, [0, 2 ** 31 - 1, -5, T], [-2 ** 31, 0, T, T + 1], [T, 0, T, 0], [T + 7, T + 8, T + 9, T + 10]):
                b.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
                b.q_starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
                buf = sentinel_bf16((T + 4, 8, 128))
                image = buf.clone()
                b.call(out=buf[2:T + 2])
                torch.cuda.synchronize()
                assert same(buf[:2], image[:2]) and same(buf[T + 2:], image[T + 2:])


def test_attention_behind_32_bits(gpu_device):
    """Pages further than 2^32 bytes into a cache that is keys and values at once; the write and the read there too."""
    page, heads, D = 16, 1, 128
    pages = (2 ** 32 + 2 ** 25) // (page * heads * D)
    codes = torch.zeros((pages, page, heads, D), dtype=torch.uint8, device="cuda")
    s = torch.ones((pages, page, heads), device="cuda")
    for lengths in ([(1, 300)], [(70, 300)]):
        b = Batch(lengths, 4, 1, D, page, 18)
        b.v = b.k
        want = b.call()
        first = pages - b.k[0].shape[0]
        codes[first:], s[first:] = b.k
        b.k = b.v = codes, s
        b.table = torch.where(b.table >= 0, b.table + first, b.table)
        assert torch.equal(b.call(), want)
    x = normal((3, heads, D), 1)
    slots = torch.tensor([pages * page - 1, 2 ** 32 // D, 0], device="cuda")
    other, s2 = torch.zeros_like(codes), torch.ones_like(s)
    ops.dg_fp8_rope_cache_write(x, x, codes, s, other, s2, slots)
    want = quantized(x.cpu())
    at = slots // page, slots % page
    assert torch.equal(codes[at].cpu(), want[0]) and torch.equal(s[at].cpu(), want[1])
    assert torch.equal(other[at].cpu(), want[0]) and torch.equal(s2[at].cpu(), want[1])
    got = ops.dg_fp8_cache_read(codes, s, slots, dtype=F32)
    assert torch.equal(got.cpu(), want[0].view(F8).float() * want[1][..., None])


# ---------------------------------------------------------------- a step's calls together

def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_decode_step.py")
    spec = importlib.util.spec_from_file_location("moe_decode_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("heads,kv_heads,page", [(4, 2, 16), (8, 1, 7), (16, 4, 64)])
def test_example_attention_steps(gpu_device, heads, kv_heads, page):
    """Prompts in chunks, then token by token, of sequences that join and leave: each step's attention against 64 bits
    over what the cache holds then, the output product against 64 bits from the same codes."""
    ex = example()
    block = ex.AttentionBlock(hidden=384, heads=heads, kv_heads=kv_heads, pages=100, page_size=page, max_tokens=300,
                              max_batch=3)
    table = torch.randperm(99, device="cuda").int().view(3, 33)
    most = 33 * page
    at = [0, 0, 0]
    for i, new in enumerate(([100, 3, 1], [120, 0, 1], [1, 1, 1], [1, 60, 1], [1, 1, 40], [1, 1, 1])):
        new = [min(m, most - n) for m, n in zip(new, at)]
        at = [n + m for n, m in zip(at, new)]
        batch = ex.batch_of(table, page, new, at)
        x, residual = normal((sum(new), 384), 20 + i).to(BF16), normal((sum(new), 384), 40 + i).to(BF16)
        total = (x.float() + residual.float()).to(BF16)
        copy = residual.clone()
        o, q = block.attend(x, residual, **batch)
        assert torch.equal(residual, total)
        exact, size = block.reference(q, table, batch["kv_lens"], batch["q_starts"])
        # scores below 64 in magnitude here, exact to 2^-24 132 64: 2^-11, and 2^-9 as above
        assert bool(((o.double() - exact).abs() <= half(BF16) * exact.abs() + (2.0 ** -9 + 2.0 ** -10) * size).all())
        out = block.step(x, copy, **batch)
        codes, s = ops.dg_fp8_quantize_1x128(o.flatten(1))
        want = (codes.view(F8).double() * s.double().repeat_interleave(128, 1)) @ ex.value(block.w_out, block.s_out).t()
        assert float((out.double() - want).norm()) <= half(BF16) * float(want.norm())


def test_step_of_padded_tokens(gpu_device):
    """A batch padded to a fixed number of tokens and sequences (slots -1, no new tokens) gives the rows of the same
    batch without padding, and leaves the cache as that does."""
    T, Hq, H, D, page = 5, 8, 2, 128, 16
    freqs, _ = ops.dg_rope_frequencies(D)
    qkv = normal((64, Hq + 2 * H, D), 1).to(BF16)
    results = []
    for pad in (0, 59):
        b = Batch([(1, 40), (3, 70), (1, 1)], Hq, H, D, page, 2)
        n = T + pad
        q, k, v = qkv[:n].clone().split([Hq, H, H], 1)
        positions = torch.zeros(n, dtype=torch.int32, device="cuda")
        positions[:T] = torch.tensor([39, 67, 68, 69, 0])
        slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
        seq = torch.tensor([0, 1, 1, 1, 2], device="cuda")
        slots[:T] = b.table[seq, positions[:T].long() // page].long() * page + positions[:T].long() % page
        lens, starts = b.kv_lens, b.q_starts
        table = b.table
        if pad:
            lens = torch.cat([lens, torch.zeros(6, dtype=torch.int32, device="cuda")])
            starts = torch.cat([starts, torch.full((6,), T, dtype=torch.int32, device="cuda")])
            table = torch.cat([table, torch.full((6, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
        q = ops.dg_fp8_rope_cache_write(k, v, *b.k, *b.v, slots, positions, freqs, q=q)
        ws = ops.workspace(ops.dg_fp8_paged_attention_workspace_bytes(n, len(lens), Hq, H, D, 3))
        out = ops.dg_fp8_paged_attention(q, *b.k, *b.v, table, lens, starts, 3, ws, out=torch.full_like(q, 0.25))
        assert bool((out[T:] == 0.25).all())
        b.q = q[:T]
        b.check(out[:T])
        results.append([out[:T], *b.k, *b.v])
    assert all(same(x, y) for x, y in zip(*(r[1:] for r in results)))


# ---------------------------------------------------------------- streams, graphs, builds

KINDS = {  # lengths of calls through each kernel, and of the two together
    "singles": ([(1, 700), (1, 3), (1, 1500)], 8, 2, 128), "few": ([(3, 300), (4, 900)], 8, 1, 64),
    "cut": ([(40, 2000)], 8, 2, 128), "cut batch": ([(33, 900)] * 5, 4, 2, 64), "chunks": ([(300, 700), (90, 90)], 8, 2, 128),
    "mixed": ([(1, 400)] * 4 + [(150, 600)], 8, 2, 128)}


@pytest.mark.parametrize("kind", KINDS)
def test_attention_on_a_stream(gpu_device, kind):
    """`stream=`, and a side stream as the current one; the caller orders the streams."""
    b = Batch(*KINDS[kind], 16, 21)
    want = b.call()
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    for _ in range(3):
        b.ws.fill_(0xFF)
        b.q = b.q.clone()
        side.wait_stream(main)
        got = b.call(stream=side)
        main.wait_stream(side)
        assert torch.equal(got, want)
        with torch.cuda.stream(side):
            again = b.call()
        side.synchronize()
        assert torch.equal(again, want)


def test_write_and_read_on_a_stream(gpu_device):
    T, H, D = 100, 2, 128
    side = torch.cuda.Stream()
    slots = torch.randperm(128, device="cuda")[:T]
    freqs, _ = ops.dg_rope_frequencies(D)
    results = []
    for kw in ({}, dict(stream=side)):
        x = normal((T, H, D), 3)
        c = [*make_cache(8, 16, H, D, 1), *make_cache(8, 16, H, D, 2)]
        positions = slots.int()
        side.wait_stream(torch.cuda.current_stream())
        q = ops.dg_fp8_rope_cache_write(x, x, *c, slots, positions, freqs, q=x, **kw)
        results.append([q, *c, ops.dg_fp8_cache_read(c[0], c[1], slots, **kw)])
        torch.cuda.current_stream().wait_stream(side)
    assert all(same(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("kind", KINDS)
def test_attention_in_a_graph(gpu_device, kind):
    """A captured step (write, attention, read), replayed with other lengths, pages and contents, and a second graph
    that shares its workspace, with eager work between."""
    lengths, heads, kv_heads, D = KINDS[kind]
    b = Batch(lengths, heads, kv_heads, D, 16, 22)
    T, page = b.q.shape[0], 16
    freqs, _ = ops.dg_rope_frequencies(D)
    kv = normal((2, T, kv_heads, D), 5)
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    positions = torch.zeros(T, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(b.q), torch.zeros_like(b.q)]
    turned = torch.zeros_like(b.q)
    rows = torch.zeros((T, kv_heads, D), dtype=F32, device="cuda")

    def step(out, window):
        q = b.q
        ops.dg_fp8_rope_cache_write(kv[0].to(BF16), kv[1].to(BF16), *b.k, *b.v, slots, positions, freqs, q=q, q_out=turned)
        ops.dg_fp8_paged_attention(turned, *b.k, *b.v, b.table, b.kv_lens, b.q_starts, b.longest, b.ws, out=out,
                                   window=window)
        ops.dg_fp8_cache_read(*b.k, slots, out=rows)

    step(outs[0], 0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    for i, window in enumerate((0, 77)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(outs[i], window)
        graphs.append(graph)
    torch.cuda.synchronize()
    g = torch.Generator(device="cuda").manual_seed(9)
    for turn in range(4):
        # shorter sequences, other pages, other rows
        lens = [max(m, (n * (4 - turn)) // 4) for m, n in lengths]
        b.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        b.table.copy_(b.table.roll(1, 0) if turn % 2 else b.table)
        b.q.copy_(torch.randn(b.q.shape, generator=g, device="cuda"))
        kv.copy_(torch.randn(kv.shape, generator=g, device="cuda"))
        for i, (m, _) in enumerate(lengths):
            at = torch.arange(lens[i] - m, lens[i], device="cuda")
            held = b.table[i].long()[at // page]
            slots[b.starts[i]:b.starts[i + 1]] = torch.where(held >= 0, held * page + at % page, -1)
            positions[b.starts[i]:b.starts[i + 1]] = at.int()
        for i, window in enumerate((0, 77)):
            for out in outs:
                out.zero_()
            b.ws.fill_(0xFF)
            graphs[i].replay()
            torch.cuda.synchronize()
            got, got_rows = outs[i].clone(), rows.clone()
            outs[i].zero_()
            rows.zero_()
            step(outs[i], window)
            torch.cuda.synchronize()
            assert torch.equal(got, outs[i]) and torch.equal(got_rows, rows), "replay %d of graph %d" % (turn, i)
            assert bool(got.any())


@pytest.mark.parametrize("kind", KINDS)
def test_attention_release_equals_O1(gpu_device, debug_lib, kind):  # noqa: F811
    """And a hundred repeats, from a workspace of NaN bytes each."""
    b = Batch(*KINDS[kind], 16, 23)
    out = sentinel_bf16(b.q.shape)

    def run():
        b.ws.fill_(0xFF)
        b.call(out=out)
        torch.cuda.synchronize()
        assert guards_intact(out)
        return out.clone()
    rel, dbg = both(debug_lib, run)
    assert torch.equal(rel, dbg), "-O1 build differs from the release build"
    for r in range(100):
        assert torch.equal(run(), rel), "repeat %d differs" % r


@pytest.mark.parametrize("T,D,dtype", [(1, 128, BF16), (61, 64, F32), (700, 128, BF16)])
def test_write_and_read_release_equal_O1(gpu_device, debug_lib, T, D, dtype):  # noqa: F811
    Hq, H = 8, 2
    x = normal((T, Hq + 2 * H, D), 1).to(dtype)
    q, k, v = x.split([Hq, H, H], 1)
    slots = torch.randperm(1024, device="cuda")[:T]
    positions = (7919 * slots).int()
    freqs, _ = ops.dg_rope_frequencies(D)

    def run():
        c = [*make_cache(64, 16, H, D, 1), *make_cache(64, 16, H, D, 2)]
        out = ops.dg_fp8_rope_cache_write(k, v, *c, slots, positions, freqs, q=q)
        back = ops.dg_fp8_cache_read(c[2], c[3], slots, dtype=dtype)
        torch.cuda.synchronize()
        return [out, *c, back]
    rel, dbg = both(debug_lib, run)
    # (The library's sine and cosine may be compiled to other instructions: an fp32 step before the rounding.)
    for a, b in zip(rel[3:], dbg[3:]):
        assert same(a, b)
    for _ in range(20):
        assert all(same(a, b) for a, b in zip(run(), rel))
    ref, size = rotated(q, positions, freqs, 1.0, False)
    assert bool(((dbg[0].double() - ref).abs() <= half(BF16) * ref.abs() + 2.0 ** -19 * size).all())


def test_attention_of_many_few_rows(gpu_device):
    """More rows to join than workgroups that would take one each: a wave a row, whose last ones end in a workgroup."""
    for lengths, heads, kv_heads, D in (([(4, 400 + 137 * i) for i in range(39)], 16, 8, 128),
                                        ([(1, 300 + 61 * i) for i in range(67)], 35, 7, 64)):
        b = Batch(lengths, heads, kv_heads, D, 16, 24)
        b.check(b.call())


@pytest.mark.parametrize("window", [0, 300])
def test_attention_of_many_chunks(gpu_device, window):
    """More sequences than a wave has lanes, whose tiles are cut, beside single tokens and sequences without new ones."""
    lengths = [((40, 1, 33, 0)[i % 4], 900 + 11 * i) for i in range(131)]
    b = Batch(lengths, 2, 1, 64, 16, 25)
    got = b.call(window=window)
    b.check(got, window=window)
    b.ws.fill_(0xFF)
    assert torch.equal(b.call(window=window), got)
