"""Attention over a paged cache of e4m3 codes where scales of values lie far apart: keys that a row does not see, and
those that it gives next to no weight, do not touch what the others give it.

Tolerances: those of tests/test_gpu_attention_step.py, but for the last one, of weights below fp16's normal numbers. A
weight p |sV| is off by 2^-25 there where the largest that its row sees is 2^7 or more, in units of 2^12 for sV; and it
may drop out in fp32, below 2^-126 of an exponential that is 2^19 / |sV| or more where it counts most: with |sV| up to
2^113 that is 2^-25 of the weight again. With M = max p |sV| / sum p over the keys that the row sees and codes below 2^9
in magnitude, n keys are off by n 2 2^-32 2^9 M = n 2^-22 M together. Above 2^113 what drops out grows in proportion:
`widen`. Exponentials end at 2^115, where 2^-25 of a weight is 2^-25 2^12 / 2^115 = 2^-32 2^-96 of p |sV| for the largest
p: in M no scale counts as less than 2^-96, whatever it is. bf16's numbers below 2^-126 are 2^-133 apart, so the rounding
of an output is off by up to 2^-134 there, which is more than 2^-8 of it (the smallest outputs here are about 2^-125).
"""
import math

import pytest
import torch

from fp8_block_scaled_sa_amd import DGError, ops
from tests.gpu_util import guards_intact, sentinel_bf16
from tests.test_gpu_attention_step import BF16, F32, F64, KINDS, MIXES, Batch, half, make_cache, normal, same, values
from tests.test_gpu_debug_build import both, debug_lib  # noqa: F401

pytestmark = pytest.mark.gpu

ALIASING, SCRATCH = 7, 8


def reference(b, window=0, widen=1.0):
    """Outputs of a Batch in 64 bits and how far each may be off, from what its row sees alone."""
    scale, page, pages = b.D ** -0.5, b.page, b.k[0].shape[0]
    group = b.q.shape[1] // b.k[0].shape[2]
    out = torch.full(b.q.shape, math.nan, dtype=F64, device="cuda")
    tol = torch.zeros_like(out)
    for i, (m, n) in enumerate(b.lengths):
        if m == 0:
            continue
        j = torch.arange(n, device="cuda")
        held = b.table[i].long()[j // page]
        there = (held >= 0) & (held < pages)
        held = torch.where(there, held, 0)
        k, v = (values(c[held, j % page], s[held, j % page]) for c, s in (b.k, b.v))
        weigh = torch.where((v != 0).any(-1), b.v[1][held, j % page].double().abs(), 0.0).clamp(min=2.0 ** -96)
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        seen = (j <= pos) & there
        if window:
            seen &= j > pos - window
        rows = slice(b.starts[i], b.starts[i] + m)
        for h in range(b.q.shape[1]):
            q, kh, vh, w = b.q[rows, h].double(), k[:, h // group], v[:, h // group], weigh[:, h // group]
            x = torch.where(seen, scale * (q @ kh.t()), -math.inf)
            p = torch.softmax(x, 1).nan_to_num(0.0)
            # how far each weight may be off by its score, which moves numerator and denominator
            pe = p * 2 * (b.D + 4) * 2.0 ** -24 * scale * (q.abs() @ kh.abs().t())
            out[rows, h] = p @ vh
            a = p @ vh.abs()
            tol[rows, h] = half(BF16) * out[rows, h].abs() + 2.0 ** -134 * (a > 0)
            tol[rows, h] += (2.0 ** -9 + 2.0 ** -19 + n * 2.0 ** -23) * a + pe @ vh.abs() + pe.sum(1, keepdim=True) * a
            tol[rows, h] += widen * n * 2.0 ** -22 * (p * w).amax(1, keepdim=True)
    return out, tol


def hold(got, ref, tol, rows):
    off = (got[rows].double() - ref[rows]).abs()
    assert bool((off <= tol[rows]).all()), "off by %.3g more than allowed" % float((off - tol[rows]).amax())


def last_key(b, i):
    """Page and offset of a sequence's last token."""
    n = b.lengths[i][1]
    return int(b.table[i, (n - 1) // b.page]), (n - 1) % b.page


@pytest.mark.parametrize("power", [22, 30, 100, 127])
@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES + [([(8, 20)], 2, 1, 128, 16), ([(20, 20)], 1, 1, 64, 16)])
def test_a_large_scale_in_the_future(gpu_device, lengths, heads, kv_heads, D, page, power):
    """The last key's values have a scale of 2^power: for the rows before it they are not there."""
    b = Batch(lengths, heads, kv_heads, D, page, 31)
    clean, (ref, tol) = b.call(), reference(b)
    for i in range(len(lengths)):
        b.v[1][last_key(b, i)] = 2.0 ** power
    got = b.call()
    after = reference(b) if power <= 100 else None
    for i, (m, _) in enumerate(lengths):
        rows = slice(b.starts[i], b.starts[i] + m - 1)
        hold(got, ref, tol, rows)
        assert torch.equal(got[rows], clean[rows])
        if after:
            hold(got, *after, slice(b.starts[i] + m - 1, b.starts[i] + m))


@pytest.mark.parametrize("power", [22, 30, 100])
@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_a_large_scale_that_has_left_the_window(gpu_device, lengths, heads, kv_heads, D, page, power):
    """The first key that the first row sees: the first row's alone, in a window."""
    b = Batch(lengths, heads, kv_heads, D, page, 32)
    for i, (m, n) in enumerate(lengths):
        j = max(0, n - m - 49)
        b.v[1][int(b.table[i, j // page]), j % page] = 2.0 ** power
    got = b.call(window=50)
    hold(got, *reference(b, 50), slice(b.starts[0], b.starts[-1]))


@pytest.mark.parametrize("power", [30, 60, 100])
@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_a_large_scale_of_next_to_no_weight(gpu_device, lengths, heads, kv_heads, D, page, power):
    """A key that every row sees and gives a weight of about exp(-150); scales of the others on both sides of 1."""
    b = Batch(lengths, heads, kv_heads, D, page, 33)
    b.q[...] = b.q.abs().clamp(0.25, 4.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    b.v[1].mul_(2.0 ** torch.randint(-8, 9, b.v[1].shape, generator=g, device="cuda"))
    for i, (m, n) in enumerate(lengths):
        j = max(0, n - m - 20)
        at = int(b.table[i, j // page]), j % page
        b.k[0][at] = 0xFE                # -448
        b.k[1][at] = 150 / (0.25 * 448 * D ** 0.5)
        b.v[1][at] = 2.0 ** power
    hold(b.call(), *reference(b), slice(b.starts[0], b.starts[-1]))


@pytest.mark.parametrize("power", [-20, -35, -60, -90])
@pytest.mark.parametrize("where", ["first", "spread"])
@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_rows_of_zeros_beside_small_values(gpu_device, lengths, heads, kv_heads, D, page, where, power):
    """Values of scales about 2^power, and rows of zeros, which have the scale 1: the first 150 keys of each sequence
    but its last, or every third one."""
    b = Batch(lengths, heads, kv_heads, D, page, 34)
    b.v[1].mul_(2.0 ** power)
    for i, (m, n) in enumerate(lengths):
        j = torch.arange(n, device="cuda")
        j = j[:min(150, n - 1)] if where == "first" else j[::3]
        at = b.table[i].long()[j // page], j % page
        b.v[0][at] = torch.tensor([0x00, 0x80], dtype=torch.uint8, device="cuda").repeat(D // 2)
        b.v[1][at] = 1.0
    hold(b.call(), *reference(b), slice(b.starts[0], b.starts[-1]))


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_pieces_whose_scales_lie_apart(gpu_device, lengths, heads, kv_heads, D, page):
    """Scales from 2^-60 to 2^100 in runs of 64 keys, of both signs: largest first, largest last and in between."""
    for turn in range(3):
        b = Batch(lengths, heads, kv_heads, D, page, 35)
        for i, (m, n) in enumerate(lengths):
            j = torch.arange(n, device="cuda")
            power = torch.tensor([[100, -60, 30, 0], [-60, 0, 30, 100], [0, 100, -60, 30]][turn], device="cuda")[j // 64 % 4]
            at = b.table[i].long()[j // page], j % page
            b.v[1][at] = torch.where(j % 5 == 0, -1.0, 1.0)[:, None] * 2.0 ** power.float()[:, None]
        hold(b.call(), *reference(b), slice(b.starts[0], b.starts[-1]))


@pytest.mark.parametrize("power", [-112, -106, -100, 105, 112, 118])
@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_scales_at_the_ends(gpu_device, lengths, heads, kv_heads, D, page, power):
    """All scales within a factor of two at the ends of what fp32 holds."""
    b = Batch(lengths, heads, kv_heads, D, page, 37)
    g = torch.Generator(device="cuda").manual_seed(2)
    b.v = (b.v[0], 2.0 ** power * (1 + torch.rand(b.v[1].shape, generator=g, device="cuda")))
    got = b.call()
    rows = slice(b.starts[0], b.starts[-1])
    assert bool(got[rows].any(-1).all())
    hold(got, *reference(b, widen=2.0 ** max(0, power + 1 - 113)), rows)


@pytest.mark.parametrize("lengths,heads,kv_heads,D,page", MIXES)
def test_scales_of_nothing(gpu_device, lengths, heads, kv_heads, D, page):
    """Scales of 0 and below 2^-114 count as 0, among others and by themselves."""
    for small in (0.0, 2.0 ** -115, 2.0 ** -149):
        b = Batch(lengths, heads, kv_heads, D, page, 36)
        some = torch.arange(b.v[1].numel(), device="cuda").view(b.v[1].shape) % 3 == 0
        b.v[1][some] = small
        got = b.call()
        b.v[1][some] = 0.0
        hold(got, *reference(b), slice(b.starts[0], b.starts[-1]))
        b.v[1][...] = small
        assert bool((b.call()[b.starts[0]:b.starts[-1]] == 0).all())


# ---------------------------------------------------------------- large batches

@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("lengths,checked", [
    ([(1, 30 + i % 50) for i in range(500)] + [(64, 5000)], [0, 63, 64, 499, 500]),
    ([(64, 5000)] + [(1, 30 + i % 50) for i in range(500)], [0, 1, 64, 500]),
    ([(1, 200), (40, 3000)] + [(1, 30 + i % 50) for i in range(700)] + [(300, 900), (1, 1)], [0, 1, 2, 64, 701, 702, 703])])
def test_chunks_beside_hundreds_of_single_tokens(gpu_device, lengths, checked, window):
    b = Batch(lengths, 64, 8, 64, 16, 41)
    got = b.call(window=window)
    for i in checked:
        b.lengths = [(m if j == i else 0, n) for j, (m, n) in enumerate(lengths)]
        hold(got, *reference(b, window), slice(b.starts[i], b.starts[i] + lengths[i][0]))


@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (4, 1), (16, 2), (28, 4), (16, 1), (17, 1), (32, 1), (33, 1)])
def test_few_tokens_beside_a_chunk(gpu_device, heads, kv_heads):
    """Sequences of all numbers of rows about the two tiles of the few-rows kernel, and the chunk first or last."""
    few = [(m, 100 + 37 * m) for m in (1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33)]
    for lengths in (few + [(70, 400)], [(70, 400)] + few):
        b = Batch(lengths, heads, kv_heads, 64, 16, 45)
        hold(b.call(), *reference(b), slice(b.starts[0], b.starts[-1]))


@pytest.mark.parametrize("lengths", [[(2100, 2100)], [(700, 700), (1400, 1500), (1, 40)]])
def test_thousands_of_tiles(gpu_device, lengths):
    """64 key heads of 8 query heads each: more than 4096 tiles of 256 rows."""
    b = Batch(lengths, 512, 64, 64, 16, 42)
    got = b.call()
    hold(got, *reference(b), slice(b.starts[0], b.starts[-1]))
    b.ws.fill_(0xFF)
    assert torch.equal(b.call(), got)


# ---------------------------------------------------------------- workspace

def needed(b):
    """Bytes of workspace without which a Batch's call is refused: with them it is refused for its output in the
    queries' place."""
    def status(n):
        with pytest.raises(DGError) as e:
            b.call(out=b.q, ws=b.ws[:n])
        return e.value.status
    low, high = 0, b.ws.numel()
    assert status(low) == SCRATCH and status(high) == ALIASING
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (mid, high) if status(mid) == SCRATCH else (low, mid)
    return high


def guarded(b):
    """The workspace as just the bytes that the call needs, and a check that what lies around them is as it was."""
    n = needed(b)
    buf = torch.full((n + 2 * 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    b.ws = buf[65536:65536 + n]

    def intact():
        torch.cuda.synchronize()
        return bool((buf[:65536] == 0xA5).all()) and bool((buf[65536 + n:] == 0xA5).all())
    return intact


@pytest.mark.parametrize("lengths,heads,kv_heads,D", list(KINDS.values()) + [
    ([(1, 100 + i) for i in range(131)], 8, 8, 64), ([(1, 16000)], 32, 1, 128), ([(16, 5000)] * 3, 4, 2, 64),
    ([(33, 9000)], 2, 2, 128), ([(40, 900 + 11 * i) for i in range(70)] + [(1, 300)] * 9, 2, 1, 64)])
def test_workspace_of_just_the_bytes_that_a_call_needs(gpu_device, lengths, heads, kv_heads, D):
    b = Batch(lengths, heads, kv_heads, D, 16, 43)
    want = b.call()
    intact = guarded(b)
    for _ in range(3):
        assert torch.equal(b.call(), want) and intact()


@pytest.mark.parametrize("lengths", [[(1, 100), (1, 40), (1, 7)], [(70, 100), (1, 40), (90, 90)], [(300, 3000)],
                                     [(1, 50)] * 70 + [(40, 2000)]])
def test_workspace_whatever_the_lengths(gpu_device, lengths):
    """Lengths and starts out of range and out of order write nothing beside the workspace and the output."""
    b = Batch(lengths, 8, 2, 128, 16, 44)
    intact = guarded(b)
    T, n = b.q.shape[0], len(lengths)
    for lens in ([2 ** 31 - 1] * n, [-1, -2 ** 31, 5] * n, [1 << 20, 0, 33] * n):
        for starts in (b.starts, [0, T] * n, [0, 2 ** 31 - 1, -5, T] * n, [-2 ** 31, 0, T, T + 1] * n, [T, 0, T, 0] * n):
            b.kv_lens = torch.tensor(lens[:n], dtype=torch.int32, device="cuda")
            b.q_starts = torch.tensor(starts[:n + 1], dtype=torch.int32, device="cuda")
            out = sentinel_bf16(b.q.shape)
            b.call(out=out)
            assert intact() and guards_intact(out)


@pytest.mark.parametrize("T,D,dtype,interleaved", [(1, 128, BF16, False), (61, 64, F32, True), (700, 128, BF16, False),
                                                   (700, 128, F32, False), (300, 64, BF16, True)])
def test_write_release_equals_O1_in_every_output(gpu_device, debug_lib, T, D, dtype, interleaved):  # noqa: F811
    """Turned queries, the keys' codes and scales and the values', bit for bit."""
    Hq, H = 8, 2
    q, k, v = normal((T, Hq + 2 * H, D), 1).to(dtype).split([Hq, H, H], 1)
    slots = torch.randperm(1024, device="cuda")[:T]
    freqs, _ = ops.dg_rope_frequencies(D)

    def run():
        c = [*make_cache(64, 16, H, D, 1), *make_cache(64, 16, H, D, 2)]
        out = ops.dg_fp8_rope_cache_write(k, v, *c, slots, (7919 * slots).int(), freqs, q=q, interleaved=interleaved)
        torch.cuda.synchronize()
        return [out, *c]
    rel, dbg = both(debug_lib, run)
    assert all(same(a, b) for a, b in zip(rel, dbg))


# ---------------------------------------------------------------- long sequences

@pytest.mark.parametrize("m,n", [(300, 1 << 21), (1, 1 << 21), (300, 40000)])
def test_a_long_run_of_zeros(gpu_device, m, n):
    """Values that are zeros but for 100 rows near the end, scores that fall by 7.9 powers of two for 32 keys of each 64:
    as much as exponentials and their sum can grow without a move of the reference. All rows and keys of a kind alike, so
    the outputs are ratios of counts; they are off as above, where n keys' sums are off by n 2^-24 each."""
    heads, D, page = 8, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    pages = -(-n // page)
    q = torch.ones((m, heads, D), dtype=BF16, device="cuda")
    k = torch.full((pages, page, 1, D), 0x38, dtype=torch.uint8, device="cuda")            # 1.0
    v = torch.zeros_like(k)
    j = torch.arange(pages * page, device="cuda")
    low = j // 32 % 2 == 0
    ks = torch.where(low, -7.9 * math.log(2) / D ** 0.5, 0.0).view(pages, page, 1).float()
    some = (j >= n - m - 100) & (j < n - m)
    v.view(-1, D)[some] = 0x38
    vs = torch.where(some, 0.75, 1.0).view(pages, page, 1)
    table = torch.randperm(pages, generator=g, device="cuda").int()
    at = torch.empty_like(table).long()
    at[table.long()] = torch.arange(pages, device="cuda")
    k, v, ks, vs = (t[at].contiguous() for t in (k, v, ks, vs))
    ws = ops.workspace(ops.dg_fp8_paged_attention_workspace_bytes(m, 1, heads, 1, D, m))
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    got = ops.dg_fp8_paged_attention(q, k, ks, v, vs, table[None], lens, starts, m, ws)
    p = torch.where(low, 2.0 ** -7.9, 1.0).double()[:n]
    want = 0.75 * (p * some[:n]).sum() / p.cumsum(0)[n - m:]
    off = (got.double() - want[:, None, None]).abs()
    assert bool((off <= (half(BF16) + 2.0 ** -9 + 2.0 ** -19 + n * 2.0 ** -23) * want[:, None, None]).all())
