"""The serving step's operators on the GPU against plain 64-bit forms: the
residual norm to codes, the router's top-k and the expert layer for a few
tokens.

Tolerances. A value rounded once is off by half a step of its type
(torch.finfo(t).eps / 2, relative); fp32 arithmetic before it adds:
  norm   the mean of K squares is summed over at most 64 + 30 additions in
         sequence: under 100 * 2^-24 = 6e-6, halved by the square root; the
         remaining handful of operations stay under 4e-6: 1e-5 in all;
  gate   exp(l - l0) of |l - l0| <= 100: the difference rounded to 2^-24 moves
         the result by at most 100 * 2^-24 = 6e-6, the exponentials' and the
         sums' own roundings (at most 64 + 4 terms in sequence) by under 6e-6
         more: 2e-5 covers it;
  layer  the products' own tolerance (tests/check.py), and exact equality
         where every sum is a whole number that fp32 holds.
"""
import math

import numpy as np
import pytest
import torch

from fp8_block_scaled_sa_amd import DGError, ops
from tests.check import assert_close
from tests.gpu_util import GUARD, bits, guards_intact, sentinel_bf16

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BF16, F32 = torch.bfloat16, torch.float32


def normal(shape, seed, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if outliers:
        x[torch.rand(shape, generator=g) < 1e-3] *= 50
    return x


def padded(t, pad, fill=None):
    """A device copy of t [M, K] inside rows of K + pad elements, and the whole buffer."""
    M, K = t.shape
    buf = torch.full((M, K + pad), 7 if fill is None else fill, dtype=t.dtype, device="cuda")
    buf[:, :K] = t.cuda()
    return buf[:, :K], buf


# ---------------------------------------------------------------- norm

def norm_reference(x, w, eps, r):
    h = x.double() + (r.double() if r is not None else 0)
    return h, h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def within(got, ref, rel, absolute=0.0):
    err = (got.double() - ref).abs()
    return bool((err <= rel * ref.abs() + absolute).all())


def half(dtype):
    return torch.finfo(dtype).eps / 2


def check_norm(x, w, eps, r, q, s, r_out, y):
    h, ref = norm_reference(x, w, eps, r)
    if r is not None:
        # the fp32 sum's rounding, then the type's (fp32: the same one); against cancellation, absolute
        assert within(r_out.cpu(), h, half(r.dtype), 2.0 ** -24 * float((x.double().abs() + r.double().abs()).max()))
    if y is not None:
        assert within(y.cpu(), ref, half(BF16) + 1e-5, 1e-38)
    M, K = x.shape
    blocks = ref.view(M, K // 128, 128)
    amax = blocks.abs().amax(2)
    s_ref = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert within(s.cpu(), s_ref, 1e-5)
    t = blocks / s_ref[:, :, None]
    got = q.cpu().view(F8).double().view(M, K // 128, 128)
    # half a step of a normal code is 2^-4 of the value, of a subnormal one 2^-10
    assert bool(((got - t).abs() <= torch.clamp(t.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 1e-3) + 1e-5 * t.abs()).all())
    # the largest value of a block takes the largest code
    assert bool((got.abs().amax(2) == torch.where(amax > 0, 448.0, 0.0)).all())


NORM_SHAPES = [(1, 128), (5, 512), (3, 640), (2, 1024), (70, 1152), (3, 2048), (9, 2176), (4, 4096), (3, 4224),
               (300, 7168), (2, 8192), (3, 8320), (2, 32768), (2, 32896), (1, 65536)]


@pytest.mark.parametrize("M,K", NORM_SHAPES)
@pytest.mark.parametrize("xt,rt,wt,normed", [(BF16, BF16, BF16, True), (BF16, F32, F32, False), (F32, F32, BF16, True),
                                             (F32, None, F32, False), (BF16, None, BF16, True), (F32, BF16, F32, True)])
def test_norm(gpu_device, M, K, xt, rt, wt, normed):
    x = normal((M, K), 1 + M + K).to(xt)
    w = (1 + 0.3 * normal((K,), 2, False)).to(wt)
    r = None if rt is None else (3 * normal((M, K), 3)).to(rt)
    out = ops.dg_fp8_rmsnorm_quantize_1x128(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda(),
                                            normed=normed)
    torch.cuda.synchronize()
    assert (out[2] is None) == (r is None) and (out[3] is None) == (not normed)
    check_norm(x, w, 1e-5, r, *out)


def test_norm_strides_in_place_and_guards(gpu_device):
    """Padded rows of every operand, row-major scales, the residual updated in
    place: same values, and nothing outside the outputs is written."""
    M, K = 37, 1408
    x, r, w = normal((M, K), 11).to(BF16), normal((M, K), 12).to(F32), normal((K,), 13, False).to(BF16)
    want = ops.dg_fp8_rmsnorm_quantize_1x128(x.cuda(), w.cuda(), 1e-6, residual=r.cuda(), normed=True)
    xd, _ = padded(x, 8)
    rd, rbuf = padded(r, 12)
    y, ybuf = padded(torch.zeros((M, K), dtype=BF16), 16)
    q, qbuf = padded(torch.zeros((M, K), dtype=torch.uint8), 32)
    sbuf = torch.full((M, K // 128 + 3), math.nan, device="cuda")
    got = ops.dg_fp8_rmsnorm_quantize_1x128(xd, w.cuda(), 1e-6, residual=rd, residual_out=rd, y=y, q=q,
                                            s=sbuf[:, :K // 128])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert got[2].data_ptr() == rd.data_ptr()
    for buf in (rbuf, ybuf, qbuf):
        assert bool((buf[:, K:] == 7).all())
    assert bool(sbuf[:, K // 128:].isnan().all())


def test_norm_special_rows(gpu_device):
    M, K = 6, 512
    x = normal((M, K), 21)
    x[0] = 0                            # a row of zeros: scale 1, codes 0
    x[1, 128:256] = 0                   # a block of zeros
    x[2] *= 1e-30                       # far below eps
    x[3] *= 1e15
    x[4, 5] = math.nan                  # the rows beside it stay what they are
    x[5, 200] = math.inf
    w = 1 + 0.1 * normal((K,), 22, False)
    q, s, _, y = ops.dg_fp8_rmsnorm_quantize_1x128(x.cuda(), w.cuda(), 1e-6, normed=True)
    torch.cuda.synchronize()
    # 1e-27 after the norm: values and scales near 2^-90, still normal numbers
    check_norm(x[:4], w, 1e-6, None, q[:4], s[:4], None, y[:4])
    assert bool((q[0] == 0).all()) and bool((s[0] == 1).all()) and float(s[1, 1]) == 1.0
    assert bool(y[4].isnan().all())
    assert bool(y[5, 200].isnan()) and bool((y[5, :200] == 0).all())


def test_norm_codes_are_the_quantisers(gpu_device):
    """With weight 1 and rows whose mean square plus eps is exactly 1, y is x
    itself: codes and scales equal the quantiser's bit for bit."""
    M, K = 20, 1024
    g = torch.Generator().manual_seed(5)
    x = torch.where(torch.rand((M, K), generator=g) < 0.5, -1.0, 1.0)  # squares: all 1
    x[:, ::2] *= 0.5                                                   # and 1/4: the mean is 0.625
    q, s, _, _ = ops.dg_fp8_rmsnorm_quantize_1x128(x.cuda(), torch.ones(K, device="cuda"), 0.375)
    q2, s2 = ops.dg_fp8_quantize_1x128(x.cuda())
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_norm_empty(gpu_device):
    x = torch.empty((0, 256), dtype=BF16, device="cuda")
    q, s, r, y = ops.dg_fp8_rmsnorm_quantize_1x128(x, torch.ones(256, device="cuda"), residual=x, normed=True)
    assert q.shape == (0, 256) and s.shape == (0, 2) and r.shape == (0, 256) and y.shape == (0, 256)


# ---------------------------------------------------------------- gate

def gate_reference(logits, k, score, renormalize, factor):
    l = logits.double().numpy().copy()  # noqa: E741
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        order = np.argsort(-l[t], kind="stable")[:k]
        order = order[l[t, order] > -np.inf]
        n = len(order)
        if not n:
            continue
        ids[t, :n] = order
        v = l[t, order]
        if score == "softmax":
            top = v[0]
            w = np.exp(v - top) / (np.exp(v - top) if renormalize else np.exp(l[t] - top)).sum()
        else:
            log = -np.logaddexp(0, -v)      # of the sigmoid
            w = np.exp(log)
            if renormalize:                 # a ratio, also where every sigmoid underflows
                w = np.exp(log - log.max())
                w = w / w.sum()
        weights[t, :n] = w * factor
    return ids, weights


def check_gate(logits, k, score, renormalize, factor=1.0, device_logits=None):
    d = logits.cuda() if device_logits is None else device_logits
    ids, weights = ops.dg_moe_gate_topk(d, k, score=score, renormalize=renormalize, factor=factor)
    torch.cuda.synchronize()
    ref_ids, ref_w = gate_reference(logits.cpu(), k, score, renormalize, factor)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    w = weights.cpu().double().numpy()
    assert np.all(np.abs(w - ref_w) <= 2e-5 * np.abs(ref_w) + 1e-37)
    assert np.all(w[ref_ids < 0] == 0)


GATE_SIZES = [(1, 1), (2, 2), (15, 3), (16, 16), (17, 5), (32, 8), (33, 1), (64, 6), (65, 16), (128, 8), (129, 7),
              (256, 8), (257, 8), (300, 10), (512, 16), (513, 4), (1000, 9), (1024, 16)]


@pytest.mark.parametrize("E,k", GATE_SIZES)
@pytest.mark.parametrize("T", [1, 37])
@pytest.mark.parametrize("dtype,score,renormalize", [(F32, "softmax", True), (BF16, "softmax", False),
                                                     (BF16, "sigmoid", True), (F32, "sigmoid", False)])
def test_gate(gpu_device, T, E, k, dtype, score, renormalize):
    check_gate((3 * normal((T, E), E + k, False)).to(dtype), k, score, renormalize, factor=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(5, 3), (48, 8), (200, 16), (700, 12)])
def test_gate_ties_and_masks(gpu_device, score, E, k):
    """A handful of distinct values (ties everywhere, of both zeros too), -inf
    and NaN in masked places, tokens with fewer candidates than slots or none."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randint(-2, 3, (60, E), generator=g).float() * 0.5
    logits[torch.rand((60, E), generator=g) < 0.3] = -math.inf
    logits[torch.rand((60, E), generator=g) < 0.1] = math.nan
    logits[::7] = -math.inf
    logits[1::7] = math.nan
    logits[2::7] = -math.inf
    logits[2::7, E - 1] = 1.5
    logits[3, :] = torch.tensor([0.0, -0.0]).repeat(E)[:E]
    logits[4, :] = torch.finfo(F32).min      # the type's lowest value is a candidate
    check_gate(logits, k, score, True)
    check_gate(logits, k, score, False)


def test_gate_far_logits(gpu_device):
    """Sigmoids that all underflow still renormalise; far apart logits give zeros, not NaN."""
    logits = torch.tensor([[-200.0, -201.0, -202.0, -300.0], [90.0, 60.0, -90.0, 0.0], [-3e38, -3e38, 3e38, 0.0]])
    ids, w = ops.dg_moe_gate_topk(logits.cuda(), 3, score="sigmoid")
    e = np.exp([0.0, -1.0, -2.0])
    assert np.allclose(w[0].cpu().numpy(), e / e.sum(), rtol=2e-5, atol=0)
    assert ids[2].tolist() == [2, 3, 0] and np.allclose(w[2].cpu().numpy(), [2 / 3, 1 / 3, 0], rtol=1e-6)
    ids, w = ops.dg_moe_gate_topk(logits.cuda(), 3)
    assert ids[1].tolist() == [0, 1, 3] and np.allclose(w[1].cpu().numpy(), [1, np.exp(-30.0), np.exp(-90.0)], rtol=2e-5)
    assert w[2].tolist() == [1.0, 0.0, 0.0]


def test_gate_strided_rows_given_outputs_and_empty(gpu_device):
    logits = normal((23, 96), 4, False)
    d, _ = padded(logits, 5, fill=99)        # larger values right behind each row
    check_gate(logits, 6, "softmax", True, device_logits=d)
    ids = torch.full((25, 6), -5, dtype=torch.int32, device="cuda")
    w = torch.full((25, 6), -5.0, device="cuda")
    got = ops.dg_moe_gate_topk(d, 6, ids=ids[1:24], weights=w[1:24])
    assert got[0].data_ptr() == ids[1:].data_ptr()
    assert bool((ids[[0, 24]] == -5).all()) and bool((w[[0, 24]] == -5).all())
    i, w = ops.dg_moe_gate_topk(logits[:0].cuda(), 6)
    assert i.shape == (0, 6) and w.shape == (0, 6)


def test_gate_many_tokens(gpu_device):
    check_gate(2 * normal((3000, 64), 8, False), 8, "softmax", True)


# ---------------------------------------------------------------- layer

def decode(codes):
    return codes.cpu().view(F8).double().numpy()


def spread(s, rows):
    s = np.repeat(s.cpu().double().numpy(), 128, axis=-1)
    return np.repeat(s, 128, axis=-2) if rows else s


def layer_reference(x, sx, w13, s13, w2, s2, ids, weights):
    xf = decode(x) * spread(sx, False)
    T, H = xf.shape
    E, I = w2.shape[0], w2.shape[2]  # noqa: E741
    ids, weights = ids.cpu().numpy(), weights.cpu().double().numpy()
    out = np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        both = xf[t] @ (decode(w13[e]) * spread(s13[e], True)).T
        g, u = both[:, :I], both[:, I:]
        y = (g / (1 + np.exp(-g)) * u) @ (decode(w2[e]) * spread(s2[e], True)).T
        np.add.at(out, t, weights[t, j][:, None] * y)
    return out


def to_bf16_bits(a):
    """bf16 bits of float64 values, rounded once."""
    f = a.astype(np.float32)
    # values here are exact in fp32, or far from a bf16 midpoint's neighbourhood that double rounding could cross
    return torch.from_numpy(f).to(BF16).view(torch.int16).numpy().view(np.uint16)


def make_layer(T, k, E, H, I, seed, ids="distinct"):  # noqa: E741
    g = torch.Generator().manual_seed(seed)
    rows = normal((T, H), seed + 1).view(T, H // 128, 128)
    sx = rows.abs().amax(2) / 448
    x = (rows / sx[:, :, None]).to(F8).view(torch.uint8).view(T, H)

    def weights(N, K):
        w = torch.randn((E, N // 128, 128, K // 128, 128), generator=g) * K ** -0.5
        s = w.abs().amax((2, 4)) / 448
        return (w / s[:, :, None, :, None]).to(F8).view(torch.uint8).view(E, N, K), s

    w13, s13 = weights(2 * I, H)
    w2, s2 = weights(H, I)
    if ids == "distinct":
        i = torch.rand((T, E), generator=g).argsort(1)[:, :k]
    elif ids == "one":
        i = torch.full((T, k), E // 2)
    elif ids == "sparse":   # most slots are another GPU's, or nonsense
        i = torch.randint(-3, 4 * E, (T, k), generator=g)
        i[0, 0], i[T // 2, 0] = -2 ** 31, 2 ** 31 - 1
    elif ids == "repeated":
        i = torch.randint(0, min(E, 2), (T, k), generator=g)
    else:
        i = torch.full((T, k), -1)
    w = torch.rand((T, k), generator=g) + 0.1
    w = w / w.sum(1, keepdim=True)
    return [t.cuda() for t in (x, sx, w13, s13, w2, s2, i.to(torch.int32), w)]


def run_layer(a, out=None, workspace=None, stream=None):
    T, H = a[0].shape
    if workspace is None:
        n = ops.dg_fp8_moe_layer_workspace_bytes(T, a[6].shape[1], H, a[4].shape[2])
        buf = torch.full((n + 2 * 2048,), 0xA5, dtype=torch.uint8, device="cuda")   # NaN-like garbage, guarded
        workspace = buf[2048:2048 + n]
    else:
        buf = None
    out = sentinel_bf16((T, H)) if out is None else out
    ops.dg_fp8_moe_layer(*a, workspace, out=out, stream=stream)
    torch.cuda.synchronize()
    if buf is not None:
        assert bool((buf[:2048] == 0xA5).all()) and bool((buf[-2048:] == 0xA5).all())
    return out


LAYERS = [
    (1, 1, 1, 128, 128, "distinct"), (1, 2, 8, 256, 384, "distinct"), (1, 8, 32, 1024, 512, "distinct"),
    (3, 2, 4, 384, 128, "distinct"), (5, 2, 8, 1024, 384, "distinct"), (16, 4, 8, 512, 256, "distinct"),
    (17, 3, 5, 640, 640, "distinct"), (33, 6, 16, 896, 384, "sparse"), (64, 8, 16, 512, 256, "distinct"),
    (64, 1, 4, 256, 256, "one"), (64, 16, 24, 256, 128, "distinct"), (64, 16, 3, 256, 128, "one"),
    (40, 5, 9, 256, 256, "repeated"), (2, 16, 1024, 128, 128, "distinct"), (7, 3, 6, 384, 256, "sparse"),
    (9, 4, 7, 256, 128, "none"), (32, 2, 3, 2944, 1152, "distinct"), (8, 8, 64, 256, 256, "distinct"),
]


@pytest.mark.parametrize("T,k,E,H,I,ids", LAYERS)
def test_layer(gpu_device, T, k, E, H, I, ids):  # noqa: E741
    a = make_layer(T, k, E, H, I, 100 + T + E, ids)
    out = run_layer(a)
    ref = layer_reference(*a)
    if ids != "none":
        assert_close(bits(out), to_bf16_bits(ref), "layer")
    none = ~((a[6] >= 0) & (a[6] < E)).any(1).cpu().numpy()
    assert not bits(out)[none].any(), "a token without an expert gets a row of zeros"


@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 3, 256, 128), (4, 2, 8, 384, 384), (20, 3, 4, 512, 256),
                                       (40, 2, 2, 256, 128), (64, 12, 16, 128, 256)])
def test_layer_whole_numbers(gpu_device, T, k, E, H, I):  # noqa: E741
    """Every operand a small whole number, gates of at least 32 (there
    g / (1 + exp(-g)) is g in fp32), up to 20 bits in the sums: the result has
    one right answer, whatever the order of the sums."""
    g = torch.Generator().manual_seed(T * 7 + k)
    ri = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g)  # noqa: E731
    x = torch.zeros((T, H))
    for t in range(T):
        x[t, torch.randperm(H, generator=g)[:9]] = 4.0
    w13 = torch.cat([ri(1, 2, E, I, H), ri(-1, 1, E, I, H)], 1).float()
    w2 = ri(-1, 1, E, H, I).float()
    code = lambda v: v.to(F8).view(torch.uint8)  # noqa: E731
    sx = 2.0 ** ri(0, 1, T, H // 128)
    x = x / sx.repeat_interleave(128, 1)          # exact: 4 or 2
    s13 = torch.ones((E, 2 * I // 128, H // 128))
    s2 = 2.0 ** ri(-1, 1, E, H // 128, I // 128)
    ids = torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32)
    weights = 2.0 ** ri(-1, 1, T, k)
    a = [t.cuda() for t in (code(x), sx.float(), code(w13), s13, code(w2), s2.float(), ids, weights.float())]
    ref = layer_reference(*a)
    whole = np.round(ref * 4) / 4      # 1 + exp(-36) is not quite 1 in fp64
    assert np.abs(ref - whole).max() < 1e-6 and np.abs(ref).max() < 2 ** 20
    ref = whole
    assert np.array_equal(bits(run_layer(a)), to_bf16_bits(ref))


def test_layer_strides_and_scale_layouts(gpu_device):
    """Padded rows, experts apart, broadcast and transposed scale tables, rows of
    a wider output: the same result, and nothing else is written."""
    T, k, E, H, I = 6, 2, 3, 256, 128  # noqa: E741
    a = make_layer(T, k, E, H, I, 31)
    a[3] = a[3][:, :, :1].expand(E, 2, 2)                    # one scale for all of K
    a[5] = a[5][:1, :1, :1].expand(E, 2, 1)                  # one scale for everything
    want = bits(run_layer([t.contiguous() for t in a]))
    x, _ = padded(a[0].cpu(), 48)
    w13 = torch.full((E, 2 * I + 8, H + 16), 0x7F, dtype=torch.uint8, device="cuda")   # NaN codes around
    w13[:, :2 * I, :H] = a[2]
    w2 = torch.full((E, H + 1, I + 32), 0x7F, dtype=torch.uint8, device="cuda")
    w2[:, :H, :I] = a[4]
    wide = torch.full((T, H + 24), 5.0, dtype=BF16, device="cuda")
    b = [x, a[1].t().contiguous().t(), w13[:, :2 * I, :H], a[3], w2[:, :H, :I], a[5], a[6], a[7]]
    run_layer(b, out=wide[:, :H])
    assert np.array_equal(bits(wide[:, :H]), want)
    assert bool((wide[:, H:] == 5).all())
    b[0] = b[0].view(F8)
    b[2], b[4] = b[2].view(F8), b[4].view(F8)
    assert np.array_equal(bits(run_layer(b)), want)


def test_layer_skipped_slots_read_nothing(gpu_device):
    """The weight of a slot without an expert is not used (NaN there), nor are
    the experts that no token chose (NaN codes), nor other tokens' rows."""
    T, k, E, H, I = 18, 3, 6, 256, 256  # noqa: E741
    a = make_layer(T, k, E, H, I, 41)
    a[6][a[6] >= 4] = -1                       # experts 4 and 5 are not chosen
    a[6][5] = -1                               # token 5 has none
    want = bits(run_layer(a))
    b = [t.clone() for t in a]
    b[2][4:], b[4][4:] = 0x7F, 0x7F
    b[3][4:], b[5][4:] = math.nan, math.nan
    b[7][a[6] < 0] = math.nan
    b[0][5], b[1][5] = 0x7F, math.nan
    assert np.array_equal(bits(run_layer(b)), want)
    b[0][3, 7] = 0x7F                          # a NaN in token 3 stays in its row
    got = bits(run_layer(b))
    other = [t for t in range(T) if t != 3]
    assert np.array_equal(got[other], want[other])
    if bool((a[6][3] >= 0).any()):
        assert np.all((got[3] & 0x7FFF) > 0x7F80)


def test_layer_infinite_h(gpu_device):
    """g * u beyond fp32 is infinite, and so is what positive weights make of
    it, not NaN; the other token is not touched."""
    T, k, E, H, I = 2, 1, 1, 128, 128  # noqa: E741
    one = torch.full((E, 2 * I, H), 0x38, dtype=torch.uint8)        # code of 1
    x = torch.full((T, H), 0x38, dtype=torch.uint8)
    sx = torch.tensor([[2.0 ** 70], [1.0]])
    a = [t.cuda() for t in (x, sx, one, torch.ones((E, 2, 1)), one[:, :H, :I].contiguous(), torch.ones((E, 1, 1)),
                            torch.zeros((T, k), dtype=torch.int32), torch.ones((T, k)))]
    out = run_layer(a).float().cpu()
    assert bool((out[0] == math.inf).all())
    assert bool((out[1] == 128.0 ** 3).all())


def test_layer_same_on_every_run_and_stream(gpu_device):
    a = make_layer(24, 4, 8, 512, 384, 51)
    want = bits(run_layer(a))
    side = torch.cuda.Stream()
    for i in range(20):
        side.wait_stream(torch.cuda.current_stream())
        assert np.array_equal(bits(run_layer(a, stream=side if i % 2 else None)), want)


def test_layer_workspace_too_small(gpu_device):
    a = make_layer(4, 2, 4, 256, 128, 61)
    n = ops.dg_fp8_moe_layer_workspace_bytes(4, 2, 256, 128)
    out = sentinel_bf16((4, 256))
    before = bits(out).copy()
    for ws in (None, torch.empty(n - 16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(DGError):
            ops.dg_fp8_moe_layer(*a, ws, out=out)
    torch.cuda.synchronize()
    assert np.array_equal(bits(out), before)


def test_layer_empty(gpu_device):
    a = make_layer(2, 2, 4, 256, 128, 62)
    for i in (0, 1, 6, 7):
        a[i] = a[i][:0]
    assert ops.dg_fp8_moe_layer(*a, None).shape == (0, 256)


# ---------------------------------------------------------------- offsets past 32 bits

def test_norm_offsets_past_32_bits(gpu_device):
    """More than 2^31 elements: the last rows are what a call on them alone gives."""
    M, K = 270000, 8192
    x = torch.empty((M, K), dtype=BF16, device="cuda")
    x[-4:] = normal((4, K), 7).to(BF16).cuda()
    w = torch.ones(K, dtype=BF16, device="cuda")
    q, s, _, _ = ops.dg_fp8_rmsnorm_quantize_1x128(x, w)
    q2, s2, _, _ = ops.dg_fp8_rmsnorm_quantize_1x128(x[-4:].clone(), w)
    assert torch.equal(q[-4:], q2) and torch.equal(s[-4:], s2)


def test_gate_offsets_past_32_bits(gpu_device):
    T, E = 2200000, 1024
    logits = torch.empty((T, E), dtype=BF16, device="cuda")
    logits[-5:] = normal((5, E), 8).to(BF16).cuda()
    ids, weights = ops.dg_moe_gate_topk(logits, 8)
    ids2, weights2 = ops.dg_moe_gate_topk(logits[-5:].clone(), 8)
    assert torch.equal(ids[-5:], ids2) and torch.equal(weights[-5:], weights2)


def test_layer_offsets_past_32_bits(gpu_device):
    """Experts more than 4 GiB apart."""
    T, k, E, H, I = 3, 2, 3, 256, 128  # noqa: E741
    a = make_layer(T, k, E, H, I, 91)
    want = bits(run_layer(a))
    apart = (1 << 32) + 4096
    pool = torch.empty(2 * apart + (2 << 20), dtype=torch.uint8, device="cuda")
    for i, rows, cols in ((2, 2 * I, H), (4, H, I)):
        far = pool.as_strided((E, rows, cols), (apart, cols, 1), 0 if i == 2 else 1 << 20)
        far.copy_(a[i])
        a[i] = far
    assert np.array_equal(bits(run_layer(a)), want)


# ---------------------------------------------------------------- together

def test_step_in_a_graph(gpu_device):
    """Norm, router and layer captured once and replayed with new activations
    (other experts chosen): every replay equals the eager calls bit for bit."""
    T, k, E, H, I = 12, 3, 8, 512, 256  # noqa: E741
    _, _, w13, s13, w2, s2, _, _ = make_layer(T, k, E, H, I, 71)
    x, r = torch.zeros((T, H), dtype=BF16, device="cuda"), torch.zeros((T, H), dtype=BF16, device="cuda")
    logits = torch.zeros((T, E), device="cuda")
    norm_w = (1 + 0.1 * normal((H,), 72, False)).to(BF16).cuda()
    ws = ops.workspace(ops.dg_fp8_moe_layer_workspace_bytes(T, k, H, I))

    def step():
        q, s, r_out, _ = ops.dg_fp8_rmsnorm_quantize_1x128(x, norm_w, residual=r)
        ids, weights = ops.dg_moe_gate_topk(logits, k)
        return r_out, ids, weights, ops.dg_fp8_moe_layer(q, s, w13, s13, w2, s2, ids, weights, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(5):
        x.copy_(normal((T, H), 80 + seed).to(BF16))
        r.copy_(normal((T, H), 90 + seed).to(BF16))
        logits.copy_(normal((T, E), 95 + seed, False))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_guard_band_helper_sees_writes(gpu_device):
    out = sentinel_bf16((2, 128))
    assert guards_intact(out) and GUARD > 0


def test_example_step(gpu_device):
    """examples/moe_decode_step.py on a small block: the step is its own 64-bit form up to the output's rounding."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_decode_step.py")
    spec = importlib.util.spec_from_file_location("moe_decode_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    block = example.MoeBlock(hidden=512, width=256, experts=8, top_k=3, max_tokens=20)
    x, residual = normal((20, 512), 5).to(BF16).cuda(), normal((20, 512), 6).to(BF16).cuda()
    exact = block.reference(x, residual)
    total = (x.float() + residual.float()).to(BF16)
    out = block.step(x, residual)
    torch.cuda.synchronize()
    assert torch.equal(residual, total)
    # the norm of a sum of rounding errors of half a step each
    assert float((out.double() - exact).norm()) <= half(BF16) * float(exact.norm())
