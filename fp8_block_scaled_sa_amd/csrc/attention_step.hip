// attention_step.hip -- C ABI of the operators over a paged cache of e4m3 codes
// (declared in include/dg_fp8.h): rotary positions and the cache's write, its
// read, and attention of new tokens over it. Host-side validation, kernel
// choice and launch; nothing is allocated and no stream is synchronised.
// Compiled behind moe_step.hip (library.hip), whose checks it shares.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <math.h>
#include <numeric>
#include <stdint.h>
#include <utility>

#include "attend.hpp"
#include "cache.hpp"
#include "dg_fp8.h"

namespace {

constexpr int64_t kMaxPageSize = (int64_t)1 << 20;
constexpr int64_t kMaxContext = (int64_t)1 << 30;      // tokens that a row of the page table spans
constexpr int64_t kMaxCacheStride = (int64_t)1 << 40;

// One strided dimension of an output: size and stride in elements.
struct Dim {
    int64_t size, stride;
};

// Whether rows of `inner` elements at all index combinations lie apart, with the dimensions nested in some order.
bool rows_apart(std::initializer_list<Dim> dims, int64_t inner)
{
    Dim d[3];
    int n = 0;
    for (const Dim &x : dims)
        if (x.size > 1)
            d[n++] = x;
    std::sort(d, d + n, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    int64_t span = inner;
    for (int i = 0; i < n; ++i) {
        if (d[i].stride < span)
            return false;
        span += (d[i].size - 1) * d[i].stride;
    }
    return true;
}

// A dimension of two sets of rows: how far an index of the second may lie from one of the first.
struct Step {
    int64_t stride, low, high;
};

constexpr int64_t kFar = (int64_t)1 << 60;

// Whether blocks of two sets may meet, of `first` and `second` elements, the second set's `offset` behind the first's
// where all indices are 0. Steps with strides falling, none 0. Exact where the dimensions nest; where a step has more
// indices than these to look at, they do not.
bool blocks_meet(const Step *steps, int n, int64_t offset, int64_t first, int64_t second)
{
    if (n == 0)
        return offset > -second && offset < first;
    int64_t reach = std::max(first, second), more;
    for (int i = 1; i < n; ++i)
        if (__builtin_mul_overflow(std::max(-steps[i].low, steps[i].high), steps[i].stride, &more) || more > kFar ||
            (reach += more) > kFar)
            return true;
    // |offset + i stride| < reach
    const auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    const int64_t from = std::max(steps->low, floor_div(-reach - offset, steps->stride) + 1);
    const int64_t to = std::min(steps->high, -floor_div(offset - reach, steps->stride) - 1);
    constexpr int64_t kTries = 16;
    if (to - from >= kTries)
        return true;
    for (int64_t i = from; i <= to; ++i)
        if (blocks_meet(steps + 1, n - 1, offset + i * steps->stride, first, second))
            return true;
    return false;
}

// Whether a row of one set may meet one of the other, both of `inner` elements: not where a reading of the strides
// shows them apart. Strides that differ are read as blocks as long as the dimension reaches, or as all places that the
// two can come to.
bool rows_meet(std::initializer_list<std::pair<Dim, Dim>> dims, int64_t offset, int64_t inner)
{
    for (const bool blocks : {true, false}) {
        Step steps[3];
        int n = 0;
        int64_t first = inner, second = inner, more, and_more;
        for (const auto &[a, b] : dims) {
            const int64_t s = a.size > 1 ? a.stride : 0, t = b.size > 1 ? b.stride : 0;
            if (s == 0 && t == 0)
                continue;
            if (s == 0 || t == 0 || s == t) {
                steps[n++] = Step{std::max(s, t), s ? 1 - a.size : 0, t ? b.size - 1 : 0};
            } else if (!blocks) {
                steps[n++] = Step{std::gcd(s, t), -((int64_t)1 << 40), (int64_t)1 << 40};
            } else {
                if (__builtin_mul_overflow(a.size - 1, s, &more) || __builtin_mul_overflow(b.size - 1, t, &and_more) ||
                    more > kFar || and_more > kFar)
                    return true;
                first = std::min(first + more, kFar);
                second = std::min(second + and_more, kFar);
            }
        }
        std::sort(steps, steps + n, [](const Step &a, const Step &b) { return a.stride > b.stride; });
        if (!blocks_meet(steps, n, offset, first, second))
            return false;
    }
    return true;
}

int check_head_dim(int64_t D)
{
    return D <= 0 ? DG_ERR_BAD_SHAPE : D == 64 || D == 128 ? DG_OK : DG_ERR_UNSUPPORTED;
}

int check_cache_sizes(const dg_fp8_cache &c)
{
    if (c.pages <= 0 || c.page_size <= 0 || c.heads <= 0)
        return DG_ERR_BAD_SHAPE;
    const int st = check_head_dim(c.head_dim);
    if (st != DG_OK)
        return st;
    if (c.page_size > kMaxPageSize || c.pages > kInt32Max / c.page_size || c.heads > 65536)
        return DG_ERR_UNSUPPORTED;
    return DG_OK;
}

int check_cache(const dg_fp8_cache &c, bool written)
{
    if (!c.codes || !c.scales)
        return DG_ERR_NULL_POINTER;
    const int64_t strides[6] = {c.stride_page,   c.stride_token,   c.stride_head,
                                c.s_stride_page, c.s_stride_token, c.s_stride_head};
    for (int64_t s : strides)
        if (s < 0)
            return DG_ERR_BAD_STRIDE;
    for (int64_t s : strides)
        if (s > kMaxCacheStride)
            return DG_ERR_UNSUPPORTED;
    if (written && (!rows_apart({{c.pages, c.stride_page}, {c.page_size, c.stride_token}, {c.heads, c.stride_head}},
                                c.head_dim) ||
                    !rows_apart({{c.pages, c.s_stride_page}, {c.page_size, c.s_stride_token}, {c.heads, c.s_stride_head}},
                                1)))
        return DG_ERR_BAD_STRIDE;
    // The kernels keep a slot's offset in units of 16 bytes in 32 bits.
    if ((c.pages - 1) * (c.stride_page / 16) >= ((int64_t)1 << 32) ||
        (c.pages - 1) * (c.stride_page / 16) + (c.page_size - 1) * (c.stride_token / 16) >= ((int64_t)1 << 32))
        return DG_ERR_UNSUPPORTED;
    if (!aligned(c.codes, 16) || !aligned(c.scales, 4) || (c.pages > 1 && c.stride_page % 16) ||
        (c.page_size > 1 && c.stride_token % 16) || (c.heads > 1 && c.stride_head % 16))
        return DG_ERR_MISALIGNED;
    return DG_OK;
}

Extent codes_extent(const dg_fp8_cache &c)
{
    return extent(c.codes, 1, (c.pages - 1) * c.stride_page + (c.page_size - 1) * c.stride_token +
                                  (c.heads - 1) * c.stride_head + c.head_dim - 1);
}

Extent scales_extent(const dg_fp8_cache &c)
{
    return extent(c.scales, 4, (c.pages - 1) * c.s_stride_page + (c.page_size - 1) * c.s_stride_token +
                                   (c.heads - 1) * c.s_stride_head);
}

// Strides of a [T, heads, D] tensor of rows: 16-byte multiples.
int check_rows(int64_t stride_t, int64_t stride_h, int64_t T, int64_t heads, int64_t size)
{
    if (stride_t < 0 || stride_h < 0)
        return DG_ERR_BAD_STRIDE;
    if (!strides_fit({stride_t, stride_h}))
        return DG_ERR_UNSUPPORTED;
    if ((T > 1 && (stride_t * size) % 16) || (heads > 1 && (stride_h * size) % 16))
        return DG_ERR_MISALIGNED;
    return DG_OK;
}

Extent rows_extent(const void *p, int64_t size, int64_t T, int64_t stride_t, int64_t heads, int64_t stride_h, int64_t D)
{
    return extent(p, size, (T - 1) * stride_t + (heads - 1) * stride_h + D - 1);
}

dgc::Pages pages_of(const dg_fp8_cache &c)
{
    return dgc::Pages{(uint8_t *)c.codes, c.stride_page,   c.stride_token,   c.stride_head,
                      c.scales,           c.s_stride_page, c.s_stride_token, c.s_stride_head};
}

dga::Rows rows_of(const dg_fp8_cache &c)
{
    return dga::Rows{(const uint8_t *)c.codes, (uint32_t)(c.stride_page / 16), (uint32_t)(c.stride_token / 16),
                     c.stride_head,            c.scales,                       c.s_stride_page,
                     c.s_stride_token,         c.s_stride_head};
}

// ---------------------------------------------------------------- write, read

template <bool BF16>
int launch_write(dgc::WriteParams &p, int64_t D, hipStream_t stream)
{
    const int in_round = dgc::kThreads / ((int)D / 8), rows = p.q_heads + 2 * p.heads;
    p.tokens = std::min(std::max(in_round / rows, 1), dgc::kMaxTokens);
    const int grid = (p.T + p.tokens - 1) / p.tokens;
    // Few tokens: one round of rows a workgroup, for latency.
    const int rounds = (p.tokens * rows + in_round - 1) / in_round;
    const dim3 blocks((unsigned)grid, (unsigned)(grid < 256 ? std::min(rounds, 64) : 1));
    if (D == 64)
        hipLaunchKernelGGL((dgc::rope_cache_write_kernel<BF16, 64>), blocks, dim3(dgc::kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((dgc::rope_cache_write_kernel<BF16, 128>), blocks, dim3(dgc::kThreads), 0, stream, p);
    return launched();
}

template <bool BF16>
int launch_read(const dgc::ReadParams &p, int64_t D, hipStream_t stream)
{
    const int64_t rows = dgc::kReadRows * dgc::kThreads / (D / (BF16 ? 8 : 4));
    const dim3 blocks((unsigned)((p.rows + rows - 1) / rows));
    if (D == 64)
        hipLaunchKernelGGL((dgc::cache_read_kernel<BF16, 64>), blocks, dim3(dgc::kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((dgc::cache_read_kernel<BF16, 128>), blocks, dim3(dgc::kThreads), 0, stream, p);
    return launched();
}

// ---------------------------------------------------------------- attention

// Which kernels take a call, and what they need, from what the host knows.
struct AttendPlan {
    int tiles;             // 16-row tiles of the few-rows kernel (0: none of the sequences is its)
    int few_rows;          // rows up to which a sequence is its
    int64_t pieces;        // its workgroups at most, which is what its partial results take
    int64_t part_rows;     // rows of a piece's partial result
    bool many;             // whether there can be sequences of more rows, the many-rows kernel's
    int64_t many_tiles;    // their tiles, of all key heads, at most
    int64_t many_rows;     // rows of a cut tile's partial result
    int64_t bytes;         // of the workspace
    int64_t most_bytes;    // of the workspace of any call with at most these sizes
};

// Pieces that the few-rows kernel's work is cut into: four workgroups for each CU, of which two run at a time. (64
// sequences up to 16384 tokens and 16 of 4 tokens up to 8192: 251 and 55 us with 512, 227 and 56 with 1024, 225 and 64
// with 2048.)
constexpr int kFewTarget = 1024;
// Rows from which on each wave of the joining launch takes one by itself; below, the four of a workgroup share it (one
// token over 4000: 10.4 us, 12.4 with a wave a row; 4096 rows: 59 us, 56 with a wave a row).
constexpr int64_t kRowAWave = 2048;
// Workgroups up to which the many-rows kernel's tiles are cut, three rounds of one a CU. How many tiles there are, and
// whether they are cut, is found on the device: the host knows sizes for which there can be thousands (500 single tokens
// and a chunk of 64, 8 heads of 8: 2248) where there are few (16): 100 tokens each and the chunk's 32768 take 1087 us
// uncut, 348 us cut.
constexpr int64_t kMostPieces = 768;

AttendPlan plan_attend(int64_t T, int64_t B, int64_t heads, int64_t group, int64_t D, int64_t max_q_len)
{
    AttendPlan a = {};
    const int64_t longest = std::min(max_q_len, T), rows = longest * group;
    const bool many = a.many = rows > dga::kFewRows;
    // Beside chunks, the few-rows kernel has all sequences of up to 32 rows, which a tile of 256 would pay for in full
    // (16 sequences of 4 tokens up to 8192 beside a chunk of 512, 8 heads of 8: 366 us with up to 16 rows, 249 with 32;
    // 60 of 4 up to 2000 beside 300: 141 and 91); but where the longest leaves no more than a token for each other one,
    // it has these alone, in its form of one tile if that holds them (64 single tokens up to 8192 beside a chunk of 512:
    // 333 us, 341 in the form of two; 500 of 100 beside 64 over 32768: 348 and 398). One sequence alone takes one kernel.
    const int64_t beside = T - longest < B ? group : dga::kFewRows;
    const int64_t few = !many ? rows : B > 1 && group <= dga::kFewRows ? beside : 0;
    a.tiles = few == 0 ? 0 : few <= 16 ? 1 : 2;
    a.few_rows = 16 * a.tiles;
    if (a.tiles) {
        a.pieces = kFewTarget + B * heads;
        a.part_rows = many ? a.few_rows : rows;
        a.bytes = a.pieces * a.part_rows * (D + 2) * 4;
    }
    a.most_bytes = (kFewTarget + B * heads) * std::min<int64_t>(dga::kFewRows, rows) * (D + 2) * 4;
    if (many) {
        // Sequences that have tiles have more rows than the few-rows kernel's.
        const int64_t sequences = std::min(std::min(B, T), T * group / (a.few_rows + 1));
        a.many_tiles = (T * group + sequences * (dga::kTileRows - 1)) / dga::kTileRows * heads;
        a.many_rows = std::min<int64_t>(dga::kTileRows, rows);
        a.bytes += kMostPieces * a.many_rows * (D + 2) * 4;
        a.most_bytes += kMostPieces * a.many_rows * (D + 2) * 4;
    }
    return a;
}

int check_attend_sizes(int64_t T, int64_t B, int64_t q_heads, int64_t heads, int64_t D, int64_t max_q_len)
{
    if (T < 0 || B < 0 || q_heads <= 0 || heads <= 0 || q_heads % heads || max_q_len <= 0)
        return DG_ERR_BAD_SHAPE;
    const int st = check_head_dim(D);
    if (st != DG_OK)
        return st;
    constexpr int64_t kMaxPieces = ((int64_t)1 << 24) - 1;     // of 256 threads
    if (T > kInt32Max || B > kMaxPieces || q_heads > 65536 || T * q_heads > kInt32Max)
        return DG_ERR_UNSUPPORTED;
    if (T == 0 || B == 0)
        return DG_OK;
    const AttendPlan a = plan_attend(T, B, heads, q_heads / heads, D, max_q_len);
    if (a.pieces > kMaxPieces || a.many_tiles > kMaxPieces / 3 || B * heads * a.part_rows > kMaxPieces - dga::kJoinGroups)
        return DG_ERR_UNSUPPORTED;
    return DG_OK;
}

template <int D>
int launch_attend(dga::AttendParams &p, const AttendPlan &a, int64_t units, hipStream_t stream)
{
    const dim3 threads(dga::kThreads);
    p.few_rows = a.few_rows;
    int st;
    int64_t joined = 0;
    float *parts = p.few.o;
    if (a.tiles) {
        p.target = kFewTarget;
        p.few = dga::Parts{(int)a.part_rows, parts, parts + a.pieces * a.part_rows * D};
        parts += a.pieces * a.part_rows * (D + 2);
        // A sequence and head has a piece for each unit at most.
        const dim3 grid((unsigned)std::min<int64_t>(a.pieces, p.B * p.heads * std::max<int64_t>(units, 1)));
        if (a.tiles == 1)
            hipLaunchKernelGGL((dga::attend_few_kernel<D, 1>), grid, threads, 0, stream, p);
        else
            hipLaunchKernelGGL((dga::attend_few_kernel<D, 2>), grid, threads, 0, stream, p);
        if ((st = launched()) != DG_OK)
            return st;
        if (units > 1) {
            joined = p.B * p.heads * a.part_rows;
            p.row_a_wave = joined >= kRowAWave;
            p.few_joined = (int)(joined = p.row_a_wave ? (joined + 3) / 4 : joined);
        }
    }
    if (a.many) {
        p.most_pieces = (int)kMostPieces;
        p.many = dga::Parts{(int)a.many_rows, parts, parts + kMostPieces * a.many_rows * D};
        hipLaunchKernelGGL((dga::attend_many_kernel<D>), dim3((unsigned)std::max(a.many_tiles, kMostPieces)),
                           dim3(dga::kManyThreads), 0, stream, p);
        if ((st = launched()) != DG_OK)
            return st;
        joined += std::min<int64_t>(dga::kJoinGroups, std::min(a.many_tiles, kMostPieces / 2) *
                                                          ((a.many_rows + dga::kJoinRows - 1) / dga::kJoinRows));
    }
    if (joined) {
        hipLaunchKernelGGL((dga::join_kernel<D>), dim3((unsigned)joined), threads, 0, stream, p);
        return launched();
    }
    return DG_OK;
}

}  // namespace

extern "C" {

dg_status dg_fp8_rope_cache_write(const void *Q, int64_t q_stride_t, int64_t q_stride_h, void *Q_out,
                                  int64_t qo_stride_t, int64_t qo_stride_h, int64_t q_heads, const void *K,
                                  int64_t k_stride_t, int64_t k_stride_h, const void *V, int64_t v_stride_t,
                                  int64_t v_stride_h, int x_dtype, const int32_t *positions, const double *freqs,
                                  int64_t rot, int interleaved, float factor, const int64_t *slots,
                                  const dg_fp8_cache *k_cache, const dg_fp8_cache *v_cache, int64_t T, void *stream)
{
    if (!k_cache || !v_cache)
        return DG_ERR_NULL_POINTER;
    const dg_fp8_cache &kc = *k_cache, &vc = *v_cache;
    int st;
    if ((st = check_cache_sizes(kc)) != DG_OK || (st = check_cache_sizes(vc)) != DG_OK)
        return (dg_status)st;
    const int64_t D = kc.head_dim, heads = kc.heads;
    if (T < 0 || vc.pages != kc.pages || vc.page_size != kc.page_size || vc.heads != heads || vc.head_dim != D ||
        rot < 0 || rot > D || rot % 16 || (Q ? q_heads <= 0 : q_heads != 0))
        return DG_ERR_BAD_SHAPE;
    if (!is_float_type(x_dtype) || q_heads > 65536 || T > kInt32Max || !threads_fit(std::max<int64_t>(T, 256 * 64), 256))
        return DG_ERR_UNSUPPORTED;
    if (T == 0)
        return DG_OK;
    if (!K || !V || !slots || (Q && !Q_out) || (rot && (!positions || !freqs)))
        return DG_ERR_NULL_POINTER;
    const int64_t size = x_dtype == DG_DTYPE_BF16 ? 2 : 4;
    if ((st = check_cache(kc, true)) != DG_OK || (st = check_cache(vc, true)) != DG_OK ||
        (st = check_rows(k_stride_t, k_stride_h, T, heads, size)) != DG_OK ||
        (st = check_rows(v_stride_t, v_stride_h, T, heads, size)) != DG_OK)
        return (dg_status)st;
    if (Q && ((st = check_rows(q_stride_t, q_stride_h, T, q_heads, size)) != DG_OK ||
              (st = check_rows(qo_stride_t, qo_stride_h, T, q_heads, 2)) != DG_OK))
        return (dg_status)st;
    if (Q && !rows_apart({{T, qo_stride_t}, {q_heads, qo_stride_h}}, D))
        return DG_ERR_BAD_STRIDE;
    if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 8) || (Q && (!aligned(Q, 16) || !aligned(Q_out, 16))) ||
        (rot && (!aligned(positions, 4) || !aligned(freqs, 8))))
        return DG_ERR_MISALIGNED;
    const Extent none = {0, 0};
    const Extent ins[6] = {Q ? rows_extent(Q, size, T, q_stride_t, q_heads, q_stride_h, D) : none,
                           rows_extent(K, size, T, k_stride_t, heads, k_stride_h, D),
                           rows_extent(V, size, T, v_stride_t, heads, v_stride_h, D),
                           extent(slots, 8, T - 1), rot ? extent(positions, 4, T - 1) : none,
                           rot ? extent(freqs, 8, rot / 2 - 1) : none};
    const Extent outs[5] = {codes_extent(kc), codes_extent(vc), scales_extent(kc), scales_extent(vc),
                            Q ? rows_extent(Q_out, 2, T, qo_stride_t, q_heads, qo_stride_h, D) : none};
    // Q_out may be Q itself (each row is read before it is written), also where Q, K and V are columns of one tensor, but
    // not where a row of K or V is one of Q.
    const bool in_place = Q && Q_out == Q && size == 2 && (T == 1 || qo_stride_t == q_stride_t) &&
                          (q_heads == 1 || qo_stride_h == q_stride_h);
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < 6; ++j)
            if (overlaps(outs[i], ins[j]) && !(i == 4 && in_place && j < 3))
                return DG_ERR_ALIASING;
    const auto among_queries = [&](const void *X, int64_t x_t, int64_t x_h) {
        return rows_meet({{{T, q_stride_t}, {T, x_t}}, {{q_heads, q_stride_h}, {heads, x_h}}},
                         ((const uint8_t *)X - (const uint8_t *)Q) / size, D);
    };
    if (in_place && ((overlaps(outs[4], ins[1]) && among_queries(K, k_stride_t, k_stride_h)) ||
                     (overlaps(outs[4], ins[2]) && among_queries(V, v_stride_t, v_stride_h))))
        return DG_ERR_ALIASING;
    // The two caches may be halves of one tensor, page by page or row by row, with no row in both; codes and scales lie
    // apart.
    if ((overlaps(outs[0], outs[1]) &&
         rows_meet({{{kc.pages, kc.stride_page}, {vc.pages, vc.stride_page}},
                    {{kc.page_size, kc.stride_token}, {vc.page_size, vc.stride_token}},
                    {{heads, kc.stride_head}, {heads, vc.stride_head}}},
                   (const uint8_t *)vc.codes - (const uint8_t *)kc.codes, D)) ||
        (overlaps(outs[2], outs[3]) &&
         rows_meet({{{kc.pages, kc.s_stride_page}, {vc.pages, vc.s_stride_page}},
                    {{kc.page_size, kc.s_stride_token}, {vc.page_size, vc.s_stride_token}},
                    {{heads, kc.s_stride_head}, {heads, vc.s_stride_head}}},
                   vc.scales - kc.scales, 1)))
        return DG_ERR_ALIASING;
    for (int i = 0; i < 2; ++i)
        for (int j = 2; j < 4; ++j)
            if (overlaps(outs[i], outs[j]))
                return DG_ERR_ALIASING;
    for (int i = 0; i < 4; ++i)
        if (overlaps(outs[i], outs[4]))
            return DG_ERR_ALIASING;
    DeviceInfo dev;
    if ((st = current_device(dev)) != DG_OK)
        return (dg_status)st;
    dgc::WriteParams p = {};
    p.Q = Q; p.q_t = q_stride_t; p.q_h = q_stride_h;
    p.Q_out = (uint16_t *)Q_out; p.qo_t = qo_stride_t; p.qo_h = qo_stride_h;
    p.K = K; p.k_t = k_stride_t; p.k_h = k_stride_h;
    p.V = V; p.v_t = v_stride_t; p.v_h = v_stride_h;
    p.positions = positions; p.freqs = freqs; p.slots = slots;
    p.k = pages_of(kc); p.v = pages_of(vc);
    p.page = dgc::divisor((uint32_t)kc.page_size);
    p.slots_in_all = kc.pages * kc.page_size;
    p.T = (int)T; p.q_heads = (int)q_heads; p.heads = (int)heads;
    p.half = (int)rot / 2; p.interleaved = interleaved != 0; p.factor = factor;
    const hipStream_t s = (hipStream_t)stream;
    return (dg_status)(x_dtype == DG_DTYPE_BF16 ? launch_write<true>(p, D, s) : launch_write<false>(p, D, s));
}

dg_status dg_fp8_cache_read(const dg_fp8_cache *cache, const int64_t *slots, void *out, int out_dtype,
                            int64_t out_stride_t, int64_t out_stride_h, int64_t T, void *stream)
{
    if (!cache)
        return DG_ERR_NULL_POINTER;
    const dg_fp8_cache &c = *cache;
    int st = check_cache_sizes(c);
    if (st != DG_OK)
        return (dg_status)st;
    if (T < 0)
        return DG_ERR_BAD_SHAPE;
    if (!is_float_type(out_dtype) || T > kInt32Max / c.heads || !threads_fit(T * c.heads / 4, c.head_dim / 4))
        return DG_ERR_UNSUPPORTED;
    if (T == 0)
        return DG_OK;
    if (!slots || !out)
        return DG_ERR_NULL_POINTER;
    const int64_t size = out_dtype == DG_DTYPE_BF16 ? 2 : 4, D = c.head_dim;
    if ((st = check_cache(c, false)) != DG_OK || (st = check_rows(out_stride_t, out_stride_h, T, c.heads, size)) != DG_OK)
        return (dg_status)st;
    if (!rows_apart({{T, out_stride_t}, {c.heads, out_stride_h}}, D))
        return DG_ERR_BAD_STRIDE;
    if (!aligned(slots, 8) || !aligned(out, 16))
        return DG_ERR_MISALIGNED;
    const Extent eo = rows_extent(out, size, T, out_stride_t, c.heads, out_stride_h, D);
    if (overlaps(eo, codes_extent(c)) || overlaps(eo, scales_extent(c)) || overlaps(eo, extent(slots, 8, T - 1)))
        return DG_ERR_ALIASING;
    DeviceInfo dev;
    if ((st = current_device(dev)) != DG_OK)
        return (dg_status)st;
    dgc::ReadParams p = {};
    p.from = pages_of(c); p.slots = slots;
    p.out = out; p.o_t = out_stride_t; p.o_h = out_stride_h;
    p.page = dgc::divisor((uint32_t)c.page_size);
    p.head = dgc::divisor((uint32_t)c.heads);
    p.slots_in_all = c.pages * c.page_size;
    p.rows = T * c.heads;
    const hipStream_t s = (hipStream_t)stream;
    return (dg_status)(out_dtype == DG_DTYPE_BF16 ? launch_read<true>(p, D, s) : launch_read<false>(p, D, s));
}

int64_t dg_fp8_paged_attention_workspace_bytes(int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads,
                                               int64_t head_dim, int64_t max_q_len)
{
    const int st = check_attend_sizes(T, B, q_heads, kv_heads, head_dim, max_q_len);
    if (st != DG_OK)
        return -st;
    return T == 0 || B == 0 ? 0 : plan_attend(T, B, kv_heads, q_heads / kv_heads, head_dim, max_q_len).most_bytes;
}

dg_status dg_fp8_paged_attention(const void *Q, int64_t q_stride_t, int64_t q_stride_h, int64_t q_heads,
                                 const dg_fp8_cache *k_cache, const dg_fp8_cache *v_cache, const int32_t *block_table,
                                 int64_t table_stride, int64_t table_width, const int32_t *kv_lens,
                                 const int32_t *q_starts, int64_t B, int64_t T, int64_t max_q_len, float scale,
                                 int64_t window, void *out, int64_t out_stride_t, int64_t out_stride_h,
                                 void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!k_cache || !v_cache)
        return DG_ERR_NULL_POINTER;
    const dg_fp8_cache &kc = *k_cache, &vc = *v_cache;
    int st;
    if ((st = check_cache_sizes(kc)) != DG_OK || (st = check_cache_sizes(vc)) != DG_OK)
        return (dg_status)st;
    const int64_t D = kc.head_dim, heads = kc.heads;
    if (vc.pages != kc.pages || vc.page_size != kc.page_size || vc.heads != heads || vc.head_dim != D ||
        table_width < 0 || window < 0 || !(fabsf(scale) < INFINITY))
        return DG_ERR_BAD_SHAPE;
    if ((st = check_attend_sizes(T, B, q_heads, heads, D, max_q_len)) != DG_OK)
        return (dg_status)st;
    if (table_width > kMaxContext / kc.page_size)
        return DG_ERR_UNSUPPORTED;
    if (T == 0 || B == 0)
        return DG_OK;
    const int64_t units = (table_width * kc.page_size + dga::kUnit - 1 + 31) / dga::kUnit;
    if (B * heads * (units + 1) > kInt32Max)
        return DG_ERR_UNSUPPORTED;
    if (!Q || !out || !kv_lens || !q_starts || (!block_table && table_width))
        return DG_ERR_NULL_POINTER;
    if ((st = check_cache(kc, false)) != DG_OK || (st = check_cache(vc, false)) != DG_OK ||
        (st = check_rows(q_stride_t, q_stride_h, T, q_heads, 2)) != DG_OK ||
        (st = check_rows(out_stride_t, out_stride_h, T, q_heads, 2)) != DG_OK)
        return (dg_status)st;
    if ((B > 1 && table_stride < table_width) || !rows_apart({{T, out_stride_t}, {q_heads, out_stride_h}}, D))
        return DG_ERR_BAD_STRIDE;
    if (!strides_fit({table_stride}))
        return DG_ERR_UNSUPPORTED;
    if (!aligned(Q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(kv_lens, 4) ||
        !aligned(q_starts, 4) || !aligned(workspace, 16))
        return DG_ERR_MISALIGNED;
    const AttendPlan a = plan_attend(T, B, heads, q_heads / heads, D, max_q_len);
    if (workspace_bytes < a.bytes)
        return DG_ERR_SCRATCH;
    if (a.bytes && !workspace)
        return DG_ERR_NULL_POINTER;
    const Extent none = {0, 0};
    const Extent ins[8] = {rows_extent(Q, 2, T, q_stride_t, q_heads, q_stride_h, D), codes_extent(kc), codes_extent(vc),
                           scales_extent(kc), scales_extent(vc), extent(kv_lens, 4, B - 1), extent(q_starts, 4, B),
                           table_width ? extent(block_table, 4, (B - 1) * table_stride + table_width - 1) : none};
    const Extent eo = rows_extent(out, 2, T, out_stride_t, q_heads, out_stride_h, D);
    const Extent ews = workspace_bytes > 0 && workspace ? extent(workspace, 1, workspace_bytes - 1) : none;
    if (overlaps(eo, ews))
        return DG_ERR_ALIASING;
    for (const Extent &e : ins)
        if (overlaps(eo, e) || overlaps(ews, e))
            return DG_ERR_ALIASING;
    DeviceInfo dev;
    if ((st = current_device(dev)) != DG_OK)
        return (dg_status)st;
    dga::AttendParams p = {};
    p.Q = (const uint16_t *)Q; p.q_t = q_stride_t; p.q_h = q_stride_h;
    p.out = (uint16_t *)out; p.o_t = out_stride_t; p.o_h = out_stride_h;
    p.k = rows_of(kc); p.v = rows_of(vc);
    p.table = block_table; p.table_stride = table_stride;
    p.width = (int)table_width; p.pages = (int)kc.pages;
    p.page = dgc::divisor((uint32_t)kc.page_size);
    p.kv_lens = kv_lens; p.q_starts = q_starts;
    p.B = (int)B; p.T = (int)T; p.heads = (int)heads;
    p.max_q_len = (int)std::min(max_q_len, T);
    p.window = window > kMaxContext ? 0 : (int)window;
    p.group = dgc::divisor((uint32_t)(q_heads / heads));
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.few.o = (float *)workspace;
    const hipStream_t s = (hipStream_t)stream;
    return (dg_status)(D == 64 ? launch_attend<64>(p, a, units, s) : launch_attend<128>(p, a, units, s));
}

}  // extern "C"
