// attend.hpp -- gfx950 kernels of attention over a paged cache of e4m3 codes.
//
// A sequence's new tokens i = 0 .. m - 1 are the last m of its n tokens. Token
// i, at position pos = n - m + i, sees the keys j <= pos (and j > pos - window):
//   x_ij = scale sK_j (q_i . K_j)          o_i = sum_j p_ij sV_j V_j / sum_j p_ij,   p_ij = exp(x_ij)
// with codes K_j, V_j and one fp32 scale for each key and head. The query heads
// of a group share a key head: their rows (token i, head of the group) stand
// side by side as columns of the same products, so the cache is read once for
// all of them.
//
// Roundings. The codes are exact in bf16 and fp16, so the products q . K are
// exact bf16 products summed in fp32; both scales are applied in fp32. The
// second product takes the weights w_j = p_j sV_j in fp16 (11 bits, off by 2^-11;
// bf16's 8 would add as much error as the output's own rounding) and the codes.
// The denominator's exponentials, all sums, the references and the outputs
// before their rounding are fp32.
// fp16's range is kept by one reference for each row: p is exp2(x - m), and m
// follows the row's largest weight, not its largest p: the largest |w| was 2^7
// when m was set, and m moves when one passes 2^15, so that rows rarely move
// their sums. So what a row does not see, or sees with next to no weight, has no
// say in how its other weights are rounded, whatever its scale. Weights below
// fp16's normal numbers are off by 2^-25, 2^-32 of the row's largest. p takes up
// fp32's exponents for this: with the row's largest weight on a key of scale s
// it lies about 2^19 / s (sV goes into weights in units of 2^12). It is kept below
// 2^115, so weights are rounded as beside one of the largest p and a scale of
// 2^-96 where that is more than the row's largest; scales below 2^-114 count as 0;
// and what lies below 2^-145 s of that key's p drops out (2^-26 at the largest
// scale that bf16 values have).
//
// Masked keys never count, whatever their rows hold: their p is set to 0, scales
// that are not finite and codes of V that are NaN there are replaced (0 * NaN
// would be NaN). A row that sees a NaN code comes out as NaN: in that column, or
// in all of them where the code lies in a tile that is masked for some rows; a
// row that sees a scale that is not finite, in all of them. A row of zeros has
// the scale 1, which says nothing about values beside it: it counts as 2^-114.
//
// Which kernel. The cache's bytes bound few rows: each key is read once, at
// 2 D + 8 bytes, and costs 4 D operations a row, so up to some 60 rows the read
// takes longer. The few-rows kernel takes up to 32 (33 rows of 64 sequences, in
// a form of it with four tiles of 16: 1087 us, its registers spilled; 397 us
// here in the other). Both split keys over workgroups by the lengths on the
// device, and one launch behind them joins what was split.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "cache.hpp"

namespace dga {

using dgc::Divisor;
using dgc::quotient;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kUnit = 128;               // keys that a workgroup of the few-rows kernel takes at once
constexpr int kFewRows = 32;             // most rows (tokens x heads of a group) of its sequences
constexpr int kTileRows = 256;           // rows of a workgroup of the many-rows kernel
constexpr int kJoinRows = 4;             // of a cut tile, that a workgroup joins at a time
constexpr int kJoinGroups = 1024;        // workgroups that do
constexpr int kTileKeys = 64;            // keys that a workgroup of the many-rows kernel takes at once
constexpr float kNoMax = -1e30f;         // reference of a row that has seen nothing; finite, so that differences are
constexpr float kTopWeight = 7.0f;       // log2 of a row's largest weight when its reference is set
constexpr float kMostWeight = 0x1p15f;   // how far a weight may go before the reference moves (fp16 ends at 65504)
constexpr float kUnset = -1.0f;          // limit of a row whose reference has not been set
constexpr float kMostSum = 0x1p120f;     // how far a lane's exponentials of a tile may go
constexpr float kTopExponential = 115.0f;  // log2 of a row's largest when its reference is set, at most
constexpr float kScaleUnit = 0x1p-12f;   // of values' scales in weights
constexpr float kLeastScale = 0x1p-114f; // of values; what lies below counts as 0
constexpr float kSumUnit = 0x1p-20f;     // in which exponentials are summed: 2^26 times 2^120 stays in fp32's range
constexpr float kOutUnit = kSumUnit / kScaleUnit;      // of sums of weights over those of exponentials

// One of the two caches: rows of 16-byte multiples, addressed in units of 16 bytes.
struct Rows {
    const uint8_t *codes;
    uint32_t page16, token16;
    int64_t head;
    const float *scales;
    int64_t s_page, s_token, s_head;
};

// Where pieces leave their partial results.
struct Parts {
    int rows;                            // of a piece
    float *o;                            // [piece][rows][D], sums over p sV V, sV in kScaleUnit
    float *ml;                           // [piece][rows][2], reference and sum of p in kSumUnit
};

struct AttendParams {
    const uint16_t *Q;                   // bf16 [T, heads * group, D]
    int64_t q_t, q_h;
    uint16_t *out;                       // bf16 [T, heads * group, D]
    int64_t o_t, o_h;
    Rows k, v;
    const int32_t *table;                // [B, width]
    int64_t table_stride;
    int width, pages;
    Divisor page;                        // tokens of a page
    const int32_t *kv_lens, *q_starts;
    int B, T, heads, max_q_len, window;
    Divisor group;                       // query heads of a key head
    float scale_log2;                    // scale / ln 2
    int few_rows;                        // sequences of up to so many rows are the few-rows kernel's
    int target;                          // few rows: workgroups aimed at
    int most_pieces;                     // many rows: workgroups up to which tiles may be cut
    Parts few, many;                     // partial results of the two kernels
    int few_joined;                      // workgroups of the joining launch that join the first kernel's,
    int row_a_wave;                      // and whether each of their waves joins a row
};

// A sequence as the device arrays give it; anything out of range counts as nothing.
struct Sequence {
    int start, m, n, low;                // first row of Q, new tokens, tokens, first key that any of them sees
    int rows;                            // 0: none, or more tokens than max_q_len
};

__device__ __forceinline__ Sequence sequence(const AttendParams &p, int b)
{
    Sequence s;
    s.start = min(max(p.q_starts[b], 0), p.T);
    const int end = min(max(p.q_starts[b + 1], s.start), p.T);
    s.m = end - s.start;
    s.n = (int)min((int64_t)max(p.kv_lens[b], 0), (int64_t)p.width * p.page.d);
    s.low = p.window ? max(0, s.n - s.m + 1 - p.window) : 0;
    s.rows = s.m <= p.max_q_len ? s.m * (int)p.group.d : 0;
    return s;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int shifted(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}

// Inclusive sums over the 64 lanes: shifts within rows of 16, then the rows' totals onwards.
__device__ __forceinline__ int scan(int v)
{
    v += shifted<0x111, 0xF>(v);
    v += shifted<0x112, 0xF>(v);
    v += shifted<0x114, 0xF>(v);
    v += shifted<0x118, 0xF>(v);
    v += shifted<0x142, 0xA>(v);
    return v + shifted<0x143, 0xC>(v);
}

__device__ __forceinline__ int lane_int(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Orders a wave's LDS accesses for the compiler; the hardware runs them in order.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float max_across(float v)  // over the lanes l, l ^ 16, l ^ 32, l ^ 48
{
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}

__device__ __forceinline__ float sum_across(float v)
{
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// Two codes (the low or high half of a dword) as packed bf16 or fp16, exactly.
template <bool HIGH>
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t codes)
{
    return __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, HIGH));
}

template <bool HIGH>
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t codes)
{
    return __builtin_bit_cast(uint32_t, (f16x2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, HIGH));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ bool has_nan_code(uint32_t codes)  // 0x7f or 0xff among four
{
    return (((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}

// The codes with NaNs replaced by zeros.
__device__ __forceinline__ uint32_t without_nan_codes(uint32_t codes)
{
    const uint32_t nan = (((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    return codes & ~(nan * 0xffu);
}

// The value that lane I of a lane's 16 has: an operand of the instruction that takes it.
template <int I>
__device__ __forceinline__ float from_lane(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + I, 0xF, 0xF, true));
}

// f(0), f(1), .. f(N - 1), with the numbers as types.
template <typename F, int... I>
__device__ __forceinline__ void for_each(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}

// Whether a scale of values can go into weights as it is.
__device__ __forceinline__ bool usable(float scale)
{
    return fabsf(scale) >= kLeastScale && fabsf(scale) < __builtin_inff();
}

// Bits of the 32 keys whose codes are all zeros; a lane holds some elements of the keys 16 (i / 4) + 4 (lane / 16) + i % 4.
template <int VW>
__device__ __forceinline__ uint32_t rows_of_zeros(const uint32_t (&codes)[8][VW])
{
    uint32_t zeros = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t some = 0;
#pragma unroll
        for (int l = 0; l < VW; ++l)
            some |= codes[i][l] & 0x7f7f7f7fu;
        const uint64_t lanes = __ballot(some != 0);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            zeros |= (uint32_t)((lanes >> (16 * g) & 0xffff) == 0) << (16 * (i / 4) + 4 * g + i % 4);
    }
    return zeros;
}

// A row's move to a reference at which its largest weight is 2^kTopWeight, or its largest exponential as large as it may
// be: by how much (exactly, as x is moved too).
__device__ __forceinline__ float move_reference(float &ref, float top_weight, float top_exponential)
{
    const float next = ref + fmaxf(top_weight - kTopWeight, top_exponential - kTopExponential), by = next - ref;
    ref = next;
    return by;
}

// exp2(2 half) v, for exponentials whose sum lies far from 1: the factor alone could leave fp32's range.
__device__ __forceinline__ float scaled(float v, float half)
{
    const float f = __builtin_amdgcn_exp2f(half);
    return v * f * f;
}

// ---------------------------------------------------------------- few rows

// Where a piece of the few-rows kernel lies: its units of a sequence's keys, for one head.
struct Piece {
    Sequence s;
    int b, head, first, units;           // units [first, first + units) of the sequence's
    int pieces, index;                   // pieces of each of its heads; this one's number among the launch's
};

// Units of kUnit keys that a sequence's rows read, counted from the 32 keys that hold the first one.
__device__ __forceinline__ int units_of(const Sequence &s)
{
    return max(0, (s.n - (s.low & ~31) + kUnit - 1) / kUnit);
}

// The launch's keys are cut into pieces of about the same size, so that uneven
// sequences fill the CUs evenly: `chunk` units a piece, as many as give
// p.target pieces in all. Each wave finds its piece by itself from the
// sequences' lengths (64 at a time, a scan over the lanes), without a planning
// launch and without the host knowing them. Workgroups that follow each other go
// to the XCDs in turn, so pieces are numbered such that the heads of a page, whose
// rows lie next to each other, are read by one XCD.
struct Cut {
    Sequence s;                          // of this lane, of 64
    int units, pieces, before;           // pieces of each of its heads; pieces of the lanes (and sequences) before
};

__device__ __forceinline__ int lane_units(const AttendParams &p, int b, Sequence &s)
{
    s.rows = 0;
    if (b < p.B)
        s = sequence(p, b);
    return s.rows > 0 && s.rows <= p.few_rows ? units_of(s) : -1;
}

// Units of a piece. c: the first 64 sequences' cut is begun.
__device__ __forceinline__ int chunk_of(const AttendParams &p, Cut &c)
{
    const int lane = threadIdx.x & 63;
    c.units = lane_units(p, lane, c.s);
    int all = max(0, c.units);
    for (int b0 = 64; b0 < p.B; b0 += 64) {
        Sequence s;
        all += max(0, lane_units(p, b0 + lane, s));
    }
    all = lane_int(scan(all), 63) * p.heads;
    return max(1, (all + p.target - 1) / p.target);
}

// Cuts the sequences from b0 on; returns the pieces up to and with them.
__device__ __forceinline__ int cut(const AttendParams &p, int b0, int chunk, int before, Cut &c)
{
    if (b0)
        c.units = lane_units(p, b0 + (threadIdx.x & 63), c.s);
    c.pieces = c.units < 0 ? 0 : max(1, (c.units + chunk - 1) / chunk);
    const int upto = scan(c.pieces * p.heads);
    c.before = before + upto - c.pieces * p.heads;
    return before + lane_int(upto, 63);
}

__device__ __forceinline__ bool find_piece(const AttendParams &p, int block, Piece &w)
{
    Cut c;
    const int chunk = chunk_of(p, c);
    int total = cut(p, 0, chunk, 0, c);
    for (int b0 = 64; b0 < p.B; b0 += 64)
        total = cut(p, b0, chunk, total, c);
    // Workgroups are dealt to the 8 XCDs in turn. Renumbered, each XCD takes a contiguous range of pieces, so that the
    // heads of a page, whose rows lie side by side, are read by the same one at the same time (64 sequences up to 16384
    // tokens: 259 -> 232 us).
    const int xcd = block % 8, per = total / 8, extra = total % 8, turn = block / 8;
    if (turn >= per + (xcd < extra))
        return false;
    const int index = xcd * per + min(xcd, extra) + turn;
    int b0 = 0;
    if (p.B > 64) {
        c.units = lane_units(p, threadIdx.x & 63, c.s);
        for (int upto = cut(p, 0, chunk, 0, c); upto <= index; ) {
            b0 += 64;
            upto = cut(p, b0, chunk, upto, c);
        }
    }
    const int lane = __builtin_ctzll(__ballot(index >= c.before && index < c.before + c.pieces * p.heads));
    w.b = b0 + lane;
    w.s.start = lane_int(c.s.start, lane);
    w.s.m = lane_int(c.s.m, lane);
    w.s.n = lane_int(c.s.n, lane);
    w.s.low = lane_int(c.s.low, lane);
    w.s.rows = lane_int(c.s.rows, lane);
    w.pieces = lane_int(c.pieces, lane);
    w.index = index;
    const int at = index - lane_int(c.before, lane), all = lane_int(c.units, lane);
    // Heads next to each other: they read the same pages.
    const int i = at / p.heads;
    w.head = at - i * p.heads;
    w.first = (int)((int64_t)all * i / w.pieces);
    w.units = (int)((int64_t)all * (i + 1) / w.pieces) - w.first;
    return true;
}

// Writes D / 16 values of a finished row.
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t *to, const float *v)
{
    if (N == 8)
        *(u32x4 *)to = u32x4{dgn::pack_bf16(v[0], v[1]), dgn::pack_bf16(v[2], v[3]), dgn::pack_bf16(v[N - 4], v[N - 3]),
                             dgn::pack_bf16(v[N - 2], v[N - 1])};
    else
        *(u32x2 *)to = u32x2{dgn::pack_bf16(v[0], v[1]), dgn::pack_bf16(v[2], v[3])};
}

// One piece: up to 16 NT rows of one key head over some units of its keys.
//
// Bound by the bytes of the cache. Each wave streams 32 of a unit's 128 keys
// from HBM straight into the operands' registers, the next unit's loads in
// flight while it computes one; nothing goes through LDS but addresses and
// scales. The products are transposed, so that each lane keeps one row's
// statistics and the first product's output is the second one's operand as it
// stands: S^T = K Q^T (16x16x32 bf16: lane l holds key l % 16 of K and 32 of
// its codes, and receives row l % 16, keys 4 (l / 16) + i), O^T = V^T P^T (the
// order of keys within an operand is free, as long as both have the same: lane
// group g takes the keys 4 g + i and 16 + 4 g + i; column c of V^T's tile t
// stands for element (D / 16) c + t, so that a lane reads consecutive codes).
// K's loads cover whole 128-byte lines, 8 lanes a row, and lanes l and l ^ 8
// then exchange halves. V's pairs of keys are brought together byte by byte
// (v_perm) before the conversion, which takes two codes at once.
//
// Two units are in flight, in registers of their own (one: 260 us for 64
// sequences of up to 16384 tokens, 8 key heads of 8; two: 226 us, 5.1 TB/s of
// 6.6 to 7.2 that kernels which only load reach here; 512 sequences of 4096 tokens
// 5.8 TB/s). What it reads from HBM is what it needs, 1.17 GB; matrix units and
// VALU are busy for 7% and 37% of the time. 198 registers for one tile of rows,
// two waves a SIMD; with two tiles 250, where the queries' would spill: they stay
// in LDS, the same for all waves (16 sequences of 4 tokens up to 8192: 56 -> 54 us
// with the joining launch, 62% of a copy's rate without it: a workgroup has four
// units or so, and the first and the last are not hidden). The look for rows of
// zeros costs a cache whose scales are all 1 a few percent (222 -> 229 us).
template <int D, int NT>
__global__ __launch_bounds__(kThreads, 2) void attend_few_kernel(AttendParams p)
{
    constexpr int DT = D / 16;           // codes of a key in a lane of V, and tiles of O^T
    constexpr int KS = D / 32;           // matrix instructions of a tile of S^T
    constexpr int KL = D / 64;           // 16-byte loads of K in a lane, for 16 keys
    constexpr int VW = D / 64;           // dwords of V in a lane, for one key
    constexpr int kPad = D + 4;
    __shared__ uint32_t offsets[4][64];  // of a wave's 32 keys in K, then in V
    __shared__ __align__(16) float scales[4][64];
    __shared__ float refs[4][2][16 * NT];
    __shared__ __align__(16) float sums[4][16][kPad];
    // Queries of two tiles.
    __shared__ __align__(16) u32x4 queries[NT > 1 ? NT * KS : 1][64];

    Piece w;
    if (!find_piece(p, blockIdx.x, w))
        return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int key0 = (w.s.low & ~31) + w.first * kUnit + 32 * wave;    // this wave's first key
    const int units = w.units;
    const int32_t *table = p.table + w.b * p.table_stride;
    const uint8_t *kbase = p.k.codes + w.head * p.k.head, *vbase = p.v.codes + w.head * p.v.head;
    const bool values = lane >= 32;      // lanes 0..31 look after K's rows, 32..63 after V's
    const float *sbase = values ? p.v.scales + w.head * p.v.s_head : p.k.scales + w.head * p.k.s_head;

    bf16x8 q[NT][KS];
    int pos[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = 16 * nt + c;
        const int token = (int)quotient(r, p.group), h = r - token * (int)p.group.d;
        const bool present = r < w.s.rows;
        pos[nt] = present ? w.s.n - w.s.m + token : -1;
        const uint16_t *row = p.Q + (int64_t)(w.s.start + token) * p.q_t + (int64_t)(w.head * (int)p.group.d + h) * p.q_h;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
            u32x4 v = {0, 0, 0, 0};
            if (present)
                v = *(const u32x4 *)(row + (D / 4) * g + 8 * t);
            q[nt][t] = __builtin_bit_cast(bf16x8, v);
            if (NT > 1 && wave == t % 4)
                queries[NT > 1 ? nt * KS + t : 0][lane] = v;
        }
    }
    if (NT > 1)
        __syncthreads();

    const auto query = [&](int nt, int t) {
        return NT > 1 ? __builtin_bit_cast(bf16x8, (u32x4)queries[NT > 1 ? nt * KS + t : 0][lane]) : q[nt][t];
    };

    // What a unit brings: its codes, the scale of this lane's key, which keys are there, and the page of this lane's key
    // in the unit after the next.
    struct Raw {
        u32x4 k[2][KL];
        uint32_t v[8][VW];
        float scale;
        uint32_t there;
        int page;
    } even, odd;
    // Without a branch around it, so that nothing waits for it before its use; units are at most the sequence's.
    const auto load_page = [&](int u) {
        return table[quotient(min(key0 + u * kUnit + (lane & 31), w.s.n - 1), p.page)];
    };
    const auto load = [&](int u, Raw &raw) {
        const int j = key0 + u * kUnit + (lane & 31);
        const bool valid = u < units && j >= w.s.low && j < w.s.n && raw.page >= 0 && raw.page < p.pages;
        // A key that is not there reads slot 0, and is masked later.
        const uint32_t pg = valid ? raw.page : 0, token = valid ? j - quotient(j, p.page) * p.page.d : 0;
        raw.there = (uint32_t)__ballot(valid);
        raw.page = load_page(u + 2);
        offsets[wave][lane] = values ? pg * p.v.page16 + token * p.v.token16 : pg * p.k.page16 + token * p.k.token16;
        raw.scale = values ? sbase[pg * p.v.s_page + token * p.v.s_token] : sbase[pg * p.k.s_page + token * p.k.s_token];
        wave_sync();
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            if (D == 128) {
#pragma unroll
                for (int l = 0; l < KL; ++l)
                    raw.k[sub][l] = __builtin_nontemporal_load(
                        (const u32x4 *)(kbase + 16 * (int64_t)offsets[wave][16 * sub + 8 * l + (lane & 7)] + 32 * g +
                                        16 * ((lane >> 3) & 1)));
            } else {
                raw.k[sub][0] = __builtin_nontemporal_load(
                    (const u32x4 *)(kbase + 16 * (int64_t)offsets[wave][16 * sub + c] + 16 * g));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *at = vbase + 16 * (int64_t)offsets[wave][32 + 16 * sub + 4 * g + i] + DT * c;
                if (VW == 2) {
                    const u32x2 v = __builtin_nontemporal_load((const u32x2 *)at);
                    raw.v[4 * sub + i][0] = v[0];
                    raw.v[4 * sub + i][VW - 1] = v[1];
                } else {
                    raw.v[4 * sub + i][0] = __builtin_nontemporal_load((const uint32_t *)at);
                }
            }
        }
        wave_sync();
    };

    f32x4 o[NT][DT];
    float ref[NT], limit[NT], sum[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        ref[nt] = sum[nt] = 0.0f;
        limit[nt] = pos[nt] >= 0 ? kUnset : kMostWeight;
#pragma unroll
        for (int t = 0; t < DT; ++t)
            o[nt][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const auto attend = [&](int u, Raw &raw) {
        const uint32_t there = raw.there;
        const float found = raw.scale;
        const int first = key0 + u * kUnit;
        // Scales that cannot be weighed with are replaced; their keys are looked at below.
        const bool mine = values && (there >> (lane & 31) & 1);
        const bool masked = there != 0xffffffffu || first + 31 > w.s.n - w.s.m ||
                            (p.window && first <= w.s.n - 1 - p.window) || __ballot(mine && !usable(found)) != 0;
        scales[wave][lane] = !values ? found * p.scale_log2 : (usable(found) ? found : kLeastScale) * kScaleUnit;
        wave_sync();
        float ks[8], vs[8];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            const f32x4 a = *(const f32x4 *)&scales[wave][16 * sub + 4 * g];
            const f32x4 b = *(const f32x4 *)&scales[wave][32 + 16 * sub + 4 * g];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ks[4 * sub + i] = a[i];
                vs[4 * sub + i] = b[i];
            }
        }
        wave_sync();
        if (__ballot(mine && found == 1.0f)) {
            const uint32_t zeros = rows_of_zeros(raw.v) >> (4 * g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                vs[i] = (zeros >> (16 * (i / 4) + i % 4) & 1) && vs[i] == kScaleUnit ? kLeastScale * kScaleUnit : vs[i];
        }

        // This lane's keys whose values are not finite: codes are replaced by zeros, and a row that sees one becomes NaN.
        uint32_t bad = 0;
        if (masked) {
            const uint32_t infinite = (uint32_t)(__ballot(mine && !(fabsf(found) < __builtin_inff())) >> 32) >> (4 * g);
            const uint32_t none = (uint32_t)(__ballot(mine && fabsf(found) < kLeastScale) >> 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = 16 * (i / 4) + i % 4;
                const bool here = (there & ~none) >> (4 * g) >> at & 1;
                bool nan = false;
#pragma unroll
                for (int l = 0; l < VW; ++l) {
                    nan |= has_nan_code(raw.v[i][l]);
                    raw.v[i][l] = here ? without_nan_codes(raw.v[i][l]) : 0;
                }
                if ((infinite >> at & 1) || (__ballot(nan) >> (16 * g) & 0xffff) != 0)
                    bad |= 1u << i;
            }
        }

        // S^T, 2 x 16 keys.
        f32x4 s[NT][2];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            uint32_t row[8];
            if (D == 128) {
                // From load order to operand order: lanes 8..15 of each 16 take the first from lane ^ 8's second.
                const bool upper = lane & 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = raw.k[sub][0][i], b = raw.k[sub][KL - 1][i];
                    const uint32_t give = upper ? a : b;
                    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xF, 0xF, false);
                    row[i] = upper ? got : a;
                    row[4 + i] = upper ? b : got;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    row[i] = raw.k[sub][0][i];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                s[nt][sub] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                const u32x4 a = {codes_to_bf16<false>(row[2 * t]), codes_to_bf16<true>(row[2 * t]),
                                 codes_to_bf16<false>(row[2 * t + 1]), codes_to_bf16<true>(row[2 * t + 1])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[nt][sub] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), query(nt, t),
                                                                         s[nt][sub], 0, 0, 0);
            }
        }

        // Weights.
        f16x8 weights[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __builtin_fmaf(s[nt][i / 4][i % 4], ks[i], -ref[nt]);
            if (masked) {
                // From this lane's first key on: keys [from, to] are seen, where they are there.
                const int to = pos[nt] - first - 4 * g, from = p.window ? to - p.window + 1 : -kUnit;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 16 * (i / 4) + i % 4;
                    const bool sees = (there >> (4 * g) >> at & 1) && at <= to && at >= from;
                    x[i] = sees ? x[i] : -__builtin_inff();
                    if (sees && (bad >> i & 1))
                        sum[nt] = __builtin_nanf("");
                }
            }
            float most, part;
            const auto weigh = [&]() {
                most = part = 0.0f;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float e = __builtin_amdgcn_exp2f(x[i]);
                    part += e;
                    y[i] = e * vs[i];
                    most = fmaxf(most, fabsf(y[i]));
                }
                const u32x4 packed = {pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]), pack_f16(y[6], y[7])};
                weights[nt] = __builtin_bit_cast(f16x8, packed);
            };
            weigh();
            if (__ballot(most > limit[nt] || part > kMostSum)) {
                float top = -__builtin_inff(), top_x = top;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    top = fmaxf(top, x[i] + __builtin_amdgcn_logf(fabsf(vs[i])));
                    top_x = fmaxf(top_x, x[i]);
                }
                top = max_across(top);
                top_x = max_across(top_x);
                const float over = most > limit[nt] || part > kMostSum ? 1.0f : 0.0f;
                const bool moves = max_across(over) > 0.0f && top > -__builtin_inff();
                const float by = moves ? move_reference(ref[nt], top, top_x) : 0.0f;
                const float half = limit[nt] == kUnset ? 0.0f : -0.5f * by;
                const float shrink = scaled(1.0f, half);
                sum[nt] = scaled(sum[nt], half);
#pragma unroll
                for (int t = 0; t < DT; ++t)
                    o[nt][t] *= shrink;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] -= by;
                limit[nt] = moves ? kMostWeight : limit[nt];
                weigh();
            }
            sum[nt] = __builtin_fmaf(part, kSumUnit, sum[nt]);
        }

        // O^T += V^T P^T
#pragma unroll
        for (int l = 0; l < VW; ++l) {
            uint32_t low[4], high[4];    // elements 0, 1 and 2, 3 of the dword, each for two keys
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                low[i] = __builtin_amdgcn_perm(raw.v[2 * i + 1][l], raw.v[2 * i][l], 0x05010400);
                high[i] = __builtin_amdgcn_perm(raw.v[2 * i + 1][l], raw.v[2 * i][l], 0x07030602);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                u32x4 a;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t both = d < 2 ? low[i] : high[i];
                    a[i] = d % 2 ? codes_to_f16<true>(both) : codes_to_f16<false>(both);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    o[nt][4 * l + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), weights[nt],
                                                                              o[nt][4 * l + d], 0, 0, 0);
            }
        }
    };

    // Each wave loads two units ahead: while it computes one, the next is on its way. The queries are there before the
    // loop, or its first use of them would wait for every load in each round.
    if (units > 0) {
        even.page = load_page(0);
        odd.page = load_page(1);
        load(0, even);
        load(1, odd);
        if (NT == 1) {
#pragma unroll
            for (int t = 0; t < KS; ++t)
                asm volatile("" : "+v"(q[0][t]));
        }
        // (No way out in the middle: where two ways join, loads are waited for as on the shorter one.)
        for (int u = 0; u + 1 < units; u += 2) {
            attend(u, even);
            load(u + 2, even);
            attend(u + 1, odd);
            load(u + 3, odd);
        }
        if (units & 1)
            attend(units - 1, even);
    }

    // The four waves' sums, over their largest reference.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float all = sum_across(sum[nt]);
        ref[nt] = limit[nt] == kUnset ? kNoMax : ref[nt];
        if (g == 0) {
            refs[wave][0][16 * nt + c] = ref[nt];
            refs[wave][1][16 * nt + c] = all;
        }
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (16 * nt >= w.s.rows)
            break;
        float top = kNoMax;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = fmaxf(top, refs[i][0][16 * nt + c]);
        const float factor = __builtin_amdgcn_exp2f(ref[nt] - top);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < DT; t += 4)
                *(f32x4 *)&sums[wave][c][(4 * g + i) * DT + t] =
                    f32x4{o[nt][t][i], o[nt][t + 1][i], o[nt][t + 2][i], o[nt][t + 3][i]} * factor;
        __syncthreads();
        const int row = threadIdx.x >> 4, r = 16 * nt + row, col = DT * (threadIdx.x & 15);
        if (r < w.s.rows) {
            float most = kNoMax, total = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                most = fmaxf(most, refs[i][0][r]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                total += scaled(refs[i][1][r], 0.5f * (refs[i][0][r] - most));
            float y[DT];
#pragma unroll
            for (int t = 0; t < DT; ++t)
                y[t] = (sums[0][row][col + t] + sums[1][row][col + t]) + (sums[2][row][col + t] + sums[3][row][col + t]);
            if (w.pieces == 1) {
                const int token = (int)quotient(r, p.group), h = r - token * (int)p.group.d;
#pragma unroll
                for (int t = 0; t < DT; ++t)
                    y[t] = total == 0.0f ? 0.0f : y[t] * kOutUnit / total;
                store_bf16<DT>(p.out + (int64_t)(w.s.start + token) * p.o_t +
                                   (int64_t)(w.head * (int)p.group.d + h) * p.o_h + col, y);
            } else {
                const int64_t at = (int64_t)w.index * p.few.rows + r;
#pragma unroll
                for (int t = 0; t < DT; t += 4)
                    *(f32x4 *)(p.few.o + at * D + col + t) = f32x4{y[t], y[t + 1], y[t + 2], y[t + 3]};
                if (col == 0)
                    *(f32x2 *)(p.few.ml + 2 * at) = f32x2{most, total};
            }
        }
        __syncthreads();
    }
}

// Joins this wave's share (every `waves`-th from `first` on) of `count` partial results of a row, the i-th at index(i).
template <int D, typename Index>
__device__ __forceinline__ void join_pieces(const Parts &parts, int count, int first, int waves, Index index, float &total,
                                            float (&y)[D / 64])
{
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    float top = kNoMax;
    for (int i = lane; i < count; i += 64)
        top = fmaxf(top, parts.ml[2 * index(i)]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d, 64));
    // (By the lanes: as two more products for each piece in the loop below it took twice as long, 66 pieces of 256 rows
    // 19.7 us instead of 8.6.)
    total = 0.0f;
    for (int i = lane; i < count; i += 64)
        if (i % waves == first) {
            const f32x2 ml = *(const f32x2 *)(parts.ml + 2 * index(i));
            total += scaled(ml[1], 0.5f * (ml[0] - top));
        }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        total += __shfl_xor(total, d, 64);
#pragma unroll
    for (int e = 0; e < E; ++e)
        y[e] = 0.0f;
#pragma unroll 8
    for (int i = first; i < count; i += waves) {
        const int64_t at = index(i);
        const float weight = __builtin_amdgcn_exp2f(parts.ml[2 * at] - top);
        const float *o = parts.o + at * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e)
            y[e] = __builtin_fmaf(o[e], weight, y[e]);
    }
}

// A joined row, E elements of it in each lane.
template <int E>
__device__ __forceinline__ void store_row(uint16_t *to, float total, const float (&y)[E])
{
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < E; ++e)
        v[e] = total == 0.0f ? 0.0f : y[e] * kOutUnit / total;
    to += E * (threadIdx.x & 63);
    if (E == 2)
        *(uint32_t *)to = dgn::pack_bf16(v[0], v[1]);
    else
        *to = (uint16_t)dgn::pack_bf16(v[0], 0.0f);
}

// One row of a sequence that several pieces share, by a wave; or by the four of a workgroup, for few rows.
template <int D>
__device__ __forceinline__ void join_few(const AttendParams &p, int block)
{
    constexpr int E = D / 64;
    __shared__ float part[4][D + 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = p.row_a_wave ? 4 * block + wave : block;
    const int of = row / p.few.rows, r = row - of * p.few.rows, b = of / p.heads, head = of - b * p.heads;
    if (b >= p.B)
        return;
    Cut c;
    const int chunk = chunk_of(p, c);
    int upto = 0;
    for (int b0 = 0; b0 <= b; b0 += 64)
        upto = cut(p, b0, chunk, upto, c);
    const int pieces = lane_int(c.pieces, b % 64), before = lane_int(c.before, b % 64);
    const int start = lane_int(c.s.start, b % 64), rows = lane_int(c.s.rows, b % 64);
    if (pieces < 2 || r >= rows)
        return;
    const int token = (int)quotient(r, p.group), h = r - token * (int)p.group.d;
    uint16_t *to = p.out + (int64_t)(start + token) * p.o_t + (int64_t)(head * (int)p.group.d + h) * p.o_h;
    const auto index = [&](int i) { return (int64_t)(before + i * p.heads + head) * p.few.rows + r; };
    float total, y[E];
    if (p.row_a_wave) {
        join_pieces<D>(p.few, pieces, 0, 1, index, total, y);
        store_row(to, total, y);
        return;
    }
    join_pieces<D>(p.few, pieces, wave, 4, index, total, y);
#pragma unroll
    for (int e = 0; e < E; ++e)
        part[wave][E * lane + e] = y[e];
    if (lane == 0)
        part[wave][D] = total;
    __syncthreads();
    if (wave)
        return;
#pragma unroll
    for (int e = 0; e < E; ++e)
        y[e] = (part[0][E * lane + e] + part[1][E * lane + e]) + (part[2][E * lane + e] + part[3][E * lane + e]);
    store_row(to, (part[0][D] + part[1][D]) + (part[2][D] + part[3][D]), y);
}

// ---------------------------------------------------------------- many rows

// A tile of rows of one key head, and the piece of its keys that a workgroup takes.
struct Tile {
    Sequence s;
    int b, first, head;                  // sequence, first row
    int pieces, piece, slot;             // pieces of its keys; this one's number; the place of its partial result
};

// How the tiles of 64 sequences are cut, this lane's one.
struct Cuts {
    Sequence s;
    int tiles, keys;                     // tiles of rows; tiles of keys that the longest of them reads
    int pieces;                          // of each tile's keys
};

__device__ __forceinline__ void lane_tiles(const AttendParams &p, int b, Cuts &c)
{
    c.s.rows = 0;
    if (b < p.B)
        c.s = sequence(p, b);
    c.tiles = c.s.rows > p.few_rows ? (c.s.rows + kTileRows - 1) / kTileRows : 0;
    c.keys = c.tiles ? max(1, (c.s.n - (c.s.low & ~(kTileKeys - 1)) + kTileKeys - 1) / kTileKeys) : 0;
}

constexpr float kPieceStart = 3.0f, kPieceJoin = 0.15f;    // in units of the time of a tile of keys

// Pieces of a tile of this lane's sequence, of about 1 / rate tiles of keys each.
__device__ __forceinline__ int pieces_of(const Cuts &c, float rate)
{
#pragma clang fp contract(off)           // the joining kernel has to come to the same numbers
    return max(1, (int)((float)c.keys * rate + 0.5f));
}

// How tiles are cut: the reciprocal of the tiles of keys of a piece, 0 for not at
// all. Every workgroup comes to the same estimate from the lengths, in units of
// the time that a workgroup takes for one tile of keys (2.1 us; 1.9 where no row
// moves its reference): pieces that fill the 256 CUs at most once take as long as
// the longest; one sequence's, equal ones, as many rounds as they fill; uneven
// ones their average and a part of the longest. Cutting costs the joining launch's
// work (2), and for each piece its partial result's way out and back. Measured,
// 8 heads of 8, uncut and cut: 16 sequences of 16 tokens up to 8192, 366 and 150
// us; chunks of 100 tokens over 30000 and 500 over 600 in one batch, 1330 and 221;
// 512 tokens of 32 heads over 32768, 990 and 323; a prompt of 300 by itself, 29.5
// and 29.8, is not worth a cut. A piece's start is more than kPieceStart says:
// 512 tokens of 64 heads over 4096 to 32768 keys, in two pieces each, take 51 us
// and 2.1 for each tile of a piece, 39 and 1.9 with keys that are all the same.
// (More candidates than powers of two gained up to 15% for some batches and lost
// as much for others.)
__device__ __forceinline__ float cut_tiles(const AttendParams &p, Cuts &first)
{
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63;
    float total = 0.0f;
    int most = 0, pieces = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64) {
        Cuts c;
        lane_tiles(p, b0 + lane, c);
        if (b0 == 0)
            first = c;
        total += (float)c.tiles * (float)c.keys;
        pieces += c.tiles;
        most = max(most, c.keys);
    }
    const float cost = 0.03f * (float)p.many.rows / kTileRows, heads = (float)p.heads;
    float best = 0.0f;
    if (p.B == 1) {
        const float tiles = (float)lane_int(pieces, 0) * heads, keys = (float)lane_int(most, 0);
        float least = (keys + kPieceStart) * __builtin_ceilf(tiles / 256.0f);
#pragma unroll
        for (int rounds = 1; rounds <= 3; ++rounds) {
            const float parts = fminf(__builtin_floorf(256.0f * (float)rounds / tiles), keys);
            const float time = (float)rounds * (keys / parts + kPieceStart) + 2.0f + kPieceJoin * parts + cost * tiles * parts;
            if (parts >= 2.0f && time < least) {
                least = time;
                best = parts / keys;
            }
        }
        return best;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        total += __shfl_xor(total, d, 64);
        most = max(most, __shfl_xor(most, d, 64));
    }
    total *= heads / 256.0f;
    pieces = lane_int(scan(pieces), 63) * p.heads;
    const auto estimate = [&](float longest) { return pieces <= 256 ? longest : fmaxf(longest, 1.1f * total + 0.3f * longest); };
    float least = estimate((float)most);
    for (int parts = 2; parts <= 16 && parts <= most && least > total + 2.0f; parts *= 2) {
        const float rate = (float)parts / (float)most;
        pieces = 0;
        for (int b0 = 0; b0 < p.B; b0 += 64) {
            Cuts c = first;
            if (b0)
                lane_tiles(p, b0 + lane, c);
            pieces += c.tiles * pieces_of(c, rate);
        }
        pieces = lane_int(scan(pieces), 63) * p.heads;
        const float time = estimate((float)most / (float)parts) + 2.0f + cost * (float)pieces;
        if (pieces > p.most_pieces || time >= least)
            break;
        least = time;
        best = rate;
    }
    return best;
}

// The block's piece: of a sequence, the last (longest) tiles first, heads next to each other.
__device__ __forceinline__ bool find_tile(const AttendParams &p, int block, Tile &w)
{
    Cuts c;
    float rate = 0.0f;
    // Tiles are cut into up to most_pieces pieces; behind them lie uncut ones, or nothing.
    if (block < p.most_pieces)
        rate = cut_tiles(p, c);
    else
        lane_tiles(p, threadIdx.x & 63, c);
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64) {
        if (b0)
            lane_tiles(p, b0 + (threadIdx.x & 63), c);
        c.pieces = pieces_of(c, rate);
        const int all = c.tiles * c.pieces * p.heads, upto = before + scan(all);
        const uint64_t mine = __ballot(block >= upto - all && block < upto);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            w.b = b0 + l;
            w.s.start = lane_int(c.s.start, l);
            w.s.m = lane_int(c.s.m, l);
            w.s.n = lane_int(c.s.n, l);
            w.s.low = 0;
            w.s.rows = lane_int(c.s.rows, l);
            w.pieces = lane_int(c.pieces, l);
            const int at = block - lane_int(upto - all, l), share = at / p.heads, tile = share / w.pieces;
            w.head = at - share * p.heads;
            w.piece = share - tile * w.pieces;
            w.first = (lane_int(c.tiles, l) - 1 - tile) * kTileRows;
            w.slot = block;
            return true;
        }
        before = lane_int(upto, 63);
    }
    return false;
}

// The index-th cut tile (of all key heads), with the place of its first piece's partial result.
__device__ __forceinline__ bool find_cut_tile(const AttendParams &p, float rate, const Cuts &first, int index, Tile &w)
{
    Cuts c = first;
    int tiles_before = 0, pieces_before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64) {
        if (b0)
            lane_tiles(p, b0 + (threadIdx.x & 63), c);
        c.pieces = pieces_of(c, rate);
        const int tiles = c.pieces > 1 ? c.tiles * p.heads : 0, all = c.tiles * c.pieces * p.heads;
        const int tiles_upto = tiles_before + scan(tiles), upto = pieces_before + scan(all);
        const uint64_t mine = __ballot(index >= tiles_upto - tiles && index < tiles_upto);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            w.s.start = lane_int(c.s.start, l);
            w.s.rows = lane_int(c.s.rows, l);
            w.pieces = lane_int(c.pieces, l);
            const int at = index - lane_int(tiles_upto - tiles, l), tile = at / p.heads;
            w.head = at - tile * p.heads;
            w.first = (lane_int(c.tiles, l) - 1 - tile) * kTileRows;
            w.slot = lane_int(upto - all, l) + tile * w.pieces * p.heads + w.head;
            return w.slot >= 0 && w.slot + (w.pieces - 1) * p.heads < p.most_pieces;
        }
        tiles_before = lane_int(tiles_upto, 63);
        pieces_before = lane_int(upto, 63);
    }
    return false;
}

// LDS rows: K by key, D bf16; V^T by element, 64 fp16 keys. The padding spreads the lanes of a read (consecutive rows,
// one 16-byte chunk) over all banks, and lets every place be one address and a constant. Element (D / 16) c + i of V
// has row 16 i + c, so that the lanes that write one i write consecutive rows.
template <int D>
constexpr int kRowBytes = 2 * D + 16;
constexpr int kColumnBytes = 2 * kTileKeys + 16;

constexpr int kComputeWaves = kTileRows / 32;
constexpr int kManyThreads = 64 * (kComputeWaves + 4);  // two waves bring in K, two bring in V
constexpr int kHalf = kTileKeys / 2;                    // keys of a tile that a wave brings in

// What the many-rows kernel's waves share: two buffers, one computed while the other is filled, with what goes for each
// half of a tile.
template <int D>
struct ManyLds {
    __align__(16) uint8_t k[2][kTileKeys * kRowBytes<D>];
    __align__(16) uint8_t v[2][D * kColumnBytes];
    __align__(16) float kscales[2][kTileKeys];
    float vscales[2][kTileKeys];
    struct {
        uint32_t present[2];             // bits of the keys that are there
        uint32_t bad[2];                 // bits of keys whose values are not finite, where they were looked at
    } __align__(16) about[2];
    __align__(16) uint32_t offsets[4][kHalf];            // of the rows that a wave loads next
};

// The keys of a workgroup.
struct Keys {
    int key0, tiles, low, last;          // first key of the first tile, tiles, first and last key that count
    int pos_first, pos_last;             // positions of the first and the last row
};

// Whether some row between two positions does not see every one of the kHalf keys from `first` on.
__device__ __forceinline__ bool masked(int first, uint32_t there, int pos_first, int pos_last, int window)
{
    return there != ~0u || first + kHalf - 1 > pos_first || (window && first <= pos_last - window);
}

// Pages, rows and scales of a half tile of one of the caches, a key a lane (twice).
struct Rider {
    const Rows &rows;
    const int32_t *table;
    const float *scales;
    const AttendParams &p;
    const Keys &k;
    int part, lane;

    __device__ __forceinline__ int first(int t) const { return k.key0 + t * kTileKeys + kHalf * part; }
    __device__ __forceinline__ int page(int t) const
    {
        return table[quotient(min(first(t) + (lane & 31), k.last), p.page)];
    }
    // Offset and scale of this lane's key, and which of the keys are there. What is not there reads slot 0, and is
    // masked.
    __device__ __forceinline__ uint32_t place(int t, int page, uint32_t &offset, float &scale) const
    {
        const int j = first(t) + (lane & 31);
        const bool valid = j >= k.low && j <= k.last && page >= 0 && page < p.pages;
        const uint32_t pg = valid ? page : 0, token = valid ? j - quotient(j, p.page) * p.page.d : 0;
        offset = pg * rows.page16 + token * rows.token16;
        scale = scales[pg * rows.s_page + token * rows.s_token];
        return (uint32_t)__ballot(valid);
    }
};

// The loop of a wave that brings in a cache: tile t + 1 is stored while the others compute tile t, and tile t + 3
// loaded, so that a tile's loads have more than a round to arrive.
template <typename Load, typename Store, typename Raw>
__device__ __forceinline__ void bring(int tiles, const Rider &rider, Load load, Store store, Raw &even, Raw &odd)
{
    even.page = rider.page(0);
    odd.page = rider.page(1);
    load(0, even);
    load(1, odd);
    store(0, even);
    load(2, even);
    __syncthreads();
    // (No way out in the middle: where two ways join, loads are waited for as on the shorter one.)
    for (int t = 0; t + 1 < tiles; t += 2) {
        store(t + 1, odd);
        load(t + 3, odd);
        __syncthreads();
        store(t + 2, even);
        load(t + 4, even);
        __syncthreads();
    }
    if (tiles & 1)                       // there is nothing to bring in any more
        __syncthreads();
}

// K: codes to bf16.
template <int D>
__device__ __forceinline__ void bring_k(const AttendParams &p, const Keys &k, const int32_t *table, int head, int part,
                                        ManyLds<D> &lds)
{
    constexpr int L = D / 16;            // lanes of a row
    constexpr int N = kHalf * L / 64;    // 16-byte loads of a lane
    const int lane = threadIdx.x & 63, row = lane / L, col = lane % L;
    const Rider rider = {p.k, table, p.k.scales + head * p.k.s_head, p, k, part, lane};
    const uint8_t *base = p.k.codes + head * p.k.head + 16 * col;
    uint32_t *offsets = lds.offsets[part];
    struct Raw {
        u32x4 codes[N];
        float scale;
        uint32_t there;
        int page;                        // of the tile after the next
    } even, odd;
    const auto load = [&](int t, Raw &raw) {
        uint32_t offset;
        raw.there = rider.place(t, raw.page, offset, raw.scale);
        raw.page = rider.page(t + 2);
        offsets[lane & 31] = offset;
        wave_sync();
#pragma unroll
        for (int l = 0; l < N; ++l)
            raw.codes[l] = *(const u32x4 *)(base + 16 * (int64_t)offsets[row + l * (64 / L)]);
        wave_sync();
    };
    const auto store = [&](int t, const Raw &raw) {
        uint8_t *to = lds.k[t & 1] + (kHalf * part + row) * kRowBytes<D> + 32 * col;
#pragma unroll
        for (int l = 0; l < N; ++l)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t low = raw.codes[l][2 * i], high = raw.codes[l][2 * i + 1];
                *(u32x4 *)(to + l * (64 / L) * kRowBytes<D> + 16 * i) =
                    u32x4{codes_to_bf16<false>(low), codes_to_bf16<true>(low), codes_to_bf16<false>(high),
                          codes_to_bf16<true>(high)};
            }
        if (lane < kHalf)
            lds.kscales[t & 1][kHalf * part + lane] = raw.scale * p.scale_log2;
        if (lane == 0)
            lds.about[t & 1].present[part] = raw.there;
    };
    bring(k.tiles, rider, load, store, even, odd);
}

// V: codes to fp16, transposed.
template <int D>
__device__ __forceinline__ void bring_v(const AttendParams &p, const Keys &k, const int32_t *table, int head, int part,
                                        ManyLds<D> &lds)
{
    constexpr int VW = D / 64;           // dwords of a lane, for one key
    const int lane = threadIdx.x & 63, group = lane >> 4, col = lane & 15;
    const Rider rider = {p.v, table, p.v.scales + head * p.v.s_head, p, k, part, lane};
    const uint8_t *base = p.v.codes + head * p.v.head + (D / 16) * col;
    uint32_t *offsets = lds.offsets[2 + part];
    struct Raw {
        uint32_t codes[8][VW];           // keys 16 (i / 4) + 4 group + i % 4
        float scale;
        uint32_t there;
        int page;                        // of the tile after the next
    } even, odd;
    const auto load = [&](int t, Raw &raw) {
        uint32_t offset;
        raw.there = rider.place(t, raw.page, offset, raw.scale);
        raw.page = rider.page(t + 2);
        offsets[lane & 31] = offset;
        wave_sync();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const u32x4 rows = *(const u32x4 *)&offsets[16 * r + 4 * group];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *at = base + 16 * (int64_t)rows[i];
                if (VW == 2) {
                    const u32x2 v = *(const u32x2 *)at;
                    raw.codes[4 * r + i][0] = v[0];
                    raw.codes[4 * r + i][VW - 1] = v[1];
                } else {
                    raw.codes[4 * r + i][0] = *(const uint32_t *)at;
                }
            }
        }
        wave_sync();
    };
    const auto store = [&](int t, Raw &raw) {
        const uint32_t there = raw.there;
        const float found = raw.scale;
        const bool mine = there >> (lane & 31) & 1;
        // Scales that cannot be weighed with are replaced.
        float scale = mine && usable(found) ? found : kLeastScale;
        if (__ballot(mine && found == 1.0f)) {
            const uint32_t zeros = rows_of_zeros(raw.codes);
            scale = (zeros >> (lane & 31) & 1) && scale == 1.0f ? kLeastScale : scale;
        }
        uint32_t bad = 0;
        if (masked(rider.first(t), there, k.pos_first, k.pos_last, p.window) || __ballot(mine && !usable(found))) {
            // What is not there becomes zeros (0 * NaN would be NaN), and so do NaN codes; keys that hold them or have
            // scales that are not finite are noted.
            const uint32_t none = (uint32_t)__ballot(mine && fabsf(found) < kLeastScale);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int key = 16 * (i / 4) + i % 4;    // of group 0
                const bool here = (there & ~none) >> (4 * group) >> key & 1;
                bool nan = false;
#pragma unroll
                for (int l = 0; l < VW; ++l) {
                    nan |= has_nan_code(raw.codes[i][l]);
                    raw.codes[i][l] = here ? without_nan_codes(raw.codes[i][l]) : 0;
                }
                const uint64_t some = __ballot(nan);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    bad |= (uint32_t)((some >> (16 * g) & 0xffff) != 0) << (key + 4 * g);
            }
            bad |= (uint32_t)__ballot(mine && !(fabsf(found) < __builtin_inff()));
        }
        if (lane < kHalf)
            lds.vscales[t & 1][kHalf * part + lane] = scale * kScaleUnit;
        if (lane == 0)
            lds.about[t & 1].bad[part] = bad;
        // Keys 4 x + i of each 16 go to chunk x % 2, half x / 2: the order of S^T's registers. Element (D / 16) col + i
        // has row 16 i + col, so that lanes write consecutive rows.
        uint8_t *to = lds.v[t & 1] + col * kColumnBytes + 2 * kHalf * part + 16 * (group & 1) + 8 * (group >> 1);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int l = 0; l < VW; ++l) {
                uint32_t both[2][2];     // keys 0, 1 and 2, 3; elements 0, 1 and 2, 3
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t one = raw.codes[4 * r + 2 * i][l], two = raw.codes[4 * r + 2 * i + 1][l];
                    both[i][0] = __builtin_amdgcn_perm(two, one, 0x05010400);
                    both[i][1] = __builtin_amdgcn_perm(two, one, 0x07030602);
                }
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    u32x2 v;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        v[i] = d % 2 ? codes_to_f16<true>(both[i][d / 2]) : codes_to_f16<false>(both[i][d / 2]);
                    *(u32x2 *)(to + 16 * (4 * l + d) * kColumnBytes + 32 * r) = v;
                }
            }
        }
    };
    bring(k.tiles, rider, load, store, even, odd);
}

// One tile of 256 rows of one key head over its keys, or over a piece of them.
//
// The products are transposed as in the few-rows kernel, on 32x32x16
// instructions: each of eight waves holds 32 rows (Q^T and O^T in registers), a
// lane a row with half of the keys. Four more waves bring in K and V, 64 keys at
// a time: they look up the pages, load the codes two tiles ahead, convert them
// (K to bf16, V times its scale to fp16) and store them to LDS while the other
// waves compute the tile before; V transposed, its keys in the order in which
// the first product leaves them. One barrier a tile.
//
// Bound by the matrix units and the vector instructions beside them: 2048 tokens
// of 64 heads over 32768 keys take 2.09 to 2.18 ms, 977 to 1019 TFLOP/s of 1155
// to 1317 that large bf16 products reach here, with the matrix units busy for
// 45% of the cycles and the VALU for 56%, at 1.9 GHz. With V times its scale in
// fp16 on the way into LDS, and weights without it, it took 2.03 ms, but a row's
// accuracy then hung on the scales of keys that it does not see; the scale in the
// weights costs a product and a sum for each. The same waves bringing in and
// computing took 2.39 ms (conversion and exponentials beside each other), sums and
// queries in fewer registers spilled (6.45 ms). 256 rows share each conversion;
// 768 threads and 168 registers leave room for one workgroup a CU. A short
// sequence pays its rows' moves of the reference: a prompt of 2048 tokens by
// itself takes 121 us, 92 with keys that are all the same.
template <int D>
__global__ __launch_bounds__(kManyThreads, 3) void attend_many_kernel(AttendParams p)
{
    constexpr int KS = D / 16;           // matrix instructions of 32 keys of S^T
    constexpr int DT = D / 32;           // tiles of O^T
    __shared__ ManyLds<D> lds;

    Tile w;
    if (!find_tile(p, blockIdx.x, w))
        return;
    const int head = w.head;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int last = min(w.first + kTileRows, w.s.rows) - 1;
    const int base = w.s.n - w.s.m;      // position of the first new token
    Keys k;
    k.pos_first = base + (int)quotient(w.first, p.group);
    k.pos_last = base + (int)quotient(last, p.group);
    k.low = p.window ? max(0, k.pos_first - p.window + 1) : 0;
    const int start = k.low & ~(kTileKeys - 1);
    const int tiles_in_all = max(0, (k.pos_last - start + kTileKeys) / kTileKeys);
    const int tile0 = (int)((int64_t)tiles_in_all * w.piece / w.pieces);
    k.tiles = (int)((int64_t)tiles_in_all * (w.piece + 1) / w.pieces) - tile0;
    k.key0 = start + tile0 * kTileKeys;
    k.last = min(k.pos_last, k.key0 + k.tiles * kTileKeys - 1);           // of this piece

    if (wave >= kComputeWaves) {
        if (k.tiles == 0)
            return;
        const int32_t *table = p.table + w.b * p.table_stride;
        const int part = wave & 1;
        if (wave < kComputeWaves + 2)
            bring_k<D>(p, k, table, head, part, lds);
        else
            bring_v<D>(p, k, table, head, part, lds);
        return;
    }

    // This lane's row.
    const int n = lane & 31, hf = lane >> 5;
    const int r = w.first + 32 * wave + n;
    const int token = (int)quotient(r, p.group), h = r - token * (int)p.group.d;
    const bool row_present = r < w.s.rows;
    const int pos = row_present ? base + token : -1;
    bf16x8 q[KS];
    {
        const uint16_t *row = p.Q + (int64_t)(w.s.start + token) * p.q_t +
                              (int64_t)(head * (int)p.group.d + h) * p.q_h + 8 * hf;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
            u32x4 v = {0, 0, 0, 0};
            if (row_present)
                v = *(const u32x4 *)(row + 16 * t);
            q[t] = __builtin_bit_cast(bf16x8, v);
        }
    }
    // The positions of the wave's rows, between which a tile is masked for some of them (a wave without rows: all are).
    const int r0 = w.first + 32 * wave;
    const int wave_first = r0 < w.s.rows ? base + (int)quotient(r0, p.group) : -1;
    const int wave_last = r0 < w.s.rows ? base + (int)quotient(min(r0 + 32, w.s.rows) - 1, p.group) : -1;

    f32x16 o[DT];
    // A weight past `limit` moves the reference.
    float ref = 0.0f, limit = pos >= 0 ? kUnset : kMostWeight, sum = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[d][i] = 0.0f;
    // The queries are there before the loop, or its first use of them would wait for every load in each round.
#pragma unroll
    for (int i = 0; i < KS; ++i)
        asm volatile("" : "+v"(q[i]));
    if (k.tiles > 0)
        __syncthreads();
    for (int t = 0; t < k.tiles; ++t) {
        const int first = k.key0 + t * kTileKeys;
        const uint8_t *kfrom = lds.k[t & 1] + n * kRowBytes<D> + 16 * hf;
        const uint8_t *vfrom = lds.v[t & 1] + n * kColumnBytes + 16 * hf;
        f32x16 x[2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[b][i] = 0.0f;
        const u32x4 about = *(const u32x4 *)&lds.about[t & 1];
        const auto multiply_k = [&](int b) {
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const bf16x8 a = *(const bf16x8 *)(kfrom + 32 * b * kRowBytes<D> + 32 * i);
                x[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[i], x[b], 0, 0, 0);
            }
        };
        multiply_k(0);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // Register i of x[b] is key 32 b + 8 (i / 4) + 4 hf + i % 4.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 ks = *(const f32x4 *)&lds.kscales[t & 1][32 * b + 8 * i + 4 * hf];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    x[b][4 * i + c] = __builtin_fmaf(x[b][4 * i + c], ks[c], -ref);
            }
            const uint32_t there = (uint32_t)__builtin_amdgcn_readfirstlane((int)about[b]);
            const uint32_t unfit = (uint32_t)__builtin_amdgcn_readfirstlane((int)about[2 + b]);
            if (masked(first + 32 * b, there, wave_first, wave_last, p.window) || unfit) {
                // A row that sees a key whose values are not finite (they are zeros now) becomes NaN. From this lane's
                // first key on, keys [from, to] are seen, where they are there.
                const uint32_t mine = there >> (4 * hf), bad = unfit >> (4 * hf);
                const int to = pos - (first + 32 * b) - 4 * hf, from = p.window ? to - p.window + 1 : -kTileKeys;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int at = 8 * (i / 4) + i % 4;
                    const bool sees = (mine >> at & 1) && at <= to && at >= from;
                    x[b][i] = sees ? x[b][i] : -__builtin_inff();
                    if (sees && (bad >> at & 1))
                        sum = __builtin_nanf("");
                }
            }
            // The next half's scores, while this one's weights are formed.
            if (b == 0)
                multiply_k(1);
            // The weights in fp16, as the second product takes them, and the sum of the exponentials. The values' scales
            // of a lane's 16 keys lie in the 16 lanes around it, which takes one register instead of 16.
            const float scale = lds.vscales[t & 1][32 * b + 8 * (lane >> 2 & 3) + 4 * hf + (lane & 3)];
            u32x4 weights[2];
            float part, most;
            const auto weigh = [&]() {
                part = most = 0.0f;
                for_each([&](auto pair) {
                    constexpr int i = pair.value;
                    const float e0 = __builtin_amdgcn_exp2f(x[b][2 * i]), e1 = __builtin_amdgcn_exp2f(x[b][2 * i + 1]);
                    part += e0;
                    part += e1;
                    const float y0 = e0 * from_lane<2 * i>(scale), y1 = e1 * from_lane<2 * i + 1>(scale);
                    most = fmaxf(fmaxf(most, fabsf(y0)), fabsf(y1));
                    uint32_t two = pack_f16(y0, y1);
                    // Here and now, or all exponentials wait in registers for their sum, and others are spilled.
                    asm volatile("" : "+v"(two), "+v"(part));
                    weights[i / 4][i % 4] = two;
                }, std::make_integer_sequence<int, 8>());
            };
            weigh();
            if (__ballot(most > limit || part > kMostSum)) {
                const float log = __builtin_amdgcn_logf(fabsf(scale));
                float top = -__builtin_inff(), top_x = top;
                for_each([&](auto i) {
                    top = fmaxf(top, x[b][i.value] + from_lane<i.value>(log));
                    top_x = fmaxf(top_x, x[b][i.value]);
                }, std::make_integer_sequence<int, 16>());
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                top_x = fmaxf(top_x, __shfl_xor(top_x, 32, 64));
                const int over = most > limit || part > kMostSum, other = __shfl_xor(over, 32, 64);
                const bool moves = (over | other) != 0 && top > -__builtin_inff();      // the row's other half too
                const float by = moves ? move_reference(ref, top, top_x) : 0.0f;
                const float half = limit == kUnset ? 0.0f : -0.5f * by;
                const float shrink = scaled(1.0f, half);
                sum = scaled(sum, half);
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] *= shrink;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[b][i] -= by;
                limit = moves ? kMostWeight : limit;
                weigh();
            }
            sum = __builtin_fmaf(part, kSumUnit, sum);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const f16x8 a = *(const f16x8 *)(vfrom + 32 * d * kColumnBytes + 64 * b + 32 * c);
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, __builtin_bit_cast(f16x8, weights[c]), o[d], 0, 0, 0);
                }
        }
        __syncthreads();
    }

    sum += __shfl_xor(sum, 32, 64);
    if (!row_present)
        return;
    // Registers i % 8 of all tiles hold consecutive elements.
    constexpr int E = 2 * DT;
    uint16_t *to = p.out + (int64_t)(w.s.start + token) * p.o_t + (int64_t)(head * (int)p.group.d + h) * p.o_h;
    const int64_t at = (int64_t)w.slot * p.many.rows + r - w.first;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int element = E * (8 * (i / 4) + 4 * hf + i % 4);
        float y[E];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                y[2 * d + e] = o[d][i + 8 * e];
        if (w.pieces == 1) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                y[e] = sum == 0.0f ? 0.0f : y[e] * kOutUnit / sum;
            store_bf16<E>(to + element, y);
        } else {
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *(f32x4 *)(p.many.o + at * D + element + e) = f32x4{y[e], y[e + 1], y[e + 2], y[e + 3]};
        }
    }
    if (w.pieces > 1 && hf == 0)
        *(f32x2 *)(p.many.ml + 2 * at) = f32x2{limit == kUnset ? kNoMax : ref, sum};
}

// The rows of the cut tiles, kJoinRows at a time, a wave a row.
template <int D>
__device__ __forceinline__ void join_many(const AttendParams &p, int block, int blocks)
{
    constexpr int E = D / 64;
    const int wave = threadIdx.x >> 6;
    const int shares = (p.many.rows + kJoinRows - 1) / kJoinRows;
    Cuts c;
    const float rate = cut_tiles(p, c);
    Tile w;
    for (; find_cut_tile(p, rate, c, block / shares, w); block += blocks) {
        const int from = kJoinRows * (block % shares);
        for (int i = from + wave; i < from + kJoinRows && w.first + i < w.s.rows; i += 4) {
            const auto index = [&](int piece) { return (int64_t)(w.slot + piece * p.heads) * p.many.rows + i; };
            const int r = w.first + i, token = (int)quotient(r, p.group), h = r - token * (int)p.group.d;
            float total, y[E];
            join_pieces<D>(p.many, w.pieces, 0, 1, index, total, y);
            store_row(p.out + (int64_t)(w.s.start + token) * p.o_t +
                          (int64_t)(w.head * (int)p.group.d + h) * p.o_h, total, y);
        }
    }
}

template <int D>
__global__ __launch_bounds__(kThreads) void join_kernel(AttendParams p)
{
    if ((int)blockIdx.x < p.few_joined)
        join_few<D>(p, blockIdx.x);
    else
        join_many<D>(p, blockIdx.x - p.few_joined, gridDim.x - p.few_joined);
}

}  // namespace dga
