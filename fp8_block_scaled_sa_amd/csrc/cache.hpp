// cache.hpp -- gfx950 kernels of a paged cache of e4m3 codes: rotary positions
// and quantisation on the way in, dequantisation on the way out.
//
// A cache holds a row of D codes and one fp32 scale for each slot (a page and
// an offset in it) and head, in the format of the 1x128 quantiser:
//   amax = max |x| over the row's D values,  s = amax / 448 (1 for a row of zeros),
//   code = e4m3(x / s), rounded to nearest even.
// The rotary positions turn rot / 2 pairs (x, y) of a head by a = pos * freq_i:
//   (x, y) -> factor * (x cos a - y sin a, x sin a + y cos a)
// with the pairs (i, i + rot/2) or (2i, 2i + 1).
//
// Both kernels touch each byte once and are bound by HBM.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm.hpp"

namespace dgc {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Quotient of a number below 2^31 by a divisor fixed at launch: with
// l = ceil(log2 d), mul = ceil(2^(31 + l) / d) is below 2^32 and
// floor(j mul / 2^(31 + l)) = floor(j / d), since mul d - 2^(31 + l) < d <= 2^l.
struct Divisor {
    uint32_t d, mul, shift;
};

inline Divisor divisor(uint32_t d)
{
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d)
        ++l;
    return Divisor{d, (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), 31 + l};
}

__device__ __forceinline__ uint32_t quotient(uint32_t j, const Divisor &v)
{
    return (uint32_t)(((uint64_t)j * v.mul) >> v.shift);
}

struct Pages {
    uint8_t *codes;                      // row of slot (page, token) and head at page * c_page + token * c_token + head * c_head
    int64_t c_page, c_token, c_head;
    float *scales;
    int64_t s_page, s_token, s_head;
};

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;            // of a workgroup of the write kernel
constexpr int kMaxHalf = 64;             // rotating pairs of a head

struct WriteParams {
    const void *Q;                       // [T, q_heads, D]; NULL: no queries
    int64_t q_t, q_h;
    uint16_t *Q_out;                     // bf16 [T, q_heads, D]
    int64_t qo_t, qo_h;
    const void *K, *V;                   // [T, heads, D]
    int64_t k_t, k_h, v_t, v_h;
    const int32_t *positions;
    const double *freqs;
    const int64_t *slots;
    Pages k, v;
    Divisor page;                        // slots of a page
    int64_t slots_in_all;
    int T, q_heads, heads, half, interleaved;
    float factor;
    int tokens;                          // of a workgroup
};

// A workgroup takes the rows (queries, keys, values) of one token, or of a few
// where a token has few, D / 8 lanes a row and 8 elements a lane, whole
// 128-byte lines with every load and store. The angles' sines and cosines are
// formed once per workgroup into LDS: the angle in 64 bits as turns (pos * freq
// / 2 pi), of which the whole turns are dropped exactly, so that far positions
// cost no precision; the rest is 32-bit. The other element of a pair lies in
// the same lane (interleaved) or rot / 16 lanes away (half), one lane exchange.
// The table of a program that keeps cosines and sines would be read for every
// token instead; forming them takes one wave for the 64 pairs of a token.
template <bool BF16, int D>
__global__ __launch_bounds__(kThreads) void rope_cache_write_kernel(WriteParams p)
{
    constexpr int LANES = D / 8;                 // of a row
    constexpr int ROWS = kThreads / LANES;       // of a round
    constexpr int NW = BF16 ? 1 : 2;             // 16-byte loads of a lane
    __shared__ float turn[kMaxTokens][2][kMaxHalf];  // cosines, sines
    const int c = threadIdx.x % LANES;
    // Workgroups are dealt to the 8 XCDs in turn; renumbered, each XCD takes a
    // contiguous range of tokens, whose scales share lines.
    const int nwg = gridDim.x, xcd = blockIdx.x % 8, per = nwg / 8, extra = nwg % 8;
    const int first = (xcd * per + min(xcd, extra) + (int)blockIdx.x / 8) * p.tokens;
    const int tokens = min(p.tokens, p.T - first);
    const int rows = p.q_heads + 2 * p.heads, all = tokens * rows;

    const auto load = [&](int r, u32x4 *w) {
        const int t = p.tokens == 1 ? 0 : r / rows, row = r - t * rows;
        const int64_t token = first + t;
        const void *base;
        int64_t at;
        if (row < p.q_heads) {
            base = p.Q;
            at = token * p.q_t + row * p.q_h;
        } else if (row < p.q_heads + p.heads) {
            base = p.K;
            at = token * p.k_t + (row - p.q_heads) * p.k_h;
        } else {
            base = p.V;
            at = token * p.v_t + (row - p.q_heads - p.heads) * p.v_h;
        }
        const u32x4 *from = (const u32x4 *)((const uint8_t *)base + (at + 8 * c) * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < NW; ++i)
            w[i] = __builtin_nontemporal_load(from + i);
    };

    const int step = ROWS * gridDim.y;
    int r = blockIdx.y * ROWS + (int)threadIdx.x / LANES;
    u32x4 w[NW] = {};
    if (r < all)
        load(r, w);
    for (int i = threadIdx.x; i < tokens * p.half; i += kThreads) {
        const int t = i / p.half, pair = i - t * p.half;
        const double turns = (double)p.positions[first + t] * p.freqs[pair] * 0.15915494309189533577;
        float s, co;
        sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &co);
        turn[t][0][pair] = co * p.factor;
        turn[t][1][pair] = s * p.factor;
    }
    __syncthreads();

    // Every lane of a wave takes part in each round (the lane exchange needs its neighbours).
    for (int base = blockIdx.y * ROWS; base < all; base += step, r += step) {
        u32x4 next[NW] = {};
        if (r + step < all)
            load(r + step, next);
        const bool present = r < all;
        const int t = p.tokens == 1 ? 0 : min(r, all - 1) / rows, row = r - t * rows;
        float x[8];
        if (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = dgq::bf16_to_f32(w[0][i] & 0xffffu);
                x[2 * i + 1] = __uint_as_float(w[0][i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __uint_as_float(w[i / 4][i % 4]);
        }
        if (p.half > 0) {
            const bool turns = row < p.q_heads + p.heads && 8 * c < 2 * p.half;
            if (p.interleaved) {
                if (turns) {
                    const f32x4 co = *(const f32x4 *)&turn[t][0][4 * c], s = *(const f32x4 *)&turn[t][1][4 * c];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = __builtin_fmaf(a, co[i], -b * s[i]);
                        x[2 * i + 1] = __builtin_fmaf(a, s[i], b * co[i]);
                    }
                }
            } else {
                const int apart = p.half / 8;
                const bool second = c >= apart;
                const int other = (threadIdx.x & 63) + (second ? -apart : apart);
                float y[8];
#pragma unroll
                for (int i = 0; i < NW * 4; ++i) {
                    const uint32_t v = (uint32_t)__shfl((int)w[i / 4][i % 4], other, 64);
                    if (BF16) {
                        y[2 * i] = dgq::bf16_to_f32(v & 0xffffu);
                        y[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
                    } else {
                        y[i] = __uint_as_float(v);
                    }
                }
                if (turns) {
                    const int pair = 8 * (second ? c - apart : c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float co = turn[t][0][pair + i], s = turn[t][1][pair + i];
                        x[i] = __builtin_fmaf(x[i], co, second ? y[i] * s : -y[i] * s);
                    }
                }
            }
        }
        if (present && row < p.q_heads) {
            dgn::store8<true>(p.Q_out, (int64_t)(first + t) * p.qo_t + row * p.qo_h + 8 * c, x);
        } else {
            // The row's scale and codes, as the 1x128 quantiser forms them; every lane of the wave takes part.
            uint32_t abits = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                abits = max(abits, __float_as_uint(x[i]) & 0x7fffffffu);
            abits = LANES == 16 ? dgn::max_over_16_lanes(abits) : dgq::max_over_8_lanes(abits);
            // A row with an infinity or NaN gets the scale NaN, and comes back as NaN.
            const float amax = abits < 0x7f800000u ? __uint_as_float(abits) : __uint_as_float(0x7fc00000u);
            const float s = amax == 0.0f ? 1.0f : amax / dgq::kE4m3Max;
            float q[8];
            if (s >= 0x1p-64f) {
                const float rc = 1.0f / s;
                const float rc_lo = __builtin_fmaf(-s, rc, 1.0f) * rc;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = dgq::quotient(x[i], s, rc, rc_lo);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = x[i] / s;
            }
            uint32_t code[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = fminf(fmaxf(q[4 * half + i], -dgq::kE4m3Max), dgq::kE4m3Max);
                const int low = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                code[half] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], low, true);
            }
            const int64_t slot = present ? p.slots[first + t] : -1;
            if (slot >= 0 && slot < p.slots_in_all) {
                const bool key = row < p.q_heads + p.heads;
                const Pages &to = key ? p.k : p.v;
                const int head = row - p.q_heads - (key ? 0 : p.heads);
                const uint32_t page = quotient((uint32_t)slot, p.page), token = (uint32_t)slot - page * p.page.d;
                *(u32x2 *)(to.codes + page * to.c_page + token * to.c_token + head * to.c_head + 8 * c) =
                    u32x2{code[0], code[1]};
                if (c == 0)
                    to.scales[page * to.s_page + token * to.s_token + head * to.s_head] = s;
            }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i)
            w[i] = next[i];
    }
}

struct ReadParams {
    Pages from;
    const int64_t *slots;
    void *out;                           // bf16 or fp32 [T, heads, D]
    int64_t o_t, o_h;
    Divisor page, head;
    int64_t slots_in_all;
    int64_t rows;                        // T * heads
};

constexpr int kReadRows = 4;             // rows of a thread, all of whose loads are in flight together

// Each thread turns 16 bytes of output (8 bf16 or 4 fp32 values) of kReadRows
// rows, so that every load and store instruction covers whole rows.
template <bool BF16, int D>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(ReadParams p)
{
    constexpr int E = BF16 ? 8 : 4;
    constexpr int LANES = D / E;
    constexpr int ROWS = kThreads / LANES;
    const int c = threadIdx.x % LANES;
    const int64_t first = (int64_t)blockIdx.x * (ROWS * kReadRows) + threadIdx.x / LANES;
    uint32_t code[kReadRows][2];
    float scale[kReadRows];
    int64_t to[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const uint32_t r = (uint32_t)min(first + i * ROWS, p.rows - 1);
        const uint32_t t = quotient(r, p.head), head = r - t * p.head.d;
        const int64_t slot = p.slots[t];
        to[i] = t * p.o_t + head * p.o_h + E * c;
        code[i][0] = code[i][1] = 0;
        scale[i] = 0.0f;
        if (slot >= 0 && slot < p.slots_in_all) {
            const uint32_t page = quotient((uint32_t)slot, p.page), token = (uint32_t)slot - page * p.page.d;
            const uint8_t *at = p.from.codes + page * p.from.c_page + token * p.from.c_token + head * p.from.c_head + E * c;
            if (BF16) {
                const u32x2 v = __builtin_nontemporal_load((const u32x2 *)at);
                code[i][0] = v[0];
                code[i][1] = v[1];
            } else {
                code[i][0] = __builtin_nontemporal_load((const uint32_t *)at);
            }
            scale[i] = p.from.scales[page * p.from.s_page + token * p.from.s_token + head * p.from.s_head];
        }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        if (first + i * ROWS >= p.rows)
            return;
        float x[E];
#pragma unroll
        for (int h = 0; h < E / 4; ++h) {
            const f32x2 low = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[i][h], false);
            const f32x2 high = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[i][h], true);
            x[4 * h] = low[0] * scale[i];
            x[4 * h + 1] = low[1] * scale[i];
            x[4 * h + 2] = high[0] * scale[i];
            x[4 * h + 3] = high[1] * scale[i];
        }
        if (BF16)
            __builtin_nontemporal_store(u32x4{dgn::pack_bf16(x[0], x[1]), dgn::pack_bf16(x[2], x[3]),
                                              dgn::pack_bf16(x[E - 4], x[E - 3]), dgn::pack_bf16(x[E - 2], x[E - 1])},
                                        (u32x4 *)((uint16_t *)p.out + to[i]));
        else
            __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, (f32x4 *)((float *)p.out + to[i]));
    }
}

}  // namespace dgc
