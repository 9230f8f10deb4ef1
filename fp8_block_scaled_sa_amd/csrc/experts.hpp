// experts.hpp -- gfx950 kernels of a mixture-of-experts layer for a few tokens.
//
// With x_t = sX[t, kb] X[t, k], for every slot j of a token t with expert e:
//   g = W13_e[0, I) x_t,  u = W13_e[I, 2I) x_t      (e4m3 codes, 128x128 scales)
//   h = g / (1 + exp(-g)) * u
//   out_t = bf16( sum_j w_tj W2_e h )
//
// A few tokens leave the layer bound by the chosen experts' weights, which
// have to come from HBM once: 3 H I bytes an expert. The two kernels stream
// them as operand A of the matrix instructions (16 rows of weights), with up
// to 16 of the expert's tokens as operand B. Each weight row is read by one
// workgroup only, for all of the expert's tokens.
//
// h is kept as the sum of two bf16 numbers (its rounding to bf16, and the
// rounding of what that leaves: 16 bits of mantissa), so that no rounding
// comes between the products but the last one to bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mfma.hpp"

namespace dge {

using dgk::mfma_e4m3_16x16x128;
using dgk::v4f;
using dgk::v8i;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxTokens = 64;
constexpr int kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kMaxExperts = 1024;
// The kernels keep a lane's offsets in 32 bits: 63 rows of X or 15 rows of
// weights, and both parts of h for all pairs, stay below 2^31 bytes.
constexpr int kMaxWidth = 1 << 18;                // H and I
constexpr int64_t kMaxRowStride = 1 << 25;
constexpr int64_t kMaxTokenScaleStride = 1 << 22;

struct LayerParams {
    const uint8_t *X;       // e4m3 [T, H]
    int64_t ldx;
    const float *sX;
    int64_t sx_m, sx_kb;
    const uint8_t *W13;     // e4m3 [E, 2 I, H]
    int64_t ld13, w13_e;
    const float *s13;
    int64_t s13_e, s13_nb, s13_kb;
    const uint8_t *W2;      // e4m3 [E, H, I]
    int64_t ld2, w2_e;
    const float *s2;
    int64_t s2_e, s2_nb, s2_kb;
    const int32_t *ids;     // [T, top_k]
    const float *weights;   // [T, top_k]
    uint16_t *out;          // bf16 [T, H]
    int64_t ldo;
    uint16_t *h;            // workspace: bf16 [hi, lo][pairs][I]
    int T, top_k, E, H, I;
};

__device__ __forceinline__ u32x4 load16(const uint8_t *base, uint32_t offset)
{
    return *(const u32x4 *)(base + offset);
}

// For data that is read once.
__device__ __forceinline__ u32x4 load16_once(const uint8_t *base, uint32_t offset)
{
    return __builtin_nontemporal_load((const u32x4 *)(base + offset));
}

__device__ __forceinline__ v8i join(const u32x4 &a, const u32x4 &b)
{
    return v8i{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Offset of this lane's 16 bytes in load 0 of a block of 16 rows x 128 bytes
// (load 1: 8 rows further on).
__device__ __forceinline__ uint32_t block_offset(int lane, int64_t ld)
{
    return (uint32_t)((lane & 7) * (int)ld + 32 * (lane >> 4) + 16 * ((lane >> 3) & 1));
}

// From load order to operand order: lanes 8..15 of each 16 take a from lane ^ 8's b, lanes 0..7 b from its a.
__device__ __forceinline__ void exchange_halves(u32x4 &a, u32x4 &b)
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int va = (int)a[c], vb = (int)b[c];
        a[c] = (uint32_t)__builtin_amdgcn_update_dpp(va, vb, 0x128, 0xF, 0xC, false);  // row_ror:8
        b[c] = (uint32_t)__builtin_amdgcn_update_dpp(vb, va, 0x128, 0xF, 0x3, false);
    }
}

__device__ __forceinline__ float from_lane_xor_8(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x128, 0xF, 0xF, false));
}

// The pairs (token * top_k + slot) of expert e, in ascending order, into list;
// returns how many. One wave.
template <typename Id>
__device__ __forceinline__ int list_pairs(const Id *ids, int pairs, int e, int lane, uint16_t *list)
{
    int n = 0;
    for (int c = 0; c < pairs; c += 64) {
        const bool hit = c + lane < pairs && ids[c + lane] == e;
        const uint64_t m = __ballot(hit);
        if (hit)
            list[n + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(c + lane);
        n += __popcll(m);
    }
    __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses stay in program order
    return n;
}

// ---------------------------------------------------------------- gate and up

constexpr int kUpWaves = 4;
constexpr int kUpThreads = 64 * kUpWaves;

template <int NT>
struct UpStage {
    u32x4 g[2], u[2];       // 16 gate rows and 16 up rows, 128 bytes of K
    u32x4 x[NT][2];         // NT x 16 tokens
    float sx[NT], sg, su;
};

template <int NT, int D>
__device__ __forceinline__ void up_tiles(const LayerParams &p, int e, int n0, const uint16_t *list, int base, int np,
                                         v4f (*red)[64])
{
    const int lane = threadIdx.x & 63, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int nkb = p.H >> 7;
    const uint8_t *gate = p.W13 + e * p.w13_e + n0 * p.ld13;
    const uint8_t *up = gate + p.I * p.ld13;
    const uint32_t row0 = block_offset(lane, p.ld13), row8 = row0 + 8 * (uint32_t)p.ld13;
    const float *sg = p.s13 + e * p.s13_e + (n0 >> 7) * p.s13_nb;
    const float *su = p.s13 + e * p.s13_e + ((p.I + n0) >> 7) * p.s13_nb;
    uint32_t xo[NT], so[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int token = list[min(base + 16 * i + (lane & 15), np - 1)] / p.top_k;
        xo[i] = (uint32_t)(token * (int)p.ldx + 32 * lg);
        so[i] = (uint32_t)(token * (int)p.sx_m);
    }
    v4f ag[NT], au[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        ag[i] = au[i] = v4f{0.f, 0.f, 0.f, 0.f};

    // This wave's K blocks: wave, wave + kUpWaves, ...; D of them in flight.
    const int n = (nkb - wave + kUpWaves - 1) / kUpWaves;
    UpStage<NT> st[D];
    auto load = [&](int j, UpStage<NT> &s) {
        const int kb = min(wave + j * kUpWaves, nkb - 1);
        const int64_t k = (int64_t)kb * 128;
        s.g[0] = load16_once(gate + k, row0);
        s.g[1] = load16_once(gate + k, row8);
        s.u[0] = load16_once(up + k, row0);
        s.u[1] = load16_once(up + k, row8);
        const float *sx = p.sX + kb * p.sx_kb;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            s.x[i][0] = load16(p.X + k, xo[i]);
            s.x[i][1] = load16(p.X + k + 16, xo[i]);
            s.sx[i] = sx[so[i]];
        }
        s.sg = sg[kb * p.s13_kb];
        s.su = su[kb * p.s13_kb];
    };
    auto compute = [&](UpStage<NT> &s) {
        exchange_halves(s.g[0], s.g[1]);
        exchange_halves(s.u[0], s.u[1]);
        const v8i wg = join(s.g[0], s.g[1]), wu = join(s.u[0], s.u[1]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const v8i xi = join(s.x[i][0], s.x[i][1]);
            ag[i] += mfma_e4m3_16x16x128(wg, xi) * (s.sx[i] * s.sg);
            au[i] += mfma_e4m3_16x16x128(wu, xi) * (s.sx[i] * s.su);
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        load(d, st[d]);
    for (int j = 0; j < n; j += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (j + d < n)
                compute(st[d]);
            load(j + d + D, st[d]);
        }
    }

    // red[wave][i][gate, up][lane]: rows 4 lg .. 4 lg + 3 of token lane % 16
    __syncthreads();  // the previous pass's reads
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        red[(wave * NT + i) * 2][lane] = ag[i];
        red[(wave * NT + i) * 2 + 1][lane] = au[i];
    }
    __syncthreads();
    for (int i = wave; i < NT; i += kUpWaves) {
        v4f g = {0.f, 0.f, 0.f, 0.f}, u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kUpWaves; ++w) {
            g += red[(w * NT + i) * 2][lane];
            u += red[(w * NT + i) * 2 + 1][lane];
        }
        const int at = base + 16 * i + (lane & 15);
        if (at < np) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float h = g[c] / (1.0f + __expf(-g[c])) * u[c];
                hi[c] = dgk::bf16_rne(h);
                lo[c] = dgk::bf16_rne(h - __uint_as_float(hi[c] << 16));
            }
            uint16_t *to = p.h + (int64_t)list[at] * p.I + n0 + 4 * lg;
            *(u32x2 *)to = u32x2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
            to += (int64_t)p.T * p.top_k * p.I;
            *(u32x2 *)to = u32x2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
        }
    }
}

// One workgroup per 16 columns of h of one expert. by_pair: slot s of the grid
// is the expert of pair s, if no earlier pair has it (fewer pairs than
// experts); else slot s is expert s. With up to 64 pairs every wave lists the
// expert's pairs for itself.
template <int NT, int D, bool FEW>
__global__ __launch_bounds__(kUpThreads) void gate_up_kernel(LayerParams p, int by_pair)
{
    __shared__ uint16_t list[FEW ? 64 * kUpWaves : kMaxPairs];
    __shared__ int count;
    __shared__ v4f red[kUpWaves * NT * 2][64];
    const int tiles = p.I >> 4, pairs = p.T * p.top_k;
    const int slot = blockIdx.x / tiles, n0 = (blockIdx.x - slot * tiles) * 16;
    const int e = __builtin_amdgcn_readfirstlane(by_pair ? p.ids[slot] : slot);
    if (e < 0 || e >= p.E)
        return;
    int np;
    uint16_t *mine = list;
    if (FEW) {
        mine = list + 64 * (threadIdx.x >> 6);
        np = list_pairs(p.ids, pairs, e, threadIdx.x & 63, mine);
    } else {
        if (threadIdx.x < 64) {
            const int n = list_pairs(p.ids, pairs, e, threadIdx.x, list);
            if (threadIdx.x == 0)
                count = n;
        }
        __syncthreads();
        np = count;
    }
    np = __builtin_amdgcn_readfirstlane(np);
    if (np == 0 || (by_pair && mine[0] != slot))
        return;
    int base = 0;
    if (NT >= 4)
        for (; np - base > 32; base += 64)
            up_tiles<NT, D>(p, e, n0, mine, base, np, red);
    if (NT >= 2)
        for (; np - base > 16; base += 32)
            up_tiles<NT < 2 ? NT : 2, D>(p, e, n0, mine, base, np, red);
    for (; base < np; base += 16)
        up_tiles<1, D>(p, e, n0, mine, base, np, red);
}

// ---------------------------------------------------------------- down

constexpr int kDownWaves = 8;
constexpr int kDownThreads = 64 * kDownWaves;

// 16 e4m3 codes as two operands of 8 bf16 numbers (exact).
__device__ __forceinline__ void to_bf16(const u32x4 &w, bf16x8 *out)
{
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[2 * m + c], 1.0f, false);
            const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[2 * m + c], 1.0f, true);
            out[m][4 * c] = a[0];
            out[m][4 * c + 1] = a[1];
            out[m][4 * c + 2] = b[0];
            out[m][4 * c + 3] = b[1];
        }
    }
}

template <int NT, int NR>
struct DownStage {
    u32x4 w[NR][2];         // 16 NR rows, 128 bytes of K
    u32x4 h[NT][4];         // NT x 8 pairs, hi and lo: this lane's 32 of 128 values
    float s;
};

// Pairs base .. base + 8 NT of expert e's list against rows n0 .. n0 + 16 NR
// of W2, K blocks [kb0, kb1): res[pair][16 NR] = weight * product.
template <int NT, int NR, int D>
__device__ __forceinline__ void down_tiles(const LayerParams &p, int e, int n0, const uint16_t *list, int base, int np,
                                           int kb0, int kb1, float *res)
{
    const int lane = threadIdx.x & 63, lg = lane >> 4, col = lane & 15;
    const uint8_t *w = p.W2 + e * p.w2_e + n0 * p.ld2;
    const uint32_t row0 = block_offset(lane, p.ld2), row8 = row0 + 8 * (uint32_t)p.ld2;
    const float *sw = p.s2 + e * p.s2_e + (n0 >> 7) * p.s2_nb;
    const uint8_t *h = (const uint8_t *)p.h;
    uint32_t ho[NT];
    int pair[NT];
    float weight[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        pair[i] = list[min(base + 8 * i + (col & 7), np - 1)];
        weight[i] = p.weights[pair[i]];
        // column col: the hi (col < 8) or lo part of pair col % 8
        ho[i] = (uint32_t)(((col >> 3) * p.T * p.top_k + pair[i]) * p.I * 2 + 64 * lg);
    }
    v4f acc[NT][NR];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r)
            acc[i][r] = v4f{0.f, 0.f, 0.f, 0.f};
    DownStage<NT, NR> st[D];
    auto load = [&](int j, DownStage<NT, NR> &s) {
        const int kb = min(j, kb1 - 1);
        const int64_t k = (int64_t)kb * 128;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            s.w[r][0] = load16_once(w + 16 * r * p.ld2 + k, row0);
            s.w[r][1] = load16_once(w + 16 * r * p.ld2 + k, row8);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                s.h[i][q] = load16(h + 2 * k + 16 * q, ho[i]);
        s.s = sw[kb * p.s2_kb];
    };
    auto compute = [&](DownStage<NT, NR> &s) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            exchange_halves(s.w[r][0], s.w[r][1]);
            bf16x8 wr[4];
            to_bf16(s.w[r][0], wr);
            to_bf16(s.w[r][1], wr + 2);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                v4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wr[q], __builtin_bit_cast(bf16x8, s.h[i][q]), part,
                                                                   0, 0, 0);
                acc[i][r] += part * s.s;
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        load(kb0 + d, st[d]);
    for (int j = kb0; j < kb1; j += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (j + d < kb1)
                compute(st[d]);
            load(j + d + D, st[d]);
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            v4f sum;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sum[c] = (acc[i][r][c] + from_lane_xor_8(acc[i][r][c])) * weight[i];
            if (col < 8 && base + 8 * i + col < np)
                *(v4f *)(res + pair[i] * 16 * NR + 16 * r + 4 * lg) = sum;
        }
    }
}

// One workgroup per 16 NR columns of out, for all chosen experts. Their K
// blocks, one expert's after the other's, are dealt to the waves in equal
// runs; each wave's part of an expert goes to a place of its own in LDS, and
// the sum over a token's slots and an expert's parts runs in a fixed order.
template <int NR, int PAIRS, int RES, int NT, int D>
__global__ __launch_bounds__(kDownThreads) void down_kernel(LayerParams p)
{
    constexpr bool kFew = PAIRS <= 64;
    __shared__ float res[RES];                // [part][pair][16 NR]
    __shared__ int16_t active_of[PAIRS];      // each pair's place in active, -1 without an expert
    __shared__ uint16_t list[kDownWaves][PAIRS];
    __shared__ int16_t ids[kFew ? 1 : PAIRS];
    __shared__ int16_t active[kFew ? 1 : PAIRS];       // the chosen experts
    __shared__ int first[kFew ? 1 : kMaxExperts];      // each expert's first pair
    __shared__ int16_t place[kFew ? 1 : kMaxExperts];  // ... and its place in active
    static_assert(RES >= 2 * PAIRS * 16 * NR, "an expert has two parts where the waves' runs cut it");
    __shared__ int count;
    const int pairs = p.T * p.top_k;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16 * NR;

    int nact = 0;
    int my_expert = -1;                       // kFew: lane a's chosen expert a ...
    uint64_t my_pairs = 0;                    // ... and the pairs that have it
    if (kFew) {
        int id = lane < pairs ? p.ids[lane] : -1;
        if (id >= p.E)
            id = -1;
        int at = -1;
        for (uint64_t left = __ballot(id >= 0); left; ++nact) {
            const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
            const uint64_t m = __ballot(id == e);
            left &= ~m;
            if (id == e)
                at = nact;
            if (lane == nact) {
                my_expert = e;
                my_pairs = m;
            }
        }
        if (wave == 0 && lane < pairs)
            active_of[lane] = (int16_t)at;
    } else {
        for (int i = tid; i < p.E; i += kDownThreads)
            first[i] = kMaxPairs;
        __syncthreads();
        for (int i = tid; i < pairs; i += kDownThreads) {
            const int e = p.ids[i];
            const bool in = e >= 0 && e < p.E;
            ids[i] = (int16_t)(in ? e : -1);
            if (in)
                atomicMin(&first[e], i);
        }
        __syncthreads();
        if (wave == 0) {
            int n = 0;
            for (int c = 0; c < pairs; c += 64) {
                const int e = c + lane < pairs ? ids[c + lane] : -1;
                const bool lead = e >= 0 && first[e] == c + lane;
                const uint64_t m = __ballot(lead);
                if (lead) {
                    const int at = n + __popcll(m & ((1ull << lane) - 1));
                    active[at] = (int16_t)e;
                    place[e] = (int16_t)at;
                }
                n += __popcll(m);
            }
            if (lane == 0)
                count = n;
        }
        __syncthreads();
        nact = count;
        for (int i = tid; i < pairs; i += kDownThreads)
            active_of[i] = ids[i] >= 0 ? place[ids[i]] : (int16_t)-1;
    }
    nact = __builtin_amdgcn_readfirstlane(nact);

    // Waves in use: an expert's parts, (waves / nact rounded up) + 1 at most, have to fit res.
    const int nkb = p.I >> 7, total = nact * nkb;
    const int parts_cap = RES / (pairs * 16 * NR);
    const int waves = max(1, min(min(kDownWaves, total), nact * (parts_cap - 1)));
    if (wave < waves && nact > 0) {
        int b = total * wave / waves;
        const int end = total * (wave + 1) / waves;
        while (b < end) {
            const int a = b / nkb, kb0 = b - a * nkb, kb1 = min(nkb, kb0 + end - b);
            int e, np;
            if (kFew) {
                e = __builtin_amdgcn_readlane(my_expert, a);
                const uint64_t m = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)my_pairs, a) |
                                   (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(my_pairs >> 32), a) << 32;
                if (m >> lane & 1)
                    list[wave][__popcll(m & ((1ull << lane) - 1))] = (uint16_t)lane;
                __builtin_amdgcn_wave_barrier();
                np = __popcll(m);
            } else {
                e = __builtin_amdgcn_readfirstlane(active[a]);
                np = __builtin_amdgcn_readfirstlane(list_pairs(ids, pairs, e, lane, list[wave]));
            }
            // the part's number: this wave among those that have blocks of the expert
            const int part = wave - ((a * nkb + 1) * waves - 1) / total;
            float *to = res + part * pairs * 16 * NR;
            int base = 0;
            if (NT >= 2)
                for (; np - base > 8; base += 16)
                    down_tiles<NT < 2 ? NT : 2, NR, D>(p, e, n0, list[wave], base, np, kb0, kb1, to);
            for (; base < np; base += 8)
                down_tiles<1, NR, D>(p, e, n0, list[wave], base, np, kb0, kb1, to);
            b += kb1 - kb0;
        }
    }
    __syncthreads();
    for (int i = tid; i < p.T * 4 * NR; i += kDownThreads) {
        const int t = i / (4 * NR), c = (i - t * 4 * NR) * 4;
        v4f sum = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < p.top_k; ++j) {
            const int pair = t * p.top_k + j, a = active_of[pair];
            if (a < 0)
                continue;
            const int parts = ((a + 1) * nkb * waves - 1) / total - ((a * nkb + 1) * waves - 1) / total + 1;
            for (int s = 0; s < parts; ++s)
                sum += *(const v4f *)(res + (s * pairs + pair) * 16 * NR + c);
        }
        const uint2 packed = dgk::pack_bf16x4(sum);
        *(u32x2 *)(p.out + t * p.ldo + n0 + c) = u32x2{packed.x, packed.y};
    }
}

}  // namespace dge
