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
    uint16_t *h;            // workspace: [pairs][I / 8][hi 8, lo 8] bf16
    int T, top_k, E, H, I;
};

__device__ __forceinline__ u32x4 load16(const uint8_t *p) { return *(const u32x4 *)p; }
__device__ __forceinline__ u32x4 load16_once(const uint8_t *p)
{
    return __builtin_nontemporal_load((const u32x4 *)p);
}

__device__ __forceinline__ v8i join(const u32x4 &a, const u32x4 &b)
{
    return v8i{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// The pairs (token * top_k + slot) of expert e, in ascending order, into list;
// returns how many. One wave.
__device__ __forceinline__ int list_pairs(const int32_t *ids, int pairs, int e, int lane, uint16_t *list)
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
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lg = lane >> 4;
    const int nkb = p.H >> 7;
    const uint8_t *gate = p.W13 + e * p.w13_e + (n0 + (lane & 15)) * p.ld13 + 16 * lg;
    const uint8_t *up = gate + p.I * p.ld13;
    const float *sg = p.s13 + e * p.s13_e + (n0 >> 7) * p.s13_nb;
    const float *su = p.s13 + e * p.s13_e + ((p.I + n0) >> 7) * p.s13_nb;
    const uint8_t *x[NT];
    const float *sx[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int token = list[min(base + 16 * i + (lane & 15), np - 1)] / p.top_k;
        x[i] = p.X + token * p.ldx + 16 * lg;
        sx[i] = p.sX + token * p.sx_m;
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
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            s.g[c] = load16_once(gate + k + 64 * c);
            s.u[c] = load16_once(up + k + 64 * c);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
                s.x[i][c] = load16(x[i] + k + 64 * c);
            s.sx[i] = sx[i][kb * p.sx_kb];
        }
        s.sg = sg[kb * p.s13_kb];
        s.su = su[kb * p.s13_kb];
    };
    auto compute = [&](const UpStage<NT> &s) {
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

    // red[wave][2 i + (0 gate, 1 up)][lane]: rows 4 lg .. 4 lg + 3 of token lane % 16
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
            const int row = n0 + 4 * lg;
            uint16_t *to = p.h + ((int64_t)list[at] * p.I + (row & ~7)) * 2 + (row & 7);
            *(u32x2 *)to = u32x2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
            *(u32x2 *)(to + 8) = u32x2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
        }
    }
}

// One workgroup per 16 columns of h of one expert. by_pair: slot s of the grid
// is the expert of pair s, if no earlier pair has it (fewer pairs than
// experts); else slot s is expert s.
template <int NT, int D>
__global__ __launch_bounds__(kUpThreads) void gate_up_kernel(LayerParams p, int by_pair)
{
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    __shared__ v4f red[kUpWaves * NT * 2][64];
    const int tiles = p.I >> 4;
    const int slot = blockIdx.x / tiles, n0 = (blockIdx.x - slot * tiles) * 16;
    const int e = by_pair ? p.ids[slot] : slot;
    if (e < 0 || e >= p.E)
        return;
    if (threadIdx.x < 64) {
        const int n = list_pairs(p.ids, p.T * p.top_k, e, threadIdx.x, list);
        if (threadIdx.x == 0)
            count = n;
    }
    __syncthreads();
    const int np = count;
    if (np == 0 || (by_pair && list[0] != slot))
        return;
    int base = 0;
    if (NT >= 4)
        for (; np - base > 32; base += 64)
            up_tiles<NT, D>(p, e, n0, list, base, np, red);
    if (NT >= 2)
        for (; np - base > 16; base += 32)
            up_tiles<NT < 2 ? NT : 2, D>(p, e, n0, list, base, np, red);
    for (; base < np; base += 16)
        up_tiles<1, D>(p, e, n0, list, base, np, red);
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
    u32x4 w[NR];            // 16 NR rows, 64 bytes of K
    u32x4 h[NT][2][2];      // NT x 16 pairs: [operand][hi, lo]
};

// Pairs base .. base + 16 NT of expert e's list against rows n0 .. n0 + 16 NR
// of W2, K blocks [kb0, kb1): res[pair][16 NR] = weight * product.
template <int NT, int NR, int D>
__device__ __forceinline__ void down_tiles(const LayerParams &p, int e, int n0, const uint16_t *list, int base, int np,
                                           int kb0, int kb1, float *res)
{
    const int lane = threadIdx.x & 63, lg = lane >> 4;
    const uint8_t *w = p.W2 + e * p.w2_e + (n0 + (lane & 15)) * p.ld2 + 16 * lg;
    const float *sw = p.s2 + e * p.s2_e + (n0 >> 7) * p.s2_nb;
    const uint16_t *h[NT];
    int pair[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        pair[i] = list[min(base + 16 * i + (lane & 15), np - 1)];
        h[i] = p.h + (int64_t)pair[i] * p.I * 2 + 32 * lg;
    }
    v4f acc[NT][NR], part[NT][NR];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r)
            acc[i][r] = part[i][r] = v4f{0.f, 0.f, 0.f, 0.f};
    DownStage<NT, NR> st[D];
    const int first = 2 * kb0, last = 2 * kb1;  // halves of K blocks
    auto load = [&](int half, DownStage<NT, NR> &s) {
        const int64_t k = (int64_t)min(half, last - 1) * 64;
#pragma unroll
        for (int r = 0; r < NR; ++r)
            s.w[r] = load16_once(w + 16 * r * p.ld2 + k);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    s.h[i][m][c] = *(const u32x4 *)(h[i] + 2 * k + 16 * m + 8 * c);
    };
    auto compute = [&](const DownStage<NT, NR> &s) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            bf16x8 wr[2];
            to_bf16(s.w[r], wr);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        part[i][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wr[m], __builtin_bit_cast(bf16x8, s.h[i][m][c]), part[i][r], 0, 0, 0);
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        load(first + d, st[d]);
    for (int half = first; half < last; half += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {   // D is even: a K block's two halves are in one turn
            if (half + d < last)
                compute(st[d]);
            load(half + d + D, st[d]);
            if (d % 2 && half + d < last) {
                const float s = sw[((half + d) >> 1) * p.s2_kb];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        acc[i][r] += part[i][r] * s;
                        part[i][r] = v4f{0.f, 0.f, 0.f, 0.f};
                    }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
        if (base + 16 * i + (lane & 15) < np) {
            const float weight = p.weights[pair[i]];
#pragma unroll
            for (int r = 0; r < NR; ++r)
                *(v4f *)(res + pair[i] * 16 * NR + 16 * r + 4 * lg) = acc[i][r] * weight;
        }
}

// One workgroup per 16 NR columns of out, for all chosen experts: its waves
// take the items (expert, slice of K), each result goes to its place in LDS,
// and the sum over a token's slots and slices runs in a fixed order.
template <int NR, int PAIRS, int RES>
__global__ __launch_bounds__(kDownThreads) void down_kernel(LayerParams p)
{
    __shared__ float res[RES];          // [slice][pair][16 NR]
    __shared__ int ids[PAIRS];
    __shared__ int first[kMaxExperts];  // each expert's first pair
    __shared__ int active[PAIRS];       // the chosen experts
    __shared__ uint16_t list[kDownWaves][PAIRS];
    __shared__ int count;
    const int pairs = p.T * p.top_k;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n0 = blockIdx.x * 16 * NR;
    for (int i = tid; i < p.E; i += kDownThreads)
        first[i] = kMaxPairs;
    __syncthreads();
    for (int i = tid; i < pairs; i += kDownThreads) {
        const int e = p.ids[i];
        const bool in = e >= 0 && e < p.E;
        ids[i] = in ? e : -1;
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
            if (lead)
                active[n + __popcll(m & ((1ull << lane) - 1))] = e;
            n += __popcll(m);
        }
        if (lane == 0)
            count = n;
    }
    __syncthreads();
    const int nact = count, nkb = p.I >> 7;
    int slices = 1;
    if (nact > 0)
        slices = max(1, min(min((kDownWaves + nact - 1) / nact, nkb), RES / (pairs * 16 * NR)));
    for (int item = wave; item < nact * slices; item += kDownWaves) {
        const int a = item / slices, sl = item - a * slices;
        const int e = __builtin_amdgcn_readfirstlane(active[a]);
        const int np = __builtin_amdgcn_readfirstlane(list_pairs(ids, pairs, e, lane, list[wave]));
        const int kb0 = nkb * sl / slices, kb1 = nkb * (sl + 1) / slices;
        float *to = res + sl * pairs * 16 * NR;
        int base = 0;
        for (; np - base > 16; base += 32)
            down_tiles<2, NR, 2>(p, e, n0, list[wave], base, np, kb0, kb1, to);
        for (; base < np; base += 16)
            down_tiles<1, NR, 2>(p, e, n0, list[wave], base, np, kb0, kb1, to);
    }
    __syncthreads();
    for (int i = tid; i < p.T * 4 * NR; i += kDownThreads) {
        const int t = i / (4 * NR), c = (i - t * 4 * NR) * 4;
        v4f sum = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < p.top_k; ++j) {
            const int pair = t * p.top_k + j;
            if (ids[pair] < 0)
                continue;
            for (int s = 0; s < slices; ++s)
                sum += *(const v4f *)(res + (s * pairs + pair) * 16 * NR + c);
        }
        const uint2 packed = dgk::pack_bf16x4(sum);
        *(u32x2 *)(p.out + t * p.ldo + n0 + c) = u32x2{packed.x, packed.y};
    }
}

}  // namespace dge
