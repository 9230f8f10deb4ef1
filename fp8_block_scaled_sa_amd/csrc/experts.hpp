// experts.hpp -- gfx950 kernels of a mixture-of-experts layer for a few tokens.
//
// With x_t = sX[t, kb] X[t, k], for every slot j of a token t with expert e:
//   g = W13_e[0, I) x_t,  u = W13_e[I, 2I) x_t      (e4m3 codes, 128x128 scales)
//   h = g / (1 + exp(-g)) * u
//   out_t = bf16( sum_j w_tj W2_e h )
//
// A few tokens leave the layer bound by the chosen experts' weights, which
// have to come from HBM once: 3 H I bytes an expert. Two kernels stream them as
// operand A of the matrix instructions (16 rows of weights), with up to 16 of
// the expert's tokens as operand B: each weight row is read by one workgroup
// only, for all of the expert's tokens. A third, small one adds a token's slots.
// Doing that in the second kernel, by the workgroup of a column block that
// arrives last, took three times the second kernel's time: the device-wide
// fences write back and drop what the XCDs' L2s hold.
//
// Lane order of the weight loads. The matrix instructions want lane l to hold
// row l % 16 and the K bytes of group g = l / 16, 32 a lane. A load in that
// order takes half of each 128-byte line and leaves the other half to the next
// load, which costs a quarter of the bandwidth. So load p of a 16 x 128 byte
// block reads the rows 8p + l % 8 and the 16 bytes 2g + l / 8 % 2 of the line
// (whole lines: 6.6 to 7.2 TB/s in a kernel that only reads, against 4.9 for
// 16 rows x 64 bytes, both non-temporal; 6.1 against 4.7 in the first kernel
// for one token, 38.5 against 49.9 us), and the two registers' halves are then
// exchanged between lanes l and l ^ 8, two DPP moves for each pair of dwords.
//
// h is kept as the sum of two bf16 numbers (its rounding to bf16, and the
// rounding of what that leaves: 16 bits of mantissa), so that no rounding
// comes between the products but the last one to bf16. The second product
// takes them as 8 + 8 columns of one operand and adds the two results.
//
// Measured for H 7168, I 2048, graph replays over three inputs in turn (in
// brackets the first and the second kernel's median under the kernel trace):
//   1 token, 8 of 32 experts:    65 us (38.0, 23.7), 352 MB
//   8 tokens, 8 of 32:          226 us (136, 86), 1268 MB
//   16 tokens, 8 of 32:         249 us (147, 90), 1396 MB
//   64 tokens, 8 of 32:         337 us (215, 117), 1411 MB
// With one tile of tokens the layer runs at 5.4 to 5.6 TB/s, near what a kernel
// that only reads reaches; with more, it falls to 4.1 or 4.2 TB/s: in the first
// the waves split K and each reads its own tokens' blocks from L2, two loads a
// tile beside the four of the weights, in the second the chunks get shorter.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kernels.hpp"

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
constexpr int kDownWaves = 8;
constexpr int kDownRows = 16 * kDownWaves;
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
    float *part;            // and fp32 [pairs][H], each pair's weighted product
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
__device__ __forceinline__ int list_pairs(const LayerParams &p, int e, int lane, uint16_t *list)
{
    const int pairs = p.T * p.top_k;
    int n = 0;
    for (int c = 0; c < pairs; c += 64) {
        const bool hit = c + lane < pairs && p.ids[c + lane] == e;
        const uint64_t m = __ballot(hit);
        if (hit)
            list[n + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(c + lane);
        n += __popcll(m);
    }
    __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses stay in program order
    return n;
}

// The expert of one slot of the grid, or -1: by_pair (fewer pairs than experts)
// slot s has the expert of pair s, else slot s is expert s.
__device__ __forceinline__ int slot_expert(const LayerParams &p, int by_pair, int slot)
{
    const int e = __builtin_amdgcn_readfirstlane(by_pair ? p.ids[slot] : slot);
    return e >= 0 && e < p.E ? e : -1;
}

// ---------------------------------------------------------------- gate and up

constexpr int kUpWaves = 4;
constexpr int kUpThreads = 64 * kUpWaves;

// h as two bf16 numbers. A finite h that rounds to infinity keeps bf16's largest
// number as hi, and its lo the rest of it; an infinite or NaN h has no rest (hi +
// lo would be NaN). That is decided from hi, not from h - hi: the compiler fuses
// h's last product into that subtraction, which leaves an infinity where h and hi
// are both infinite (and makes lo the rest of the product before its rounding).
__device__ __forceinline__ void split_bf16(float h, uint32_t &hi, uint32_t &lo)
{
    hi = dgk::bf16_rne(h);
    if ((hi & 0x7fffu) == 0x7f80u && __builtin_fabsf(h) < INFINITY)
        hi -= 1;
    const float rest = h - __uint_as_float(hi << 16);
    lo = (hi & 0x7f80u) == 0x7f80u ? 0 : dgk::bf16_rne(rest);
}

// Four consecutive values of h of one pair, from row on.
__device__ __forceinline__ void store_h(const LayerParams &p, int pair, int row, const v4f &g, const v4f &u)
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        split_bf16(g[c] / (1.0f + __expf(-g[c])) * u[c], hi[c], lo[c]);
    uint16_t *to = p.h + (int64_t)pair * p.I + row;
    *(u32x2 *)to = u32x2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
    to += (int64_t)p.T * p.top_k * p.I;
    *(u32x2 *)to = u32x2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
}

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
    // Past the last one the last block of K is read again (a wave may have none).
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
        if (at < np)
            store_h(p, list[at], n0 + 4 * lg, g, u);
    }
}

// One workgroup per 16 columns of h of one expert (a later pair with an
// expert that an earlier one has leaves it to that one's slot), its waves
// taking the K blocks in turn: for one token and 8 experts of I = 2048 that
// makes 1024 workgroups, 16 waves a CU, each with D = 2 blocks of 32 rows (8 KB)
// in flight. D = 3 changed nothing there (38.6 us) and cost a tenth where K is
// short (19.6 against 22.9 us at H 2048). One wave lists the expert's pairs:
// where every wave listed up to 64 of them for itself, without the barrier, 17
// cases from 1 to 64 tokens kept their time within 1%.
template <int NT, int D>
__global__ __launch_bounds__(kUpThreads) void gate_up_kernel(LayerParams p, int by_pair)
{
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    __shared__ v4f red[kUpWaves * NT * 2][64];
    const int tiles = p.I >> 4;
    const int slot = blockIdx.x / tiles, n0 = (blockIdx.x - slot * tiles) * 16;
    const int e = slot_expert(p, by_pair, slot);
    if (e < 0)
        return;
    if (threadIdx.x < 64) {
        const int n = list_pairs(p, e, threadIdx.x, list);
        if (threadIdx.x == 0)
            count = n;
    }
    __syncthreads();
    const int np = __builtin_amdgcn_readfirstlane(count);
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

// LDS writes of all waves before, LDS reads after. Loads in flight stay in
// flight, which __syncthreads would wait for.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Pairs base .. base + 8 NT of expert e's list against this wave's 16 rows
// of W2: part[pair][row] = weight * product.
//
// All waves read the same h, so it goes through LDS in chunks of KC blocks
// of K, two buffers deep: the chunk after the present one is loaded to
// registers before the present one's products and stored after them. Read
// from L2 by each wave, h took four loads beside the two of a block's weights,
// and the load path became the bound: a copy of such a form without the h
// loads ran 74 instead of 104 us (8 tokens, 8 of 32 experts). A chunk's 16-byte units lie
// [block][tile][unit][column], the column exchanged by the unit's number so
// that neither the stores (a row's units) nor the reads (a unit's columns)
// meet in a bank. Column c of a tile is the hi (c < 8) or lo part of pair c % 8.
template <int NT, int KC>
__device__ __forceinline__ void down_tiles(const LayerParams &p, int e, int n0, const uint16_t *list, int base, int np,
                                           u32x4 *lds)
{
    constexpr int kUnits = KC * NT * 256;             // of 16 bytes, in one buffer
    constexpr int kMine = kUnits / kDownThreads;
    static_assert(kUnits % kDownThreads == 0, "");
    const int tid = threadIdx.x, lane = tid & 63, lg = lane >> 4, col = lane & 15;
    const int nkb = p.I >> 7, nch = (nkb + KC - 1) / KC;
    const int turn = (int)(blockIdx.x % nch);
    const uint8_t *w = p.W2 + e * p.w2_e + n0 * p.ld2;
    const uint32_t row0 = block_offset(lane, p.ld2), row8 = row0 + 8 * (uint32_t)p.ld2;
    const float *sw = p.s2 + e * p.s2_e + (n0 >> 7) * p.s2_nb;
    const uint8_t *h = (const uint8_t *)p.h;
    // This thread's units: n = 0, 1, ... are kRowStep rows (of columns) apart, unit and block are the same.
    constexpr int kRowStep = kDownThreads / (KC * 16);
    const int unit = tid % 16, hd = tid / 16 % KC, hrow = tid / (KC * 16);
    uint32_t ho[kMine];
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
        const int row = hrow + n * kRowStep, c = row % 16;
        const int pair = list[min(base + row / 16 * 8 + (c & 7), np - 1)];
        ho[n] = (uint32_t)(((c >> 3) * p.T * p.top_k + pair) * p.I * 2 + 16 * unit);
    }
    v4f acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        acc[i] = v4f{0.f, 0.f, 0.f, 0.f};

    u32x4 st[KC][2], hs[kMine];
    float sc[KC];
    // first block of the c-th chunk of this workgroup's order
    auto chunk = [&](int c) {
        c = min(c, nch - 1) + turn;
        return (c >= nch ? c - nch : c) * KC;
    };
    auto load_w = [&](int d, int kb0) {
        const int kb = min(kb0 + d, nkb - 1);
        st[d][0] = load16_once(w + (int64_t)kb * 128, row0);
        st[d][1] = load16_once(w + (int64_t)kb * 128, row8);
        sc[d] = sw[kb * p.s2_kb];
    };
    auto load_h = [&](int kb0) {
#pragma unroll
        for (int n = 0; n < kMine; ++n)
            hs[n] = load16(h, ho[n] + (uint32_t)min(kb0 + hd, nkb - 1) * 256);
    };
    auto store_h = [&](u32x4 *to) {
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
            const int row = hrow + n * kRowStep;
            to[((hd * NT + row / 16) * 16 + unit) * 16 + (row % 16 ^ unit)] = hs[n];
        }
    };
    load_h(chunk(0));
#pragma unroll
    for (int d = 0; d < KC; ++d)
        load_w(d, chunk(0));
    lds_barrier();  // the previous pass's reads
    store_h(lds);
    lds_barrier();
    for (int c = 0; c < nch; ++c) {
        const u32x4 *from = lds + (c & 1) * kUnits;
        const int kb0 = chunk(c), next = chunk(c + 1);
        load_h(next);
#pragma unroll
        for (int d = 0; d < KC; ++d) {
            if (kb0 + d < nkb) {
                exchange_halves(st[d][0], st[d][1]);
                bf16x8 wr[4];
                to_bf16(st[d][0], wr);
                to_bf16(st[d][1], wr + 2);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    v4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int u = 4 * lg + q;
                        const u32x4 b = from[((d * NT + i) * 16 + u) * 16 + (col ^ u)];
                        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wr[q], __builtin_bit_cast(bf16x8, b), part, 0,
                                                                       0, 0);
                    }
                    acc[i] += part * sc[d];
                }
            }
            if (c + 1 < nch)
                load_w(d, next);
        }
        store_h(lds + ((c + 1) & 1) * kUnits);
        lds_barrier();
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        v4f sum;
        const int at = base + 8 * i + col;
        const bool mine = col < 8 && at < np;
        const int pair = list[min(at, np - 1)];
        const float weight = p.weights[pair];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            sum[c] = (acc[i][c] + from_lane_xor_8(acc[i][c])) * weight;
        if (mine)
            *(v4f *)(p.part + (int64_t)pair * p.H + n0 + 4 * lg) = sum;
    }
}

// One workgroup per 128 columns of out and expert, 16 columns a wave: 448
// workgroups of 8 waves for one token, 8 experts and H = 7168, two a CU (so at
// most 128 registers). Every pair's product goes to the workspace: fp32, 4 H
// bytes a pair, little beside an expert's weights. One workgroup per 16 columns
// that went through all experts needed no sum after it, but the layer took 74
// instead of 67 us for one token and 481 instead of 345 for 64.
template <int NT>
__global__ __launch_bounds__(kDownThreads, 4) void down_kernel(LayerParams p, int by_pair)
{
    __shared__ u32x4 lds[NT >= 4 ? 4096 : 2048];  // two buffers of the widest pass
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int blocks = p.H / kDownRows;
    const int slot = blockIdx.x / blocks, n0 = (blockIdx.x - slot * blocks) * kDownRows + 16 * wave;
    const int e = slot_expert(p, by_pair, slot);
    if (e < 0)
        return;
    if (tid < 64) {
        const int n = list_pairs(p, e, tid, list);
        if (tid == 0)
            count = n;
    }
    __syncthreads();
    const int np = __builtin_amdgcn_readfirstlane(count);
    if (np == 0 || (by_pair && list[0] != slot))
        return;
    int base = 0;
    if (NT >= 4) {
        for (; np - base > 24; base += 32)
            down_tiles<4, 2>(p, e, n0, list, base, np, lds);
        for (; np - base > 16; base += 24)
            down_tiles<3, 2>(p, e, n0, list, base, np, lds);
    }
    if (NT >= 2)
        for (; np - base > 8; base += 16)
            down_tiles<2, 2>(p, e, n0, list, base, np, lds);
    for (; base < np; base += 8)
        down_tiles<1, 4>(p, e, n0, list, base, np, lds);
}

// ---------------------------------------------------------------- sum over a token's slots

// Four columns of out a thread, the slots' products added in their order. A
// slot without an expert has no product: what its place holds is not used.
constexpr int kSumThreads = 256;

__global__ __launch_bounds__(kSumThreads) void sum_slots_kernel(LayerParams p)
{
    const int t = blockIdx.y, at = (blockIdx.x * kSumThreads + threadIdx.x) * 4;
    if (at >= p.H)
        return;
    const float *part = p.part + (int64_t)t * p.top_k * p.H + at;
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < p.top_k; j0 += 4) {
        v4f v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = *(const v4f *)(part + (int64_t)min(j0 + j, p.top_k - 1) * p.H);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int id = p.ids[t * p.top_k + min(j0 + j, p.top_k - 1)];
            if (j0 + j < p.top_k && id >= 0 && id < p.E)
                sum += v[j];
        }
    }
    const uint2 packed = dgk::pack_bf16x4(sum);
    *(u32x2 *)(p.out + t * p.ldo + at) = u32x2{packed.x, packed.y};
}

}  // namespace dge
