// norm.hpp -- gfx950 kernel of the residual addition and root-mean-square norm
// whose output is the products' LHS: e4m3 codes with one scale per 1x128 block.
//
// Per row m of K elements, in fp32 from the loads to the last store:
//   h = x + r                               (h = x without a residual)
//   R_out = h, rounded once to its type     (the residual stream of the next layer)
//   y = h * (1 / sqrt(mean(h^2) + eps)) * w
//   Y = y, rounded once to bf16             (what a router reads; optional)
//   s = max|y| over the block / 448, or 1 for a block of zeros
//   q = the e4m3 code nearest to y / s, as quant.hpp computes it
// The norm is taken of the unrounded h.
//
// HBM bounds it for many rows: x, r and w are read once, the row stays in
// registers between the sum and the output, and what is written is written in
// 16-byte stores (codes: 8). 8192 x 7168, bf16 in, residual and normed rows:
// 105.5 us for 530 MB, 5.03 TB/s, the rate of a 2 GiB copy (4.93 TB/s); 2048
// rows 29.7 us (graph replays over three inputs in turn). One row: 4.8 us, a
// launch and the latency of two dependent reads. 16 lanes hold a 1x128 block
// (8 elements each), so the block's amax and the row's sum are DPP steps, and
// the rows are dealt to the XCDs in contiguous ranges, as the quantiser's are,
// for the M-major scales' lines.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "quant.hpp"

namespace dgn {

using dgq::dpp;
using dgq::f32x4;
using dgq::u32x2;
using dgq::u32x4;

struct NormParams {
    const void *X;      // fp32 or bf16 [M, K]
    int64_t ldx;
    const void *R;      // fp32 or bf16 [M, K], or NULL
    int64_t ldr;
    void *R_out;        // the type of R
    int64_t ldro;
    const void *W;      // fp32 or bf16 [K]
    int w_bf16;
    float eps;
    uint16_t *Y;        // bf16 [M, K], or NULL
    int64_t ldy;
    uint8_t *Q;
    int64_t ldq;
    float *S;
    int64_t s_m, s_kb;
    int M, K;
};

enum Residual { kNoResidual = 0, kResidualBf16 = 1, kResidualF32 = 2 };

// Sum over each row of 16 lanes, the same in all of them (quad permutes, half
// mirror, mirror): a fixed tree.
__device__ __forceinline__ float sum_over_16_lanes(float v)
{
    v += __uint_as_float(dpp<0xB1>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x4E>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x141>(__float_as_uint(v)));
    return v + __uint_as_float(dpp<0x140>(__float_as_uint(v)));
}

__device__ __forceinline__ uint32_t max_over_16_lanes(uint32_t v)
{
    v = dgq::max_over_8_lanes(v);
    return max(v, dpp<0x140>(v));
}

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

// Two fp32 values rounded to bf16 (round to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// Eight consecutive elements from 16-byte aligned memory.
template <bool BF16>
__device__ __forceinline__ void load8(const void *base, int64_t index, float *v)
{
    if (BF16) {
        const u32x4 w = *(const u32x4 *)((const uint16_t *)base + index);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[2 * c] = dgq::bf16_to_f32(w[c] & 0xffffu);
            v[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
        }
    } else {
        const f32x4 a = *(const f32x4 *)((const float *)base + index);
        const f32x4 b = *(const f32x4 *)((const float *)base + index + 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[c] = a[c];
            v[4 + c] = b[c];
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t index, const float *v)
{
    if (BF16) {
        *(u32x4 *)((uint16_t *)base + index) =
            u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    } else {
        *(f32x4 *)((float *)base + index) = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4 *)((float *)base + index + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
}

// ROW threads per row (64, four rows a workgroup, or the whole workgroup), NC
// chunks of 8 elements a thread: a row of up to 8 * ROW * NC elements stays in registers between the
// two passes over it, so HBM is read once.
template <bool XBF16, int RES, int ROW, int NC>
__global__ __launch_bounds__(ROW < 256 ? 256 : ROW) void rmsnorm_quantize_kernel(NormParams p)
{
    constexpr int kThreads = ROW < 256 ? 256 : ROW;
    constexpr int kRows = kThreads / ROW;       // rows per workgroup
    constexpr int kWaves = ROW / 64;            // waves per row
    __shared__ float part[kWaves];
    const int t = threadIdx.x % ROW;
    const int nwg = gridDim.x, xcd = blockIdx.x % 8, per = nwg / 8, extra = nwg % 8;
    const int wg = xcd * per + min(xcd, extra) + (int)blockIdx.x / 8;
    const int row = __builtin_amdgcn_readfirstlane(wg * kRows + (int)threadIdx.x / ROW);
    if (row >= p.M)
        return;
    const int chunks = p.K / 8;

    float h[NC][8];
    float r[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t at = 8 * (int64_t)min(i * ROW + t, chunks - 1);
        load8<XBF16>(p.X, row * p.ldx + at, h[i]);
        if (RES != kNoResidual)
            load8<RES == kResidualBf16>(p.R, row * p.ldr + at, r[i]);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int chunk = i * ROW + t;
        if (RES != kNoResidual) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                h[i][c] += r[i][c];
            if (chunk < chunks)
                store8<RES == kResidualBf16>(p.R_out, row * p.ldro + 8 * (int64_t)chunk, h[i]);
        }
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            s = __builtin_fmaf(h[i][c], h[i][c], s);
        sum += chunk < chunks ? s : 0.0f;
    }
    sum = sum_over_16_lanes(sum);
    sum = (lane_value(sum, 0) + lane_value(sum, 16)) + (lane_value(sum, 32) + lane_value(sum, 48));
    if (kWaves > 1) {
        part[threadIdx.x / 64] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            sum += part[w];
    }
    const float inv = 1.0f / sqrtf(sum / (float)p.K + p.eps);

#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int chunk = i * ROW + t;
        if (chunk >= chunks)  // the same for all 16 lanes of a block
            continue;
        const int64_t at = 8 * (int64_t)chunk;
        float w[8];
        if (p.w_bf16)
            load8<true>(p.W, at, w);
        else
            load8<false>(p.W, at, w);
        uint32_t abits = 0;
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            y[c] = h[i][c] * inv * w[c];
            abits = max(abits, __float_as_uint(y[c]) & 0x7fffffffu);
        }
        if (p.Y)
            store8<true>(p.Y, row * p.ldy + at, y);
        const float amax = __uint_as_float(max_over_16_lanes(abits));
        const float s = amax == 0.0f ? 1.0f : amax / dgq::kE4m3Max;
        float q[8];
        if (s >= 0x1p-64f) {
            const float rc = 1.0f / s;
            const float rc_lo = __builtin_fmaf(-s, rc, 1.0f) * rc;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                q[c] = dgq::quotient(y[c], s, rc, rc_lo);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                q[c] = y[c] / s;
        }
        uint32_t code[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = fminf(fmaxf(q[4 * half + c], -dgq::kE4m3Max), dgq::kE4m3Max);
            const int low = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            code[half] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], low, true);
        }
        *(u32x2 *)(p.Q + row * p.ldq + at) = u32x2{code[0], code[1]};
        if (t % 16 == 0)
            p.S[row * p.s_m + (int64_t)(chunk / 16) * p.s_kb] = s;
    }
}

}  // namespace dgn
