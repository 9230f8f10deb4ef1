// gate.hpp -- gfx950 kernel of a mixture-of-experts router's choice: for each
// token the k largest of its E logits, and their weights.
//
//   ids[t, j]     the expert of the j-th largest logit; equal logits go to the lower expert first
//   softmax:      w_j = exp(l_j - l_0) / sum, over the chosen (renormalised) or over all E
//   sigmoid:      w_j = 1 / (1 + exp(-l_j)), divided by their sum when renormalised
//   weights[t, j] factor * w_j
// A NaN or -inf logit is no candidate and has no share in a sum; a slot with no
// candidate left gets id -1 and weight 0.
//
// The selection is top_k rounds of a maximum and the lowest index that holds
// it, on the logits themselves: no key is built, so equal logits are equal. 16
// lanes take a token (four tokens a wave), which keeps every reduction inside a
// DPP row, four steps and no LDS; a lane holds E / 16 logits in registers. The
// logits are read once, but the vector instructions of the rounds bound it, not
// HBM: 8192 tokens x 256 experts, 8 chosen, fp32: 6.8 us with the softmax over
// all (8.9 MB, 1.3 TB/s), 6.0 us over the chosen; 64 experts 4.1 us, 512
// experts 10.6 us; one token of 32 experts 3.2 us, a launch (graph replays over
// three inputs in turn; 6.2 us instead of 6.8 where the calls are eager, one
// after the other).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "norm.hpp"

namespace dgg {

using dgn::sum_over_16_lanes;
using dgq::dpp;

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;    // one lane of a token's 16 holds one slot
constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 16;

struct GateParams {
    const void *logits;  // fp32 or bf16 [T, E]
    int64_t ldl;
    int32_t *ids;        // [T, top_k]
    float *weights;      // [T, top_k]
    int64_t T;
    int E, top_k;
    int sigmoid, renormalize;
    float factor;
};

__device__ __forceinline__ float max_over_16_lanes(float v)
{
    v = fmaxf(v, __uint_as_float(dpp<0xB1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<0x4E>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<0x141>(__float_as_uint(v))));
    return fmaxf(v, __uint_as_float(dpp<0x140>(__float_as_uint(v))));
}

__device__ __forceinline__ int min_over_16_lanes(int v)
{
    v = min(v, (int)dpp<0xB1>((uint32_t)v));
    v = min(v, (int)dpp<0x4E>((uint32_t)v));
    v = min(v, (int)dpp<0x141>((uint32_t)v));
    return min(v, (int)dpp<0x140>((uint32_t)v));
}

// 16 lanes per token; lane i holds experts i, i + 16, ..., NV of them.
template <bool BF16, int NV>
__global__ __launch_bounds__(kThreads) void gate_topk_kernel(GateParams p)
{
    const int lane = threadIdx.x & 15;
    const int64_t token = (int64_t)blockIdx.x * kTokens + threadIdx.x / 16;
    if (token >= p.T)
        return;
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 16 * i + lane;
        const int64_t at = token * p.ldl + min(e, p.E - 1);
        const float l = BF16 ? dgq::bf16_to_f32(((const uint16_t *)p.logits)[at]) : ((const float *)p.logits)[at];
        // false for NaN: it becomes -inf
        v[i] = e < p.E && l > -INFINITY ? l : -INFINITY;
    }
    float all = 0.0f;   // softmax over all experts: the sum of exp(l - largest)
    float mine = -INFINITY;
    int id = -1;
    float largest = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
        float best = v[0];
#pragma unroll
        for (int i = 1; i < NV; ++i)
            best = fmaxf(best, v[i]);
        best = max_over_16_lanes(best);
        if (best == -INFINITY)
            break;
        if (j == 0) {
            largest = best;
            if (!p.sigmoid && !p.renormalize) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    all += expf(v[i] - largest);
                all = sum_over_16_lanes(all);
            }
        }
        // the lowest expert that holds it
        int e = 0x7fffffff;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
            e = v[i] == best ? 16 * i + lane : e;
        e = min_over_16_lanes(e);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = e == 16 * i + lane ? -INFINITY : v[i];
        if (lane == j) {
            mine = best;
            id = e;
        }
    }
    float w = 0.0f;
    if (p.sigmoid) {
        // Renormalised weights are ratios, so that all of them may be scaled
        // by exp(-largest) where the sigmoids themselves would underflow.
        const float shift = p.renormalize ? fminf(largest, 0.0f) : 0.0f;
        if (id >= 0)
            w = mine > 0.0f ? 1.0f / (1.0f + expf(-mine)) : expf(mine - shift) / (1.0f + expf(mine));
    } else if (id >= 0) {
        w = expf(mine - largest);
    }
    if (p.renormalize)
        all = sum_over_16_lanes(w);
    if (id >= 0 && (p.renormalize || !p.sigmoid))
        w /= all;
    if (lane < p.top_k) {
        p.ids[token * p.top_k + lane] = id;
        p.weights[token * p.top_k + lane] = w * p.factor;
    }
}

}  // namespace dgg
