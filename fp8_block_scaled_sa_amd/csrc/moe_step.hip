// moe_step.hip -- C ABI of the operators around the experts of a
// mixture-of-experts serving step (declared in include/dg_fp8.h): the residual
// norm to codes, the router's choice and the expert layer for a few tokens.
// Host-side validation, kernel choice and launch; nothing is allocated and no
// stream is synchronised. Compiled behind dg_fp8.hip (library.hip), whose
// device check, argument checks and error record it shares.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <stdint.h>

#include "dg_fp8.h"
#include "experts.hpp"
#include "gate.hpp"
#include "norm.hpp"

namespace {

// Strides up to this keep every byte offset below 2^62 (sizes are int32).
constexpr int64_t kMaxStride = (int64_t)1 << 28;

bool strides_fit(std::initializer_list<int64_t> strides)
{
    for (int64_t s : strides)
        if (s > kMaxStride)
            return false;
    return true;
}

// A launch takes fewer than 2^32 threads in all.
bool threads_fit(int64_t workgroups, int64_t threads) { return workgroups * threads < ((int64_t)1 << 32); }

int launched()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? DG_OK : fail_hip(e);
}

bool is_float_type(int t) { return t == DG_DTYPE_F32 || t == DG_DTYPE_BF16; }

// ---------------------------------------------------------------- norm

// Threads that a row takes (see launch_norm).
int64_t norm_row_threads(int64_t K) { return K <= 1024 ? 64 : K <= 8192 ? 256 : 1024; }

// Row layouts of the norm kernel: ROW threads per row, NC chunks of 8 a thread.
// Short rows share a workgroup; past 1024 elements a row has one to itself, of
// 256 threads while 4 chunks a thread hold it, then of 1024. A layout holds up
// to twice, the first of 1024 threads up to four times the row that it is used
// for; the loads past a row's end repeat its last chunk, which the cache holds.
// bf16, residual and normed rows: 8192 x 1024 runs at 5.2 TB/s, x 4096 at 5.3,
// x 5120 and x 7168 at 5.0, x 8192 at 4.4, x 8320 at 4.6, x 12288 at 5.2, x
// 16384 at 5.4, 4096 x 32768 and 2048 x 65536 at 4.9.
template <bool XBF16, int RES>
int launch_norm(const dgn::NormParams &p, hipStream_t stream)
{
#define DG_NORM(ROW, NC)                                                                                              \
    hipLaunchKernelGGL((dgn::rmsnorm_quantize_kernel<XBF16, RES, ROW, NC>),                                           \
                       dim3((unsigned)((p.M + (ROW < 256 ? 256 / ROW : 1) - 1) / (ROW < 256 ? 256 / ROW : 1))),       \
                       dim3(ROW < 256 ? 256 : ROW), 0, stream, p)
    const int chunks = p.K / 8;
    if (chunks <= 64)
        DG_NORM(64, 1);
    else if (chunks <= 128)
        DG_NORM(64, 2);
    else if (chunks <= 256)
        DG_NORM(256, 1);
    else if (chunks <= 512)
        DG_NORM(256, 2);
    else if (chunks <= 1024)
        DG_NORM(256, 4);
    else if (chunks <= 4096)
        DG_NORM(1024, 4);
    else
        DG_NORM(1024, 8);
#undef DG_NORM
    return launched();
}

constexpr int64_t kNormMaxK = 65536;

// ---------------------------------------------------------------- gate

template <bool BF16>
int launch_gate(const dgg::GateParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.T + dgg::kTokens - 1) / dgg::kTokens)), block(dgg::kThreads);
#define DG_GATE(NV) hipLaunchKernelGGL((dgg::gate_topk_kernel<BF16, NV>), grid, block, 0, stream, p)
    if (p.E <= 16)
        DG_GATE(1);
    else if (p.E <= 32)
        DG_GATE(2);
    else if (p.E <= 64)
        DG_GATE(4);
    else if (p.E <= 128)
        DG_GATE(8);
    else if (p.E <= 256)
        DG_GATE(16);
    else if (p.E <= 512)
        DG_GATE(32);
    else
        DG_GATE(64);
#undef DG_GATE
    return launched();
}

// ---------------------------------------------------------------- layer

int check_layer_sizes(int64_t T, int64_t top_k, int64_t E, int64_t H, int64_t I)
{
    if (T < 0 || top_k <= 0 || E <= 0 || H <= 0 || I <= 0 || H % 128 || I % 128)
        return DG_ERR_BAD_SHAPE;
    if (T > dge::kMaxTokens || top_k > dge::kMaxTopK || E > dge::kMaxExperts ||
        H > dge::kMaxWidth || I > dge::kMaxWidth)
        return DG_ERR_UNSUPPORTED;
    return DG_OK;
}

// Both bf16 parts of h, and the pairs' products.
int64_t layer_bytes(int64_t T, int64_t top_k, int64_t H, int64_t I) { return T * top_k * (4 * I + 4 * H); }

// Grid slots are pairs or experts, whichever are fewer. The kernels' tiles of
// tokens follow T, the most tokens an expert can have (a token that names an
// expert twice only makes it take another pass): fewer tiles, fewer registers,
// more waves (gate_up: 98 registers for 16 tokens, 130 for 32, 140 for 64). For
// 64 tokens gate_up keeps one block of K in flight: two (208 registers) took
// 220 instead of 215 us at 16 tokens an expert and 28 instead of 26 on a share
// of the experts, but 89 instead of 99 where every expert has 64. The down
// kernel with tiles of 16 pairs for T of 64 (top-1, 4 experts) read W2 four
// times: the layer took 70.6 instead of 58.5 us.
int launch_layer(const dge::LayerParams &p, hipStream_t stream)
{
    const int pairs = p.T * p.top_k;
    const int by_pair = pairs < p.E;
    const dim3 grid((unsigned)((by_pair ? pairs : p.E) * (p.I / 16))), block(dge::kUpThreads);
    if (p.T <= 16)
        hipLaunchKernelGGL((dge::gate_up_kernel<1, 2>), grid, block, 0, stream, p, by_pair);
    else if (p.T <= 32)
        hipLaunchKernelGGL((dge::gate_up_kernel<2, 2>), grid, block, 0, stream, p, by_pair);
    else
        hipLaunchKernelGGL((dge::gate_up_kernel<4, 1>), grid, block, 0, stream, p, by_pair);
    int st = launched();
    if (st != DG_OK)
        return st;
    const dim3 dgrid((unsigned)((by_pair ? pairs : p.E) * (p.H / dge::kDownRows))), threads(dge::kDownThreads);
    if (p.T <= 8)
        hipLaunchKernelGGL((dge::down_kernel<1>), dgrid, threads, 0, stream, p, by_pair);
    else if (p.T <= 16)
        hipLaunchKernelGGL((dge::down_kernel<2>), dgrid, threads, 0, stream, p, by_pair);
    else
        hipLaunchKernelGGL((dge::down_kernel<4>), dgrid, threads, 0, stream, p, by_pair);
    if ((st = launched()) != DG_OK)
        return st;
    hipLaunchKernelGGL(dge::sum_slots_kernel, dim3((p.H / 4 + dge::kSumThreads - 1) / dge::kSumThreads, p.T),
                       dim3(dge::kSumThreads), 0, stream, p);
    return launched();
}

}  // namespace

extern "C" {

dg_status dg_fp8_rmsnorm_quantize_1x128(const void *X, int x_dtype, int64_t ldx, const void *R, int r_dtype,
                                        int64_t ldr, void *R_out, int64_t ldro, const void *W, int w_dtype,
                                        float eps, void *Y, int64_t ldy, void *Q, int64_t ldq, float *S,
                                        int64_t s_stride_m, int64_t s_stride_kb, int64_t M, int64_t K, void *stream)
{
    if (M < 0 || K <= 0 || K % 128 || !(eps >= 0.0f))
        return DG_ERR_BAD_SHAPE;
    if (!is_float_type(x_dtype) || (R && !is_float_type(r_dtype)) || !is_float_type(w_dtype) || M > kInt32Max ||
        K > kNormMaxK)
        return DG_ERR_UNSUPPORTED;
    const int64_t row_threads = norm_row_threads(K), group = std::max<int64_t>(row_threads, 256);
    if (!threads_fit((M * row_threads + group - 1) / group, group))
        return DG_ERR_UNSUPPORTED;
    if (M == 0)
        return DG_OK;
    if (!X || !W || !Q || !S || (R && !R_out))
        return DG_ERR_NULL_POINTER;
    const int64_t nkb = K / 128;
    const int64_t xs = x_dtype == DG_DTYPE_BF16 ? 2 : 4, rs = r_dtype == DG_DTYPE_BF16 ? 2 : 4;
    const int64_t wsz = w_dtype == DG_DTYPE_BF16 ? 2 : 4;
    if (ldx < K || ldq < K || (R && (ldr < K || ldro < K)) || (Y && ldy < K) || s_stride_m < 0 || s_stride_kb < 0)
        return DG_ERR_BAD_STRIDE;
    // Every (m, kb) owns a distinct scale slot.
    const bool row_major = (M == 1 || s_stride_m >= nkb * std::max<int64_t>(s_stride_kb, 1)) &&
                           (nkb == 1 || s_stride_kb >= 1);
    const bool m_major = (nkb == 1 || s_stride_kb >= M * std::max<int64_t>(s_stride_m, 1)) &&
                         (M == 1 || s_stride_m >= 1);
    if (!row_major && !m_major)
        return DG_ERR_BAD_STRIDE;
    if (!strides_fit({ldx, ldq, s_stride_m, s_stride_kb}) || (R && !strides_fit({ldr, ldro})) ||
        (Y && !strides_fit({ldy})))
        return DG_ERR_UNSUPPORTED;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Q, 16) || !aligned(S, 4) || (ldx * xs) % 16 || ldq % 16 ||
        (R && (!aligned(R, 16) || !aligned(R_out, 16) || (ldr * rs) % 16 || (ldro * rs) % 16)) ||
        (Y && (!aligned(Y, 16) || ldy % 8)))
        return DG_ERR_MISALIGNED;
    const Extent ex = extent(X, xs, (M - 1) * ldx + K - 1), ew = extent(W, wsz, K - 1);
    const Extent none = {0, 0};
    const Extent er = R ? extent(R, rs, (M - 1) * ldr + K - 1) : none;
    const Extent outs[4] = {extent(Q, 1, (M - 1) * ldq + K - 1),
                            extent(S, 4, (M - 1) * s_stride_m + (nkb - 1) * s_stride_kb),
                            R ? extent(R_out, rs, (M - 1) * ldro + K - 1) : none,
                            Y ? extent(Y, 2, (M - 1) * ldy + K - 1) : none};
    // R_out may be R itself (each row is read before it is written).
    const bool in_place = R && R_out == R && ldro == ldr;
    for (int i = 0; i < 4; ++i) {
        if (overlaps(outs[i], ex) || overlaps(outs[i], ew) || (!(i == 2 && in_place) && overlaps(outs[i], er)))
            return DG_ERR_ALIASING;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outs[j]))
                return DG_ERR_ALIASING;
    }
    DeviceInfo dev;
    const int st = current_device(dev);
    if (st != DG_OK)
        return (dg_status)st;
    dgn::NormParams p = {};
    p.X = X; p.ldx = ldx; p.R = R; p.ldr = ldr; p.R_out = R_out; p.ldro = ldro;
    p.W = W; p.w_bf16 = w_dtype == DG_DTYPE_BF16; p.eps = eps;
    p.Y = (uint16_t *)Y; p.ldy = ldy; p.Q = (uint8_t *)Q; p.ldq = ldq;
    p.S = S; p.s_m = s_stride_m; p.s_kb = s_stride_kb;
    p.M = (int)M; p.K = (int)K;
    const hipStream_t s = (hipStream_t)stream;
    const bool xb = x_dtype == DG_DTYPE_BF16;
    if (!R)
        return (dg_status)(xb ? launch_norm<true, dgn::kNoResidual>(p, s) : launch_norm<false, dgn::kNoResidual>(p, s));
    if (r_dtype == DG_DTYPE_BF16)
        return (dg_status)(xb ? launch_norm<true, dgn::kResidualBf16>(p, s)
                              : launch_norm<false, dgn::kResidualBf16>(p, s));
    return (dg_status)(xb ? launch_norm<true, dgn::kResidualF32>(p, s) : launch_norm<false, dgn::kResidualF32>(p, s));
}

dg_status dg_moe_gate_topk(const void *logits, int l_dtype, int64_t ldl, int score, int renormalize, float factor,
                           int32_t *ids, float *weights, int64_t T, int64_t E, int64_t top_k, void *stream)
{
    if (T < 0 || E <= 0 || top_k <= 0 || top_k > E)
        return DG_ERR_BAD_SHAPE;
    if (!is_float_type(l_dtype) || (score != DG_GATE_SOFTMAX && score != DG_GATE_SIGMOID) || E > dgg::kMaxExperts ||
        top_k > dgg::kMaxTopK || T > kInt32Max ||
        !threads_fit((T + dgg::kTokens - 1) / dgg::kTokens, dgg::kThreads))
        return DG_ERR_UNSUPPORTED;
    if (T == 0)
        return DG_OK;
    if (!logits || !ids || !weights)
        return DG_ERR_NULL_POINTER;
    if (ldl < E)
        return DG_ERR_BAD_STRIDE;
    if (!strides_fit({ldl}))
        return DG_ERR_UNSUPPORTED;
    const int64_t size = l_dtype == DG_DTYPE_BF16 ? 2 : 4;
    if (!aligned(logits, size) || !aligned(ids, 4) || !aligned(weights, 4))
        return DG_ERR_MISALIGNED;
    const Extent el = extent(logits, size, (T - 1) * ldl + E - 1);
    const Extent ei = extent(ids, 4, T * top_k - 1), ew = extent(weights, 4, T * top_k - 1);
    if (overlaps(ei, el) || overlaps(ew, el) || overlaps(ei, ew))
        return DG_ERR_ALIASING;
    DeviceInfo dev;
    const int st = current_device(dev);
    if (st != DG_OK)
        return (dg_status)st;
    dgg::GateParams p = {};
    p.logits = logits; p.ldl = ldl; p.ids = ids; p.weights = weights;
    p.T = T; p.E = (int)E; p.top_k = (int)top_k;
    p.sigmoid = score == DG_GATE_SIGMOID; p.renormalize = renormalize != 0; p.factor = factor;
    return (dg_status)(l_dtype == DG_DTYPE_BF16 ? launch_gate<true>(p, (hipStream_t)stream)
                                                : launch_gate<false>(p, (hipStream_t)stream));
}

int64_t dg_fp8_moe_layer_workspace_bytes(int64_t T, int64_t top_k, int64_t H, int64_t I)
{
    const int st = check_layer_sizes(T, top_k, 1, H, I);
    return st == DG_OK ? layer_bytes(T, top_k, H, I) : -st;
}

dg_status dg_fp8_moe_layer(const void *X, int64_t ldx, const float *sX, int64_t sx_stride_m, int64_t sx_stride_kb,
                           const void *W13, int64_t ld13, int64_t w13_stride_e, const float *s13,
                           int64_t s13_stride_e, int64_t s13_stride_nb, int64_t s13_stride_kb, const void *W2,
                           int64_t ld2, int64_t w2_stride_e, const float *s2, int64_t s2_stride_e,
                           int64_t s2_stride_nb, int64_t s2_stride_kb, const int32_t *topk_ids,
                           const float *topk_weights, void *out, int64_t ldo, int64_t T, int64_t top_k, int64_t E,
                           int64_t H, int64_t I, void *workspace, int64_t workspace_bytes, void *stream)
{
    int st = check_layer_sizes(T, top_k, E, H, I);
    if (st != DG_OK)
        return (dg_status)st;
    if (!threads_fit(std::min(T * top_k, E) * (I / 16), dge::kUpThreads))
        return DG_ERR_UNSUPPORTED;
    if (T == 0)
        return DG_OK;
    if (!X || !sX || !W13 || !s13 || !W2 || !s2 || !topk_ids || !topk_weights || !out || !workspace)
        return DG_ERR_NULL_POINTER;
    if (ldx < H || ld13 < H || ld2 < I || ldo < H || sx_stride_m < 0 || sx_stride_kb < 0 || s13_stride_e < 0 ||
        s13_stride_nb < 0 || s13_stride_kb < 0 || s2_stride_e < 0 || s2_stride_nb < 0 || s2_stride_kb < 0)
        return DG_ERR_BAD_STRIDE;
    if (!strides_fit({sx_stride_kb, s13_stride_nb, s13_stride_kb, s2_stride_nb, s2_stride_kb}) ||
        std::max({ldx, ld13, ld2, ldo}) > dge::kMaxRowStride || sx_stride_m > dge::kMaxTokenScaleStride)
        return DG_ERR_UNSUPPORTED;
    const int64_t last13 = (2 * I - 1) * ld13 + H - 1, last2 = (H - 1) * ld2 + I - 1;
    const int64_t last_s13 = (2 * I / 128 - 1) * s13_stride_nb + (H / 128 - 1) * s13_stride_kb;
    const int64_t last_s2 = (H / 128 - 1) * s2_stride_nb + (I / 128 - 1) * s2_stride_kb;
    if (E > 1 && (w13_stride_e <= last13 || w2_stride_e <= last2))
        return DG_ERR_BAD_STRIDE;
    constexpr int64_t kMaxGroupStride = (int64_t)1 << 50;
    if (E > 1 && (w13_stride_e > kMaxGroupStride || w2_stride_e > kMaxGroupStride || s13_stride_e > kMaxGroupStride ||
                  s2_stride_e > kMaxGroupStride))
        return DG_ERR_UNSUPPORTED;
    if (!aligned(X, 16) || !aligned(W13, 16) || !aligned(W2, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(sX, 4) || !aligned(s13, 4) || !aligned(s2, 4) || !aligned(topk_ids, 4) ||
        !aligned(topk_weights, 4) || ldx % 16 || ld13 % 16 || ld2 % 16 || ldo % 8 ||
        (E > 1 && (w13_stride_e % 16 || w2_stride_e % 16)))
        return DG_ERR_MISALIGNED;
    if (workspace_bytes < layer_bytes(T, top_k, H, I))
        return DG_ERR_SCRATCH;
    const Extent ins[8] = {
        extent(X, 1, (T - 1) * ldx + H - 1),
        extent(sX, 4, (T - 1) * sx_stride_m + (H / 128 - 1) * sx_stride_kb),
        extent(W13, 1, (E - 1) * w13_stride_e + last13), extent(s13, 4, (E - 1) * s13_stride_e + last_s13),
        extent(W2, 1, (E - 1) * w2_stride_e + last2), extent(s2, 4, (E - 1) * s2_stride_e + last_s2),
        extent(topk_ids, 4, T * top_k - 1), extent(topk_weights, 4, T * top_k - 1)};
    const Extent eo = extent(out, 2, (T - 1) * ldo + H - 1), ews = extent(workspace, 1, workspace_bytes - 1);
    if (overlaps(eo, ews))
        return DG_ERR_ALIASING;
    for (const Extent &e : ins)
        if (overlaps(eo, e) || overlaps(ews, e))
            return DG_ERR_ALIASING;
    DeviceInfo dev;
    if ((st = current_device(dev)) != DG_OK)
        return (dg_status)st;
    dge::LayerParams p = {};
    p.X = (const uint8_t *)X; p.ldx = ldx; p.sX = sX; p.sx_m = sx_stride_m; p.sx_kb = sx_stride_kb;
    p.W13 = (const uint8_t *)W13; p.ld13 = ld13; p.w13_e = w13_stride_e;
    p.s13 = s13; p.s13_e = s13_stride_e; p.s13_nb = s13_stride_nb; p.s13_kb = s13_stride_kb;
    p.W2 = (const uint8_t *)W2; p.ld2 = ld2; p.w2_e = w2_stride_e;
    p.s2 = s2; p.s2_e = s2_stride_e; p.s2_nb = s2_stride_nb; p.s2_kb = s2_stride_kb;
    p.ids = topk_ids; p.weights = topk_weights; p.out = (uint16_t *)out; p.ldo = ldo;
    p.h = (uint16_t *)workspace;
    p.part = (float *)workspace + T * top_k * I;
    p.T = (int)T; p.top_k = (int)top_k; p.E = (int)E; p.H = (int)H; p.I = (int)I;
    return (dg_status)launch_layer(p, (hipStream_t)stream);
}

}  // extern "C"
