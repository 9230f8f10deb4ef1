// mfma.hpp -- device pieces shared by the product kernels: the e4m3 MFMA of
// one 128-wide K block and the rounding to bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dgk {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// One e4m3 x e4m3 -> fp32 MFMA over a 16x16x128 block, C = 0 + A.B.
// Format selectors 0/0 = OCP e4m3 for both operands; zero scale operands make
// the compiler emit the plain (unscaled) v_mfma_f32_16x16x128_f8f6f4.
__device__ __forceinline__ v4f mfma_e4m3_16x16x128(const v8i &a, const v8i &b)
{
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// fp32 -> bf16 bits, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_rne(float f)
{
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return 0x7fc0u;
    u += 0x7fffu + ((u >> 16) & 1u);
    return u >> 16;
}

__device__ __forceinline__ uint2 pack_bf16x4(const v4f &v)
{
    uint2 r;
    r.x = bf16_rne(v[0]) | (bf16_rne(v[1]) << 16);
    r.y = bf16_rne(v[2]) | (bf16_rne(v[3]) << 16);
    return r;
}

}  // namespace dgk
