// The epilogue of the linear layer, shared by its engines: bias, activation, residual and the
// one rounding to bf16, in fp32.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace mx {
namespace linear {

// z / (1 + e^-v): the hardware's exponential and quotient are off by less than 2^-17 of the
// result here, far below bf16's half step.
__device__ __forceinline__ float over_one_plus_exp(float z, float v) { return __fdividef(z, 1.f + __expf(-v)); }

// The activation of one output in fp32 (u: the gated activation's second factor).
__device__ __forceinline__ float activate(int act, float z, float u) {
    switch (act) {
        case MXFP4_ACT_RELU: return z < 0.f ? 0.f : z;   // keeps NaN
        case MXFP4_ACT_SILU: return over_one_plus_exp(z, z);
        case MXFP4_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);   // 1 + erf without cancellation
        case MXFP4_ACT_GELU_TANH:   // 0.5 (1 + tanh(v)) = 1 / (1 + e^(-2 v))
            return over_one_plus_exp(z, 1.5957691216057308f * (z + 0.044715f * z * z * z));
        case MXFP4_ACT_SWIGLU: return over_one_plus_exp(z, z) * u;
        default: return z;
    }
}

// Four outputs.  One copy of this code per kernel: inlined at every element, the activations fill
// the instruction cache, and a launch this short meets its code cold.
static __device__ __noinline__ float4 activate4(int act, float4 z, float4 u) {
    return make_float4(activate(act, z.x, u.x), activate(act, z.y, u.y), activate(act, z.z, u.z), activate(act, z.w, u.w));
}

__device__ __forceinline__ float bias_at(const LinearArgs& a, int64_t n) {
    if (!a.bias) return 0.f;
    return a.bias_f32 ? static_cast<const float*>(a.bias)[n]
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[n]);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace linear
}  // namespace mx
