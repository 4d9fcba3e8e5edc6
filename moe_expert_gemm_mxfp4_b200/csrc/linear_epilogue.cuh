// The epilogue of the linear layer, shared by its engines: bias, activation, residual and the
// one rounding to bf16, in fp32.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace mx {
namespace linear {

// z / (1 + e^-v) by h = e^(-|v| / 2), which stays a normal number wherever the result is one in fp32: z h^2 / (1 + h^2)
// for negative v (e^-v itself passes a reciprocal's range at 2^126, and the result would be 0 from
// v = -87.3 on, where SiLU is -5e-37).  The rounded argument and the hardware's 2^x leave h off by less than
// (|v| + 5) 2^-24 of itself, so the result by twice that and some 2^-21: below 2^-15 where it is not 0.
__device__ __forceinline__ float over_one_plus_exp(float z, float v) {
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(-0.72134752044448170f * fabsf(v)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + h * h));
    return (v < 0.f ? z * h * h : z) * r;
}

// z -> act(z) for four outputs in fp32 (u: the gated activation's second factors).  One copy of
// this code per kernel and one switch per four outputs: inlined at every element, the
// activations fill the instruction cache, and a launch this short meets its code cold.
static __device__ __noinline__ float4 activate4(int act, float4 z, float4 u) {
    float v[4] = {z.x, z.y, z.z, z.w};
    switch (act) {
        case MXFP4_ACT_RELU:
#pragma unroll
            for (float& x : v) x = x < 0.f ? 0.f : x;   // keeps NaN
            break;
        case MXFP4_ACT_GELU:   // erfc: 1 + erf without cancellation
#pragma unroll
            for (float& x : v) x = 0.5f * x * erfcf(-0.70710678118654752f * x);
            break;
        case MXFP4_ACT_GELU_TANH:   // 0.5 (1 + tanh(v)) = 1 / (1 + e^(-2 v))
#pragma unroll
            for (float& x : v) x = over_one_plus_exp(x, 1.5957691216057308f * (x + 0.044715f * x * x * x));
            break;
        default:   // SILU, and SWIGLU's first factor
#pragma unroll
            for (float& x : v) x = over_one_plus_exp(x, x);
    }
    if (act == MXFP4_ACT_SWIGLU) v[0] *= u.x, v[1] *= u.y, v[2] *= u.z, v[3] *= u.w;
    return make_float4(v[0], v[1], v[2], v[3]);
}

// mbar_wait_spin that polls a while before it first reads the clock: the read takes longer than the
// waits that end soon.  Bounded the same way.
__device__ __forceinline__ bool wait_poll(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_test_wait(bar, parity)) return true;
    return mbar_wait_spin(bar, parity, abort);
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
