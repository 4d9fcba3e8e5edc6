// Linear layer on MXFP4 weights with a fused epilogue:
//   y = bf16( act(x . dequant(W)^T + bias) + residual ).
#include "linear_epilogue.cuh"

namespace mx {

namespace {

using namespace linear;

constexpr int kTM = 64, kTN = 64;   // tokens and output features per CTA

// One 64 x 64 tile of outputs per CTA, a 32-element weight block of K at a time.
template <bool kGated>
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a) {
    constexpr int NW = kGated ? 2 : 1;
    __shared__ float xs[32][kTM + 1], ws[NW][32][kTN + 1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTM, n0 = static_cast<int64_t>(blockIdx.x) * kTN;
    const int tid = threadIdx.x, tm = tid / 16, tn = tid % 16;
    float acc[NW][4][4] = {};
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
    for (int64_t k0 = 0; k0 < a.K; k0 += 32) {
        for (int i = tid; i < kTM * 32; i += 256) {
            const int r = i / 32, k = i % 32;
            xs[k][r] = m0 + r < a.M ? __bfloat162float(x[(m0 + r) * a.K + k0 + k]) : 0.f;
        }
        for (int i = tid; i < NW * kTN * 16; i += 256) {
            const int h = i / (kTN * 16), r = i / 16 % kTN, b = i % 16;
            const int64_t n = n0 + r;
            float lo = 0.f, hi = 0.f;
            if (n < a.n_out) {
                const int64_t row = n + h * a.n_out;
                const uint32_t byte = a.codes[row * (a.K / 2) + k0 / 2 + b];
                const float s = e8m0_f32(a.scales[row * (a.K / 32) + k0 / 32]);
                lo = e2m1_f32(byte & 15u) * s;
                hi = e2m1_f32(byte >> 4) * s;
            }
            ws[h][2 * b][r] = lo;
            ws[h][2 * b + 1][r] = hi;
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
#pragma unroll
            for (int h = 0; h < NW; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[h][i][j] += xs[k][tm * 4 + i] * ws[h][k][tn + 16 * j];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + tm * 4 + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tn + 16 * j;
            if (m < a.M && n < a.n_out) {
                float v = activate(a.act, acc[0][i][j] + bias_at(a, n),
                                   kGated ? acc[NW - 1][i][j] + bias_at(a, n + a.n_out) : 0.f);
                const int64_t at = m * a.n_out + n;
                if (a.residual) v += __bfloat162float(static_cast<const __nv_bfloat16*>(a.residual)[at]);
                static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
            }
        }
    }
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.n_out + kTN - 1) / kTN), static_cast<unsigned>((a.M + kTM - 1) / kTM));
    if (a.act == MXFP4_ACT_SWIGLU) linear_kernel<true><<<grid, 256, 0, stream>>>(a);
    else linear_kernel<false><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace mx
