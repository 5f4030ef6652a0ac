// Products of 8-bit floating-point operands with block scales (fp8.cuh):
//   C[m, n] = sum_b sA[b, m] sW[b, n / 128] sum_{k in block b} a[m, k] w[n, k]
// with every block's inner sum and the outer sum in fp32.
#pragma once

#include "fp8.cuh"

namespace bnn {

// Operands of a (grouped) product.  Dense: offsets == nullptr, one group of R
// rows.  Grouped: rows offsets[e] .. offsets[e + 1] of A meet W[e].
struct Fp8Gemm {
    const uint8_t* A;
    int64_t lda;
    const float* sa;
    int64_t ldsa;
    const uint8_t* W;
    int64_t ldw, w_stride;
    const float* sw;
    int64_t ldsw, sw_stride;
    const int32_t* offsets;
    int R, E, N, K;
    void* out;
    int64_t ldo;
};

template <typename T>
__device__ __forceinline__ T fp8_out(float v);
template <>
__device__ __forceinline__ float fp8_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 fp8_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float fp8_value(uint8_t c) {
    __nv_fp8_e4m3 t;
    t.__x = c;
    return (float)t;
}

// 64 x 64 outputs per CTA, 4 x 4 per thread, operands decoded to fp32 in
// shared memory 32 columns of K at a time.
template <typename T>
__global__ void __launch_bounds__(256) fp8_gemm_simple_kernel(Fp8Gemm g) {
    constexpr int KC = 32;
    __shared__ float as[KC][64 + 4], ws[KC][64 + 4];
    const int e = blockIdx.z;
    int r0 = 0, r1 = g.R;
    if (g.offsets != nullptr) {
        r0 = max(0, min(g.offsets[e], g.R));
        r1 = max(r0, min(g.offsets[e + 1], g.R));
    }
    const int m0 = r0 + blockIdx.y * 64, n0 = blockIdx.x * 64;
    if (m0 >= r1) return;
    const uint8_t* W = g.W + e * g.w_stride;
    const float* sw = g.sw + e * g.sw_stride;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float y[4][4] = {};
    for (int kb = 0; kb * fp8::BLOCK < g.K; ++kb) {
        float p[4][4] = {};
        for (int k0 = kb * fp8::BLOCK; k0 < min(g.K, (kb + 1) * fp8::BLOCK); k0 += KC) {
            __syncthreads();
            for (int i = threadIdx.x; i < 64 * KC; i += 256) {
                const int r = i / KC, k = k0 + i % KC;
                as[i % KC][r] = m0 + r < r1 && k < g.K ? fp8_value(g.A[(int64_t)(m0 + r) * g.lda + k]) : 0.0f;
                ws[i % KC][r] = n0 + r < g.N && k < g.K ? fp8_value(W[(int64_t)(n0 + r) * g.ldw + k]) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < KC; ++k) {
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) p[i][j] = fmaf(as[k][ty * 4 + i], ws[k][tx * 4 + j], p[i][j]);
                }
            }
        }
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = min(m0 + ty * 4 + i, r1 - 1);
            const int n = min(n0 + tx * 4, g.N - 1);
            const float s = g.sa[kb * g.ldsa + m] * sw[kb * g.ldsw + n / fp8::BLOCK];
            #pragma unroll
            for (int j = 0; j < 4; ++j) y[i][j] = fmaf(p[i][j], s, y[i][j]);
        }
    }
    T* out = static_cast<T*>(g.out);
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m < r1 && n < g.N) out[(int64_t)m * g.ldo + n] = fp8_out<T>(y[i][j]);
        }
    }
}

}  // namespace bnn
