// 8-bit floating-point operands with one fp32 scale per block of 128: the
// quantise-and-pack kernels, and the element helpers of the products on them.
//
// A real x in a block with scale s is stored as the e4m3 code of x / s
// (4 exponent bits, 3 mantissa bits, largest value 448, NaN 0x7F, no
// infinities): s = max(amax / 448, 2^-126) with amax the largest finite |x| of
// the block, so the largest element lands on 448 and no quotient is larger.
// The quotient is taken as x * (1 / s), both roundings in fp32 (each 2^-24,
// against the 2^-4 of the code itself).  Blocks are 1 x 128 (activations: one
// row's 128 consecutive elements of K) or 128 x 128 (weights).  The scale of
// row block i and K block b is scales[b * ld + i]: a product walks K block by
// block and then reads consecutive rows' scales together.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace bnn {
namespace fp8 {
constexpr int BLOCK = 128;                  // elements of K (and weight rows) per scale
constexpr float CODE_MAX = 448.0f;
constexpr float SCALE_MIN = 1.17549435e-38f;   // 2^-126: the reciprocal stays finite

// Magnitude bits of a finite value, 0 for infinities and NaN: ordered as
// unsigned integers exactly as the magnitudes are.
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
    const uint32_t a = __float_as_uint(v) & 0x7FFFFFFFu;
    return a < 0x7F800000u ? a : 0u;
}

__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    return fmaxf(__fdiv_rn(__uint_as_float(amax_bits), CODE_MAX), SCALE_MIN);
}

// Two codes of a, b times inv (a in the low byte).  x * 0 is 0 for a finite x
// and NaN for an infinity or NaN, so those become the NaN code and not 448.
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv) {
    const float2 q = make_float2(fmaf(a, 0.0f, a * inv), fmaf(b, 0.0f, b * inv));
    return (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
    return codes2(v[0], v[1], inv) | (codes2(v[2], v[3], inv) << 16);
}

// E = 16 / sizeof(T) consecutive elements from column c of a row of K (0 past
// K).  ALIGN: the alignment in bytes that the row start and c * sizeof(T)
// share (16, 8, or sizeof(T)).
template <typename T, int ALIGN>
__device__ __forceinline__ void load_elems(const T* row, int64_t c, int64_t K, float (&v)[16 / sizeof(T)]) {
    constexpr int E = 16 / (int)sizeof(T);
    if (ALIGN >= 8 && c + E <= K) {
        uint32_t w[4];
        if constexpr (ALIGN == 16) {
            const uint4 q = ldg_stream_v4(row + c);
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        } else {
            const uint2 p = __ldg(reinterpret_cast<const uint2*>(row + c));
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(row + c) + 1);
            w[0] = p.x; w[1] = p.y; w[2] = q.x; w[3] = q.y;
        }
        #pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
            else v[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
        }
    } else {
        #pragma unroll
        for (int i = 0; i < E; ++i) v[i] = c + i < K ? to_float(row[c + i]) : 0.0f;
    }
}

// E codes at column c of a code row (ld a multiple of 16, so 4- and 8-byte
// stores are aligned); columns from kp (K rounded up to 16) on stay unwritten.
template <int E>
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c, int64_t kp, const float (&v)[E], float inv) {
    if (c >= kp) return;
    if constexpr (E == 8) {
        *reinterpret_cast<uint2*>(row + c) = make_uint2(codes4(v, inv), codes4(v + 4, inv));
    } else {
        *reinterpret_cast<uint32_t*>(row + c) = codes4(v, inv);
    }
}
}  // namespace fp8

// Blocks of 1 x 128.  A warp takes U vectors of one row (a 16-byte vector per
// lane: 256 bf16 or 128 fp32 elements per vector); the 16 (or 32) lanes of a
// block find its amax by shuffles, and every element is read once.  Warps of
// consecutive rows run next to each other, so their scales, consecutive in
// memory, meet in L2.
template <typename T, int ALIGN, int U>
__global__ void __launch_bounds__(256)
fp8_pack_rows_kernel(const T* __restrict__ x, int64_t x_rows, int64_t K, int64_t ld_x,
                     const int32_t* __restrict__ row_index, int64_t rows, uint8_t* __restrict__ codes, int64_t ldc,
                     float* __restrict__ scales, int64_t lds, int64_t tasks) {
    using namespace fp8;
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int LANES = BLOCK / E;                 // lanes per block
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (task >= tasks) return;
    const int64_t r = task % rows;
    const int64_t c0 = task / rows * (32 * E * U);
    int64_t src = r;
    if (row_index != nullptr) {
        src = __ldg(row_index + r);
        if (src < 0 || src >= x_rows) return;        // the row is left as it was
    }
    const T* xr = x + src * ld_x;
    const int64_t kp = (K + 15) / 16 * 16;
    float v[U][E];
    #pragma unroll
    for (int u = 0; u < U; ++u) load_elems<T, ALIGN>(xr, c0 + (u * 32 + lane) * E, K, v[u]);
    #pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + (u * 32 + lane) * E;
        uint32_t a = 0;
        #pragma unroll
        for (int i = 0; i < E; ++i) a = max(a, finite_abs_bits(v[u][i]));
        #pragma unroll
        for (int off = 1; off < LANES; off <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
        const float s = block_scale(a);
        store_codes<E>(codes + r * ldc, c, kp, v[u], __frcp_rn(s));
        if ((lane & (LANES - 1)) == 0 && c < K) scales[c / BLOCK * lds + r] = s;
    }
}

// Blocks of 128 x 128, one per CTA: 256 threads hold the block in registers
// (64 elements each) between finding its amax and writing its codes.
template <typename T, int ALIGN>
__global__ void __launch_bounds__(256)
fp8_pack_blocks_kernel(const T* __restrict__ x, int64_t rows, int64_t K, int64_t ld_x, uint8_t* __restrict__ codes,
                       int64_t ldc, float* __restrict__ scales, int64_t lds, int64_t kblocks) {
    using namespace fp8;
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int LANES = BLOCK / E;                 // lanes per row of the block
    constexpr int RPW = 32 / LANES;                  // rows per warp and vector
    constexpr int U = BLOCK / (8 * RPW);             // vectors per lane
    __shared__ uint32_t part[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t kb = blockIdx.x % kblocks, rb = blockIdx.x / kblocks;
    const int64_t c = kb * BLOCK + (lane & (LANES - 1)) * E;
    const int64_t r0 = rb * BLOCK + warp * (U * RPW) + lane / LANES;
    const int64_t kp = (K + 15) / 16 * 16;
    float v[U][E];
    #pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * RPW;
        if (r < rows) {
            load_elems<T, ALIGN>(x + r * ld_x, c, K, v[u]);
        } else {
            #pragma unroll
            for (int i = 0; i < E; ++i) v[u][i] = 0.0f;
        }
    }
    uint32_t a = 0;
    #pragma unroll
    for (int u = 0; u < U; ++u) {
        #pragma unroll
        for (int i = 0; i < E; ++i) a = max(a, finite_abs_bits(v[u][i]));
    }
    a = __reduce_max_sync(0xffffffffu, a);
    if (lane == 0) part[warp] = a;
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < 8; ++w) a = max(a, part[w]);
    const float s = block_scale(a);
    const float inv = __frcp_rn(s);
    #pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * RPW;
        if (r < rows) store_codes<E>(codes + r * ldc, c, kp, v[u], inv);
    }
    if (threadIdx.x == 0) scales[kb * lds + rb] = s;
}

}  // namespace bnn
