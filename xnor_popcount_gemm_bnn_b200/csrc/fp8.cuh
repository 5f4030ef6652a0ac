// 8-bit floating-point operands with one fp32 scale per block of 128: the
// quantise-and-pack kernels, and the element helpers of the products on them.
//
// A real x in a block with scale s is stored as the e4m3 code of x / s
// (4 exponent bits, 3 mantissa bits, largest value 448, NaN 0x7F, no
// infinities): s = max(amax / 448, 2^-126) with amax the largest finite |x| of
// the block, so the largest element lands on 448 and no quotient is larger.
// The quotient is that of x * 448 by amax, rounded once to fp32 (2^-24, against
// the 2^-4 of the code itself; see Quotient for fp32 x).  Blocks are 1 x 128 (activations: one
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
constexpr float SCALE_MIN = 1.17549435e-38f;   // 2^-126, the least normal number: no scale is subnormal or 0

__device__ __forceinline__ float block_scale(float amax) { return fmaxf(__fdiv_rn(amax, CODE_MAX), SCALE_MIN); }

// Two codes of a, b (a in the low byte); NaN gives the NaN code.
__device__ __forceinline__ uint32_t codes2(float2 v) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}

// x * 448 / amax as x * m / d: d is amax's significand in [1, 2) and m = 448 *
// 2^-exponent, so that nothing over- or underflows that matters; 2^126 and 1
// where the scale is 2^-126.
struct Quotient {
    float m, d, inv;                        // inv = 1 / d, rounded
    __device__ __forceinline__ void set(float amax) {
        const uint32_t b = __float_as_uint(amax), e = b >> 23;
        const bool least = amax < 448.0f * SCALE_MIN;
        m = least ? 0x1p126f : __uint_as_float((262u - e) << 23 | 0x600000u);
        d = least ? 1.0f : __uint_as_float((b & 0x7FFFFFu) | 0x3F800000u);
    }
    // Two quotients: q = y inv with y = x m is off by less than one and a half
    // units, and q - remainder * inv, the remainder q d - y from one fused
    // multiply-add, rounds correctly where the remainder is exact (Markstein,
    // IBM J. Res. Dev. 34, 1990); written so that a zero keeps its sign.
    // EXACT (bf16): y has 8 + 3 bits and d 8, so y and the remainder are exact,
    // and no quotient lies within 2^-9 of a unit of the middle of two numbers.
    // Else y's error joins the remainder, which may take a 25th bit: the
    // remainder's two roundings and that of inv are 2^-23 of a unit each, and a
    // quotient that lies within 2^-21 of a unit of the middle of two numbers may
    // go to either.  (With 27 bits over 24 it can be the middle itself: 10335963 *
    // 448 / 12582912 = 368 - 2^-16 goes to 368 - 2^-15.)
    template <bool EXACT>
    __device__ __forceinline__ float2 of(float2 x) const {
        const float2 i2 = make_float2(-inv, -inv);
        const float2 ny = mul2(x, make_float2(-m, -m)), q = mul2(ny, i2);
        float2 r = fma2(q, make_float2(d, d), ny);
        if constexpr (!EXACT) r = fma2(fma2(x, make_float2(m, m), ny), make_float2(-1.0f, -1.0f), r);
        return fma2(r, i2, q);
    }
};

// 32 bytes, read-only and not kept in L1 (one access where a row's lanes would
// otherwise touch every 32-byte sector twice).
__device__ __forceinline__ void ldg_stream_v8(const void* p, uint32_t* w) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

// What a lane packs at a time: 16 consecutive elements as loaded (fp32, or
// pairs of bf16), an eighth of a block.
template <typename T>
struct Elems {
    static constexpr int WORDS = 16 * (int)sizeof(T) / 4;
    uint32_t w[WORDS];

    // Elements c .. c + 15 of a row of K, 0 past K.  ALIGN: the alignment in
    // bytes of every row's start (32 or 16).
    template <int ALIGN>
    __device__ __forceinline__ void load(const T* row, int64_t c, int64_t K) {
        if (c + 16 <= K) {
            if constexpr (ALIGN == 32) {
                #pragma unroll
                for (int i = 0; i < WORDS; i += 8) ldg_stream_v8(reinterpret_cast<const uint32_t*>(row + c) + i, w + i);
            } else {
                #pragma unroll
                for (int i = 0; i < WORDS; i += 4) {
                    const uint4 q = ldg_stream_v4(reinterpret_cast<const uint32_t*>(row + c) + i);
                    w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
                }
            }
        } else {
            #pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = c + i < K ? __float_as_uint(to_float(row[c + i])) : 0u;
                } else {
                    const uint32_t lo = c + 2 * i < K ? __bfloat16_as_ushort(row[c + 2 * i]) : 0u;
                    const uint32_t hi = c + 2 * i + 1 < K ? __bfloat16_as_ushort(row[c + 2 * i + 1]) : 0u;
                    w[i] = lo | (hi << 16);
                }
            }
        }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    }
    // Largest |x|: NaN left out (unless all are), infinities not.
    __device__ __forceinline__ float amax() const {
        if constexpr (sizeof(T) == 4) {
            float a = fabsf(value(0));
            #pragma unroll
            for (int i = 1; i < 16; ++i) a = fmaxf(a, fabsf(value(i)));
            return a;
        } else {
            __nv_bfloat162 a = __habs2(reinterpret_cast<const __nv_bfloat162&>(w[0]));
            #pragma unroll
            for (int i = 1; i < WORDS; ++i) a = __hmax2(a, __habs2(reinterpret_cast<const __nv_bfloat162&>(w[i])));
            return fmaxf(__low2float(a), __high2float(a));
        }
    }
    __device__ __forceinline__ float finite_amax() const {
        float a = 0.0f;
        #pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = fabsf(value(i));
            if (v < __int_as_float(0x7F800000)) a = fmaxf(a, v);
        }
        return a;
    }
    // 16 codes.  SPECIAL (the block holds an infinity or nothing but NaN): x * 0
    // is 0 for a finite x and NaN otherwise, which then gets the NaN code.
    template <bool SPECIAL>
    __device__ __forceinline__ uint4 codes(const Quotient& by) const {
        uint32_t o[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c[2];
            #pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 v = make_float2(value(4 * i + 2 * j), value(4 * i + 2 * j + 1));
                float2 q = by.of<sizeof(T) == 2>(v);
                if constexpr (SPECIAL) q = make_float2(fmaf(v.x, 0.0f, q.x), fmaf(v.y, 0.0f, q.y));
                c[j] = codes2(q);
            }
            o[i] = c[0] | (c[1] << 16);
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
};

// Rows of a lesser alignment: a warp takes a row of a block, four elements per
// lane in 4 / V loads of V elements (V * sizeof(T) the alignment, 8 bytes at
// most), each load of the warp one contiguous piece.
template <typename T, int V>
struct Narrow {
    float v[4];
    static __device__ __forceinline__ int column(int i, int lane) { return (i / V) * (32 * V) + lane * V + i % V; }
    // `n`: the columns of the block that the row has (128, less at the row's
    // end, none past it).  Predicated loads, so that all of a lane's are in
    // flight together; V elements that the row ends among come by rest().
    __device__ __forceinline__ void load(const T* p, int n, int lane) {
        #pragma unroll
        for (int i = 0; i < 4; i += V) {
            const int c = column(i, lane);
            const int on = c + V <= n ? 1 : 0;
            if constexpr (V * sizeof(T) == 8) {
                uint32_t lo, hi;
                asm volatile(
                    "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
                    "@p ld.global.nc.v2.b32 {%0, %1}, [%2];\n\t}"
                    : "=&r"(lo), "=&r"(hi)
                    : "l"(p + c), "r"(on));
                if constexpr (sizeof(T) == 4) {
                    v[i] = __uint_as_float(lo);
                    v[i + 1] = __uint_as_float(hi);
                } else {
                    v[0] = __uint_as_float(lo << 16);
                    v[1] = __uint_as_float(lo & 0xFFFF0000u);
                    v[2] = __uint_as_float(hi << 16);
                    v[3] = __uint_as_float(hi & 0xFFFF0000u);
                }
            } else if constexpr (V == 2) {
                uint32_t q;
                asm volatile(
                    "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
                    "@p ld.global.nc.b32 %0, [%1];\n\t}"
                    : "=&r"(q)
                    : "l"(p + c), "r"(on));
                v[i] = __uint_as_float(q << 16);
                v[i + 1] = __uint_as_float(q & 0xFFFF0000u);
            } else {
                v[i] = on ? to_float(p[c]) : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void rest(const T* p, int n, int lane) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = column(i, lane);
            if (c < n && c - c % V + V > n) v[i] = to_float(p[c]);
        }
    }
    __device__ __forceinline__ float amax() const {
        return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    }
    __device__ __forceinline__ float finite_amax() const {
        float a = 0.0f;
        #pragma unroll
        for (int i = 0; i < 4; ++i)
            if (fabsf(v[i]) < __int_as_float(0x7F800000)) a = fmaxf(a, fabsf(v[i]));
        return a;
    }
    // Codes to columns below `np` (n rounded up to 16) of the block's row.
    __device__ __forceinline__ void store(uint8_t* p, int np, int lane, const Quotient& by, bool special) const {
        float2 q[2];
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            q[i] = by.of<sizeof(T) == 2>(make_float2(v[2 * i], v[2 * i + 1]));
            if (special) q[i] = make_float2(fmaf(v[2 * i], 0.0f, q[i].x), fmaf(v[2 * i + 1], 0.0f, q[i].y));
        }
        const uint32_t lo = codes2(q[0]), hi = codes2(q[1]);
        #pragma unroll
        for (int i = 0; i < 4; i += V) {
            const int c = column(i, lane);
            if (c >= np) continue;
            const uint32_t two = i < 2 ? lo : hi;
            if constexpr (V == 1) p[c] = (uint8_t)((i & 1) ? two >> 8 : two);
            else if constexpr (V == 2) *reinterpret_cast<uint16_t*>(p + c) = (uint16_t)two;
            else *reinterpret_cast<uint32_t*>(p + c) = lo | (hi << 16);
        }
    }
};

// Largest of the lanes' non-negative numbers or NaN (above them all), by their
// bits: those of magnitudes order as unsigned integers.
__device__ __forceinline__ float warp_max_bits(float a) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}

// No number, or an infinity.
__device__ __forceinline__ bool not_finite(float a) { return !(a < __int_as_float(0x7F800000)); }
constexpr int LANES = BLOCK / 16;           // lanes per block of a row
}  // namespace fp8

// Blocks of 1 x 128.  Eight lanes share a block; a warp takes U x 512 elements
// of one row and reads every element once.  Warps of consecutive rows run next
// to each other, so their scales, consecutive in memory, meet in L2.  Measured:
// 16384 rows of 4096 bf16 gathered from 4096, 27 to 28 us (134 MB read through L2,
// 69 MB written): a row is read, reduced and divided once for each of its packed
// rows (61 % of the issue slots, two dependent loads before the first element).
// 4096 x 4096 fp32 15 us, 0.86 of the measured HBM rate.
template <typename T, int ALIGN, int U>
__global__ void __launch_bounds__(256)
fp8_pack_rows_kernel(const T* __restrict__ x, int64_t x_rows, int64_t K, int64_t ld_x,
                     const int32_t* __restrict__ row_index, int64_t rows, uint8_t* __restrict__ codes, int64_t ldc,
                     float* __restrict__ scales, int64_t lds) {
    using namespace fp8;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    int64_t src = r;
    if (row_index != nullptr) {
        src = __ldg(row_index + r);
        if (src < 0 || src >= x_rows) return;        // the row is left as it was
    }
    const T* xr = x + src * ld_x;
    for (int64_t c0 = (int64_t)blockIdx.y * (512 * U) + lane * 16; c0 - lane * 16 < K; c0 += (int64_t)gridDim.y * (512 * U)) {
        Elems<T> v[U];
        #pragma unroll
        for (int u = 0; u < U; ++u) v[u].template load<ALIGN>(xr, c0 + u * 512, K);
        // Lane u of a block's eight keeps the amax of its u-th vector, so that
        // one division and one reciprocal serve all U.
        float a = 0.0f;
        bool special = false;
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            float m = v[u].amax();
            special |= not_finite(m);
            #pragma unroll
            for (int off = 1; off < LANES; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            if ((lane & (LANES - 1)) == u) a = m;
        }
        special = __any_sync(0xffffffffu, special);
        if (special) {
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                float m = v[u].finite_amax();
                #pragma unroll
                for (int off = 1; off < LANES; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                if ((lane & (LANES - 1)) == u) a = m;
            }
        }
        const float s = block_scale(a);
        Quotient by;
        by.set(a);
        const float inv = __frcp_rn(by.d);
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + u * 512;
            const int from = (lane & ~(LANES - 1)) | u;
            by.set(__shfl_sync(0xffffffffu, a, from));
            by.inv = __shfl_sync(0xffffffffu, inv, from);
            if (c < K)
                *reinterpret_cast<uint4*>(codes + r * ldc + c) =
                    special ? v[u].template codes<true>(by) : v[u].template codes<false>(by);
        }
        // Lane u of the eight writes the scale of the block in its u-th vector.
        const int64_t cs = c0 - lane * 16 + (lane & ~(LANES - 1)) * 16 + (lane & (LANES - 1)) * 512;
        if ((lane & (LANES - 1)) < U && cs < K) scales[cs / BLOCK * lds + r] = s;
    }
}

// The same for rows of any alignment: a warp takes U blocks of one row.
template <typename T, int V, int U>
__global__ void __launch_bounds__(256)
fp8_pack_rows_narrow_kernel(const T* __restrict__ x, int64_t x_rows, int64_t K, int64_t ld_x,
                            const int32_t* __restrict__ row_index, int64_t rows, uint8_t* __restrict__ codes,
                            int64_t ldc, float* __restrict__ scales, int64_t lds) {
    using namespace fp8;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    int64_t src = r;
    if (row_index != nullptr) {
        src = __ldg(row_index + r);
        if (src < 0 || src >= x_rows) return;        // the row is left as it was
    }
    const T* xr = x + src * ld_x;
    for (int64_t b0 = (int64_t)blockIdx.y * U; b0 * BLOCK < K; b0 += (int64_t)gridDim.y * U) {
        Narrow<T, V> v[U];
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t n = K - (b0 + u) * BLOCK;
            v[u].load(xr + (b0 + u) * BLOCK, n < BLOCK ? (n < 0 ? 0 : (int)n) : BLOCK, lane);
        }
        if (V > 1 && K % V != 0) {
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t n = K - (b0 + u) * BLOCK;
                if (n > 0 && n < BLOCK) v[u].rest(xr + (b0 + u) * BLOCK, (int)n, lane);
            }
        }
        float a = 0.0f;                              // lane u's: the amax of block u
        bool special = false;
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const float m = warp_max_bits(v[u].amax());
            special |= not_finite(m);
            if (lane == u) a = m;
        }
        if (special) {
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                const float m = warp_max_bits(v[u].finite_amax());
                if (lane == u) a = m;
            }
        }
        const float s = block_scale(a);
        Quotient by;
        by.set(a);
        const float inv = __frcp_rn(by.d);
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            by.set(__shfl_sync(0xffffffffu, a, u));
            by.inv = __shfl_sync(0xffffffffu, inv, u);
            const int64_t n = (K + 15) / 16 * 16 - (b0 + u) * BLOCK;
            v[u].store(codes + r * ldc + (b0 + u) * BLOCK, n < BLOCK ? (n < 0 ? 0 : (int)n) : BLOCK, lane, by, special);
        }
        if (lane < U && (b0 + lane) * BLOCK < K) scales[(b0 + lane) * lds + r] = s;
    }
}

// Blocks of 128 x 128, one per CTA: 256 threads hold the block in registers
// (64 elements each) between finding its amax and writing its codes.  Bound by
// HBM: 4096 x 4096 bf16 9.7 us, 0.79 of the measured rate.
template <typename T, int ALIGN>
__global__ void __launch_bounds__(256)
fp8_pack_blocks_kernel(const T* __restrict__ x, int64_t rows, int64_t K, int64_t ld_x, uint8_t* __restrict__ codes,
                       int64_t ldc, float* __restrict__ scales, int64_t lds, unsigned kblocks) {
    using namespace fp8;
    constexpr int U = 4;                             // passes of 8 warps x 4 rows
    __shared__ float part[8];
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t kb = blockIdx.x % kblocks, rb = blockIdx.x / kblocks;
    const int64_t c = kb * BLOCK + (lane & (LANES - 1)) * 16;
    const int64_t r0 = rb * BLOCK + warp * 4 + lane / LANES;
    Elems<T> v[U];
    #pragma unroll
    for (int u = 0; u < U; ++u) v[u].template load<ALIGN>(x + min(r0 + 32 * u, rows - 1) * ld_x, c, K);
    // A row past the end is read as the last one: its elements change no amax
    // of a block that holds that row.
    float a = v[0].amax();
    #pragma unroll
    for (int u = 1; u < U; ++u) a = fmaxf(a, v[u].amax());
    bool special = __syncthreads_or(not_finite(a));
    if (special) {
        a = 0.0f;
        #pragma unroll
        for (int u = 0; u < U; ++u) a = fmaxf(a, v[u].finite_amax());
    }
    a = warp_max_bits(a);
    if (lane == 0) part[warp] = a;
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < 8; ++w) a = fmaxf(a, part[w]);
    const float s = block_scale(a);
    Quotient by;
    by.set(a);
    by.inv = __frcp_rn(by.d);
    #pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + 32 * u;
        if (r < rows && c < K)
            *reinterpret_cast<uint4*>(codes + r * ldc + c) =
                special ? v[u].template codes<true>(by) : v[u].template codes<false>(by);
    }
    if (threadIdx.x == 0) scales[kb * lds + rb] = s;
}

// The same for rows of any alignment: a warp takes 16 rows of the block.
// 11008 x 4090 fp32 (rows on 8-byte boundaries) 44 to 47 us, 0.78 to 0.73 of the
// measured HBM rate; with 16 elements per lane in 8-byte loads it took 46 us
// before the quotient was refined, this layout 40.
template <typename T, int V>
__global__ void __launch_bounds__(256)
fp8_pack_blocks_narrow_kernel(const T* __restrict__ x, int64_t rows, int64_t K, int64_t ld_x,
                              uint8_t* __restrict__ codes, int64_t ldc, float* __restrict__ scales, int64_t lds,
                              unsigned kblocks) {
    using namespace fp8;
    constexpr int U = 16;
    __shared__ float part[8];
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t kb = blockIdx.x % kblocks, rb = blockIdx.x / kblocks;
    const int64_t left = K - kb * BLOCK, r0 = rb * BLOCK + warp;
    const int n = left < BLOCK ? (int)left : BLOCK;
    Narrow<T, V> v[U];
    #pragma unroll
    for (int u = 0; u < U; ++u) v[u].load(x + min(r0 + 8 * u, rows - 1) * ld_x + kb * BLOCK, n, lane);
    if (V > 1 && n % V != 0) {
        #pragma unroll
        for (int u = 0; u < U; ++u) v[u].rest(x + min(r0 + 8 * u, rows - 1) * ld_x + kb * BLOCK, n, lane);
    }
    float a = v[0].amax();
    #pragma unroll
    for (int u = 1; u < U; ++u) a = fmaxf(a, v[u].amax());
    const bool special = __syncthreads_or(not_finite(a));
    if (special) {
        a = 0.0f;
        #pragma unroll
        for (int u = 0; u < U; ++u) a = fmaxf(a, v[u].finite_amax());
    }
    a = warp_max_bits(a);
    if (lane == 0) part[warp] = a;
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < 8; ++w) a = fmaxf(a, part[w]);
    const float s = block_scale(a);
    Quotient by;
    by.set(a);
    by.inv = __frcp_rn(by.d);
    #pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + 8 * u;
        if (r < rows) v[u].store(codes + r * ldc + kb * BLOCK, (n + 15) / 16 * 16, lane, by, special);
    }
    if (threadIdx.x == 0) scales[kb * lds + rb] = s;
}

}  // namespace bnn
