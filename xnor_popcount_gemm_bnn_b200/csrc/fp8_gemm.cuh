// Products of 8-bit floating-point operands with block scales (fp8.cuh):
//   C[m, n] = sum_b sA[b, m] sW[b, n / 128] sum_{k in block b} a[m, k] w[n, k]
//
// The inner sum of a block is four tcgen05.mma kind::f8f6f4 (K = 32 each) into
// a fresh fp32 accumulator in tensor memory; the sum over blocks is kept in
// fp32 registers, C += s * inner, because every block has its own scale.  s =
// sA sW is rounded to fp32 before it meets the sum (one multiplication per row
// and block instead of one per element), which limits the scales' range: see
// bnn_fp8_gemm.  K tails need no care: the tensor maps end at K, so the copies
// fill zeros.
//
// Two kernels share the work:
//  * fp8_gemm_split_kernel, few rows: the weights are the 128-row operand of
//    the MMA and the rows of A its N (16 .. 128), so that a small batch wastes
//    nothing; K is split over a cluster.
//  * fp8_gemm_pair_kernel, many rows: CTA pairs on 256 rows x 128 or 256
//    columns.
// Every mbarrier wait is bounded as in gemm_tc.cuh: on time-out the roles stop
// at their next wait, outstanding copies and MMAs are waited for (bounded),
// and tensor memory is freed before exit.
#pragma once

#include "fp8.cuh"
#include "gemm_f4.cuh"

namespace bnn {

// Operands of a (grouped) product.  Dense: offsets == nullptr, one group of R
// rows.  Grouped: rows offsets[e] .. offsets[e + 1] of A meet W[e].  A and W
// themselves come through tensor maps.
struct Fp8Gemm {
    const float* sa;
    int64_t ldsa;
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

// Four consecutive outputs, aligned to four elements.
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(reinterpret_cast<const uint32_t&>(a), reinterpret_cast<const uint32_t&>(b));
}

// Rows [r0, r1) of group e, clamped to [0, R] whatever the offsets hold.
__device__ __forceinline__ int2 fp8_group_rows(const Fp8Gemm& g, int e) {
    if (g.offsets == nullptr) return make_int2(0, g.R);
    const int r0 = max(0, min(g.offsets[e], g.R));
    return make_int2(r0, max(r0, min(g.offsets[e + 1], g.R)));
}

template <int CTAS>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    if constexpr (CTAS == 2) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}

// kind::f8f6f4 instruction descriptor: D fp32 (bits 4-5 = 1), A and B e4m3
// (0 at bits 7-9 and 10-12), both K-major, N >> 3 at bits 17-22, M >> 4 at 24-28.
__host__ __device__ constexpr uint32_t f8_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// True in one lane of a converged warp.  The compiler knows that one lane
// runs what this guards, and issues tensor-core and copy instructions there
// without a loop over the lanes.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
// TMEM -> registers in two statements, so that arithmetic runs between them: the
// load is started, and the wait names the registers, which hold their values
// only after it (every use has to come through the wait's outputs).
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// tc_wait by all lanes of a converged warp, which stay converged, for waits that
// come once per K block: the timer is read only after the wait has failed for a
// while.
__device__ __forceinline__ bool f8_wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    #pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag));
}

// Whether the phase of parity `parity` is complete, without waiting.  Asked for
// the next K block while this one's work goes on, it hides what a wait costs
// even when there is nothing to wait for (about 180 cycles with the vote).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Arrive on an mbarrier given by its address in the cluster's shared memory,
// without ordering earlier memory operations (a release over the cluster costs
// about a thousand cycles here): for an arrival that only says that values
// have come into registers.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// acc += t * s on pairs of fp32 (one instruction per two products).
__device__ __forceinline__ void scale_add2(float2& acc, float2 t, float2 s) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<unsigned long long&>(acc))
        : "l"(reinterpret_cast<unsigned long long&>(t)), "l"(reinterpret_cast<unsigned long long&>(s)));
}

// 16 bytes of the cluster's shared memory; zeros where `on` is 0.
__device__ __forceinline__ float4 ld_shared_cluster_v4_if(uint32_t addr, int on) {
    float4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&f"(v.x), "=&f"(v.y), "=&f"(v.z), "=&f"(v.w)
        : "r"(addr), "r"(on)
        : "memory");
    return v;
}
// Orders the accesses to the cluster's shared memory so far before the
// asynchronous copies that a barrier lets go after it.
__device__ __forceinline__ void fence_proxy_async_cluster() {
    asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}
__device__ __forceinline__ uint32_t mapa_shared(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// ---------------------------------------------------------------------------
// Few rows: out^T tile of 128 weight rows x NT rows of A per cluster.
// ---------------------------------------------------------------------------
namespace f8s {
constexpr int BN = 128;                      // weight rows per CTA = TMEM lanes
constexpr int W_BYTES = BN * fp8::BLOCK;     // 16 KiB of weights per stage
constexpr int WARP_PRODUCER = 0, WARP_MMA = 1, WARP_SCALE = 2, WARP_EPI0 = 4;
constexpr int AHEAD = 8;                     // K blocks whose scales are in flight
constexpr int MAX_SPLIT = 8;
constexpr int SMEM_SM = 228 * 1024;          // shared memory of an SM, 1 KiB of it reserved per CTA
template <int NT, bool DEEP>
struct Cfg {
    static constexpr int STAGE = W_BYTES + NT * fp8::BLOCK;
    static constexpr int NBUF = 4;                           // accumulators in tensor memory
    static constexpr int TMEM_COLS = NBUF * NT;
    // CTAs per SM: weights stream from HBM for one while another starts or
    // ends.  Whatever variants meet on an SM, their shared memory lets no more
    // in than tensor memory has room for: a cluster's CTAs wait for one another
    // and must not wait for an allocation.
    static constexpr int PER_SM = NT <= 64 ? 2 : 1;
    static constexpr int PARTS = NT <= 64 ? 1 : 2;           // warps per quadrant, each with its columns
    static constexpr int CW = NT / PARTS;
    static constexpr int THREADS = (WARP_EPI0 + 4 * PARTS) * 32;
    static constexpr int SC = (NT + 31) / 32;                // columns per lane of the scale warp
    static constexpr int RAW_BYTES = AHEAD * (SC + 1) * 32 * 4;
    static constexpr int PROD_BYTES = 2 * NBUF * NT * 4;
    static constexpr int FIXED = RAW_BYTES + PROD_BYTES + 512 + 1024;
    // DEEP: as many stages as fit.  Else three, enough in flight for a short
    // stream, and room for a CTA of the next launch to set up beside the two of
    // this one (NT = 16 only, see the launcher).
    static constexpr int STAGES = DEEP ? (SMEM_SM / PER_SM - 1024 - FIXED) / STAGE : 3;
    static constexpr int SMEM_BYTES = FIXED + STAGES * STAGE;
    static_assert(TMEM_COLS >= 32 && (TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS * PER_SM <= 512, "tensor memory");
    static_assert(NT * BN * 4 <= STAGES * STAGE, "the partial sums reuse the ring");
    static_assert(STAGE % 1024 == 0, "128B swizzle");
    static_assert((2 * STAGES + 2 * NBUF + 1) * 8 + 16 <= 512, "barriers");
    static constexpr int SHARE = SMEM_BYTES + 1024;          // of SMEM_SM
};
// What fits together in shared memory has its tensor memory: two CTAs of 256
// columns leave no room for another, one of 512 for none.
constexpr int SMALLEST = Cfg<16, false>::SHARE;
static_assert(SMALLEST <= Cfg<16, true>::SHARE && SMALLEST <= Cfg<32, true>::SHARE &&
                  2 * Cfg<64, true>::SHARE + SMALLEST > SMEM_SM && Cfg<64, true>::SHARE <= Cfg<32, true>::SHARE &&
                  Cfg<128, true>::SHARE + SMALLEST > SMEM_SM,
              "tensor memory of the CTAs that share an SM");
}  // namespace f8s

// The sums of S CTAs: parts[column][128] fp32 at the same shared-memory offset
// in each.  Rank q adds the columns q, q + S, ... in rank order; a warp takes
// whole columns, four rows of weights per lane, and several of them at a time,
// since every remote load takes about half a microsecond.
struct Fp8Parts {
    uint32_t parts;
    int rank, warp, warps, cols, m0, n0, vec_out;
};
template <int S, typename T>
__device__ __forceinline__ void add_parts(const Fp8Parts& p, const Fp8Gemm& g, int lane) {
    constexpr int C = 16 / S;                    // columns whose loads are in flight together
    const int step = S * p.warps, n = p.n0 + 4 * lane;
    for (int c0 = p.rank + p.warp * S; c0 < p.cols; c0 += C * step) {
        float4 v[C][S];
        #pragma unroll
        for (int i = 0; i < C; ++i) {
            const uint32_t at = p.parts + ((c0 + i * step) * f8s::BN + 4 * lane) * 4;
            const int on = c0 + i * step < p.cols ? 1 : 0;
            #pragma unroll
            for (int r = 0; r < S; ++r) v[i][r] = ld_shared_cluster_v4_if(mapa_shared(at, r), on);
        }
        #pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = c0 + i * step;
            if (c >= p.cols) break;
            float4 y = v[i][0];
            #pragma unroll
            for (int r = 1; r < S; ++r) {
                y.x += v[i][r].x;
                y.y += v[i][r].y;
                y.z += v[i][r].z;
                y.w += v[i][r].w;
            }
            T* out = static_cast<T*>(g.out) + (int64_t)(p.m0 + c) * g.ldo + n;
            if (p.vec_out && n + 4 <= g.N) {
                store4(out, y);
            } else {
                if (n < g.N) out[0] = fp8_out<T>(y.x);
                if (n + 1 < g.N) out[1] = fp8_out<T>(y.y);
                if (n + 2 < g.N) out[2] = fp8_out<T>(y.z);
                if (n + 3 < g.N) out[3] = fp8_out<T>(y.w);
            }
        }
    }
}

// grid: (tiles of 128 weight rows x E) * S CTAs in clusters of S; a group's
// rows are walked NT at a time.  Cluster rank r takes K blocks [r nk / S, (r + 1) nk / S).
//  warp 0     producer: TMA of 128 weight rows and NT rows of A per K block.
//  warp 1     issues the block's four MMAs (M = 128, N = NT) and commits them
//             to the accumulator and to the stage.
//  warp 2     scales: sA[b, column] * sW[b, tile] of the NT columns, copied AHEAD
//             blocks ahead and put into shared memory; its arrival on the
//             accumulator's barrier goes with the MMAs' commit.
//  warps 4 .. epilogue: thread = one weight row; per block its columns' sums
//             from tensor memory times their scales, added in registers.
// With S > 1 the CTAs leave their partial sums in shared memory and each adds
// the columns r, r + S, ... of all of them in rank order: the same sum on every run.
// Bound by the weights' stream and, when it is short, by the launch: 11008 x 4096
// and one row 10.4 to 11.1 us (45 MB, 0.66 of the measured HBM rate; 0.5 us of it
// the parts' addition), 64 experts of 2048 x 4096 with 128 rows 65 to 72 us (387 MB
// read, 0.91 to 0.82).  The scales, whose loads a register would have waited for in every
// block, were what bound it first (13.8 and 107 us).
template <int NT, bool DEEP, typename T>
__global__ void __launch_bounds__(f8s::Cfg<NT, DEEP>::THREADS, f8s::Cfg<NT, DEEP>::PER_SM)
fp8_gemm_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, Fp8Gemm g,
                      int tiles_n, int S, int vec_out) {
    using namespace f8s;
    using C = Cfg<NT, DEEP>;
    constexpr int STAGES = C::STAGES, NBUF = C::NBUF, SC = C::SC, CW = C::CW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* prod = reinterpret_cast<float*>(ring + STAGES * C::STAGE);      // [2 NBUF][NT]
    float* raw = prod + C::PROD_BYTES / 4;                                 // [AHEAD][SC + 1][32]
    uint64_t* full = reinterpret_cast<uint64_t*>(raw + C::RAW_BYTES / 4);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + NBUF;
    uint64_t* drain = tempty + NBUF;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cid = (int)blockIdx.x / S, rank = (int)blockIdx.x % S;
    const int e = cid / tiles_n, tile = cid % tiles_n, n0 = tile * BN;
    const int nk = (g.K + fp8::BLOCK - 1) / fp8::BLOCK;
    const int kb0 = (int)((int64_t)rank * nk / S), kb1 = (int)((int64_t)(rank + 1) * nk / S);

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmW);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&tfull[b], 2);                   // the MMAs' commit and the scales
            mbar_init(&tempty[b], 4 * C::PARTS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // Everything above may overlap the previous kernel; operands, offsets and
    // outputs are touched only after it.
    grid_dependency_wait();
    grid_dependents_launch();
    const int2 rows = fp8_group_rows(g, e);

    uint32_t it = 0;                          // K blocks this role has handled, over all chunks
    uint32_t issued = 0;
    bool ok = true;
    bool ready = false;                       // what this role waits for is there for its next block
    for (int m0 = rows.x; m0 < rows.y; m0 += NT) {
        if (warp == WARP_PRODUCER) {
            for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                const uint32_t s = it % STAGES;
                ok = it < STAGES || f8_wait_all(&empty[s], ((it / STAGES) - 1) & 1, abort_flag);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t* dst = ring + s * C::STAGE;
                    mbar_arrive_expect_tx(&full[s], C::STAGE);
                    tma_load_3d(dst, &tmW, kb * fp8::BLOCK, n0, e, &full[s]);
                    tma_load_2d(dst + W_BYTES, &tmA, kb * fp8::BLOCK, m0, &full[s]);
                }
                __syncwarp();
                ++issued;
            }
        } else if (warp == WARP_MMA) {
            // Stages lie 16-byte units apart in the descriptor's address field
            // (a shared-memory address never carries out of it).
            const uint64_t wdesc = umma_desc_sw128(smem_u32(ring));
            for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                const uint32_t s = it % STAGES, b = it % NBUF;
                const uint64_t dw = wdesc + (uint64_t)(s * (C::STAGE >> 4)), da = dw + (W_BYTES >> 4);
                ok = ready || (f8_wait_all(&full[s], (it / STAGES) & 1, abort_flag) &&
                               (it < NBUF || f8_wait_all(&tempty[b], ((it / NBUF) - 1) & 1, abort_flag)));
                if (!ok) break;
                tc_fence_after();
                const uint32_t nx = it + 1;
                const bool fn = mbar_test(&full[nx % STAGES], (nx / STAGES) & 1);
                const bool en = nx < NBUF || mbar_test(&tempty[nx % NBUF], ((nx / NBUF) - 1) & 1);
                if (elect_one()) {
                    #pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8<1>(tmem_base + b * NT, dw + kk * 2, da + kk * 2, f8_idesc(BN, NT), kk != 0 ? 1u : 0u);
                    mma_commit(&tfull[b]);
                    mma_commit(&empty[s]);
                }
                ready = __all_sync(0xffffffffu, fn && en);
            }
        } else if (warp == WARP_SCALE) {
            const float* sa = g.sa + m0 + lane;
            const float* sw = g.sw + e * g.sw_stride + tile;
            const int cols = rows.y - m0;
            // Every lane copies what it needs itself, so only its own copies
            // are waited for; columns past the group's end keep what the slot
            // held (their sums are not stored).
            auto load = [&](int kb) {
                if (kb < kb1) {
                    float* d = raw + ((kb - kb0) % AHEAD) * (SC + 1) * 32 + lane;
                    #pragma unroll
                    for (int i = 0; i < SC; ++i)
                        if (32 * i + lane < min(cols, NT)) cp_async4(d + 32 * i, sa + kb * g.ldsa + 32 * i);
                    cp_async4(d + 32 * SC, sw + kb * g.ldsw);
                }
                cp_async_commit();
            };
            #pragma unroll
            for (int i = 0; i < AHEAD - 1; ++i) load(kb0 + i);
            for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                const uint32_t b = it % NBUF;
                load(kb + AHEAD - 1);
                cp_async_wait<AHEAD - 1>();
                // The accumulator's previous use is committed: its barrier can
                // take this block's arrival, and the epilogue is done with the
                // block 2 NBUF before this one (the MMAs had waited for it).
                ok = it < NBUF || f8_wait_all(&tfull[b], ((it / NBUF) - 1) & 1, abort_flag);
                if (!ok) break;
                const float* d = raw + ((kb - kb0) % AHEAD) * (SC + 1) * 32 + lane;
                float* p = prod + (it % (2 * NBUF)) * NT + lane;
                const float w = d[32 * SC];
                #pragma unroll
                for (int i = 0; i < SC; ++i)
                    if (32 * i + lane < NT) p[32 * i] = d[32 * i] * w;
                __syncwarp();
                if (lane == 0) mbar_arrive(&tfull[b]);
            }
            cp_async_wait<0>();
        } else if (warp >= WARP_EPI0) {
            const int quad = warp & 3, part = (warp - WARP_EPI0) >> 2;
            const int cols = min(NT, rows.y - m0);
            const uint32_t tq = tmem_base + ((uint32_t)(32 * quad) << 16) + part * CW;
            constexpr int CH = 16;                          // columns per load
            float2 acc[CW / 2];
            #pragma unroll
            for (int c = 0; c < CW / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            #pragma unroll 1
            for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                const uint32_t b = it % NBUF;
                ok = ready || f8_wait_all(&tfull[b], (it / NBUF) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const bool next = mbar_test(&tfull[(it + 1) % NBUF], ((it + 1) / NBUF) & 1);
                const float* s = prod + (it % (2 * NBUF)) * NT + part * CW;
                #pragma unroll
                for (int c = 0; c < CW; c += CH) {
                    uint32_t r[CH];
                    tmem_ld16_sync(tq + b * NT + c, r);
                    #pragma unroll
                    for (int j = 0; j < CH; j += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(s + c + j);
                        scale_add2(acc[(c + j) / 2], make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                             make_float2(f.x, f.y));
                        scale_add2(acc[(c + j) / 2 + 1], make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])),
                             make_float2(f.z, f.w));
                    }
                }
                tc_fence_before();
                ready = __all_sync(0xffffffffu, next);   // and every lane has used its scales
                if (elect_one()) mbar_arrive(&tempty[b]);
            }
            const int n = 32 * quad + lane;
            T* out = static_cast<T*>(g.out) + n0 + n;
            if (S == 1) {
                if (ok && n0 + n < g.N) {
                    #pragma unroll
                    for (int c = 0; c < CW; ++c) {
                        const int m = part * CW + c;
                        if (m < cols) out[(int64_t)(m0 + m) * g.ldo] = fp8_out<T>(c & 1 ? acc[c / 2].y : acc[c / 2].x);
                    }
                }
            } else {
                // The last block's commit covers all MMAs of this chunk, so the
                // ring is free for the partial sums.
                float* sum = reinterpret_cast<float*>(ring) + part * CW * BN + n;
                #pragma unroll
                for (int c = 0; c < CW; ++c)
                    if (part * CW + c < cols) sum[c * BN] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
            }
        }
        if (S > 1) {
            __syncwarp();
            cluster_sync_all();
            if (warp >= WARP_EPI0) {
                const int cols = ok ? min(NT, rows.y - m0) : 0;
                const Fp8Parts to{smem_u32(ring), rank, warp - WARP_EPI0, 4 * C::PARTS, cols, m0, n0, vec_out};
                switch (S) {
                    case 2: add_parts<2, T>(to, g, lane); break;
                    case 3: add_parts<3, T>(to, g, lane); break;
                    case 4: add_parts<4, T>(to, g, lane); break;
                    case 5: add_parts<5, T>(to, g, lane); break;
                    case 6: add_parts<6, T>(to, g, lane); break;
                    case 7: add_parts<7, T>(to, g, lane); break;
                    default: add_parts<8, T>(to, g, lane); break;
                }
                // Ordered before the next chunk's copies into the ring, which this
                // CTA's threads have written and the cluster's have read.
                fence_proxy_async_cluster();
            }
            __syncwarp();
            cluster_sync_all();
        }
    }
    if (warp == WARP_PRODUCER && lane == 0 && !ok) {
        for (uint32_t q = issued > STAGES ? issued - STAGES : 0; q < issued; ++q)
            if (!mbar_wait_bounded(&full[q % STAGES], (q / STAGES) & 1)) break;
    }
    if (warp == WARP_MMA && elect_one()) {
        mma_commit(drain);
        mbar_wait_bounded(drain, 0);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Many rows: CTA pairs on tiles of 256 rows x BN columns.
// ---------------------------------------------------------------------------
namespace f8p {
constexpr int BM = 128;                      // rows of A per CTA = TMEM lanes
constexpr int A_BYTES = BM * fp8::BLOCK;     // 16 KiB per stage
constexpr int WARP_PRODUCER = 0, WARP_MMA = 1, WARP_SCALE = 2, SCALE_WARPS = 2, WARP_EPI0 = 4, EPI_WARPS = 8;
constexpr int THREADS = (WARP_EPI0 + EPI_WARPS) * 32;
constexpr int AHEAD = 4;                     // K blocks whose scales a scale warp has in flight
constexpr int OUT_ROW = 64;                  // bytes per row of an epilogue warp's staging block
constexpr int OUT_BLOCK = 32 * OUT_ROW;
constexpr int BAND = 8;                      // row tiles that a band of concurrent tiles spans
template <int BN>
struct Cfg {
    static constexpr int W_BYTES = BN / 2 * fp8::BLOCK;      // this CTA's half of the weight rows
    static constexpr int STAGE = A_BYTES + W_BYTES;
    static constexpr int NBUF = 512 / BN;                    // accumulators in tensor memory
    static constexpr int NBK = BN / fp8::BLOCK;              // column blocks of a tile
    static constexpr int RAW_BYTES = SCALE_WARPS * AHEAD * (4 + NBK) * 32 * 4;
    static constexpr int PROD_BYTES = 2 * NBUF * NBK * BM * 4;
    static constexpr int FIXED = EPI_WARPS * OUT_BLOCK + RAW_BYTES + PROD_BYTES + 512 + 1024;
    static constexpr int STAGES = (tc::SMEM_LIMIT - FIXED) / STAGE;
    static constexpr int SMEM_BYTES = FIXED + STAGES * STAGE;
    static_assert((2 * STAGES + 2 * NBUF + 1) * 8 + 16 <= 512, "barriers");
    static_assert(STAGE % 1024 == 0, "128B swizzle");
};
}  // namespace f8p

// TMA load into this CTA's shared memory whose bytes count on the barrier at
// the same offset in the pair's even CTA.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Where a tile lies: group, first row, first column.
struct Fp8Tile {
    int e, m0, n0, r1;
};

// Walks the tiles of all groups in order.  A whole warp holds a window of 32
// groups, one per lane, with the running sum of their tiles; t grows from call
// to call, so the window only moves forward.
template <int BN>
struct Fp8Tiles {
    int tiles_n, first, base, incl;          // window's first group, tiles before it, this lane's inclusive sum
    int2 rows;
    __device__ __forceinline__ void load(const Fp8Gemm& g, int lane) {
        rows = make_int2(0, 0);
        if (first + lane < g.E) rows = fp8_group_rows(g, first + lane);
        incl = (rows.y - rows.x + 2 * f8p::BM - 1) / (2 * f8p::BM) * tiles_n;
        #pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
    }
    __device__ __forceinline__ void init(const Fp8Gemm& g, int lane) {
        tiles_n = (g.N + BN - 1) / BN;
        first = base = 0;
        load(g, lane);
    }
    // False past the last tile.  The whole warp calls it.
    __device__ __forceinline__ bool find(const Fp8Gemm& g, int lane, int t, Fp8Tile& out) {
        while (true) {
            const int total = __shfl_sync(0xffffffffu, incl, 31);
            if (t < base + total) break;
            base += total;
            first += 32;
            if (first >= g.E) return false;
            load(g, lane);
        }
        const int j = __ffs(__ballot_sync(0xffffffffu, t < base + incl)) - 1;
        const int r0 = __shfl_sync(0xffffffffu, rows.x, j), r1 = __shfl_sync(0xffffffffu, rows.y, j);
        const int before = __shfl_sync(0xffffffffu, incl, j > 0 ? j - 1 : 0);
        const int lt = t - base - (j > 0 ? before : 0);
        // Bands of BAND row tiles, column by column: the tiles in flight span
        // about as many rows as columns and share operands in L2.
        const int tiles_m = (r1 - r0 + 2 * f8p::BM - 1) / (2 * f8p::BM);
        const int band = lt / (f8p::BAND * tiles_n), in = lt - band * (f8p::BAND * tiles_n);
        const int mt = min(f8p::BAND, tiles_m - band * f8p::BAND);
        out.e = first + j;
        out.m0 = r0 + (band * f8p::BAND + in % mt) * (2 * f8p::BM);
        out.n0 = in / mt * BN;
        out.r1 = r1;
        return true;
    }
};

// Persistent pairs of CTAs (cta_group::2), one CTA per SM:
//  warp 0     producer in each CTA: its 128 rows of A and its half of the BN
//             weight rows per K block, counted on the even CTA's barrier.
//  warp 1     in the even CTA issues the four MMAs of a K block (M = 256,
//             N = BN) for both.
//  warps 2-3  scales, taking turns: per K block sA[b, row] * sW[b, column
//             block] for the CTA's rows and the tile's column blocks, copied
//             ahead and put into shared memory; the arrival on the
//             accumulator's barrier goes with the MMAs' commit.
//  warps 4-11 epilogue: two warps per quadrant of 32 rows, half of the columns
//             each; thread = one row, BN / 2 fp32 sums in registers,
//             C += scale * inner, one scale per thread and block.
// The tensor memory holds 512 / BN accumulators: the MMAs of the next blocks
// run while the epilogue adds this one.  What bounds the kernel is the
// latency of each role's loop per block (wait, issue, hand on), which is why
// the loops hold nothing else and ask for the next block's barriers early.
// Measured: 8192 x 8192 x 8192 to bf16 480 to 490 us in a call by itself = 2.26
// PFLOP/s, 0.70 of twice the measured bf16 rate (tensor pipe active 46 %), and 550 to
// 570 us = 1.96 in a loop under the power limit, 0.72 of twice the sustained rate;
// without the sums over blocks, one accumulation over K, the single call took 401
// us.  The 256-column variants spill 20 (fp32) and 56 bytes (bf16) a thread.  On the way: a release
// over the cluster in every hand-back cost 470 us, scales loaded into registers
// 280, copies and MMAs issued by a lane the compiler did not know to be alone 60.
// The finished tile is rounded, put into shared memory (16-byte chunks swizzled
// by row, no bank conflicts) and stored by row, rows and columns outside left
// out.
template <int BN, typename T>
__global__ void __launch_bounds__(f8p::THREADS, 1)
fp8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, Fp8Gemm g,
                     int vec_out) {
    using namespace f8p;
    using C = Cfg<BN>;
    constexpr int STAGES = C::STAGES, NBUF = C::NBUF, NBK = C::NBK;
    constexpr int CW = BN / (EPI_WARPS / 4);                               // columns of an epilogue warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* oring = ring + STAGES * C::STAGE;
    float* raw = reinterpret_cast<float*>(oring + EPI_WARPS * OUT_BLOCK);  // [SCALE_WARPS][AHEAD][4 + NBK][32]
    float* prod = raw + C::RAW_BYTES / 4;                                  // [2 NBUF][NBK][BM]
    uint64_t* full = reinterpret_cast<uint64_t*>(prod + C::PROD_BYTES / 4);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + NBUF;
    uint64_t* drain = tempty + NBUF;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cid = (int)blockIdx.x / 2, ncl = (int)gridDim.x / 2;
    const int nk = (g.K + fp8::BLOCK - 1) / fp8::BLOCK;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmW);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&tfull[b], 2);                   // the MMAs' commit and the scales
            mbar_init(&tempty[b], EPI_WARPS * 2);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == WARP_MMA) f4_tmem_alloc<true>(tmem_slot, 512);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependency_wait();
    grid_dependents_launch();

    Fp8Tiles<BN> tiles;
    tiles.init(g, lane);
    Fp8Tile tl;
    uint32_t it = 0;
    bool ok = true;
    // The epilogue's sums and the loads beside them take more registers than the
    // other four warps: 128 * 80 + 256 * 208 of the launch's 384 * 168.
    if (warp < WARP_EPI0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == WARP_PRODUCER) {
            uint32_t issued = 0;
            for (int t = cid; ok && tiles.find(g, lane, t, tl); t += ncl) {
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t s = it % STAGES;
                    ok = it < STAGES || f8_wait_all(&empty[s], ((it / STAGES) - 1) & 1, abort_flag);
                    if (!ok) break;
                    if (elect_one()) {
                        uint8_t* dst = ring + s * C::STAGE;
                        const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE);
                        tma_load_2d_pair(dst, &tmA, kb * fp8::BLOCK, tl.m0 + (int)rank * BM, bar);
                        tma_load_3d_pair(dst + A_BYTES, &tmW, kb * fp8::BLOCK, tl.n0 + (int)rank * (BN / 2), tl.e, bar);
                    }
                    __syncwarp();
                    ++issued;
                }
            }
            // After a failed wait: both CTAs' copies count on the even CTA's barriers.
            if (lane == 0 && !ok && rank == 0) {
                for (uint32_t q = issued > STAGES ? issued - STAGES : 0; q < issued; ++q)
                    if (!mbar_wait_bounded(&full[q % STAGES], (q / STAGES) & 1)) break;
            }
            __syncwarp();
        } else if (warp == WARP_MMA) {
            if (rank == 0) {
                // Stages lie 16-byte units apart in the descriptor's address field
                // (a shared-memory address never carries out of it).
                const uint64_t adesc = umma_desc_sw128(smem_u32(ring));
                bool ready = false;                        // the next block's stage and accumulator
                for (int t = cid; ok && tiles.find(g, lane, t, tl); t += ncl) {
                    for (int kb = 0; kb < nk; ++kb, ++it) {
                        const uint32_t s = it % STAGES, b = it % NBUF;
                        const uint64_t da = adesc + (uint64_t)(s * (C::STAGE >> 4)), dw = da + (A_BYTES >> 4);
                        ok = ready || (f8_wait_all(&full[s], (it / STAGES) & 1, abort_flag) &&
                                       (it < NBUF || f8_wait_all(&tempty[b], ((it / NBUF) - 1) & 1, abort_flag)));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t nx = it + 1;
                        const bool f = mbar_test(&full[nx % STAGES], (nx / STAGES) & 1);
                        const bool e = nx < NBUF || mbar_test(&tempty[nx % NBUF], ((nx / NBUF) - 1) & 1);
                        if (elect_one()) {
                            #pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_f8<2>(tmem_base + b * BN, da + kk * 2, dw + kk * 2, f8_idesc(2 * BM, BN),
                                          kk != 0 ? 1u : 0u);
                            f4_commit<true>(&tfull[b], 0x3);
                            f4_commit<true>(&empty[s], 0x3);
                        }
                        ready = __all_sync(0xffffffffu, f && e);
                    }
                }
                if (elect_one()) {
                    f4_commit<true>(drain, 0x1);
                    mbar_wait_bounded(drain, 0);
                }
                __syncwarp();
            }
        } else {
            const int sw_id = warp - WARP_SCALE;           // takes the blocks whose `it` is this modulo SCALE_WARPS
            float* mine = raw + sw_id * AHEAD * (4 + NBK) * 32 + lane;
            for (int t = cid; ok && tiles.find(g, lane, t, tl); t += ncl) {
                // Rows and columns past the ends take the last one's scale; they are not stored.
                const float* sa[4];
                const float* sw[NBK];
                #pragma unroll
                for (int i = 0; i < 4; ++i) sa[i] = g.sa + min(tl.m0 + (int)rank * BM + 32 * i + lane, tl.r1 - 1);
                #pragma unroll
                for (int i = 0; i < NBK; ++i)
                    sw[i] = g.sw + tl.e * g.sw_stride + min(tl.n0 + i * fp8::BLOCK, g.N - 1) / fp8::BLOCK;
                // Every lane copies what it needs itself, so only its own copies are waited for.
                auto load = [&](int kb) {
                    if (kb < nk) {
                        float* d = mine + (kb / SCALE_WARPS % AHEAD) * (4 + NBK) * 32;
                        #pragma unroll
                        for (int i = 0; i < 4; ++i) cp_async4(d + 32 * i, sa[i] + kb * g.ldsa);
                        #pragma unroll
                        for (int i = 0; i < NBK; ++i) cp_async4(d + 32 * (4 + i), sw[i] + kb * g.ldsw);
                    }
                    cp_async_commit();
                };
                const uint32_t it0 = it;
                const int first = (int)((uint32_t)(sw_id - (int)it0) % SCALE_WARPS);
                #pragma unroll
                for (int i = 0; i < AHEAD - 1; ++i) load(first + i * SCALE_WARPS);
                for (int kb = first; kb < nk; kb += SCALE_WARPS) {
                    it = it0 + kb;
                    const uint32_t b = it % NBUF;
                    load(kb + (AHEAD - 1) * SCALE_WARPS);
                    cp_async_wait<AHEAD - 1>();
                    // The accumulator's previous use is committed: its barrier can
                    // take this block's arrival, and the epilogue is done with the
                    // block 2 NBUF before this one (the MMAs had waited for it).
                    ok = it < NBUF || f8_wait_all(&tfull[b], ((it / NBUF) - 1) & 1, abort_flag);
                    if (!ok) break;
                    const float* d = mine + (kb / SCALE_WARPS % AHEAD) * (4 + NBK) * 32;
                    float* p = prod + (it % (2 * NBUF)) * NBK * BM + lane;
                    #pragma unroll
                    for (int n = 0; n < NBK; ++n) {
                        const float w = d[32 * (4 + n)];
                        #pragma unroll
                        for (int i = 0; i < 4; ++i) p[n * BM + 32 * i] = d[32 * i] * w;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tfull[b]);
                }
                it = it0 + nk;
            }
            cp_async_wait<0>();                            // (after a failed wait some are in flight)
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int quad = warp & 3, part = (warp - WARP_EPI0) >> 2;
        uint8_t* stage = oring + (warp - WARP_EPI0) * OUT_BLOCK;
        const uint32_t hand_back = mapa_shared(smem_u32(tempty), 0);
        const float* sp = prod + part * CW / fp8::BLOCK * BM + 32 * quad + lane;
        const uint32_t tq = tmem_base + ((uint32_t)(32 * quad) << 16) + part * CW;
        T* out = static_cast<T*>(g.out);
        bool ready = false;                            // the next accumulator and its scales
        for (int t = cid; ok && tiles.find(g, lane, t, tl); t += ncl) {
            const int mq = tl.m0 + (int)rank * BM + 32 * quad;       // first row of this warp
            const int nh = tl.n0 + part * CW;                        // first column
            float2 acc[CW / 2];
            #pragma unroll
            for (int c = 0; c < CW / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            #pragma unroll 1
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t b = it % NBUF;
                ok = ready || f8_wait_all(&tfull[b], (it / NBUF) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const float f = sp[(it % (2 * NBUF)) * NBK * BM];
                const float2 s = make_float2(f, f);
                bool next = false;
                // The load of the next 32 columns runs beside the sums of these.
                const uint32_t t0 = tq + b * BN;
                uint32_t r[2][32];
                tmem_ld32_start(t0, r[0]);
                #pragma unroll
                for (int c = 0; c < CW; c += 32) {
                    uint32_t(&v)[32] = r[(c / 32) & 1];
                    tmem_ld32_wait(v);
                    if (c + 32 < CW) {
                        tmem_ld32_start(t0 + c + 32, r[(c / 32 + 1) & 1]);
                    } else {
                        // Everything has been read and the scale is used: nothing of
                        // this block is touched after the arrival.
                        tc_fence_before();
                        if (elect_one()) mbar_arrive_relaxed(hand_back + b * 8);
                        next = mbar_test(&tfull[(it + 1) % NBUF], ((it + 1) / NBUF) & 1);
                    }
                    #pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        scale_add2(acc[(c + j) / 2], make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), s);
                }
                ready = __all_sync(0xffffffffu, next);
            }
            if (!ok) break;
            // 32 rows x 64 bytes at a time: chunk q of row r at (q ^ (r >> 1 & 3)) * 16.
            constexpr int CE = 16 / (int)sizeof(T);                  // elements per 16-byte chunk
            constexpr int CQ = OUT_ROW / 16;                         // chunks per row and pass
            constexpr int PER = CQ * CE;                             // columns per pass
            static_assert(CW % PER == 0, "whole passes");
            #pragma unroll
            for (int c = 0; c < CW; c += PER) {
                #pragma unroll
                for (int q = 0; q < CQ; ++q) {
                    uint4 v;
                    T* e = reinterpret_cast<T*>(&v);
                    #pragma unroll
                    for (int i = 0; i < CE; ++i) {
                        const int j = c + q * CE + i;
                        e[i] = fp8_out<T>(j & 1 ? acc[j / 2].y : acc[j / 2].x);
                    }
                    *reinterpret_cast<uint4*>(stage + lane * OUT_ROW + ((q ^ ((lane >> 1) & 3)) << 4)) = v;
                }
                __syncwarp();
                const int nb = nh + c;
                if (vec_out) {
                    #pragma unroll
                    for (int p = 0; p < CQ; ++p) {
                        const int r = p * (32 / CQ) + lane / CQ, q = lane % CQ, m = mq + r, n = nb + q * CE;
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * OUT_ROW + ((q ^ ((r >> 1) & 3)) << 4));
                        if (m < tl.r1 && n < g.N) {
                            T* dst = out + (int64_t)m * g.ldo + n;
                            if (n + CE <= g.N) {
                                *reinterpret_cast<uint4*>(dst) = v;
                            } else {
                                const T* e = reinterpret_cast<const T*>(&v);
                                #pragma unroll
                                for (int i = 0; i < CE; ++i)
                                    if (n + i < g.N) dst[i] = e[i];
                            }
                        }
                    }
                } else {
                    // Any alignment: elements one by one, a row's next to each other.
                    for (int i = lane; i < 32 * PER; i += 32) {
                        const int r = i / PER, j = i % PER, m = mq + r, n = nb + j;
                        const T v = *reinterpret_cast<const T*>(stage + r * OUT_ROW +
                                                                (((j / CE) ^ ((r >> 1) & 3)) << 4) + (j % CE) * sizeof(T));
                        if (m < tl.r1 && n < g.N) out[(int64_t)m * g.ldo + n] = v;
                    }
                }
                __syncwarp();
            }
        }
    }
    // The even CTA's MMAs read the odd one's shared and tensor memory.
    tc_fence_before();
    cluster_sync_all();
    if (warp == WARP_MMA) {
        tc_fence_after();
        f4_tmem_dealloc<true>(tmem_base, 512);
    }
}

}  // namespace bnn
