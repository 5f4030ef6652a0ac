// Routing of tokens to experts: scores, choice, weights, the plan of rows by
// expert, and the weighted sum of the experts' rows.
#pragma once

#include <math_constants.h>

#include "common.cuh"

namespace bnn {
namespace route {
constexpr int MAX_E = 512;
constexpr int MAX_K = 16;
constexpr int MAX_GROUPS = 32;
constexpr int PLAN_CLUSTER = 8;
constexpr int PLAN_THREADS = 512;
}  // namespace route

struct RouteParams {
    int T, E, k;
    int64_t ld;
    int sigmoid, groups, kept, group_top, renorm;
    double scale;
    const float* bias;
    int32_t* idx;
    float* weights;
};

// Doubles as unsigned keys in the same order (negative ones reversed); 0 is
// below every number's key and marks what cannot be chosen.
__device__ __forceinline__ unsigned long long order_key(double v) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);   // -0 -> +0
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// Largest key of the warp and the lowest index that has it.
__device__ __forceinline__ void warp_best(unsigned long long& key, int& id) {
    #pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, key, off);
        const int i2 = __shfl_xor_sync(0xffffffffu, id, off);
        if (k2 > key || (k2 == key && i2 < id)) { key = k2; id = i2; }
    }
}
__device__ __forceinline__ double warp_max(double v) {
    #pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
    #pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// One warp per token; lane l holds experts l, l + 32, ...  Scores and the
// choice in fp64: neighbouring scores of a few hundred experts are often
// closer than fp32 tells apart, and the chosen set is a whole-number result.
template <typename T, int NI>
__global__ void __launch_bounds__(256) route_topk_kernel(const T* __restrict__ logits, RouteParams p) {
    using namespace route;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T* row = logits + (int64_t)t * p.ld;
    double score[NI];
    unsigned long long key[NI];
    double top = -CUDART_INF;
    #pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        float l = e < p.E ? to_float(row[e]) : -CUDART_INF_F;
        if (!(l > -CUDART_INF_F)) l = -CUDART_INF_F;          // NaN masks an expert as -inf does
        if (l == CUDART_INF_F) l = 3.402823466e38f;
        score[i] = (double)l;
        top = fmax(top, score[i]);
    }
    if (!p.sigmoid) {
        top = warp_max(top);
        double sum = 0.0;
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool on = score[i] > -CUDART_INF;
            key[i] = on ? 1ull : 0ull;
            score[i] = on ? exp(score[i] - top) : 0.0;
            sum += score[i];
        }
        sum = warp_sum(sum);
        #pragma unroll
        for (int i = 0; i < NI; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
    } else {
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool on = score[i] > -CUDART_INF;
            key[i] = on ? 1ull : 0ull;
            score[i] = on ? 1.0 / (1.0 + exp(-score[i])) : 0.0;
        }
    }
    #pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        if (key[i] == 0) continue;
        double c = score[i];
        if (p.bias != nullptr) c += (double)__ldg(p.bias + e);
        key[i] = c > -CUDART_INF ? order_key(c) : 0ull;       // a NaN or -inf bias masks too
    }
    if (p.groups > 1 && p.kept < p.groups) {
        // Lane g keeps group g's score: its largest choice value, or the sum
        // of its two largest.
        const int per = p.E / p.groups;
        unsigned long long mine = 0;
        for (int g = 0; g < p.groups; ++g) {
            unsigned long long k1 = 0, k2 = 0;
            #pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                if (e / per == g && e < p.E) {
                    if (key[i] > k1) { k2 = k1; k1 = key[i]; }
                    else if (key[i] > k2) k2 = key[i];
                }
            }
            #pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                const unsigned long long o1 = __shfl_xor_sync(0xffffffffu, k1, off);
                const unsigned long long o2 = __shfl_xor_sync(0xffffffffu, k2, off);
                if (o1 > k1) { k2 = max(k1, o2); k1 = o1; }
                else k2 = max(k2, o1);
            }
            unsigned long long gk = k1;
            if (p.group_top > 1 && k2 != 0) {
                auto val = [](unsigned long long q) {
                    return __longlong_as_double((long long)((q >> 63) ? q & 0x7FFFFFFFFFFFFFFFull : ~q));
                };
                gk = order_key(val(k1) + val(k2));
            }
            if (lane == g) mine = gk;
        }
        unsigned kept = 0;
        for (int j = 0; j < p.kept; ++j) {
            unsigned long long b = mine;
            int id = lane;
            warp_best(b, id);
            if (b == 0) break;
            kept |= 1u << id;
            if (lane == id) mine = 0;
        }
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E && ((kept >> (e / per)) & 1u) == 0) key[i] = 0;
        }
    }
    // k rounds: every lane offers its best, the winner's lane gives it up.
    int my_e = -1;
    double my_s = 0.0;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long b = 0;
        int id = 0x7fffffff;
        double s = 0.0;
        #pragma unroll
        for (int i = 0; i < NI; ++i)
            if (key[i] > b) { b = key[i]; id = lane + 32 * i; s = score[i]; }
        int win = id;
        warp_best(b, win);
        if (b == 0) break;
        const double ws = __shfl_sync(0xffffffffu, s, win & 31);
        if (lane == j) { my_e = win; my_s = ws; }
        if (lane == (win & 31)) {
            #pragma unroll
            for (int i = 0; i < NI; ++i)
                if (lane + 32 * i == win) key[i] = 0;
        }
    }
    const double sum = warp_sum(my_s);
    if (lane < p.k) {
        double w = my_s;
        if (p.renorm) w = sum > 0.0 ? w / sum : 0.0;
        p.idx[(int64_t)t * p.k + lane] = my_e;
        p.weights[(int64_t)t * p.k + lane] = (float)(w * p.scale);
    }
}

// The plan: slots (t, j) in the order of t * k + j, sorted stably by expert.
//   offsets[e]    first row of expert e, offsets[E] the rows in use
//   row_token[r]  token of row r (-1 from offsets[E] on)
//   slot_row[s]   row of slot s (-1 for a slot without an expert)
// One cluster: CTA c counts its share of the slots per warp and expert in
// shared memory, the counts of the CTAs before it come over distributed
// shared memory, and each slot's row is the expert's start + the earlier
// CTAs' and warps' counts + its place in the warp.  No atomics order the
// result: it is the same on every run.
__global__ void __launch_bounds__(route::PLAN_THREADS)
route_plan_kernel(const int32_t* __restrict__ idx, int slots, int k, int E, int32_t* __restrict__ offsets,
                  int32_t* __restrict__ row_token, int32_t* __restrict__ slot_row) {
    using namespace route;
    constexpr int WARPS = PLAN_THREADS / 32;
    extern __shared__ int32_t plan_smem[];
    int32_t* total = plan_smem;                       // [E] this CTA's counts
    int32_t* start = total + MAX_E;                   // [E] first row of this CTA's slots of each expert
    int32_t* cnt = start + MAX_E;                     // [WARPS][E] counts, then running starts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    // Shares of whole warp steps: CTA c has slots [s0, s1), warp w of it [a, b).
    const int steps = (slots + 31) / 32;
    const int per_cta = (steps + PLAN_CLUSTER - 1) / PLAN_CLUSTER;
    const int per_warp = (per_cta + WARPS - 1) / WARPS;
    const int c0 = (int)rank * per_cta, c1 = min(steps, c0 + per_cta);
    const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);
    for (int i = threadIdx.x; i < WARPS * E; i += PLAN_THREADS) cnt[i] = 0;
    __syncthreads();
    int32_t* mine = cnt + warp * E;
    for (int st = w0; st < w1; ++st) {
        const int s = st * 32 + lane;
        const int e = s < slots ? idx[s] : -1;
        const bool on = e >= 0 && e < E;
        const unsigned same = __match_any_sync(0xffffffffu, on ? e : -1);
        if (on && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS) {
        int run = 0;
        for (int w = 0; w < WARPS; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        total[e] = run;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // Counts of the earlier CTAs and of all of them, per expert.
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS) {
        int before = 0, all = 0;
        for (int c = 0; c < PLAN_CLUSTER; ++c) {
            uint32_t a;
            int v;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(total + e)), "r"(c));
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
            if (c < (int)rank) before += v;
            all += v;
        }
        start[e] = all;
        for (int w = 0; w < WARPS; ++w) cnt[w * E + e] += before;
    }
    __syncthreads();
    if (warp == 0) {                                  // exclusive scan of the experts' totals
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int v = e0 + lane < E ? start[e0 + lane] : 0;
            int x = v;
            #pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            if (e0 + lane < E) start[e0 + lane] = carry + x - v;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        if (rank == 0) {
            __syncwarp();
            for (int e = lane; e < E; e += 32) offsets[e] = start[e];
            if (lane == 0) offsets[E] = carry;
        }
        // rows without a slot
        if (row_token != nullptr)
            for (int r = carry + (int)rank * 32 + lane; r < slots; r += 32 * PLAN_CLUSTER) row_token[r] = -1;
    }
    __syncthreads();
    for (int st = w0; st < w1; ++st) {
        const int s = st * 32 + lane;
        const int e = s < slots ? idx[s] : -1;
        const bool on = e >= 0 && e < E;
        const unsigned same = __match_any_sync(0xffffffffu, on ? e : -1);
        int r = -1;
        if (on) r = start[e] + mine[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (on && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
        if (s < slots) {
            if (slot_row != nullptr) slot_row[s] = r;
            if (on && row_token != nullptr) row_token[r] = s / k;
        }
    }
    // No CTA leaves while another may still read its counts.
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// out[t, n] = sum_j weights[t, j] * Y[slot_row[t, j], n], in j order, fp32.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ T route_out(float v);
template <>
__device__ __forceinline__ float route_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 route_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 16 bytes, read-only and not kept in L1; zeros where `on` is 0.
__device__ __forceinline__ uint4 ldg_stream_v4_if(const void* p, int on) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(on));
    return v;
}

__device__ __forceinline__ float ldg_if(const float* p, int on) {
    float v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.f32 %0, [%1];\n\t}"
        : "=&f"(v)
        : "l"(p), "r"(on));
    return v;
}
__device__ __forceinline__ float ldg_if(const __nv_bfloat16* p, int on) {
    unsigned short v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
        : "=&h"(v)
        : "l"(p), "r"(on));
    return __uint_as_float((uint32_t)v << 16);
}

// Bound by reading the k rows of a token, each once.  A block takes one token
// and C pieces of V elements per thread, THREADS * V apart; the lanes hold the
// token's rows and weights, and the loads of eight rows are in flight
// together (predicated: a branch would wait for each).  V = 16 bytes of T
// where every row of Y and out allows it, else 1.
constexpr int kCombineThreads = 128;
template <typename T, typename O, int V, int C>
__global__ void __launch_bounds__(kCombineThreads)
route_combine_kernel(const T* __restrict__ Y, int64_t R, int64_t N, int64_t ldy, const int32_t* __restrict__ slot_row,
                     const float* __restrict__ weights, int k, O* __restrict__ out, int64_t ldo) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    static_assert(V == 1 || C == 1, "one vector per thread");
    const int64_t t = blockIdx.x;
    constexpr int PER = kCombineThreads * C * V;
    for (int64_t base = (int64_t)blockIdx.y * PER; base < N; base += (int64_t)gridDim.y * PER) {
        const int64_t n0 = base + threadIdx.x * V;
        float y[C][V];
        #pragma unroll
        for (int c = 0; c < C; ++c) {
            #pragma unroll
            for (int i = 0; i < V; ++i) y[c][i] = 0.0f;
        }
        for (int j0 = 0; j0 < k; j0 += 32) {
            int row = -1;
            float w = 0.0f;
            if (j0 + lane < k) {
                row = __ldg(slot_row + t * k + j0 + lane);
                w = __ldg(weights + t * k + j0 + lane);
            }
            const int n_j = min(32, k - j0);
            constexpr int J = V == 1 ? 4 : 8;
            for (int j = 0; j < n_j; j += J) {
                // Slots past k hold row -1 and weight 0.
                uint4 q[V == 1 ? 1 : J];
                float s[V == 1 ? J : 1][C], f[J];
                #pragma unroll
                for (int i = 0; i < J; ++i) {
                    const int64_t r = __shfl_sync(0xffffffffu, row, j + i);
                    const bool on = r >= 0 && r < R;
                    f[i] = __shfl_sync(0xffffffffu, w, j + i);
                    f[i] = on ? f[i] : 0.0f;
                    #pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int64_t n = n0 + c * (kCombineThreads * V);
                        if constexpr (V == 1) s[i][c] = ldg_if(Y + r * ldy + n, on && n < N ? 1 : 0);
                        else q[i] = ldg_stream_v4_if(Y + r * ldy + n, on && n < N ? 1 : 0);
                    }
                }
                #pragma unroll
                for (int i = 0; i < J; ++i) {
                    #pragma unroll
                    for (int c = 0; c < C; ++c) {
                        if constexpr (V == 1) {
                            y[c][0] = fmaf(f[i], s[i][c], y[c][0]);
                        } else {
                            const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
                            #pragma unroll
                            for (int e = 0; e < V; ++e) {
                                float v;
                                if constexpr (sizeof(T) == 4) v = __uint_as_float(u[e]);
                                else v = __uint_as_float((e & 1) ? (u[e >> 1] & 0xFFFF0000u) : (u[e >> 1] << 16));
                                y[c][e] = fmaf(f[i], v, y[c][e]);
                            }
                        }
                    }
                }
            }
        }
        #pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t n = n0 + (int64_t)c * (kCombineThreads * V);
            if (n >= N) continue;
            O* o = out + t * ldo + n;
            if constexpr (V == 1) {
                o[0] = route_out<O>(y[c][0]);
            } else {
                union {
                    O e[V];
                    uint2 w[V * sizeof(O) / 8];
                } q;
                #pragma unroll
                for (int i = 0; i < V; ++i) q.e[i] = route_out<O>(y[c][i]);
                #pragma unroll
                for (int i = 0; i < (int)(V * sizeof(O) / 8); ++i) reinterpret_cast<uint2*>(o)[i] = q.w[i];
            }
        }
    }
}

}  // namespace bnn
