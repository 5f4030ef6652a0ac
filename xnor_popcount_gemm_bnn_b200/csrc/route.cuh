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
constexpr int PLAN_CLUSTER = 16;             // opt-in size: the scattered rows are bound by the SMs that write
constexpr int PLAN_THREADS = 512;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int SMALL_T = 16;                  // tokens that one CTA chooses for and plans in one launch
}  // namespace route

struct RouteParams {
    int T, E, k;
    int64_t ld;
    int sigmoid, groups, kept, group_top, renorm;
    double scale;
    const float* bias;
    int32_t* idx;
    float* weights;
    int vec;                                     // rows of logits can be read in vectors
};

// ---------------------------------------------------------------------------
// The choice in fp64: what the result is defined by.
// ---------------------------------------------------------------------------
// Doubles as unsigned keys in the same order (negative ones reversed); 0 is
// below every number's key and marks what cannot be chosen.
__device__ __forceinline__ unsigned long long order_key(double v) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);   // -0 -> +0
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_value(unsigned long long q) {
    return __longlong_as_double((long long)((q >> 63) ? q & 0x7FFFFFFFFFFFFFFFull : ~q));
}

// Largest key of the warp.
__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long key) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
    return (unsigned long long)hi << 32 | lo;
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

// NaN masks an expert as -inf does; +inf counts as the largest finite number.
__device__ __forceinline__ float logit_of(float l) {
    return l > -CUDART_INF_F ? fminf(l, 3.402823466e38f) : -CUDART_INF_F;
}

// Logits lane * NI .. lane * NI + NI - 1 of a row, -inf past E and where
// masked (-inf or NaN), +inf as the largest finite number; in vectors of up to
// 16 bytes where p.vec says that rows and E allow them.
template <int NI, typename T>
__device__ __forceinline__ void load_logits(const T* __restrict__ row, const RouteParams& p, int lane, float (&l)[NI]) {
    constexpr int VE = NI * (int)sizeof(T) < 16 ? NI : 16 / (int)sizeof(T);
    if (p.vec) {
        #pragma unroll
        for (int i = 0; i < NI; i += VE) {
            union {
                T e[VE];
                uint32_t w[VE * sizeof(T) / 4];
            } q;
            const int e = lane * NI + i;
            if (e < p.E) {
                if constexpr (VE * sizeof(T) == 16) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e));
                    q.w[0] = v.x; q.w[1] = v.y; q.w[2] = v.z; q.w[3] = v.w;
                } else if constexpr (VE * sizeof(T) == 8) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + e));
                    q.w[0] = v.x; q.w[1] = v.y;
                } else {
                    q.w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + e));
                }
            }
            #pragma unroll
            for (int j = 0; j < VE; ++j) l[i + j] = e < p.E ? to_float(q.e[j]) : -CUDART_INF_F;
        }
    } else {
        #pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = lane * NI + i < p.E ? to_float(row[lane * NI + i]) : -CUDART_INF_F;
    }
    #pragma unroll
    for (int i = 0; i < NI; ++i) l[i] = logit_of(l[i]);
}

// One warp, one token.  Lane j < k gets the j-th expert (-1: none) and its weight.
template <int NI, typename T>
__device__ __noinline__ void route_exact(const T* __restrict__ row, const RouteParams& p, int lane, int& my_e,
                                         float& my_w) {
    float l[NI];
    load_logits<NI>(row, p, lane, l);
    double score[NI];
    unsigned long long key[NI];
    double top = -CUDART_INF;
    #pragma unroll
    for (int i = 0; i < NI; ++i) top = fmax(top, (double)l[i]);
    if (!p.sigmoid) {
        top = warp_max(top);
        double sum = 0.0;
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            score[i] = l[i] > -CUDART_INF_F ? exp((double)l[i] - top) : 0.0;
            sum += score[i];
        }
        sum = warp_sum(sum);
        #pragma unroll
        for (int i = 0; i < NI; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
    } else {
        #pragma unroll
        for (int i = 0; i < NI; ++i) score[i] = l[i] > -CUDART_INF_F ? 1.0 / (1.0 + exp(-(double)l[i])) : 0.0;
    }
    #pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane * NI + i;
        key[i] = 0ull;
        if (!(l[i] > -CUDART_INF_F)) continue;
        const double c = score[i] + (p.bias != nullptr ? (double)__ldg(p.bias + e) : 0.0);
        key[i] = c > -CUDART_INF ? order_key(c) : 0ull;       // a NaN or -inf bias masks too
    }
    if (p.kept < p.groups) {
        // Lane g keeps group g's score: its largest choice value, or the sum
        // of its two largest.
        const int per = p.E / p.groups;
        unsigned long long mine = 0;
        for (int g = 0; g < p.groups; ++g) {
            unsigned long long k1 = 0, k2 = 0;
            #pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane * NI + i;
                if (e / per == g && e < p.E) {
                    if (key[i] > k1) { k2 = k1; k1 = key[i]; }
                    else if (key[i] > k2) k2 = key[i];
                }
            }
            const unsigned long long t1 = warp_max_key(k1);
            // The second: the winner's lane (one of them) offers its other.
            const unsigned has = __ballot_sync(0xffffffffu, k1 == t1);
            k2 = warp_max_key(lane == __ffs(has) - 1 ? k2 : k1);
            k1 = t1;
            if (p.group_top > 1 && k2 != 0) k1 = order_key(key_value(k1) + key_value(k2));
            if (lane == g) mine = k1;
        }
        unsigned kept = 0;
        for (int j = 0; j < p.kept; ++j) {
            const unsigned long long b = warp_max_key(mine);
            if (b == 0) break;
            const int id = __ffs(__ballot_sync(0xffffffffu, mine == b)) - 1;
            kept |= 1u << id;
            if (lane == id) mine = 0;
        }
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane * NI + i;
            if (e < p.E && ((kept >> (e / per)) & 1u) == 0) key[i] = 0;
        }
    }
    // k rounds: every lane offers its best, the winner's lane gives it up.
    my_e = -1;
    double my_s = 0.0;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long b = 0;
        int at = 0;
        double s = 0.0;
        #pragma unroll
        for (int i = 0; i < NI; ++i)
            if (key[i] > b) { b = key[i]; at = i; s = score[i]; }
        const unsigned long long best = warp_max_key(b);
        if (best == 0) break;
        // The lowest lane's first is the lowest index.
        const int from = __ffs(__ballot_sync(0xffffffffu, b == best)) - 1;
        const int win = from * NI + __shfl_sync(0xffffffffu, at, from);
        const double ws = __shfl_sync(0xffffffffu, s, from);
        if (lane == j) { my_e = win; my_s = ws; }
        #pragma unroll
        for (int i = 0; i < NI; ++i)
            if (lane * NI + i == win) key[i] = 0;
    }
    const double sum = warp_sum(my_s);
    my_w = (float)((p.renorm ? (sum > 0.0 ? my_s / sum : 0.0) : my_s) * p.scale);
}

// ---------------------------------------------------------------------------
// The choice in fp32, where it is certain.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t q) {
    return __uint_as_float((q >> 31) ? q & 0x7FFFFFFFu : ~q);
}

// Batcher's odd-even merge sort of N = 2^n values, as a list of compared pairs.
template <int N>
struct SortPairs {
    int a[N * N], b[N * N], n;
    constexpr SortPairs() : a{}, b{}, n(0) {
        for (int p = 1; p < N; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < N; j += 2 * k)
                    for (int i = 0; i < k && i + j + k < N; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            a[n] = i + j;
                            b[n++] = i + j + k;
                        }
    }
};
// Sorts a lane's keys, largest first, with their places (equal keys in any order).
template <int NI>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[NI], uint32_t (&at)[NI]) {
    constexpr SortPairs<NI> net;
    #pragma unroll
    for (int c = 0; c < net.n; ++c) {
        const int a = net.a[c], b = net.b[c];
        const bool swap = key[a] < key[b];
        const uint32_t ka = key[a], pa = at[a];
        key[a] = swap ? key[b] : ka;
        at[a] = swap ? at[b] : pa;
        key[b] = swap ? ka : key[b];
        at[b] = swap ? pa : at[b];
    }
}

// A choice value in fp64.  (A softmax's common divisor, which changes no order
// where there is no bias, is left out.)
template <typename T>
__device__ __forceinline__ double choice_exact(const T* __restrict__ row, const RouteParams& p, int e, float top) {
    const double l = (double)logit_of(to_float(row[e]));
    const double s = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top);
    return p.bias != nullptr ? s + (double)__ldg(p.bias + e) : s;
}

// Groups whose scores are too near on the border: each group's two best experts
// (they have to be certainly its two best) again in fp64, and the groups ranked
// by that.  Groups of whole lanes, a power of two of them.  True in lane g if
// group g is kept.
template <int NI, typename T>
__device__ __forceinline__ bool groups_exact(const T* __restrict__ row, const RouteParams& p, int lane,
                                             const uint32_t (&key)[NI], float top, float slack, bool& sure) {
    const int lanes = p.E / p.groups / NI;
    uint32_t k1 = 0, k2 = 0, k3 = 0;
    int e1 = -1, e2 = -1;
    auto insert = [&](uint32_t q, int e) {
        if (q > k1) {
            k3 = k2; k2 = k1; e2 = e1; k1 = q; e1 = e;
        } else if (q > k2) {
            k3 = k2; k2 = q; e2 = e;
        } else {
            k3 = max(k3, q);
        }
    };
    #pragma unroll
    for (int i = 0; i < NI; ++i) insert(key[i], lane * NI + i);
    for (int off = 1; off < lanes; off <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, off), o2 = __shfl_xor_sync(0xffffffffu, k2, off);
        const uint32_t o3 = __shfl_xor_sync(0xffffffffu, k3, off);
        const int f1 = __shfl_xor_sync(0xffffffffu, e1, off), f2 = __shfl_xor_sync(0xffffffffu, e2, off);
        insert(o1, f1);
        insert(o2, f2);
        k3 = max(k3, o3);
    }
    double v = -CUDART_INF;
    if (k1 != 0) {
        v = choice_exact(row, p, e1, top);
        if (k2 != 0) {
            const double w = choice_exact(row, p, e2, top);
            v = p.group_top > 1 ? v + w : fmax(v, w);
        }
    }
    sure = sure && __all_sync(0xffffffffu, k3 == 0 || key_value(k2) - key_value(k3) > slack);
    const double mine = __shfl_sync(0xffffffffu, v, (lane * lanes) & 31);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
        const double o = __shfl_sync(0xffffffffu, mine, g);
        rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    return lane < p.groups && mine > -CUDART_INF && rank < p.kept;
}

// One warp, one token, lane l holding experts l * NI .. l * NI + NI - 1.  Scores
// are taken in fp32 and every decision is checked against their errors.
// Choice values nearer than that (other than the same logit and bias, a tie in
// any precision) are compared again in fp64, one candidate per lane, and so are
// groups on the border, by their two best experts; what that does not settle --
// a softmax with a bias, scores that underflow -- goes to route_exact().  In
// fp64 throughout, the exponentials alone would take several times the kernel's
// time.  The weights are made of the chosen experts' scores in fp64 (one
// exponential per lane: 8192 tokens of 256 experts 12.1 us against 12.0 with
// fp32 weights, off by up to 2^-20); only a softmax that is not renormalised
// needs every expert's, 16.7 us against 12.1.
//   Errors: expf 2^-22 relative (2 ulp), rcp.approx 2^-23 (1 ulp), sums and
//   products 2^-24 each.  Sigmoid s = 1 / (1 + e): at most 2^-22 + 2^-23 +
//   2^-24 of it, and in absolute terms s (1 - s) 2^-22 + s (2^-23 + 2^-24) <=
//   2^-22.  Softmax: 2^-19 + |l - max| 2^-24 of the score (21 additions for 512
//   experts), taken for up to 30 below the maximum.
//   Softmax beside a bias, in units of 2^-24 of the largest score.  Each value:
//   e^-a (4 for the exponential + a for its argument, a = max - l, + 1 for the
//   product) <= 5.  The common divisor: 4 for the exponentials, at most 3.9 for
//   their arguments (sum of a e^-a over sum of e^-a, 511 experts at the worst a),
//   1 for the rounded sum, 2 for the reciprocal: 10.9, but it moves two values by
//   that times their difference.  Two values so come out in order from 2 * 5 +
//   10.9 = 20.9 units (1.25e-6) apart, where 2 * 7.5e-7 is taken, and two sums of
//   two from 4 * 5 + 2 * 10.9 (2.5e-6), where twice that is.  The bias' addition
//   and that of a group's two: 2^-24 of the choice value each, 2^-23 taken.
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Sum of a softmax's exponentials in fp64, four of a lane's in flight.
template <int NI, typename T>
__device__ __noinline__ double softmax_sum(const T* __restrict__ row, const RouteParams& p, int lane, float top) {
    constexpr int C = NI < 4 ? NI : 4;
    double sum = 0.0;
    #pragma unroll 1
    for (int i = 0; i < NI; i += C) {
        float l[C];
        #pragma unroll
        for (int j = 0; j < C; ++j) {
            const int e = (i + j) * 32 + lane;
            l[j] = e < p.E ? logit_of(to_float(row[e])) : -CUDART_INF_F;
        }
        #pragma unroll
        for (int j = 0; j < C; ++j) sum += exp((double)l[j] - (double)top);
    }
    return warp_sum(sum);
}
template <int NI, typename T>
__device__ __forceinline__ void route_token(const T* __restrict__ row, const RouteParams& p, int lane, int& my_e,
                                            float& my_w) {
    uint32_t key[NI];
    float top = -CUDART_INF_F, inv = 0.0f, big = 0.0f;         // big: largest |choice value| or score
    const float rel = p.sigmoid ? 4.2e-7f : 4.0e-6f;
    {
        float s[NI];
        load_logits<NI>(row, p, lane, s);
        uint32_t on = 0;                                       // experts that are not masked
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            on |= (s[i] > -CUDART_INF_F ? 1u : 0u) << i;
            top = fmaxf(top, s[i]);
        }
        if (!p.sigmoid) {
            #pragma unroll
            for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            #pragma unroll
            for (int i = 0; i < NI; ++i) s[i] = (on >> i) & 1u ? expf(s[i] - top) : 0.0f;
            // Beside a bias the sum's error counts too: there it is taken in fp64.
            if (p.bias != nullptr) {
                double sum = 0.0;
                #pragma unroll
                for (int i = 0; i < NI; ++i) sum += (double)s[i];
                sum = warp_sum(sum);
                inv = sum > 0.0 ? rcp_approx((float)sum) : 0.0f;
            } else {
                float sum = 0.0f;
                #pragma unroll
                for (int i = 0; i < NI; ++i) sum += s[i];
                #pragma unroll
                for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                inv = sum > 0.0f ? rcp_approx(sum) : 0.0f;
            }
            #pragma unroll
            for (int i = 0; i < NI; ++i) s[i] *= inv;
        } else {
            #pragma unroll
            for (int i = 0; i < NI; ++i) s[i] = rcp_approx(1.0f + expf(-s[i]));
        }
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane * NI + i;
            const float c = p.bias != nullptr && e < p.E ? s[i] + __ldg(p.bias + e) : s[i];
            const bool ok = ((on >> i) & 1u) && c > -CUDART_INF_F;
            key[i] = ok ? order_key(c) : 0u;
            if (ok) big = fmaxf(big, fmaxf(s[i], fabsf(c)));
        }
    }
    bool sure = true;
    float slack = 0.0f;                                        // two errors of any choice value
    if (p.bias != nullptr || p.kept < p.groups) {
        big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
        const float err = p.sigmoid ? 2.4e-7f : p.bias != nullptr ? 7.5e-7f * inv : rel * big;
        slack = 2.0f * (err + 1.2e-7f * big);
        sure = big < 1e30f;
    }
    if (p.kept < p.groups) {
        const int per = p.E / p.groups;
        uint32_t mine = 0;                                     // lane g: group g's score
        const bool whole = per % NI == 0 && ((per / NI) & (per / NI - 1)) == 0;
        if (whole) {
            // Groups of whole lanes, a power of two of them.
            uint32_t k1 = 0, k2 = 0;
            #pragma unroll
            for (int i = 0; i < NI; ++i) {
                k2 = max(k2, min(k1, key[i]));
                k1 = max(k1, key[i]);
            }
            const int lanes = per / NI;
            for (int off = 1; off < lanes; off <<= 1) {
                const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, off), o2 = __shfl_xor_sync(0xffffffffu, k2, off);
                k2 = max(max(k2, o2), min(k1, o1));
                k1 = max(k1, o1);
            }
            if (p.group_top > 1 && k2 != 0) k1 = order_key(key_value(k1) + key_value(k2));
            mine = __shfl_sync(0xffffffffu, k1, (lane * lanes) & 31);
        } else {
            for (int g = 0; g < p.groups; ++g) {
                uint32_t k1 = 0, k2 = 0;
                #pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const uint32_t q = (lane * NI + i) / per == g ? key[i] : 0u;
                    k2 = max(k2, min(k1, q));
                    k1 = max(k1, q);
                }
                const uint32_t t1 = __reduce_max_sync(0xffffffffu, k1);
                // The second: the winner's lane (one of them) offers its other.
                const unsigned has = __ballot_sync(0xffffffffu, k1 == t1);
                const uint32_t t2 = __reduce_max_sync(0xffffffffu, lane == __ffs(has) - 1 ? k2 : k1);
                uint32_t q = t1;
                if (p.group_top > 1 && t2 != 0) q = order_key(key_value(t1) + key_value(t2));
                if (lane == g) mine = q;
            }
        }
        if (lane >= p.groups) mine = 0;
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const uint32_t o = __shfl_sync(0xffffffffu, mine, g);
            rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
        }
        bool in = mine != 0 && rank < p.kept;
        const uint32_t least = __reduce_min_sync(0xffffffffu, in ? mine : 0xFFFFFFFFu);
        const uint32_t next = __reduce_max_sync(0xffffffffu, in ? 0u : mine);
        if (next != 0 && !(key_value(least) - key_value(next) > 2.0f * slack)) {
            if (whole && (p.sigmoid || p.bias == nullptr)) in = groups_exact<NI>(row, p, lane, key, top, slack, sure);
            else sure = false;
        }
        const unsigned kept = __ballot_sync(0xffffffffu, in);
        if (whole) {                                           // (a lane's experts are one group's)
            if (((kept >> (lane * NI / per)) & 1u) == 0) {
                #pragma unroll
                for (int i = 0; i < NI; ++i) key[i] = 0;
            }
        } else {
            #pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane * NI + i;
                if (e < p.E && ((kept >> (e / per)) & 1u) == 0) key[i] = 0;
            }
        }
    }
    // Candidates in order, the j-th to lane j: k of them, and on to the first
    // that is certainly below.  Every lane sorts its keys and offers the first,
    // the winner's lane moves on.  Without a bias the order is that of the scores, whose errors
    // are relative: no score below has a larger one.
    const float step = 2.0f * rel;
    int cand = -1, m = 0;
    float my_c = 0.0f, last = 0.0f;
    uint32_t at[NI];
    #pragma unroll
    for (int i = 0; i < NI; ++i) at[i] = lane * NI + i;
    sort_keys<NI>(key, at);
    for (; m < 32; ++m) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
        if (best == 0) break;
        const float c = key_value(best);
        if (m >= p.k && last - c > (p.bias != nullptr ? slack : step * last)) break;
        last = c;
        const int from = __ffs(__ballot_sync(0xffffffffu, key[0] == best)) - 1;
        const int win = __shfl_sync(0xffffffffu, at[0], from);
        if (lane == m) { cand = win; my_c = c; }
        const bool mine = lane == from;
        #pragma unroll
        for (int i = 0; i + 1 < NI; ++i) {
            key[i] = mine ? key[i + 1] : key[i];
            at[i] = mine ? at[i + 1] : at[i];
        }
        if (mine) key[NI - 1] = 0;
    }
    sure = sure && (m < 32 || p.E <= 32);
    float l = 0.0f, bias = 0.0f;
    if (cand >= 0) {
        l = logit_of(to_float(row[cand]));
        if (p.bias != nullptr) bias = __ldg(p.bias + cand);
    }
    const float c0 = __shfl_up_sync(0xffffffffu, my_c, 1), l0 = __shfl_up_sync(0xffffffffu, l, 1);
    const float b0 = __shfl_up_sync(0xffffffffu, bias, 1);
    const int e0 = __shfl_up_sync(0xffffffffu, cand, 1);
    const bool near = lane > 0 && lane < m && !(l == l0 && bias == b0 && e0 < cand) &&
                      !(c0 - my_c > (p.bias != nullptr ? slack : step * c0));
    // The candidates' scores in fp64, one exponential per lane: the weights are
    // made of them.  A softmax's common divisor is still left out.
    double s = 0.0;
    if (cand >= 0) s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top);
    if (__any_sync(0xffffffffu, near)) {
        // Each candidate's rank by its fp64 value.  (The divisor changes no order.)
        sure = sure && (p.sigmoid || p.bias == nullptr);
        const double c = s + (double)bias;
        int rank = lane < m ? 0 : 32;
        for (int j = 0; j < m; ++j) {
            const double o = __shfl_sync(0xffffffffu, c, j);
            const int oe = __shfl_sync(0xffffffffu, cand, j);
            if (lane < m && (o > c || (o == c && oe < cand))) ++rank;
        }
        int src = 31;
        for (int j = 0; j < m; ++j)
            if (__shfl_sync(0xffffffffu, rank, j) == lane) src = j;
        const int e = __shfl_sync(0xffffffffu, cand, src);
        l = __shfl_sync(0xffffffffu, l, src);
        s = __shfl_sync(0xffffffffu, s, src);
        cand = lane < m ? e : -1;
    }
    const bool mine = lane < p.k && cand >= 0;
    sure = sure && !(mine && (s < 1e-30 || (!p.sigmoid && l < top - 30.0f)));
    if (!__all_sync(0xffffffffu, sure)) {
        route_exact<NI>(row, p, lane, my_e, my_w);
        return;
    }
    // Renormalised weights need the chosen scores alone, a softmax's others the
    // sum over all experts.  The scale is a double, and may lie outside of fp32
    // where the weight does not: one rounding at the end.
    double sum = 1.0;
    if (p.renorm) sum = warp_sum(mine ? s : 0.0);
    else if (!p.sigmoid) sum = softmax_sum<NI>(row, p, lane, top);
    my_e = mine ? cand : -1;
    my_w = (float)(mine && sum > 0.0 ? s / sum * p.scale : 0.0);
}

// (Registers limited for occupancy: only route_exact() would take more.)  Bound
// by issue and latency of about 900 instructions a token: 45 % of the issue slots
// in a cold launch of 20 us, about 65 % of them in a stream of calls.  8192 tokens,
// 256 experts 12 us, with groups 14 us (21 us with groups on the border left to
// route_exact(), whose last token the launch waits for).
// Everything in fp64 and by shuffles it took 62 us.
template <typename T, int NI>
__global__ void __launch_bounds__(256, 4) route_topk_kernel(const T* __restrict__ logits, RouteParams p) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.T) return;
    int e;
    float w;
    route_token<NI>(logits + (int64_t)t * p.ld, p, lane, e, w);
    if (lane < p.k) {
        p.idx[(int64_t)t * p.k + lane] = e;
        p.weights[(int64_t)t * p.k + lane] = w;
    }
}

// ---------------------------------------------------------------------------
// The plan: slots (t, j) in the order of t * k + j, sorted stably by expert.
//   offsets[e]    first row of expert e, offsets[E] the rows in use
//   row_token[r]  token of row r (-1 from offsets[E] on)
//   slot_row[s]   row of slot s (-1 for a slot without an expert)
// CTAS CTAs of a cluster (or one) count their shares of the slots per warp and
// expert in shared memory, the counts of the CTAs before come over distributed
// shared memory, and each slot's row is the expert's start + the earlier CTAs'
// and warps' counts + its place in the warp.  Counts are added by atomics, but
// no atomic orders the result: it is the same on every run.  65536 slots of 256
// experts take 9 us, mostly scattered 4-byte stores (15 us on 8 CTAs).
// ---------------------------------------------------------------------------
template <int CTAS>
__device__ __forceinline__ void plan_sync() {
    if constexpr (CTAS > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
        __syncthreads();
}

template <int CTAS>
__device__ __forceinline__ void route_plan(const int32_t* idx, int slots, int k, int E, int32_t* __restrict__ offsets,
                                           int32_t* __restrict__ row_token, int32_t* __restrict__ slot_row,
                                           int32_t* smem) {
    using namespace route;
    constexpr int STEPS = 8;                          // steps of 32 slots whose loads are in flight together
    int32_t* total = smem;                            // [E] this CTA's counts
    int32_t* start = total + MAX_E;                   // [E] first row of each expert's slots in this CTA
    int32_t* part = start + MAX_E;                    // [32] sums of 32 experts
    int32_t* cnt = part + 32;                         // [PLAN_WARPS][E], zero: counts, then starts within the CTA
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t rank = 0;
    if constexpr (CTAS > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int steps = (slots + 31) / 32;
    const int per_cta = (steps + CTAS - 1) / CTAS, per_warp = (per_cta + PLAN_WARPS - 1) / PLAN_WARPS;
    const int c0 = min(steps, (int)rank * per_cta), c1 = min(steps, c0 + per_cta);
    const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);
    int32_t* mine = cnt + warp * E;
    int ex[STEPS];
    auto load = [&](int st) {
        #pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int s = (st + i) * 32 + lane;
            ex[i] = st + i < w1 && s < slots ? idx[s] : -1;
            if (ex[i] >= E) ex[i] = -1;
        }
    };
    for (int st = w0; st < w1; st += STEPS) {
        load(st);
        #pragma unroll
        for (int i = 0; i < STEPS; ++i)
            if (ex[i] >= 0) atomicAdd(mine + ex[i], 1);
    }
    __syncthreads();
    static_assert(PLAN_THREADS >= MAX_E, "a thread per expert");
    const int e = threadIdx.x;
    int run = 0;
    if (e < E) {
        #pragma unroll
        for (int w = 0; w < PLAN_WARPS; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        total[e] = run;
    }
    plan_sync<CTAS>();
    // Counts of the earlier CTAs and of all of them, and the scan over experts.
    int before = 0, all = run;
    if constexpr (CTAS > 1) {
        if (e < E) {
            int v[CTAS];
            #pragma unroll
            for (int c = 0; c < CTAS; ++c) {
                uint32_t a;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(total + e)), "r"(c));
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[c]) : "r"(a) : "memory");
            }
            all = 0;
            #pragma unroll
            for (int c = 0; c < CTAS; ++c) {
                before += c < (int)rank ? v[c] : 0;
                all += v[c];
            }
        }
    }
    int incl = all;
    #pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int rows = 0;                                     // rows before this warp's experts, then in use
    #pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) {
        const int v = part[w];
        if (w < warp) incl += v;
        rows += v;
    }
    if (e < E) {
        start[e] = incl - all + before;
        if (rank == 0) offsets[e] = incl - all;
    }
    if (rank == 0 && threadIdx.x == 0) offsets[E] = rows;
    __syncthreads();
    for (int64_t r = rows + (int64_t)rank * PLAN_THREADS + threadIdx.x; r < slots; r += PLAN_THREADS * CTAS)
        row_token[r] = -1;                            // rows without a slot
    for (int st = w0; st < w1; st += STEPS) {
        if (per_warp > STEPS) load(st);               // else the first pass's are still here
        #pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (st + i >= w1) break;
            const int s = (st + i) * 32 + lane;
            const unsigned same = __match_any_sync(0xffffffffu, ex[i]);
            int r = -1;
            if (ex[i] >= 0) r = start[ex[i]] + mine[ex[i]] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (ex[i] >= 0 && lane == __ffs(same) - 1) mine[ex[i]] += __popc(same);
            __syncwarp();
            if (s < slots) {
                slot_row[s] = r;
                if (r >= 0) row_token[r] = s / k;
            }
        }
    }
    // No CTA leaves while another may still read its counts.
    if constexpr (CTAS > 1) plan_sync<CTAS>();
}

// Zeroes the counts of route_plan (before its barrier; may run ahead of the inputs).
__device__ __forceinline__ void route_plan_clear(int32_t* smem, int E) {
    int32_t* cnt = smem + 2 * route::MAX_E + 32;
    for (int i = threadIdx.x; i < route::PLAN_WARPS * E; i += route::PLAN_THREADS) cnt[i] = 0;
    __syncthreads();
}

constexpr int route_plan_smem(int E) { return (2 * route::MAX_E + 32 + route::PLAN_WARPS * E) * 4; }

__global__ void __launch_bounds__(route::PLAN_THREADS)
route_plan_kernel(const int32_t* idx, int slots, int k, int E, int32_t* __restrict__ offsets,
                  int32_t* __restrict__ row_token, int32_t* __restrict__ slot_row) {
    extern __shared__ int32_t plan_smem[];
    route_plan_clear(plan_smem, E);
    grid_dependency_wait();
    grid_dependents_launch();
    route_plan<route::PLAN_CLUSTER>(idx, slots, k, E, offsets, row_token, slot_row, plan_smem);
}

// Choice and plan of up to SMALL_T tokens in one CTA: one launch for a decode step.
template <typename T, int NI>
__global__ void __launch_bounds__(route::PLAN_THREADS)
route_small_kernel(const T* __restrict__ logits, RouteParams p, int32_t* __restrict__ offsets,
                   int32_t* __restrict__ row_token, int32_t* __restrict__ slot_row) {
    using namespace route;
    extern __shared__ int32_t plan_smem[];
    __shared__ int32_t chosen[SMALL_T * MAX_K];
    route_plan_clear(plan_smem, p.E);
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    for (int t = threadIdx.x >> 5; t < p.T; t += PLAN_WARPS) {
        int e;
        float w;
        route_token<NI>(logits + (int64_t)t * p.ld, p, lane, e, w);
        if (lane < p.k) {
            chosen[t * p.k + lane] = e;
            p.idx[(int64_t)t * p.k + lane] = e;
            p.weights[(int64_t)t * p.k + lane] = w;
        }
    }
    __syncthreads();
    route_plan<1>(chosen, p.T * p.k, p.k, p.E, offsets, row_token, slot_row, plan_smem);
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
// token's rows and weights, and the loads of J rows are in flight together
// (predicated: a branch would wait for each).  V = 16 bytes of T
// where every row of Y and out allows it, else 1.  4096 tokens of 4 rows of 4096
// bf16: 29.4 us, 0.87 of the measured HBM rate; odd rows, one element per load,
// 43 us.
constexpr int kCombineThreads = 256;
template <typename T, typename O, int V, int C, int J>
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
