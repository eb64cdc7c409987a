// Expert choice by scores with a selection bias and groups of experts:
//   s = sigmoid(z) or softmax(z),  c = s + bias;
//   the topk_groups groups of largest (sum of two best c | best c);
//   the topk experts of largest c in them;  w = s / sum s * scale.
//
// One warp per token.  The lanes are dealt to the groups (32 / groups lanes
// each, groups rounded up to a power of two), and every lane keeps its experts'
// logits and choice values in registers, so that a group's two best values are
// a few shuffles and the top-k is one warp maximum per choice.
//
// The chosen experts are those of exact scores.  Scores are computed in 32
// bits with a known error; where two neighbours in the order (of groups or of
// experts) are closer than that error and not equal by their inputs, the warp
// makes the token's choice again with 64-bit scores.  Without a bias the order
// of the experts is the order of the logits themselves, which is exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "block.h"
#include "ptx.cuh"

namespace wna16 {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kWarps = 8;   // tokens per block

// Order-preserving map of a float (no NaN) to unsigned, above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 as 0
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float sigmoid_of(float z) { return 1.0f / (1.0f + expf(-z)); }

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Which experts a lane holds: its group's experts at position pos(i) of the
// group, i < PL, four neighbours at a time.
struct Lanes {
    int per_group;   // lanes of a group
    int group;       // this lane's group (>= groups: an idle lane)
    int sub;         // lane within the group
    int size;        // experts per group
    bool live;
    __device__ __forceinline__ Lanes(int E, int groups) {
        int g2 = 1;
        while (g2 < groups) g2 <<= 1;
        per_group = 32 / g2;
        const int lane = threadIdx.x & 31;
        group = lane / per_group;
        sub = lane & (per_group - 1);
        size = E / groups;
        live = group < groups;
    }
    __device__ __forceinline__ int pos(int i) const { return (i >> 2) * 4 * per_group + sub * 4 + (i & 3); }
    __device__ __forceinline__ bool has(int i) const { return live && pos(i) < size; }
    __device__ __forceinline__ int expert(int i) const { return group * size + pos(i); }
};

// The softmax's shift and the sum of its exponentials over all experts.
// With no logit above -inf all scores are 0.
template <int PL>
__device__ __forceinline__ void softmax_of(const Lanes& L, const float (&z)[PL], float& m, float& total) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PL; ++i) m = fmaxf(m, z[i]);
    m = key_value(__reduce_max_sync(kAll, order_key(m)));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i)
        if (L.has(i) && m > -INFINITY) sum += z[i] == m ? 1.0f : expf(z[i] - m);
    total = warp_sum(sum);
}

__device__ __forceinline__ float score_of(float z, bool softmax, float m, float total) {
    if (!softmax) return sigmoid_of(z);
    if (!(m > -INFINITY)) return 0.0f;
    return (z == m ? 1.0f : expf(z - m)) / total;
}

// The token's choice with 64-bit scores: lane j gets choice j's expert and
// logit.  z: the lane's n logits.  Rarely run, so kept small: its arrays are in
// local memory and its loops are not unrolled.
constexpr int kMaxPerLane = 64;
__device__ __noinline__ void choose64(const ScoredRouteParams& p, const float* z, int n, int& my_id, float& my_z) {
    const Lanes L(p.E, p.groups);
    const int lane = threadIdx.x & 31;
    double total = 0.0;
    float m = -INFINITY;
    if (p.softmax) {
        for (int i = 0; i < n; ++i) m = fmaxf(m, z[i]);
        m = key_value(__reduce_max_sync(kAll, order_key(m)));
    }
    double c[kMaxPerLane];
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        c[i] = -INFINITY;
        if (!L.has(i)) continue;
        // sigmoid: 1 / (1 + exp(-z)); softmax: exp(z - m), divided below
        const double e = p.softmax && z[i] == m ? 1.0 : exp(p.softmax ? static_cast<double>(z[i]) - static_cast<double>(m) : -static_cast<double>(z[i]));
        c[i] = !p.softmax ? 1.0 / (1.0 + e) : m > -INFINITY ? e : 0.0;
        total += c[i];
    }
    total = p.softmax && m > -INFINITY ? warp_sum(total) : 1.0;
    double b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        if (!L.has(i)) continue;
        c[i] = c[i] / total + (p.bias ? static_cast<double>(p.bias[L.expert(i)]) : 0.0);
        if (c[i] > b0) {
            b1 = b0;
            b0 = c[i];
        } else if (c[i] > b1) {
            b1 = c[i];
        }
    }
    uint64_t taken = 0;
    if (p.topk_groups < p.groups) {
        for (int o = 1; o < L.per_group; o <<= 1) {
            const double a0 = __shfl_xor_sync(kAll, b0, o), a1 = __shfl_xor_sync(kAll, b1, o);
            b1 = b0 > a0 ? (b1 > a0 ? b1 : a0) : (a1 > b0 ? a1 : b0);
            b0 = b0 > a0 ? b0 : a0;
        }
        const double gs = p.group_max || L.size < 2 ? b0 : b0 + b1;
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const double o = __shfl_sync(kAll, gs, g * L.per_group);
            rank += o > gs || (o == gs && g < L.group);
        }
        if (rank >= p.topk_groups) taken = ~0ull;
    }
    constexpr int kNone = 0x7fffffff;
#pragma unroll 1
    for (int j = 0; j < p.topk; ++j) {
        double bv = -INFINITY;
        int bi = kNone, at = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (L.has(i) && !((taken >> i) & 1) && (bi == kNone || c[i] > bv)) {
                bv = c[i];
                bi = L.expert(i);
                at = i;
            }
        }
        const int mine = bi;
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(kAll, bv, o);
            const int oi = __shfl_xor_sync(kAll, bi, o);
            if (oi != kNone && (bi == kNone || ov > bv || (ov == bv && oi < bi))) {
                bv = ov;
                bi = oi;
            }
        }
        const bool own = mine == bi;   // one lane: a candidate is always left (topk <= topk_groups * size)
        if (own) taken |= 1ull << at;
        const float zv = __shfl_sync(kAll, z[at], __ffs(__ballot_sync(kAll, own)) - 1);
        if (lane == j) {
            my_id = bi;
            my_z = zv;
        }
    }
}

template <typename T>
__device__ __forceinline__ float logit_of(T v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else if constexpr (std::is_same<T, __half>::value)
        return __half2float(v);
    else
        return __bfloat162float(v);
}

template <typename T, int PL>
__global__ void __launch_bounds__(32 * kWarps) route_scored_kernel(const ScoredRouteParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= p.T) return;   // whole warps leave together
    const Lanes L(p.E, p.groups);
    const T* row = static_cast<const T*>(p.logits) + static_cast<int64_t>(t) * p.ld;

    float z[PL];
#pragma unroll
    for (int i = 0; i < PL; i += 4) {
        if (p.vec && L.has(i)) {
            alignas(16) T e[4];
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<uint4*>(e) = __ldg(reinterpret_cast<const uint4*>(row + L.expert(i)));
            else
                *reinterpret_cast<uint2*>(e) = __ldg(reinterpret_cast<const uint2*>(row + L.expert(i)));
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i + j] = logit_of(e[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i + j] = !p.vec && L.has(i + j) ? logit_of(row[L.expert(i + j)]) : -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
        if (!(z[i] == z[i])) z[i] = -INFINITY;   // NaN: never preferred

    float m = 0.0f, total = 1.0f;
    if (p.softmax) {
        softmax_of<PL>(L, z, m, total);
        if (m == INFINITY) {   // infinite logits share the whole weight; the others' scores are 0
#pragma unroll
            for (int i = 0; i < PL; ++i) z[i] = z[i] == m ? 0.0f : -INFINITY;
            m = 0.0f;
        }
    }
    const bool pick_groups = p.topk_groups < p.groups;
    const bool by_logit = p.bias == nullptr;       // the experts' order is the logits' order
    // choice values; with by_logit needed for the sums of groups only
    const bool need_c = !by_logit || (pick_groups && !p.group_max);
    float c[PL];
    float big = 0.0f;   // largest magnitude among scores and choice values
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        c[i] = z[i];
        if (need_c) {
            c[i] = -INFINITY;
            if (L.has(i)) {
                const float s = score_of(z[i], p.softmax, m, total);
                c[i] = p.bias ? s + __ldg(p.bias + L.expert(i)) : s;
                big = fmaxf(big, fmaxf(s, fabsf(c[i])));
            }
        }
    }
    // Two choice values closer than tol may be in either order.  Sigmoid: a
    // score's error is at most 5 units of 2^-24, a sum's rounding one more, for
    // each of the two; softmax: besides, the shifted logit's rounding (at most
    // 0.37 units after the exponential) and the error of the total, a sum of up
    // to PL + 5 roundings.
    big = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(big)));
    const float tol = big * (p.softmax ? static_cast<float>(2 * PL + 32) * 0x1p-24f : 0x1p-20f);
    bool unsure = false;

    bool out = !L.live;
    if (pick_groups) {
        const bool by_c = need_c;
        float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const float v = L.has(i) ? c[i] : -INFINITY;
            b1 = fmaxf(b1, fminf(b0, v));
            b0 = fmaxf(b0, v);
        }
        for (int o = 1; o < L.per_group; o <<= 1) {
            const float a0 = __shfl_xor_sync(kAll, b0, o), a1 = __shfl_xor_sync(kAll, b1, o);
            b1 = fmaxf(fmaxf(b1, a1), fminf(b0, a0));
            b0 = fmaxf(b0, a0);
        }
        const float gs = p.group_max || L.size < 2 ? b0 : b0 + b1;
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float o = __shfl_sync(kAll, gs, g * L.per_group);
            rank += o > gs || (o == gs && g < L.group);
        }
        if (rank >= p.topk_groups) out = true;
        if (by_c) {
            const uint32_t kept = L.live && rank < p.topk_groups ? order_key(gs) : 0xffffffffu;
            const uint32_t left = L.live && rank >= p.topk_groups ? order_key(gs) : 0u;
            unsure = key_value(__reduce_min_sync(kAll, kept)) - key_value(__reduce_max_sync(kAll, left)) <= 4.0f * tol;
        }
    }

    if (by_logit) {
#pragma unroll
        for (int i = 0; i < PL; ++i) c[i] = z[i];
    }
    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) key[i] = !out && L.has(i) ? order_key(c[i]) : 0u;

    int my_id = 0;
    float my_z = 0.0f;
    uint32_t last_key = 0, last_id = 0;
    float last_z = 0.0f;
    const int candidates = p.topk_groups * L.size;
    const int rounds = by_logit ? p.topk : min(p.topk + 1, candidates);   // one more, for the last one's margin
    for (int j = 0; j < rounds; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        }
        const uint32_t top = __reduce_max_sync(kAll, best);
        const uint32_t e = best == top ? static_cast<uint32_t>(L.expert(at)) : 0xffffffffu;
        const uint32_t id = __reduce_min_sync(kAll, e);
        float zv = 0.0f;
        const bool mine = e == id;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            if (i == at) {
                zv = z[i];
                if (mine) key[i] = 0u;
            }
        }
        zv = __shfl_sync(kAll, zv, __ffs(__ballot_sync(kAll, mine)) - 1);
        if (lane == j) {
            my_id = static_cast<int>(id);
            my_z = zv;
        }
        if (!by_logit) {
            // Equal inputs give equal scores in any precision, and their order is
            // the index's (but behind the last choice a third one may be as near).
            if (j > 0 && key_value(last_key) - key_value(top) <= tol)
                unsure = unsure || j == p.topk || last_z != zv || __ldg(p.bias + last_id) != __ldg(p.bias + id);
            last_key = top;
            last_id = id;
            last_z = zv;
        }
    }
    if (unsure) {
        float copy[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) copy[i] = z[i];
        choose64(p, copy, PL, my_id, my_z);
    }

    float w = lane < p.topk ? score_of(my_z, p.softmax, m, total) : 0.0f;
    if (p.renormalize) {
        const float sum = warp_sum(w);
        w = sum > 0.0f ? w / sum : 0.0f;
    }
    if (lane < p.topk) {
        p.ids[static_cast<int64_t>(t) * p.topk + lane] = my_id;
        p.weights[static_cast<int64_t>(t) * p.topk + lane] = w * p.scale;
    }
}

template <typename T>
cudaError_t launch_typed(const ScoredRouteParams& p, cudaStream_t s) {
    int g2 = 1;
    while (g2 < p.groups) g2 <<= 1;
    const int span = 4 * (32 / g2);                      // experts per four register slots of a group's lanes
    const int pl = (p.E / p.groups + span - 1) / span * 4;
    // few tokens: one warp per block, each on an SM of its own
    const int warps = p.T >= 2048 ? kWarps : 1;
    const dim3 grid(static_cast<unsigned>((p.T + warps - 1) / warps)), block(32 * warps);
    if (pl <= 4) return launch_pdl(route_scored_kernel<T, 4>, grid, block, 0, s, p);
    if (pl <= 8) return launch_pdl(route_scored_kernel<T, 8>, grid, block, 0, s, p);
    if (pl <= 16) return launch_pdl(route_scored_kernel<T, 16>, grid, block, 0, s, p);
    if (pl <= 32) return launch_pdl(route_scored_kernel<T, 32>, grid, block, 0, s, p);
    if (pl <= 64) return launch_pdl(route_scored_kernel<T, 64>, grid, block, 0, s, p);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_route_scored(int type, const ScoredRouteParams& p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    if (type == kBf16) return launch_typed<__nv_bfloat16>(p, s);
    if (type == kFp16) return launch_typed<__half>(p, s);
    return launch_typed<float>(p, s);
}

}  // namespace wna16
