// Expert choice by scores with a selection bias and groups of experts:
//   s = sigmoid(z) or softmax(z),  c = s + bias;
//   the topk_groups groups of largest (sum of two best c | best c);
//   the topk experts of largest c in them;  w = s / sum s * scale.
//
// One warp per token.  The lanes are dealt to the groups (32 / groups lanes
// each, groups rounded up to a power of two), and every lane keeps its experts'
// choice values in registers, so that a group's two best values are a few
// shuffles.  The top-k: the (k + 1)-th greatest of the lanes' maxima is a
// lower bound of the (k + 1)-th best value, the few values above it are dealt
// to the lanes, and each counts those above it.  (One warp maximum per choice,
// the way for the rare token with more than 64 values above the bound, takes
// about four times the instructions.)
//
// The chosen experts are those of exact scores.  Scores are computed in 32
// bits with a known error; where two neighbours in the order (of groups or of
// experts) are closer than the error of their own magnitudes and not equal by their
// inputs, the values in question, and only those, are computed again in 64 bits and
// ordered by them (all of the token's, where they are too many).  Without a bias the order of the experts is the order of the logits
// themselves, which is exact.
//
// Bound by latency: 1.3 us would read the logits of 8192 tokens of 256 experts, and 36 %
// of the issue slots are used; a token is one dependent chain, and its 2048 blocks are
// 1.7 waves.  Small cases are one launch, and a token that needs 64 bits takes some 8 us by
// itself (fp64 is slow on this chip).  Measured (us), 256 experts, 8 chosen, sigmoid
// with a bias and 4 of 8 groups: 4 tokens 2.8, 2048 6.9, 8192 10.5; without bias and
// groups 8192 6.6; with the softmax 19.4; with every token in 64 bits 122.  1024 experts,
// 32 chosen, with a bias: 8192 43.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "block.h"
#include "ptx.cuh"

namespace wna16 {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLowest = -3.402823466e38f;   // stands for -INFINITY among values that may be chosen
constexpr int kWarps = 4;   // tokens per block

// Order-preserving map of a float (no NaN) to unsigned, above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 as 0
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// 64 bits: the order of doubles as unsigned integers
__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double key_value64(uint64_t k) {
    return __longlong_as_double(static_cast<long long>(k ^ ((k >> 63) ? 1ull << 63 : ~0ull)));
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a minimum that a NaN wins
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A bias as a finite number (NaN: the lowest).  The 32-bit path takes biases as they
// are: a choice value of NaN or -INFINITY is not collected there, and a token with one
// of +INFINITY or with too few others is chosen in 64 bits, with these biases.
__device__ __forceinline__ float finite_bias(float b) { return fminf(fmaxf(b, kLowest), -kLowest); }

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
    int held;        // experts of this lane: i < held (positions grow with i)
    __device__ __forceinline__ explicit Lanes(const ScoredRouteParams& p) {
        per_group = 32 >> p.groups_log;
        const int lane = threadIdx.x & 31;
        group = lane >> (5 - p.groups_log);
        sub = lane & (per_group - 1);
        size = p.group_size;
        live = group < p.groups;
        const int block = 4 << (5 - p.groups_log);   // positions per four slots of the group's lanes
        const int rest = (size & (block - 1)) - 4 * sub;
        held = live ? (size >> (7 - p.groups_log)) * 4 + min(max(rest, 0), 4) : 0;
    }
    __device__ __forceinline__ int pos(int i) const { return (i >> 2) * 4 * per_group + sub * 4 + (i & 3); }
    __device__ __forceinline__ bool has(int i) const { return i < held; }
    __device__ __forceinline__ int expert(int i) const { return group * size + pos(i); }
};

// One token's logits and how its scores are made of them.  (Passed by value to the
// rare paths, which are not inlined: what they took by address would live in
// local memory on the common path too.)
struct Token {
    const ScoredRouteParams& p;
    int type;
    const void* row;
    bool infinite = false;   // softmax with logits of +inf: they share the whole weight, the others' scores are 0
    float m = 0.0f;          // softmax: the largest logit (-inf: all scores are 0)
    float total = 1.0f;      // softmax: sum of exp(z - m)

    __device__ __forceinline__ float clean(float z) const {
        if (!(z == z)) return -INFINITY;   // NaN: never preferred
        if (infinite) return z == INFINITY ? 0.0f : -INFINITY;
        return z;
    }
    __device__ __forceinline__ float logit(int e) const {
        if (type == kFp32) return clean(static_cast<const float*>(row)[e]);
        if (type == kFp16) return clean(__half2float(static_cast<const __half*>(row)[e]));
        return clean(__bfloat162float(static_cast<const __nv_bfloat16*>(row)[e]));
    }
    // Scores relative to a logit of `most` from here on: weights that are divided by their
    // sum do not depend on it, and keep their bits where the chosen ones are far below the largest.
    __device__ __forceinline__ void softmax_of(float most) {
        m = most;
        total = 1.0f;
    }
    // For the weights.
    __device__ __forceinline__ float score(float z) const {
        if (!p.softmax) return 1.0f / (1.0f + expf(-z));
        if (!(m > -INFINITY)) return 0.0f;
        return (z == m ? 1.0f : expf(z - m)) / total;
    }
    // 64-bit choice value; total64: the softmax's sum (any positive number without a bias: the order is the same)
    __device__ __forceinline__ double choice64(int e, double total64) const {
        const float z = logit(e);
        double s;
        if (!p.softmax)
            s = 1.0 / (1.0 + exp(-static_cast<double>(z)));
        else if (!(m > -INFINITY))
            s = 0.0;
        else
            s = (z == m ? 1.0 : exp(static_cast<double>(z) - static_cast<double>(m))) / total64;
        return p.bias ? s + static_cast<double>(finite_bias(p.bias[e])) : s;
    }
    __device__ __forceinline__ double total64() const {
        if (!p.softmax || !p.bias) return 1.0;
        double sum = 0.0;
#pragma unroll 1
        for (int e = threadIdx.x & 31; e < p.E; e += 32) {
            const float z = logit(e);
            if (m > -INFINITY) sum += z == m ? 1.0 : exp(static_cast<double>(z) - static_cast<double>(m));
        }
        return m > -INFINITY ? warp_sum(sum) : 1.0;
    }
};

// A warp's values under consideration: key << 32 | ~expert, so that the greater
// is the better one and, of equal keys, the lower expert's.  0: none.
constexpr int kMost = 64;   // values considered at a time, at most two per lane
struct alignas(16) Candidates {   // (v is read 16 bytes at a time, in every warp's copy)
    uint64_t v[kMost];
    uint2 found[kMost + 1];   // (value, expert) in no order; the last one takes what is too much
};
__device__ __forceinline__ uint64_t pack(uint32_t key, int expert) {
    return static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(expert);
}
__device__ __forceinline__ int expert_of(uint64_t v) { return static_cast<int>(~static_cast<uint32_t>(v)); }

// Collects the experts whose value is at least the lane's `bound`; their number, of
// which the first 64 are in c.v (the rest of it is 0).  A bound is kLowest at least:
// slots without an expert hold -INFINITY, and would index logits and biases past E.
// Of a lane with the bound kNone, which no value reaches (a logit of +INFINITY would
// reach +INFINITY), nothing is collected.
constexpr float kNone = __builtin_nanf("");
template <int PL>
__device__ __forceinline__ int collect(const Lanes& L, const float (&value)[PL], float bound, Candidates& c) {
    const int lane = threadIdx.x & 31;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) mine += value[i] >= bound ? 1 : 0;
    int at = mine;   // places of this lane's values: after those of the lanes below
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, at, o);
        if (lane >= o) at += v;
    }
    const int count = __shfl_sync(kAll, at, 31);
    at -= mine;
    __syncwarp();
    if (mine > 0) {
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            if (value[i] >= bound) {
                c.found[min(at, kMost)] = make_uint2(__float_as_uint(value[i]), static_cast<uint32_t>(L.expert(i)));
                ++at;
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < kMost; h += 32) {
        if (h > 0 && count <= 32) {
            c.v[lane + h] = 0ull;
            break;
        }
        const uint2 f = c.found[lane + h];
        c.v[lane + h] = lane + h < count ? pack(order_key(__uint_as_float(f.x)), static_cast<int>(f.y)) : 0ull;
    }
    __syncwarp();
    return count;
}

// How many of the first `count` values are greater than v.
__device__ __forceinline__ int rank_of(uint64_t v, const Candidates& c, int count) {
    int rank = 0;
    for (int j = 0; j < count; j += 4) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&c.v[j]), b = *reinterpret_cast<const ulonglong2*>(&c.v[j + 2]);
        rank += (a.x > v) + (a.y > v) + (b.x > v) + (b.y > v);
    }
    return rank;
}

// All of the token's choice with 64-bit scores: lane j gets choice j's expert.
// For tokens with more than 64 values in question; kept small (arrays in local
// memory, loops not unrolled).
constexpr int kMaxPerLane = 64;
__device__ __noinline__ int choose64(Token t, int n) {
    const ScoredRouteParams& p = t.p;
    const Lanes L(p);
    const int lane = threadIdx.x & 31;
    const double total = t.total64();
    uint64_t key[kMaxPerLane];
    uint64_t b0 = 0, b1 = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        key[i] = L.has(i) ? order_key64(t.choice64(L.expert(i), total)) : 0ull;
        if (key[i] > b0) {
            b1 = b0;
            b0 = key[i];
        } else if (key[i] > b1) {
            b1 = key[i];
        }
    }
    if (p.topk_groups < p.groups) {
        for (int o = 1; o < L.per_group; o <<= 1) {
            const uint64_t a0 = __shfl_xor_sync(kAll, b0, o), a1 = __shfl_xor_sync(kAll, b1, o);
            b1 = b0 > a0 ? (b1 > a0 ? b1 : a0) : (a1 > b0 ? a1 : b0);
            b0 = b0 > a0 ? b0 : a0;
        }
        const double gs = !L.live ? 0.0 : p.group_max || L.size < 2 ? key_value64(b0) : key_value64(b0) + key_value64(b1);
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const double o = __shfl_sync(kAll, gs, g * L.per_group);
            rank += o > gs || (o == gs && g < L.group);
        }
        if (rank >= p.topk_groups)
            for (int i = 0; i < n; ++i) key[i] = 0ull;
    }
    int my_id = 0;
#pragma unroll 1
    for (int j = 0; j < p.topk; ++j) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        }
        const uint64_t top = warp_max64(best);
        const uint32_t e = best == top && top != 0ull ? static_cast<uint32_t>(L.expert(at)) : kAll;
        const uint32_t id = __reduce_min_sync(kAll, e);
        if (e == id) key[at] = 0ull;
        if (lane == j) my_id = static_cast<int>(id);
    }
    return my_id;
}

// Whether this lane's group stays, when 32 bits cannot tell: gs is its score, off by
// `margin` at most, `kept` the decision so far, `lo` the least that a kept group's score
// may be and `hi` the most that another one's may be.  from: the last of the group's best
// two (one) values, -INFINITY if there are not as many.  Returns false if there are too many
// values to look at, or too few.
template <int PL>
__device__ __noinline__ bool settle_groups(Token t, Lanes L, const float* value, float gs, float margin, float lo, float hi,
                                           float from, Candidates& cand, bool& kept) {
    const ScoredRouteParams& p = t.p;
    const int lane = threadIdx.x & 31;
    const bool open = L.live && (kept ? gs - margin <= hi : gs + margin >= lo);
    if (__any_sync(kAll, open && !(from >= kLowest))) return false;
    const int open_kept = __popc(__ballot_sync(kAll, open && kept && L.sub == 0));   // places to give
    float v[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) v[i] = value[i];
    const int count = collect(L, v, open ? fmaxf(from - (p.bias ? margin : 0.0f), kLowest) : kNone, cand);   // what may be among them
    if (count > 32) return false;
    const double total = t.total64();
    const int e = lane < count ? expert_of(cand.v[lane]) : -1;
    const int my_group = e >= 0 ? e / L.size : -1;
    const uint64_t k = e >= 0 ? order_key64(t.choice64(e, total)) : 0ull;
    double sum = 0.0;   // of group `lane`
    for (int g = 0; g < p.groups; ++g) {
        const uint64_t v = my_group == g ? k : 0ull;
        const uint64_t first = warp_max64(v);
        if (first == 0ull) continue;   // not open
        double s = key_value64(first);
        if (!p.group_max && L.size >= 2) {
            const int owner = __ffs(__ballot_sync(kAll, v == first)) - 1;
            s += key_value64(warp_max64(lane == owner ? 0ull : v));
        }
        if (lane == g) sum = s;
    }
    const uint32_t open_mask = __ballot_sync(kAll, open && L.sub == 0);   // by the groups' first lanes
    const double mine = __shfl_sync(kAll, sum, L.live ? L.group : 0);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
        const double o = __shfl_sync(kAll, sum, g);
        if (open_mask >> (g * L.per_group) & 1u) rank += o > mine || (o == mine && g < L.group);
    }
    if (open) kept = rank < open_kept;
    return true;
}

// Sorts the `count` collected experts by their 64-bit values.
__device__ __noinline__ void settle_order(Token t, Candidates& cand, int count) {
    const int lane = threadIdx.x & 31;
    const double total = t.total64();
    int e[2], rank[2] = {0, 0};
    uint64_t k[2];
    for (int h = 0; h < 2; ++h) {
        const bool in = lane + 32 * h < count;
        e[h] = in ? expert_of(cand.v[lane + 32 * h]) : 0;
        k[h] = in ? order_key64(t.choice64(e[h], total)) : 0ull;
        if (count <= 32) break;
    }
    for (int j = 0; j < count; ++j) {
        const uint64_t ok = __shfl_sync(kAll, j < 32 ? k[0] : k[1], j & 31);
        const int oe = __shfl_sync(kAll, j < 32 ? e[0] : e[1], j & 31);
        rank[0] += ok > k[0] || (ok == k[0] && oe < e[0]);
        if (count > 32) rank[1] += ok > k[1] || (ok == k[1] && oe < e[1]);
    }
    __syncwarp();
    if (lane < count) cand.v[rank[0]] = pack(0u, e[0]);
    if (lane + 32 < count) cand.v[rank[1]] = pack(0u, e[1]);
    __syncwarp();
}

// Weights of a token with a sigmoid near or below fp32's smallest normal number (z: the
// lane's chosen logit, -INFINITY: none).  Where they will be divided by their sum they are
// taken relative to the largest, so that they keep their bits.  A logit below -709
// (softmax: 709 below the largest) scores 0, as where the score is computed in 64 bits:
// masks with a type's lowest value are down there, and share no weight among them.
__device__ __noinline__ float deep_sigmoid(float z, int renormalize) {
    const float most = key_value(__reduce_max_sync(kAll, order_key(z)));
    const float shift = renormalize ? fminf(most, 0.0f) : 0.0f;
    if (z < -709.0f) return 0.0f;
    return z < 0.0f ? expf(z - shift) / (1.0f + expf(z)) : 1.0f / (1.0f + expf(-z));
}

template <int PL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kWarps, PL <= 8 ? 8 : 1) route_scored_kernel(const __grid_constant__ ScoredRouteParams p, int type) {
    __shared__ Candidates shared[kWarps];
    static_assert(sizeof(Candidates) % 16 == 0, "every warp's copy is 16-byte aligned");
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int ti = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (ti >= p.T) return;   // whole warps leave together
    Candidates& cand = shared[threadIdx.x >> 5];
    const Lanes L(p);
    Token t{p, type, static_cast<const uint8_t*>(p.logits) + static_cast<int64_t>(ti) * p.ld * (type == kFp32 ? 4 : 2)};

    // logits, -INFINITY where the lane has no expert
    float z[PL];
    if (p.vec) {
        if (type == kFp32) {
            const float* row = static_cast<const float*>(t.row) + L.expert(0);
#pragma unroll
            for (int i = 0; i < PL; i += 4) {
                float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (L.has(i)) v = __ldg(reinterpret_cast<const float4*>(row + i * L.per_group));
                z[i] = v.x;
                z[i + 1] = v.y;
                z[i + 2] = v.z;
                z[i + 3] = v.w;
            }
        } else {
            const uint16_t* row = static_cast<const uint16_t*>(t.row) + L.expert(0);
            const uint32_t none = type == kFp16 ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
            for (int i = 0; i < PL; i += 4) {
                uint2 v = make_uint2(none, none);
                if (L.has(i)) v = __ldg(reinterpret_cast<const uint2*>(row + i * L.per_group));
                const uint32_t h[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    z[i + j] = type == kFp16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(h[j]))) : __uint_as_float(h[j] << 16);
            }
        }
#pragma unroll
        for (int i = 0; i < PL; ++i) z[i] = fmaxf(z[i], -INFINITY);   // NaN: -INFINITY, as Token::clean
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) z[i] = L.has(i) ? t.logit(L.expert(i)) : -INFINITY;
    }

    float bias[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) bias[i] = -INFINITY;   // no expert
    if (p.bias) {
        const float* src = p.bias + L.expert(0);
#pragma unroll
        for (int i = 0; i < PL; i += 4) {
            if (p.bias_vec) {
                if (L.has(i)) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(src + i * L.per_group));
                    bias[i] = v.x;
                    bias[i + 1] = v.y;
                    bias[i + 2] = v.z;
                    bias[i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (L.has(i + j)) bias[i + j] = __ldg(src + i * L.per_group + j);
            }
        }
    }

    constexpr float kLog2e = 1.44269504f;
    float top_score = 1.0f;   // no score is greater
    if constexpr (SOFTMAX) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) m = fmaxf(m, z[i]);
        t.m = key_value(__reduce_max_sync(kAll, order_key(m)));
        if (t.m == INFINITY) {
            t.infinite = true;
            t.m = 0.0f;
#pragma unroll
            for (int i = 0; i < PL; ++i) z[i] = t.clean(z[i]);
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) sum += t.m > -INFINITY ? exp2_approx((z[i] - t.m) * kLog2e) : 0.0f;   // (0 without an expert)
        t.total = warp_sum(sum);
        top_score = t.m > -INFINITY ? rcp_approx(t.total) : 0.0f;
    }
    auto fast_score = [&](float x) {   // with the fast exponential: see unit
        if constexpr (SOFTMAX)
            return exp2_approx((t.m > -INFINITY ? x - t.m : -INFINITY) * kLog2e) * top_score;
        else
            return rcp_approx(1.0f + exp2_approx(x * -kLog2e));
    };
    // What the experts are ordered by: choice values or, without a bias, the logits.
    // -INFINITY: no expert.
    const bool by_logit = p.bias == nullptr;
    float value[PL];
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < PL; ++i) value[i] = L.has(i) ? fmaxf(z[i], kLowest) : -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) value[i] = fast_score(z[i]) + bias[i];
    }
    // Two choice values that differ by at most unit times the greatest of the scores
    // and of their own magnitudes may be in either order.  Errors in units of
    // 2^-24 of that.  Sigmoid: the exponential's relative error is 4 and 1.5 |z| for
    // its argument's rounding, of which the score sees s (1 - s): 1 + 1.5 * 0.37;
    // the sum 1, the reciprocal 2, the bias 1; for both values 12.  Softmax: 4 and
    // at most 2.5 * 0.37 likewise, the reciprocal and product 3, the bias 1, and the
    // total's, a sum of up to PL + 5 roundings and its terms' 5; for both values.
    constexpr float unit = SOFTMAX ? static_cast<float>(2 * PL + 48) * 0x1p-24f : 24.0f * 0x1p-24f;

    float best = -INFINITY, second = -INFINITY;   // of the lane (a value of NaN is neither)
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        second = fmaxf(second, min_nan(best, value[i]));
        best = fmaxf(best, value[i]);
    }
    bool out = !L.live;
    bool all64 = !by_logit && __any_sync(kAll, best == INFINITY);
    if (!all64 && p.topk_groups < p.groups) {
        float b0 = best, b1 = second;             // of the group
        for (int o = 1; o < L.per_group; o <<= 1) {
            const float a0 = __shfl_xor_sync(kAll, b0, o), a1 = __shfl_xor_sync(kAll, b1, o);
            b1 = fmaxf(fmaxf(b1, a1), fminf(b0, a0));
            b0 = fmaxf(b0, a0);
        }
        const bool best_only = p.group_max || L.size < 2;
        const float from = best_only ? b0 : b1;
        if (by_logit && !best_only) {
            b0 = fast_score(b0);
            b1 = fast_score(b1);
        }
        const float gs = best_only ? b0 : b0 + b1;
        int rank = 0;
#pragma unroll 4
        for (int g = 0; g < p.groups; ++g) {
            const float o = __shfl_sync(kAll, gs, g << (5 - p.groups_log));
            rank += g < L.group ? o >= gs : o > gs;
        }
        bool kept = L.live && rank < p.topk_groups;
        if (!by_logit || !best_only) {   // (the best logits' order is exact)
            // Each group's score may be off by a margin of its own (a sum's error is twice a value's): with
            // one margin for all, a group masked by a bias of -1e9 brought every group's order in question.
            const float margin = unit * fmaxf(top_score, L.live ? fminf(fmaxf(fabsf(b0), best_only ? 0.0f : fabsf(b1)), -kLowest) : 0.0f);
            const float lo = key_value(__reduce_min_sync(kAll, kept ? order_key(gs - margin) : 0xffffffffu));
            const float hi = key_value(__reduce_max_sync(kAll, L.live && !kept ? order_key(gs + margin) : 0u));
            if (!(lo > hi)) {
                float copy[PL];
#pragma unroll
                for (int i = 0; i < PL; ++i) copy[i] = value[i];
                bool stays = kept;
                all64 = !settle_groups<PL>(t, L, copy, gs, margin, lo, hi, from, cand, stays);
                kept = stays;
            }
        }
        out = !kept;
    }

    int my_id = 0;
    if (all64) {
        my_id = choose64(t, PL);
    } else {
        // A bound that at least topk + 1 values (or all there are) reach: the lanes'
        // (topk + 1)-th greatest maximum, or where that takes most of the lanes, the
        // (topk / 2 + 1)-th greatest second best, each of which has its lane's best above it.
        const bool seconds = 2 * (p.topk + 1) > p.topk_groups * L.per_group;
        uint32_t mine = out ? 0u : order_key(seconds ? second : best), top = 0u;
        for (int j = seconds ? p.topk / 2 : p.topk; j >= 0; --j) {
            top = __reduce_max_sync(kAll, mine);
            if (mine == top) mine = 0u;   // (several lanes at once where values are equal)
        }
        const float bound = out ? kNone : top == 0u ? kLowest : fmaxf(key_value(top), kLowest);
        int count = collect(L, value, bound, cand);
        bool unsure = count < p.topk;   // (only by biases of NaN or -INFINITY)
        if (count <= kMost) {
            // sort: each value goes to the place of its rank
            const bool two = count > 32;
            uint64_t v = cand.v[lane], v2 = two ? cand.v[lane + 32] : 0ull;
            {
                const int rank = rank_of(v, cand, count), rank2 = two ? rank_of(v2, cand, count) : 0;
                __syncwarp();
                if (lane < count) cand.v[rank] = v;
                if (lane + 32 < count) cand.v[rank2] = v2;
                __syncwarp();
            }
            v = cand.v[lane];
            my_id = expert_of(v);
            if (!by_logit) {
                const uint64_t next = lane + 1 < count ? cand.v[lane + 1] : 0ull;
                const float mine = key_value(static_cast<uint32_t>(v >> 32));
                // Neighbours are compared by their own size: by the largest choice's, an expert that a bias
                // of 1e9 forces brought all the others' order in question.
                const float after = key_value(static_cast<uint32_t>(next >> 32));
                bool close = lane < p.topk && lane + 1 < count &&
                             mine - after <= unit * fmaxf(top_score, fmaxf(fabsf(mine), fabsf(after)));
                // Equal inputs give equal scores in any precision, and their order is the
                // index's (but behind the last choice a third one may be as near).
                if (close && lane + 1 < p.topk)
                    close = t.logit(my_id) != t.logit(expert_of(next)) || p.bias[my_id] != p.bias[expert_of(next)];
                if (__any_sync(kAll, close)) {
                    // every value that may be among the choices, in 64 bits
                    const float last = __shfl_sync(kAll, mine, p.topk - 1);
                    count = collect(L, value, out ? kNone : fmaxf(last - unit * fmaxf(top_score, fabsf(last)), kLowest), cand);
                    if (count <= kMost) {
                        settle_order(t, cand, count);
                        my_id = expert_of(cand.v[lane]);
                    } else {
                        unsure = true;
                    }
                }
            }
        } else {
            // many values above the bound: one warp maximum per choice
            if (out) {
#pragma unroll
                for (int i = 0; i < PL; ++i) value[i] = -INFINITY;
            }
            float last = INFINITY, chosen = 0.0f;
            int last_id = 0;
            const int rounds = by_logit ? p.topk : min(p.topk + 1, p.topk_groups * L.size);   // one more, for the last one's margin
            for (int j = 0; j < rounds; ++j) {
                float top = -INFINITY;
                int at = 0;
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    if (value[i] > top) {
                        top = value[i];
                        at = i;
                    }
                }
                const uint32_t key = order_key(top), all = __reduce_max_sync(kAll, key);
                const uint32_t e = key == all && top > -INFINITY ? static_cast<uint32_t>(L.expert(at)) : kAll;
                const uint32_t id = __reduce_min_sync(kAll, e);
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    if (i == at && e == id && j < p.topk) value[i] = -INFINITY;
                if (lane == j) {
                    my_id = static_cast<int>(id);
                    chosen = key_value(all);
                }
                if (!by_logit) {
                    const float now = key_value(all);
                    if (j > 0 && last - now <= unit * fmaxf(top_score, fmaxf(fabsf(last), fabsf(now))))
                        unsure = unsure || j == p.topk || t.logit(last_id) != t.logit(static_cast<int>(id)) ||
                                 p.bias[last_id] != p.bias[id];
                    last = now;
                    last_id = static_cast<int>(id);
                }
            }
            if (unsure) {   // the choices and what may be among them, in 64 bits
                const float least = __shfl_sync(kAll, chosen, p.topk - 1);
                const int more = collect(L, value, out ? kNone : fmaxf(least - unit * fmaxf(top_score, fabsf(least)), kLowest), cand);
                if (more + p.topk <= kMost) {
                    if (lane < p.topk) cand.v[more + lane] = pack(0u, my_id);
                    __syncwarp();
                    settle_order(t, cand, more + p.topk);
                    my_id = expert_of(cand.v[lane]);
                    unsure = false;
                }
            }
        }
        if (unsure) my_id = choose64(t, PL);
    }

    float z_mine = lane < p.topk ? t.logit(my_id) : -INFINITY;
    if (SOFTMAX && z_mine < t.m - 709.0f) z_mine = -INFINITY;   // a score of 0: see deep_sigmoid
    if (SOFTMAX && p.renormalize) t.softmax_of(key_value(__reduce_max_sync(kAll, order_key(z_mine))));
    float w = lane < p.topk ? t.score(z_mine) : 0.0f;
    if (!SOFTMAX && __any_sync(kAll, z_mine < -87.0f && z_mine > -INFINITY)) w = deep_sigmoid(z_mine, p.renormalize);
    if (p.renormalize) {
        const float sum = warp_sum(w);
        // (the fast division is not for sums near fp32's smallest)
        w = sum > 0x1p-100f ? __fdividef(w, sum) : sum > 0.0f ? w / sum : 0.0f;
    }
    if (lane < p.topk) {
        p.ids[static_cast<int64_t>(ti) * p.topk + lane] = my_id;
        p.weights[static_cast<int64_t>(ti) * p.topk + lane] = w * p.scale;
    }
}

template <bool SOFTMAX>
cudaError_t launch_score(int type, const ScoredRouteParams& p, cudaStream_t s) {
    const int span = 4 << (5 - p.groups_log);            // experts per four register slots of a group's lanes
    const int pl = (p.group_size + span - 1) / span * 4;
    // few tokens: one warp per block, each on an SM of its own
    const int warps = p.T >= 1024 ? kWarps : 1;
    const dim3 grid(static_cast<unsigned>((p.T + warps - 1) / warps)), block(32 * warps);
    if (pl <= 4) return launch_pdl(route_scored_kernel<4, SOFTMAX>, grid, block, 0, s, p, type);
    if (pl <= 8) return launch_pdl(route_scored_kernel<8, SOFTMAX>, grid, block, 0, s, p, type);
    if (pl <= 16) return launch_pdl(route_scored_kernel<16, SOFTMAX>, grid, block, 0, s, p, type);
    if (pl <= 32) return launch_pdl(route_scored_kernel<32, SOFTMAX>, grid, block, 0, s, p, type);
    if (pl <= kMaxPerLane) return launch_pdl(route_scored_kernel<64, SOFTMAX>, grid, block, 0, s, p, type);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_route_scored(int type, ScoredRouteParams p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    p.group_size = p.E / p.groups;
    p.groups_log = 0;
    while ((1 << p.groups_log) < p.groups) ++p.groups_log;
    return p.softmax ? launch_score<true>(type, p, s) : launch_score<false>(type, p, s);
}

}  // namespace wna16
