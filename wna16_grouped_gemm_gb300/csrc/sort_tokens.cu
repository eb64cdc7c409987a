// Tokens to rows in the order of their experts, and back.
//
//   inv[f]  = (slots of lower experts) + (earlier slots of the same expert)
//   rows[inv[f]] = x[t]                        f = t * topk + j
//   out[t]  = sum_j w[t][j] y[inv[t][j]]       (without w: the gradient of the line above)
//   dy[inv[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[inv[t][j]]>
//
// Bound by the bytes of the rows.  Sums are fp32, in an order that the sizes alone fix.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "f8.h"
#include "gemm.h"
#include "ptx.cuh"

namespace wna16 {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------ sort

constexpr int kSmallThreads = 256;
// Slots up to which every token counts its own positions, in one launch.
constexpr int kSmallSlots = 4096;

// One block per token, and one for the offsets.  A slot's row is the number of slots
// that sort before it; a warp counts them.  Experts are unsigned offsets from
// expert_begin, so ids below it are large numbers.
template <typename V>
__global__ void __launch_bounds__(kSmallThreads) sort_small_kernel(const SortParams p) {
    __shared__ int pos[1024];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned E = static_cast<unsigned>(p.E), begin = static_cast<unsigned>(p.expert_begin);
    const int R = static_cast<int>(p.T) * p.topk;
    const unsigned* ids = reinterpret_cast<const unsigned*>(p.ids);
    if (blockIdx.x == p.T) {
        for (int e = tid; e < 1024; e += kSmallThreads) pos[e] = 0;
        __syncthreads();
        for (int f = tid; f < R; f += kSmallThreads) {
            const unsigned e = __ldg(ids + f) - begin;
            if (e < E) atomicAdd(&pos[e], 1);
        }
        __syncthreads();
        // four experts per thread, warps' sums by the first warp
        __shared__ int sums[kSmallThreads / 32];
        int c[4], total = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = total;
            total += pos[tid * 4 + i];
        }
        int run = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kAll, run, d);
            if (lane >= d) run += o;
        }
        if (lane == 31) sums[warp] = run;
        __syncthreads();
        int before = run - total;
        for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (tid * 4 + i <= p.E) p.offsets[tid * 4 + i] = before + c[i];
        if (tid == kSmallThreads - 1 && p.E == 1024) p.offsets[1024] = before + total;
        return;
    }
    const int t = blockIdx.x;
    for (int j = warp; j < p.topk; j += kSmallThreads / 32) {
        const int f = t * p.topk + j;
        const unsigned e = __ldg(ids + f) - begin;
        int n = 0;
        if (e < E) {
            for (int i = lane; i < R; i += 32) {
                const unsigned o = __ldg(ids + i) - begin;
                n += o < e || (o == e && i < f);
            }
            n = __reduce_add_sync(kAll, n);
        } else {
            n = -1;
        }
        if (lane == 0) {
            pos[j] = n;
            p.inv[f] = n;
        }
    }
    if (!p.x) return;
    const int64_t n_vec = p.row_bytes / static_cast<int64_t>(sizeof(V));
    const V* src = reinterpret_cast<const V*>(static_cast<const char*>(p.x) + t * p.x_pitch);
    V* dst = static_cast<V*>(p.rows);
    __syncthreads();
    for (int64_t v = tid; v < n_vec; v += kSmallThreads) {
        const V a = src[v];
        for (int j = 0; j < p.topk; ++j)
            if (pos[j] >= 0) dst[pos[j] * n_vec + v] = a;
    }
    if (p.x_scales)
        for (int64_t v = tid; v < p.groups; v += kSmallThreads) {
            const float a = p.x_scales[t * p.groups + v];
            for (int j = 0; j < p.topk; ++j)
                if (pos[j] >= 0) p.row_scales[pos[j] * p.groups + v] = a;
        }
}

constexpr int kListThreads = 1024;
constexpr int kListWarps = kListThreads / 32;
constexpr int kListBlocks = 8;   // one cluster

// The lists of many slots, by one cluster: a stable counting sort.  Every warp has a run
// of slots and counts its experts; the blocks exchange their counts through distributed
// shared memory; then every warp places its slots.
__global__ void __launch_bounds__(kListThreads, 1) sort_lists_kernel(const SortParams p) {
    extern __shared__ int sm[];
    __shared__ int sums[kListWarps];
    const int E = p.E;
    int* hist = sm;                        // [kListWarps][E]
    int* table = hist + kListWarps * E;    // [kListBlocks][E]
    int* base = table + kListBlocks * E;   // [E]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const unsigned begin = static_cast<unsigned>(p.expert_begin);
    const unsigned* ids = reinterpret_cast<const unsigned*>(p.ids);
    pdl_wait();
    pdl_trigger();
    const int64_t R = p.T * p.topk;
    const int64_t per_warp = (R + kListBlocks * kListWarps * 32 - 1) / (kListBlocks * kListWarps * 32) * 32;
    const int64_t f0 = (rank * kListWarps + warp) * per_warp, f1 = min(R, f0 + per_warp);
    int* my = hist + warp * E;
    for (int e = lane; e < E; e += 32) my[e] = 0;
    __syncwarp();
    for (int64_t at = f0; at < f1; at += 32) {
        const int64_t f = at + lane;
        unsigned e = f < f1 ? __ldg(ids + f) - begin : ~0u;
        if (e >= static_cast<unsigned>(E)) e = ~0u;
        const unsigned peers = __match_any_sync(kAll, e);
        if (e != ~0u && lane == __ffs(peers) - 1) my[e] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    if (tid < E) {
        int c = 0;
#pragma unroll 8
        for (int w = 0; w < kListWarps; ++w) {
            const int v = hist[w * E + tid];
            hist[w * E + tid] = c;
            c += v;
        }
        const uint32_t at = smem_u32(table + rank * E + tid);
#pragma unroll
        for (int r = 0; r < kListBlocks; ++r)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_shared(at, r)), "r"(c) : "memory");
    }
    cluster_sync();
    int total = 0, before = 0;
    if (tid < E) {
#pragma unroll
        for (int r = 0; r < kListBlocks; ++r) {
            const int v = table[r * E + tid];
            if (r < rank) before += v;
            total += v;
        }
    }
    int run = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, run, d);
        if (lane >= d) run += o;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    const int s = __reduce_add_sync(kAll, lane < warp ? sums[lane] : 0);
    const int off = s + run - total;
    if (tid < E) {
        base[tid] = off + before;
        if (rank == 0) {
            p.offsets[tid] = off;
            if (tid == E - 1) p.offsets[E] = off + total;
        }
    }
    __syncthreads();
    const unsigned lower = (1u << lane) - 1u;
    for (int64_t at = f0; at < f1; at += 32) {
        const int64_t f = at + lane;
        unsigned e = f < f1 ? __ldg(ids + f) - begin : ~0u;
        if (e >= static_cast<unsigned>(E)) e = ~0u;
        const unsigned peers = __match_any_sync(kAll, e);
        const int pos = e != ~0u ? base[e] + my[e] + __popc(peers & lower) : -1;
        __syncwarp();
        if (e != ~0u && lane == __ffs(peers) - 1) my[e] += __popc(peers);
        __syncwarp();
        if (f < f1) p.inv[f] = pos;
    }
}

constexpr int kCopyWarps = 8;

// rows[inv[t][j]] = x[t]: a warp per token, which reads its row once.
template <typename V>
__global__ void __launch_bounds__(32 * kCopyWarps) sort_copy_kernel(const SortParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int64_t n_vec = p.row_bytes / static_cast<int64_t>(sizeof(V));
    const V* src = reinterpret_cast<const V*>(static_cast<const char*>(p.x) + t * p.x_pitch);
    V* dst = static_cast<V*>(p.rows);
    const int32_t* inv = p.inv + t * p.topk;
    for (int j0 = 0; j0 < p.topk; j0 += 32) {
        const int count = min(32, p.topk - j0);
        const int mine = lane < count ? __ldg(inv + j0 + lane) : -1;
        for (int64_t v0 = lane; v0 - lane < n_vec; v0 += 4 * 32) {   // the same turns for every lane
            V a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (v0 + c * 32 < n_vec) a[c] = __ldg(src + v0 + c * 32);
            for (int j = 0; j < count; ++j) {
                const int r = __shfl_sync(kAll, mine, j);
                if (r < 0) continue;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (v0 + c * 32 < n_vec) dst[r * n_vec + v0 + c * 32] = a[c];
            }
        }
        if (p.x_scales)
            for (int64_t v = lane; v - lane < p.groups; v += 32) {
                const float a = v < p.groups ? __ldg(p.x_scales + t * p.groups + v) : 0.0f;
                for (int j = 0; j < count; ++j) {
                    const int r = __shfl_sync(kAll, mine, j);
                    if (r >= 0 && v < p.groups) p.row_scales[r * p.groups + v] = a;
                }
            }
    }
}

template <typename V>
cudaError_t launch_sort(const SortParams& p, cudaStream_t s) {
    const int64_t R = p.T * p.topk;
    if (R <= kSmallSlots)
        return launch_pdl(sort_small_kernel<V>, dim3(static_cast<unsigned>(p.T + 1)), dim3(kSmallThreads), 0, s, p);
    const int smem = (kListWarps + kListBlocks + 1) * p.E * 4;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(sort_lists_kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kListBlocks);
    cfg.blockDim = dim3(kListThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kListBlocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, sort_lists_kernel, p);
    if (e != cudaSuccess || !p.x) return e;
    return launch_pdl(sort_copy_kernel<V>, dim3(static_cast<unsigned>((p.T + kCopyWarps - 1) / kCopyWarps)),
                      dim3(32 * kCopyWarps), 0, s, p);
}

// ------------------------------------------------------------------ back

constexpr int kV = 8;   // values per chunk
constexpr int kBackThreads = 256;
constexpr int kBatch = 8;   // rows read at the same time

template <typename T>
__device__ __forceinline__ float to_f(T v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else if constexpr (std::is_same<T, __half>::value)
        return __half2float(v);
    else
        return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else if constexpr (std::is_same<T, __half>::value)
        return __float2half_rn(v);
    else
        return __float2bfloat16_rn(v);
}

template <typename T>
struct alignas(16) Chunk {
    T v[kV];
};

// 8 values at p (n of them exist, the others are 0)
template <typename T, bool VEC>
__device__ __forceinline__ Chunk<T> load_chunk(const T* p, int64_t n) {
    Chunk<T> c;
    if (VEC) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(c) / 16); ++i)
            reinterpret_cast<uint4*>(c.v)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) c.v[i] = i < n ? p[i] : from_f<T>(0.0f);
    }
    return c;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* p, int64_t n, const Chunk<T>& c) {
    if (VEC) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(c) / 16); ++i)
            reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(c.v)[i];
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < n) p[i] = c.v[i];
    }
}

// A block per token and run of 2048 values; a thread has 8 of them.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kBackThreads) unsort_kernel(const UnsortParams p) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int64_t k = (static_cast<int64_t>(blockIdx.y) * kBackThreads + threadIdx.x) * kV;
    if (k >= p.K) return;
    const int64_t n = p.K - k;
    const T* y = static_cast<const T*>(p.y);
    float sum[kV] = {};
    for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
        Chunk<T> c[kBatch];
        float w[kBatch];
        bool used[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t f = t * p.topk + j0 + i;
            const int64_t r = j0 + i < p.topk ? __ldg(p.inv + f) : -1;
            used[i] = r >= 0 && r < p.R;
            if (used[i]) {
                w[i] = p.weights ? __ldg(p.weights + f) : 1.0f;
                c[i] = load_chunk<T, VEC>(y + r * p.K + k, n);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (used[i]) {
#pragma unroll
                for (int v = 0; v < kV; ++v) sum[v] = fmaf(w[i], to_f(c[i].v[v]), sum[v]);
            }
    }
    if (p.addend) {
        const Chunk<T> a = load_chunk<T, VEC>(static_cast<const T*>(p.addend) + t * p.K + k, n);
#pragma unroll
        for (int v = 0; v < kV; ++v) sum[v] += to_f(a.v[v]);
    }
    Chunk<T> o;
#pragma unroll
    for (int v = 0; v < kV; ++v) o.v[v] = from_f<T>(sum[v]);
    store_chunk<T, VEC>(static_cast<T*>(p.out) + t * p.K + k, n, o);
}

// A block per token: a thread has its chunks of dout and, for up to 8 slots at a time,
// the same chunks of their rows of y.  The dot products are summed over a thread's chunks, the
// lanes and the warps, in that order.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kBackThreads) unsort_grad_kernel(const UnsortParams p) {
    __shared__ float part[kBackThreads / 32][kBatch];
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* y = static_cast<const T*>(p.y);
    T* dy = static_cast<T*>(p.out);
    for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
        int64_t row[kBatch];
        float w[kBatch], dot[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t f = t * p.topk + j0 + i;
            const int64_t r = j0 + i < p.topk ? __ldg(p.inv + f) : -1;
            row[i] = r < p.R ? r : -1;
            w[i] = row[i] >= 0 && p.weights ? __ldg(p.weights + f) : 1.0f;
            dot[i] = 0.0f;
        }
        for (int64_t k = threadIdx.x * kV; k < p.K; k += kBackThreads * kV) {
            const int64_t n = p.K - k;
            const Chunk<T> d = load_chunk<T, VEC>(static_cast<const T*>(p.dout) + t * p.K + k, n);
            if (p.dweights) {
                Chunk<T> c[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (row[i] >= 0) c[i] = load_chunk<T, VEC>(y + row[i] * p.K + k, n);
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (row[i] >= 0) {
#pragma unroll
                        for (int v = 0; v < kV; ++v) dot[i] = fmaf(to_f(d.v[v]), to_f(c[i].v[v]), dot[i]);
                    }
            }
            if (dy) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (row[i] >= 0) {
                        Chunk<T> o;
#pragma unroll
                        for (int v = 0; v < kV; ++v) o.v[v] = from_f<T>(w[i] * to_f(d.v[v]));
                        store_chunk<T, VEC>(dy + row[i] * p.K + k, n, o);
                    }
            }
        }
        if (!p.dweights) continue;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) dot[i] += __shfl_xor_sync(kAll, dot[i], d);
            if (lane == 0) part[warp][i] = dot[i];
        }
        __syncthreads();
        if (threadIdx.x < kBatch && j0 + static_cast<int>(threadIdx.x) < p.topk) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kBackThreads / 32; ++i) s += part[i][threadIdx.x];
            p.dweights[t * p.topk + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_back(const UnsortParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>((p.K + kBackThreads * kV - 1) / (kBackThreads * kV)));
    return launch_pdl(p.vec ? unsort_kernel<T, true> : unsort_kernel<T, false>, grid, dim3(kBackThreads), 0, s, p);
}
template <typename T>
cudaError_t launch_back_grad(const UnsortParams& p, cudaStream_t s) {
    return launch_pdl(p.vec ? unsort_grad_kernel<T, true> : unsort_grad_kernel<T, false>, dim3(static_cast<unsigned>(p.T)),
                      dim3(kBackThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_sort_tokens(const SortParams& p, cudaStream_t s) {
    // the widest accesses that every row allows
    const uint64_t all = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.rows) |
                         (p.T > 1 ? static_cast<uint64_t>(p.x_pitch) : 0) | static_cast<uint64_t>(p.row_bytes);
    if (all % 16 == 0) return launch_sort<uint4>(p, s);
    if (all % 4 == 0) return launch_sort<uint32_t>(p, s);
    if (all % 2 == 0) return launch_sort<uint16_t>(p, s);
    return launch_sort<uint8_t>(p, s);
}

cudaError_t launch_unsort_tokens(int type, const UnsortParams& p, cudaStream_t s) {
    if (type == kBf16) return launch_back<__nv_bfloat16>(p, s);
    if (type == kFp16) return launch_back<__half>(p, s);
    return launch_back<float>(p, s);
}

cudaError_t launch_unsort_tokens_grad(int type, const UnsortParams& p, cudaStream_t s) {
    if (type == kBf16) return launch_back_grad<__nv_bfloat16>(p, s);
    if (type == kFp16) return launch_back_grad<__half>(p, s);
    return launch_back_grad<float>(p, s);
}

}  // namespace wna16
