// Tokens to rows in the order of their experts, and back.
//
//   inv[f]  = (slots of lower experts) + (earlier slots of the same expert)
//   rows[inv[f]] = x[t]                        f = t * topk + j
//   out[t]  = sum_j w[t][j] y[inv[t][j]]       (without w: the gradient of the line above)
//   dy[inv[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[inv[t][j]]>
//
// Bound by the bytes of the rows.  Sums are fp32, in an order that the sizes alone fix.
// Measured (us; 8 slots per token on 256 experts, rows of 4096 bf16; of a measured copy's 6793 GB/s):
//   8192 tokens   lists 8.9, lists and rows 106 (0.84 of it; the copies alone 0.91), back 90 (0.98), gradient 173 (0.97)
//   4 tokens      3.2, 2.1, 4.1 (a launch); 1024 tokens: 17.7, 14.7, 25
//   8192 tokens   fp32 202, 171, 338; e4m3 58; rows of 4100 bf16 (4-byte accesses) 122, 121, 212; of 4097 205, 232, 443
// The gradient of a few thousand tokens is further from it, since a block's items are whole tokens: 2047 of them with about half of
// their 8 slots in use 31 to 33 us, of 22 that the bytes take (608 blocks, 3.4 turns of unequal length).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "f8.h"
#include "gemm.h"
#include "ptx.cuh"

namespace wna16 {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// The status word of the index checks here (the bounds-checked build; these operators have no workspace).
#ifdef WNA16_DEBUG
__device__ int g_index_status;
__device__ __forceinline__ int* index_status() { return &g_index_status; }
#else
__device__ __forceinline__ constexpr int* index_status() { return nullptr; }
#endif
// A row of R, which the bounds-checked build leaves out if it is none.
__device__ __forceinline__ int row_in_bounds(int row, int64_t R) {
    return in_bounds(row >= 0 && row < R, index_status()) ? row : -1;
}

// ------------------------------------------------------------------ sort

constexpr int kSmallThreads = 256;
// Slots up to which every token counts its own positions, in one launch.  Lists and rows of 4096 bf16 this way / with the
// cluster's lists (us): 512 slots 3.3 / 13, 4096 11.4 / 16, 6144 15.5 / 17, 8192 21 / 19, 16384 65 / 33.
constexpr int kSmallSlots = 6144;

// The sums over a warp of 8 values per lane: lane l has that of value l / 4 (halves of the values go to halves of the
// lanes, then the lanes of each are added).
template <typename N>
__device__ __forceinline__ N warp_sums(const N (&v)[8], int lane) {
    N a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        a[i] = (up ? v[4 + i] : v[i]) + __shfl_xor_sync(kAll, up ? v[i] : v[4 + i], 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        b[i] = (up ? a[2 + i] : a[i]) + __shfl_xor_sync(kAll, up ? a[i] : a[2 + i], 8);
    }
    const bool up = lane & 4;
    N c = (up ? b[1] : b[0]) + __shfl_xor_sync(kAll, up ? b[0] : b[1], 4);
    c += __shfl_xor_sync(kAll, c, 2);
    c += __shfl_xor_sync(kAll, c, 1);
    return c;
}

// One block per token, and one for the offsets.  A slot's row is the number of slots
// that sort before it; the block's threads count them, for up to 8 slots at a time.  Experts are unsigned
// offsets from expert_begin, so ids below it are large numbers.
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
            const unsigned e = ids[f] - begin;
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
    __shared__ int part[kSmallThreads / 32][8];
    for (int j0 = 0; j0 < p.topk; j0 += 8) {
        const int f = t * p.topk + j0;
        unsigned e[8];
        int n[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            e[q] = j0 + q < p.topk ? ids[f + q] - begin : ~0u;
            n[q] = 0;
        }
#pragma unroll 4
        for (int i = tid; i < R; i += kSmallThreads) {
            const unsigned o = ids[i] - begin;
#pragma unroll
            for (int q = 0; q < 8; ++q) n[q] += o < e[q] || (o == e[q] && i < f + q);
        }
        const int sum = warp_sums(n, lane);
        if ((lane & 3) == 0) part[warp][lane >> 2] = sum;
        __syncthreads();
        if (tid < 8 && j0 + tid < p.topk) {
            int row = 0;
#pragma unroll
            for (int w = 0; w < kSmallThreads / 32; ++w) row += part[w][tid];
            row = ids[f + tid] - begin >= E ? -1 : row_in_bounds(row, R);
            pos[j0 + tid] = row;
            p.inv[f + tid] = row;
        }
        __syncthreads();
    }
    if (!p.x) return;
    const int64_t n_vec = p.row_bytes / static_cast<int64_t>(sizeof(V));
    const V* src = reinterpret_cast<const V*>(static_cast<const char*>(p.x) + t * p.x_pitch);
    V* dst = static_cast<V*>(p.rows);
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
constexpr int kListBlocks = 16;  // one cluster
constexpr int kKeep = 8;         // slots of a lane at a time

// The lists of many slots, by one cluster (65536 slots 8.8 us; by one of 8 blocks 12.3): a stable counting sort.  Every warp has a run
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
    cluster_arrive();   // (the wait for it is behind the counting)
    pdl_wait();
    pdl_trigger();
    const int64_t R = p.T * p.topk;
    const int64_t per_warp = (R + kListBlocks * kListWarps * 32 - 1) / (kListBlocks * kListWarps * 32) * 32;
    const int64_t f0 = (rank * kListWarps + warp) * per_warp, f1 = min(R, f0 + per_warp);
    const bool kept = per_warp <= 32 * kKeep;   // the experts and ranks of all of a lane's slots stay in registers
    int* my = hist + warp * E;
    for (int e = lane; e < E; e += 32) my[e] = 0;
    __syncwarp();
    const unsigned lower = (1u << lane) - 1u;
    unsigned e[kKeep];
    int at_rank[kKeep];
    auto load = [&](int64_t at) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int64_t f = at + i * 32 + lane;
            e[i] = f < f1 ? ids[f] - begin : ~0u;
        }
    };
    // every slot's rank among its expert's, and the counts of the warp
    auto count = [&] {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if (e[i] >= static_cast<unsigned>(E)) e[i] = ~0u;
            const unsigned peers = __match_any_sync(kAll, e[i]);
            const int before = e[i] != ~0u ? my[e[i]] : 0;
            at_rank[i] = before + __popc(peers & lower);
            __syncwarp();
            if (e[i] != ~0u && lane == __ffs(peers) - 1) my[e[i]] = before + __popc(peers);
            __syncwarp();
        }
    };
    for (int64_t at = f0; at < f1; at += 32 * kKeep) {
        load(at);
        count();
    }
    __syncthreads();
    cluster_wait();     // every block has started: their shared memory is theirs
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
    // now hist holds the slots of the expert in the block's lower warps, and base its first row of the block
    if (kept) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int64_t f = f0 + i * 32 + lane;
            if (f < f1) p.inv[f] = e[i] != ~0u ? row_in_bounds(base[e[i]] + my[e[i]] + at_rank[i], R) : -1;
        }
        return;
    }
    for (int64_t at = f0; at < f1; at += 32 * kKeep) {
        load(at);
        count();
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int64_t f = at + i * 32 + lane;
            if (f < f1) p.inv[f] = e[i] != ~0u ? row_in_bounds(base[e[i]] + at_rank[i], R) : -1;
        }
    }
}

constexpr int kCopyWarps = 8;
// The rows go ahead to L2 while the lists are made, 8 KB of each, if those of all tokens are few: 1024 tokens of 8 KB 19.2 us
// without and 17.6 with, 2047 31.9 and 30.0, 8192 of 4 KB 57.7 and 56.3; of 8 KB 105.8 and 107.1, 32768 of 4 KB 221.7 and 223.9.
constexpr int64_t kAheadBytes = 8192, kAheadTotal = 40 << 20;

// (16 bytes at a time past L1, by an instruction that stays where it is written: 8192 x 2 of 4096 bf16 38.6 us, 39.8 without.)
template <typename V>
__device__ __forceinline__ V load_row(const V* p) {
    if constexpr (sizeof(V) == 16)
        return ld_stream(p);
    else
        return *p;
}

// rows[inv[t][j]] = x[t]: a warp per token, which reads its row once.  (Six blocks per SM: with five, 8192 x 8 of 4100 bf16 134 us,
// not 122; with seven, of 4096 118, not 105.)
template <typename V>
__global__ void __launch_bounds__(32 * kCopyWarps, 6) sort_copy_kernel(const SortParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5);
    const char* row = static_cast<const char*>(p.x) + t * p.x_pitch;
    const int64_t ahead = min(p.row_bytes, kAheadBytes);
    if (t < p.T && p.T * ahead <= kAheadTotal)
        for (int64_t b = lane * 128; b < ahead; b += 32 * 128) prefetch_l2(row + b);
    pdl_wait();
    pdl_trigger();
    if (t >= p.T) return;
    const int64_t n_vec = p.row_bytes / static_cast<int64_t>(sizeof(V));
    const V* src = reinterpret_cast<const V*>(row);
    V* dst = static_cast<V*>(p.rows);
    const int32_t* inv = p.inv + t * p.topk;
    for (int j0 = 0; j0 < p.topk; j0 += 32) {
        const int count = min(32, p.topk - j0);
        const int mine = lane < count ? inv[j0 + lane] : -1;
        for (int64_t v0 = lane; v0 - lane < n_vec; v0 += 4 * 32) {   // the same turns for every lane
            V a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (v0 + c * 32 < n_vec) a[c] = load_row(src + v0 + c * 32);
            for (int j = 0; j < count; ++j) {
                const int r = __shfl_sync(kAll, mine, j);
                if (r < 0 || row_in_bounds(r, p.T * p.topk) < 0) continue;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (v0 + c * 32 < n_vec) dst[r * n_vec + v0 + c * 32] = a[c];
            }
        }
        if (p.x_scales)
            for (int64_t v = lane; v - lane < p.groups; v += 32) {
                const float a = v < p.groups ? p.x_scales[t * p.groups + v] : 0.0f;
                for (int j = 0; j < count; ++j) {
                    const int r = __shfl_sync(kAll, mine, j);
                    if (r >= 0 && v < p.groups && row_in_bounds(r, p.T * p.topk) >= 0) p.row_scales[r * p.groups + v] = a;
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
    e = cudaFuncSetAttribute(sort_lists_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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

constexpr int kBackThreads = 256;
constexpr int kBatch = 8;   // rows read at the same time
// Per SM.  (The gradient of 8192 x 8 slots with three blocks, whose registers then spill, 179 us, with two 177; of 512
// x 8 slots 17.8 and 14.6.)
constexpr int kBackBlocks = 3, kGradBlocks = 2;
constexpr int kRunThreads = 128; // of a run of unsort, and of the gradient's of short rows

// The values of a thread, 16 bytes of them: neighbours where rows are read 16 bytes at a time, else every 32nd access
// of a warp's (of W = 4 or 2 bytes), so that its lanes read neighbours.
template <typename T>
constexpr int kV = 16 / static_cast<int>(sizeof(T));
constexpr int kWords = 4;
struct Chunk {
    uint32_t w[kWords];
};
// the place of a thread's first value in a run
template <typename T, int W>
__device__ __forceinline__ int chunk_start() {
    constexpr int kOne = W / static_cast<int>(sizeof(T));   // values per access
    return W == 16 ? static_cast<int>(threadIdx.x) * kV<T>
                   : static_cast<int>(threadIdx.x / 32) * 32 * kV<T> + static_cast<int>(threadIdx.x & 31) * kOne;
}

// the chunk at p (of n values from there on; those past them are 0)
template <typename T, int W>
__device__ __forceinline__ Chunk load_chunk(const T* p, int64_t n) {
    Chunk c;
    if constexpr (W == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        c.w[0] = v.x;
        c.w[1] = v.y;
        c.w[2] = v.z;
        c.w[3] = v.w;
    } else if constexpr (W == 4) {   // (rows are of whole accesses)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c.w[i] = 32 * i * (4 / static_cast<int>(sizeof(T))) < n ? reinterpret_cast<const uint32_t*>(p)[32 * i] : 0u;
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 64 * i < n ? h[64 * i] : 0u, hi = 64 * i + 32 < n ? h[64 * i + 32] : 0u;
            c.w[i] = lo | hi << 16;
        }
    }
    return c;
}
template <typename T, int W>
__device__ __forceinline__ void store_chunk(T* p, int64_t n, const Chunk& c) {
    if constexpr (W == 16) {
        *reinterpret_cast<uint4*>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    } else if constexpr (W == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (32 * i * (4 / static_cast<int>(sizeof(T))) < n) reinterpret_cast<uint32_t*>(p)[32 * i] = c.w[i];
    } else {
        uint16_t* h = reinterpret_cast<uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * i < n) h[32 * i] = static_cast<uint16_t>(c.w[i / 2] >> (i % 2 * 16));
    }
}
template <typename T>
__device__ __forceinline__ void to_floats(const Chunk& c, float (&v)[kV<T>]) {
#pragma unroll
    for (int i = 0; i < kV<T>; ++i) {
        if constexpr (sizeof(T) == 4) {
            v[i] = __uint_as_float(c.w[i]);
        } else if constexpr (std::is_same<T, __half>::value) {
            if (i % 2 == 0) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c.w[i / 2]));
                v[i] = f.x;
                v[i + 1] = f.y;
            }
        } else {
            v[i] = __uint_as_float(i % 2 ? c.w[i / 2] & 0xffff0000u : c.w[i / 2] << 16);
        }
    }
}
template <typename T>
__device__ __forceinline__ Chunk from_floats(const float (&v)[kV<T>]) {
    Chunk c;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 4) {
            c.w[i] = __float_as_uint(v[i]);
        } else if constexpr (std::is_same<T, __half>::value) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            c.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            c.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return c;
}

// The rows and weights of up to 32 slots of a token from slot j0 on, one per lane; -1: left out.
struct Slots {
    int row = -1;
    float w = 1.0f;
};
__device__ __forceinline__ Slots load_slots(const UnsortParams& p, int64_t t, int j0, int lane) {
    Slots s;
    if (t < p.T && j0 + lane < p.topk) {
        const int64_t f = t * p.topk + j0 + lane;
        const int r = p.inv[f];
        s.row = r >= 0 && r < p.R ? r : -1;
        if (p.weights) s.w = p.weights[f];
    }
    return s;
}

// A block takes RUNS neighbouring runs of 2 KB of one token, item after item, and has the next one's slots
// loaded while it works on one; a thread has 16 bytes of a run.  Several runs at a time keep as many loads in flight
// with few slots per token as one does with eight.
template <typename T, int W, int RUNS>
__global__ void __launch_bounds__(kBackThreads, RUNS == 4 ? kGradBlocks : kBackBlocks) unsort_kernel(const UnsortParams p, int groups, int64_t items) {
    constexpr int kSlots = kBatch / RUNS;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int start = chunk_start<T, W>(), width = static_cast<int>(blockDim.x) * kV<T>;   // values of a run
    const T* y = static_cast<const T*>(p.y);
    int64_t t = blockIdx.x / groups;
    int group = static_cast<int>(blockIdx.x - t * groups);
    const int64_t step_t = gridDim.x / groups;
    const int step_group = static_cast<int>(gridDim.x - step_t * groups);
    Slots next = load_slots(p, t, 0, lane);
    for (int64_t v = blockIdx.x; v < items; v += gridDim.x) {
        const int64_t now = t, k = static_cast<int64_t>(group) * RUNS * width + start, n = p.K - k;
        Slots s = next;
        t += step_t;
        group += step_group;
        if (group >= groups) {
            group -= groups;
            ++t;
        }
        next = load_slots(p, t, 0, lane);
        float sum[RUNS][kV<T>] = {};
        for (int j0 = 0; j0 < p.topk; j0 += kSlots) {
            if (j0 > 0 && j0 % 32 == 0) s = load_slots(p, now, j0, lane);
            Chunk c[kSlots][RUNS];
            int row[kSlots];
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                row[i] = __shfl_sync(kAll, s.row, (j0 + i) & 31);
#pragma unroll
                for (int q = 0; q < RUNS; ++q)
                    if (row[i] >= 0 && n > q * width) c[i][q] = load_chunk<T, W>(y + row[i] * p.K + k + q * width, n - q * width);
            }
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const float w = __shfl_sync(kAll, s.w, (j0 + i) & 31);
                if (row[i] >= 0) {
#pragma unroll
                    for (int q = 0; q < RUNS; ++q) {
                        float f[kV<T>];
                        to_floats<T>(c[i][q], f);
#pragma unroll
                        for (int e = 0; e < kV<T>; ++e) sum[q][e] = fmaf(w, f[e], sum[q][e]);
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < RUNS; ++q) {
            if (n <= q * width || !in_bounds(now < p.T, index_status())) break;
            const int64_t at = now * p.K + k + q * width;
            if (p.addend) {
                float a[kV<T>];
                to_floats<T>(load_chunk<T, W>(static_cast<const T*>(p.addend) + at, n - q * width), a);
#pragma unroll
                for (int e = 0; e < kV<T>; ++e) sum[q][e] += a[e];
            }
            store_chunk<T, W>(static_cast<T*>(p.out) + at, n - q * width, from_floats<T>(sum[q]));
        }
    }
}

// A block takes token after token: a thread has its chunks of dout, RUNS of them at a time, and, for up to 8 / RUNS slots at a time,
// the same chunks of their rows of y.  The dot products are summed over a thread's chunks, the
// lanes and the warps, in that order.
template <typename T, int W, int RUNS>
__global__ void __launch_bounds__(kBackThreads, kGradBlocks) unsort_grad_kernel(const UnsortParams p) {
    constexpr int kSlots = kBatch / RUNS;
    __shared__ float part[2][kBackThreads / 32][kBatch];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int start = chunk_start<T, W>(), width = static_cast<int>(blockDim.x) * kV<T>;   // values of a run
    const T* y = static_cast<const T*>(p.y);
    const T* dout = static_cast<const T*>(p.dout);
    T* dy = static_cast<T*>(p.out);
    int turn = 0;
    Slots next = load_slots(p, blockIdx.x, 0, lane);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        Slots s = next;
        next = load_slots(p, t + gridDim.x, 0, lane);
        for (int j0 = 0; j0 < p.topk; j0 += kSlots) {
            if (j0 > 0 && j0 % 32 == 0) s = load_slots(p, t, j0, lane);
            float dot[kBatch] = {};
            for (int64_t k0 = 0; k0 < p.K; k0 += RUNS * width) {   // the same turns for every thread
                const int64_t k = k0 + start, n = p.K - k;
                Chunk g[RUNS], c[kSlots][RUNS];
                int row[kSlots];
#pragma unroll
                for (int q = 0; q < RUNS; ++q)
                    if (n > q * width) g[q] = load_chunk<T, W>(dout + t * p.K + k + q * width, n - q * width);
#pragma unroll
                for (int i = 0; i < kSlots; ++i) {
                    row[i] = __shfl_sync(kAll, s.row, (j0 + i) & 31);
#pragma unroll
                    for (int q = 0; q < RUNS; ++q)
                        if (p.dweights && row[i] >= 0 && n > q * width)
                            c[i][q] = load_chunk<T, W>(y + row[i] * p.K + k + q * width, n - q * width);
                }
#pragma unroll
                for (int q = 0; q < RUNS; ++q) {
                    const bool mine = n > q * width;
                    float d[kV<T>];
                    to_floats<T>(g[q], d);
                    if (p.dweights) {
#pragma unroll
                        for (int i = 0; i < kSlots; ++i)
                            if (mine && row[i] >= 0) {
                                float f[kV<T>];
                                to_floats<T>(c[i][q], f);
#pragma unroll
                                for (int e = 0; e < kV<T>; ++e) dot[i] = fmaf(d[e], f[e], dot[i]);
                            }
                    }
                    if (dy) {
#pragma unroll
                        for (int i = 0; i < kSlots; ++i) {
                            const float w = __shfl_sync(kAll, s.w, (j0 + i) & 31);
                            if (mine && row[i] >= 0 && in_bounds(row[i] < p.R, index_status())) {
                                float o[kV<T>];
#pragma unroll
                                for (int e = 0; e < kV<T>; ++e) o[e] = w * d[e];
                                store_chunk<T, W>(dy + row[i] * p.K + k + q * width, n - q * width, from_floats<T>(o));
                            }
                        }
                    }
                }
            }
            if (!p.dweights) continue;
            const float sum = warp_sums(dot, lane);
            if ((lane & 3) == 0) part[turn][warp][lane >> 2] = sum;
            __syncthreads();   // (and the other half of `part` has been read)
            if (threadIdx.x < kSlots && j0 + static_cast<int>(threadIdx.x) < p.topk) {
                float total = 0.0f;
                for (int i = 0; i < static_cast<int>(blockDim.x / 32); ++i) total += part[turn][i][threadIdx.x];
                p.dweights[t * p.topk + j0 + threadIdx.x] = total;
            }
            turn ^= 1;
        }
    }
}

// Threads of a block: those that a row needs, `most` at most.
template <typename T>
int back_threads(int64_t K, int most) {
    return static_cast<int>(std::min<int64_t>(most, (K + 32 * kV<T> - 1) / (32 * kV<T>) * 32));
}

// Runs at a time: what keeps eight loads in flight, of those that a row has, and fewer if blocks would go without items.
// us with one run / so, 8192 tokens of 4096 bf16: 1 slot 53 / 28, gradient 81 / 40; 2 slots 66 / 34, 93 / 54; 4 slots 76 / 52,
// 119 / 93.
int runs_at_a_time(const UnsortParams& p, int64_t runs, int64_t blocks) {
    if (p.access != 16) return 1;
    int q = p.topk <= 2 ? 4 : p.topk <= 4 ? 2 : 1;
    while (q > 1 && (q > runs || p.T * ((runs + q - 1) / q) < blocks)) q /= 2;
    return q;
}

template <typename T>
cudaError_t launch_back(const UnsortParams& p, int sms, cudaStream_t s) {
    const int threads = back_threads<T>(p.K, kRunThreads), width = threads * kV<T>;
    const int64_t runs = (p.K + width - 1) / width, per_sm = kBackThreads / threads;
    const int q = runs_at_a_time(p, runs, sms * kBackBlocks * per_sm);
    const int64_t blocks = sms * (q == 4 ? kGradBlocks : kBackBlocks) * per_sm;
    const int groups = static_cast<int>((runs + q - 1) / q);
    const int64_t items = p.T * groups;
    const dim3 grid(static_cast<unsigned>(std::min(items, blocks)));
    const auto kernel = q == 4             ? unsort_kernel<T, 16, 4>
                        : q == 2           ? unsort_kernel<T, 16, 2>
                        : p.access == 16   ? unsort_kernel<T, 16, 1>
                        : p.access == 4    ? unsort_kernel<T, 4, 1>
                                           : unsort_kernel<T, sizeof(T), 1>;
    return launch_pdl(kernel, grid, dim3(threads), 0, s, p, groups, items);
}
template <typename T>
cudaError_t launch_back_grad(const UnsortParams& p, int sms, cudaStream_t s) {
    // Short rows have more blocks with half the threads, if there are tokens for them: 8192 x 8 slots of 4096 bf16 173 us, not 178, 1024
    // x 8 25.1 (27.2), 4096 x 8 of 2048 47.2 (52.7), 8192 x 2 54 (75); 2047 x 8 49.4 (48.0), 200 x 8 9.7 (7.9), 8192 x 8 of 4096
    // fp32 352 (335).
    const bool narrow = p.K * static_cast<int64_t>(sizeof(T)) <= 8192 && p.T >= 2 * sms;
    const int threads = back_threads<T>(p.K, narrow ? kRunThreads : kBackThreads), width = threads * kV<T>;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(p.T, static_cast<int64_t>(sms) * kGradBlocks * kBackThreads / threads)));
    const int q = runs_at_a_time(p, (p.K + width - 1) / width, 0);
    const auto kernel = q == 4             ? unsort_grad_kernel<T, 16, 4>
                        : q == 2           ? unsort_grad_kernel<T, 16, 2>
                        : p.access == 16   ? unsort_grad_kernel<T, 16, 1>
                        : p.access == 4    ? unsort_grad_kernel<T, 4, 1>
                                           : unsort_grad_kernel<T, sizeof(T), 1>;
    return launch_pdl(kernel, grid, dim3(threads), 0, s, p);
}

}  // namespace

#ifdef WNA16_DEBUG
// The bounds-checked build only: what the index checks of these operators have recorded (0, or WNA16_ERR_INDEX), after
// all work on the device; cleared.  Returns a CUDA error code.
extern "C" __attribute__((visibility("default"))) int wna16_moe_debug_index_status(int* status) {
    cudaError_t e = cudaDeviceSynchronize();
    const int clear = 0;
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(status, g_index_status, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_index_status, &clear, sizeof(int));
    return e;
}
#endif

cudaError_t launch_sort_tokens(const SortParams& p, cudaStream_t s) {
    // the widest accesses that every row allows
    const uint64_t all = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.rows) |
                         (p.T > 1 ? static_cast<uint64_t>(p.x_pitch) : 0) | static_cast<uint64_t>(p.row_bytes);
    if (all % 16 == 0) return launch_sort<uint4>(p, s);
    if (all % 8 == 0) return launch_sort<uint2>(p, s);
    if (all % 4 == 0) return launch_sort<uint32_t>(p, s);
    if (all % 2 == 0) return launch_sort<uint16_t>(p, s);
    return launch_sort<uint8_t>(p, s);
}

cudaError_t launch_unsort_tokens(int type, const UnsortParams& p, int sms, cudaStream_t s) {
    if (type == kBf16) return launch_back<__nv_bfloat16>(p, sms, s);
    if (type == kFp16) return launch_back<__half>(p, sms, s);
    return launch_back<float>(p, sms, s);
}

cudaError_t launch_unsort_tokens_grad(int type, const UnsortParams& p, int sms, cudaStream_t s) {
    if (type == kBf16) return launch_back_grad<__nv_bfloat16>(p, sms, s);
    if (type == kFp16) return launch_back_grad<__half>(p, sms, s);
    return launch_back_grad<float>(p, sms, s);
}

}  // namespace wna16
