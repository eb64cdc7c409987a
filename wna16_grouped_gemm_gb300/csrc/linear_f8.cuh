// What the kernels of the block-scaled e4m3 products share: the list of tiles, waits, conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "f8.h"
#include "ptx.cuh"

namespace wna16 {

// Launch parameters of a product.
struct LinearF8Launch {
    LinearF8Params p;
    int blocks = 0;     // K / 128
    int n_tiles = 0;    // tiles of output channels
    int n_blocks = 0;   // rows of scales per weight
    int ksplit = 1;     // blocks of a cluster that share a tile's K
    int stages = 0;     // operand buffers
    int wide = 0;       // rows of results are stored 16 bytes at a time
};

// kernels' launches (linear_f8_small.cu, linear_f8_thin.cu, linear_f8_wide.cu); return a wna16_status
int launch_linear_f8_small(const LinearF8Params& p, int nt, cudaStream_t stream);
int launch_linear_f8_thin(const LinearF8Params& p, int nt, int ksplit, cudaStream_t stream);
int launch_linear_f8_wide(const LinearF8Params& p, cudaStream_t stream);
// Codes [matrices][rows][K] as boxes of `box_rows` rows x 128 k (zeros past the end)
int f8_code_map(CUtensorMap* map, const uint8_t* q, int64_t matrices, int64_t rows, int64_t K, int box_rows);

#ifdef __CUDACC__

template <typename T>
__device__ __forceinline__ float elem_to_f(T v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else if constexpr (std::is_same<T, __half>::value)
        return __half2float(v);
    else
        return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T elem_from_f(float v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else if constexpr (std::is_same<T, __half>::value)
        return __float2half_rn(v);
    else
        return __float2bfloat16_rn(v);
}

// acc += v * s on a value of a tensor memory load: volatile, so that it stays behind the wait for it.
__device__ __forceinline__ void fma_loaded(float& acc, uint32_t v, float s) {
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(v)), "f"(s));
}
// Position in a ring of n slots and the parity of its current phase.
struct RingSlot {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            phase ^= 1u;
        }
    }
};

// Wait of a whole warp: true only if every lane saw the phase complete.
__device__ __forceinline__ bool warp_wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
    return __all_sync(0xffffffffu, mbar_wait_at(smem_u32(bar), parity, abort, status));
}

// The same without a call: a function's registers do not go with setmaxnreg.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile int* abort, int* status) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t began = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity)) {
        if (*abort) return false;
        if (globaltimer_ns() - began > kWaitLimitNs) {
            *abort = 1;
            atomicExch(status, kStatusTimeout);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool warp_wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
    return __all_sync(0xffffffffu, wait_inline(smem_u32(bar), parity, abort, status));
}

// The offsets into rows [E + 1], by the whole block; a barrier of the block is behind them.
__device__ __forceinline__ void f8_load_offsets(const LinearF8Params& p, int* rows) {
    if (!p.offsets) return;
    for (int i = threadIdx.x; i <= p.E; i += blockDim.x) rows[i] = p.offsets[i];
    __syncthreads();
}
// The list of tiles: rows[e] is the first row of expert e (rows[E] the end), tiles[e] the number
// of tiles of `tile` rows before it.  Written by one warp, from the offsets (which the block has
// loaded into rows) held to [their predecessor, T]; returns whether one had to be.
__device__ inline bool f8_tile_list(const LinearF8Params& p, int tile, int* rows, int* tiles) {
    const int lane = threadIdx.x & 31;
    if (!p.offsets) {
        if (lane == 0) {
            rows[0] = tiles[0] = 0;
            rows[1] = p.T;
            tiles[1] = (p.T + tile - 1) / tile;
        }
        __syncwarp();
        return false;
    }
    bool bad = false;
    {
        const int per = (p.E + 1 + 31) / 32, i0 = lane * per, i1 = min(i0 + per, p.E + 1);
        int top = 0;
        for (int i = i0; i < i1; ++i) {
            const int o = rows[i], c = min(max(o, 0), p.T);
            bad = bad || c != o;
            rows[i] = c;
            top = max(top, c);
        }
        int before = top;   // inclusive, then of the lanes before
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before = max(before, o);
        }
        before = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 0) before = 0;
        for (int i = i0; i < i1; ++i) {
            bad = bad || rows[i] < before;
            before = max(before, rows[i]);
            rows[i] = before;
        }
    }
    __syncwarp();
    const int per = (p.E + 31) / 32, i0 = min(lane * per, p.E), i1 = min(i0 + per, p.E);
    int total = 0;
    for (int i = i0; i < i1; ++i) total += (rows[i + 1] - rows[i] + tile - 1) / tile;
    int run = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
    }
    int at = run - total;
    for (int i = i0; i < i1; ++i) {
        tiles[i] = at;
        at += (rows[i + 1] - rows[i] + tile - 1) / tile;
    }
    if (lane == 31) tiles[p.E] = run;
    __syncwarp();
    return __any_sync(0xffffffffu, bad);
}

// A tile: rows [r0, r1) of expert e (r1 may be past the tile's last row), output channels from tile `nt` on.
// Tiles of an expert are in the order of the channels, those of the same channels side by side:
// they are worked on at the same time and share the weights in L2.
struct F8Tile {
    int e = 0;
    int r0 = 0, r1 = 0, nt = 0;
    // the tile of item v (items of a walk come in ascending order); the bounds-checked build takes the first expert's first
    // one where the lists lead outside the buffers
    __device__ __forceinline__ void locate(int v, int n_tiles, int tile, const int* rows, const int* tiles,
                                           const LinearF8Params& p, int* status) {
        const int q = v / n_tiles;
        while (in_bounds(e < p.E, status) && tiles[e + 1] <= q) ++e;
        if (!in_bounds(e < p.E, status)) e = 0;
        const int count = tiles[e + 1] - tiles[e], local = v - tiles[e] * n_tiles;
        nt = local / count;
        r0 = rows[e] + (local - nt * count) * tile;
        r1 = rows[e + 1];
        if (!in_bounds(nt >= 0 && nt < n_tiles && r0 >= 0 && r0 < r1 && r1 <= p.T, status)) nt = r0 = r1 = 0;
    }
};

#endif  // __CUDACC__

}  // namespace wna16
