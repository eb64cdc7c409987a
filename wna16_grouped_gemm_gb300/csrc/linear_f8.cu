// Products of e4m3 rows with block-scaled e4m3 weights, one weight or one per expert:
//   out[t][n] = sum_b xs[t][b] ws[n / 128][b] sum_{k in b} xq[t][k] wq[n][k]  (+ bias[n]) (+ addend[t][n])
//
// A block has 16 rows of one expert and 64 output channels, a thread 4 sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "../../include/wna16_moe_f8.h"
#include "f8.h"
#include "gemm.h"
#include "ptx.cuh"

namespace wna16 {

namespace {

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

__device__ __forceinline__ float code_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

constexpr int kRows = 16, kCols = 64;

template <typename T>
__global__ void __launch_bounds__(256) simple_kernel(const LinearF8Params p) {
    __shared__ float sx[kRows][kScaleBlock + 1], sw[kCols][kScaleBlock + 1];
    pdl_wait();
    pdl_trigger();
    if (p.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        bool bad = false;
        if (p.offsets) {
            int at = 0;
            for (int i = 0; i <= p.E; ++i) {
                const int o = p.offsets[i], c = min(max(o, at), p.T);
                bad = bad || c != o;
                at = c;
            }
        }
        *p.status = bad ? kStatusBadRouting : kStatusOk;
    }
    // the tile's expert and rows: tiles of 16 rows, expert after expert
    int e = 0, r0 = 0, r1 = p.T;
    if (p.offsets) {
        int tile = blockIdx.x, at = min(max(p.offsets[0], 0), p.T);
        for (; e < p.E; ++e) {
            const int next = min(max(p.offsets[e + 1], at), p.T), tiles = (next - at + kRows - 1) / kRows;
            if (tile < tiles) {
                r0 = at + tile * kRows;
                r1 = next;
                break;
            }
            tile -= tiles;
            at = next;
        }
        if (e == p.E) return;
    } else {
        r0 = blockIdx.x * kRows;
    }
    const int n0 = blockIdx.y * kCols, blocks = p.K / kScaleBlock, n_blocks = (p.N + kScaleBlock - 1) / kScaleBlock;
    const int c = threadIdx.x % kCols, g = threadIdx.x / kCols;
    const uint8_t* w = p.wq + static_cast<int64_t>(e) * p.N * p.K;
    float sum[4] = {};
    for (int b = 0; b < blocks; ++b) {
        __syncthreads();
        for (int i = threadIdx.x; i < kRows * kScaleBlock; i += 256) {
            const int r = i / kScaleBlock, k = i % kScaleBlock;
            sx[r][k] = r0 + r < r1 ? code_value(p.xq[static_cast<int64_t>(r0 + r) * p.K + b * kScaleBlock + k]) : 0.0f;
        }
        for (int i = threadIdx.x; i < kCols * kScaleBlock; i += 256) {
            const int n = i / kScaleBlock, k = i % kScaleBlock;
            sw[n][k] = n0 + n < p.N ? code_value(w[static_cast<int64_t>(n0 + n) * p.K + b * kScaleBlock + k]) : 0.0f;
        }
        __syncthreads();
        const float ws = p.ws[(static_cast<int64_t>(e) * n_blocks + n0 / kScaleBlock) * blocks + b];
        for (int i = 0; i < 4; ++i) {
            const int r = g * 4 + i;
            if (r0 + r >= r1) continue;
            float s = 0.0f;
            for (int k = 0; k < kScaleBlock; ++k) s = fmaf(sx[r][k], sw[c][k], s);
            sum[i] = fmaf(s, p.xs[static_cast<int64_t>(r0 + r) * blocks + b] * ws, sum[i]);
        }
    }
    const int n = n0 + c;
    if (n >= p.N) return;
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + g * 4 + i;
        if (r >= r1) continue;
        const int64_t at = static_cast<int64_t>(r) * p.N + n;
        float v = sum[i];
        if (p.bias) v += p.bias[n];
        if (p.addend) v += to_f(static_cast<const T*>(p.addend)[at]);
        static_cast<T*>(p.out)[at] = from_f<T>(v);
    }
}

template <typename T>
int run_typed(const LinearF8Params& p, cudaStream_t s) {
    const int tiles = (p.T + kRows - 1) / kRows + (p.offsets ? p.E : 0);
    const cudaError_t e = launch_pdl(simple_kernel<T>, dim3(tiles, (p.N + kCols - 1) / kCols), dim3(256), 0, s, p);
    return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "8-bit float linear: %s", cudaGetErrorString(e));
}

}  // namespace

int run_linear_f8(LinearF8Params p, cudaStream_t s) {
    if (p.type == kBf16) return run_typed<__nv_bfloat16>(p, s);
    if (p.type == kFp16) return run_typed<__half>(p, s);
    return run_typed<float>(p, s);
}

}  // namespace wna16
