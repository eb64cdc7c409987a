// Block-scaled e4m3 product for a few rows and one weight: out[t][n] = sum_b xs[t][b] ws[b] P_b[t][n].
//
// Bound by latency and the weights' bytes.  A block of the grid owns 16 output channels and up to 32 rows (the weights
// come from L2 for the second and later groups of rows); its 8 warps take the blocks of 128 k in turns, each lane
// loading 16 consecutive bytes of two weight rows and of a row of the input straight into registers, as operands of
// mma.sync m16n8k32 (the order of k inside a product is free, so both operands use the order in which the bytes lie).
// A block's fp32 sums are scaled and added in registers, the warps' through shared memory.
// Measured (us): 4 x 4096 x 4096 4.3 (3.9 TB/s), 4 x 4096 x 32768 27 (5.0 TB/s), 77 x 2048 x 1000 5.2.  (Codes
// converted to fp16 for m16n8k16: 5.7, 32, 6.6, with the same errors against 64 bits.)
#include "../../include/wna16_moe_f8.h"
#include "gemm.h"
#include "linear_f8.cuh"

namespace wna16 {

namespace {

constexpr int kWarps = 8;
constexpr int kChannels = 16;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Blocks of 128 k in flight per warp, and blocks of the grid per SM.  Measured (us; 4 x 4096 x 4096 / 16 x 4096 x 4096 /
// 32 x 4096 x 4096, then x 32768 channels):  2, 2: 4.3 5.8 8.7, 27 35 55   2, 3: 5.3 9.6 -, 27 41 -   4, 2: 4.6 - -, 28 - -
// 4, 1: - 7.6 -, - 46 -   2, 1: - - 10.1, - - 64   1, 2: - - 9.1, - - 58.
constexpr int kInFlight = 2, kPerSm = 2;

// NT tiles of 8 rows
template <typename T, int NT>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) small_kernel(const LinearF8Params p) {
    __shared__ float part[kWarps][kChannels][NT * 8 + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * kChannels, t0 = blockIdx.y * NT * 8;
    const int K = p.K, blocks = K / kScaleBlock;
    // the block's weights on their way to L2 while the kernel before finishes (nothing of them is used)
    for (int64_t i = threadIdx.x * 128; i < static_cast<int64_t>(min(kChannels, p.N - n0)) * K; i += 32 * kWarps * 128)
        prefetch_l2(p.wq + static_cast<int64_t>(n0) * K + i);
    pdl_wait();
    pdl_trigger();
    if (p.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = kStatusOk;
    // rows past the end read the last one; their results are not stored
    const uint8_t* w0 = p.wq + static_cast<int64_t>(min(n0 + g, p.N - 1)) * K + q * 16;
    const uint8_t* w1 = p.wq + static_cast<int64_t>(min(n0 + g + 8, p.N - 1)) * K + q * 16;
    const float* ws = p.ws + static_cast<int64_t>(n0 / kScaleBlock) * blocks;
    const uint8_t* x[NT];
    const float* xs[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        x[j] = p.xq + static_cast<int64_t>(min(t0 + j * 8 + g, p.T - 1)) * K + q * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) xs[j][i] = p.xs + static_cast<int64_t>(min(t0 + j * 8 + 2 * q + i, p.T - 1)) * blocks;
    }
    float sum[NT][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int b0 = warp; b0 < blocks; b0 += kWarps * kInFlight) {   // the same turns for every lane of the warp
        uint4 a[kInFlight][4], c[kInFlight][NT][2];
        float s[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int b = b0 + u * kWarps, k = b * kScaleBlock;
            const bool some = b < blocks;
            a[u][0] = some ? ld_stream(w0 + k) : zero;
            a[u][1] = some ? ld_stream(w1 + k) : zero;
            a[u][2] = some ? ld_stream(w0 + k + 64) : zero;
            a[u][3] = some ? ld_stream(w1 + k + 64) : zero;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                c[u][j][0] = some ? ld_again(x[j] + k) : zero;
                c[u][j][1] = some ? ld_again(x[j] + k + 64) : zero;
            }
            s[u] = some ? ws[b] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int b = b0 + u * kWarps;
            if (b >= blocks) break;
            float acc[NT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t aw[4] = {a[u][2 * h].x, a[u][2 * h].y, a[u][2 * h].z, a[u][2 * h].w};
                const uint32_t bw[4] = {a[u][2 * h + 1].x, a[u][2 * h + 1].y, a[u][2 * h + 1].z, a[u][2 * h + 1].w};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint32_t xw[4] = {c[u][j][h].x, c[u][j][h].y, c[u][j][h].z, c[u][j][h].w};
                    mma_e4m3(acc[j], aw[0], bw[0], aw[1], bw[1], xw[0], xw[1]);
                    mma_e4m3(acc[j], aw[2], bw[2], aw[3], bw[3], xw[2], xw[3]);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float s0 = xs[j][0][b] * s[u], s1 = xs[j][1][b] * s[u];
                sum[j][0] = fmaf(acc[j][0], s0, sum[j][0]);
                sum[j][1] = fmaf(acc[j][1], s1, sum[j][1]);
                sum[j][2] = fmaf(acc[j][2], s0, sum[j][2]);
                sum[j][3] = fmaf(acc[j][3], s1, sum[j][3]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        part[warp][g][j * 8 + 2 * q] = sum[j][0];
        part[warp][g][j * 8 + 2 * q + 1] = sum[j][1];
        part[warp][g + 8][j * 8 + 2 * q] = sum[j][2];
        part[warp][g + 8][j * 8 + 2 * q + 1] = sum[j][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kChannels * NT * 8; i += 32 * kWarps) {
        const int r = i % kChannels, tt = i / kChannels, t = t0 + tt, n = n0 + r;
        if (n >= p.N || t >= p.T) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part[w][r][tt];
        if (p.bias) v += p.bias[n];
        const int64_t o = static_cast<int64_t>(t) * p.N + n;
        if (p.addend) v += elem_to_f(static_cast<const T*>(p.addend)[o]);
        static_cast<T*>(p.out)[o] = elem_from_f<T>(v);
    }
}

template <typename T>
cudaError_t launch(const LinearF8Params& p, int nt, cudaStream_t s) {
    const unsigned channels = static_cast<unsigned>((p.N + kChannels - 1) / kChannels);
    const unsigned groups = static_cast<unsigned>((p.T + 8 * nt - 1) / (8 * nt));
    const dim3 grid(channels, groups), block(32 * kWarps);
    const auto kernel = nt == 1 ? small_kernel<T, 1> : nt == 2 ? small_kernel<T, 2> : small_kernel<T, 4>;
    return launch_pdl(kernel, grid, block, 0, s, p);
}

}  // namespace

int launch_linear_f8_small(const LinearF8Params& p, int nt, cudaStream_t s) {
    const cudaError_t e = p.type == kBf16 ? launch<__nv_bfloat16>(p, nt, s)
                          : p.type == kFp16 ? launch<__half>(p, nt, s)
                                            : launch<float>(p, nt, s);
    return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "8-bit float linear launch: %s", cudaGetErrorString(e));
}

}  // namespace wna16
