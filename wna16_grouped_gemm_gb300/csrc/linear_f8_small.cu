// Block-scaled e4m3 product for a few rows and one weight: out[t][n] = sum_b xs[t][b] ws[b] P_b[t][n].
//
// Bound by latency and the weights' bytes.  A block of the grid owns 16 output channels and up to 32 rows (the weights
// come from L2 for the second and later groups of rows); its 8 warps take the blocks of 128 k in turns, each lane
// loading 16 consecutive bytes of two weight rows and of a row of the input straight into registers, where the codes
// become the fp16 operands of mma.sync m16n8k16 (exact: e4m3 has 4 significant bits and exponents within fp16's; the
// order of k inside a product is free, so both operands use the order in which the bytes lie).  A block's fp32 sums are
// scaled and added in registers, the warps' through shared memory.
#include <cuda_fp8.h>

#include "../../include/wna16_moe_f8.h"
#include "gemm.h"
#include "linear_f8.cuh"

namespace wna16 {

namespace {

constexpr int kWarps = 8;
constexpr int kChannels = 16;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 4 codes -> 4 fp16 (exact)
__device__ __forceinline__ uint2 fp16x4_of(uint32_t w) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    return make_uint2(static_cast<uint32_t>(lo.x) | static_cast<uint32_t>(lo.y) << 16,
                      static_cast<uint32_t>(hi.x) | static_cast<uint32_t>(hi.y) << 16);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT tiles of 8 rows; U blocks of 128 k in flight per warp, at least PER_SM blocks of the grid per SM
template <typename T, int NT, int U, int PER_SM>
__global__ void __launch_bounds__(32 * kWarps, PER_SM) small_kernel(const LinearF8Params p) {
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
    for (int b0 = warp; b0 < blocks; b0 += kWarps * U) {   // the same turns for every lane of the warp
        uint4 a[U][4], c[U][2];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kWarps, k = b * kScaleBlock;
            const bool some = b < blocks;
            a[u][0] = some ? ld_stream(w0 + k) : zero;
            a[u][1] = some ? ld_stream(w1 + k) : zero;
            a[u][2] = some ? ld_stream(w0 + k + 64) : zero;
            a[u][3] = some ? ld_stream(w1 + k + 64) : zero;
            c[u][0] = some ? __ldg(reinterpret_cast<const uint4*>(x[0] + k)) : zero;
            c[u][1] = some ? __ldg(reinterpret_cast<const uint4*>(x[0] + k + 64)) : zero;
            s[u] = some ? __ldg(ws + b) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kWarps, k = b * kScaleBlock;
            if (b >= blocks) break;
            float acc[NT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t aw[4] = {a[u][2 * h].x, a[u][2 * h].y, a[u][2 * h].z, a[u][2 * h].w};
                const uint32_t bw[4] = {a[u][2 * h + 1].x, a[u][2 * h + 1].y, a[u][2 * h + 1].z, a[u][2 * h + 1].w};
                uint2 fa[4], fb[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    fa[m] = fp16x4_of(aw[m]);
                    fb[m] = fp16x4_of(bw[m]);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 xc = j == 0 ? c[u][h] : __ldg(reinterpret_cast<const uint4*>(x[j] + k + 64 * h));
                    const uint32_t xw[4] = {xc.x, xc.y, xc.z, xc.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const uint2 fx = fp16x4_of(xw[m]);
                        mma_f16(acc[j], fa[m].x, fb[m].x, fa[m].y, fb[m].y, fx.x, fx.y);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float s0 = __ldg(xs[j][0] + b) * s[u], s1 = __ldg(xs[j][1] + b) * s[u];
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
        if (p.bias) v += __ldg(p.bias + n);
        const int64_t o = static_cast<int64_t>(t) * p.N + n;
        if (p.addend) v += elem_to_f(static_cast<const T*>(p.addend)[o]);
        static_cast<T*>(p.out)[o] = elem_from_f<T>(v);
    }
}

template <typename T>
cudaError_t launch(const LinearF8Params& p, int nt, int sms, cudaStream_t s) {
    const unsigned channels = static_cast<unsigned>((p.N + kChannels - 1) / kChannels);
    const unsigned groups = static_cast<unsigned>((p.T + 8 * nt - 1) / (8 * nt));
    const dim3 grid(channels, groups), block(32 * kWarps);
    const bool turns = static_cast<int64_t>(channels) * groups > 2 * sms;
    if (nt == 1) return launch_pdl(turns ? small_kernel<T, 1, 2, 3> : small_kernel<T, 1, 2, 2>, grid, block, 0, s, p);
    if (nt == 2) return launch_pdl(turns ? small_kernel<T, 2, 1, 4> : small_kernel<T, 2, 2, 2>, grid, block, 0, s, p);
    return launch_pdl(small_kernel<T, 4, 1, 2>, grid, block, 0, s, p);
}

}  // namespace

int launch_linear_f8_small(const LinearF8Params& p, int nt, cudaStream_t s) {
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    const cudaError_t e = p.type == kBf16 ? launch<__nv_bfloat16>(p, nt, sms, s)
                          : p.type == kFp16 ? launch<__half>(p, nt, sms, s)
                                            : launch<float>(p, nt, sms, s);
    return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "8-bit float linear launch: %s", cudaGetErrorString(e));
}

}  // namespace wna16
