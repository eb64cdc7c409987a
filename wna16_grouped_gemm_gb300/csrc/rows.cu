// Rows to 8 bits: residual addition + RMS norm, the clamped SwiGLU, or nothing,
// then one scale and K codes per row (or per group of a row), and back.
//
//   norm    h = x + r,  y = h / sqrt(mean h^2 + eps) * w;  writes h, y (16 bits), y (8 bits)
//   swiglu  y = silu(min(g, L)) * clamp(u, -L, L)
//   plain   y = x
//   m = max |y|,  scale = m / Q,  code = round(y * (Q / m))
//
// One block per row.  A thread owns chunks of 8 consecutive values (chunk
// i * blockDim + thread, i < CH), which stay in registers from the one read of
// the row to its last write; sums and maxima are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "block.h"
#include "ptx.cuh"

namespace wna16 {

namespace {

constexpr int kV = 8;   // values per chunk

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
    static __device__ __forceinline__ float to_f(float v) { return v; }
    static __device__ __forceinline__ float from_f(float v) { return v; }
};

// 8 values at p (n of them, the others 0); vec: 16-byte loads.  Plain loads:
// the residual may be updated in place.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[kV]) {
    if (vec) {
        constexpr int W = 16 / sizeof(T);
        alignas(16) T e[kV];
#pragma unroll
        for (int i = 0; i < kV / W; ++i) reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = Elem<T>::to_f(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = i < n ? Elem<T>::to_f(p[i]) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const float (&v)[kV]) {
    if (vec) {
        constexpr int W = 16 / sizeof(T);
        alignas(16) T e[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) e[i] = Elem<T>::from_f(v[i]);
#pragma unroll
        for (int i = 0; i < kV / W; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(e)[i];
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < n) p[i] = Elem<T>::from_f(v[i]);
    }
}

// 8 codes of v * inv in 8 bytes
__device__ __forceinline__ uint2 codes8(const float (&v)[kV], float inv, int q_type) {
    uint32_t w[2];
    if (q_type == kInt8) {
        // |v * inv| exceeds 127 by at most the two roundings, so rounding gives -127..127
        int c[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) c[i] = __float2int_rn(v[i] * inv);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __byte_perm(static_cast<uint32_t>(c[4 * h]), static_cast<uint32_t>(c[4 * h + 1]), 0x0040);
            const uint32_t hi = __byte_perm(static_cast<uint32_t>(c[4 * h + 2]), static_cast<uint32_t>(c[4 * h + 3]), 0x0040);
            w[h] = __byte_perm(lo, hi, 0x5410);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h] * inv, v[4 * h + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2] * inv, v[4 * h + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | (hi << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(uint8_t* p, int n, bool vec, uint2 c) {
    if (vec) {
        *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

// Scale and code factor of a maximum magnitude, given as the bits of |y| (as
// integers they order like the values, with NaN above infinity).
__device__ __forceinline__ void scale_of(uint32_t m_bits, int q_type, float& scale, float& inv) {
    const float Q = q_type == kInt8 ? 127.0f : 448.0f;
    const float m = __uint_as_float(m_bits);
    const bool tiny = m < 0x1p-100f;
    scale = tiny ? 0.0f : m / Q;
    // not finite: codes 0, by a factor of 0 (the row reads back as 0 * scale = NaN)
    inv = tiny || m_bits >= 0x7f800000u ? 0.0f : Q / m;
}

// sum over the block; every thread gets it.  red: 32 floats
__device__ __forceinline__ float block_sum(float v, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (nw == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < nw ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    v = __reduce_max_sync(0xffffffffu, v);
    if (nw == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
}

template <RowOp OP, typename T, int CH>
__global__ void __launch_bounds__(1024) rows_kernel(const RowParams p) {
    __shared__ float red_sum[32];
    __shared__ uint32_t red_max[32];
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int K = p.K;
    const bool vec = p.vec != 0;
    const T* x = static_cast<const T*>(p.x) + t * p.ldx;
    const T* r = OP == RowOp::norm && p.residual ? static_cast<const T*>(p.residual) + t * p.ldr : nullptr;

    float v[CH][kV];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * blockDim.x + threadIdx.x) * kV;
        const int n = K - k;
        if (n > 0) {
            load8(x + k, n, vec, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < kV; ++j) v[i][j] = 0.0f;
        }
    }
    if constexpr (OP == RowOp::norm) {
        if (r) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int k = (i * blockDim.x + threadIdx.x) * kV;
                const int n = K - k;
                if (n > 0) {
                    float a[kV];
                    load8(r + k, n, vec, a);
#pragma unroll
                    for (int j = 0; j < kV; ++j) v[i][j] += a[j];
                }
            }
        }
        if (p.residual_out) {
            T* o = static_cast<T*>(p.residual_out) + t * K;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int k = (i * blockDim.x + threadIdx.x) * kV;
                if (k < K) store8(o + k, K - k, vec, v[i]);
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) ss += v[i][j] * v[i][j];
        ss = block_sum(ss, red_sum);
        const float inv = rsqrtf(ss / static_cast<float>(K) + p.eps);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = (i * blockDim.x + threadIdx.x) * kV;
            const int n = K - k;
            if (n > 0) {
                float w[kV];
                if (p.weight_f32)
                    load8(static_cast<const float*>(p.weight) + k, n, vec, w);
                else
                    load8(static_cast<const T*>(p.weight) + k, n, vec, w);
#pragma unroll
                for (int j = 0; j < kV; ++j) v[i][j] = v[i][j] * inv * w[j];
            }
        }
        if (p.norm_out) {
            T* o = static_cast<T*>(p.norm_out) + t * K;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int k = (i * blockDim.x + threadIdx.x) * kV;
                if (k < K) store8(o + k, K - k, vec, v[i]);
            }
        }
        if (!p.q) return;
    }
    if constexpr (OP == RowOp::swiglu) {
        const float L = p.limit;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = (i * blockDim.x + threadIdx.x) * kV;
            const int n = K - k;
            if (n > 0) {
                float u[kV];
                load8(x + K + k, n, vec, u);
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    // comparisons that a NaN fails: it passes through
                    const float g = v[i][j] > L ? L : v[i][j];
                    const float c = u[j] > L ? L : (u[j] < -L ? -L : u[j]);
                    v[i][j] = g / (1.0f + expf(-g)) * c;
                }
            }
        }
    }

    uint32_t m[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        m[i] = 0;
#pragma unroll
        for (int j = 0; j < kV; ++j) m[i] = max(m[i], __float_as_uint(v[i][j]) & 0x7fffffffu);
    }
    uint8_t* q = static_cast<uint8_t*>(p.q) + t * K;
    if (p.group == 0) {
        uint32_t mm = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i) mm = max(mm, m[i]);
        float scale, inv;
        scale_of(block_max(mm, red_max), p.q_type, scale, inv);
        if (threadIdx.x == 0) p.scales[t] = scale;
        const bool zero = inv == 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = (i * blockDim.x + threadIdx.x) * kV;
            if (k < K) store_codes(q + k, K - k, vec, zero ? make_uint2(0u, 0u) : codes8(v[i], inv, p.q_type));
        }
    } else {
        // a group is group / 8 neighbouring chunks: 4, 8, 16 or 32 lanes of one warp
        const int lanes = p.group / kV;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = (i * blockDim.x + threadIdx.x) * kV;
            uint32_t mm = m[i];
            for (int o = lanes >> 1; o > 0; o >>= 1) mm = max(mm, __shfl_xor_sync(0xffffffffu, mm, o));
            float scale, inv;
            scale_of(mm, p.q_type, scale, inv);
            if (k < K) {
                if ((threadIdx.x & (lanes - 1)) == 0) p.scales[t * (K / p.group) + k / p.group] = scale;
                store_codes(q + k, K - k, vec, inv == 0.0f ? make_uint2(0u, 0u) : codes8(v[i], inv, p.q_type));
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scales, int K, int q_type, int group,
                      bool vec, T* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int k = (blockIdx.y * blockDim.x + threadIdx.x) * kV;
    if (k >= K) return;
    const float s = __ldg(scales + (group ? t * (K / group) + k / group : t));   // a group is a multiple of 8
    const uint8_t* src = q + t * K + k;
    uint32_t w[2] = {0u, 0u};
    if (vec) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(src));
        w[0] = c.x;
        w[1] = c.y;
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (k + i < K) w[i >> 2] |= static_cast<uint32_t>(src[i]) << (8 * (i & 3));
    }
    float v[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const uint8_t b = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
        const float c = q_type == kInt8 ? static_cast<float>(static_cast<int8_t>(b))
                                        : __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
        v[i] = c * s;
    }
    store8(out + t * K + k, K - k, vec, v);
}

template <RowOp OP, typename T>
cudaError_t launch_typed(const RowParams& p, cudaStream_t s) {
    const int chunks = (p.K + kV - 1) / kV;
    auto threads = [&](int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; };
    const dim3 grid(static_cast<unsigned>(p.T));
    if (threads(1) <= 256) return launch_pdl(rows_kernel<OP, T, 1>, grid, dim3(threads(1)), 0, s, p);
    if (threads(2) <= 512) return launch_pdl(rows_kernel<OP, T, 2>, grid, dim3(threads(2)), 0, s, p);
    return launch_pdl(rows_kernel<OP, T, 4>, grid, dim3(threads(4)), 0, s, p);
}

template <RowOp OP>
cudaError_t launch_op(int type, const RowParams& p, cudaStream_t s) {
    if (type == kBf16) return launch_typed<OP, __nv_bfloat16>(p, s);
    if (type == kFp16) return launch_typed<OP, __half>(p, s);
    return launch_typed<OP, float>(p, s);
}

}  // namespace

cudaError_t launch_rows(RowOp op, int type, const RowParams& p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    if (op == RowOp::norm) return launch_op<RowOp::norm>(type, p, s);
    if (op == RowOp::swiglu) return launch_op<RowOp::swiglu>(type, p, s);
    return launch_op<RowOp::plain>(type, p, s);
}

cudaError_t launch_dequantize_q8(const void* q, const float* scales, int64_t T, int K, int q_type, int group, int type,
                                 void* out, bool vec, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    const int chunks = (K + kV - 1) / kV;
    const int threads = chunks >= 256 ? 256 : (chunks + 31) / 32 * 32;
    const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>((chunks + threads - 1) / threads));
    const auto* qb = static_cast<const uint8_t*>(q);
    if (type == kBf16)
        return launch_pdl(dequantize_kernel<__nv_bfloat16>, grid, dim3(threads), 0, s, qb, scales, K, q_type, group,
                          vec, static_cast<__nv_bfloat16*>(out));
    if (type == kFp16)
        return launch_pdl(dequantize_kernel<__half>, grid, dim3(threads), 0, s, qb, scales, K, q_type, group, vec,
                          static_cast<__half*>(out));
    return launch_pdl(dequantize_kernel<float>, grid, dim3(threads), 0, s, qb, scales, K, q_type, group, vec,
                      static_cast<float*>(out));
}

}  // namespace wna16
