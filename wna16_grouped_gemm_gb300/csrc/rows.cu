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

#include <atomic>
#include <type_traits>

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

// 8 values as they lie in memory
template <typename T>
struct Raw {
    static constexpr int kWords = kV * sizeof(T) / 16;
    uint4 w[kWords];
};

// 8 values at p (n of them exist, the others are 0).  Plain loads: the residual
// may be updated in place.
template <typename T, bool VEC>
__device__ __forceinline__ void load_raw(const T* p, int n, Raw<T>& r) {
    if (VEC) {
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
        T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
        for (int i = 0; i < kV; ++i) e[i] = i < n ? p[i] : Elem<T>::from_f(0.0f);
    }
}

template <typename T>
__device__ __forceinline__ void to_floats(const Raw<T>& r, float (&v)[kV]) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = Elem<T>::to_f(e[i]);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[kV]) {
    if (VEC) {
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

// maxima and minima that a NaN wins
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_abs8(const float (&v)[kV]) {
    float m = fabsf(v[0]);
#pragma unroll
    for (int j = 1; j < kV; ++j) m = max_nan(m, fabsf(v[j]));
    return m;
}

// g * sigmoid(g).  2^t with the rounding of t = -g log2(e) made good: off by
// 4 units of 2^-24 (and 0.2 |g| for the constant), the rest by 1 to 2 each.
__device__ __forceinline__ float silu(float g) {
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
    const float t = g * -kLog2e;
    const float rest = fmaf(g, -kLog2e, -t);
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    // (an infinite t has no rest; e is then 0 or infinite already)
    e = fabsf(t) < 1000.0f ? fmaf(e, rest * kLn2, e) : e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r;
}

// 8 codes of v * factor in 8 bytes
__device__ __forceinline__ uint2 codes8(const float (&v)[kV], float factor, int q_type) {
    uint32_t w[2];
    if (q_type == kInt8) {
        // 1.5 * 2^23 + x holds x rounded to an integer (ties to even) in its low
        // bits; |x| exceeds 127 by at most the roundings before it
        uint32_t c[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) c[i] = __float_as_uint(fmaf(v[i], factor, 12582912.0f));
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = __byte_perm(__byte_perm(c[4 * h], c[4 * h + 1], 0x0040), __byte_perm(c[4 * h + 2], c[4 * h + 3], 0x0040), 0x5410);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h] * factor, v[4 * h + 1] * factor), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2] * factor, v[4 * h + 3] * factor), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | (hi << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 c) {
    if (VEC) {
        *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

// Scale of a row (group) with greatest magnitude most * inv, and the factor that
// makes codes of its values before the product with inv.
__device__ __forceinline__ void scale_of(float most, float inv, int q_type, float& scale, float& factor) {
    const float Q = q_type == kInt8 ? 127.0f : 448.0f;
    const float m = most * inv;
    const bool tiny = m < 0x1p-100f;
    scale = tiny ? 0.0f : m / Q;
    // not finite: codes 0 (the row reads back as 0 * scale = NaN)
    factor = tiny || !(m < INFINITY) ? 0.0f : Q / most;
}

// Sum and maximum over the block; every thread gets them.  red: this row's 32 + 32 words.
__device__ __forceinline__ void block_reduce(float& sum, float& most, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // magnitudes order like their bits, with NaN above infinity
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu));
    if (nw == 1) return;
    if (lane == 0) {
        red[warp] = sum;
        red[32 + warp] = most;
    }
    __syncthreads();
    sum = lane < nw ? red[lane] : 0.0f;
    most = lane < nw ? red[32 + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
}

// What a thread reads of a chunk of a row: the values, and a second tensor's
// (norm: the residual, swiglu: the other half of the row).
template <RowOp OP, typename T>
struct Input {
    Raw<T> x;
    Raw<T> y;
};
template <RowOp OP, typename T, bool VEC>
__device__ __forceinline__ void load_chunk(const RowParams& p, int64_t t, int k, Input<OP, T>& in) {
    const T* x = static_cast<const T*>(p.x) + t * p.ldx + k;
    load_raw<T, VEC>(x, p.K - k, in.x);
    if (OP == RowOp::swiglu) load_raw<T, VEC>(x + p.K, p.K - k, in.y);
    if (OP == RowOp::norm && p.residual) load_raw<T, VEC>(static_cast<const T*>(p.residual) + t * p.ldr + k, p.K - k, in.y);
}

// One block per row, row after row; with PREFETCH the next row is on its way
// while a row is worked on, so that reads stay in flight through the reductions.
template <RowOp OP, typename T, int CH, bool VEC, bool PREFETCH>
__global__ void __launch_bounds__(CH >= 4 ? 1024 : 512) rows_kernel(const RowParams p) {
    __shared__ float red[2][64];
    pdl_wait();
    pdl_trigger();
    const int K = p.K;
    Input<OP, T> next[PREFETCH ? CH : 1];
    int64_t t = blockIdx.x;
    if constexpr (PREFETCH) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = (i * blockDim.x + threadIdx.x) * kV;
            if (k < K) load_chunk<OP, T, VEC>(p, t, k, next[i]);
        }
    }
    for (int turn = 0; t < p.T; ++turn) {
        Input<OP, T> in[PREFETCH ? CH : 1];
        if constexpr (PREFETCH) {
#pragma unroll
            for (int i = 0; i < CH; ++i) in[i] = next[i];
            const int64_t after = t + gridDim.x;
            if (after < p.T) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int k = (i * blockDim.x + threadIdx.x) * kV;
                    if (k < K) load_chunk<OP, T, VEC>(p, after, k, next[i]);
                }
            }
        }
        float v[CH][kV];   // norm: h, then h * w; swiglu: h
        float sum = 0.0f, most[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = (i * blockDim.x + threadIdx.x) * kV;
            most[i] = 0.0f;
            if (k < K) {
                Input<OP, T>& c = in[PREFETCH ? i : 0];
                if constexpr (!PREFETCH) load_chunk<OP, T, VEC>(p, t, k, c);
                to_floats(c.x, v[i]);
                if constexpr (OP == RowOp::norm) {
                    if (p.residual) {
                        float a[kV];
                        to_floats(c.y, a);
#pragma unroll
                        for (int j = 0; j < kV; ++j) v[i][j] += a[j];
                        store8<T, VEC>(static_cast<T*>(p.residual_out) + t * K + k, K - k, v[i]);
                    }
#pragma unroll
                    for (int j = 0; j < kV; ++j) sum = fmaf(v[i][j], v[i][j], sum);
                    float w[kV];
                    if (p.weight_f32) {
                        Raw<float> r;
                        load_raw<float, VEC>(static_cast<const float*>(p.weight) + k, K - k, r);
                        to_floats(r, w);
                    } else {
                        Raw<T> r;
                        load_raw<T, VEC>(static_cast<const T*>(p.weight) + k, K - k, r);
                        to_floats(r, w);
                    }
#pragma unroll
                    for (int j = 0; j < kV; ++j) v[i][j] *= w[j];
                }
                if constexpr (OP == RowOp::swiglu) {
                    float u[kV];
                    to_floats(c.y, u);
#pragma unroll
                    for (int j = 0; j < kV; ++j)
                        v[i][j] = silu(min_nan(v[i][j], p.limit)) * max_nan(min_nan(u[j], p.limit), -p.limit);
                }
                most[i] = max_abs8(v[i]);
            }
        }
        float row_most = most[0];
#pragma unroll
        for (int i = 1; i < CH; ++i) row_most = max_nan(row_most, most[i]);
        float inv = 1.0f;
        if (OP == RowOp::norm || p.group == 0) block_reduce(sum, row_most, red[turn & 1]);
        if constexpr (OP == RowOp::norm) {
            inv = rsqrtf(sum / static_cast<float>(K) + p.eps);
            if (p.norm_out) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int k = (i * blockDim.x + threadIdx.x) * kV;
                    if (k < K) {
                        float y[kV];
#pragma unroll
                        for (int j = 0; j < kV; ++j) y[j] = v[i][j] * inv;
                        store8<T, VEC>(static_cast<T*>(p.norm_out) + t * K + k, K - k, y);
                    }
                }
            }
        }
        if (OP != RowOp::norm || p.q) {
            uint8_t* q = static_cast<uint8_t*>(p.q) + t * K;
            if (p.group == 0) {
                float scale, factor;
                scale_of(row_most, inv, p.q_type, scale, factor);
                if (threadIdx.x == 0) p.scales[t] = scale;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int k = (i * blockDim.x + threadIdx.x) * kV;
                    if (k < K) store_codes<VEC>(q + k, K - k, factor == 0.0f ? make_uint2(0u, 0u) : codes8(v[i], factor, p.q_type));
                }
            } else {
                // a group is group / 8 neighbouring chunks: 4, 8, 16 or 32 lanes of one warp
                const int lanes = p.group / kV;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int k = (i * blockDim.x + threadIdx.x) * kV;
                    float m = most[i];
                    for (int o = lanes >> 1; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    float scale, factor;
                    scale_of(m, inv, p.q_type, scale, factor);
                    if (k < K) {
                        if ((threadIdx.x & (lanes - 1)) == 0) p.scales[t * (K / p.group) + k / p.group] = scale;
                        store_codes<VEC>(q + k, K - k, factor == 0.0f ? make_uint2(0u, 0u) : codes8(v[i], factor, p.q_type));
                    }
                }
            }
        }
        t += gridDim.x;
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scales, int K, int q_type, int group,
                      T* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int k = (blockIdx.y * blockDim.x + threadIdx.x) * kV;
    if (k >= K) return;
    const float s = __ldg(scales + (group ? t * (K / group) + k / group : t));   // a group is a multiple of 8
    const uint8_t* src = q + t * K + k;
    uint32_t w[2] = {0u, 0u};
    if (VEC) {
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
    store8<T, VEC>(out + t * K + k, K - k, v);
}

template <RowOp OP, typename T, int CH, bool VEC, bool PREFETCH>
cudaError_t launch_chunks(const RowParams& p, int threads, cudaStream_t s) {
    auto kern = rows_kernel<OP, T, CH, VEC, PREFETCH>;
    int64_t blocks = p.T;
    if (PREFETCH) {
        // as many blocks as run at the same time
        static std::atomic<int> known[33];   // per SM, by warps per block
        int per_sm = known[threads / 32].load();
        if (per_sm == 0) {
            const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0);
            if (e != cudaSuccess) return e;
            if (per_sm < 1) per_sm = 1;
            known[threads / 32].store(per_sm);
        }
        int sms = 0, smem = 0;
        if (device_limits(sms, smem) != 0) return cudaErrorInvalidDevice;
        if (blocks > static_cast<int64_t>(per_sm) * sms) blocks = static_cast<int64_t>(per_sm) * sms;
    }
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, p);
}

template <RowOp OP, typename T, bool VEC>
cudaError_t launch_vec(const RowParams& p, cudaStream_t s) {
    const int chunks = (p.K + kV - 1) / kV;
    auto threads = [&](int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; };
    constexpr bool pre = VEC && sizeof(T) == 2;
    if (threads(1) <= 256) return launch_chunks<OP, T, 1, VEC, pre>(p, threads(1), s);
    if (threads(2) <= 512) return launch_chunks<OP, T, 2, VEC, pre>(p, threads(2), s);
    return launch_chunks<OP, T, 4, VEC, false>(p, threads(4), s);
}

template <RowOp OP, typename T>
cudaError_t launch_typed(const RowParams& p, cudaStream_t s) {
    return p.vec ? launch_vec<OP, T, true>(p, s) : launch_vec<OP, T, false>(p, s);
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
    auto run = [&](auto* o) {
        using T = std::remove_pointer_t<decltype(o)>;
        return vec ? launch_pdl(dequantize_kernel<T, true>, grid, dim3(threads), 0, s, qb, scales, K, q_type, group, o)
                   : launch_pdl(dequantize_kernel<T, false>, grid, dim3(threads), 0, s, qb, scales, K, q_type, group, o);
    };
    if (type == kBf16) return run(static_cast<__nv_bfloat16*>(out));
    if (type == kFp16) return run(static_cast<__half*>(out));
    return run(static_cast<float*>(out));
}

}  // namespace wna16
