// Rows to 8 bits: residual addition + RMS norm, the clamped SwiGLU, or nothing,
// then one scale and K codes per row (or per group of a row), and back.
//
//   norm    h = x + r,  y = h / sqrt(mean h^2 + eps) * w;  writes h, y (16 bits), y (8 bits)
//   swiglu  y = silu(min(g, L)) * clamp(u, -L, L)
//   plain   y = x
//   m = max |y|,  scale = m / Q,  code = round(y * (Q / m))
//
// Bound by the bytes of the rows, each read and written once, and close behind by
// issue slots (66 % of them used at 8192 x 4096).  One block works on one row: a
// thread owns chunks of 8 consecutive values (chunk i * blockDim + thread, i < CH),
// which stay in registers from the one read of the row to its last write, and one
// block reduction gives both the sum of squares and the maximum (the greatest |h w|
// times 1 / rms is the greatest |y|).  Sums and maxima are fp32.  A block takes row
// after row and has the next one's reads in flight.  Few blocks of more registers
// beat more blocks: norm 8192 x 4096 held to 38 registers and three blocks per SM
// 55.0 us, with 45 and two 49.2.
// Measured (us, of the measured copy bandwidth of 6782 GB/s), back to back:
//   norm 8192 x 4096 bf16, four outputs   49.2   0.91    2047 x 5120 fp16, e4m3 in groups of 128   17.6   0.61
//   swiglu 8192 x 2048 bf16               16.3   0.76    8192 x 4096   30.3   0.82
//   plain 8192 x 4096 bf16                16.5   0.90    back to bf16   16.6   0.89
//   4 rows: norm 2.2, swiglu 1.6 (a launch)
//   fp32: norm 8192 x 4096 89.1   0.94    swiglu 8192 x 2048 22.6   0.98
//   rows that are not read 16 bytes at a time: norm 8192 x 4097 bf16 185   0.24, swiglu 8192 x 2049 28.6   0.43
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

// Two floats in a register pair, for the packed fp32 instructions (one issue slot
// for two results: these kernels are bound by issue slots before memory).
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 parts(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

constexpr int kP = kV / 2;   // pairs per chunk

template <typename T>
__device__ __forceinline__ void to_floats(const Raw<T>& r, F2 (&v)[kP]) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < kP; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else if constexpr (std::is_same<T, __half>::value) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[i] = f2(f.x, f.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kP; ++i)
            v[i] = i & 1 ? f2(__uint_as_float(r.w[i / 2].z), __uint_as_float(r.w[i / 2].w))
                         : f2(__uint_as_float(r.w[i / 2].x), __uint_as_float(r.w[i / 2].y));
    }
}

template <typename T>
__device__ __forceinline__ Raw<T> from_floats(const F2 (&v)[kP]) {
    Raw<T> r;
    uint32_t w[4 * Raw<T>::kWords];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
        const float2 f = parts(v[i]);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else if constexpr (std::is_same<T, __half>::value) {
            const __half2 h = __floats2half2_rn(f.x, f.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            w[2 * i] = __float_as_uint(f.x);
            w[2 * i + 1] = __float_as_uint(f.y);
        }
    }
#pragma unroll
    for (int i = 0; i < Raw<T>::kWords; ++i) r.w[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const F2 (&v)[kP]) {
    const Raw<T> r = from_floats<T>(v);
    if (VEC) {
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
    } else {
        const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < n) p[i] = e[i];
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
__device__ __forceinline__ float max_abs8(const F2 (&v)[kP]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
        const float2 f = parts(v[i]);
        asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(f.x)), "f"(fabsf(f.y)));
    }
    return m;
}

// silu(min(g, L)) * clamp(u, -L, L), with sigmoid(g) = 1 / (1 + 2^t), t = -g log2(e)
// (g in [-100, 100] there: beyond, the sigmoid is 0 or 1 to fp32).  The rounding
// of t is made good, which leaves 2^t off by 5 units of 2^-24 (and 0.2 |g| for
// the constant); the rest is off by 1 to 2 each.  Below g = -87 the sigmoid is
// taken as 0.  NaN passes the clamps.
__device__ __forceinline__ F2 swiglu2(F2 gate, F2 up, float L) {
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
    float2 g = parts(gate), u = parts(up);
    g = make_float2(min_nan(g.x, L), min_nan(g.y, L));
    u = make_float2(max_nan(min_nan(u.x, L), -L), max_nan(min_nan(u.y, L), -L));
    const F2 x = f2(max_nan(min_nan(g.x, 100.0f), -100.0f), max_nan(min_nan(g.y, 100.0f), -100.0f));
    const F2 t = mul2(x, f2(-kLog2e, -kLog2e));
    const F2 rest = fma2(x, f2(kLog2e, kLog2e), t);   // what rounding added to t
    const float2 tt = parts(t);
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(tt.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(tt.y));
    const F2 ee = f2(e.x, e.y);
    const F2 one = f2(1.0f, 1.0f);   // (2^t may be infinite: its factor is positive, so that the sum is too)
    const float2 d = parts(fma2(ee, fma2(rest, f2(-kLn2, -kLn2), one), one));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    return mul2(mul2(f2(g.x, g.y), f2(r.x, r.y)), f2(u.x, u.y));
}

// 8 codes of v * factor in 8 bytes
__device__ __forceinline__ uint2 codes8(const F2 (&v)[kP], float factor, int q_type) {
    uint32_t w[2];
    const F2 ff = f2(factor, factor);
    if (q_type == kInt8) {
        // 1.5 * 2^23 + x holds x rounded to an integer (ties to even) in its low
        // bits; |x| exceeds 127 by at most the roundings before it
        const F2 base = f2(12582912.0f, 12582912.0f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 a = parts(fma2(v[2 * h], ff, base)), b = parts(fma2(v[2 * h + 1], ff, base));
            w[h] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                               __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(parts(mul2(v[2 * h], ff)), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(parts(mul2(v[2 * h + 1], ff)), __NV_SATFINITE, __NV_E4M3);
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
    scale = tiny ? 0.0f : m * (q_type == kInt8 ? 1.0f / 127.0f : 1.0f / 448.0f);
    // not finite: codes 0 (the row reads back as 0 * scale = NaN)
    if (tiny || !(m < INFINITY)) {
        factor = 0.0f;
    } else if (most > 0x1p-100f && most < 0x1p100f) {   // where the fast reciprocal is good to 1 ulp
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(factor) : "f"(most));
        factor *= Q;
    } else {
        factor = Q / most;
        // Below 2^-119 there is no such factor in fp32.  (For an eps above 1e-11 these rows are below 2^-100.)
        if (factor == INFINITY) scale = factor = 0.0f;
    }
}

// Sum (if SUM) and maximum (if MAX) over the block; every thread gets them.  red: this row's 32 + 32 words.
template <bool SUM, bool MAX>
__device__ __forceinline__ void block_reduce(float& sum, float& most, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (SUM) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    // magnitudes order like their bits, with NaN above infinity
    if (MAX) most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu));
    if (nw == 1) return;
    if (lane == 0) {
        if (SUM) red[warp] = sum;
        if (MAX) red[32 + warp] = most;
    }
    __syncthreads();
    if (MAX) most = lane < nw ? red[32 + lane] : 0.0f;
    if (SUM) {
        sum = lane < nw ? red[lane] : 0.0f;
        for (int o = nw > 16 ? 16 : nw > 8 ? 8 : nw > 4 ? 4 : nw > 2 ? 2 : 1; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum = __shfl_sync(0xffffffffu, sum, 0);
    }
    if (MAX) most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
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

// One block per row, row after row; with PREFETCH the next row's values are on
// their way as soon as this row's are in fp32, so that reads stay in flight
// through the reductions and stores.
template <RowOp OP, typename T, int CH, bool VEC, bool PREFETCH>
__global__ void __launch_bounds__(CH == 4 && PREFETCH ? 512 : 1024) rows_kernel(const __grid_constant__ RowParams p) {
    __shared__ float red[2][64];
    pdl_wait();
    pdl_trigger();
    const int K = p.K;
    const int k0 = threadIdx.x * kV, step = blockDim.x * kV;   // this thread's chunks: k0 + i * step
    Input<OP, T> in[PREFETCH ? CH : 1];
    int64_t t = blockIdx.x;
    if constexpr (PREFETCH) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (k0 + i * step < K) load_chunk<OP, T, VEC>(p, t, k0 + i * step, in[i]);
    }
    for (int turn = 0; t < p.T; ++turn, t += gridDim.x) {
        F2 v[CH][kP];   // norm: h, then h * w; swiglu: h
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = k0 + i * step;
            if (k < K) {
                Input<OP, T>& c = in[PREFETCH ? i : 0];
                if constexpr (!PREFETCH) load_chunk<OP, T, VEC>(p, t, k, c);
                to_floats(c.x, v[i]);
                if constexpr (OP == RowOp::norm) {
                    if (p.residual) {
                        F2 a[kP];
                        to_floats(c.y, a);
#pragma unroll
                        for (int j = 0; j < kP; ++j) v[i][j] = add2(v[i][j], a[j]);
                    }
                }
                if constexpr (OP == RowOp::swiglu) {
                    F2 u[kP];
                    to_floats(c.y, u);
#pragma unroll
                    for (int j = 0; j < kP; ++j) v[i][j] = swiglu2(v[i][j], u[j], p.limit);
                }
            }
        }
        if constexpr (PREFETCH) {
            const int64_t after = t + gridDim.x;
            if (after < p.T) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (k0 + i * step < K) load_chunk<OP, T, VEC>(p, after, k0 + i * step, in[i]);
            }
        }
        F2 sum2 = f2(0.0f, 0.0f);
        float most[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = k0 + i * step;
            most[i] = 0.0f;
            if (k < K) {
                if constexpr (OP == RowOp::norm) {
                    if (p.residual_out) store8<T, VEC>(static_cast<T*>(p.residual_out) + t * K + k, K - k, v[i]);
#pragma unroll
                    for (int j = 0; j < kP; ++j) sum2 = fma2(v[i][j], v[i][j], sum2);
                    F2 w[kP];
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
                    for (int j = 0; j < kP; ++j) v[i][j] = mul2(v[i][j], w[j]);
                }
                most[i] = max_abs8(v[i]);
            }
        }
        float row_most = most[0];
#pragma unroll
        for (int i = 1; i < CH; ++i) row_most = max_nan(row_most, most[i]);
        const float2 halves = parts(sum2);
        float sum = halves.x + halves.y, inv = 1.0f;
        if (p.group == 0)
            block_reduce<OP == RowOp::norm, true>(sum, row_most, red[turn & 1]);
        else if (OP == RowOp::norm)
            block_reduce<true, false>(sum, row_most, red[turn & 1]);
        if constexpr (OP == RowOp::norm) {
            inv = rsqrtf(sum / static_cast<float>(K) + p.eps);
            if (p.norm_out) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int k = k0 + i * step;
                    if (k < K) {
                        F2 y[kP];
#pragma unroll
                        for (int j = 0; j < kP; ++j) y[j] = mul2(v[i][j], f2(inv, inv));
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
                    const int k = k0 + i * step;
                    if (k < K) store_codes<VEC>(q + k, K - k, factor == 0.0f ? make_uint2(0u, 0u) : codes8(v[i], factor, p.q_type));
                }
            } else {
                // a group is group / 8 neighbouring chunks: 4, 8, 16 or 32 lanes of one warp
                const int lanes = 1 << (p.group_log - 3);
                float* scales = p.scales + t * (K >> p.group_log);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int k = k0 + i * step;
                    float m = most[i];
                    for (int o = lanes >> 1; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    float scale, factor;
                    scale_of(m, inv, p.q_type, scale, factor);
                    if (k < K) {
                        if ((threadIdx.x & (lanes - 1)) == 0) scales[k >> p.group_log] = scale;
                        store_codes<VEC>(q + k, K - k, factor == 0.0f ? make_uint2(0u, 0u) : codes8(v[i], factor, p.q_type));
                    }
                }
            }
        }
    }
}

// 8 codes as 4 pairs of values
__device__ __forceinline__ void values8(uint32_t lo, uint32_t hi, float scale, int q_type, F2 (&v)[kP]) {
    const uint32_t w[2] = {lo, hi};
    if (q_type == kInt8) {
        // a code plus 128 in the low bits of 2^23 .., less that base: the code
        const F2 base = f2(-8388736.0f, -8388736.0f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u = w[h] ^ 0x80808080u;
            v[2 * h] = add2(f2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)), __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441))), base);
            v[2 * h + 1] = add2(f2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)), __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443))), base);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
            v[i] = f2(f.x, f.y);
        }
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) v[i] = mul2(v[i], f2(scale, scale));
}

// 16 codes per thread.  (Four rows per block with all their reads first were slower:
// 8192 x 4096 21.5 us against 18.8.)
constexpr int kDequant = 16;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const uint8_t* q, const float* scales, int K, int q_type, int group_log,
                      T* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int k = (blockIdx.y * blockDim.x + threadIdx.x) * kDequant;
    if (k >= K) return;
    // (a group is a multiple of 16)
    const float s = scales[group_log ? t * (K >> group_log) + (k >> group_log) : t];
    const uint8_t* src = q + t * K + k;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (VEC) {
        const uint4 c = *reinterpret_cast<const uint4*>(src);
        w[0] = c.x;
        w[1] = c.y;
        w[2] = c.z;
        w[3] = c.w;
    } else {
#pragma unroll
        for (int i = 0; i < kDequant; ++i)
            if (k + i < K) w[i >> 2] |= static_cast<uint32_t>(src[i]) << (8 * (i & 3));
    }
    T* dst = out + t * K + k;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        F2 v[kP];
        values8(w[2 * h], w[2 * h + 1], s, q_type, v);
        store8<T, VEC>(dst + h * kV, K - k - h * kV, v);
    }
}

template <RowOp OP, typename T, int CH, bool VEC, bool PREFETCH>
struct Rows {
    static constexpr auto kern = rows_kernel<OP, T, CH, VEC, PREFETCH>;
    // rows that are worked on at the same time (0: an error)
    static int64_t resident(int threads) {
        static std::atomic<int> known[33];   // blocks per SM, by warps per block
        int per_sm = known[threads / 32].load();
        if (per_sm == 0) {
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0) != cudaSuccess) return 0;
            if (per_sm < 1) per_sm = 1;
            known[threads / 32].store(per_sm);
        }
        int sms = 0, smem = 0;
        return device_limits(sms, smem) == 0 ? static_cast<int64_t>(per_sm) * sms : 0;
    }
    static cudaError_t launch(const RowParams& p, int threads, cudaStream_t s) {
        int64_t blocks = p.T;
        if (PREFETCH) {
            const int64_t most = resident(threads);
            if (most == 0) return cudaErrorInvalidConfiguration;
            if (blocks > most) blocks = most;
        }
        return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, p);
    }
};

template <RowOp OP, typename T, bool VEC>
cudaError_t launch_vec(const RowParams& p, cudaStream_t s) {
    const int chunks = (p.K + kV - 1) / kV;
    auto threads = [&](int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; };
    constexpr bool pre = VEC && sizeof(T) == 2;
    if constexpr (pre) {
        // Chunks per thread, measured (us) at 8192 rows of 4096 (2 x 2048 for swiglu):
        //   norm    1: 49.2, 2: 49.0, 4: 50.6 (without the reads ahead 67, 57, 71); 2047 x 5120 e4m3 in groups
        //           17.6, 19.9, 22.1; 4 rows 2.2, 2.6, 3.1; but 512 rows 6.0, 5.3, 6.3: there 2 have all
        //           rows worked on at the same time and 1 has not
        //   swiglu  1: 19.4, 2: 17.0, 4: 16.8
        //   plain   1: 19.8, 2: 18.6, 4: 16.7; in groups 11.5, 10.9, 13.2 (4096 rows)
        if (OP == RowOp::norm && threads(1) <= 1024) {
            const bool two = threads(2) <= 512 && p.T > Rows<OP, T, 1, VEC, true>::resident(threads(1)) &&
                             p.T <= Rows<OP, T, 2, VEC, true>::resident(threads(2));
            if (!two) return Rows<OP, T, 1, VEC, true>::launch(p, threads(1), s);
        }
        if (OP == RowOp::plain && p.group == 0 && threads(4) >= 64 && threads(4) <= 512)
            return Rows<OP, T, 4, VEC, true>::launch(p, threads(4), s);
        if (threads(2) <= 1024 && p.K <= 8192) return Rows<OP, T, 2, VEC, true>::launch(p, threads(2), s);
        if (threads(4) <= 512) return Rows<OP, T, 4, VEC, true>::launch(p, threads(4), s);
    }
    // long rows, 4-byte values, unaligned rows
    if (threads(1) <= 256) return Rows<OP, T, 1, VEC, false>::launch(p, threads(1), s);
    if (threads(2) <= 512) return Rows<OP, T, 2, VEC, false>::launch(p, threads(2), s);
    return Rows<OP, T, 4, VEC, false>::launch(p, threads(4), s);
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

cudaError_t launch_rows(RowOp op, int type, RowParams p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    p.group_log = 0;
    while ((1 << p.group_log) < p.group) ++p.group_log;
    if (op == RowOp::norm) return launch_op<RowOp::norm>(type, p, s);
    if (op == RowOp::swiglu) return launch_op<RowOp::swiglu>(type, p, s);
    return launch_op<RowOp::plain>(type, p, s);
}

cudaError_t launch_dequantize_q8(const void* q, const float* scales, int64_t T, int K, int q_type, int group, int type,
                                 void* out, bool vec, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    const int units = (K + kDequant - 1) / kDequant;
    const int threads = units >= 256 ? 256 : (units + 31) / 32 * 32;
    int group_log = 0;
    while ((1 << group_log) < group) ++group_log;
    const auto* qb = static_cast<const uint8_t*>(q);
    const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>((units + threads - 1) / threads));
    auto run = [&](auto* o) {
        using E = std::remove_pointer_t<decltype(o)>;
        return launch_pdl(vec ? dequantize_kernel<E, true> : dequantize_kernel<E, false>, grid, dim3(threads), 0, s, qb,
                          scales, K, q_type, group_log, o);
    };
    if (type == kBf16) return run(static_cast<__nv_bfloat16*>(out));
    if (type == kFp16) return run(static_cast<__half*>(out));
    return run(static_cast<float*>(out));
}

}  // namespace wna16
