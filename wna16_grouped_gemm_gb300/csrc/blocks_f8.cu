// Weights to e4m3 with one scale per block of 128 x 128:
//   m = max |w|,  scale = m / 448,  code = e4m3(w * (448 / m))
//
// Bound by the bytes of the weights, read once.  A thread block has one block of
// the weight in registers from its reads to the codes (four of them per SM with 16-bit values, three with fp32; with three, 16 x
// 4096 x 4096 bf16 126 us and transposed 134; with five fp16 135 and 150).
// Measured (us), 16 x 4096 x 4096: fp32 184 (7.3 TB/s), transposed 188; bf16 120 (6.7), transposed 122; fp16 122, 127.  1000 x
// 2048 bf16 2.5, transposed 2.8.  With four blocks per SM the fp16 kernels spill 48 to 96 bytes per thread, bf16 transposed off 16-byte
// boundaries 60.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "f8.h"
#include "ptx.cuh"

namespace wna16 {

namespace {

constexpr int kThreads = 256;
constexpr int kV = 8;                                              // neighbouring values per load
constexpr int kTurns = kScaleBlock * kScaleBlock / (kThreads * kV);
constexpr float kTiny = 7.888609052210118e-31f;                    // 2^-100
constexpr float kQ = 448.0f;

// A thread's 8 neighbouring values, in words (as an array of 16-bit values they cost a permutation each).
template <typename T>
struct alignas(16) Chunk {
    static constexpr int kPer = 4 / static_cast<int>(sizeof(T));   // values per word
    uint32_t w[kV / kPer];
    __device__ __forceinline__ float operator[](int j) const {
        const uint32_t v = w[j / kPer];
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(v);
        else if constexpr (std::is_same<T, __half>::value)
            return __half2float(__ushort_as_half(static_cast<unsigned short>(j % 2 ? v >> 16 : v & 0xffffu)));
        else
            return __uint_as_float(j % 2 ? v & 0xffff0000u : v << 16);
    }
};
// the values at p, `count` of them, then zeros
template <typename T>
__device__ __forceinline__ Chunk<T> load_some(const T* p, int count) {
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    const Bits* b = reinterpret_cast<const Bits*>(p);
    Chunk<T> c;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const uint32_t v = j < count ? b[j] : 0u;
        if (j % Chunk<T>::kPer == 0)
            c.w[j / Chunk<T>::kPer] = v;
        else
            c.w[j / Chunk<T>::kPer] |= v << 16;
    }
    return c;
}

// Bytes r of the words a become the bytes of word r (byte by byte, by shifts: 16 x 4096 x 4096 bf16 transposed 254 us).
__device__ __forceinline__ void transpose_bytes(const uint32_t (&a)[4], uint32_t (&o)[4]) {
    const uint32_t t0 = __byte_perm(a[0], a[1], 0x5140), t1 = __byte_perm(a[2], a[3], 0x5140);
    const uint32_t t2 = __byte_perm(a[0], a[1], 0x7362), t3 = __byte_perm(a[2], a[3], 0x7362);
    o[0] = __byte_perm(t0, t1, 0x5410);
    o[1] = __byte_perm(t0, t1, 0x7632);
    o[2] = __byte_perm(t2, t3, 0x5410);
    o[3] = __byte_perm(t2, t3, 0x7632);
}

// COLUMNS: w's columns are contiguous (a transposed weight), else its rows.
template <typename T, bool COLUMNS, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) blocks_kernel(const BlocksParams p) {
    __shared__ uint32_t warp_max[kThreads / 32];
    __shared__ alignas(16) uint8_t tile[COLUMNS ? kScaleBlock * kScaleBlock : 16];
    pdl_wait();
    pdl_trigger();
    const int k_blocks = static_cast<int>(p.K / kScaleBlock), n_blocks = static_cast<int>((p.N + kScaleBlock - 1) / kScaleBlock);
    const int64_t b = blockIdx.x;   // (e, n block, k block)
    const int kb = static_cast<int>(b % k_blocks), nb = static_cast<int>(b / k_blocks % n_blocks);
    const int64_t e = b / k_blocks / n_blocks;
    const int64_t n0 = static_cast<int64_t>(nb) * kScaleBlock, k0 = static_cast<int64_t>(kb) * kScaleBlock;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kScaleBlock), p.N - n0));
    const T* w = static_cast<const T*>(p.w) + e * p.se + n0 * p.sn + k0 * p.sk;
    // a thread's 8 values of turn i: `fast` along the contiguous axis, `slow` along the other (with columns,
    // neighbouring k in its turns: 8 x 8 values, whose codes are 8 bytes of each of 8 rows)
    const int fast = threadIdx.x % (kScaleBlock / kV) * kV, group = threadIdx.x / (kScaleBlock / kV);
    constexpr int kGroups = kThreads / (kScaleBlock / kV);
    static_assert(kTurns == kV, "8 x 8");
    auto slow_of = [&](int i) { return COLUMNS ? group * kTurns + i : group + i * kGroups; };
    Chunk<T> c[kTurns];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int slow = slow_of(i);
        const T* at = w + (COLUMNS ? slow * p.sk : slow * p.sn) + fast;
        const int count = COLUMNS ? rows - fast : (slow < rows ? kV : 0);
        if (VEC && count >= kV) {
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(c[i]) / 16); ++j)
                reinterpret_cast<uint4*>(c[i].w)[j] = reinterpret_cast<const uint4*>(at)[j];
        } else {
            c[i] = load_some(at, count);
        }
    }
    // the largest magnitude as bits: infinities and NaN are above all numbers
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
#pragma unroll
        for (int j = 0; j < kV; ++j) top = max(top, __float_as_uint(c[i][j]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, warp_max[i]);
    const float m = __uint_as_float(top);
    const bool some = m >= kTiny && top < 0x7f800000u;
    const float by = some ? kQ / m : 0.0f;
    if (threadIdx.x == 0) p.scales[b] = m < kTiny ? 0.0f : m / kQ;   // not finite where m is not
    uint8_t* q = p.q + (e * p.N + n0) * p.K + k0;
    // the codes of turn i
    auto codes_of = [&](int i, uint32_t (&code)[2]) {
        code[0] = code[1] = 0;
        if (!some) return;
#pragma unroll
        for (int j = 0; j < kV; j += 2) {
            const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(c[i][j] * by, c[i][j + 1] * by),
                                                          __NV_SATFINITE, __NV_E4M3);
            code[j / 4] |= two << (j % 4 * 8);
        }
    };
    if constexpr (!COLUMNS) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int slow = slow_of(i);
            uint32_t code[2];
            codes_of(i, code);
            if (slow >= rows) continue;
            uint8_t* to = q + slow * p.K + fast;
            if (reinterpret_cast<uintptr_t>(p.q) % 8 == 0) {
                *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
            } else {
#pragma unroll
                for (int j = 0; j < kV; ++j) to[j] = static_cast<uint8_t>(code[j / 4] >> (j % 4 * 8));
            }
        }
    } else {
        uint32_t code[kTurns][2];
#pragma unroll
        for (int i = 0; i < kTurns; ++i) codes_of(i, code[i]);
        // Row n's 8 bytes of group g lie at place g ^ (n / 8) of its 16: the writes of a warp, 8 bytes to each of 16 rows
        // of different n / 8, then meet no bank twice.
        const int f = fast / kV;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {code[0][h], code[1][h], code[2][h], code[3][h]}, b[4] = {code[4][h], code[5][h], code[6][h], code[7][h]};
            uint32_t lo[4], hi[4];
            transpose_bytes(a, lo);
            transpose_bytes(b, hi);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint2*>(tile + (fast + h * 4 + j) * kScaleBlock + (group ^ f) * 8) = make_uint2(lo[j], hi[j]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * (kScaleBlock / 16); i += kThreads) {
            const int n = i / (kScaleBlock / 16), piece = i % (kScaleBlock / 16), r = n / kV;
            uint4 v = *reinterpret_cast<const uint4*>(tile + n * kScaleBlock + (piece ^ (r >> 1)) * 16);
            if (r & 1) v = make_uint4(v.z, v.w, v.x, v.y);
            uint8_t* to = q + static_cast<int64_t>(n) * p.K + piece * 16;
            if (reinterpret_cast<uintptr_t>(p.q) % 16 == 0) {
                *reinterpret_cast<uint4*>(to) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 16; ++j) to[j] = static_cast<uint8_t>(w[j / 4] >> (j % 4 * 8));
            }
        }
    }
}

template <typename T>
cudaError_t launch(const BlocksParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.E * ((p.N + kScaleBlock - 1) / kScaleBlock) * (p.K / kScaleBlock)));
    const bool columns = p.sk != 1;
    const uint64_t pitch = static_cast<uint64_t>(columns ? p.sk : p.sn) | static_cast<uint64_t>(p.se);
    const bool vec = (pitch * sizeof(T)) % 16 == 0 && reinterpret_cast<uintptr_t>(p.w) % 16 == 0;
    if (columns) return launch_pdl(vec ? blocks_kernel<T, true, true> : blocks_kernel<T, true, false>, grid, dim3(kThreads), 0, s, p);
    return launch_pdl(vec ? blocks_kernel<T, false, true> : blocks_kernel<T, false, false>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_quantize_blocks_f8(int type, const BlocksParams& p, cudaStream_t s) {
    if (type == kBf16) return launch<__nv_bfloat16>(p, s);
    if (type == kFp16) return launch<__half>(p, s);
    return launch<float>(p, s);
}

}  // namespace wna16
