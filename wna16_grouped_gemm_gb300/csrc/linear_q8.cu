// Product of 8-bit integers with a scale per token and per output channel:
//   out[t][n] = (sum_k xq[t][k] wq[n][k]) xs[t] ws[n] (+ bias[n]) (+ addend[t][n])
//
// Two kernels, by the number of tokens:
//
// small_kernel (a few tokens): bound by the weights' bytes.  A block owns 16
// output channels; its 8 warps take the K range in turns of 64, each lane
// loading 16 consecutive bytes of two weight rows straight into the registers
// of two mma.sync m16n8k32 (the order of k inside a product is free, so both
// operands use the order in which the bytes lie).  The integer sums of the
// warps are added in shared memory.
//
// tile_kernel (many tokens): bound by the tensor cores.  sm_103a has no 8-bit
// integer kind of tcgen05.mma, but 8-bit integers are exact in fp16, and their
// products and sums (below 2^24) exact in the fp32 accumulator, so the
// codes run through kind::f16.  The weights are the M side: a block owns 128
// output channels and one tile of tokens.
//   convert kernel            xq -> fp16 in the workspace (rows padded with 0 to a multiple of 64 k)
//   TMA producer (warp 0)     64-k stages: weight codes (128 x 64 bytes) and the token tile (fp16)
//   converter warps (4..11)   thread = weight row: 64 codes -> fp16 -> tcgen05.st into a TMEM buffer
//   MMA issuer (warp 1)       tcgen05.mma, A from TMEM, B from shared memory
//   epilogue (warps 12..19)   tcgen05.ld, scales, bias, addend, store
// The weights' fp16 form never passes through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/wna16_moe_block.h"
#include "block.h"
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

// ------------------------------------------------------------------ few tokens

constexpr int kSmallWarps = 8;
constexpr int kSmallRows = 16;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT tiles of 8 tokens
template <typename T, int NT>
__global__ void __launch_bounds__(32 * kSmallWarps) small_kernel(const LinearParams p) {
    __shared__ int part[kSmallWarps][kSmallRows][NT * 8 + 1];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * kSmallRows;
    const int K = p.K;
    // rows past the end read the last one; their results are not stored
    const int8_t* w0 = p.wq + static_cast<int64_t>(min(n0 + g, p.N - 1)) * K;
    const int8_t* w1 = p.wq + static_cast<int64_t>(min(n0 + g + 8, p.N - 1)) * K;
    const int8_t* x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = p.xq + static_cast<int64_t>(min(j * 8 + g, p.T - 1)) * K;

    int acc[NT][4] = {};
    constexpr int kUnroll = NT <= 2 ? 4 : 2;
    constexpr int kStep = 64 * kSmallWarps;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int k0 = warp * 64; k0 < K; k0 += kStep * kUnroll) {   // the same turns for every lane of the warp
        uint4 a[kUnroll], b[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int k = k0 + u * kStep + q * 16;
            a[u] = k < K ? ld_stream(w0 + k) : zero;
            b[u] = k < K ? ld_stream(w1 + k) : zero;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int k = k0 + u * kStep + q * 16;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint4 c = k < K ? __ldg(reinterpret_cast<const uint4*>(x[j] + k)) : zero;
                mma_s8(acc[j], a[u].x, b[u].x, a[u].y, b[u].y, c.x, c.y);
                mma_s8(acc[j], a[u].z, b[u].z, a[u].w, b[u].w, c.z, c.w);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        part[warp][g][j * 8 + 2 * q] = acc[j][0];
        part[warp][g][j * 8 + 2 * q + 1] = acc[j][1];
        part[warp][g + 8][j * 8 + 2 * q] = acc[j][2];
        part[warp][g + 8][j * 8 + 2 * q + 1] = acc[j][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kSmallRows * NT * 8; i += 32 * kSmallWarps) {
        const int r = i % kSmallRows, t = i / kSmallRows;
        const int n = n0 + r;
        if (n >= p.N || t >= p.T) continue;
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) sum += part[w][r][t];
        float v = static_cast<float>(sum) * __ldg(p.xs + t) * __ldg(p.ws + n);
        if (p.bias) v += __ldg(p.bias + n);
        const int64_t o = static_cast<int64_t>(t) * p.N + n;
        if (p.addend) v += to_f(static_cast<const T*>(p.addend)[o]);
        static_cast<T*>(p.out)[o] = from_f<T>(v);
    }
}

// ------------------------------------------------------------------ many tokens

// 4 codes -> 4 fp16 (exact): the code plus 128 as the low bits of 1024 .. 1279, minus 1152
__device__ __forceinline__ uint2 fp16x4_of(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

constexpr int kConvertThreads = 256;
// x16[t][k] = xq[t][k], k < K; 0 for K <= k < Kp.  16 codes per thread and step; also clears the status word.
__global__ void __launch_bounds__(kConvertThreads)
    convert_kernel(const int8_t* __restrict__ xq, int64_t T, int K, int Kp, __half* __restrict__ x16, int* status) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = kStatusOk;
    const int per_row = Kp / 16;
    const int64_t total = T * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kConvertThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kConvertThreads) {
        const int64_t t = i / per_row;
        const int k = static_cast<int>(i - t * per_row) * 16;
        uint4 c = make_uint4(0, 0, 0, 0);
        if (k < K) c = __ldg(reinterpret_cast<const uint4*>(xq + t * K + k));
        const uint2 a = fp16x4_of(c.x), b = fp16x4_of(c.y), d = fp16x4_of(c.z), e = fp16x4_of(c.w);
        uint4* o = reinterpret_cast<uint4*>(x16 + t * Kp + k);
        o[0] = make_uint4(a.x, a.y, b.x, b.y);
        o[1] = make_uint4(d.x, d.y, e.x, e.y);
    }
}

constexpr int kM = 128;            // weight rows per tile
constexpr int kStageK = 64;        // k per stage and per TMEM buffer (32 columns)
constexpr int kABufs = 8;
constexpr int kProducer = 0, kIssuer = 1, kAlloc = 2;
constexpr int kFirstConverter = 4, kConverters = 8;
constexpr int kFirstEpilogue = kFirstConverter + kConverters, kEpilogues = 8;
constexpr int kTileThreads = 32 * (kFirstEpilogue + kEpilogues);
constexpr int kCols = 512;
constexpr int kMaxStages = 8;

struct TileParams {
    LinearParams p;
    int nt = 0;            // tokens per tile
    int nstage = 0;        // even: a stage's slot belongs to one set of converter warps
    int kblocks = 0;       // stages over the whole K
    int n_tiles = 0, t_tiles = 0;
    int ksplit = 1;
    float* partial = nullptr;   // [ksplit][T][N] (ksplit > 1)
    int* status = nullptr;
};

template <typename T>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                const TileParams tp) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const LinearParams& p = tp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nt = tp.nt, nstage = tp.nstage;
    constexpr int w_bytes = kM * kStageK;
    const int x_bytes = nt * kStageK * 2;
    uint8_t* sX = smem;
    uint8_t* sW = smem + nstage * x_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(sW + nstage * w_bytes);
    uint64_t* empty = full + kMaxStages;
    uint64_t* afull = empty + kMaxStages;
    uint64_t* aempty = afull + kABufs;
    uint64_t* accfull = aempty + kABufs;
    uint64_t* accempty = accfull + 1;
    uint64_t* drain = accempty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < nstage; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kConverters / 2 + 1);   // its converter set's warps and the MMAs' commit
        }
        for (int i = 0; i < kABufs; ++i) {
            mbar_init(&afull[i], kConverters / 2);
            mbar_init(&aempty[i], 1);
        }
        mbar_init(accfull, 1);
        mbar_init(accempty, kEpilogues);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    if (warp == kAlloc) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t a_col = 512 - kABufs * (kStageK / 2);   // accumulator below, buffers above
    pdl_wait();
    pdl_trigger();
    int* status = tp.status;

    const int items = tp.n_tiles * tp.t_tiles * tp.ksplit;
    // item -> (token tile, K split, weight tile), weight tiles fastest
    auto decode = [&](int v, int& n0, int& t0, int& kb0, int& kb1) {
        const int s = v / tp.n_tiles;
        n0 = (v - s * tp.n_tiles) * kM;
        const int split = s % tp.ksplit;
        t0 = (s / tp.ksplit) * nt;
        kb0 = static_cast<int>(static_cast<int64_t>(tp.kblocks) * split / tp.ksplit);
        kb1 = static_cast<int>(static_cast<int64_t>(tp.kblocks) * (split + 1) / tp.ksplit);
        return split;
    };

    if (warp == kProducer) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            const uint32_t tx = static_cast<uint32_t>(w_bytes + x_bytes);
            uint32_t kc = 0;   // stages so far
            bool ok = true;
            for (int v = blockIdx.x; v < items && ok; v += gridDim.x) {
                int n0, t0, kb0, kb1;
                decode(v, n0, t0, kb0, kb1);
                for (int kb = kb0; kb < kb1; ++kb, ++kc) {
                    const int slot = kc % nstage;
                    const uint32_t ph = (kc / nstage) & 1u;
                    if (!mbar_wait(&empty[slot], ph ^ 1u, abort_flag, status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[slot], tx);
                    tma_load_3d(sW + slot * w_bytes, &tm_w, &full[slot], kb * kStageK, n0, 0, pol);
                    tma_load_3d(sX + slot * x_bytes, &tm_x, &full[slot], 0, t0, kb, pol);
                }
            }
            // no copy may be in flight when the block ends: wait for the last issue of every slot
            for (uint32_t c = kc > static_cast<uint32_t>(nstage) ? kc - nstage : 0; c < kc; ++c) {
                const uint32_t a = smem_u32(&full[c % nstage]);
                const uint64_t b = globaltimer_ns();
                while (!mbar_try_wait(a, (c / nstage) & 1u)) {
                    if (globaltimer_ns() - b > kWaitLimitNs) {
                        atomicExch(status, kStatusTimeout);
                        break;
                    }
                }
            }
        }
    } else if (warp == kIssuer) {
        auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool r = true;
            if (lane == 0) r = mbar_wait(bar, parity, abort_flag, status);
            return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
        };
        // f16 A and B, f32 D, both K-major
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(nt >> 3) << 17) | (static_cast<uint32_t>(kM >> 4) << 24);
        uint32_t kc = 0, it = 0;
        bool ok = true, issued = false;
        for (int v = blockIdx.x; v < items && ok; v += gridDim.x, ++it) {
            int n0, t0, kb0, kb1;
            decode(v, n0, t0, kb0, kb1);
            if (!warp_wait(accempty, (it & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            for (int kb = kb0; kb < kb1; ++kb, ++kc) {
                const int slot = kc % nstage;
                const int ab = kc % kABufs;
                if (!warp_wait(&full[slot], (kc / nstage) & 1u) || !warp_wait(&afull[ab], (kc / kABufs) & 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t b_lo = smem_desc_sw128_lo(smem_u32(sX + slot * x_bytes));
                const uint32_t a0 = tmem + a_col + ab * (kStageK / 2);
                if (elect_one(status)) {
                    tc_fence_after();
#pragma unroll
                    for (int k16 = 0; k16 < kStageK / 16; ++k16)
                        tc_mma_ts_lohi(tmem, a0 + k16 * 8, b_lo + k16 * 2, kSmemDescSw128Hi, idesc,
                                       kb > kb0 || k16 > 0 ? 1u : 0u);
                    tc_commit(&aempty[ab]);
                    tc_commit(&empty[slot]);
                    if (kb + 1 == kb1) tc_commit(accfull);
                }
                __syncwarp();
                issued = true;
            }
        }
        if (issued && (!ok || *abort_flag)) {   // no MMA may still run when TMEM is released
            if (elect_one(status)) {
                tc_commit(drain);
                const uint32_t a = smem_u32(drain);
                const uint64_t b = globaltimer_ns();
                while (!mbar_try_wait(a, 0)) {
                    if (globaltimer_ns() - b > kWaitLimitNs) break;
                }
            }
            __syncwarp();
        }
    } else if (warp >= kFirstConverter && warp < kFirstConverter + kConverters) {
        // Two sets of four warps (one warp per TMEM lane quarter) take the stages in
        // turn.  nstage and kABufs are even, so a slot or buffer always
        // belongs to the same set, which waits for each of its phases in order.
        const uint32_t set = static_cast<uint32_t>(warp - kFirstConverter) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t xr = (static_cast<uint32_t>(row) >> 1) & 3u;   // 64-byte swizzle
        const uint32_t abase = tmem + a_col + (static_cast<uint32_t>(quarter * 32) << 16);
        uint32_t kc = 0;
        bool ok = true;
        for (int v = blockIdx.x; v < items && ok; v += gridDim.x) {
            int n0, t0, kb0, kb1;
            decode(v, n0, t0, kb0, kb1);
            for (int kb = kb0; kb < kb1; ++kb, ++kc) {
                if ((kc & 1u) != set) continue;
                const int slot = kc % nstage;
                const int ab = kc % kABufs;
                const uint32_t aph = ((kc / kABufs) & 1u) ^ 1u;
                if (!mbar_wait(&full[slot], (kc / nstage) & 1u, abort_flag, status)) {
                    ok = false;
                    break;
                }
                const bool ready = mbar_test_wait(smem_u32(&aempty[ab]), aph);
                const uint8_t* src = sW + slot * w_bytes + row * kStageK;
                uint32_t a[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4*>(src + ((static_cast<uint32_t>(c) ^ xr) << 4));
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint2 h = fp16x4_of(ww[j]);
                        a[c * 8 + j * 2] = h.x;
                        a[c * 8 + j * 2 + 1] = h.y;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);   // the codes are in registers
                if (!ready && !mbar_wait(&aempty[ab], aph, abort_flag, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                tc_st_32x32b_x32(abase + ab * (kStageK / 2), a);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&afull[ab]);
            }
        }
    } else if (warp >= kFirstEpilogue) {
        // two sets of four warps: the lower and the upper half of the tile's tokens
        const int half = (warp - kFirstEpilogue) >> 2;
        const int quarter = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        uint32_t it = 0;
        for (int v = blockIdx.x; v < items; v += gridDim.x, ++it) {
            int n0, t0, kb0, kb1;
            const int split = decode(v, n0, t0, kb0, kb1);
            if (!mbar_wait_bounded(accfull, it & 1u, abort_flag, status, true)) break;
            tc_fence_after();
            const int n = n0 + quarter * 32 + lane;
            const bool live = n < p.N;
            const float ws = live && tp.ksplit == 1 ? __ldg(p.ws + n) : 1.0f;
            const float bias = live && tp.ksplit == 1 && p.bias ? __ldg(p.bias + n) : 0.0f;
            const int j1 = (half + 1) * (nt / 2);
            for (int j = half * (nt / 2); j < j1; j += 16) {
                uint32_t d[16];
                tc_ld_32x32b_x16(tmem + lane_base + static_cast<uint32_t>(j), d);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = t0 + j + i;
                    if (t < p.T && live && j + i < j1) {
                        const int64_t o = static_cast<int64_t>(t) * p.N + n;
                        if (tp.ksplit > 1) {
                            tp.partial[static_cast<int64_t>(split) * p.T * p.N + o] = __uint_as_float(d[i]);
                        } else {
                            float r = __uint_as_float(d[i]) * __ldg(p.xs + t) * ws;
                            if (p.bias) r += bias;
                            if (p.addend) r += to_f(static_cast<const T*>(p.addend)[o]);
                            static_cast<T*>(p.out)[o] = from_f<T>(r);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(accempty);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kAlloc) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// sums of the K splits in split order, then the epilogue
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const LinearParams p, const float* __restrict__ partial, int ksplit) {
    pdl_wait();
    pdl_trigger();
    const int64_t total = static_cast<int64_t>(p.T) * p.N;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / p.N;
        const int n = static_cast<int>(i - t * p.N);
        float s = 0.0f;
        for (int k = 0; k < ksplit; ++k) s += partial[k * total + i];
        s = s * __ldg(p.xs + t) * __ldg(p.ws + n);
        if (p.bias) s += __ldg(p.bias + n);
        if (p.addend) s += to_f(static_cast<const T*>(p.addend)[i]);
        static_cast<T*>(p.out)[i] = from_f<T>(s);
    }
}

// ------------------------------------------------------------------ plans

constexpr int kSmallTokens = 32;   // up to here: small_kernel
constexpr int kSms = 152;

struct Plan {
    int nt = 0, ksplit = 1, kblocks = 0, n_tiles = 0, t_tiles = 0;
    int64_t kp = 0;
    size_t status = 0, x16 = 0, partial = 0, total = 0;
};

Plan make_plan(int64_t T, int64_t K, int64_t N) {
    Plan L;
    L.kblocks = static_cast<int>((K + kStageK - 1) / kStageK);
    L.kp = static_cast<int64_t>(L.kblocks) * kStageK;
    L.nt = T <= 64 ? 64 : T <= 128 ? 128 : 256;
    L.n_tiles = static_cast<int>((N + kM - 1) / kM);
    L.t_tiles = static_cast<int>((T + L.nt - 1) / L.nt);
    const int64_t tiles = static_cast<int64_t>(L.n_tiles) * L.t_tiles;
    while (L.ksplit < 8 && tiles * L.ksplit * 2 <= kSms && L.kblocks >= 2 * L.ksplit * 4) L.ksplit *= 2;
    size_t o = 256;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = (o + bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    L.x16 = take(static_cast<size_t>(T * L.kp) * 2);
    L.partial = L.ksplit > 1 ? take(static_cast<size_t>(T * N) * 4 * L.ksplit) : 0;
    L.total = o;
    return L;
}

template <typename T>
cudaError_t launch_small(const LinearParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.N + kSmallRows - 1) / kSmallRows)), block(32 * kSmallWarps);
    if (p.T <= 8) return launch_pdl(small_kernel<T, 1>, grid, block, 0, s, p);
    if (p.T <= 16) return launch_pdl(small_kernel<T, 2>, grid, block, 0, s, p);
    return launch_pdl(small_kernel<T, 4>, grid, block, 0, s, p);
}

template <typename T>
int run_typed(const LinearParams& p, void* workspace, cudaStream_t s) {
    auto cuda_error = [](cudaError_t e, const char* what) {
        return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    };
    if (p.T <= kSmallTokens) return cuda_error(launch_small<T>(p, s), "8-bit linear launch");
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    const Plan L = make_plan(p.T, p.K, p.N);
    auto* base = static_cast<uint8_t*>(workspace);
    auto* x16 = reinterpret_cast<__half*>(base + L.x16);
    TileParams tp;
    tp.p = p;
    tp.nt = L.nt;
    tp.kblocks = L.kblocks;
    tp.n_tiles = L.n_tiles;
    tp.t_tiles = L.t_tiles;
    tp.ksplit = L.ksplit;
    tp.partial = reinterpret_cast<float*>(base + L.partial);
    tp.status = reinterpret_cast<int*>(base);
    const int stage = kM * kStageK + L.nt * kStageK * 2;
    const int bars = 8 * (2 * kMaxStages + 2 * kABufs + 3) + 16;
    int ns = (max_smem - 1024 - bars) / stage;
    ns = (ns > kMaxStages ? kMaxStages : ns) & ~1;
    tp.nstage = ns;
    const int smem = ns * stage + bars + 1024;

    CUtensorMap tm_w, tm_x;
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.N), 1};
        const uint64_t strides[2] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.K) * p.N};
        const uint32_t box[3] = {kStageK, kM, 1};
        if (int rc = encode_tma_3d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.wq, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B))
            return rc;
    }
    {
        const uint64_t dims[3] = {64, static_cast<uint64_t>(p.T), static_cast<uint64_t>(L.kblocks)};
        const uint64_t strides[2] = {static_cast<uint64_t>(L.kp) * 2, 128};
        const uint32_t box[3] = {64, static_cast<uint32_t>(L.nt), 1};
        if (int rc = encode_tma_3d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return rc;
    }
    auto kern = tile_kernel<T>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return cuda_error(e, "shared memory of the 8-bit linear");
    const int64_t units = static_cast<int64_t>(p.T) * (L.kp / 16);
    const int64_t blocks = (units + kConvertThreads - 1) / kConvertThreads;
    e = launch_pdl(convert_kernel, dim3(static_cast<unsigned>(blocks < 8 * sms ? blocks : 8 * sms)), dim3(kConvertThreads), 0, s,
                   p.xq, static_cast<int64_t>(p.T), p.K, static_cast<int>(L.kp), x16, tp.status);
    if (e != cudaSuccess) return cuda_error(e, "8-bit linear conversion launch");
    const int64_t items = static_cast<int64_t>(L.n_tiles) * L.t_tiles * L.ksplit;
    e = launch_pdl(kern, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(kTileThreads),
                   static_cast<size_t>(smem), s, tm_w, tm_x, tp);
    if (e != cudaSuccess) return cuda_error(e, "8-bit linear launch");
    if (L.ksplit > 1) {
        const int64_t n = static_cast<int64_t>(p.T) * p.N;
        const int64_t jb = (n + 255) / 256;
        e = launch_pdl(join_kernel<T>, dim3(static_cast<unsigned>(jb < 8 * sms ? jb : 8 * sms)), dim3(256), 0, s, p,
                       static_cast<const float*>(tp.partial), L.ksplit);
        if (e != cudaSuccess) return cuda_error(e, "8-bit linear join launch");
    }
    return WNA16_OK;
}

}  // namespace

size_t linear_q8_workspace(int64_t T, int64_t K, int64_t N) {
    return T <= kSmallTokens ? 0 : make_plan(T, K, N).total;
}

int run_linear_q8(const LinearParams& p, void* workspace, cudaStream_t s) {
    if (p.type == kBf16) return run_typed<__nv_bfloat16>(p, workspace, s);
    if (p.type == kFp16) return run_typed<__half>(p, workspace, s);
    return run_typed<float>(p, workspace, s);
}

}  // namespace wna16
