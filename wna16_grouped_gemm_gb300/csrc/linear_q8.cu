// Product of 8-bit integers with a scale per token and per output channel:
//   out[t][n] = (sum_k xq[t][k] wq[n][k]) xs[t] ws[n] (+ bias[n]) (+ addend[t][n])
//
// Two kernels: small_kernel up to 32 tokens and where it is estimated to be faster
// (few channels: a tile's prologue, ring and join take 4 us), else tile_kernel.
//
// small_kernel: bound by the weights' bytes.  A block owns 16 output channels and up
// to 32 tokens (the weights come from L2 for the second and later groups of tokens);
// its 8 warps take the K range in turns of 64, each lane loading 16 consecutive bytes
// of two weight rows and of a token straight into registers, where they become the
// fp16 operands of four mma.sync m16n8k16 (the order of k inside a product is free,
// so both operands use the order in which the bytes lie).  The fp32 sums of at most 1024 products are exact integers;
// they are added as integers, over the warps in shared memory.  (mma.sync on
// 8-bit integers, a 40th of the fp16 rate on this chip: 4 x 4096 x 4096 5.0 us,
// 32 x 4096 x 4096 17.6 us.)  Measured, tokens x 4096 x 4096: 4 4.7 us (3.6 TB/s),
// 16 6.1, 32 8.3 (the conversions); 4 x 4096 x 32768 24.8 us (5.4 TB/s, 0.80 of the
// measured copy bandwidth); 77 x 2048 x 1000 5.0.
//
// tile_kernel: bound by the tensor cores.  sm_103a has no 8-bit
// integer kind of tcgen05.mma, but 8-bit integers are exact in fp16, and their
// products and sums (up to 2^24) exact in the fp32 accumulator, so the
// codes run through kind::f16.  (A larger sum loses bits in every product of 16 k:
// each of the 16 terms is cut at about 2^-25 of the largest one or of the sum, and the result
// at 2^-23, 5 * 2^-23 together; measured at most 1.7 * 2^-23 of the largest partial sum, for
// 65536 k, products of 1023 after 32768 of 16129.  Sums held in integers, as the other
// kernel has them, would need half of the accumulator's columns and a pass over it
// every 1024 k.)  A pair of CTAs (cta_group::2) owns 256 rows of
// operand A (the M side, 128 per CTA) and a tile of up to 256 rows of operand B
// (half of them in each CTA's shared memory).  A is the weights where tokens are
// few (tiles of B fit them) and the tokens where they are many (a thread then
// holds neighbouring output channels and stores 32 bytes at a time):
//   TMA producer (warp 0)      128-k stages: codes of the CTA's rows of A and B
//   A converters (warps 4..11) thread = row: 128 codes -> fp16 -> TMEM, in two sets for
//   B converters (12..19)      thread = row: 128 codes -> fp16 -> shared memory, even and odd stages
//   MMA issuer (warp 1 of the even CTA)   256 x nt x 128 per pair of operand buffers
//   epilogue (warps 20..27)    tcgen05.ld, scales, bias, addend, store
// (with few rows of B: four sets for A, and the epilogue's warps convert B first)
// Only codes cross the memory system, and A's fp16 form never passes through
// shared memory.  (Operands are handed to the leader's issuer by arrivals that release at CTA
// scope, also from the other CTA; what reads them are the pair's tensor cores.  That this is
// enough is not in the PTX memory model: it rests on the fences before the arrival and on
// the comparison with integers.)  When there are few tiles, 2 to 4 pairs form a cluster
// that shares a tile's K and adds its sums through distributed shared memory.
// Measured, tokens x 4096 x 4096 (of the 1917 TFLOP/s of a measured bf16 product):
// 64 11.6 us, 512 20.6, 1024 24.3, 2048 42.3 (0.85), 4096 79 (0.91), 8192 151 to 160
// (0.90 to 0.95, power); 8192 x 2048 x 4096 88 (0.82: the accumulator takes half of TMEM
// and the operands of a stage the rest, so a tile's epilogue is not under the next
// tile's products; there with a bias 102, an addend 118, fp32 results 102); 2048 has 152 tiles of
// 224 columns, two for each pair.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

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

// 4 codes -> 4 fp16 (exact): the code plus 128 as the low bits of 1024 .. 1279, minus 1152.
// (Masks and a shift in place of the two permutations made the converters a third slower.)
__device__ __forceinline__ uint2 fp16x4_of(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// ------------------------------------------------------------------ few tokens

constexpr int kSmallWarps = 8;
constexpr int kSmallRows = 16;
constexpr int kExactSteps = 16;   // 64-k steps whose sums stay below 2^24 (1024 * 2^14)

__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT tiles of 8 tokens; U steps of 64 k in flight per warp, at least BLOCKS blocks per SM
template <typename T, int NT, int U, int BLOCKS>
__global__ void __launch_bounds__(32 * kSmallWarps, BLOCKS) small_kernel(const LinearParams p, int* status) {
    __shared__ int part[kSmallWarps][kSmallRows][NT * 8 + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * kSmallRows, t0 = blockIdx.y * NT * 8;
    const int K = p.K;
    // the block's weights on their way to L2 while the kernel before finishes (nothing of them is used)
    for (int64_t i = threadIdx.x * 128; i < static_cast<int64_t>(min(kSmallRows, p.N - n0)) * K; i += 32 * kSmallWarps * 128)
        prefetch_l2(p.wq + static_cast<int64_t>(n0) * K + i);
    pdl_wait();
    pdl_trigger();
    if (status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = kStatusOk;
    // rows past the end read the last one; their results are not stored
    const int8_t* w0 = p.wq + static_cast<int64_t>(min(n0 + g, p.N - 1)) * K;
    const int8_t* w1 = p.wq + static_cast<int64_t>(min(n0 + g + 8, p.N - 1)) * K;
    const int8_t* x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = p.xq + static_cast<int64_t>(min(t0 + j * 8 + g, p.T - 1)) * K;

    int sum[NT][4] = {};
    float acc[NT][4] = {};
    constexpr int kStep = 64 * kSmallWarps;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int held = 0;   // steps in acc
    for (int k0 = warp * 64; k0 < K; k0 += kStep * U) {   // the same turns for every lane of the warp
        uint4 a[U], b[U], c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * kStep + q * 16;
            a[u] = k < K ? ld_stream(w0 + k) : zero;
            b[u] = k < K ? ld_stream(w1 + k) : zero;
            c[u] = k < K ? __ldg(reinterpret_cast<const uint4*>(x[0] + k)) : zero;
        }
        if (held + U > kExactSteps) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[j][i] += __float2int_rn(acc[j][i]);
                    acc[j][i] = 0.0f;
                }
            held = 0;
        }
        held += U;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * kStep + q * 16;
            const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
            uint2 fa[4], fb[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                fa[m] = fp16x4_of(aw[m]);
                fb[m] = fp16x4_of(bw[m]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint4 xc = j == 0 ? c[u] : k < K ? __ldg(reinterpret_cast<const uint4*>(x[j] + k)) : zero;
                const uint32_t xw[4] = {xc.x, xc.y, xc.z, xc.w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint2 fx = fp16x4_of(xw[m]);
                    mma_f16(acc[j], fa[m].x, fb[m].x, fa[m].y, fb[m].y, fx.x, fx.y);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[j][i] += __float2int_rn(acc[j][i]);
        part[warp][g][j * 8 + 2 * q] = sum[j][0];
        part[warp][g][j * 8 + 2 * q + 1] = sum[j][1];
        part[warp][g + 8][j * 8 + 2 * q] = sum[j][2];
        part[warp][g + 8][j * 8 + 2 * q + 1] = sum[j][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kSmallRows * NT * 8; i += 32 * kSmallWarps) {
        const int r = i % kSmallRows, tt = i / kSmallRows, t = t0 + tt;
        const int n = n0 + r;
        if (n >= p.N || t >= p.T) continue;
        int total = 0;
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) total += part[w][r][tt];
        float v = static_cast<float>(total) * __ldg(p.xs + t) * __ldg(p.ws + n);
        if (p.bias) v += __ldg(p.bias + n);
        const int64_t o = static_cast<int64_t>(t) * p.N + n;
        if (p.addend) v += to_f(static_cast<const T*>(p.addend)[o]);
        static_cast<T*>(p.out)[o] = from_f<T>(v);
    }
}

// ------------------------------------------------------------------ many tokens

// Position in a ring of n slots and the parity of its current phase.
struct Slot {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

constexpr int kM = 128;            // rows of A per CTA (256 per pair)
constexpr int kStageK = 128;       // k per stage of codes: one 128-byte swizzle row
constexpr int kHalfK = 64;         // k converted at a time: 32 TMEM columns, one 128-byte swizzle row of fp16
constexpr int kBufs = 3;           // operand buffers, one stage each: 64 TMEM columns, two swizzle atoms of fp16
constexpr int kMaxSplit = 4;
constexpr int kProducer = 0, kIssuer = 1, kAlloc = 2;
constexpr int kFirstA = 4, kFirstB = 12, kFirstEpilogue = 20;   // 8 warps each
constexpr int kSet = 4, kEpilogues = 8;
// How the converters are dealt out.  A set takes every kSets-th stage, and slots and
// barriers come in multiples of that: a wait by parity must not take the turn of another
// set at the same barrier for its own.
template <bool SMALL_B>
struct Roles {
    static constexpr int kSets = 2;      // of four warps for A (warps 4..11) and four for B (12..19)
    static constexpr int kBWarps = 4;
    static constexpr int kStages = 4;    // slots of codes
    static constexpr int kFree = 6;      // barriers of the operand buffers' release, in turns
};
// At most 96 rows of B, one item per pair, and enough stages that it is estimated to be faster:
// four sets for A (warps 4..19), and the epilogue's warps convert B before they have anything
// else to do, two per set; twice the slots fit.  Like this / with two sets (us): 64 x 4096 x 4096
// 11.6 / 12.2, 100 x 8192 x 2048 15.0 / 17.6, 128 x 4096 x 4096 13.1 / 13.8, 64 x 4096 x 16384 18.2 / 21.5; but with 6
// stages per pair, 40 x 2048 x 4096, 9.9 / 9.3.  (Six operand buffers, which fit with 64 rows: 64 x 4096 x
// 4096 11.7, 96 x 4096 x 4096 13.1 against 12.3.)
constexpr int kSmallCols = 96;
template <>
struct Roles<true> {
    static constexpr int kSets = 4;
    static constexpr int kBWarps = 2;
    static constexpr int kStages = 8;
    static constexpr int kFree = 12;
};
template <bool SMALL_B>
constexpr int kBars = 2 * Roles<SMALL_B>::kStages + kBufs + Roles<SMALL_B>::kFree + 3;
constexpr int kTileThreads = 32 * (kFirstEpilogue + kEpilogues);
constexpr int kCols = 512;
constexpr uint32_t kACol = 256;    // TMEM: accumulator in columns 0..nt-1, operand buffers from here
constexpr int kMaxCols = 256;      // rows of B per tile (columns of the result)

struct TileParams {
    LinearParams p;
    int nt = 0;            // rows of B per tile, half of them in each CTA of the pair
    int kblocks = 0;       // stages over the whole K
    int m_tiles = 0, c_tiles = 0;   // tiles of 256 rows of A, of nt rows of B
    int addend16 = 0;      // the addend is 16-byte aligned
    int ksplit = 1;        // pairs per cluster: each takes a part of K
    int* status = nullptr;
};

// Operand A: the weights, B: the tokens; with TM the other way round.
template <typename T, bool TM, bool SMALL_B>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const TileParams tp) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const LinearParams& p = tp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t leader = rank & ~1u, side = rank & 1u;
    const int split = static_cast<int>(rank >> 1);
    const int nt = tp.nt, brows = nt / 2, ksplit = tp.ksplit;
    using R = Roles<SMALL_B>;
    constexpr int kStages = R::kStages, kSets = R::kSets, kFree = R::kFree;
    static_assert(kStages % kSets == 0 && kFree % kSets == 0 && kFree % kBufs == 0, "every set has its own");
    constexpr int a_bytes = kM * kStageK;
    const int b_bytes = brows * kStageK;
    const int h_bytes = brows * kStageK * 2;
    uint8_t* sA = smem;
    uint8_t* sB = sA + kStages * a_bytes;
    uint8_t* sH = sB + kStages * b_bytes;      // B's codes as fp16
    float* sScale = reinterpret_cast<float*>(sH + kBufs * h_bytes);   // the scales of B's rows
    uint64_t* full = reinterpret_cast<uint64_t*>(sScale + kMaxCols);
    uint64_t* empty = full + kStages;
    uint64_t* bfull = empty + kStages;         // the leader's: both CTAs' operands of a buffer are in place
    uint64_t* bempty = bfull + kBufs;          // stage s + kBufs waits for the products of stage s at barrier (s + kBufs) % kFree
    uint64_t* accfull = bempty + kFree;
    uint64_t* accempty = accfull + 1;          // the leader's
    uint64_t* drain = accempty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* acc_ok = abort_flag + 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kSet + R::kBWarps);   // a set of either kind of converters
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&bfull[i], 2 * (kSet + R::kBWarps));   // those of both CTAs
        }
        for (int i = 0; i < kFree; ++i) mbar_init(&bempty[i], 1);
        mbar_init(accfull, 1);
        mbar_init(accempty, 2 * kEpilogues);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
    }
    if (warp == kAlloc) {
        tmem_alloc_pair(tmem_slot, kCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                    // the other CTA's barriers exist
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_wait();
    pdl_trigger();
    int* status = tp.status;
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = kStatusOk;   // any timeout is seconds away

    const int items = tp.m_tiles * tp.c_tiles;
    const int first = static_cast<int>(blockIdx.x) / (2 * ksplit);
    const int stride = static_cast<int>(gridDim.x) / (2 * ksplit);
    const int kb0 = static_cast<int>(static_cast<int64_t>(tp.kblocks) * split / ksplit);
    const int kb1 = static_cast<int>(static_cast<int64_t>(tp.kblocks) * (split + 1) / ksplit);
    // item -> (tile of B, tile of A), tiles of A fastest: first rows of this CTA's A and of the pair's B
    auto a_row = [&](int v) { return (v % tp.m_tiles) * (2 * kM) + static_cast<int>(side) * kM; };
    auto b_row = [&](int v) { return (v / tp.m_tiles) * nt; };

    if (warp == kProducer) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            const uint32_t tx = static_cast<uint32_t>(a_bytes + b_bytes);
            Slot st;
            uint32_t kc = 0;   // stages so far
            bool ok = true;
            for (int v = first; v < items && ok; v += stride) {
                const int a0 = a_row(v), b0 = b_row(v) + static_cast<int>(side) * brows;
                for (int kb = kb0; kb < kb1; ++kb, ++kc, st.next(kStages)) {
                    const int slot = st.i;
                    if (!mbar_wait(&empty[slot], st.phase ^ 1u, abort_flag, status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[slot], tx);
                    tma_load_3d(sA + slot * a_bytes, &tm_a, &full[slot], kb * kStageK, a0, 0, pol);
                    tma_load_3d(sB + slot * b_bytes, &tm_b, &full[slot], kb * kStageK, b0, 0, pol);
                }
            }
            // no copy may be in flight when the block ends: wait for the last issue of every slot
            for (uint32_t c = kc > kStages ? kc - kStages : 0; c < kc; ++c) {
                const uint32_t a = smem_u32(&full[c % kStages]);
                const uint64_t b = globaltimer_ns();
                while (!mbar_try_wait(a, (c / kStages) & 1u)) {
                    if (globaltimer_ns() - b > kWaitLimitNs) {
                        atomicExch(status, kStatusTimeout);
                        break;
                    }
                }
            }
        }
    } else if (warp == kIssuer) {
        if (side == 0) {
            auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                bool r = true;
                if (lane == 0) r = mbar_wait(bar, parity, abort_flag, status);
                return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
            };
            // f16 A and B, f32 D, both K-major, 256 x nt
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(nt >> 3) << 17) | (static_cast<uint32_t>((2 * kM) >> 4) << 24);
            const uint16_t mask = static_cast<uint16_t>(3u << rank);
            Slot bs, be;   // operand buffer, and the barrier of its release
            be.i = kBufs;
            uint32_t it = 0;
            bool ok = true, issued = false;
            for (int v = first; v < items && ok; v += stride, ++it) {
                if (!warp_wait(accempty, (it & 1u) ^ 1u)) {
                    ok = false;
                    break;
                }
                for (int kb = kb0; kb < kb1; ++kb, bs.next(kBufs), be.next(kFree)) {
                    const int b = bs.i;
                    if (!warp_wait(&bfull[b], bs.phase)) {
                        ok = false;
                        break;
                    }
                    const uint32_t b_lo = smem_desc_sw128_lo(smem_u32(sH + b * h_bytes));
                    const uint32_t atom = static_cast<uint32_t>(h_bytes) >> 5;   // 64 k of the tokens, >> 4
                    const uint32_t a0 = tmem + kACol + b * (kStageK / 2);
                    if (elect_one(status)) {
                        tc_fence_after();
#pragma unroll
                        for (int k16 = 0; k16 < kStageK / 16; ++k16)
                            tc_mma_ts_pair(tmem, a0 + k16 * 8, b_lo + (k16 >> 2) * atom + (k16 & 3) * 2,
                                           kSmemDescSw128Hi, idesc, kb > kb0 || k16 > 0 ? 1u : 0u);
                        tc_commit_pair(&bempty[be.i], mask);
                        if (kb + 1 == kb1) tc_commit_pair(accfull, mask);
                    }
                    __syncwarp();
                    issued = true;
                }
            }
            if (issued && (!ok || *abort_flag)) {   // no MMA may still run when TMEM is released
                if (elect_one(status)) {
                    tc_commit_pair(drain, static_cast<uint16_t>(1u << rank));
                    const uint32_t a = smem_u32(drain);
                    const uint64_t b = globaltimer_ns();
                    while (!mbar_try_wait(a, 0)) {
                        if (globaltimer_ns() - b > kWaitLimitNs) break;
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp >= kFirstA && (SMALL_B || warp < kFirstEpilogue)) {
        // Converters.  Set s of either kind takes the stages s, s + kSets, .. (With two sets, a half of
        // every stage per set, with twice the waits and arrivals: 2048 x 4096 x 4096 45.3 us against 42.6, 2500 x
        // 8192 x 1536 44.7 against 39.7; only products of a few stages were faster, 100 x 512 x 4096 6.4 against 6.6.)
        // Chunk c of a row lies at chunk c ^ (row & 7) of its 128 bytes (the swizzle), so
        // with the row's part of that in an address, c enters by one exclusive or.
        constexpr int kFirstOfB = SMALL_B ? kFirstEpilogue : kFirstB;
        const bool is_b = warp >= kFirstOfB;
        const uint32_t set = is_b ? static_cast<uint32_t>(warp - kFirstOfB) / R::kBWarps : static_cast<uint32_t>(warp - kFirstA) / kSet;
        // row of A (= TMEM lane) or of this CTA's half of B
        const uint32_t row = static_cast<uint32_t>((is_b ? warp % R::kBWarps : warp & 3) * 32 + lane);
        const uint32_t bfull0 = map_shared(smem_u32(bfull), leader), bempty0 = smem_u32(bempty), empty0 = smem_u32(empty);
        const uint32_t turns = first < items ? static_cast<uint32_t>((items - 1 - first) / stride + 1) : 0;
        const uint32_t total = turns * static_cast<uint32_t>(kb1 - kb0);
        // put(buffer, h, fp16 pairs): 64 converted codes of the row, for the k half h of operand buffer
        // `buffer`; placed(): after both
        auto convert = [&](uint32_t codes, uint32_t code_bytes, auto&& put, auto&& placed) {
            uint32_t src = codes + set * code_bytes, empty_at = empty0 + set * 8;   // this stage's codes
            uint32_t phase = 0, buf = set % kBufs;
            uint32_t free_at = bempty0 + set * 8, free_phase = 0;   // the buffer's barrier of this turn (the first one of each is free)
            for (uint32_t stage = set; stage < total; stage += kSets) {
                if (!mbar_wait_at(empty_at - kStages * 8, phase, abort_flag, status)) return;
                const uint32_t parity = free_phase ^ (free_at < bempty0 + kBufs * 8 ? 1u : 0u);
                const bool ready = mbar_test_wait(free_at, parity);
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    uint32_t a[32];
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c) {
                        const uint4 raw = ld_shared_16(src ^ ((h * 4 + c) << 4));
                        const uint32_t ww[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint2 v = fp16x4_of(ww[j]);
                            a[c * 8 + j * 2] = v.x;
                            a[c * 8 + j * 2 + 1] = v.y;
                        }
                    }
                    if (h == 0 && !ready && !mbar_wait_at(free_at, parity, abort_flag, status)) return;
                    put(buf, h, a);
                }
                // The slot is given back only when every word read from it has been used by a store.
                // An arrival does not wait for the data of loads issued before it: right after
                // them, the loads were served after the refill where the epilogue filled the
                // memory pipe (an addend, fp32 results), and the sums were wrong.
                __syncwarp();
                if (lane == 0) mbar_arrive_at(empty_at);
                placed();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(bfull0 + buf * 8);
                src += kSets * code_bytes;
                empty_at += kSets * 8;
                if (empty_at >= empty0 + kStages * 8) {
                    empty_at -= kStages * 8;
                    src -= kStages * code_bytes;
                    phase ^= 1u;
                }
                free_at += kSets * 8;
                if (free_at >= bempty0 + kFree * 8) {
                    free_at -= kFree * 8;
                    free_phase ^= 1u;
                }
                buf = (buf + kSets) % kBufs;
            }
        };
        if (is_b) {
            if (SMALL_B && first < items) {   // (one item: the scales are not in its way then)
                const float* scale = TM ? p.ws : p.xs;
                const int i = static_cast<int>(threadIdx.x) - 32 * kFirstEpilogue;
                if (i < nt) sScale[i] = __ldg(scale + min(b_row(first) + i, (TM ? p.N : p.T) - 1));
            }
            const bool live = row < static_cast<uint32_t>(brows);   // a tile of fewer rows leaves threads without one
            const uint32_t r = live ? row : 0;
            const uint32_t dst0 = smem_u32(sH) + r * (kHalfK * 2) + ((r & 7u) << 4);
            convert((smem_u32(sB) + r * kStageK) ^ ((r & 7u) << 4), b_bytes, [&](uint32_t b, uint32_t h, const uint32_t (&a)[32]) {
                if (live) {
                    const uint32_t dst = dst0 + b * h_bytes + h * (h_bytes / 2);
#pragma unroll
                    for (uint32_t j = 0; j < 8; ++j) st_shared_16(dst ^ (j << 4), a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]);
                }
            }, [] { fence_proxy_async_shared(); });
        } else {
            const uint32_t a0 = tmem + kACol + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            convert((smem_u32(sA) + row * kStageK) ^ ((row & 7u) << 4), a_bytes, [&](uint32_t b, uint32_t h, const uint32_t (&a)[32]) {
                if (h == 0) tc_fence_after();
                tc_st_32x32b_x32(a0 + b * (kStageK / 2) + h * (kHalfK / 2), a);
            }, [] {
                tc_wait_st();
                tc_fence_before();
            });
        }
    }

    // Epilogue: thread = row of A; two sets of four warps, the lower and the
    // upper half of the tile's columns (rows of B).
    const int eset = (warp - kFirstEpilogue) / kSet;
    const int quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int a_len = TM ? p.T : p.N, b_len = TM ? p.N : p.T;
    const float* a_scale = TM ? p.xs : p.ws;
    const float* b_scale = TM ? p.ws : p.xs;
    bool done = true;   // false: a wait gave up; what is missing is written as NaN
    const int row = quarter * 32 + lane;
    // 16 sums of this thread's row a of A, with the rows b .. b + 15 of B of which `count` exist
    auto emit = [&](int a, float as, float a_bias, int b, int count, const float* scale, const float (&sum)[16]) {
        if (a >= a_len || count <= 0) return;
        float r[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(scale + i);
            // (sum * token scale) * channel scale, in either orientation
            r[i] = TM ? sum[i] * as * x.x : sum[i] * x.x * as;
            r[i + 1] = TM ? sum[i + 1] * as * x.y : sum[i + 1] * x.y * as;
            r[i + 2] = TM ? sum[i + 2] * as * x.z : sum[i + 2] * x.z * as;
            r[i + 3] = TM ? sum[i + 3] * as * x.w : sum[i + 3] * x.w * as;
        }
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] += TM ? __ldg(p.bias + b + (i < count ? i : 0)) : a_bias;
        }
        const int64_t at = TM ? static_cast<int64_t>(a) * p.N + b : static_cast<int64_t>(b) * p.N + a;
        const int64_t step = TM ? 1 : p.N;
        T* out = static_cast<T*>(p.out) + at;
        if (p.addend) {
            const T* add = static_cast<const T*>(p.addend) + at;
            alignas(32) T v[16];
            if (TM && tp.addend16) {
#pragma unroll
                for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
                    reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(add)[i];
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = add[(i < count ? i : 0) * step];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] += to_f(v[i]);
        }
        if constexpr (TM) {   // 16 neighbouring outputs (all exist, on a 32-byte boundary: N is a multiple of 16)
            alignas(32) T v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = from_f<T>(r[i]);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
                st_global_32(reinterpret_cast<uint8_t*>(out) + 32 * i, reinterpret_cast<const uint32_t*>(v) + 8 * i);
        } else if (count >= 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) out[i * step] = from_f<T>(r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < count) out[i * step] = from_f<T>(r[i]);
        }
    };
    auto load_acc = [&](int column, float (&v)[16]) {
        uint32_t d[16];
        tc_ld_32x32b_x16(tmem + lane_base + static_cast<uint32_t>(column), d);
        tc_wait_ld_of(d);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = done ? __uint_as_float(d[i]) : NAN;
    };
    if (warp >= kFirstEpilogue) {
        const uint32_t accempty0 = map_shared(smem_u32(accempty), leader);
        const int thread = threadIdx.x - 32 * kFirstEpilogue;
        uint32_t it = 0;
        for (int v = first; v < items; v += stride, ++it) {
            const int b0 = b_row(v), a = a_row(v) + row;
            const float as = a < a_len ? __ldg(a_scale + a) : 0.0f;
            const float bias = !TM && a < a_len && p.bias ? __ldg(p.bias + a) : 0.0f;
            if (it > 0) named_barrier(1, 32 * kEpilogues);   // the last tile's scales have been read
            if (!SMALL_B)
                for (int i = thread; i < nt; i += 32 * kEpilogues) sScale[i] = __ldg(b_scale + min(b0 + i, b_len - 1));
            // one warp polls; the others wait in a barrier, which costs the converters no issue slots
            if (warp == kFirstEpilogue) {
                done = done && mbar_wait_bounded(accfull, it & 1u, abort_flag, status, true);
                done = __all_sync(0xffffffffu, done);
                if (lane == 0) *acc_ok = done;
            }
            named_barrier(1, 32 * kEpilogues);
            done = *acc_ok != 0;
            tc_fence_after();
            if (ksplit > 1) break;   // one item per cluster: joined below
            for (int j = eset * brows; j < (eset + 1) * brows; j += 16) {
                float s[16];
                load_acc(j, s);
                emit(a, as, bias, b0 + j, b_len - b0 - j, sScale + j, s);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(accempty0);
        }
    }
    if (ksplit > 1) {
        // The cluster's pairs hold sums over parts of K: pair s gets the others'
        // sums of its share of the tile's columns in shared memory (free now: all
        // operands have been read) and adds them in the order of the parts.
        const int share = (nt / 16 + ksplit - 1) / ksplit * 16;   // the last one may be smaller
        const int v = first;
        float* sums = reinterpret_cast<float*>(smem);   // [ksplit][share][kM]
        __syncwarp();
        cluster_sync();
        if (warp >= kFirstEpilogue) {
            for (int d = 0; d < ksplit; ++d) {
                if (d == split) continue;
                const uint32_t to = map_shared(smem_u32(sums + (split * share) * kM + row), static_cast<uint32_t>(2 * d) + side);
                const int mine = min(share, nt - d * share);
                for (int j = eset * 16; j < mine; j += 32) {
                    float x[16];
                    load_acc(d * share + j, x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) st_shared_cluster_f32(to + (j + i) * kM * 4, x[i]);
                }
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= kFirstEpilogue) {
            const int a = a_row(v) + row;
            const float as = a < a_len ? __ldg(a_scale + a) : 0.0f;
            const float bias = !TM && a < a_len && p.bias ? __ldg(p.bias + a) : 0.0f;
            const int mine = min(share, nt - split * share);
            for (int j = eset * 16; j < mine; j += 32) {
                float x[16], s[16];
                load_acc(split * share + j, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.0f;
                for (int d = 0; d < ksplit; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] += d == split ? x[i] : sums[(d * share + j + i) * kM + row];
                const int c = split * share + j;   // column of the tile
                emit(a, as, bias, b_row(v) + c, b_len - b_row(v) - c, sScale + c, s);
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    cluster_sync();     // the pair's TMEM is not in use, and no CTA leaves while another may reach its barriers
    if (warp == kAlloc) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kCols);
    }
}

// Status word of calls without a workspace.
__device__ int g_linear_status;

// ------------------------------------------------------------------ plans

constexpr int kSmallTokens = 32;   // up to here: small_kernel
// Costs in cycles (clock traces): a stage of 128 k is bound by the converters or
// by the tensor cores' 4 cycles per column; a column's way through the epilogue,
// with B's rows as the tokens (2-byte stores) or as the output channels (32-byte
// stores); the join of a shared K.
// With four sets of converters (see Roles) a stage takes less, but the first ones come later.
constexpr double kStageCycles = 1050, kSmallStageCycles = 650, kSmallFillCycles = 3000;
constexpr double kColumnCycles = 21, kRowColumnCycles = 8, kJoinCycles = 3000, kJoinColumnCycles = 20;

// Launch, prologue and exit of a call (tile_kernel, small_kernel), a block of small_kernel, and 1024 k of its 32 tokens.
constexpr double kTileCycles = 4500, kSmallCycles = 3800, kSmallBlockCycles = 1000, kSmallKCycles = 1500;

struct Plan {
    double cycles = 0.0;   // estimated time
    bool tokens_m = false;
    bool small_b = false;   // see Roles
    int nt = 0, ksplit = 1, kblocks = 0, m_tiles = 0, c_tiles = 0;
};

// The plan of least estimated time (cycles).  active[k]: clusters of k + 1 pairs
// that run at the same time; wide: 32-byte stores are possible (without them
// tokens on the M side lose: 3000 x 1024 x 1000 41 us against 14).
Plan make_plan(int64_t T, int64_t K, int64_t N, bool wide, const int (&active)[kMaxSplit]) {
    Plan best;
    const int kblocks = static_cast<int>((K + kStageK - 1) / kStageK);
    for (int tm = 0; tm < (wide ? 2 : 1); ++tm) {
        const int64_t a_len = tm ? T : N, b_len = tm ? N : T;
        const int64_t m_tiles = (a_len + 2 * kM - 1) / (2 * kM);
        const int64_t min_tiles = (b_len + kMaxCols - 1) / kMaxCols;
        // tiles of B of about the same size, as few as fit and some more
        for (int64_t c_tiles = min_tiles; c_tiles <= 4 * min_tiles && c_tiles < min_tiles + 8; ++c_tiles) {
            const int64_t nt = ((b_len + c_tiles - 1) / c_tiles + 31) / 32 * 32;
            if (nt > kMaxCols || nt * (c_tiles - 1) >= b_len) continue;
            const int64_t tiles = m_tiles * c_tiles;
            const double column = tm ? kRowColumnCycles : kColumnCycles;
            for (int ks = 1; ks <= kMaxSplit && ks <= kblocks; ++ks) {
                const int64_t waves = (tiles + active[ks - 1] - 1) / active[ks - 1];
                if (ks > 1 && waves > 1) break;   // (only ever faster for a single wave)
                const int64_t per = (kblocks + ks - 1) / ks;
                const double two_sets = per * std::max(kStageCycles, nt * 4.0);
                const double four_sets = kSmallFillCycles + per * std::max(kSmallStageCycles, nt * 4.0);
                const bool small_b = tm == 0 && nt <= kSmallCols && waves == 1 && four_sets < two_sets;
                const double cost = kTileCycles + waves * ((small_b ? four_sets : two_sets) + nt * column) +
                                    (ks > 1 ? kJoinCycles + nt * kJoinColumnCycles : 0);
                if (best.nt == 0 || cost < best.cycles) {
                    best.cycles = cost;
                    best.tokens_m = tm != 0;
                    best.small_b = small_b;
                    best.nt = static_cast<int>(nt);
                    best.ksplit = ks;
                    best.kblocks = kblocks;
                    best.m_tiles = static_cast<int>(m_tiles);
                    best.c_tiles = static_cast<int>(c_tiles);
                }
            }
        }
    }
    return best;
}

// Estimated time of small_kernel for more than kSmallTokens tokens (32 per block).  Few channels leave
// tile_kernel few tiles, each with the time of a pair's prologue, ring and join; tile_kernel / small_kernel (us):
//   33 x 2048 x 1000 7.7 / 3.7    77 x 2048 x 1000 8.1 / 5.1    128 x 4096 x 1024 10.2 / 7.9   64 x 512 x 512 6.0 / 2.5
//   64 x 4096 x 4096 12.8 / 15.0   100 x 512 x 4096 6.4 / 9.6    256 x 8192 x 512 14.4 / 13.1   40 x 2048 x 4096 9.4 / 8.9
double small_cycles(int64_t T, int64_t K, int64_t N, int sms) {
    const int64_t groups = (T + kSmallTokens - 1) / kSmallTokens;
    const double per_sm = static_cast<double>(groups * ((N + kSmallRows - 1) / kSmallRows)) / sms;
    if (groups > 65535) return HUGE_VAL;   // a grid's limit
    return kSmallCycles + std::max(per_sm, 1.0) * (kSmallBlockCycles + kSmallKCycles * static_cast<double>(K) / 1024.0);
}

// Steps in flight and blocks per SM, measured (us) with the weights streamed from memory:
//   tokens x 4096 x N      4, 4096   4, 32768   16, 4096   16, 32768   32, 4096
//   chosen                 4.7       24.0       6.0        32.7        8.2
//   the other blocks/SM    5.2       27.4       6.6        37.4        8.2
//   twice the steps        4.9       29.8       6.1        34.9        10.3
// More blocks hide one another's loads and ends where there are several turns of
// them; with one turn (at most two blocks per SM) registers for loads count.
// Tokens per block: the fewest of 8, 16, 32 that hold all or leave one block per SM.
template <typename T>
cudaError_t launch_small(const LinearParams& p, int sms, int* status, cudaStream_t s) {
    const int64_t channels = (p.N + kSmallRows - 1) / kSmallRows;
    auto blocks = [&](int nt) { return channels * ((p.T + 8 * nt - 1) / (8 * nt)); };
    int nt = p.T <= 8 ? 1 : p.T <= 16 ? 2 : 4;
    while (nt > 1 && blocks(nt / 2) <= sms) nt /= 2;
    const dim3 grid(static_cast<unsigned>(channels), static_cast<unsigned>(blocks(nt) / channels)), block(32 * kSmallWarps);
    const bool turns = blocks(nt) > 2 * sms;
    if (nt == 1)
        return launch_pdl(turns ? small_kernel<T, 1, 4, 3> : small_kernel<T, 1, 4, 2>, grid, block, 0, s, p, status);
    if (nt == 2)
        return launch_pdl(turns ? small_kernel<T, 2, 2, 4> : small_kernel<T, 2, 2, 2>, grid, block, 0, s, p, status);
    return launch_pdl(small_kernel<T, 4, 2, 2>, grid, block, 0, s, p, status);
}

int cuda_error(cudaError_t e, const char* what) {
    return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The address of g_linear_status on the current device.
int status_word(int** p) {
    constexpr int kDevices = 64;
    static std::atomic<int*> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    *p = dev < kDevices ? known[dev].load() : nullptr;
    if (*p) return WNA16_OK;
    void* a = nullptr;
    e = cudaGetSymbolAddress(&a, g_linear_status);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetSymbolAddress");
    *p = static_cast<int*>(a);
    if (dev < kDevices) known[dev].store(*p);
    return WNA16_OK;
}

// Codes [rows][K] as boxes of `box_rows` rows x 128 k (zeros past the end)
int code_map(CUtensorMap* map, const int8_t* q, int64_t rows, int64_t K, int box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows), 1};
    const uint64_t strides[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(K) * static_cast<uint64_t>(rows)};
    const uint32_t box[3] = {kStageK, static_cast<uint32_t>(box_rows), 1};
    return encode_tma_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Clusters of 1 .. kMaxSplit pairs of `kern` (one CTA per SM) that the device runs at the same time.
template <typename K>
int active_clusters(K kern, int smem, int (&active)[kMaxSplit]) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][kMaxSplit];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    bool all = dev < kDevices;
    for (int i = 0; all && i < kMaxSplit; ++i) all = (active[i] = known[dev][i].load()) > 0;
    if (all) return WNA16_OK;
    e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return cuda_error(e, "shared memory of the 8-bit linear");
    for (int i = 0; i < kMaxSplit; ++i) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(2 * (i + 1));
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(2 * (i + 1)));
        cfg.blockDim = dim3(kTileThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&active[i], kern, &cfg);
        if (e != cudaSuccess || active[i] < 1)
            return cuda_error(e == cudaSuccess ? cudaErrorInvalidConfiguration : e, "cudaOccupancyMaxActiveClusters");
        if (dev < kDevices) known[dev][i].store(active[i]);
    }
    return WNA16_OK;
}

template <typename T, bool TM, bool SMALL_B>
int launch_tiles(const LinearParams& p, const Plan& L, int max_smem, int pairs, void* workspace, cudaStream_t s) {
    TileParams tp;
    tp.p = p;
    tp.nt = L.nt;
    tp.kblocks = L.kblocks;
    tp.m_tiles = L.m_tiles;
    tp.c_tiles = L.c_tiles;
    tp.ksplit = L.ksplit;
    tp.addend16 = reinterpret_cast<uintptr_t>(p.addend) % 16 == 0;
    tp.status = static_cast<int*>(workspace);
    if (!workspace)
        if (int rc = status_word(&tp.status)) return rc;
    const int ring = Roles<SMALL_B>::kStages * (kM + L.nt / 2) * kStageK + kBufs * (L.nt / 2) * kStageK * 2;
    const int sums = L.ksplit > 1 ? L.ksplit * ((L.nt / 16 + L.ksplit - 1) / L.ksplit * 16) * kM * 4 : 0;
    if (sums > ring) return set_error(WNA16_ERR_UNSUPPORTED, "8-bit linear: the join does not fit");   // (the rings hold it)
    const int smem = ring + kMaxCols * 4 + kBars<SMALL_B> * 8 + 16 + 1024;
    if (smem > max_smem) return set_error(WNA16_ERR_UNSUPPORTED, "8-bit linear: %d bytes of shared memory", smem);

    CUtensorMap tm_a, tm_b;
    if (int rc = code_map(&tm_a, TM ? p.xq : p.wq, TM ? p.T : p.N, p.K, kM)) return rc;
    if (int rc = code_map(&tm_b, TM ? p.wq : p.xq, TM ? p.N : p.T, p.K, L.nt / 2)) return rc;
    auto kern = tile_kernel<T, TM, SMALL_B>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return cuda_error(e, "shared memory of the 8-bit linear");
    const int64_t items = static_cast<int64_t>(L.m_tiles) * L.c_tiles;
    // a pair runs item after item; with a shared K every cluster has one item
    const int64_t clusters = L.ksplit > 1 || items < pairs ? items : pairs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * L.ksplit));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(2 * L.ksplit);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_error(cudaLaunchKernelEx(&cfg, kern, tm_a, tm_b, tp), "8-bit linear launch");
}

template <typename T>
int run_typed(const LinearParams& p, void* workspace, cudaStream_t s) {
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    auto* status = static_cast<int*>(workspace);
    auto small = [&] { return cuda_error(launch_small<T>(p, sms, status, s), "8-bit linear launch"); };
    if (p.T <= kSmallTokens) return small();
    int active[kMaxSplit];
    if (int rc = active_clusters(tile_kernel<T, false, false>, max_smem, active)) return rc;
    const bool wide = p.N % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
    const Plan L = make_plan(p.T, p.K, p.N, wide, active);
    if (small_cycles(p.T, p.K, p.N, sms) < L.cycles) return small();
    if (L.tokens_m) return launch_tiles<T, true, false>(p, L, max_smem, active[0], workspace, s);
    return L.small_b ? launch_tiles<T, false, true>(p, L, max_smem, active[0], workspace, s)
                     : launch_tiles<T, false, false>(p, L, max_smem, active[0], workspace, s);
}

}  // namespace

size_t linear_q8_workspace(int64_t T, int64_t, int64_t) { return T <= kSmallTokens ? 0 : 256; }

int run_linear_q8(const LinearParams& p, void* workspace, cudaStream_t s) {
    if (p.type == kBf16) return run_typed<__nv_bfloat16>(p, workspace, s);
    if (p.type == kFp16) return run_typed<__half>(p, workspace, s);
    return run_typed<float>(p, workspace, s);
}

}  // namespace wna16
