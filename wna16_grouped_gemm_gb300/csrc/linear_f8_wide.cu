// Block-scaled e4m3 product for many rows per weight: out[t][n] = sum_b xs[t][b] ws[n / 128][b] P_b[t][n].
//
// A block of the grid takes tile after tile of 128 rows (the tensor cores' M side) x 256 output channels (the N side):
//   producer (warp 0)     TMA: the rows and the channels x 128 k per stage
//   issuers (warps 2, 3)  one per half of the channels: four tcgen05.mma kind::f8f6f4 of 128 x 128 x 32 per stage, into
//                         alternate accumulators of the half
//   epilogue (8 warps)    thread = row, 128 channels of one scale: sum += P_b * (xs * ws) in registers
// The sum over blocks cannot stay in the accumulator (a block's scales are fp32 numbers of their own), so every
// block passes through registers: one tcgen05.ld and one fused multiply-add per value, beside the tensor cores' work on
// the next block.  That needs 128 sums, two batches of 32 loaded values and little else per thread: the epilogue's
// warps take registers from the others (setmaxnreg).
//
// Bound by what an SM gets from L2: a stage is 48 KB, at 64 bytes a cycle 770 cycles, of 835 that it takes (the tensor cores
// need 512, the multiply-adds 256 issue slots).  Measured (us, 8192 x 4096 x 4096): 114 by itself (2.4 PFLOP/s, 0.64 of twice the
// measured bf16 rate: an 8-bit product has twice the rate of a 16-bit one), 125 to 128 among other calls (with the issuers'
// waits and elections by whole warps 117; then 109 without the multiply-adds or with a quarter
// of the products, 102 with neither).  8192 x 2048 x 4096 64, 1024 x 4096 x 4096 19 (one tile per SM).  256 experts of
// 4096 x 4096, 65536 rows with skewed popularity: 1330 to 1520 (640 tiles of 128 rows for 512 that would be full, 10240 with their
// channels: at the time per tile of the line above 1100; the rest is boxes of rows that another expert follows, stored value by value,
// and weights read again, and is not told apart).  Channels whose rows are not of 16 bytes are stored so throughout: 8192 x 4096 x 4097 384.
// Lists of more than 356 experts leave room for three stages: 64 rows each of 2048 x 1024, per expert 0.597 us, 0.589 with four.
// Tried and not kept: pairs of CTAs (cta_group::2; 32 KB per stage and CTA) 116, by what is not known, and tiles of 256 rows make that
// 1790 for the experts; two blocks per SM with 128 x 128 tiles 147; 16 epilogue warps of 64 channels 128; packed multiply-adds
// (fma.rn.f32x2) 140; stages of weights sent to L2 four to 32 blocks ahead 137, experts 1600 to 2170; three stages and twice
// the room for results 124; results stored without TMA 147.  (All beside 118.)
#include <algorithm>
#include <atomic>

#include "../../include/wna16_moe_f8.h"
#include "gemm.h"
#include "linear_f8.cuh"

namespace wna16 {

namespace {

constexpr int kRows = 128;           // rows of a tile (the M side)
constexpr int kLowRows = 64;         // rows of a lower box (boxes of 32 rows, as many as a tile has: 8192 x 4096 x 4096 142 us, not 118)
constexpr int kTile = 256;           // output channels of a tile
constexpr int kHalf = 128;           // channels of an accumulator: those of one scale
constexpr int kHalves = kTile / kHalf;
constexpr int kProducer = 0, kAlloc = 1, kIssuer = 2, kFirstEpilogue = 4;   // (an issuer per half)
constexpr int kEpilogues = 8;
constexpr int kCols = 128;           // channels of an epilogue warp
constexpr int kThreads = 32 * (kFirstEpilogue + kEpilogues);
// Registers of a thread at launch, then of the first four warps and of the epilogue's.
constexpr int kLaunchRegs = 168, kOtherRegs = 56, kEpilogueRegs = 224;
static_assert(kThreads * kLaunchRegs == 128 * kOtherRegs + (kThreads - 128) * kEpilogueRegs, "a larger sum waits forever");
constexpr int kTmem = 512;
constexpr int kBufs = kTmem / kTile; // accumulators per half
constexpr int kMaxStages = 8;
constexpr int kStageBytes = (kRows + kTile) * kScaleBlock;
constexpr int kBars = 2 * kMaxStages + 2 * kBufs * kHalves + kHalves;
constexpr int kOutRow = 128;         // bytes of a row of results per turn of the store
constexpr int kOutBytes = 32 * kOutRow, kOutSlots = 1;   // of an epilogue warp

__device__ int g_status;   // of calls without a workspace

template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_low, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_out, const LinearF8Launch L) {
    extern __shared__ __align__(1024) uint8_t smem[];   // (the swizzled tiles need it)
    const LinearF8Params& p = L.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = L.stages, blocks = L.blocks;
    uint8_t* sX = smem;
    uint8_t* sW = sX + stages * kRows * kScaleBlock;
    uint8_t* sOut = sW + stages * kTile * kScaleBlock;   // [epilogue warps][kOutSlots][32 rows][kOutRow]
    uint64_t* full = reinterpret_cast<uint64_t*>(sOut + kEpilogues * kOutSlots * kOutBytes);
    uint64_t* empty = full + kMaxStages;
    uint64_t* accfull = empty + kMaxStages;
    uint64_t* accempty = accfull + kBufs * kHalves;    // (both [half][buffer])
    uint64_t* drain = accempty + kBufs * kHalves;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + kHalves);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* rows = reinterpret_cast<int*>(tmem_slot + 2);
    int* tiles = rows + p.E + 1;
    int* status = p.status ? p.status : &g_status;

    const int first = static_cast<int>(blockIdx.x), stride = static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kHalves);
        }
        for (int i = 0; i < kBufs * kHalves; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], kEpilogues / kHalves);
        }
        for (int i = 0; i < kHalves; ++i) mbar_init(&drain[i], 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_low);
        tma_prefetch_desc(&tm_w);
        if (L.wide) tma_prefetch_desc(&tm_out);
    }
    if (warp == kAlloc) {
        tmem_alloc(tmem_slot, kTmem);
        tmem_relinquish();
    }
    // one weight: the first stages of it on their way to L2 while the kernel before finishes (1024 x 4096 x 4096 19.4 us, not 19.9;
    // the tiles for few rows lose by it: 128 x 4096 x 4096 14.4, not 13.8)
    if (!p.offsets) {
        const int nt = first / ((p.T + kRows - 1) / kRows), n = min(kTile, p.N - nt * kTile);
        for (int i = threadIdx.x; i < n * min(stages, blocks); i += kThreads)
            prefetch_l2(p.wq + static_cast<int64_t>(nt * kTile + i % n) * p.K + i / n * kScaleBlock);
    }
    pdl_wait();
    f8_load_offsets(p, rows);
    if (warp == kIssuer) {
        const bool bad = f8_tile_list(p, kRows, rows, tiles);
        if (blockIdx.x == 0 && lane == 0) *status = bad ? kStatusBadRouting : kStatusOk;   // any timeout is seconds away
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();      // (this block has its TMEM: a block of the next kernel cannot take it away)
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int items = tiles[p.E] * L.n_tiles;

    if (warp < kFirstEpilogue) {
        fewer_registers<kOtherRegs>();
        F8Tile tile;
        if (warp == kProducer) {
            if (lane == 0) {
                const uint64_t pol = policy_evict_normal();
                RingSlot st;
                uint32_t issued = 0;
                bool ok = true;
                for (int v = first; v < items && ok; v += stride) {
                    tile.locate(v, L.n_tiles, kRows, rows, tiles, p, status);
                    // a tile of few rows has a lower box (what lies in the others' place goes to sums that are not stored)
                    const bool low = tile.r1 - tile.r0 <= kLowRows;
                    const uint32_t bytes = ((low ? kLowRows : kRows) + kTile) * kScaleBlock;
                    for (int kb = 0; kb < blocks; ++kb, ++issued, st.next(stages)) {
                        if (!wait_inline(smem_u32(&empty[st.i]), st.phase ^ 1u, abort_flag, status)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&full[st.i], bytes);
                        tma_load_3d(sX + st.i * kRows * kScaleBlock, low ? &tm_low : &tm_x, &full[st.i], kb * kScaleBlock, tile.r0, 0, pol);
                        tma_load_3d(sW + st.i * kTile * kScaleBlock, &tm_w, &full[st.i], kb * kScaleBlock, tile.nt * kTile, tile.e, pol);
                    }
                }
                // no copy may be in flight when the block ends: wait for the last issue of every slot
                const uint32_t n = static_cast<uint32_t>(stages);
                for (uint32_t c = issued > n ? issued - n : 0; c < issued; ++c) {
                    const uint32_t a = smem_u32(&full[c % n]);
                    const uint64_t began = globaltimer_ns();
                    while (!mbar_try_wait(a, (c / n) & 1u)) {
                        if (globaltimer_ns() - began > kWaitLimitNs) {
                            atomicExch(status, kStatusTimeout);
                            break;
                        }
                    }
                }
            }
        } else if (warp >= kIssuer && warp < kIssuer + kHalves) {
            if (elect_one(status)) {
                const int half = warp - kIssuer;
                constexpr uint32_t idesc = idesc_e4m3_f32(kRows, kHalf);
                RingSlot st, buf;
                bool ok = true, issued = false;
                for (int v = first; v < items && ok; v += stride) {
                    for (int kb = 0; kb < blocks; ++kb, st.next(stages), buf.next(kBufs)) {
                        const int acc = half * kBufs + buf.i;
                        if (!wait_inline(smem_u32(&full[st.i]), st.phase, abort_flag, status) ||
                            !wait_inline(smem_u32(&accempty[acc]), buf.phase ^ 1u, abort_flag, status)) {
                            ok = false;
                            break;
                        }
                        const uint32_t a = smem_desc_sw128_lo(smem_u32(sX + st.i * kRows * kScaleBlock));
                        const uint32_t b = smem_desc_sw128_lo(smem_u32(sW + (st.i * kHalves + half) * kHalf * kScaleBlock));
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k) tc_mma_f8(tmem + acc * kHalf, a + k * 2, b + k * 2, idesc, k > 0);
                        tc_commit(&accfull[acc]);
                        tc_commit(&empty[st.i]);
                        issued = true;
                    }
                }
                if (issued && (!ok || *abort_flag)) {   // no MMA may still run when TMEM is released
                    tc_commit(&drain[half]);
                    const uint32_t a = smem_u32(&drain[half]);
                    const uint64_t began = globaltimer_ns();
                    while (!mbar_try_wait(a, 0)) {
                        if (globaltimer_ns() - began > kWaitLimitNs) break;
                    }
                }
            }
            __syncwarp();
        }
    } else {
        more_registers<kEpilogueRegs>();
        F8Tile tile;
        const int quarter = warp & 3, half = (warp - kFirstEpilogue) / 4, row = quarter * 32 + lane;
        const uint32_t src = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(half * kBufs * kHalf);
        uint64_t* const accempty0 = accempty + half * kBufs;
        uint64_t* const accfull0 = accfull + half * kBufs;
        const uint32_t slot0 = smem_u32(sOut + (warp - kFirstEpilogue) * kOutSlots * kOutBytes);
        constexpr int kBatches = kCols / 32;
        static_assert(kBatches % 2 == 0 && kBatches > 2, "a block's first batch goes to d[0]");
        bool done = true;   // false: a wait gave up; what is missing is written as NaN
        RingSlot buf;
        for (int v = first; v < items; v += stride) {
            tile.locate(v, L.n_tiles, kRows, rows, tiles, p, status);
            // scales, two blocks ahead (past the ends: the last ones; what they scale is not stored)
            const float* xs = p.xs + static_cast<int64_t>(min(tile.r0 + row, p.T - 1)) * blocks;
            const float* ws = p.ws + (static_cast<int64_t>(tile.e) * L.n_blocks + min(tile.nt * kHalves + half, L.n_blocks - 1)) * blocks;
            float x0 = *xs, w0 = *ws, x1 = xs[min(1, blocks - 1)], w1 = ws[min(1, blocks - 1)];
            float acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
            // Batches of 32 columns, one on its way while the last one is added; over the blocks' borders too.
            uint32_t d[2][32];
            done = done && warp_wait_inline(&accfull0[buf.i], buf.phase, abort_flag, status);
            if (done) {
                tc_fence_after();
                tc_ld_32x32b_x32(src + buf.i * kHalf, d[0]);
            }
            for (int kb = 0; kb < blocks && done; ++kb) {
                const float s = x0 * w0;
                const int now = buf.i;
                buf.next(kBufs);
                bool ready = false;
#pragma unroll
                for (int c = 0; c < kBatches; ++c) {
                    tc_wait_ld();
                    if (c + 1 < kBatches) {
                        tc_ld_32x32b_x32(src + now * kHalf + (c + 1) * 32, d[(c + 1) & 1]);
                        if (c == 0) {
                            ready = mbar_test_wait(smem_u32(&accfull0[buf.i]), buf.phase);
                        } else if (c == 1) {
                            x0 = x1;
                            w0 = w1;
                            x1 = xs[min(kb + 2, blocks - 1)];
                            w1 = ws[min(kb + 2, blocks - 1)];
                        }
                    } else {   // all of it has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&accempty0[now]);
                        if (kb + 1 < blocks) {
                            done = __all_sync(0xffffffffu, ready) || warp_wait_inline(&accfull0[buf.i], buf.phase, abort_flag, status);
                            tc_fence_after();
                            if (done) tc_ld_32x32b_x32(src + buf.i * kHalf, d[0]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) fma_loaded(acc[c * 32 + j], d[c & 1][j], s);
                }
            }
            const int r = tile.r0 + row, n0 = tile.nt * kTile + half * kCols;
            T* out = static_cast<T*>(p.out) + static_cast<int64_t>(r) * p.N + n0;
            const int box_r = r - lane, cols = p.N - n0;   // columns that exist
            const bool mine = r < tile.r1 && in_bounds(r >= 0 && r < p.T, status);
            // What is not always there stands apart: this code runs once per tile, and fetching it is what it costs
            // (with the tests beside every value a tile's end took 20000 cycles).
            if (!done) {
#pragma unroll
                for (int j = 0; j < kCols; ++j) acc[j] = NAN;
            }
            if (p.bias) {
#pragma unroll
                for (int j = 0; j < kCols; ++j) acc[j] += p.bias[min(n0 + j, p.N - 1)];
            }
            if (p.addend && mine) {
                const T* add = static_cast<const T*>(p.addend) + static_cast<int64_t>(r) * p.N + n0;
#pragma unroll
                for (int j = 0; j < kCols; ++j) acc[j] += elem_to_f(add[min(j, cols - 1)]);
            }
            // Boxes of 32 rows x 128 bytes go out by TMA while the next tile is worked on; rows that
            // another expert follows are stored one by one.
            constexpr int kTurn = kOutRow / static_cast<int>(sizeof(T)), kOne = 16 / static_cast<int>(sizeof(T));
            if (L.wide && (box_r + 32 <= tile.r1 || (box_r < tile.r1 && tile.r1 == p.T))) {
#pragma unroll
                for (int c = 0; c < kCols; c += kTurn) {
                    const uint32_t slot = slot0 + (c / kTurn) % kOutSlots * kOutBytes;
                    if (lane == 0) bulk_wait_read<kOutSlots - 1>();   // the slot's last box has been read
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kTurn; i += kOne) {
                        alignas(16) T o[kOne];
#pragma unroll
                        for (int j = 0; j < kOne; ++j) o[j] = elem_from_f<T>(acc[c + i + j]);
                        // 16-byte piece i of row `lane` lies at piece i ^ (lane & 7) (the swizzle)
                        const uint32_t* w = reinterpret_cast<const uint32_t*>(o);
                        st_shared_16(slot + lane * kOutRow + ((i / kOne ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (c < cols) tma_store_3d(&tm_out, slot, n0 + c, box_r, 0);
                        bulk_commit();
                    }
                }
            } else if (mine) {
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    if (j < cols) out[j] = elem_from_f<T>(acc[j]);
            }
            __syncwarp();
        }
        if (L.wide) bulk_wait();
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == kAlloc) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

int cuda_error(cudaError_t e, const char* what) {
    return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

template <typename T>
int launch(LinearF8Launch L, cudaStream_t s) {
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    const LinearF8Params& p = L.p;
    const int fixed = kEpilogues * kOutSlots * kOutBytes + kBars * 8 + 8 + 2 * (p.E + 1) * 4;
    L.stages = std::min((max_smem - fixed) / kStageBytes, kMaxStages);
    if (L.stages < 2) return set_error(WNA16_ERR_UNSUPPORTED, "8-bit float linear: %d bytes of shared memory", fixed + 2 * kStageBytes);
    const int smem = fixed + L.stages * kStageBytes;
    L.wide = p.N * sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
    CUtensorMap tm_x, tm_low, tm_w;
    if (int rc = f8_code_map(&tm_x, p.xq, 1, p.T, p.K, kRows)) return rc;
    if (int rc = f8_code_map(&tm_low, p.xq, 1, p.T, p.K, kLowRows)) return rc;
    if (int rc = f8_code_map(&tm_w, p.wq, p.E, p.N, p.K, kTile)) return rc;
    CUtensorMap tm_out = {};
    if (L.wide) {
        const uint64_t dims[3] = {static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.T), 1};
        const uint64_t strides[2] = {dims[0] * sizeof(T), dims[0] * dims[1] * sizeof(T)};
        const uint32_t box[3] = {kOutRow / sizeof(T), 32, 1};
        const CUtensorMapDataType type = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
        if (int rc = encode_tma_3d(&tm_out, type, p.out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
    }
    auto kern = wide_kernel<T>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), max_smem);
    if (e != cudaSuccess) return cuda_error(e, "shared memory of the 8-bit float linear");
    // the registers that the warps share out have to be those of the launch
    static std::atomic<bool> checked{false};
    if (!checked.load()) {
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kern);
        if (e != cudaSuccess) return cuda_error(e, "cudaFuncGetAttributes");
        if (attr.numRegs != kLaunchRegs)
            return set_error(WNA16_ERR_CUDA, "8-bit float linear: built with %d registers, not %d", attr.numRegs, kLaunchRegs);
        checked.store(true);
    }
    const int64_t most = (static_cast<int64_t>(p.T) + kRows - 1) / kRows + (p.offsets ? std::min(p.E, p.T) - 1 : 0);
    const int64_t items = most * L.n_tiles;
    if (items >= (int64_t(1) << 31)) return set_error(WNA16_ERR_UNSUPPORTED, "8-bit float linear: too many tiles");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(items, sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_error(cudaLaunchKernelEx(&cfg, kern, tm_x, tm_low, tm_w, tm_out, L), "8-bit float linear launch");
}

}  // namespace

int launch_linear_f8_wide(const LinearF8Params& p, cudaStream_t s) {
    LinearF8Launch L;
    L.p = p;
    L.blocks = p.K / kScaleBlock;
    L.n_tiles = (p.N + kTile - 1) / kTile;
    L.n_blocks = (p.N + kScaleBlock - 1) / kScaleBlock;
    if (p.type == kBf16) return launch<__nv_bfloat16>(L, s);
    if (p.type == kFp16) return launch<__half>(L, s);
    return launch<float>(L, s);
}

}  // namespace wna16
