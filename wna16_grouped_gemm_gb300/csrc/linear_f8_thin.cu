// Block-scaled e4m3 product for few rows per weight: out[t][n] = sum_b xs[t][b] ws[b] P_b[t][n].
//
// Bound by the weights' bytes.  The weights are the tensor cores' M side (tiles of 128
// output channels, which share one scale per block of 128 k) and NT rows of the input the N side:
//   producer (warp 0)   TMA: 128 channels x 128 k and NT rows x 128 k per stage
//   issuer (warp 1)     four tcgen05.mma kind::f8f6f4 per stage, into the next of several accumulators
//   scaler (warp 2)     cp.async: the rows' scales of a block, and the weight's
//   epilogue (4 or 8 warps)  thread = channel: sum += P_b * (xs * ws) in registers, then the stores
// A block of the grid takes tile after tile; with few tiles a cluster shares a tile's K, and
// the parts are added in order through distributed shared memory.
// Eight stages of 16 KB of weights are in flight per SM.  The epilogue takes as many blocks at a time as fill 64 registers (half
// as many: 8192 rows of 256 experts 698 us, not 654).  Measured (us): 256 experts of 4096 x 4096 with a row each 599 (7.2 TB/s),
// with 32 each 648, 30 experts with a row or two 83 (6.1 TB/s; start and the last turn of tiles 10); 64 x 4096 x 4096 10.1 (K in
// four parts), 4 x 16384 x 4096 15.9.  With many rows per tile the reads of the rows' scales from shared memory count (every lane
// needs all of them): a stage takes 0.23 us with 16 rows, 0.45 with 128.
#include <algorithm>

#include "../../include/wna16_moe_f8.h"
#include "gemm.h"
#include "linear_f8.cuh"

namespace wna16 {

namespace {

constexpr int kM = 128;
constexpr int kProducer = 0, kIssuer = 1, kScaler = 2, kLister = 3, kFirstEpilogue = 4;
constexpr int kScaleSlots = 16;
// More requests in flight make memory slower, fewer do not fill it.  us with 6, 7, 8, 9 stages, 256 experts of 4096 x 4096:
// 32 rows 86, 85, 84, 84, 512 rows 535, 528, 526, 532, 2048 rows 627, 618, 615, 631 (and 658 with 12).
constexpr int kMaxStages = 8;
constexpr int kAloneBytes = 150 * 1024;

__device__ int g_status;   // of calls without a workspace

template <int NT>
struct Thin {
    static constexpr int kEpilogues = NT >= 64 ? 8 : 4;
    static constexpr int kThreads = 32 * (kFirstEpilogue + kEpilogues);
    static constexpr int kCols = NT * 4 / kEpilogues;          // rows of the input per epilogue warp
    static constexpr int kBufs = 512 / NT < 8 ? 512 / NT : 8;  // accumulators
    static constexpr int kTmem = NT * kBufs;
    static constexpr int kBatch = kCols < 64 ? 64 / kCols : 1; // blocks that the epilogue takes at a time
    static_assert(kBufs >= 2 * kBatch && kBufs % kBatch == 0 && kScaleSlots >= 2 * kBatch, "one batch is on its way while another is added");
    static constexpr int kStageBytes = (kM + NT) * kScaleBlock;
    static constexpr int kScalePitch = NT + 4;                 // floats of a block's scales: the rows', the weight's
    static constexpr int kBars = 2 * kMaxStages + 2 * kBufs + 2 * kScaleSlots + 1;
};

template <typename T, int NT>
__global__ void __launch_bounds__(Thin<NT>::kThreads, 1)
    thin_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                const LinearF8Launch L) {
    using C = Thin<NT>;
    constexpr int kBufs = C::kBufs, kCols = C::kCols;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const LinearF8Params& p = L.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = L.stages, ksplit = L.ksplit;
    uint8_t* sW = smem;
    uint8_t* sX = sW + stages * kM * kScaleBlock;
    float* sums = reinterpret_cast<float*>(sX + stages * NT * kScaleBlock);   // [NT][kM], with a shared K
    float* scales = sums + (ksplit > 1 ? NT * kM : 0);                        // [kScaleSlots][kScalePitch]
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + kScaleSlots * C::kScalePitch);
    uint64_t* empty = full + kMaxStages;
    uint64_t* accfull = empty + kMaxStages;
    uint64_t* accempty = accfull + kBufs;
    uint64_t* sfull = accempty + kBufs;
    uint64_t* sempty = sfull + kScaleSlots;
    uint64_t* drain = sempty + kScaleSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* rows = reinterpret_cast<int*>(tmem_slot + 2);
    int* tiles = rows + p.E + 1;
    int* status = p.status ? p.status : &g_status;

    const int split = ksplit > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = static_cast<int>(blockIdx.x) / ksplit, stride = static_cast<int>(gridDim.x) / ksplit;
    const int kb0 = static_cast<int>(static_cast<int64_t>(L.blocks) * split / ksplit);
    const int kb1 = static_cast<int>(static_cast<int64_t>(L.blocks) * (split + 1) / ksplit);

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], C::kEpilogues);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sfull[i], 32);
            mbar_init(&sempty[i], C::kEpilogues);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    if (warp == kScaler) {
        tmem_alloc(tmem_slot, C::kTmem);
        tmem_relinquish();
    }
    pdl_wait();
    f8_load_offsets(p, rows);
    if (warp == kLister) {
        const bool bad = f8_tile_list(p, NT, rows, tiles);
        if (blockIdx.x == 0 && lane == 0) *status = bad ? kStatusBadRouting : kStatusOk;   // any timeout is seconds away
    }
    tc_fence_before();
    __syncthreads();
    if (ksplit > 1) cluster_sync();   // the others' shared memory is theirs
    tc_fence_after();
    pdl_trigger();                    // (this block has its TMEM: a block of the next kernel cannot take it away)
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int items = tiles[p.E] * L.n_tiles;

    float acc[kCols];
    bool done = true;   // false: a wait gave up; what is missing is written as NaN
    F8Tile tile;
    // one row's sums of this thread's channel
    const int quarter = warp & 3, channel = quarter * 32 + lane, col0 = (warp - kFirstEpilogue) / 4 * kCols;
    auto store = [&](int col, float sum) {
        const int r = tile.r0 + col, n = tile.nt * kM + channel;
        if (r >= tile.r1 || n >= p.N || !in_bounds(r >= 0 && r < p.T, status)) return;
        const int64_t at = static_cast<int64_t>(r) * p.N + n;
        if (p.bias) sum += p.bias[n];
        if (p.addend) sum += elem_to_f(static_cast<const T*>(p.addend)[at]);
        static_cast<T*>(p.out)[at] = elem_from_f<T>(done ? sum : NAN);
    };

    if (warp == kProducer) {
        if (lane == 0) {
            const uint64_t first_use = policy_evict_first(), again = policy_evict_normal();
            RingSlot st;
            uint32_t issued = 0;
            bool ok = true, is_free = false;
            for (int v = first; v < items && ok; v += stride) {
                tile.locate(v, L.n_tiles, NT, rows, tiles, p, status);
                // weights that no other tile reads need not stay in L2
                const uint64_t pol = tiles[tile.e + 1] - tiles[tile.e] > 1 ? again : first_use;
                for (int kb = kb0; kb < kb1; ++kb, ++issued) {
                    if (!is_free && !wait_inline(smem_u32(&empty[st.i]), st.phase ^ 1u, abort_flag, status)) {
                        ok = false;
                        break;
                    }
                    const int at = st.i;
                    st.next(stages);
                    is_free = mbar_test_wait(smem_u32(&empty[st.i]), st.phase ^ 1u);   // (of the next turn: it takes a while)
                    mbar_arrive_expect_tx(&full[at], C::kStageBytes);
                    tma_load_3d(sW + at * kM * kScaleBlock, &tm_w, &full[at], kb * kScaleBlock, tile.nt * kM, tile.e, pol);
                    tma_load_3d(sX + at * NT * kScaleBlock, &tm_x, &full[at], kb * kScaleBlock, tile.r0, 0, again);
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
    } else if (warp == kIssuer) {
        // One thread, without the warp's votes: what a stage costs here bounds a block's rate while memory is not full (votes, and
        // an election per stage: 64 x 4096 x 4096 10.7 us, not 10.1).
        constexpr uint32_t idesc = idesc_e4m3_f32(kM, NT);
        if (elect_one(status)) {
            RingSlot st, buf;
            bool ok = true, issued = false;
            for (int v = first; v < items && ok; v += stride) {
                for (int kb = kb0; kb < kb1; ++kb, st.next(stages), buf.next(kBufs)) {
                    if (!wait_inline(smem_u32(&accempty[buf.i]), buf.phase ^ 1u, abort_flag, status) ||
                        !wait_inline(smem_u32(&full[st.i]), st.phase, abort_flag, status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = smem_desc_sw128_lo(smem_u32(sW + st.i * kM * kScaleBlock));
                    const uint32_t b = smem_desc_sw128_lo(smem_u32(sX + st.i * NT * kScaleBlock));
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_f8(tmem + buf.i * NT, a + k * 2, b + k * 2, idesc, k > 0);
                    tc_commit(&empty[st.i]);
                    tc_commit(&accfull[buf.i]);
                    issued = true;
                }
            }
            if (issued && (!ok || *abort_flag)) {   // no MMA may still run when TMEM is released
                tc_commit(drain);
                const uint32_t a = smem_u32(drain);
                const uint64_t began = globaltimer_ns();
                while (!mbar_try_wait(a, 0)) {
                    if (globaltimer_ns() - began > kWaitLimitNs) break;
                }
            }
        }
        __syncwarp();
    } else if (warp == kScaler) {
        RingSlot sl;
        bool ok = true;
        for (int v = first; v < items && ok; v += stride) {
            tile.locate(v, L.n_tiles, NT, rows, tiles, p, status);
            const float* ws = p.ws + (static_cast<int64_t>(tile.e) * L.n_blocks + tile.nt) * L.blocks;
            for (int kb = kb0; kb < kb1; ++kb, sl.next(kScaleSlots)) {
                if (!warp_wait_all(&sempty[sl.i], sl.phase ^ 1u, abort_flag, status)) {
                    ok = false;
                    break;
                }
                float* to = scales + sl.i * C::kScalePitch;
                for (int j = lane; j < NT; j += 32)   // rows past the end have the last one's; their sums are not stored
                    cp_async<4>(to + j, p.xs + static_cast<int64_t>(min(tile.r0 + j, p.T - 1)) * L.blocks + kb);
                if (lane == 0) cp_async<4>(to + NT, ws + kb);
                cp_async_arrive(&sfull[sl.i]);
            }
        }
        cp_async_wait_all();
    } else if (warp >= kFirstEpilogue) {
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        constexpr int kBatch = C::kBatch;
        // Blocks so far: block i has accumulator i % kBufs and slot i % kScaleSlots of the scales.  Products and copies complete in
        // order, so a batch waits for its last block's (even lanes for the products, odd ones for the scales).  Slots of scales
        // are given back a batch later: an arrival does not wait for the data of loads issued before it.
        uint32_t at = 0;
        int held = 0;
        for (int v = first; v < items; v += stride) {
            tile.locate(v, L.n_tiles, NT, rows, tiles, p, status);
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
            for (int kb = kb0; kb < kb1; kb += kBatch) {
                const int count = min(kBatch, kb1 - kb);
                const uint32_t end = at + count - 1;
                done = done && warp_wait_all(lane & 1 ? &sfull[end % kScaleSlots] : &accfull[end % kBufs],
                                             (lane & 1 ? end / kScaleSlots : end / kBufs) & 1u, abort_flag, status);
                if (!done) break;
                tc_fence_after();
                uint32_t d[kBatch][kCols];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (i < count) {
                        const uint32_t from = tmem + lane_base + (at + i) % kBufs * NT + static_cast<uint32_t>(col0);
#pragma unroll
                        for (int c = 0; c < kCols; c += 16) tc_ld_32x32b_x16(from + c, d[i] + c);
                    }
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane < count) mbar_arrive(&accempty[(at + lane) % kBufs]);
                if (lane < held) mbar_arrive(&sempty[(at - held + lane) % kScaleSlots]);
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (i < count) {
                        const float* s = scales + (at + i) % kScaleSlots * C::kScalePitch;
                        const float ws = s[NT];
#pragma unroll
                        for (int j = 0; j < kCols; j += 4) {
                            const float4 x = *reinterpret_cast<const float4*>(s + col0 + j);
                            fma_loaded(acc[j], d[i][j], x.x * ws);
                            fma_loaded(acc[j + 1], d[i][j + 1], x.y * ws);
                            fma_loaded(acc[j + 2], d[i][j + 2], x.z * ws);
                            fma_loaded(acc[j + 3], d[i][j + 3], x.w * ws);
                        }
                    }
                at += count;
                held = count;
            }
            if (ksplit > 1) break;   // one tile per cluster: joined below
#pragma unroll
            for (int j = 0; j < kCols; ++j) store(col0 + j, acc[j]);
        }
    }
    if (ksplit > 1) {
        // Block d of the cluster gets the others' sums of its share of the tile's rows and adds them in the order of K.
        const int share = NT / ksplit;
        __syncwarp();
        if (warp >= kFirstEpilogue && first < items) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const int col = col0 + j, d = col / share;
                const uint32_t to = smem_u32(sums + (split * share + col - d * share) * kM + channel);
                st_shared_cluster_f32(map_shared(to, static_cast<uint32_t>(d)), done ? acc[j] : NAN);
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= kFirstEpilogue && first < items) {
            for (int j = (warp - kFirstEpilogue) / 4; j < share; j += C::kEpilogues / 4) {
                float sum = 0.0f;
                for (int d = 0; d < ksplit; ++d) sum += sums[(d * share + j) * kM + channel];
                store(split * share + j, sum);
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == kScaler) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

int cuda_error(cudaError_t e, const char* what) {
    return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

template <typename T, int NT>
int launch(LinearF8Launch L, cudaStream_t s) {
    using C = Thin<NT>;
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    const LinearF8Params& p = L.p;
    const int fixed = (L.ksplit > 1 ? NT * kM * 4 : 0) + kScaleSlots * C::kScalePitch * 4 + C::kBars * 8 + 8 + 2 * (p.E + 1) * 4 + 1024;
    L.stages = std::min((max_smem - fixed) / C::kStageBytes, kMaxStages);
    if (L.ksplit > 1) L.stages = std::min(L.stages, std::max(2, (L.blocks + L.ksplit - 1) / L.ksplit));   // one turn
    if (L.stages < 2) return set_error(WNA16_ERR_UNSUPPORTED, "8-bit float linear: %d bytes of shared memory", fixed + 2 * C::kStageBytes);
    // Blocks that share a K wait for one another, and each for its columns of TMEM: two such clusters side
    // by side could hold what the other waits for.  So much shared memory keeps others off their SMs.
    const int smem = std::max(fixed + L.stages * C::kStageBytes, L.ksplit > 1 ? kAloneBytes : 0);
    CUtensorMap tm_w, tm_x;
    if (int rc = f8_code_map(&tm_w, p.wq, p.E, p.N, p.K, kM)) return rc;
    if (int rc = f8_code_map(&tm_x, p.xq, 1, p.T, p.K, NT)) return rc;
    auto kern = thin_kernel<T, NT>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return cuda_error(e, "shared memory of the 8-bit float linear");
    const int64_t most = (static_cast<int64_t>(p.T) + NT - 1) / NT + (p.offsets ? std::min(p.E, p.T) - 1 : 0);
    const int64_t items = most * L.n_tiles;
    if (items >= (int64_t(1) << 31)) return set_error(WNA16_ERR_UNSUPPORTED, "8-bit float linear: too many tiles");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(L.ksplit > 1 ? items * L.ksplit : std::min<int64_t>(items, sms)));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(L.ksplit);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_error(cudaLaunchKernelEx(&cfg, kern, tm_w, tm_x, L), "8-bit float linear launch");
}

template <int NT>
int launch_typed(const LinearF8Launch& L, cudaStream_t s) {
    if (L.p.type == kBf16) return launch<__nv_bfloat16, NT>(L, s);
    if (L.p.type == kFp16) return launch<__half, NT>(L, s);
    return launch<float, NT>(L, s);
}

}  // namespace

int launch_linear_f8_thin(const LinearF8Params& p, int nt, int ksplit, cudaStream_t s) {
    LinearF8Launch L;
    L.p = p;
    L.blocks = p.K / kScaleBlock;
    L.n_tiles = L.n_blocks = (p.N + kScaleBlock - 1) / kScaleBlock;
    L.ksplit = ksplit;
    switch (nt) {
        case 16: return launch_typed<16>(L, s);
        case 32: return launch_typed<32>(L, s);
        case 64: return launch_typed<64>(L, s);
        default: return launch_typed<128>(L, s);
    }
}

}  // namespace wna16
