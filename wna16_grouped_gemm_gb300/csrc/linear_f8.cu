// Plans of the block-scaled e4m3 products: which kernel (linear_f8_small.cu, linear_f8_thin.cu,
// linear_f8_wide.cu), how many rows per tile, how many parts of K.
#include <algorithm>

#include "../../include/wna16_moe_f8.h"
#include "gemm.h"
#include "linear_f8.cuh"

namespace wna16 {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Estimated times in us, from calls timed by themselves (T x K x N with weights that are not in L2; small with 8, 16 or
// 32 rows per block / thin with 16 to 128 rows per tile and its best split of K / wide):
//   4 x 4096 x 4096      4.3 / 8.2 / -       77 x 2048 x 1000    4.8 / 7.4 / 10.9     200 x 4096 x 4096   - / 15.4 / 18.2
//   16 x 4096 x 4096     5.8 / 8.2 / -       64 x 4096 x 4096    15.5 / 10.1 / 18.4   512 x 4096 x 4096   - / 22.9 / 18.3
//   32 x 4096 x 4096     8.7 / 9.6 / 18.1   128 x 4096 x 4096   - / 13.7 / 19.2      1024 x 4096 x 4096  - / 41.5 / 19.0
//   4 x 16384 x 4096     15 / 15.9 / -     128 x 4096 x 1024   8.4 / 9.1 / 18.0    1024 x 512 x 4096   - / 16.1 / 7.4
//   4 x 4096 x 32768     26.6 / 29.6 / 43    300 x 1024 x 4096   - / 11.7 / 8.2       64 x 4096 x 16384   - / 17.0 / 21.2
// (Wide tiles with a K shared over a cluster: 128 x 4096 x 4096 17.2 at best, 77 x 2048 x 1000 13.4; the join of 128 x 256
// sums takes 8 us.  Few rows make wide tiles slow where many read the same ones at a time.)
// A launch and a block's way through its prologue, a stage of 128 k, a tile's end, the join of a shared K.
constexpr double kSmallBase = 1.5, kSmallPer4096[3] = {1.8, 2.5, 4.1};   // (8, 16, 32 rows)
constexpr double kThinBase = 4.3, kThinEndRow = 0.018, kThinStage[4] = {0.26, 0.30, 0.34, 0.47}, kThinJoin = 1.0, kThinJoinRow = 0.025;   // (16 .. 128 rows)
constexpr double kWideBase = 3.4, kWideStage = 0.42, kWideEnd = 2.4;
constexpr int kWideRows = 32;   // at least
constexpr double kBytesPerUs = 5.5e6;   // of weights read once by tiles

struct Plan {
    enum { small, thin, wide } kernel = wide;
    int nt = 0, ksplit = 1;
    double us = 1e30;
};

// Clusters of ks blocks, one block per SM, that fit at the same time: a cluster lies in one of eight GPCs.
int64_t clusters(int ks, int sms) { return ks == 1 ? sms : sms / 8 / ks * 8; }

void consider(Plan& best, int kernel, int nt, int ksplit, double us) {
    if (us >= best.us) return;
    best.kernel = static_cast<decltype(best.kernel)>(kernel);
    best.nt = nt;
    best.ksplit = ksplit;
    best.us = us;
}

Plan plan_one_weight(const LinearF8Params& p, int sms) {
    Plan best;
    const int64_t blocks = p.K / kScaleBlock;
    const double bytes = 3.0 + static_cast<double>(p.K) * p.N / kBytesPerUs;
    for (int i = 0; i < 3; ++i) {
        const int64_t groups = ceil_div(p.T, 8 << i);
        if (groups > 65535) continue;   // a grid's limit
        const double per_sm = std::max(1.0, static_cast<double>(groups * ceil_div(p.N, 16)) / sms);
        consider(best, Plan::small, 1 << i, 1, kSmallBase + per_sm * kSmallPer4096[i] * p.K / 4096.0);
    }
    for (int i = 0; i < 4; ++i) {
        const int nt = 16 << i;
        const int64_t tiles = ceil_div(p.T, nt) * ceil_div(p.N, 128);
        for (int ks = 1; ks <= 8 && ks <= blocks; ks *= 2) {
            const int64_t waves = ceil_div(tiles, clusters(ks, sms));
            if (ks > 1 && waves > 1) break;   // a cluster has one tile
            const double us = kThinBase + waves * (ceil_div(blocks, ks) * kThinStage[i] + nt * kThinEndRow) + (ks > 1 ? kThinJoin + nt * kThinJoinRow : 0.0);
            consider(best, Plan::thin, nt, ks, std::max(us, bytes));
        }
    }
    const int64_t waves = ceil_div(ceil_div(p.T, 128) * ceil_div(p.N, 256), sms);
    if (p.T >= kWideRows) consider(best, Plan::wide, 0, 1, std::max(kWideBase + waves * (blocks * kWideStage + kWideEnd), bytes));
    return best;
}

// With a weight per expert the rows of each are known on the device only; the mean decides.  Measured (us, 256 experts of
// 4096 x 4096, rows at random; thin with 16, 32, 64 rows per tile / wide; the weights alone take 632 at the measured copy
// bandwidth, and are read faster where nothing is written):
//   mean 2   516 517 533 / 545      mean 16  715 623 623 / 702      mean 48  1640 1178 667 / 725
//   mean 8   607 608 613 / 650      mean 32  1179 862 654 / 696     mean 64  2095 1325 942 / 722
// (with skewed popularity, mean 8: 643 588 580 / 577, mean 16: 851 718 673 / 660, mean 32: 1250 935 784 / 705: wide tiles lose
// less there than thin ones gain in the first table, so they begin below its crossing.)  Other sizes and fewer experts, whose tiles
// may not fill the SMs, follow the same rule and have not been measured for it; with `expert_begin` the mean counts the slots of
// other experts too.
Plan plan_experts(const LinearF8Params& p, int sms) {
    Plan best;
    const double mean = static_cast<double>(p.T) / p.E;
    if (mean > 40.0) return best;
    best.kernel = Plan::thin;
    best.nt = mean <= 4.0 ? 16 : mean <= 12.0 ? 32 : 64;
    // few tiles whatever the offsets are: a cluster for each
    const int64_t most = (ceil_div(p.T, best.nt) + std::min(p.E, p.T) - 1) * ceil_div(p.N, 128);
    while (best.ksplit < 8 && p.K / kScaleBlock >= 4 * best.ksplit && most <= clusters(2 * best.ksplit, sms)) best.ksplit *= 2;
    return best;
}

}  // namespace

int f8_code_map(CUtensorMap* map, const uint8_t* q, int64_t matrices, int64_t rows, int64_t K, int box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows), static_cast<uint64_t>(matrices)};
    const uint64_t strides[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(K) * static_cast<uint64_t>(rows)};
    const uint32_t box[3] = {kScaleBlock, static_cast<uint32_t>(box_rows), 1};
    return encode_tma_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

int run_linear_f8(const LinearF8Params& p, cudaStream_t s) {
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    const Plan L = p.offsets ? plan_experts(p, sms) : plan_one_weight(p, sms);
    if (L.kernel == Plan::small) return launch_linear_f8_small(p, L.nt, s);
    if (L.kernel == Plan::thin) return launch_linear_f8_thin(p, L.nt, L.ksplit, s);
    return launch_linear_f8_wide(p, s);
}

}  // namespace wna16
