// Plans of the block-scaled e4m3 products (linear_f8_thin.cu, linear_f8_wide.cu).
#include <algorithm>

#include "../../include/wna16_moe_f8.h"
#include "gemm.h"
#include "linear_f8.cuh"

namespace wna16 {

int f8_code_map(CUtensorMap* map, const uint8_t* q, int64_t matrices, int64_t rows, int64_t K, int box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows), static_cast<uint64_t>(matrices)};
    const uint64_t strides[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(K) * static_cast<uint64_t>(rows)};
    const uint32_t box[3] = {kScaleBlock, static_cast<uint32_t>(box_rows), 1};
    return encode_tma_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

int run_linear_f8(LinearF8Params p, cudaStream_t s) {
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    const int mean = p.offsets ? (p.T + p.E - 1) / p.E : p.T;
    int nt = 16;
    while (nt < 128 && nt < mean) nt *= 2;
    const int64_t items = ((static_cast<int64_t>(p.T) + nt - 1) / nt + (p.offsets ? std::min(p.E, p.T) - 1 : 0)) * ((p.N + 127) / 128);
    int ksplit = 1;
    while (ksplit < 8 && items * ksplit * 2 <= sms && p.K / kScaleBlock >= ksplit * 4) ksplit *= 2;
    return launch_linear_f8_thin(p, nt, ksplit, s);
}

}  // namespace wna16
