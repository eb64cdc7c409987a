// Internal interface of the operators around the routed experts (host side).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace wna16 {

// element types and 8-bit formats (mirror wna16_type / wna16_q8_type)
enum : int { kBf16 = 0, kFp16 = 1, kFp32 = 2 };
enum : int { kInt8 = 0, kE4m3 = 1 };

// Rows to 8 bits (rows.cu).  What a row is before it is quantised:
enum class RowOp { norm, swiglu, plain };

struct RowParams {
    const void* x = nullptr;          // [T, K] (swiglu: [T, 2K], gate | up)
    const void* residual = nullptr;   // norm
    const void* weight = nullptr;     // norm, [K]
    int64_t ldx = 0, ldr = 0;         // row distances in elements
    int64_t T = 0;
    int K = 0;
    int weight_f32 = 0;
    float eps = 0.0f;
    float limit = 0.0f;
    int q_type = kInt8;
    int group = 0;                    // 0: one scale per row
    int group_log = 0;                // log2 of it, set by the launch
    void* q = nullptr;
    float* scales = nullptr;
    void* residual_out = nullptr;
    void* norm_out = nullptr;
    int vec = 0;                      // 16-byte accesses are possible
};

cudaError_t launch_rows(RowOp op, int type, RowParams p, cudaStream_t stream);
cudaError_t launch_dequantize_q8(const void* q, const float* scales, int64_t T, int K, int q_type, int group, int type,
                                 void* out, bool vec, cudaStream_t stream);

// Expert choice (route_scored.cu).
struct ScoredRouteParams {
    const void* logits = nullptr;
    int64_t ld = 0;
    const float* bias = nullptr;
    int T = 0, E = 0;
    int softmax = 0;
    int groups = 1, topk_groups = 1, group_max = 0, topk = 1;
    int group_size = 0, groups_log = 0;   // set by the launch: experts per group, log2 of groups rounded up
    int renormalize = 1;
    float scale = 1.0f;
    int32_t* ids = nullptr;
    float* weights = nullptr;
    int vec = 0;                      // four logits per load are possible
    int bias_vec = 0;                 // four biases per load are possible
};
cudaError_t launch_route_scored(int type, ScoredRouteParams p, cudaStream_t stream);

// 8-bit integer product (linear_q8.cu).
struct LinearParams {
    const int8_t* xq = nullptr;
    const float* xs = nullptr;
    const int8_t* wq = nullptr;
    const float* ws = nullptr;
    const float* bias = nullptr;
    const void* addend = nullptr;
    void* out = nullptr;
    int T = 0, K = 0, N = 0;
    int type = kBf16;
};
size_t linear_q8_workspace(int64_t T, int64_t K, int64_t N);
// returns a wna16_status and sets the error message
int run_linear_q8(const LinearParams& p, void* workspace, cudaStream_t stream);

// Provided by api.cu.
int device_limits(int& sms, int& max_smem);
int encode_tma_3d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, const uint64_t (&dims)[3],
                  const uint64_t (&strides)[2], const uint32_t (&box)[3], CUtensorMapSwizzle swz);

}  // namespace wna16
