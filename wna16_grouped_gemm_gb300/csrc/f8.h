// Internal interface of the routed experts in 8-bit floats (host side).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "block.h"

namespace wna16 {

constexpr int kScaleBlock = 128;   // values per scale (and output channels per scale of a weight)

// Tokens to rows in expert order and back (sort_tokens.cu).
struct SortParams {
    const void* x = nullptr;          // NULL: lists only
    const float* x_scales = nullptr;  // [T, groups] or NULL
    int64_t x_pitch = 0, row_bytes = 0;
    int64_t groups = 0;
    int64_t T = 0;
    int topk = 1, E = 1, expert_begin = 0;
    const int32_t* ids = nullptr;
    void* rows = nullptr;
    float* row_scales = nullptr;
    int32_t* offsets = nullptr;
    int32_t* inv = nullptr;
};
cudaError_t launch_sort_tokens(const SortParams& p, cudaStream_t stream);

struct UnsortParams {
    const void* y = nullptr;          // [R, K]
    const void* dout = nullptr;       // gradient: [T, K]
    const int32_t* inv = nullptr;
    const float* weights = nullptr;   // NULL: 1
    const void* addend = nullptr;
    int64_t T = 0, K = 0, R = 0;
    int topk = 1;
    void* out = nullptr;              // [T, K]; gradient: dy [R, K] or NULL
    float* dweights = nullptr;
    int access = 0;                   // bytes: 16, 4, or a value's
};
cudaError_t launch_unsort_tokens(int type, const UnsortParams& p, int sms, cudaStream_t stream);
cudaError_t launch_unsort_tokens_grad(int type, const UnsortParams& p, int sms, cudaStream_t stream);

// Products of e4m3 rows with block-scaled e4m3 weights (linear_f8.cu).
struct LinearF8Params {
    const uint8_t* xq = nullptr;
    const float* xs = nullptr;
    const uint8_t* wq = nullptr;
    const float* ws = nullptr;
    const float* bias = nullptr;
    const void* addend = nullptr;
    const int32_t* offsets = nullptr;   // NULL: one weight for all rows
    void* out = nullptr;
    int T = 0, K = 0, N = 0, E = 1;     // T rows
    int type = kBf16;
    int* status = nullptr;
};
// returns a wna16_status and sets the error message
int run_linear_f8(const LinearF8Params& p, cudaStream_t stream);

// Weights to e4m3 in blocks (blocks_f8.cu).
struct BlocksParams {
    const void* w = nullptr;
    int64_t E = 1, N = 0, K = 0;
    int64_t se = 0, sn = 0, sk = 0;     // strides in elements; sk or sn is 1
    uint8_t* q = nullptr;
    float* scales = nullptr;
};
cudaError_t launch_quantize_blocks_f8(int type, const BlocksParams& p, cudaStream_t stream);

}  // namespace wna16
