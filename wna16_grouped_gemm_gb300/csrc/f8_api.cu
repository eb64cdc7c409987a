// C ABI of the routed experts in 8-bit floats (include/wna16_moe_f8.h):
// argument validation and dispatch.
#include <initializer_list>

#include "../../include/wna16_moe_f8.h"
#include "block.h"
#include "checks.h"
#include "f8.h"
#include "gemm.h"

using namespace wna16;

namespace {

constexpr int64_t kMaxK = int64_t(1) << 26;

int check_slots(int64_t T, int64_t K, int topk) {
    if (int rc = check_rows(T, K, kMaxK, "K")) return rc;
    if (topk < 1 || topk > 1024) return set_error(WNA16_ERR_UNSUPPORTED, "topk=%d must be in [1, 1024]", topk);
    if (T * topk >= (int64_t(1) << 31))
        return set_error(WNA16_ERR_UNSUPPORTED, "T * topk = %lld must be < 2^31", (ll)(T * topk));
    return WNA16_OK;
}

int check_experts(int64_t E) {
    if (E < 1) return set_error(WNA16_ERR_INVALID_ARG, "E=%lld must be > 0", (ll)E);
    if (E > 1024) return set_error(WNA16_ERR_UNSUPPORTED, "E=%lld: at most 1024", (ll)E);
    return WNA16_OK;
}

// The widest accesses that contiguous rows of K values allow: 16 or 4 bytes, or one value.
int access_of(int64_t K, size_t es, std::initializer_list<const void*> rows) {
    uintptr_t all = static_cast<uintptr_t>(K) * es;
    for (const void* p : rows) all |= reinterpret_cast<uintptr_t>(p);
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : static_cast<int>(es);
}

int64_t row_blocks(int64_t N) { return (N + kScaleBlock - 1) / kScaleBlock; }

}  // namespace

extern "C" {

int wna16_moe_sort_tokens(const void* x, int64_t ldx, const float* x_scales, int64_t groups, int64_t T, int64_t K,
                          int type, const int32_t* topk_ids, int topk, int64_t E, int64_t expert_begin, void* rows,
                          float* row_scales, int32_t* offsets, int32_t* inv, void* stream) {
    clear_error();
    if (type != WNA16_TYPE_Q8)
        if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_slots(T, K, topk)) return rc;
    if (int rc = check_experts(E)) return rc;
    if (expert_begin < 0 || expert_begin >= (int64_t(1) << 30))
        return set_error(WNA16_ERR_INVALID_ARG, "expert_begin=%lld must be in [0, 2^30)", (ll)expert_begin);
    if (!x != !rows) return set_error(WNA16_ERR_INVALID_ARG, "x and rows go together");
    if (!x_scales != !row_scales) return set_error(WNA16_ERR_INVALID_ARG, "x_scales and row_scales go together");
    if (x_scales && !x) return set_error(WNA16_ERR_INVALID_ARG, "x_scales without x");
    if (x_scales && (groups < 1 || groups > K))
        return set_error(WNA16_ERR_INVALID_ARG, "groups=%lld must be in [1, %lld]", (ll)groups, (ll)K);
    if (x)
        if (int rc = check_ld(ldx, K, "ldx")) return rc;
    const size_t es = type == WNA16_TYPE_Q8 ? 1 : size_of(type);
    // an empty batch has offsets: all of them 0
    if (int rc = check_pointer(offsets, 4, "offsets")) return rc;
    if (T > 0) {
        if (int rc = check_pointer(topk_ids, 4, "topk_ids")) return rc;
        if (int rc = check_pointer(inv, 4, "inv")) return rc;
        if (x) {
            if (int rc = check_pointer(x, es, "x")) return rc;
            if (int rc = check_pointer(rows, es, "rows")) return rc;
        }
        if (x_scales) {
            if (int rc = check_pointer(x_scales, 4, "x_scales")) return rc;
            if (int rc = check_pointer(row_scales, 4, "row_scales")) return rc;
        }
        const size_t slots = static_cast<size_t>(T) * topk;
        const Range outs[4] = {{rows, slots * K * es, "rows"},
                               {row_scales, slots * groups * 4, "row_scales"},
                               {offsets, static_cast<size_t>(E + 1) * 4, "offsets"},
                               {inv, slots * 4, "inv"}};
        const Range ins[3] = {{x, x ? extent(T, ldx, K, es) : 0, "x"},
                              {x_scales, static_cast<size_t>(T) * groups * 4, "x_scales"},
                              {topk_ids, slots * 4, "topk_ids"}};
        if (int rc = check_overlap(outs, ins)) return rc;
    }
    SortParams p;
    p.x = x;
    p.x_scales = x_scales;
    p.x_pitch = ldx * static_cast<int64_t>(es);
    p.row_bytes = K * static_cast<int64_t>(es);
    p.groups = groups;
    p.T = T;
    p.topk = topk;
    p.E = static_cast<int>(E);
    p.expert_begin = static_cast<int>(expert_begin);
    p.ids = topk_ids;
    p.rows = rows;
    p.row_scales = row_scales;
    p.offsets = offsets;
    p.inv = inv;
    return launched(launch_sort_tokens(p, static_cast<cudaStream_t>(stream)), "sort_tokens launch");
}

int wna16_moe_unsort_tokens(const void* y, int64_t R, const int32_t* inv, const float* weights, const void* addend,
                            int64_t T, int64_t K, int topk, int type, void* out, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_slots(T, K, topk)) return rc;
    if (R < 0 || R >= (int64_t(1) << 31)) return set_error(WNA16_ERR_INVALID_ARG, "R=%lld must be in [0, 2^31)", (ll)R);
    if (T == 0) return WNA16_OK;
    const size_t es = size_of(type), slots = static_cast<size_t>(T) * topk;
    if (R > 0)
        if (int rc = check_pointer(y, es, "y")) return rc;
    if (int rc = check_pointer(inv, 4, "inv")) return rc;
    if (weights)
        if (int rc = check_pointer(weights, 4, "weights")) return rc;
    if (addend)
        if (int rc = check_pointer(addend, es, "addend")) return rc;
    if (int rc = check_pointer(out, es, "out")) return rc;
    const Range outs[1] = {{out, static_cast<size_t>(T * K) * es, "out"}};
    const Range ins[4] = {{y, static_cast<size_t>(R) * K * es, "y"},
                          {inv, slots * 4, "inv"},
                          {weights, slots * 4, "weights"},
                          {addend, static_cast<size_t>(T * K) * es, "addend", addend == out}};
    if (int rc = check_overlap(outs, ins)) return rc;
    UnsortParams p;
    p.y = y;
    p.inv = inv;
    p.weights = weights;
    p.addend = addend;
    p.T = T;
    p.K = K;
    p.R = R;
    p.topk = topk;
    p.out = out;
    p.access = access_of(K, es, {y, addend, out});
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    return launched(launch_unsort_tokens(type, p, sms, static_cast<cudaStream_t>(stream)), "unsort_tokens launch");
}

int wna16_moe_unsort_tokens_grad(const void* dout, const int32_t* inv, const void* y, const float* weights, int64_t T,
                                 int64_t K, int topk, int64_t R, int type, void* dy, float* dweights, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_slots(T, K, topk)) return rc;
    if (R < 0 || R >= (int64_t(1) << 31)) return set_error(WNA16_ERR_INVALID_ARG, "R=%lld must be in [0, 2^31)", (ll)R);
    if (T == 0) return WNA16_OK;
    if (R == 0 && !dweights) return WNA16_OK;   // dy has no rows
    if (!dy && !dweights) return set_error(WNA16_ERR_INVALID_ARG, "dy and dweights are both NULL");
    const size_t es = size_of(type), slots = static_cast<size_t>(T) * topk;
    if (R > 0 && !y != !dweights) return set_error(WNA16_ERR_INVALID_ARG, "y and dweights go together");
    if (int rc = check_pointer(dout, es, "dout")) return rc;
    if (int rc = check_pointer(inv, 4, "inv")) return rc;
    if (y)
        if (int rc = check_pointer(y, es, "y")) return rc;
    if (weights)
        if (int rc = check_pointer(weights, 4, "weights")) return rc;
    if (dy)
        if (int rc = check_pointer(dy, es, "dy")) return rc;
    if (dweights)
        if (int rc = check_pointer(dweights, 4, "dweights")) return rc;
    const size_t rows = static_cast<size_t>(R) * K * es;
    const Range outs[2] = {{dy, rows, "dy"}, {dweights, slots * 4, "dweights"}};
    const Range ins[4] = {{dout, static_cast<size_t>(T * K) * es, "dout"},
                          {inv, slots * 4, "inv"},
                          {y, rows, "y"},
                          {weights, slots * 4, "weights"}};
    if (int rc = check_overlap(outs, ins)) return rc;
    UnsortParams p;
    p.y = y;
    p.dout = dout;
    p.inv = inv;
    p.weights = weights;
    p.T = T;
    p.K = K;
    p.R = R;
    p.topk = topk;
    p.out = dy;
    p.dweights = dweights;
    p.access = access_of(K, es, {y, dout, dy});
    int sms = 0, max_smem = 0;
    if (int rc = device_limits(sms, max_smem)) return rc;
    return launched(launch_unsort_tokens_grad(type, p, sms, static_cast<cudaStream_t>(stream)), "unsort_tokens_grad launch");
}

static int linear_f8(const void* xq, const float* x_scales, const void* wq, const float* w_scales, const float* bias,
                     const void* addend, const int32_t* offsets, int64_t E, int64_t T, int64_t K, int64_t N, int type,
                     void* out, void* workspace, size_t workspace_bytes, bool grouped, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_rows(T, K, 65536, "K")) return rc;
    if (N <= 0) return set_error(WNA16_ERR_INVALID_ARG, "N=%lld must be > 0", (ll)N);
    if (K % kScaleBlock) return set_error(WNA16_ERR_UNSUPPORTED, "K=%lld must be a multiple of %d", (ll)K, kScaleBlock);
    if (N >= (int64_t(1) << 24) || T >= (int64_t(1) << 30))
        return set_error(WNA16_ERR_UNSUPPORTED, "N=%lld must be < 2^24 and the rows %lld < 2^30", (ll)N, (ll)T);
    if (int rc = check_experts(E)) return rc;
    if (E * N >= (int64_t(1) << 31)) return set_error(WNA16_ERR_UNSUPPORTED, "E * N = %lld must be < 2^31", (ll)(E * N));
    if (T == 0) return WNA16_OK;
    const size_t es = size_of(type);
    if (int rc = check_pointer(xq, 16, "xq")) return rc;
    if (int rc = check_pointer(wq, 16, "wq")) return rc;
    if (int rc = check_pointer(x_scales, 4, "x_scales")) return rc;
    if (int rc = check_pointer(w_scales, 4, "w_scales")) return rc;
    if (bias)
        if (int rc = check_pointer(bias, 4, "bias")) return rc;
    if (addend)
        if (int rc = check_pointer(addend, es, "addend")) return rc;
    if (grouped)
        if (int rc = check_pointer(offsets, 4, "offsets")) return rc;
    if (int rc = check_pointer(out, es, "out")) return rc;
    if (workspace) {
        if (int rc = check_pointer(workspace, 4, "workspace")) return rc;
        if (workspace_bytes < sizeof(int))
            return set_error(WNA16_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, sizeof(int));
    }
    const size_t out_bytes = static_cast<size_t>(T) * N * es, groups = static_cast<size_t>(K / kScaleBlock);
    const Range outs[2] = {{out, out_bytes, "out"}, {workspace, sizeof(int), "workspace"}};
    const Range ins[7] = {{xq, static_cast<size_t>(T) * K, "xq"},
                          {wq, static_cast<size_t>(E) * N * K, "wq"},
                          {x_scales, static_cast<size_t>(T) * groups * 4, "x_scales"},
                          {w_scales, static_cast<size_t>(E * row_blocks(N)) * groups * 4, "w_scales"},
                          {bias, static_cast<size_t>(N) * 4, "bias"},
                          {offsets, static_cast<size_t>(E + 1) * 4, "offsets"},
                          {addend, out_bytes, "addend", addend == out}};
    if (int rc = check_overlap(outs, ins)) return rc;
    LinearF8Params p;
    p.xq = static_cast<const uint8_t*>(xq);
    p.xs = x_scales;
    p.wq = static_cast<const uint8_t*>(wq);
    p.ws = w_scales;
    p.bias = bias;
    p.addend = addend;
    p.offsets = grouped ? offsets : nullptr;
    p.out = out;
    p.T = static_cast<int>(T);
    p.K = static_cast<int>(K);
    p.N = static_cast<int>(N);
    p.E = static_cast<int>(E);
    p.type = type;
    p.status = static_cast<int*>(workspace);
    return run_linear_f8(p, static_cast<cudaStream_t>(stream));
}

int wna16_moe_linear_f8(const void* xq, const float* x_scales, const void* wq, const float* w_scales, const float* bias,
                        const void* addend, int64_t T, int64_t K, int64_t N, int type, void* out, void* workspace,
                        size_t workspace_bytes, void* stream) {
    return linear_f8(xq, x_scales, wq, w_scales, bias, addend, nullptr, 1, T, K, N, type, out, workspace,
                     workspace_bytes, false, stream);
}

int wna16_moe_grouped_linear_f8(const void* xq, const float* x_scales, const void* wq, const float* w_scales,
                                const int32_t* offsets, int64_t E, int64_t R, int64_t K, int64_t N, int type, void* out,
                                void* workspace, size_t workspace_bytes, void* stream) {
    return linear_f8(xq, x_scales, wq, w_scales, nullptr, nullptr, offsets, E, R, K, N, type, out, workspace,
                     workspace_bytes, true, stream);
}

int wna16_moe_quantize_blocks_f8(const void* w, int64_t E, int64_t N, int64_t K, int64_t stride_e, int64_t stride_n,
                                 int64_t stride_k, int type, void* q, float* scales, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (E < 0 || N <= 0 || K <= 0)
        return set_error(WNA16_ERR_INVALID_ARG, "E=%lld must be >= 0, N=%lld and K=%lld > 0", (ll)E, (ll)N, (ll)K);
    if (E >= (int64_t(1) << 24) || N >= (int64_t(1) << 24) || K > kMaxK)
        return set_error(WNA16_ERR_UNSUPPORTED, "E=%lld and N=%lld must be < 2^24, K=%lld <= 2^26", (ll)E, (ll)N, (ll)K);
    if (K % kScaleBlock) return set_error(WNA16_ERR_UNSUPPORTED, "K=%lld must be a multiple of %d", (ll)K, kScaleBlock);
    if (E * row_blocks(N) >= (int64_t(1) << 31) / (K / kScaleBlock))
        return set_error(WNA16_ERR_UNSUPPORTED, "%lld x %lld x %lld: too many blocks", (ll)E, (ll)N, (ll)K);
    constexpr int64_t kFar = int64_t(1) << 40;
    const bool rows = stride_k == 1 && stride_n >= K, columns = stride_n == 1 && stride_k >= N;
    if ((!rows && !columns && !(stride_k == 1 && N == 1)) || stride_n >= kFar || stride_k >= kFar)
        return set_error(WNA16_ERR_INVALID_ARG, "strides (%lld, %lld): rows or columns of the weight must be contiguous and apart",
                         (ll)stride_n, (ll)stride_k);
    const int64_t span = (N - 1) * stride_n + (K - 1) * stride_k + 1;   // elements of one weight
    if (E > 1 && (stride_e < span || stride_e >= kFar))
        return set_error(WNA16_ERR_INVALID_ARG, "stride_e=%lld: weights of %lld elements overlap or are too far apart",
                         (ll)stride_e, (ll)span);
    if (E == 0) return WNA16_OK;
    const size_t es = size_of(type);
    if (int rc = check_pointer(w, es, "w")) return rc;
    if (int rc = check_pointer(q, 1, "q")) return rc;
    if (int rc = check_pointer(scales, 4, "scales")) return rc;
    const Range outs[2] = {{q, static_cast<size_t>(E) * N * K, "q"},
                           {scales, static_cast<size_t>(E * row_blocks(N) * (K / kScaleBlock)) * 4, "scales"}};
    const Range ins[1] = {{w, (static_cast<size_t>(E - 1) * (E > 1 ? stride_e : 0) + span) * es, "w"}};
    if (int rc = check_overlap(outs, ins)) return rc;
    BlocksParams p;
    p.w = w;
    p.E = E;
    p.N = N;
    p.K = K;
    p.se = E > 1 ? stride_e : 0;
    p.sn = stride_n;
    p.sk = stride_k;
    p.q = static_cast<uint8_t*>(q);
    p.scales = scales;
    return launched(launch_quantize_blocks_f8(type, p, static_cast<cudaStream_t>(stream)), "quantize_blocks launch");
}

}  // extern "C"
