// C ABI of the operators around the routed experts (include/wna16_moe_block.h):
// argument validation and dispatch.
#include <cmath>

#include "../../include/wna16_moe_block.h"
#include "block.h"
#include "checks.h"
#include "gemm.h"

using namespace wna16;

namespace {

int check_q8(int q_type, int group, int64_t K) {
    if (q_type != WNA16_Q8_INT8 && q_type != WNA16_Q8_E4M3)
        return set_error(WNA16_ERR_UNSUPPORTED, "q_type=%d: int8 (0) or e4m3 (1)", q_type);
    if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
        return set_error(WNA16_ERR_UNSUPPORTED, "group_size=%d: 0 (the whole row), 32, 64, 128 or 256", group);
    if (group && K % group)
        return set_error(WNA16_ERR_UNSUPPORTED, "group_size=%d must divide the row length %lld", group, (ll)K);
    return WNA16_OK;
}

size_t scale_bytes(int64_t T, int64_t K, int group) { return static_cast<size_t>(T) * (group ? K / group : 1) * 4; }

}  // namespace

extern "C" {

int wna16_moe_add_rmsnorm_q8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                             int weight_type, int64_t T, int64_t K, int type, float eps, int q_type, int group_size,
                             void* q, float* scales, void* residual_out, void* norm_out, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (weight_type != type && weight_type != WNA16_TYPE_FP32)
        return set_error(WNA16_ERR_UNSUPPORTED, "weight_type=%d must be the rows' type or fp32", weight_type);
    if (int rc = check_rows(T, K, 32768, "K")) return rc;
    if (int rc = check_ld(ldx, K, "ldx")) return rc;
    if (residual)
        if (int rc = check_ld(ldr, K, "ldr")) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps)) return set_error(WNA16_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    if (!q != !scales) return set_error(WNA16_ERR_INVALID_ARG, "q and scales go together");
    if (q)
        if (int rc = check_q8(q_type, group_size, K)) return rc;
    if (T == 0) return WNA16_OK;
    if (!q && !norm_out) return set_error(WNA16_ERR_INVALID_ARG, "norm_out and q are both NULL");
    const size_t es = size_of(type);
    if (int rc = check_pointer(x, es, "x")) return rc;
    if (residual)
        if (int rc = check_pointer(residual, es, "residual")) return rc;
    if (int rc = check_pointer(weight, size_of(weight_type), "weight")) return rc;
    if (residual_out)
        if (int rc = check_pointer(residual_out, es, "residual_out")) return rc;
    if (norm_out)
        if (int rc = check_pointer(norm_out, es, "norm_out")) return rc;
    if (q)
        if (int rc = check_pointer(scales, 4, "scales")) return rc;
    const size_t out_bytes = static_cast<size_t>(T * K) * es;
    const Range outs[4] = {{residual_out, out_bytes, "residual_out"},
                           {norm_out, out_bytes, "norm_out"},
                           {q, static_cast<size_t>(T * K), "q"},
                           {scales, scale_bytes(T, K, q ? group_size : 0), "scales"}};
    const Range ins[3] = {
        {x, extent(T, ldx, K, es), "x", residual_out == x && (ldx == K || T == 1)},
        {residual, residual ? extent(T, ldr, K, es) : 0, "residual", residual_out == residual && (ldr == K || T == 1)},
        {weight, static_cast<size_t>(K) * size_of(weight_type), "weight"}};
    if (int rc = check_overlap(outs, ins)) return rc;
    RowParams p;
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.ldx = ldx;
    p.ldr = ldr;
    p.T = T;
    p.K = static_cast<int>(K);
    p.weight_f32 = weight_type == WNA16_TYPE_FP32;
    p.eps = eps;
    p.q_type = q_type;
    p.group = q ? group_size : 0;
    p.q = q;
    p.scales = scales;
    p.residual_out = residual_out;
    p.norm_out = norm_out;
    p.vec = K % 8 == 0 && wide(x, ldx, es) && (!residual || wide(residual, ldr, es)) && aligned(weight, 16) &&
            aligned(residual_out, 16) && aligned(norm_out, 16) && aligned(q, 8);
    return launched(launch_rows(RowOp::norm, type, p, static_cast<cudaStream_t>(stream)), "norm kernel launch");
}

int wna16_moe_swiglu_q8(const void* gu, int64_t ldg, int64_t T, int64_t N, int type, float swiglu_limit, int q_type,
                        int group_size, void* q, float* scales, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_rows(T, N, 32768, "N")) return rc;
    if (int rc = check_ld(ldg, 2 * N, "ldg")) return rc;
    if (!(swiglu_limit > 0.0f)) return set_error(WNA16_ERR_INVALID_ARG, "swiglu_limit must be > 0 (or +inf)");
    if (int rc = check_q8(q_type, group_size, N)) return rc;
    if (T == 0) return WNA16_OK;
    const size_t es = size_of(type);
    if (int rc = check_pointer(gu, es, "gu")) return rc;
    if (int rc = check_pointer(q, 1, "q")) return rc;
    if (int rc = check_pointer(scales, 4, "scales")) return rc;
    const Range outs[2] = {{q, static_cast<size_t>(T * N), "q"}, {scales, scale_bytes(T, N, group_size), "scales"}};
    const Range ins[1] = {{gu, extent(T, ldg, 2 * N, es), "gu"}};
    if (int rc = check_overlap(outs, ins)) return rc;
    RowParams p;
    p.x = gu;
    p.ldx = ldg;
    p.T = T;
    p.K = static_cast<int>(N);
    p.limit = swiglu_limit;
    p.q_type = q_type;
    p.group = group_size;
    p.q = q;
    p.scales = scales;
    p.vec = N % 8 == 0 && wide(gu, ldg, es) && aligned(q, 8);
    return launched(launch_rows(RowOp::swiglu, type, p, static_cast<cudaStream_t>(stream)), "swiglu kernel launch");
}

int wna16_moe_quantize_q8(const void* x, int64_t ldx, int64_t T, int64_t K, int type, int q_type, int group_size,
                          void* q, float* scales, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_rows(T, K, 32768, "K")) return rc;
    if (int rc = check_ld(ldx, K, "ldx")) return rc;
    if (int rc = check_q8(q_type, group_size, K)) return rc;
    if (T == 0) return WNA16_OK;
    const size_t es = size_of(type);
    if (int rc = check_pointer(x, es, "x")) return rc;
    if (int rc = check_pointer(q, 1, "q")) return rc;
    if (int rc = check_pointer(scales, 4, "scales")) return rc;
    const Range outs[2] = {{q, static_cast<size_t>(T * K), "q"}, {scales, scale_bytes(T, K, group_size), "scales"}};
    const Range ins[1] = {{x, extent(T, ldx, K, es), "x"}};
    if (int rc = check_overlap(outs, ins)) return rc;
    RowParams p;
    p.x = x;
    p.ldx = ldx;
    p.T = T;
    p.K = static_cast<int>(K);
    p.q_type = q_type;
    p.group = group_size;
    p.q = q;
    p.scales = scales;
    p.vec = K % 8 == 0 && wide(x, ldx, es) && aligned(q, 8);
    return launched(launch_rows(RowOp::plain, type, p, static_cast<cudaStream_t>(stream)), "quantize kernel launch");
}

int wna16_moe_dequantize_q8(const void* q, const float* scales, int64_t T, int64_t K, int q_type, int group_size,
                            int type, void* out, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_rows(T, K, int64_t(1) << 26, "K")) return rc;
    if (int rc = check_q8(q_type, group_size, K)) return rc;
    if (T == 0) return WNA16_OK;
    const size_t es = size_of(type);
    if (int rc = check_pointer(q, 1, "q")) return rc;
    if (int rc = check_pointer(scales, 4, "scales")) return rc;
    if (int rc = check_pointer(out, es, "out")) return rc;
    const Range outs[1] = {{out, static_cast<size_t>(T * K) * es, "out"}};
    const Range ins[2] = {{q, static_cast<size_t>(T * K), "q"}, {scales, scale_bytes(T, K, group_size), "scales"}};
    if (int rc = check_overlap(outs, ins)) return rc;
    const bool vec = K % 16 == 0 && aligned(q, 16) && aligned(out, 16);
    return launched(launch_dequantize_q8(q, scales, T, static_cast<int>(K), q_type, group_size, type, out, vec,
                                         static_cast<cudaStream_t>(stream)),
                    "dequantize kernel launch");
}

int wna16_moe_route_scored(const void* logits, int64_t ld, const float* bias, int64_t T, int64_t E, int type, int score,
                           int groups, int topk_groups, int group_score, int topk, int renormalize, float scale,
                           int32_t* topk_ids, float* topk_weights, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_rows(T, E, 1024, "E")) return rc;
    if (int rc = check_ld(ld, E, "ld")) return rc;
    if (score != WNA16_SCORE_SIGMOID && score != WNA16_SCORE_SOFTMAX)
        return set_error(WNA16_ERR_UNSUPPORTED, "score=%d: sigmoid (0) or softmax (1)", score);
    if (group_score != WNA16_GROUP_TOP2 && group_score != WNA16_GROUP_MAX)
        return set_error(WNA16_ERR_UNSUPPORTED, "group_score=%d: two best (0) or best (1)", group_score);
    if (groups < 1 || groups > 32 || E % groups)
        return set_error(WNA16_ERR_INVALID_ARG, "groups=%d must be in [1, 32] and divide E=%lld", groups, (ll)E);
    if (topk_groups < 1 || topk_groups > groups)
        return set_error(WNA16_ERR_INVALID_ARG, "topk_groups=%d must be in [1, %d]", topk_groups, groups);
    if (topk < 1 || topk > 32 || topk > topk_groups * (E / groups))
        return set_error(WNA16_ERR_INVALID_ARG, "topk=%d must be in [1, min(32, %lld)]", topk,
                         (ll)(topk_groups * (E / groups)));
    if (renormalize != 0 && renormalize != 1)
        return set_error(WNA16_ERR_INVALID_ARG, "renormalize=%d must be 0 or 1", renormalize);
    if (!std::isfinite(scale)) return set_error(WNA16_ERR_INVALID_ARG, "scale must be finite");
    if (T == 0) return WNA16_OK;
    const size_t es = size_of(type);
    if (int rc = check_pointer(logits, es, "logits")) return rc;
    if (bias)
        if (int rc = check_pointer(bias, 4, "bias")) return rc;
    if (int rc = check_pointer(topk_ids, 4, "topk_ids")) return rc;
    if (int rc = check_pointer(topk_weights, 4, "topk_weights")) return rc;
    const Range outs[2] = {{topk_ids, static_cast<size_t>(T) * topk * 4, "topk_ids"},
                           {topk_weights, static_cast<size_t>(T) * topk * 4, "topk_weights"}};
    const Range ins[2] = {{logits, extent(T, ld, E, es), "logits"}, {bias, static_cast<size_t>(E) * 4, "bias"}};
    if (int rc = check_overlap(outs, ins)) return rc;
    ScoredRouteParams p;
    p.logits = logits;
    p.ld = ld;
    p.bias = bias;
    p.T = static_cast<int>(T);
    p.E = static_cast<int>(E);
    p.softmax = score == WNA16_SCORE_SOFTMAX;
    p.groups = groups;
    p.topk_groups = topk_groups;
    p.group_max = group_score == WNA16_GROUP_MAX;
    p.topk = topk;
    p.renormalize = renormalize;
    p.scale = scale;
    p.ids = topk_ids;
    p.weights = topk_weights;
    p.vec = E / groups % 4 == 0 && aligned(logits, 4 * es) && ld % 4 == 0;
    p.bias_vec = E / groups % 4 == 0 && aligned(bias, 16);
    return launched(launch_route_scored(type, p, static_cast<cudaStream_t>(stream)), "router kernel launch");
}

static int check_linear(int64_t T, int64_t K, int64_t N) {
    if (int rc = check_rows(T, K, 65536, "K")) return rc;
    if (N <= 0) return set_error(WNA16_ERR_INVALID_ARG, "N=%lld must be > 0", (ll)N);
    if (K % 16) return set_error(WNA16_ERR_UNSUPPORTED, "K=%lld must be a multiple of 16", (ll)K);
    if (N >= (int64_t(1) << 24) || T >= (int64_t(1) << 24))
        return set_error(WNA16_ERR_UNSUPPORTED, "T=%lld and N=%lld must be < 2^24", (ll)T, (ll)N);
    return WNA16_OK;
}

size_t wna16_moe_linear_q8_workspace_size(int64_t T, int64_t K, int64_t N) {
    return check_linear(T, K, N) == WNA16_OK ? linear_q8_workspace(T, K, N) : 0;
}

int wna16_moe_linear_q8(const int8_t* xq, const float* x_scales, const int8_t* wq, const float* w_scales,
                        const float* bias, const void* addend, int64_t T, int64_t K, int64_t N, int type, void* out,
                        void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    if (int rc = check_type(type, "type")) return rc;
    if (int rc = check_linear(T, K, N)) return rc;
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
    if (int rc = check_pointer(out, es, "out")) return rc;
    const size_t need = linear_q8_workspace(T, K, N);
    if (need && workspace) {
        if (int rc = check_pointer(workspace, 256, "workspace")) return rc;
        if (workspace_bytes < need)
            return set_error(WNA16_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    }
    // where none is needed, the status word is written if there is room for it
    if (workspace_bytes < sizeof(int) || !aligned(workspace, sizeof(int))) workspace = nullptr;
    const Range outs[2] = {{out, static_cast<size_t>(T * N) * es, "out"}, {workspace, need ? need : sizeof(int), "workspace"}};
    const Range ins[6] = {{xq, static_cast<size_t>(T * K), "xq"},
                          {wq, static_cast<size_t>(N * K), "wq"},
                          {x_scales, static_cast<size_t>(T) * 4, "x_scales"},
                          {w_scales, static_cast<size_t>(N) * 4, "w_scales"},
                          {bias, static_cast<size_t>(N) * 4, "bias"},
                          {addend, static_cast<size_t>(T * N) * es, "addend", addend == out}};
    if (int rc = check_overlap(outs, ins)) return rc;
    LinearParams p;
    p.xq = xq;
    p.xs = x_scales;
    p.wq = wq;
    p.ws = w_scales;
    p.bias = bias;
    p.addend = addend;
    p.out = out;
    p.T = static_cast<int>(T);
    p.K = static_cast<int>(K);
    p.N = static_cast<int>(N);
    p.type = type;
    return run_linear_q8(p, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
