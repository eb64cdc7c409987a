// Argument checks that the entry points beside the forward share (host side).
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/wna16_moe_block.h"
#include "gemm.h"

namespace wna16 {

using ll = long long;

inline int clear_error() { return set_error(WNA16_OK, "%s", ""); }

inline size_t size_of(int type) { return type == WNA16_TYPE_FP32 ? 4 : 2; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline int check_type(int type, const char* name) {
    if (type < WNA16_TYPE_BF16 || type > WNA16_TYPE_FP32)
        return set_error(WNA16_ERR_UNSUPPORTED, "%s=%d: bf16 (0), fp16 (1) or fp32 (2)", name, type);
    return WNA16_OK;
}

inline int check_pointer(const void* p, size_t align, const char* name) {
    if (!p) return set_error(WNA16_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, align)) return set_error(WNA16_ERR_INVALID_ARG, "%s must be %zu-byte aligned", name, align);
    return WNA16_OK;
}

// T rows of `len` elements, `ld` apart
inline int check_rows(int64_t T, int64_t len, int64_t max_len, const char* name) {
    if (T < 0 || len <= 0)
        return set_error(WNA16_ERR_INVALID_ARG, "T=%lld must be >= 0 and %s=%lld > 0", (ll)T, name, (ll)len);
    if (len > max_len) return set_error(WNA16_ERR_UNSUPPORTED, "%s=%lld: at most %lld", name, (ll)len, (ll)max_len);
    if (T >= (int64_t(1) << 31)) return set_error(WNA16_ERR_UNSUPPORTED, "T=%lld must be < 2^31", (ll)T);
    return WNA16_OK;
}

inline int check_ld(int64_t ld, int64_t len, const char* name) {
    if (ld < len || ld >= (int64_t(1) << 40))
        return set_error(WNA16_ERR_INVALID_ARG, "%s=%lld: rows of %lld elements overlap or are too far apart", name, (ll)ld,
                         (ll)len);
    return WNA16_OK;
}

struct Range {
    const void* p;
    size_t bytes;
    const char* name;
    bool in_place = false;   // an input that outs[0] updates in place: the same elements at the same places
};
inline bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}
// Outputs against inputs and against one another.
template <size_t NO, size_t NI>
int check_overlap(const Range (&outs)[NO], const Range (&ins)[NI]) {
    for (size_t i = 0; i < NO; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r) && !(i == 0 && r.in_place))
                return set_error(WNA16_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, r.name);
        for (size_t j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j]))
                return set_error(WNA16_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return WNA16_OK;
}

inline size_t extent(int64_t T, int64_t ld, int64_t len, size_t size) {
    return (static_cast<size_t>(T - 1) * ld + len) * size;
}

// rows readable 16 bytes at a time
inline bool wide(const void* p, int64_t ld, size_t size) { return aligned(p, 16) && ld * size % 16 == 0; }

inline int launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? WNA16_OK : set_error(WNA16_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace wna16
