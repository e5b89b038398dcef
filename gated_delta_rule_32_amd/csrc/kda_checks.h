// Argument checks shared by the entry points of the layer operators (kda_layers.cpp,
// kda_delta_api.cpp).
#pragma once

#include <cfloat>
#include <cmath>
#include <exception>
#include <initializer_list>
#include <utility>

#include "kda_host.h"

namespace kda_host {

constexpr int D = 128;
constexpr int64_t kState = (int64_t)D * D;
// Largest token stride (elements): the kernels add up to 31 of them in 32 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 25;


inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Runs an entry point's body; an exception (host memory) becomes a status.
template <class F>
inline kda_status guarded(F f) {
    try {
        return f();
    } catch (const std::exception& e) {
        return fail(KDA_ERR_HIP, "host error: %s", e.what());
    }
}

// 0 means dense rows.
inline kda_status check_stride(int64_t& stride, int heads, const char* name) {
    if (stride == 0) stride = (int64_t)heads * D;
    if (stride < (int64_t)heads * D || stride > kMaxStride || stride % 8 != 0)
        return fail(KDA_ERR_SHAPE, "%s token stride must be a multiple of 8 in [%d, %lld] (got %lld)", name, heads * D,
                    (long long)kMaxStride, (long long)stride);
    return KDA_OK;
}

inline kda_status check_align(const void* p, const char* name) {
    if (((uintptr_t)p & 15) != 0) return fail(KDA_ERR_SHAPE, "%s must be 16-byte aligned", name);
    return KDA_OK;
}
inline kda_status check_align(std::initializer_list<std::pair<const void*, const char*>> ps) {
    for (const auto& p : ps) {
        kda_status s = check_align(p.first, p.second);
        if (s != KDA_OK) return s;
    }
    return KDA_OK;
}

// (Below the normal numbers the reciprocal square root takes eps for 0, and a row of
// zeros would come out as NaN.)
inline kda_status check_eps(float eps) {
    if (!(eps >= FLT_MIN) || !std::isfinite(eps))
        return fail(KDA_ERR_SHAPE, "eps must be finite and a positive normal number (got %g)", (double)eps);
    return KDA_OK;
}

// Bytes from a strided operand's first element to behind its last.
inline size_t strided_bytes(int64_t tokens, int64_t stride, int heads) {
    return (size_t)((tokens - 1) * stride + (int64_t)heads * D) * 2;
}

// A launch holds less than 2^32 threads.
inline kda_status check_grid(int64_t blocks, int threads = 256) {
    if (blocks >= ((int64_t)1 << 32) / threads) return fail(KDA_ERR_SHAPE, "too many (sequence, head) tasks or tokens");
    return KDA_OK;
}
inline kda_status check_ws(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return KDA_OK;
    if (ws == nullptr) return fail(KDA_ERR_NULL_ARG, "workspace is NULL (needs %zu bytes)", need);
    if (bytes < need) return fail(KDA_ERR_WORKSPACE_SIZE, "workspace has %zu bytes, needs %zu", bytes, need);
    return check_align(ws, "workspace");
}

}  // namespace kda_host
