// api_common.cuh -- what the C ABI's translation units over newer operators
// share: error returns, argument checks and the workspace's bump allocator.
#pragma once

#include "moe_internal.cuh"

namespace moe {
namespace {

template <typename... Args>
moe_status fail(moe_status st, const char* fmt, Args... args) {
    set_last_error(fmt, args...);
    return st;
}
moe_status ok() {
    set_last_error("%s", "");
    return MOE_OK;
}
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

#define CHECK_PTR(p)                                                              \
    do {                                                                          \
        if (!(p)) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);             \
        if (!aligned((p), 16)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
    } while (0)

#define CUDA_TRY(expr, where)                                                     \
    do {                                                                          \
        const cudaError_t e_ = (expr);                                            \
        if (e_ != cudaSuccess)                                                    \
            return fail(MOE_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e_));   \
    } while (0)

#define STATUS_TRY(expr)                 \
    do {                                 \
        const moe_status st_ = (expr);   \
        if (st_ != MOE_OK) return st_;   \
    } while (0)

moe_status check_ws(const void* ws, size_t have, size_t need) {
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(MOE_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (have < need)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    return MOE_OK;
}

// Bump allocator over the caller's workspace (256-byte aligned regions).
struct Carver {
    uint8_t* base;
    size_t off = 0;
    explicit Carver(void* b) : base(static_cast<uint8_t*>(b)) {}
    template <typename T>
    T* take(size_t count) {
        off = align_up(off, 256);
        T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
        off += count * sizeof(T);
        return p;
    }
};

}  // namespace
}  // namespace moe
