// ld_dev.cuh -- global loads that stay behind a dependency wait.  A kernel that
// starts while the one before it still runs may load that kernel's results
// only after griddepcontrol.wait.  __ldg, __ldca and __ldcg promise no order
// against it: the compiler may take them to depend on no store and move them
// up.  The same holds for ordinary loads through const __restrict__ kernel
// arguments, which it may turn into such loads.  These are volatile with a
// memory clobber, and keep their place (as ordinary loads through plain
// pointers do).
// _cg: past L1.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace ld {

__device__ __forceinline__ uint32_t u32(const void* p) {
    uint32_t v;
    asm volatile("ld.global.ca.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t u32_cg(const void* p) {
    uint32_t v;
    asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ int32_t i32(const int32_t* p) { return (int32_t)u32(p); }
__device__ __forceinline__ int32_t i32_cg(const int32_t* p) { return (int32_t)u32_cg(p); }
__device__ __forceinline__ float f32(const float* p) { return __uint_as_float(u32(p)); }
__device__ __forceinline__ float f32_cg(const float* p) { return __uint_as_float(u32_cg(p)); }
__device__ __forceinline__ uint32_t u8(const uint8_t* p) {
    uint32_t v;
    asm volatile("ld.global.ca.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float2 f32x2(const float2* p) {
    float2 v;
    asm volatile("ld.global.ca.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float2 f32x2_cg(const float2* p) {
    float2 v;
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float4 f32x4(const float4* p) {
    float4 v;
    asm volatile("ld.global.ca.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint4 u32x4(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.ca.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint4 u32x4_cg(const void* p) {
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

}  // namespace ld
}  // namespace moe
