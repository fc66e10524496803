// quantize_dev.cuh -- the row quantiser's arithmetic for one lane, shared by
// the quantiser kernel and the small-batch prologue (the format is in fp8.cuh).
#pragma once

#include "fp8.cuh"

namespace moe {
namespace fp8 {

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = __bfloat1622float2(p[i]);
        f[2 * i] = a.x;
        f[2 * i + 1] = a.y;
    }
}

// 32 bytes in one load, for data read once (p 32-byte aligned).
struct Vec32 {
    uint4 a, b;
};
__device__ __forceinline__ Vec32 load32(const void* p) {
    Vec32 v;
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w), "=r"(v.b.x), "=r"(v.b.y),
                   "=r"(v.b.z), "=r"(v.b.w)
                 : "l"(p));
    return v;
}
// The same where p is 16-byte aligned only.
__device__ __forceinline__ Vec32 load32(const uint4* p, bool wide) {
    if (wide) return load32(p);
    return {__ldg(p), __ldg(p + 1)};
}

// Sixteen consecutive bf16 values (a, b) of a row as e4m3 and their block's
// scale byte.  The eight lanes 8i .. 8i+7 of a warp hold one block of 128 and
// call it together.
__device__ __forceinline__ uint4 quantize_lane16(const uint4& a, const uint4& b, uint32_t* sb) {
    float f[16];
    unpack8(a, f);
    unpack8(b, f + 8);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, finite_abs(f[j]));
    const unsigned lanes = 0xffu << (threadIdx.x & 24);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
    *sb = scale_byte(m);
    return quantize16(f, inverse_scale(*sb));
}

}  // namespace fp8
}  // namespace moe
