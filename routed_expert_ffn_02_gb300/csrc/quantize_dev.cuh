// quantize_dev.cuh -- the row quantiser's arithmetic for one lane, shared by
// the quantiser kernel and the small-batch prologue (the format is in fp8.cuh).
#pragma once

#include "fp8.cuh"
#include "ld_dev.cuh"

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
                 : "l"(p)
                 : "memory");
    return v;
}
// The same where p is 16-byte aligned only.
__device__ __forceinline__ Vec32 load32(const uint4* p, bool wide) {
    if (wide) return load32(p);
    return {ld::u32x4(p), ld::u32x4(p + 1)};
}

// Largest magnitude of 16 bf16 values, NaN apart (0 if there is nothing else);
// two values per instruction.
__device__ __forceinline__ float amax16(const Vec32& v) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
    __nv_bfloat162 m = __habs2(p[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(p[i]));
    return fmaxf(0.f, fmaxf(__low2float(m), __high2float(m)));   // 0: both may be NaN
}
// The same over finite values only.
__device__ __forceinline__ float amax16_finite(const Vec32& v) {
    float f[16], m = 0.f;
    unpack8(v.a, f);
    unpack8(v.b, f + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(f[i]));
    return m;
}
// e4m3 of 16 values.  has_inf: infinities must become NaN (the conversion
// would saturate them); NaN stays NaN by itself.
__device__ __forceinline__ uint4 convert16(const Vec32& v, float inv, bool has_inf) {
    float f[16];
    unpack8(v.a, f);
    unpack8(v.b, f + 8);
    if (has_inf) return quantize16(f, inv);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = pack_e4m3x4(f[4 * i] * inv, f[4 * i + 1] * inv, f[4 * i + 2] * inv, f[4 * i + 3] * inv);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sixteen consecutive bf16 values of a row as e4m3 and their block's scale
// byte.  The eight lanes 8i .. 8i+7 of a warp hold one block of 128 and call
// it together.
__device__ __forceinline__ uint4 quantize_lane16(const Vec32& v, uint32_t* sb) {
    const unsigned lanes = 0xffu << (threadIdx.x & 24);
    float m = amax16(v);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
    const bool has_inf = m > 3.402823466e38f;   // the same for the eight lanes
    if (has_inf) {
        m = amax16_finite(v);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
    }
    *sb = scale_byte(m);
    return convert16(v, inverse_scale(*sb), has_inf);
}

}  // namespace fp8
}  // namespace moe
