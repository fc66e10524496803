// fp8.cuh -- 8-bit floating point with a power-of-two scale per block of 128:
// the format, its device conversions, and the block-scaled tensor-core
// instructions (tcgen05 kind::mxf8f6f4) shared by the 8-bit kernels.
//
// Format.  A value is e4m3 (largest finite value 448); the blocks are 1 x 128
// along a row for activations and 128 x 128 for weight matrices.  A block's
// scale is one byte b, standing for 2^(b - 127): the smallest power of two,
// at least 2^-127, for which no finite value of the block exceeds 448 times
// it.  Values round to nearest even; a value that is not finite becomes NaN
// and does not count towards its block's scale.
//
// Why a power of two: the tensor core then applies the scale itself.
// kind::mxf8f6f4 multiplies each 32 values of K of a row of A (and of B) by
// 2^(byte - 127) inside the MMA, so four K steps of 32 that use the same byte
// are a block of 128, and the accumulator stays one fp32 tile in TMEM.  An
// arbitrary fp32 scale would have to be applied between blocks by CUDA cores
// reading the accumulator back every 128 of K.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "ld_dev.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace fp8 {

constexpr int kBlock = 128;

// Scale byte for a block whose largest finite magnitude is amax (fp32, >= 0).
// With amax = m * 2^x, 1 <= m < 2, and 448 = 1.75 * 2^8, the exponent is
// x - 8, one more when m > 1.75; subnormal amax and zero give byte 0.  The
// largest fp32 gives byte 247, so 255 (NaN) never occurs.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int b = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(b, 0);
}
// 2^(127 - b), the factor that divides by the scale; exact for b <= 253.
__device__ __forceinline__ float inverse_scale(uint32_t b) {
    return __uint_as_float((254u - b) << 23);
}
// |v| for the block maximum: 0 where v is not finite.
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : 0.f;
}
// v / scale, NaN where v is not finite (the conversion would saturate inf).
__device__ __forceinline__ float scaled(float v, float inv) {
    const float a = v * inv;
    return fabsf(v) <= 3.402823466e38f ? a : __uint_as_float(0x7fffffffu);
}
// Two fp32 -> two e4m3 bytes (a in the low one), round to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// Sixteen consecutive values as e4m3 bytes.
__device__ __forceinline__ uint4 quantize16(const float* v, float inv) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = pack_e4m3x4(scaled(v[4 * i], inv), scaled(v[4 * i + 1], inv),
                           scaled(v[4 * i + 2], inv), scaled(v[4 * i + 3], inv));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// silu(g) * u in fp32, by the hardware's approximate reciprocal (about one
// ulp): the result is rounded to 4 significant bits next.
__device__ __forceinline__ float swiglu(float g, float u) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-g)));
    return g * r * u;
}

// ---- tensor core ---------------------------------------------------------

// Instruction descriptor, kind::mxf8f6f4, e4m3 x e4m3, both K-major, scales
// as exponent bytes (bit 23); the byte of the scale words to use goes to bits
// 4-5 (B) and 29-30 (A), see with_scale_byte.
constexpr uint32_t make_idesc(int M, int N) {
    return (1u << 23) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_scale_byte(uint32_t idesc, int i) {
    return idesc | ((uint32_t)i << 4) | ((uint32_t)i << 29);
}

// Scale words in TMEM: four bytes of a row, one per 128 of K, make a 32-bit
// word; the words of 128 rows fill 4 columns (row r at lane r mod 32, column
// r / 32, repeated in the four lane quarters), copied from 512 bytes of
// shared memory laid out [r mod 32][r / 32].
constexpr int kScaleCols = 4;                    // TMEM columns per 128 rows
constexpr int kScaleBytes = 512;                 // shared bytes per 128 rows
constexpr int kGroupBlocks = 4;                  // blocks of 128 per scale word
// Descriptor of such a 512-byte piece: no swizzle, 8-row groups of 16-byte
// rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(128 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}
__device__ __forceinline__ void scale_copy(uint32_t tmem, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sdesc)
                 : "memory");
}
// D[tmem] (+)= (A[smem] scaled by sa[tmem]) (B[smem] scaled by sb[tmem])^T,
// K = 32, one elected thread.
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                    uint32_t idesc, uint32_t sa, uint32_t sb,
                                    uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate));
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate));
}

// The tiles of a launch: the planner's lists, or, for a single expert, the
// rows [lo, lo + n) that its two offsets give, cut into tiles here (no planner
// launch; offsets outside [0, rows] are cut, and recorded by the first CTA).
struct OneGroup {
    int lo, n;
};
__device__ __forceinline__ OneGroup one_group(const Fp8Args& args) {
    const int a = ld::i32_cg(args.group), b = ld::i32_cg(args.group + 1);
    const int lo = min(max(a, 0), args.rows);
    if ((a != 0 || b != args.rows) && blockIdx.x == 0 && threadIdx.x == 0)
        set_status(args.hdr, MOE_ERR_BAD_INDEX);
    return {lo, max(0, min(b, args.rows) - lo)};
}
__device__ __forceinline__ FatTile group_tile(const OneGroup& g, int i) {
    return FatTile{0, g.lo + i * kTileM, max(0, min(kTileM, g.n - i * kTileM)), 0};
}

// Scale word w (bytes 4w .. 4w+3) of a row of nb scale bytes; bytes past nb
// read as 127 (a factor of one, for operands that TMA filled with zeros).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int w, int nb) {
    if ((nb & 3) == 0) return ld::u32(reinterpret_cast<const uint32_t*>(row) + w);
    uint32_t v = 0;
#pragma unroll 1   // rare; unrolled, the loads of several words raise the kernels' registers
    for (int i = 3; i >= 0; --i)
        v = (v << 8) | (4 * w + i < nb ? ld::u8(row + 4 * w + i) : 127u);
    return v;
}

}  // namespace fp8
}  // namespace moe
