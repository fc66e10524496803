// quantize.cu -- bf16 to 8-bit floating point with a power-of-two scale per
// block of 128 (the format is in fp8.cuh).
//
// One pass over the data, bound by HBM: 2 bytes read and 1 + 1/128 (rows) or
// 1 + 1/16384 (matrices) written per value.
//
//   rows      eight lanes hold a 1 x 128 block, 16 values (32 bytes) each:
//             two 16-byte loads, three shuffles for the maximum, one 16-byte
//             store.  The same kernel writes the rows of the experts' input:
//             token t's quantised row goes to its k sorted positions, so a
//             token is read and quantised once however many experts it has.
//   matrices  one CTA per 128 x 128 block, 64 values per thread in registers.
#include <algorithm>

#include "quantize_dev.cuh"

namespace moe {
namespace {

using namespace fp8;

// Thread i quantises values [16 i, 16 i + 16) of x [rows, K]; dst == nullptr
// writes row r to q row r, else to rows dst[r * k .. r * k + k) (a position
// outside [0, P) is skipped: route lists of a bad index leave it unset).
__global__ void __launch_bounds__(256)
quantize_rows_kernel(const uint4* __restrict__ x, int64_t n16, int per_row,
                     const int32_t* __restrict__ dst, int k, int64_t P, uint4* __restrict__ q,
                     uint8_t* __restrict__ scales) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16;
         i += (int64_t)gridDim.x * blockDim.x) {
        // n16 is a multiple of 8, so the eight lanes of a block are together
        uint32_t sb;
        const uint4 o = quantize_lane16(__ldg(x + 2 * i), __ldg(x + 2 * i + 1), &sb);
        const int64_t r = i / per_row;
        const int c = (int)(i - r * per_row);
        if (!dst) {
            q[i] = o;
            if ((threadIdx.x & 7) == 0) scales[i >> 3] = (uint8_t)sb;
        } else {
            for (int j = 0; j < k; ++j) {
                const int64_t p = dst[r * k + j];
                if (p < 0 || p >= P) continue;
                q[p * per_row + c] = o;
                if ((threadIdx.x & 7) == 0) scales[(p * per_row + c) >> 3] = (uint8_t)sb;
            }
        }
    }
}

__global__ void __launch_bounds__(256)
quantize_matrices_kernel(const uint4* __restrict__ w, int n_rb, int n_cb, uint2* __restrict__ q,
                         uint8_t* __restrict__ scales) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ float red[8];
    const int64_t blk = blockIdx.x;               // (matrix, row block), column block
    const int64_t rb = blk / n_cb;
    const int cb = (int)(blk - rb * n_cb);
    (void)n_rb;
    const int64_t ld = (int64_t)n_cb * (kBlock / 8);       // 8-value vectors per row
    const int64_t base = rb * kBlock * ld + (int64_t)cb * (kBlock / 8) +
                         (int64_t)(threadIdx.x >> 4) * ld + (threadIdx.x & 15);
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __ldg(w + base + (int64_t)(16 * i) * ld);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(f[j]));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    const uint32_t sb = scale_byte(m);
    const float inv = inverse_scale(sb);
    if (threadIdx.x == 0) scales[blk] = (uint8_t)sb;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
        uint2 o;
        o.x = pack_e4m3x4(scaled(f[0], inv), scaled(f[1], inv), scaled(f[2], inv), scaled(f[3], inv));
        o.y = pack_e4m3x4(scaled(f[4], inv), scaled(f[5], inv), scaled(f[6], inv), scaled(f[7], inv));
        q[base + (int64_t)(16 * i) * ld] = o;
    }
}

// inv_perm[perm[p]] = p for the slots in range.
__global__ void __launch_bounds__(256)
invert_perm_kernel(const int32_t* __restrict__ perm, int64_t P, int32_t* __restrict__ inv) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    for (int64_t p = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; p < P;
         p += (int64_t)gridDim.x * blockDim.x) {
        const int32_t s = perm[p];
        if (s >= 0 && s < P) inv[s] = (int32_t)p;
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const __nv_bfloat16* x, int64_t rows, int K, const int32_t* dst,
                                 int k, int64_t P, uint8_t* q, uint8_t* scales, int num_sms,
                                 cudaStream_t s) {
    const int64_t n16 = rows * K / 16;
    if (n16 == 0) return cudaSuccess;
    const int64_t blocks = std::min<int64_t>((n16 + 255) / 256, (int64_t)num_sms * 16);
    return launch_pdl(quantize_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, s,
                      reinterpret_cast<const uint4*>(x), n16, K / 16, dst, k, P,
                      reinterpret_cast<uint4*>(q), scales);
}

cudaError_t launch_quantize_matrices(const __nv_bfloat16* w, int64_t n, int N, int K, uint8_t* q,
                                     uint8_t* scales, cudaStream_t s) {
    const int64_t blocks = n * (N / fp8::kBlock) * (K / fp8::kBlock);
    if (blocks == 0) return cudaSuccess;
    return launch_pdl(quantize_matrices_kernel, dim3((unsigned)blocks), dim3(256), 0, s,
                      reinterpret_cast<const uint4*>(w), N / fp8::kBlock, K / fp8::kBlock,
                      reinterpret_cast<uint2*>(q), scales);
}

cudaError_t launch_invert_perm(const int32_t* perm, int64_t P, int32_t* inv, int num_sms,
                               cudaStream_t s) {
    if (P == 0) return cudaSuccess;
    const int64_t blocks = std::min<int64_t>((P + 255) / 256, (int64_t)num_sms * 8);
    return launch_pdl(invert_perm_kernel, dim3((unsigned)blocks), dim3(256), 0, s, perm, P, inv);
}

}  // namespace moe
