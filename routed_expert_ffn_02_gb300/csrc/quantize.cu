// quantize.cu -- bf16 to 8-bit floating point with a power-of-two scale per
// block of 128 (the format is in fp8.cuh).
//
// One pass over the data, bound by HBM: 2 bytes read and 1 + 1/128 (rows) or
// 1 + 1/16384 (matrices) written per value.  16384 x 4096 rows take 31.9 us
// (6.3 TB/s), 64 matrices of 2048 x 4096 223.6 us (7.2 TB/s).  The arithmetic
// is kept out of the way: the maximum is taken on packed pairs of bf16, and
// values that are infinite (found by the maximum) are handled on a path of
// their own; checking each value in fp32 took 41 and 252 us.
//
//   rows      eight lanes hold a 1 x 128 block, 16 values (32 bytes) each:
//             one 32-byte load, three shuffles for the maximum, one 16-byte
//             store.  The same kernel writes the rows of the experts' input:
//             token t's quantised row goes to its k sorted positions, so a
//             token is read and quantised once however many experts it has.
//   matrices  one CTA per 128 x 128 block, 64 values per thread in registers.
#include <algorithm>

#include "ld_dev.cuh"
#include "quantize_dev.cuh"

namespace moe {
namespace {

using namespace fp8;

// Vector i is the values [16 i, 16 i + 16) of x [rows, K]; dst == nullptr
// writes row r to q row r, else to rows dst[r * k .. r * k + k) (a position
// outside [0, P) is skipped: the slot of a bad index has none).
template <int U>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(const uint4* __restrict__ x, int64_t n16, int per_row,
                     const int32_t* __restrict__ dst, int k, int64_t P, uint4* __restrict__ q,
                     uint8_t* __restrict__ scales) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    auto put = [&](int64_t i, const uint4& o, uint32_t sb) {
        if (!dst) {
            q[i] = o;
            if ((threadIdx.x & 7) == 0) scales[i >> 3] = (uint8_t)sb;
            return;
        }
        const int64_t r = i / per_row;
        const int c = (int)(i - r * per_row);
        for (int j = 0; j < k; ++j) {
            const int64_t p = ld::i32(dst + r * k + j);
            if (p < 0 || p >= P) continue;
            q[p * per_row + c] = o;
            if ((threadIdx.x & 7) == 0) scales[(p * per_row + c) >> 3] = (uint8_t)sb;
        }
    };
    // the CTA's first vector, U per thread 256 apart: n16 and the offsets are
    // multiples of 8, so the eight lanes of a block are together
    const bool wide = reinterpret_cast<uintptr_t>(x) % 32 == 0;
    const int64_t i0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
    Vec32 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (i0 + 256 * u < n16) v[u] = load32(x + 2 * (i0 + 256 * u), wide);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (i0 + 256 * u >= n16) break;
        uint32_t sb;
        const uint4 o = quantize_lane16(v[u], &sb);
        put(i0 + 256 * u, o, sb);
    }
}

__global__ void __launch_bounds__(256, 3)
quantize_matrices_kernel(const uint4* __restrict__ w, int n_cb, uint4* __restrict__ q,
                         uint8_t* __restrict__ scales) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ float red[8];
    const int64_t blk = blockIdx.x;               // (matrix, row block), column block
    const int64_t rb = blk / n_cb;
    const int cb = (int)(blk - rb * n_cb);
    const bool wide = reinterpret_cast<uintptr_t>(w) % 32 == 0;
    const int64_t ld = (int64_t)n_cb * (kBlock / 16);      // 16-value vectors per row
    const int64_t base = rb * kBlock * ld + (int64_t)cb * (kBlock / 16) +
                         (int64_t)(threadIdx.x >> 3) * ld + (threadIdx.x & 7);
    Vec32 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load32(w + 2 * (base + (int64_t)(32 * i) * ld), wide);
    auto block_max = [&](float m) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
        return m;
    };
    float m = block_max(fmaxf(fmaxf(amax16(v[0]), amax16(v[1])), fmaxf(amax16(v[2]), amax16(v[3]))));
    const bool has_inf = m > 3.402823466e38f;   // the same for the block
    if (has_inf) {
        __syncthreads();
        m = block_max(fmaxf(fmaxf(amax16_finite(v[0]), amax16_finite(v[1])),
                            fmaxf(amax16_finite(v[2]), amax16_finite(v[3]))));
    }
    const uint32_t sb = scale_byte(m);
    const float inv = inverse_scale(sb);
    if (threadIdx.x == 0) scales[blk] = (uint8_t)sb;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[base + (int64_t)(32 * i) * ld] = convert16(v[i], inv, has_inf);
}

__global__ void __launch_bounds__(256)
clear_inverse_kernel(int64_t P, int32_t* __restrict__ inv) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    for (int64_t p = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; p < P;
         p += (int64_t)gridDim.x * blockDim.x)
        inv[p] = -1;
}

// inv[perm[p]] = p for the slots in range, over -1 (unsigned: the largest).  A
// route list of a bad index ends in entries that nobody wrote: of two entries
// for one slot the first stands, and a slot without one keeps -1, so whatever
// they hold, no other token's row is written to its place.
__global__ void __launch_bounds__(256)
invert_perm_kernel(const int32_t* __restrict__ perm, int64_t P, int32_t* __restrict__ inv) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    for (int64_t p = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; p < P;
         p += (int64_t)gridDim.x * blockDim.x) {
        const int32_t s = ld::i32(perm + p);
        if (s >= 0 && s < P) atomicMin(reinterpret_cast<unsigned*>(inv + s), (unsigned)p);
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const __nv_bfloat16* x, int64_t rows, int K, const int32_t* dst,
                                 int k, int64_t P, uint8_t* q, uint8_t* scales, int num_sms,
                                 cudaStream_t s) {
    const int64_t n16 = rows * K / 16;
    if (n16 == 0) return cudaSuccess;
    // Two vectors per thread (64 bytes in flight) once they fill the GPU four
    // times (1 / 2 / 4 of them: 32.7 / 31.9 / 32.8 us at 16384 x 4096), else
    // one, which spreads a small batch over more SMs.
    auto go = [&]<int U>() {
        return launch_pdl(quantize_rows_kernel<U>, dim3((unsigned)((n16 + 256 * U - 1) / (256 * U))),
                          dim3(256), 0, s, reinterpret_cast<const uint4*>(x), n16, K / 16, dst, k, P,
                          reinterpret_cast<uint4*>(q), scales);
    };
    return n16 >= (int64_t)num_sms * 2048 ? go.template operator()<2>() : go.template operator()<1>();
}

cudaError_t launch_quantize_matrices(const __nv_bfloat16* w, int64_t n, int N, int K, uint8_t* q,
                                     uint8_t* scales, cudaStream_t s) {
    const int64_t blocks = n * (N / fp8::kBlock) * (K / fp8::kBlock);
    if (blocks == 0) return cudaSuccess;
    return launch_pdl(quantize_matrices_kernel, dim3((unsigned)blocks), dim3(256), 0, s,
                      reinterpret_cast<const uint4*>(w), K / fp8::kBlock,
                      reinterpret_cast<uint4*>(q), scales);
}

cudaError_t launch_invert_perm(const int32_t* perm, int64_t P, int32_t* inv, int num_sms,
                               cudaStream_t s) {
    if (P == 0) return cudaSuccess;
    const int64_t blocks = std::min<int64_t>((P + 255) / 256, (int64_t)num_sms * 8);
    const cudaError_t e =
        launch_pdl(clear_inverse_kernel, dim3((unsigned)blocks), dim3(256), 0, s, P, inv);
    if (e != cudaSuccess) return e;
    return launch_pdl(invert_perm_kernel, dim3((unsigned)blocks), dim3(256), 0, s, perm, P, inv);
}

}  // namespace moe
