// product_rows.cu -- the product with an epilogue for a few rows (decode): the
// weights streamed once by every SM, CUDA-core FMAs.
//
//   y[p, n] = act( sum_k x[p, k] W[n, k] + bias[n] ) + residual[p, n],  p < kRows
//
// A block takes four features; its threads stride over K in 16-byte vectors,
// up to eight loads of W in flight each, and share each vector of x (from L1) among the
// features.  Bound by HBM: the tile kernel gives 128 features to an SM, so a
// 4096 x 4096 matrix keeps 64 of 152 SMs busy there even with K split.  fp32
// sums: a thread's in order, then fixed trees over lanes and warps.
//
// In a captured graph, us here / by the split tile kernel: 4096 x 4096, one row
// 7.6 (4.4 TB/s) / 11.0, two 7.3 / 11.0, three 8.3 / 11.1, four 13.5 / 11.1 (so
// kFewRows is 3); one row: 16384 x 4096 21.5 (6.2 TB/s) / 23.8, 1024 x 16384
// 10.0 / 16.6, 384 x 4096 2.7 / 7.2, 4096 x 512 2.5 / 5.3.
#include "act_dev.cuh"
#include "ld_dev.cuh"
#include "ptx.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kFeats = 4;     // features per block

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case MOE_ACT_RELU: return v < 0.f ? 0.f : v;       // NaN stays
        case MOE_ACT_GELU: return gelu(v);
        case MOE_ACT_SILU: return v * sigmoid(v);
        default: return v;
    }
}

template <int kRows, int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
product_rows_kernel(const uint4* x, const uint4* W, int N, int vec, ProductEpilogue e) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ float parts[kWarps][kFeats * kRows];
    constexpr int kStep = 32 * kWarps;
    constexpr int kDeep = 2;          // vectors of each feature in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n0 = (int)blockIdx.x * kFeats;
    float sum[kFeats][kRows] = {};
    for (int i = threadIdx.x; i < vec; i += kStep * kDeep) {
        uint4 a[kFeats][kDeep], xv[kRows][kDeep];
#pragma unroll
        for (int f = 0; f < kFeats; ++f)
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                a[f][j] = make_uint4(0, 0, 0, 0);
                if (i + kStep * j < vec && n0 + f < N)
                    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(a[f][j].x), "=r"(a[f][j].y), "=r"(a[f][j].z), "=r"(a[f][j].w)
                                 : "l"(W + (int64_t)(n0 + f) * vec + i + kStep * j)
                                 : "memory");
            }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                xv[r][j] = make_uint4(0, 0, 0, 0);
                if (i + kStep * j < vec) xv[r][j] = x[(int64_t)r * vec + i + kStep * j];
            }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            float c[kRows][8];
#pragma unroll
            for (int r = 0; r < kRows; ++r) unpack8(xv[r][j], c[r]);
#pragma unroll
            for (int f = 0; f < kFeats; ++f) {
                float b[8];
                unpack8(a[f][j], b);
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int q = 0; q < 8; ++q) sum[f][r] = fmaf(b[q], c[r][q], sum[f][r]);
            }
        }
    }
#pragma unroll
    for (int f = 0; f < kFeats; ++f)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int o = 16; o; o >>= 1) sum[f][r] += __shfl_xor_sync(0xffffffffu, sum[f][r], o);
            if (lane == f * kRows + r) parts[warp][lane] = sum[f][r];
        }
    __syncthreads();
    // one thread per result
    const int f = (int)threadIdx.x / kRows, r = (int)threadIdx.x % kRows, n = n0 + f;
    if (threadIdx.x >= kFeats * kRows || n >= N) return;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += parts[w][threadIdx.x];
    const int64_t at = (int64_t)r * N + n;
    if (e.bias) v += e.bias[n];
    v = activate(v, e.act);
    if (e.residual) v += __bfloat162float(e.residual[at]);
    if (e.out32) e.out32[at] = v;
    else e.out[at] = __float2bfloat16_rn(v);
}

template <int kRows>
cudaError_t launch(const __nv_bfloat16* x, const __nv_bfloat16* W, int N, int K, const ProductEpilogue& e,
                   cudaStream_t s) {
    const int vec = K / 8;
    const dim3 grid((unsigned)((N + kFeats - 1) / kFeats));
    const auto *xv = reinterpret_cast<const uint4*>(x), *wv = reinterpret_cast<const uint4*>(W);
    // warps that K fills
    if (vec > 8 * 64) return launch_pdl(product_rows_kernel<kRows, 8>, grid, dim3(256), 0, s, xv, wv, N, vec, e);
    return launch_pdl(product_rows_kernel<kRows, 4>, grid, dim3(128), 0, s, xv, wv, N, vec, e);
}

}  // namespace

cudaError_t launch_product_rows(const __nv_bfloat16* x, int rows, const __nv_bfloat16* W, int N, int K,
                                const ProductEpilogue& e, cudaStream_t s) {
    switch (rows) {
        case 1: return launch<1>(x, W, N, K, e, s);
        case 2: return launch<2>(x, W, N, K, e, s);
        case 3: return launch<3>(x, W, N, K, e, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
