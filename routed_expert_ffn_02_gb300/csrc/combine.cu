// combine.cu -- gate-weighted un-permute ("split/combine on GPU",
// dsv41-flash-offload wiki, file map):
//   out[t] = bf16( sum_{j<k} gates[t,j] * y_sorted[inv_perm[t*k + j]] )
// fp32 accumulation in ascending j, no atomics, so repeated runs are
// bit-identical (combine_dev.cuh).  One block per token row (grid-stride),
// 16-byte vectors.
#include "moe_internal.cuh"
#include "combine_dev.cuh"
#include "ld_dev.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

__global__ void __launch_bounds__(256)
combine_kernel(const uint4* y, const int32_t* inv_perm, const float* gates, int T, int k, int H,
               uint4* __restrict__ out) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int vec = H / 8;
    auto load = [&](int64_t i) { return y[i]; };
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        int64_t src[kMaxK];
        float g[kMaxK];
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) {
            src[j] = (j < k) ? (int64_t)inv_perm[t * k + j] * vec : 0;
            g[j] = (j < k) ? gates[t * k + j] : 0.f;
        }
        for (int v = threadIdx.x; v < vec; v += blockDim.x)
            out[t * vec + v] = combine_vec(load, src, g, k, v);
    }
}

// The same over fp32 y: 8-bit experts of a small batch, whose y stays in L2, so
// that the output is rounded once.  One thread per 8 output values.
__global__ void __launch_bounds__(256)
combine_f32_kernel(const float4* y, const int32_t* inv_perm, const float* gates, int k, int vec,
                   int64_t n, uint4* __restrict__ out) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t t = i / vec, v = i - t * vec;
    float4 a[kMaxK], b[kMaxK];
    float g[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
        if (j >= k) continue;
        const int64_t row = (int64_t)ld::i32(inv_perm + t * k + j) * vec + v;
        a[j] = ld::f32x4(y + 2 * row);
        b[j] = ld::f32x4(y + 2 * row + 1);
        g[j] = ld::f32(gates + t * k + j);
    }
    float s[8] = {};
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
        if (j >= k) continue;
        const float x[8] = {a[j].x, a[j].y, a[j].z, a[j].w, b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] = fmaf(g[j], x[q], s[q]);
    }
    uint4 o;
    __nv_bfloat162* po = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
    for (int q = 0; q < 4; ++q) po[q] = __floats2bfloat162_rn(s[2 * q], s[2 * q + 1]);
    out[i] = o;
}

}  // namespace

cudaError_t launch_combine_f32(const float* y_sorted, const int32_t* inv_perm, const float* gates,
                               int T, int k, int H, __nv_bfloat16* out, cudaStream_t s) {
    const int64_t n = (int64_t)T * (H / 8);
    if (n == 0) return cudaSuccess;
    return launch_pdl(combine_f32_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                      reinterpret_cast<const float4*>(y_sorted), inv_perm, gates, k, H / 8, n,
                      reinterpret_cast<uint4*>(out));
}

cudaError_t launch_combine(const __nv_bfloat16* y_sorted, const int32_t* inv_perm,
                           const float* gates, int T, int k, int H,
                           __nv_bfloat16* out, int num_sms, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    const int blocks = (int)std::min<int64_t>(T, (int64_t)num_sms * 8);
    return launch_pdl(combine_kernel, dim3(blocks), dim3(256), 0, s,
                      reinterpret_cast<const uint4*>(y_sorted), inv_perm, gates, T, k, H,
                      reinterpret_cast<uint4*>(out));
}

}  // namespace moe
