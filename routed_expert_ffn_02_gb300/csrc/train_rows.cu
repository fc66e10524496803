// train_rows.cu -- the training passes' row work: lists of the groups' rows,
// the gathers, the sums over a token's slots, and the 8-bit rows' values.
#include "fp8.cuh"
#include "ld_dev.cuh"
#include "ptx.cuh"
#include "train.cuh"

namespace moe {
namespace {

// Inclusive scan over the block's threads (blockDim.x <= 1024), with op + or max.
template <bool kMax>
__device__ int block_scan(int v, int* warp_vals) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = kMax ? max(v, u) : v + u;
    }
    __syncthreads();       // the values of a scan before have been read
    if (lane == 31) warp_vals[w] = v;
    __syncthreads();
    for (int i = 0; i < w; ++i) v = kMax ? max(v, warp_vals[i]) : v + warp_vals[i];
    return v;
}

// A thread per group: offsets forced to ascend, then scans of the chunk
// counts and of the padded row counts.
__global__ void __launch_bounds__(1024)
plan_rows_kernel(const int32_t* offsets, int rows, int E, int most, RowLists l, WsHeader* hdr) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ int off[kMaxE + 1];
    __shared__ int warp_vals[32];
    const int e = threadIdx.x;
    const int given = e < E ? ld::i32(offsets + e) : 0, end = ld::i32(offsets + E);
    const int v = block_scan<true>(min(max(given, 0), rows), warp_vals);
    if (e < E) off[e] = v;
    if (e == E - 1) off[E] = max(v, min(max(end, 0), rows));
    if ((e < E && v != given) || (e == 0 && (given != 0 || end != rows)))
        set_status(hdr, MOE_ERR_BAD_INDEX);
    __syncthreads();
    const int c = e < E ? off[e + 1] - off[e] : 0;
    const int size = chunk_size(c, most);
    const int n = size ? (c + size - 1) / size : 0;
    const int pad = (c + 15) & ~15;
    const int n_incl = block_scan<false>(n, warp_vals);
    const int pad_incl = block_scan<false>(pad, warp_vals);
    if (e < E) {
        RowChunk ch = {e, v, c, pad_incl - pad};
        if (l.groups) l.groups[e] = ch;
        for (int i = 0; i < n; ++i) {
            ch.row0 = v + i * size;
            ch.rows = min(size, c - i * size);
            ch.row0_pad = pad_incl - pad + i * size;
            l.chunks[n_incl - n + i] = ch;
        }
        if (e == E - 1) *l.n_chunks = n_incl;
    }
}

// Eight e4m3 values (one 8-byte word) of one scale as bf16: exact.
__device__ __forceinline__ uint4 widen8(uint2 q, float scale) {
    uint32_t o[4];
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ float scale_of(uint32_t b) {
    return __uint_as_float(b == 0 ? 1u << 22 : b == 255 ? 0x7fc00000u : b << 23);
}

// Warps take parts of 16 rows of the chunks in turn; a row is copied in
// 16-byte vectors, eight per lane in flight.
constexpr int kPartRows = 16;
__global__ void __launch_bounds__(256)
gather_rows_kernel(GatherJob g, RowLists l, int most) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int vec = g.H / 8;
    const int per_chunk = most / kPartRows;
    const int64_t parts = (int64_t)ld::i32(l.n_chunks) * per_chunk;
    // a warp per row: the rows of a part are spread over the block's warps
    for (int64_t part = blockIdx.x; part < parts; part += gridDim.x) {
        const int4 c = *reinterpret_cast<const int4*>(l.chunks + part / per_chunk);
        const int r0 = (int)(part % per_chunk) * kPartRows;
        const int r1 = min(r0 + kPartRows, g.padded ? (c.z + 15) & ~15 : c.z);
        for (int r = r0 + (int)(threadIdx.x >> 5); r < r1; r += (int)(blockDim.x >> 5)) {
            const bool in = r < c.z;
            const int64_t to = (int64_t)((g.padded ? c.w : c.y) + r) * vec;
            const int slot = in ? ld::i32(g.perm + c.y + r) : 0;
            const bool ok = in && slot >= 0 && slot < g.P;
            const int64_t t = slot / g.k;
            uint4* d0 = reinterpret_cast<uint4*>(g.dst0) + to;
            uint4* d1 = reinterpret_cast<uint4*>(g.dst1) + to;
            for (int i0 = lane; i0 < vec; i0 += 32 * 8) {
                uint4 a[8], b[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = i0 + 32 * j;
                    a[j] = b[j] = make_uint4(0, 0, 0, 0);
                    if (i < vec && ok) {
                        if (g.src0_scales) {
                            const uint2 q = reinterpret_cast<const uint2*>(g.src0)[t * vec + i];
                            a[j] = widen8(q, scale_of(g.src0_scales[t * (g.H / 128) + (i >> 4)]));
                        } else {
                            a[j] = reinterpret_cast<const uint4*>(g.src0)[t * vec + i];
                        }
                        if (g.src1) b[j] = reinterpret_cast<const uint4*>(g.src1)[t * vec + i];
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = i0 + 32 * j;
                    if (i < vec) {
                        d0[i] = a[j];
                        if (g.src1) d1[i] = b[j];
                    }
                }
            }
        }
    }
}

// The parts are fp32: rounding each slot's part to bf16 as well would make the
// rounding error of d_x 1.22 times as large (relative RMS 2.9e-3 for 2.4e-3).
__global__ void __launch_bounds__(256)
sum_slots_kernel(const float4* y, const int32_t* inv, int T, int k, int vec, uint2* out) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t P = (int64_t)T * k;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        int64_t src[kMaxK];
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) {
            const int p = j < k ? ld::i32(inv + t * k + j) : -1;
            src[j] = p >= 0 && p < P ? (int64_t)p * vec : -1;
        }
        for (int v = threadIdx.x; v < vec; v += blockDim.x) {
            float4 r[kMaxK];
#pragma unroll
            for (int j = 0; j < kMaxK; ++j)
                r[j] = src[j] >= 0 ? y[src[j] + v] : make_float4(0.f, 0.f, 0.f, 0.f);
            float4 s = r[0];
#pragma unroll
            for (int j = 1; j < kMaxK; ++j) {
                s.x += r[j].x;
                s.y += r[j].y;
                s.z += r[j].z;
                s.w += r[j].w;
            }
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            out[t * vec + v] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                          *reinterpret_cast<const uint32_t*>(&hi));
        }
    }
}

__global__ void __launch_bounds__(256)
sum_gate_parts_kernel(const float* parts, int n, int P, const int32_t* inv, float* d_gates) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t s = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (s >= P) return;
    const int p = inv ? ld::i32(inv + s) : (int)s;
    float sum = 0.f;
    if (p >= 0 && p < P)
        for (int i = 0; i < n; ++i) sum += parts[(int64_t)i * P + p];
    d_gates[s] = sum;
}

__global__ void __launch_bounds__(256)
dequantize_rows_kernel(const uint2* q, const uint8_t* scales, int64_t n, uint4* x) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    // eight values each, sixteen of these to a block of 128
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step)
        x[i] = widen8(q[i], scale_of(scales[i >> 4]));
}

}  // namespace

cudaError_t launch_plan_rows(const int32_t* offsets, int rows, int E, int most, const RowLists& l,
                             WsHeader* hdr, cudaStream_t s) {
    return launch_pdl(plan_rows_kernel, dim3(1), dim3((E + 31) / 32 * 32), 0, s, offsets, rows, E,
                      most, l, hdr);
}

cudaError_t launch_gather_rows(const GatherJob& g, const RowLists& l, int64_t parts_bound, int most,
                               int num_sms, cudaStream_t s) {
    const int blocks = (int)(parts_bound < 8 * num_sms ? (parts_bound > 0 ? parts_bound : 1) : 8 * num_sms);
    return launch_pdl(gather_rows_kernel, dim3(blocks), dim3(256), 0, s, g, l, most);
}

cudaError_t launch_sum_slots(const float* y, const int32_t* inv, int T, int k, int H,
                             __nv_bfloat16* out, int num_sms, cudaStream_t s) {
    const int blocks = T < 8 * num_sms ? T : 8 * num_sms;
    return launch_pdl(sum_slots_kernel, dim3(blocks), dim3(256), 0, s,
                      reinterpret_cast<const float4*>(y), inv, T, k, H / 4,
                      reinterpret_cast<uint2*>(out));
}

cudaError_t launch_sum_gate_parts(const float* parts, int n, int P, const int32_t* inv,
                                  float* d_gates, cudaStream_t s) {
    return launch_pdl(sum_gate_parts_kernel, dim3((unsigned)(((int64_t)P + 255) / 256)), dim3(256), 0, s, parts, n, P,
                      inv, d_gates);
}

cudaError_t launch_dequantize_rows(const uint8_t* q, const uint8_t* scales, int64_t rows, int K,
                                   __nv_bfloat16* x, int num_sms, cudaStream_t s) {
    const int64_t n = rows * (K / 8);
    const int64_t want = (n + 255) / 256;
    const int blocks = (int)(want < 16 * num_sms ? want : 16 * num_sms);
    return launch_pdl(dequantize_rows_kernel, dim3(blocks), dim3(256), 0, s,
                      reinterpret_cast<const uint2*>(q), scales, n, reinterpret_cast<uint4*>(x));
}

}  // namespace moe
