// train_rows.cu -- the training passes' row work: lists of the groups' rows,
// the gathers, the sums over a token's slots, and the 8-bit rows' values.
#include <climits>

#include "fp8.cuh"
#include "ld_dev.cuh"
#include "ptx.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Groups per thread in the scans of E groups: 1, or enough for kMaxE.
constexpr int kMostPerThread = kMaxE / kThreads;

// Exclusive scan over the block's threads, + or max (from 0).
template <bool kMax>
__device__ int scan_before(int v, int* warp_vals) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl = kMax ? max(incl, u) : incl + u;
    }
    __syncthreads();       // the values of a scan before have been read
    if (lane == 31) warp_vals[w] = incl;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) before = 0;
    for (int i = 0; i < w; ++i) before = kMax ? max(before, warp_vals[i]) : before + warp_vals[i];
    return before;
}

// The groups of offsets [E + 1], the same in every block that asks: first row
// off[e] (forced to ascend inside [0, rows]) and first padded row pad[e].
struct Groups {
    int off[kMaxE + 1], pad[kMaxE + 1];
    int warp_vals[kThreads / 32];
};
template <int kPerThread>
__device__ void scan_groups(Groups& g, const int32_t* offsets, int rows, int E, WsHeader* hdr) {
    const int e0 = threadIdx.x * kPerThread;
    int given[kPerThread], v[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) given[i] = e0 + i < E ? ld::i32(offsets + e0 + i) : 0;
    const int end = ld::i32(offsets + E);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        v[i] = min(max(given[i], 0), rows);
        if (i) v[i] = max(v[i], v[i - 1]);
    }
    const int before = scan_before<true>(v[kPerThread - 1], g.warp_vals);
    bool bad = threadIdx.x == 0 && (given[0] != 0 || end != rows);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        v[i] = max(v[i], before);
        if (e0 + i < E) {
            g.off[e0 + i] = v[i];
            bad |= v[i] != given[i];
            if (e0 + i == E - 1) g.off[E] = max(v[i], min(max(end, 0), rows));
        }
    }
    if (bad && hdr) set_status(hdr, MOE_ERR_BAD_INDEX);
    __syncthreads();
    int p[kPerThread], sum = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        p[i] = sum;
        if (e0 + i < E) sum += (g.off[e0 + i + 1] - g.off[e0 + i] + 15) & ~15;
    }
    const int pad_before = scan_before<false>(sum, g.warp_vals);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
        if (e0 + i <= E) g.pad[e0 + i] = pad_before + p[i];
    if (threadIdx.x == kThreads - 1 && E == kThreads * kPerThread) g.pad[E] = pad_before + sum;
    __syncthreads();
}

// The lists of the groups, by one block.  Few chunks (kSorted at most: a few
// rounds of the grid) are listed from large to small (in classes of 16 rows; a
// group's stay together, they read the same weights), so that the items of one
// round cost about the same and the last round has the smallest: backward of
// 1999 tokens over 32 experts 267 us, unsorted 276; of many rounds it gains
// nothing (8192 tokens over 64 experts, forward: 2275 us, unsorted 2255).  The
// order inside a class is left to the atomics: it decides when an item runs, not
// what it computes.
constexpr int kSorted = 256;
template <int kPerThread>
__device__ void write_lists(Groups& g, int rows, int E, int most, const RowLists& l) {
    const int per_class = max_chunks(rows, E, most) <= kSorted ? 16 : INT_MAX;   // one class for all
    __shared__ int at[17];              // chunks in larger classes, then the class's next place
    const int e0 = threadIdx.x * kPerThread;
    if (threadIdx.x < 17) at[threadIdx.x] = 0;
    __syncthreads();
    for (int e = e0; e < e0 + kPerThread && e < E; ++e) {
        const int c = g.off[e + 1] - g.off[e], size = chunk_size(c, most);
        if (size) atomicAdd(&at[size / per_class], chunk_count(c, size));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int before = 0;
        for (int i = 16; i >= 0; --i) {
            const int n = at[i];
            at[i] = before;
            before += n;
        }
        *l.n_chunks = before;
        l.ends[0] = g.off[0];
        l.ends[1] = g.off[E];
    }
    __syncthreads();
    for (int e = e0; e < e0 + kPerThread && e < E; ++e) {
        const int v = g.off[e], c = g.off[e + 1] - v, size = chunk_size(c, most);
        RowChunk ch = {e, v, c, g.pad[e]};
        l.groups[e] = ch;
        if (!size) continue;
        int to = atomicAdd(&at[size / per_class], chunk_count(c, size));
        for (uint32_t r = 0; r < (uint32_t)c; r += (uint32_t)size) {
            ch.row0 = v + (int)r;
            ch.rows = min(size, c - (int)r);
            ch.row0_pad = g.pad[e] + (int)r;
            l.chunks[to++] = ch;
        }
    }
}

template <int kPerThread>
__global__ void __launch_bounds__(kThreads)
plan_rows_kernel(const int32_t* offsets, int rows, int E, int most, RowLists l, WsHeader* hdr) {
    __shared__ Groups g;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    scan_groups<kPerThread>(g, offsets, rows, E, hdr);
    write_lists<kPerThread>(g, rows, E, most, l);
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

// Forward: xs[p] = x[perm[p] / k] for the groups' rows, a warp per row, eight
// 16-byte vectors per lane in flight; block 0 writes the lists.  65536 x 4096
// rows of 8192 tokens: 132 us, 4.1 TB/s written.
template <int kPerThread>
__global__ void __launch_bounds__(kThreads)
forward_rows_kernel(const uint4* x, const int32_t* perm, int k, int vec, const int32_t* offsets, int P, int E,
                    int most, uint4* xs, RowLists l, WsHeader* hdr) {
    __shared__ Groups g;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (blockIdx.x == 0) {
        scan_groups<kPerThread>(g, offsets, P, E, hdr);
        write_lists<kPerThread>(g, P, E, most, l);
    }
    const int lane = threadIdx.x & 31;
    for (int64_t p = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); p < P; p += (int64_t)gridDim.x * (kThreads / 32)) {
        // a position without a slot (a routed index was skipped) is a zero row
        const int slot = ld::i32(perm + p);
        const bool in = slot >= 0 && slot < P;
        const uint4* from = x + (int64_t)(in ? slot / k : 0) * vec;
        uint4* to = xs + p * vec;
        for (int i0 = lane; i0 < vec; i0 += 32 * 8) {
            uint4 a[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] = make_uint4(0, 0, 0, 0);
                if (in && i0 + 32 * j < vec) a[j] = from[i0 + 32 * j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + 32 * j < vec) to[i0 + 32 * j] = a[j];
        }
    }
}

// Backward: each token's rows of x and d_out to the padded rows of its slots,
// and zeros to the padding.  A warp takes a token, so that a row is read once
// however many slots it has (by sorted row, x and d of 16384 tokens do not fit
// L2 together and were read from memory k times: 631 us at 16384 x 4096, k = 8;
// 392 this way, 6.2 TB/s).
// p: a position of the groups, off[0] <= p < off[E] (offsets that start above 0
// leave positions before the first group, which have no padded row).
__device__ __forceinline__ int64_t padded_row(const Groups& g, int E, int p) {
    int lo = 0, hi = E;          // the last group whose first row is not above p
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.off[mid] <= p) lo = mid;
        else hi = mid;
    }
    return (int64_t)g.pad[lo] + (p - g.off[lo]);
}

template <int kPerThread, bool kX>
__global__ void __launch_bounds__(kThreads)
backward_rows_kernel(BackwardRows q) {
    __shared__ Groups g;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    scan_groups<kPerThread>(g, q.offsets, q.T * q.k, q.E, blockIdx.x == 0 ? q.hdr : nullptr);
    if (blockIdx.x == 0) write_lists<kPerThread>(g, q.T * q.k, q.E, q.most, q.lists);
    const int lane = threadIdx.x & 31, vec = q.H / 8;
    const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5),
                  warps = (int64_t)gridDim.x * (kThreads / 32);
    const auto clear = [&](int64_t i) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if (kX) reinterpret_cast<uint4*>(q.x_rows)[i] = zero;
        reinterpret_cast<uint4*>(q.d_rows)[i] = zero;
    };
    for (int64_t t = warp; t < q.T; t += warps) {
        // lane j < k: the padded row of the token's slot j, -1 where it has none
        int64_t mine = -1;
        if (lane < q.k) {
            const int slot = (int)(t * q.k) + lane, p = ld::i32(q.inv_perm + slot);
            if (p >= g.off[0] && p < g.off[q.E] && ld::i32(q.perm + p) == slot)
                mine = padded_row(g, q.E, p) * vec;
        }
        for (int i0 = lane; i0 - lane < vec; i0 += 32 * 4) {
            uint4 a[4], b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 32 * j;
                if (i < vec) {
                    if (kX && q.x_scales)
                        a[j] = widen8(reinterpret_cast<const uint2*>(q.x)[t * vec + i],
                                      scale_of(q.x_scales[t * (q.H / 128) + (i >> 4)]));
                    else if (kX)
                        a[j] = reinterpret_cast<const uint4*>(q.x)[t * vec + i];
                    b[j] = reinterpret_cast<const uint4*>(q.d)[t * vec + i];
                }
            }
            for (int s = 0; s < q.k; ++s) {
                const int64_t to = __shfl_sync(0xffffffffu, mine, s);
                if (to < 0) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = i0 + 32 * j;
                    if (i < vec) {
                        if (kX) reinterpret_cast<uint4*>(q.x_rows)[to + i] = a[j];
                        reinterpret_cast<uint4*>(q.d_rows)[to + i] = b[j];
                    }
                }
            }
        }
    }
    // Positions that no slot holds (a routed index was skipped): zeros, lest what
    // the buffers held reach the weights' gradients of the last group.
    for (int64_t p0 = g.off[0] + warp * 32; p0 < g.off[q.E]; p0 += warps * 32) {
        const int p = (int)p0 + lane;
        bool none = false;
        if (p < g.off[q.E]) {
            const int slot = ld::i32(q.perm + p);
            none = slot < 0 || slot >= q.T * q.k || ld::i32(q.inv_perm + slot) != p;
        }
        for (unsigned left = __ballot_sync(0xffffffffu, none); left; left &= left - 1) {
            const int64_t to = padded_row(g, q.E, (int)p0 + __ffs(left) - 1) * vec;
            for (int i = lane; i < vec; i += 32) clear(to + i);
        }
    }
    // The padding, a row per warp.
    for (int64_t i = warp; i < (int64_t)q.E * 15; i += warps) {
        const int e = (int)(i / 15), c = g.off[e + 1] - g.off[e];
        const int64_t row = (int64_t)g.pad[e] + c + i % 15;
        if (row >= g.pad[e + 1]) continue;
        for (int v = lane; v < vec; v += 32) clear(row * vec + v);
    }
}

// Per token: d_x = the sum of its slots' parts, in order of j, and each slot's
// d_gate = the sum of its parts over the features (a warp per slot: lanes in
// order, then a fixed tree).  The parts of d_x are fp32: rounding them to bf16
// as well would make the rounding error of d_x 1.22 times as large (relative
// RMS 2.9e-3 for 2.4e-3).  16384 x 4096, k = 8: 398 us, 5.7 TB/s.
__global__ void __launch_bounds__(kThreads)
finish_kernel(const float4* y, uint2* d_x, const float* parts, int n_parts, float* d_gates, const int32_t* inv,
              const int32_t* ends, int T, int k, int vec) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t P = (int64_t)T * k;
    // rows outside the groups (bad offsets) have no parts: what the workspace
    // held of an earlier call stays out of the sums
    const int first = ends ? ld::i32(ends) : 0, end = ends ? ld::i32(ends + 1) : (int)P;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        if (d_gates && warp < k) {
            const int64_t s = t * k + warp;
            const int p = inv ? ld::i32(inv + s) : (int)s;
            float sum = 0.f;
            if (p >= first && p < end)
                for (int i = lane; i < n_parts; i += 32) sum += parts[(int64_t)i * P + p];
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) d_gates[s] = sum;
        }
        if (!d_x) continue;
        int64_t src[kMaxK];
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) {
            const int p = j < k ? ld::i32(inv + t * k + j) : -1;
            src[j] = p >= first && p < end ? (int64_t)p * vec : -1;
        }
        for (int v = threadIdx.x; v < vec; v += kThreads) {
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
            d_x[t * vec + v] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                          *reinterpret_cast<const uint32_t*>(&hi));
        }
    }
}

// 65536 x 2048: 63 us, 6.4 TB/s.
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
    return launch_pdl(E <= kThreads ? plan_rows_kernel<1> : plan_rows_kernel<kMostPerThread>, dim3(1), dim3(kThreads), 0, s, offsets, rows, E, most, l, hdr);
}

cudaError_t launch_forward_rows(const __nv_bfloat16* x, const int32_t* perm, int k, int H,
                                const int32_t* offsets, int P, int E, int most, __nv_bfloat16* xs,
                                const RowLists& l, WsHeader* hdr, int num_sms, cudaStream_t s) {
    // (four times the resident blocks: 8192 tokens over 64 experts, forward, 2208 us; once, 2222)
    const int64_t want = ((int64_t)P + 7) / 8;
    return launch_pdl(E <= kThreads ? forward_rows_kernel<1> : forward_rows_kernel<kMostPerThread>, dim3((unsigned)(want < 32 * num_sms ? want : 32 * num_sms)), dim3(kThreads), 0, s,
                      reinterpret_cast<const uint4*>(x), perm, k, H / 8, offsets, P, E, most,
                      reinterpret_cast<uint4*>(xs), l, hdr);
}

cudaError_t launch_backward_rows(const BackwardRows& q, int num_sms, cudaStream_t s) {
    // a block per few tokens: few tokens are spread over blocks of their own
    const int64_t want = q.T < num_sms ? q.T : ((int64_t)q.T + 7) / 8 < num_sms ? num_sms : ((int64_t)q.T + 7) / 8;
    const auto kernel = q.x_rows ? (q.E <= kThreads ? backward_rows_kernel<1, true> : backward_rows_kernel<kMostPerThread, true>)
                                 : (q.E <= kThreads ? backward_rows_kernel<1, false> : backward_rows_kernel<kMostPerThread, false>);
    return launch_pdl(kernel, dim3((unsigned)(want < 8 * num_sms ? want : 8 * num_sms)), dim3(kThreads), 0, s, q);
}

cudaError_t launch_finish(const float* y, __nv_bfloat16* d_x, const float* parts, int n_parts, float* d_gates,
                          const int32_t* inv, const int32_t* ends, int T, int k, int H, int num_sms, cudaStream_t s) {
    const int blocks = T < 8 * num_sms ? T : 8 * num_sms;
    return launch_pdl(finish_kernel, dim3(blocks), dim3(kThreads), 0, s, reinterpret_cast<const float4*>(y),
                      reinterpret_cast<uint2*>(d_x), parts, n_parts, d_gates, inv, ends, T, k, H / 4);
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
