// balance.cu -- the router's balance loss over packed sequences, its
// per-expert counts, and the gradient of the logits.
//
// With p_t = softmax(logits_t) over all E experts, sequence s holding the
// n_s tokens [off_s, off_s+1), T' = sum_s n_s, and c_se the slots that
// sequence s routes to expert e:
//   f_se = E c_se / (k n_s)      (1 when the slots are spread evenly)
//   P_se = (1/n_s) sum_{t in s} p_te
//   loss = coef * sum_s (n_s / T') sum_e f_se P_se
//        = sum_se a_se sum_{t in s} p_te,   a_se = coef E c_se / (k n_s T').
// Counts carry no gradient, so with d = d_loss
//   d_logits_te = d p_te (a_se - sum_j p_tj a_sj)            (t in s; else 0)
//               + [e = idx_tj] g_tj (dg_tj - sum_i g_ti dg_ti),
// the second line being the gradient of the router's gates (the softmax over
// the selected logits), added when the gates' gradient is given.
//
// Forward: bound by HBM (4 T E bytes read) for large batches, by latency for
// small ones.  One CTA per SM takes a chunk of consecutive tokens, a warp per
// token, the row in registers (16-byte loads); probabilities add up per lane
// over the warp's tokens, then over the CTA's warps in order, then over the
// chunks in order, all fp32: no floating-point atomics, so repeated runs give
// the same bits.  A chunk that several sequences share writes one partial row
// per sequence: chunk c and sequence s meet in row c + s, which no other pair
// of the staircase uses.  A second kernel adds the chunks up, a CTA per 32
// experts and sequence, and its last CTA the loss.  One sequence of at most
// kFusedChunks chunks (128 tokens) does without it: the last CTA of the first
// kernel adds up, which is one CTA's work for so few rows only.
//
// Backward: bound by HBM (4 T E read, 4 T E written).  A warp per token, as
// many consecutive ones as fill the GPU once, so that the coefficients a_se of
// their common sequence stay in registers.
#include <algorithm>

#include "ld_dev.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kFusedChunks = 4;
constexpr int kSlice = 32;           // experts per CTA of the second kernel
constexpr int kFold = 8;             // shared rows that a CTA's warps add into in turn

// Token range of sequence s, inside [0, T]; seq == nullptr: one sequence.
struct SeqRange {
    int beg, end;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* seq, int s, int T) {
    if (!seq) return {0, T};
    const int b = min(max(ld::i32(seq + s), 0), T), e = min(max(ld::i32(seq + s + 1), 0), T);
    return {b, max(b, e)};
}
// The last sequence s in [0, S) with seq[s] <= t (0 if there is none).
__device__ __forceinline__ int seq_of(const int32_t* seq, int S, int t) {
    if (!seq) return 0;
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ld::i32(seq + mid) <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ int tokens_of(const int32_t* seq, int S, int T) {
    if (!seq) return T;
    const int b = min(max(ld::i32(seq), 0), T), e = min(max(ld::i32(seq + S), 0), T);
    return max(e - b, 0);
}
// Whether the offsets descend anywhere; all threads of a block together.  A
// sequence then has no meaning (chunks would meet in one partial row, and rows
// that nobody wrote would be added up), so no token takes part.  Offsets that
// descend or lie outside [0, T] are recorded by the block that `records`.  Every
// block looks for itself: for 1 / 16 / 1024 sequences of 16384 x 384 the forward
// pass takes 13.5 / 14.5 / 44.6 us in a captured graph, 14.5 / 14.3 / 38.2 without;
// handing the first kernel's finding on to the second, 16.6 / 15.0 / 43.
__device__ __forceinline__ bool offsets_descend(const BalanceArgs& a, bool records) {
    if (!a.seq) return false;
    int down = 0;
    for (int64_t s = threadIdx.x; s < a.S; s += blockDim.x) {
        const int b = ld::i32(a.seq + s), e = ld::i32(a.seq + s + 1);
        down |= b > e;
        if (records && (b > e || b < 0 || e > a.T)) set_status(a.hdr, MOE_ERR_BAD_INDEX);
    }
    return __syncthreads_or(down) != 0;
}
// a_se per counted slot: coef E / (k n_s T').
__device__ __forceinline__ float slot_weight(float coef, int E, int k, int n, int total) {
    return n > 0 ? coef * (float)E / ((float)k * (float)n * (float)max(total, 1)) : 0.f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A row of E values in registers: lane l holds values 4 (l + 32 v) + c at
// [4 v + c].  vec: the rows are 16-byte aligned and E a multiple of 4.
template <int V>
__device__ __forceinline__ void load_row(const float* row, int E, bool vec, float fill,
                                         float (&r)[4 * V]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 4 * (lane + 32 * v);
        if (vec) {
            float4 x = make_float4(fill, fill, fill, fill);
            if (e < E) x = ld::f32x4(reinterpret_cast<const float4*>(row + e));
            r[4 * v] = x.x;
            r[4 * v + 1] = x.y;
            r[4 * v + 2] = x.z;
            r[4 * v + 3] = x.w;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) r[4 * v + c] = e + c < E ? ld::f32(row + e + c) : fill;
        }
    }
}
template <int V>
__device__ __forceinline__ void store_row(float* row, int E, bool vec, const float (&r)[4 * V]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 4 * (lane + 32 * v);
        if (vec) {
            if (e < E)
                *reinterpret_cast<float4*>(row + e) =
                    make_float4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (e + c < E) row[e + c] = r[4 * v + c];
        }
    }
}

// Chunks of sequence s and its a_se per counted slot.
struct SeqSum {
    int c0, c1;
    float w;
};
__device__ __forceinline__ SeqSum seq_sum(const BalanceArgs& a, int s, bool none) {
    if (none) return {0, 0, 0.f};
    const SeqRange r = seq_range(a.seq, s, a.T);
    const int n = r.end - r.beg;
    const int c0 = r.beg / a.chunk;
    return {c0, n > 0 ? (r.end - 1) / a.chunk + 1 : c0,
            slot_weight(a.coef, a.E, a.k, n, tokens_of(a.seq, a.S, a.T))};
}

// Partial sums of one chunk: part[c + s][e] = (sum of p, count), and each
// token's (row maximum, 1 / sum of exponentials).  A row of -inf alone has the
// pair (0, 0): no probability anywhere.
template <int V, int W>
__global__ void __launch_bounds__(32 * W)
balance_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
               float2* __restrict__ stats, BalanceArgs a, int fused) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ __align__(16) float sum[kFold][128 * V];
    __shared__ int hist[128 * V];
    __shared__ float red[W];
    __shared__ int last;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x, E = a.E, k = a.k;
    // (T and T k may reach 2^31 - 129: what may pass them by a block is 64-bit)
    const int beg = c * a.chunk, end = a.T - beg < a.chunk ? a.T : beg + a.chunk;
    const bool vec = a.vec;
    const bool none = offsets_descend(a, c == 0);
    for (int s = none ? a.S : seq_of(a.seq, a.S, beg); s < a.S; ++s) {
        const SeqRange r = seq_range(a.seq, s, a.T);
        if (r.beg >= end) break;
        const int t0 = max(beg, r.beg), t1 = min(end, r.end);
        if (t0 >= t1) continue;
        for (int e = threadIdx.x; e < E; e += 32 * W) hist[e] = 0;
        __syncthreads();
        for (int64_t i = (int64_t)t0 * k + threadIdx.x; i < (int64_t)t1 * k; i += 32 * W) {
            const int e = ld::i32(idx + i);
            if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
            else set_status(a.hdr, MOE_ERR_BAD_INDEX);
        }
        float acc[4 * V];
#pragma unroll
        for (int j = 0; j < 4 * V; ++j) acc[j] = 0.f;
        float next[4 * V];
        if (t0 + w < t1) load_row<V>(logits + (int64_t)(t0 + w) * E, E, vec, -INFINITY, next);
        for (int t = t0 + w; t < t1; t += W) {
            float v[4 * V];
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) {
                v[j] = next[j];
                m = fmaxf(m, v[j]);
            }
            if (t + W < t1) load_row<V>(logits + (int64_t)(t + W) * E, E, vec, -INFINITY, next);
            m = warp_max(m);
            if (m == -INFINITY) m = 0.f;
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) {
                v[j] = expf(v[j] - m);
                z += v[j];
            }
            z = warp_sum(z);
            const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) acc[j] = fmaf(v[j], inv, acc[j]);
            if (lane == 0) stats[t] = make_float2(m, inv);
        }
        // warps 0-7 store their sums, 8-15 add theirs, ...
#pragma unroll
        for (int f = 0; f < W / kFold; ++f) {
            if (w / kFold == f) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float4* p = reinterpret_cast<float4*>(&sum[w % kFold][4 * (lane + 32 * v)]);
                    float4 x = f ? *p : make_float4(0.f, 0.f, 0.f, 0.f);
                    x.x += acc[4 * v];
                    x.y += acc[4 * v + 1];
                    x.z += acc[4 * v + 2];
                    x.w += acc[4 * v + 3];
                    *p = x;
                }
            }
            __syncthreads();
        }
        const int64_t out = (int64_t)(c + s) * E;
        for (int e = threadIdx.x; e < E; e += 32 * W) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < kFold; ++i) x += sum[i][e];
            a.part[out + e] = make_float2(x, __int_as_float(hist[e]));
        }
        __syncthreads();
    }
    if (!fused) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last = atomicAdd(&a.hdr->ticket, 1) == (int)gridDim.x - 1;
        if (last) a.hdr->ticket = 0;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // one sequence of at most kFusedChunks chunks
    const SeqSum q = seq_sum(a, 0, none);
    float mine = 0.f;
    for (int e = threadIdx.x; e < E; e += 32 * W) {
        float p = 0.f;
        int n = 0;
        for (int i = q.c0; i < q.c1; ++i) {
            const float2 v = ld::f32x2_cg(a.part + (int64_t)i * E + e);
            p += v.x;
            n += __float_as_int(v.y);
        }
        a.counts[e] = n;
        mine = fmaf(q.w * (float)n, p, mine);
    }
    mine = warp_sum(mine);
    if (lane == 0) red[w] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        float loss = 0.f;
        for (int i = 0; i < W; ++i) loss += red[i];
        *a.loss = loss;
    }
}

// CTA (x, y): kSlice experts (a lane each) of sequences y, y + gridDim.y, ...;
// warp w adds chunks w, w + 8, ..., then the warps' sums are added in order.
// The last CTA adds the slices' shares of the loss.
__global__ void __launch_bounds__(256)
balance_finish_kernel(BalanceArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ float sum[8][kSlice];
    __shared__ int count[8][kSlice];
    __shared__ float red[8];
    __shared__ int last;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int e = blockIdx.x * kSlice + lane;
    const bool none = offsets_descend(a, blockIdx.x == 0 && blockIdx.y == 0);
    float share = 0.f;
    for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
        const SeqSum q = seq_sum(a, s, none);
        float p = 0.f;
        int n = 0;
        if (e < a.E) {
#pragma unroll 8
            for (int c = q.c0 + w; c < q.c1; c += 8) {
                const float2 v = ld::f32x2(a.part + (int64_t)(c + s) * a.E + e);
                p += v.x;
                n += __float_as_int(v.y);
            }
        }
        sum[w][lane] = p;
        count[w][lane] = n;
        __syncthreads();
        if (w == 0) {
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                p += sum[i][lane];
                n += count[i][lane];
            }
            if (e < a.E) a.counts[(int64_t)s * a.E + e] = n;
            share = fmaf(q.w * (float)n, p, share);
        }
        __syncthreads();
    }
    if (w == 0) {
        share = warp_sum(share);
        if (lane == 0) {
            a.shares[blockIdx.y * gridDim.x + blockIdx.x] = share;
            __threadfence();
            const int n = (int)(gridDim.x * gridDim.y);
            last = atomicAdd(&a.hdr->ticket, 1) == n - 1;
            if (last) a.hdr->ticket = 0;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    float loss = 0.f;
    for (int i = threadIdx.x; i < (int)(gridDim.x * gridDim.y); i += 256) loss += ld::f32_cg(a.shares + i);
    loss = warp_sum(loss);
    if (lane == 0) red[w] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        float v = 0.f;
        for (int i = 0; i < 8; ++i) v += red[i];
        *a.loss = v;
    }
}

template <int V>
__global__ void __launch_bounds__(256, V <= 3 ? 3 : 2)
balance_backward_kernel(const float* __restrict__ logits, const float2* __restrict__ stats,
                        const int32_t* __restrict__ counts, const float* __restrict__ d_loss,
                        const int32_t* __restrict__ idx, const float* __restrict__ gates,
                        const float* __restrict__ d_gates, float* __restrict__ d_logits,
                        BalanceArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int E = a.E, k = a.k;
    const bool vec = a.vec;
    const bool none = offsets_descend(a, false);
    const int total = tokens_of(a.seq, a.S, a.T);
    const float up = d_loss ? ld::f32(d_loss) : 1.f;
    const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * a.chunk;
    const int t0 = (int)min(first, (int64_t)a.T), t1 = (int)min(first + a.chunk, (int64_t)a.T);
    int s = -1;
    SeqRange r{0, 0};
    float coef[4 * V];   // d_loss * a_se of the current sequence
    float next[4 * V];   // the next token's row (read also for tokens of no sequence)
    float2 st_next = make_float2(0.f, 0.f);
    auto fetch = [&](int t) {
        load_row<V>(logits + (int64_t)t * E, E, vec, -INFINITY, next);
        st_next = ld::f32x2(stats + t);
    };
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; ++t) {
        if (s < 0 || t >= r.end) {
            s = seq_of(a.seq, a.S, t);
            r = seq_range(a.seq, s, a.T);
            const float w = up * slot_weight(a.coef, E, k, r.end - r.beg, total);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int e = 4 * (lane + 32 * v) + c;
                    coef[4 * v + c] = e < E ? w * (float)ld::i32(counts + (int64_t)s * E + e) : 0.f;
                }
        }
        const bool inside = !none && t >= r.beg && t < r.end;
        float d[4 * V];
        int e_sel = -1;
        float add = 0.f;
        if (idx && lane < k) {
            e_sel = ld::i32(idx + (int64_t)t * k + lane);
            add = ld::f32(gates + (int64_t)t * k + lane);
        }
        const float dg = idx && lane < k ? ld::f32(d_gates + (int64_t)t * k + lane) : 0.f;
        float p[4 * V];
#pragma unroll
        for (int j = 0; j < 4 * V; ++j) p[j] = next[j];
        const float2 st = st_next;
        if (t + 1 < t1) fetch(t + 1);
        if (inside) {
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) {
                p[j] = expf(p[j] - st.x) * st.y;
                dot = fmaf(p[j], coef[j], dot);
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) d[j] = p[j] * (coef[j] - dot);
        } else {
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) d[j] = 0.f;
        }
        if (idx) {
            // Lane j of the first k holds slot j's gradient; value e lives in
            // lane (e / 4) mod 32.  Each pass hands every lane the first of
            // its slots (k slots over 32 lanes: one or two passes).
            add *= dg - warp_sum(add * dg);
            unsigned left = 0;
            for (int i = 0; i < k; ++i) {
                const int e = __shfl_sync(0xffffffffu, e_sel, i);
                if (((e >> 2) & 31) == lane && (unsigned)e < (unsigned)E) left |= 1u << i;
            }
            while (__any_sync(0xffffffffu, left != 0)) {
                const int i = left ? __ffs(left) - 1 : 0;
                const int e = __shfl_sync(0xffffffffu, e_sel, i);
                const float x = __shfl_sync(0xffffffffu, add, i);
                const int at = left ? (e >> 7) * 4 + (e & 3) : -1;
#pragma unroll
                for (int j = 0; j < 4 * V; ++j)
                    if (j == at) d[j] += x;
                left &= left - 1;
            }
        }
        store_row<V>(d_logits + (int64_t)t * E, E, vec, d);
    }
}

bool rows_aligned(const void* p, int E) {
    return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// Calls f.template operator()<V>() for the smallest V with 128 V >= E.
template <typename F>
cudaError_t with_width(int E, F&& f) {
    switch ((E + 127) / 128) {
        case 1: return f.template operator()<1>();
        case 2: return f.template operator()<2>();
        case 3: return f.template operator()<3>();
        case 4: return f.template operator()<4>();
        case 5:
        case 6: return f.template operator()<6>();
        default: return f.template operator()<8>();
    }
}

constexpr int kMaxChunks = 512;   // CTAs of the forward pass
constexpr int kMaxRows = 256;     // CTAs per slice of the second kernel
constexpr int warps_for(int V) { return V <= 3 ? 32 : 16; }   // 64 / 128 registers a thread

}  // namespace

int64_t balance_partial_rows(int T, int S) {
    return std::min<int64_t>(((int64_t)T + 15) / 16, kMaxChunks) + S;
}

int64_t balance_shares(int E, int S) {
    return (int64_t)((E + kSlice - 1) / kSlice) * std::min(S, kMaxRows);
}

cudaError_t launch_balance(const float* logits, const int32_t* idx, float2* stats, BalanceArgs a,
                           int num_sms, cudaStream_t s) {
    bool fused = false;
    a.vec = rows_aligned(logits, a.E);
    a.chunk = 16;
    cudaError_t e = cudaSuccess;
    if (a.T > 0) {
        e = with_width(a.E, [&]<int V>() {
            constexpr int W = warps_for(V);
            const int most = std::min(num_sms, kMaxChunks);
            a.chunk = std::max(W, (int)(((int64_t)a.T + most - 1) / most));
            const int chunks = (int)(((int64_t)a.T + a.chunk - 1) / a.chunk);
            fused = a.S == 1 && chunks <= kFusedChunks;
            return launch_pdl(balance_kernel<V, W>, dim3(chunks), dim3(32 * W), 0, s, logits, idx,
                              stats, a, (int)fused);
        });
    }
    if (e != cudaSuccess || fused) return e;
    return launch_pdl(balance_finish_kernel,
                      dim3((a.E + kSlice - 1) / kSlice, std::min(a.S, kMaxRows)), dim3(256), 0, s, a);
}

cudaError_t launch_balance_backward(const float* logits, const float2* stats, const float* d_loss,
                                    const int32_t* idx, const float* gates, const float* d_gates,
                                    float* d_logits, BalanceArgs a, int num_sms, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    a.vec = rows_aligned(logits, a.E) && rows_aligned(d_logits, a.E);
    const int warps = num_sms * (a.E <= 384 ? 24 : 16);   // resident at once
    a.chunk = (int)(((int64_t)a.T + warps - 1) / warps);
    const int64_t per_block = 8 * (int64_t)a.chunk;
    return with_width(a.E, [&]<int V>() {
        return launch_pdl(balance_backward_kernel<V>, dim3((unsigned)((a.T + per_block - 1) / per_block)),
                          dim3(256), 0, s, logits, stats, (const int32_t*)a.counts, d_loss, idx,
                          gates, d_gates, d_logits, a);
    });
}

}  // namespace moe
