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
// Forward: a CTA takes kBalanceChunk tokens, a warp per token, the row in
// registers; probabilities add up per lane over the warp's tokens, then over
// the CTA's warps in order, then (second kernel) over the chunks in order, all
// fp32: no floating-point atomics, so repeated runs give the same bits.  A
// chunk that several sequences share writes one partial row per sequence:
// chunk c and sequence s meet in row c + s, which no other pair of the
// staircase uses.
#include <algorithm>

#include "moe_internal.cuh"
#include "ptx.cuh"
#include "route_dev.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;

// Token range of sequence s, inside [0, T]; seq == nullptr: one sequence.
struct SeqRange {
    int beg, end;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* seq, int s, int T) {
    if (!seq) return {0, T};
    const int b = min(max(__ldg(seq + s), 0), T), e = min(max(__ldg(seq + s + 1), 0), T);
    return {b, max(b, e)};
}
// The last sequence s in [0, S) with seq[s] <= t (0 if there is none).
__device__ __forceinline__ int seq_of(const int32_t* seq, int S, int t) {
    if (!seq) return 0;
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(seq + mid) <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ int tokens_of(const int32_t* seq, int S, int T) {
    if (!seq) return T;
    const int b = min(max(__ldg(seq), 0), T), e = min(max(__ldg(seq + S), 0), T);
    return max(e - b, 0);
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

// Partial sums of one chunk: part_p[c + s][e], part_c[c + s][e], and each
// token's (row maximum, 1 / sum of exponentials).  A row of -inf alone has
// the pair (0, 0): no probability anywhere.
template <int EPL>
__global__ void __launch_bounds__(32 * kWarps)
balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx, int T,
                       int E, int k, const int32_t* __restrict__ seq, int S,
                       float2* __restrict__ stats, float* __restrict__ part_p,
                       int32_t* __restrict__ part_c, WsHeader* hdr) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ float sum[kWarps][kMaxE];
    __shared__ int hist[kMaxE];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x;
    const int beg = c * kBalanceChunk, end = min(T, beg + kBalanceChunk);
    for (int s = seq_of(seq, S, beg); s < S; ++s) {
        const SeqRange r = seq_range(seq, s, T);
        if (r.beg >= end) break;
        const int t0 = max(beg, r.beg), t1 = min(end, r.end);
        if (t0 >= t1) continue;
        for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
        for (int i = t0 * k + threadIdx.x; i < t1 * k; i += blockDim.x) {
            const int e = __ldg(idx + i);
            if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
            else set_status(hdr, MOE_ERR_BAD_INDEX);
        }
        float acc[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
        for (int t = t0 + w; t < t1; t += kWarps) {
            const float* row = logits + (int64_t)t * E;
            float v[EPL];
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane + 32 * j;
                v[j] = e < E ? __ldg(row + e) : -INFINITY;
                m = fmaxf(m, v[j]);
            }
            m = warp_max(m);
            if (m == -INFINITY) m = 0.f;
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                v[j] = expf(v[j] - m);
                z += v[j];
            }
            z = warp_sum(z);
            const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] = fmaf(v[j], inv, acc[j]);
            if (lane == 0) stats[t] = make_float2(m, inv);
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane + 32 * j < E) sum[w][lane + 32 * j] = acc[j];
        __syncthreads();
        const int64_t out = (int64_t)(c + s) * E;
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) a += sum[i][e];
            part_p[out + e] = a;
            part_c[out + e] = hist[e];
        }
        __syncthreads();
    }
}

// One CTA per sequence: counts and the sequence's share of the loss; the last
// CTA adds the shares in order.
__global__ void __launch_bounds__(256)
balance_finish_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int T,
                      int E, int k, const int32_t* __restrict__ seq, int S, float coef,
                      int32_t* __restrict__ counts, float* seq_loss, float* loss, WsHeader* hdr) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ float red[8];
    __shared__ int last;
    const int s = blockIdx.x;
    const SeqRange r = seq_range(seq, s, T);
    const int n = r.end - r.beg;
    const int c0 = r.beg / kBalanceChunk, c1 = n > 0 ? (r.end - 1) / kBalanceChunk + 1 : c0;
    const float total = (float)max(tokens_of(seq, S, T), 1);
    const float scale = n > 0 ? coef * (float)E / ((float)k * (float)n * total) : 0.f;
    float mine = 0.f;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        float p = 0.f;
        int q = 0;
        for (int c = c0; c < c1; ++c) {
            p += part_p[(int64_t)(c + s) * E + e];
            q += part_c[(int64_t)(c + s) * E + e];
        }
        counts[(int64_t)s * E + e] = q;
        mine = fmaf(scale * (float)q, p, mine);
    }
    mine = warp_sum(mine);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        float a = 0.f;
        for (int i = 0; i < 8; ++i) a += red[i];
        seq_loss[s] = a;
        __threadfence();
        last = atomicAdd(&hdr->ticket, 1) == S - 1;
        if (last) hdr->ticket = 0;
    }
    __syncthreads();
    if (!last || threadIdx.x >= 32) return;
    __threadfence();
    float a = 0.f;
    for (int i = threadIdx.x; i < S; i += 32) a += __ldcg(seq_loss + i);
    a = warp_sum(a);
    if (threadIdx.x == 0) *loss = a;
}

template <int EPL>
__global__ void __launch_bounds__(32 * kWarps)
balance_backward_kernel(const float* __restrict__ logits, const float2* __restrict__ stats,
                        const int32_t* __restrict__ counts, const int32_t* __restrict__ seq, int T,
                        int E, int k, int S, float coef, const float* __restrict__ d_loss,
                        const int32_t* __restrict__ idx, const float* __restrict__ gates,
                        const float* __restrict__ d_gates, float* __restrict__ d_logits) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const float total = (float)max(tokens_of(seq, S, T), 1);
    const float up = d_loss ? __ldg(d_loss) : 1.f;
    for (int t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < T; t += gridDim.x * kWarps) {
        const int s = seq_of(seq, S, t);
        const SeqRange r = seq_range(seq, s, T);
        const bool inside = t >= r.beg && t < r.end;
        const float a0 = inside ? coef * (float)E / ((float)k * (float)(r.end - r.beg) * total) : 0.f;
        float d[EPL];
        if (inside) {
            const float* row = logits + (int64_t)t * E;
            const int32_t* cnt = counts + (int64_t)s * E;
            const float2 st = __ldg(stats + t);
            float p[EPL];
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane + 32 * j;
                p[j] = e < E ? expf(__ldg(row + e) - st.x) * st.y : 0.f;
                d[j] = e < E ? a0 * (float)__ldg(cnt + e) : 0.f;
                dot = fmaf(p[j], d[j], dot);
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int j = 0; j < EPL; ++j) d[j] = up * p[j] * (d[j] - dot);
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) d[j] = 0.f;
        }
        if (idx) {
            const float g = lane < k ? __ldg(gates + (int64_t)t * k + lane) : 0.f;
            const float dg = lane < k ? __ldg(d_gates + (int64_t)t * k + lane) : 0.f;
            const int e = lane < k ? __ldg(idx + (int64_t)t * k + lane) : -1;
            const float add = g * (dg - warp_sum(g * dg));
            for (int i = 0; i < k; ++i) {
                const int ei = __shfl_sync(0xffffffffu, e, i);
                const float ai = __shfl_sync(0xffffffffu, add, i);
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (ei == lane + 32 * j) d[j] += ai;
            }
        }
        float* out = d_logits + (int64_t)t * E;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane + 32 * j < E) out[lane + 32 * j] = d[j];
    }
}

}  // namespace

int64_t balance_partial_rows(int T, int S) {
    return ((int64_t)T + kBalanceChunk - 1) / kBalanceChunk + S;
}

cudaError_t launch_balance(const float* logits, const int32_t* idx, int T, int E, int k,
                           const int32_t* seq, int S, float coef, float* loss, int32_t* counts,
                           float2* stats, float* part_p, int32_t* part_c, float* seq_loss,
                           WsHeader* hdr, cudaStream_t s) {
    const int chunks = (T + kBalanceChunk - 1) / kBalanceChunk;
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(chunks), dim3(32 * kWarps), 0, s, logits, idx, T, E, k, seq,
                          S, stats, part_p, part_c, hdr);
    };
    if (chunks > 0) {
        switch (routing::candidates_per_lane(E)) {
            case 1: e = go(balance_partial_kernel<1>); break;
            case 2: e = go(balance_partial_kernel<2>); break;
            case 4: e = go(balance_partial_kernel<4>); break;
            case 8: e = go(balance_partial_kernel<8>); break;
            case 12: e = go(balance_partial_kernel<12>); break;
            case 16: e = go(balance_partial_kernel<16>); break;
            case 24: e = go(balance_partial_kernel<24>); break;
            default: e = go(balance_partial_kernel<32>); break;
        }
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(balance_finish_kernel, dim3(S), dim3(256), 0, s, (const float*)part_p,
                      (const int32_t*)part_c, T, E, k, seq, S, coef, counts, seq_loss, loss, hdr);
}

cudaError_t launch_balance_backward(const float* logits, const float2* stats,
                                    const int32_t* counts, const int32_t* seq, int T, int E, int k,
                                    int S, float coef, const float* d_loss, const int32_t* idx,
                                    const float* gates, const float* d_gates, float* d_logits,
                                    int num_sms, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    const int blocks = (int)std::min<int64_t>((T + kWarps - 1) / kWarps, (int64_t)num_sms * 16);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(blocks), dim3(32 * kWarps), 0, s, logits, stats, counts, seq,
                          T, E, k, S, coef, d_loss, idx, gates, d_gates, d_logits);
    };
    switch (routing::candidates_per_lane(E)) {
        case 1: return go(balance_backward_kernel<1>);
        case 2: return go(balance_backward_kernel<2>);
        case 4: return go(balance_backward_kernel<4>);
        case 8: return go(balance_backward_kernel<8>);
        case 12: return go(balance_backward_kernel<12>);
        case 16: return go(balance_backward_kernel<16>);
        case 24: return go(balance_backward_kernel<24>);
        default: return go(balance_backward_kernel<32>);
    }
}

}  // namespace moe
