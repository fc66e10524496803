// fp8_prologue.cu -- what precedes the expert kernels of a small batch on
// 8-bit experts, in one launch: routing, route lists, the planner's tile list
// and the quantised rows (at most kThinMaxTokens tokens, so every touched
// expert is a thin tile).
//
// Latency bounds it: a decode token needs 4 E bytes of logits and 2 H of x.
// As separate kernels (router, route lists and planner in one CTA, row
// quantiser) the three take 4.7 + 9.6 + 4.2 us; here one CTA per token
// quantises its own row while its warps route the whole batch, a token each, so every CTA
// knows its slots' sorted positions without waiting for another one (CTA 0
// stores the lists).  The results are those of the separate kernels: the same
// top-k routine, the stable order of the slots (position = number of slots
// with a smaller (expert, slot) key), the same quantiser.
#include <algorithm>

#include "fp8.cuh"
#include "ld_dev.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"
#include "quantize_dev.cuh"
#include "small_plan.cuh"

namespace moe {
namespace {

constexpr int kMinThreads = 256;                           // up to 1024: a warp per token
constexpr int kMaxSlots = kThinMaxTokens * kMaxK;          // 256: a thread per slot
constexpr int kRowVecs = kMaxHidden / 16 / kMinThreads;    // 16-value vectors per thread
static_assert(kMaxSlots <= kMinThreads, "a thread per slot");

__global__ void __launch_bounds__(1024)
fp8_prologue_kernel(const float* __restrict__ logits, const uint4* __restrict__ x, int T, int E,
                    int k, int per_row, int32_t* __restrict__ idx_out,
                    float* __restrict__ gates_out, int32_t* __restrict__ inv_perm,
                    FatTile* __restrict__ thin_tiles, WsHeader* hdr, uint4* __restrict__ xq,
                    uint8_t* __restrict__ xs) {
    __shared__ int32_t idx[kMaxSlots];
    __shared__ float gates[kMaxSlots];
    __shared__ __align__(16) uint32_t keys[kMaxSlots];
    __shared__ int32_t sorted[kMaxSlots];
    __shared__ int32_t pos_of[kMaxSlots];
    __shared__ int heads_before[kMaxSlots / 32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int t = blockIdx.x, tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int P = T * k;

    // this token's row, quantised in registers (per_row is a multiple of 8,
    // so the eight lanes of a block take part together)
    uint4 q[kRowVecs];
    uint32_t sb[kRowVecs];
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i) {
        const int v = tid + i * threads;
        if (v < per_row) {
            const uint4* src = x + 2 * ((int64_t)t * per_row + v);
            q[i] = fp8::quantize_lane16({ld::u32x4(src), ld::u32x4(src + 1)}, &sb[i]);
        }
    }
    for (int r = warp; r < T; r += threads / 32)
        route_token(logits + (int64_t)r * E, E, k, idx + r * k, gates + r * k);
    __syncthreads();
    uint32_t key = 0xffffffffu;
    if (tid < P) key = ((uint32_t)idx[tid] << 8) | (uint32_t)tid;   // distinct: (expert, slot)
    if (tid < kMaxSlots) keys[tid] = key;
    __syncthreads();
    if (tid < P) {
        int pos = 0;
        const uint4* k4 = reinterpret_cast<const uint4*>(keys);   // unused keys are the largest
        for (int j = 0; j < (P + 3) / 4; ++j) {
            const uint4 o = k4[j];
            pos += (o.x < key) + (o.y < key) + (o.z < key) + (o.w < key);
        }
        pos_of[tid] = pos;
        sorted[pos] = idx[tid];
    }
    __syncthreads();
    // the row to its k positions
    for (int j = 0; j < k; ++j) {
        const int64_t p = pos_of[t * k + j];
#pragma unroll
        for (int i = 0; i < kRowVecs; ++i) {
            const int v = tid + i * threads;
            if (v < per_row) {
                xq[p * per_row + v] = q[i];
                if ((tid & 7) == 0) xs[(p * per_row + v) >> 3] = (uint8_t)sb[i];
            }
        }
    }
    if (t != 0 || tid >= kMaxSlots) return;   // whole warps
    // CTA 0: routing, inverse permutation, and a thin tile per touched expert
    // in ascending order (thread p: sorted position p)
    const bool live = tid < P;
    const bool head = live && (tid == 0 || sorted[tid - 1] != sorted[tid]);
    const unsigned heads = __ballot_sync(0xffffffffu, head);
    if (lane == 0) heads_before[warp] = __popc(heads);
    asm volatile("bar.sync 1, %0;" ::"n"(kMaxSlots) : "memory");   // the first 256 threads
    int tile = __popc(heads & ((1u << lane) - 1u)), total = 0;
#pragma unroll
    for (int w = 0; w < kMaxSlots / 32; ++w) {
        if (w < warp) tile += heads_before[w];
        total += heads_before[w];
    }
    if (live) {
        idx_out[tid] = idx[tid];
        gates_out[tid] = gates[tid];
        inv_perm[tid] = pos_of[tid];
    }
    if (head) {
        int n = 1;
        while (tid + n < P && sorted[tid + n] == sorted[tid]) ++n;
        thin_tiles[tile] = FatTile{sorted[tid], tid, n, 0};
    }
    if (tid == 0) {
        hdr->n_fat_tiles = 0;
        hdr->n_solo = 0;
        hdr->n_thin_mma = total;
    }
}

}  // namespace

bool fp8_prologue_fits(int T) { return T <= kThinMaxTokens; }

cudaError_t launch_fp8_prologue(const float* logits, const __nv_bfloat16* x, int T, int E, int k,
                                int H, int32_t* idx, float* gates, int32_t* inv_perm,
                                FatTile* thin_tiles, WsHeader* hdr, uint8_t* xq, uint8_t* xs,
                                cudaStream_t s) {
    return launch_pdl(fp8_prologue_kernel, dim3(T), dim3(std::max(kMinThreads, 32 * T)), 0, s, logits,
                      reinterpret_cast<const uint4*>(x), T, E, k, H / 16, idx, gates, inv_perm,
                      thin_tiles, hdr, reinterpret_cast<uint4*>(xq), xs);
}

}  // namespace moe
