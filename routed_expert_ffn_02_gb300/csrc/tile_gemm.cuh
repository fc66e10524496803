// tile_gemm.cuh -- grouped products on CTA pairs (tcgen05 + TMEM, TMA) with the
// weights' features as the MMA's M and the groups' rows as its N: the training
// passes of the experts and the product with an epilogue.
//
// One work item computes D[m, n] = sum_k A[m, k] B[n, k] for 256 features m
// (128 per CTA of the pair) and up to 2 * NB rows n of one group.  Why rows as
// N: a group's row count is arbitrary, and N is the MMA's flexible size.  A
// group of c rows is cut into ceil(c / 2NB) chunks of nearly equal size, a
// multiple of 16, and each chunk's MMAs run with that N, so the tensor time
// follows the rows; with rows as M each group would fill up to a multiple of
// 256.  Both operands may lie K-major (the reduction dimension contiguous) or
// MN-major, so the same kernel does
//   forward   y  = h Wd^T         A = Wd[f, k]       B = h[row, k]
//   gradient  dh = dy Wd          A = Wd[k, f]       B = dy[row, k]
//   weights   dWd = dy^T h        A = h[k = row, i]  B = dy[k = row, h']
// without a transposed copy of anything.  The accumulator has a feature per
// lane and a row per column, so 32 lanes store 32 consecutive features of a
// row: 64-byte segments straight from registers, for any row stride and any
// row count.
//
// Roles per CTA (persistent, one cluster per SM pair):
//   warp 0      TMA producer (one lane);
//   warp 1      MMA issuer (one lane, even CTA only);
//   warp 2      TMEM allocator;
//   warps 4-11  epilogue, two warps per 32 lanes of the accumulator, taking
//               its 32-column blocks in turn.
// Every mbarrier wait is bounded and drained as in gemm_tc.cu: on expiry a
// role records MOE_ERR_TIMEOUT, both CTAs stop, and copies and MMAs in flight
// are waited for before TMEM is freed.
#pragma once

#include <cuda.h>

#include "fp8.cuh"
#include "moe_internal.cuh"
#include "pair_dev.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "train.cuh"

namespace moe {
namespace tg {

using namespace ptx;
using namespace tc;

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kTileFeatures = 256;   // features per item (both CTAs)

// What an item computes, and what its epilogue does with it.
enum Kind {
    kGated,      // D0 = x Wg^T, D1 = x Wu^T: h = silu(D0) * D1, D0 and D1 kept in bf16
    kGatedFp8,   // the same, D0 and D1 kept in 8 bits
    kRows,       // y = D, bf16 rows
    kHidden,     // D = d Wd: gradients of the two projections, h and d_gates' parts
    kHiddenFp8,  // the same from projections kept in 8 bits
    kInput,      // D = dg Wg + du Wu, bf16 rows
    kWeights,    // the three weight gradients: K runs over the group's rows
    kProduct,    // y = act(D + bias) + residual
};

constexpr bool gated(int kind) { return kind == kGated || kind == kGatedFp8; }
constexpr bool hidden(int kind) { return kind == kHidden || kind == kHiddenFp8; }

template <int kKind, int kNB>
struct Cfg {
    static constexpr bool kAMN = hidden(kKind) || kKind == kInput || kKind == kWeights;
    static constexpr bool kBMN = kKind == kWeights;
    static constexpr int MT = gated(kKind) ? 2 : 1;   // accumulators (A tiles) per item
    static constexpr int NB = kNB;                    // rows of B per CTA
    static constexpr int BN = 2 * NB;                 // most rows per item
    static constexpr int KSUB = MT == 2 ? 1 : 2;      // 64-wide swizzle atoms of K per stage
    static constexpr int BK = 64 * KSUB;
    static constexpr int A_SUB = 128 * BK * 2;        // one A tile
    static constexpr int A_BYTES = MT * A_SUB;
    static constexpr int B_BYTES = NB * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = (200 * 1024) / STAGE_BYTES < 8 ? (200 * 1024) / STAGE_BYTES : 8;
    static constexpr int ACC_COLS = MT * BN;          // TMEM columns of one accumulator set
    static constexpr int BUFS = 2 * ACC_COLS <= 512 ? 2 : 1;
    static constexpr int TMEM_COLS = BUFS * ACC_COLS;
    // block maxima of the 8-bit epilogue: [half][parity][gate, up][4 warps][32 rows]
    static constexpr int AMAX_BYTES = kKind == kGatedFp8 ? 2 * 2 * 2 * 4 * 32 * 4 : 0;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + AMAX_BYTES + 1024 /*align*/ + 512 /*barriers*/;
    static_assert(STAGES >= 2 && SMEM_BYTES <= 227 * 1024);
    static_assert(TMEM_COLS >= 32 && (TMEM_COLS & (TMEM_COLS - 1)) == 0);
};

// Instruction descriptor: tc::make_idesc with the operands' majors.
template <bool kAMN, bool kBMN>
__device__ __forceinline__ uint32_t idesc_for(int n) {
    return (tc::make_idesc(kTileFeatures, 0) | ((uint32_t)(n >> 3) << 17)) | (kAMN ? 1u << 15 : 0u) |
           (kBMN ? 1u << 16 : 0u);
}

// Shared-memory descriptor of an MN-major tile: 64 values of M (or N) in each
// 128-byte row, a row per k, eight rows to a swizzle atom (1024 bytes), the
// next 64 values of M `atom_bytes` on.  Sixteen k are 2048 bytes.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t atom_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(atom_bytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Item w.
struct Item {
    int expert;
    int m0;        // first feature
    int n0;        // weights: first column of B; else 0
    int mat;       // weights: which of the three
    int n;         // MMA N
    int rows;      // rows of the chunk (weights: of the group)
    int row0;      // first row among the sorted rows
    int row0_pad;  // the same in the padded buffers
    int k_blocks;
    int k16_last;  // 16-deep steps of the last block
};

template <int kKind, typename C>
__device__ __forceinline__ Item item_of(const TileArgs& a, int w) {
    Item it;
    it.mat = 0;
    it.n0 = 0;
    if constexpr (kKind == kWeights) {
        const int per_matrix = a.n_mtiles * a.n_ntiles;
        const int g = w / (3 * per_matrix), r = w - g * 3 * per_matrix;
        it.mat = r / per_matrix;
        const int t = r - it.mat * per_matrix;
        // mat 0: d_down, features I, columns H; 1, 2: d_gate, d_up, features H, columns I
        const int mts = it.mat == 0 ? a.n_mtiles : a.n_ntiles;
        it.m0 = (t % mts) * kTileFeatures;
        it.n0 = (t / mts) * C::BN;
        it.n = C::BN;
        it.expert = g;
        if (a.groups) {
            const int4 q = *reinterpret_cast<const int4*>(a.groups + g);
            it.row0 = q.y;
            it.rows = q.z;
            it.row0_pad = q.w;
        } else {
            it.row0 = it.row0_pad = 0;
            it.rows = a.rows;
        }
        it.k_blocks = (it.rows + C::BK - 1) / C::BK;
        it.k16_last = (it.rows - (it.k_blocks - 1) * C::BK + 15) / 16;
    } else {
        const int q = w / a.n_mtiles;
        it.m0 = (w - q * a.n_mtiles) * kTileFeatures;
        if (a.chunks) {
            const int4 c = *reinterpret_cast<const int4*>(a.chunks + q);
            it.expert = c.x;
            it.row0 = c.y;
            it.rows = c.z;
            it.row0_pad = c.w;
        } else {
            it.expert = 0;
            it.row0 = it.row0_pad = q * a.chunk_rows;
            it.rows = min(a.chunk_rows, a.rows - it.row0);
        }
        it.n = (it.rows + 15) & ~15;
        it.k_blocks = a.k_blocks;
        it.k16_last = C::BK / 16;
    }
    return it;
}

// Sums of 32 values per lane over the lanes: lane l gets the sum of v[l].
__device__ __forceinline__ float lane_sums(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

// e4m3 byte -> fp32 (exact).
__device__ __forceinline__ float from_e4m3(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
// 2^(b - 127); byte 255 stands for NaN.
__device__ __forceinline__ float scale_value(uint32_t b) {
    return __uint_as_float(b == 0 ? 1u << 22 : b == 255 ? 0x7fc00000u : b << 23);
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

// ---- epilogues: one 32-column block of one warp ----------------------------
// f: this lane's feature; c0: first column; the columns are rows row0 + c.

template <int kKind>
__device__ __forceinline__ void store_gated(const TileArgs& a, const Item& it, int f, int c0,
                                            int lane, const uint32_t (&g)[32],
                                            const uint32_t (&u)[32], uint32_t* amax, int quad,
                                            int bar_id) {
    const int left = it.rows - c0;                        // valid columns of the block
    const int64_t at = (int64_t)(it.row0 + c0) * a.ld + f;
    __nv_bfloat16* h = a.out + at;
    if constexpr (kKind == kGated) {
        __nv_bfloat16 *kg = static_cast<__nv_bfloat16*>(a.gate) + at,
                      *ku = static_cast<__nv_bfloat16*>(a.up) + at;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            if (c < left) {
                const float gv = __uint_as_float(g[c]), uv = __uint_as_float(u[c]);
                const int64_t o = (int64_t)c * a.ld;
                h[o] = __float2bfloat16_rn(swiglu(gv, uv));
                kg[o] = __float2bfloat16_rn(gv);
                ku[o] = __float2bfloat16_rn(uv);
            }
        }
    } else {
        // The block's scale covers 128 features: the four warps of the CTA's
        // 128 lanes exchange their maxima through shared memory.
        uint32_t mg = 0, mu = 0;                          // of column `lane`
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            const uint32_t bg = __float_as_uint(fp8::finite_abs(__uint_as_float(g[c]))),
                           bu = __float_as_uint(fp8::finite_abs(__uint_as_float(u[c])));
            const uint32_t wg = __reduce_max_sync(0xffffffffu, bg),
                           wu = __reduce_max_sync(0xffffffffu, bu);
            if (lane == c) {
                mg = wg;
                mu = wu;
            }
        }
        amax[quad * 32 + lane] = mg;
        amax[128 + quad * 32 + lane] = mu;
        asm volatile("bar.sync %0, 128;" ::"r"(bar_id) : "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            mg = max(mg, amax[q * 32 + lane]);
            mu = max(mu, amax[128 + q * 32 + lane]);
        }
        const uint32_t sg = fp8::scale_byte(__uint_as_float(mg)),
                       su = fp8::scale_byte(__uint_as_float(mu));
        if (quad == 0 && lane < left) {
            const int64_t s = (int64_t)(it.row0 + c0 + lane) * (a.ld / 128) + (f >> 7);
            a.gate_scales[s] = (uint8_t)sg;
            a.up_scales[s] = (uint8_t)su;
        }
        const float ig = fp8::inverse_scale(sg), iu = fp8::inverse_scale(su);
        uint8_t *kg = static_cast<uint8_t*>(a.gate) + at, *ku = static_cast<uint8_t*>(a.up) + at;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            const float gv = __uint_as_float(g[c]), uv = __uint_as_float(u[c]);
            const float xg = __shfl_sync(0xffffffffu, ig, c), xu = __shfl_sync(0xffffffffu, iu, c);
            if (c < left) {
                const uint32_t p = fp8::pack_e4m3x2(fp8::scaled(gv, xg), fp8::scaled(uv, xu));
                const int64_t o = (int64_t)c * a.ld;
                h[o] = __float2bfloat16_rn(swiglu(gv, uv));
                kg[o] = (uint8_t)(p & 0xffu);
                ku[o] = (uint8_t)(p >> 8);
            }
        }
    }
}

__device__ __forceinline__ void store_rows(const TileArgs& a, const Item& it, int f, int c0,
                                           const uint32_t (&v)[32]) {
    const int left = it.rows - c0;
    __nv_bfloat16* y = a.out + (int64_t)(it.row0 + c0) * a.ld + f;
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (c < left) y[(int64_t)c * a.ld] = __float2bfloat16_rn(__uint_as_float(v[c]));
}

// With q = d Wd (this accumulator), s = sigmoid(g), w the row's gate:
//   h = g s u,  dh = w q,  du = dh g s,  dg = dh u s (1 + g (1 - s)),
//   d_gate = sum_i q_i h_i  (a part of it here: this warp's 32 features).
// dg, du and w h are rounded to bf16, the operands of the next products.
template <int kKind>
__device__ __forceinline__ void store_hidden(const TileArgs& a, const Item& it, int f, int c0,
                                             int lane, const uint32_t (&v)[32]) {
    const int left = it.rows - c0, pad = it.n - c0;
    const int64_t at = (int64_t)(it.row0 + c0) * a.ld + f;
    float g[32], u[32];
    if constexpr (kKind == kHidden) {
        const __nv_bfloat16 *kg = static_cast<const __nv_bfloat16*>(a.gate) + at,
                            *ku = static_cast<const __nv_bfloat16*>(a.up) + at;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            g[c] = c < left ? __bfloat162float(kg[(int64_t)c * a.ld]) : 0.f;
            u[c] = c < left ? __bfloat162float(ku[(int64_t)c * a.ld]) : 0.f;
        }
    } else {
        const uint8_t *kg = static_cast<const uint8_t*>(a.gate) + at,
                      *ku = static_cast<const uint8_t*>(a.up) + at;
        float sg = 0.f, su = 0.f;
        if (lane < left) {
            const int64_t s = (int64_t)(it.row0 + c0 + lane) * (a.ld / 128) + (f >> 7);
            sg = scale_value(a.gate_scales[s]);
            su = scale_value(a.up_scales[s]);
        }
        uint32_t bg[32], bu[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            bg[c] = c < left ? kg[(int64_t)c * a.ld] : 0u;
            bu[c] = c < left ? ku[(int64_t)c * a.ld] : 0u;
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            g[c] = from_e4m3(bg[c]) * __shfl_sync(0xffffffffu, sg, c);
            u[c] = from_e4m3(bu[c]) * __shfl_sync(0xffffffffu, su, c);
        }
    }
    float w = 1.f;
    if (a.gates && lane < left) {
        const int r = it.row0 + c0 + lane, slot = a.perm ? a.perm[r] : r;
        w = slot >= 0 && slot < a.rows ? a.gates[slot] : 0.f;
    }
    const int64_t to = (int64_t)(it.row0_pad + c0) * a.ld + f;
    __nv_bfloat16 *dg = a.d_gate + to, *du = a.d_up + to, *ho = a.out + to;
    float part[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        const float wc = __shfl_sync(0xffffffffu, w, c);
        const float q = __uint_as_float(v[c]), s = sigmoid(g[c]);
        const float gs = g[c] * s, h = gs * u[c], dh = wc * q;
        part[c] = c < left ? q * h : 0.f;
        if (c < pad) {
            const int64_t o = (int64_t)c * a.ld;
            const bool in = c < left;          // rows up to the next multiple of 16 are zero
            dg[o] = __float2bfloat16_rn(in ? dh * u[c] * s * (1.f + g[c] * (1.f - s)) : 0.f);
            du[o] = __float2bfloat16_rn(in ? dh * gs : 0.f);
            ho[o] = __float2bfloat16_rn(in ? wc * h : 0.f);
        }
    }
    if (a.gate_parts) {
        const float sum = lane_sums(part, lane);
        if (lane < left)
            a.gate_parts[(int64_t)(f >> 5) * a.rows + it.row0 + c0 + lane] = sum;
    }
}

__device__ __forceinline__ void store_weights(const TileArgs& a, const Item& it, int f, int c0,
                                              const uint32_t (&v)[32]) {
    const int64_t ld = it.mat == 0 ? a.m_total : a.n_total;      // I, H
    const int64_t rows = it.mat == 0 ? a.n_total : a.m_total;    // H, I
    __nv_bfloat16* W = it.mat == 0 ? a.out : it.mat == 1 ? a.d_gate : a.d_up;
    W += ((int64_t)it.expert * rows + it.n0 + c0) * ld + f;
#pragma unroll
    for (int c = 0; c < 32; ++c) W[(int64_t)c * ld] = __float2bfloat16_rn(__uint_as_float(v[c]));
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case MOE_ACT_RELU: return v < 0.f ? 0.f : v;       // NaN stays
        case MOE_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
        case MOE_ACT_SILU: return v * sigmoid(v);
        default: return v;
    }
}

__device__ __forceinline__ void store_product(const TileArgs& a, const Item& it, int f, int c0,
                                              const uint32_t (&v)[32]) {
    const int left = it.rows - c0;
    if (f >= a.m_total) return;
    const float bias = a.bias ? a.bias[(int64_t)it.expert * a.m_total + f] : 0.f;
    const int64_t at = (int64_t)(it.row0 + c0) * a.ld + f;
    float r[32];
#pragma unroll
    for (int c = 0; c < 32; ++c)
        r[c] = a.residual && c < left ? __bfloat162float(a.residual[at + (int64_t)c * a.ld]) : 0.f;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        if (c < left) {
            const float y = activate(__uint_as_float(v[c]) + bias, a.act) + r[c];
            if (a.out32) a.out32[at + (int64_t)c * a.ld] = y;
            else a.out[at + (int64_t)c * a.ld] = __float2bfloat16_rn(y);
        }
    }
}

// ---- the kernel ------------------------------------------------------------

// Maps: tmA[0..1] / tmB[0..1], meaning by kind:
//   gated     A0 = Wg, A1 = Wu, B0 = x          input    A0 = Wg, A1 = Wu, B0 = dg, B1 = du
//   weights   A0 = w h, A1 = x, B0 = d, B1 = dg, B2 = du        others   A0, B0
struct Maps {
    CUtensorMap a0, a1, b0, b1, b2;
};

template <int kKind, int kNB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
tile_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ TileArgs args) {
    using C = Cfg<kKind, kNB>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    uint32_t* amax_all = reinterpret_cast<uint32_t*>(base_ptr + C::STAGES * C::STAGE_BYTES);
    const uint32_t bars = base + C::STAGES * C::STAGE_BYTES + C::AMAX_BYTES;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
    auto tfull_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + 2 + b); };
    const uint32_t done_bar = bars + 8u * (2 * C::STAGES + 4);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(
        base_ptr + C::STAGES * C::STAGE_BYTES + C::AMAX_BYTES + 8 * (2 * C::STAGES + 5));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* fills_out = reinterpret_cast<int*>(tmem_holder + 2);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t peer_abort = mapa_shared(smem_u32(tmem_holder + 1), rank ^ 1u);
    auto give_up = [&]() {
        *abort_flag = 1;
        st_shared_cluster(peer_abort, 1u);
        set_status(args.hdr, MOE_ERR_TIMEOUT);
    };
    const int cluster = (int)blockIdx.x >> 1;
    const int n_clusters = (int)gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);     // even CTA's producer + both CTAs' bytes
            mbar_init(empty_bar(s), 1);    // the pair's MMA commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kEpiWarps);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        *fills_out = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&maps.a0);
        prefetch_map(&maps.b0);
        if (gated(kKind) || kKind == kInput || kKind == kWeights) prefetch_map(&maps.a1);
        if (kKind == kInput || kKind == kWeights) prefetch_map(&maps.b1);
        if (kKind == kWeights) prefetch_map(&maps.b2);
    }
    if (warp == 2) tmem_alloc_pair(smem_u32(tmem_holder), C::TMEM_COLS);
    fence_before();
    cluster_sync();
    fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_dep_wait();
    grid_dep_launch();

    int total;
    if constexpr (kKind == kWeights) total = args.E * 3 * args.n_mtiles * args.n_ntiles;
    else total = (args.chunks ? *args.n_chunks : args.dense_chunks) * args.n_mtiles;

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        const uint32_t full0 = mapa_shared(full_bar(0), 0);
        int stage = 0;
        uint32_t phase = 0;
        int fills = 0;
        bool ok = true;
        for (int w = cluster; ok && w < total; w += n_clusters) {
            const Item it = item_of<kKind, C>(args, w);
            const int m = it.m0 + (int)rank * 128;
            for (int kb = 0; kb < it.k_blocks; ++kb) {
                if (!mbar_wait_for(empty_bar(stage), phase ^ 1u, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                const uint32_t fb = full0 + 8u * stage;
                if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * C::STAGE_BYTES);
                int k = kb * C::BK;
                const CUtensorMap *ma = &maps.a0, *mb = &maps.b0;
                if constexpr (kKind == kInput) {
                    if (kb >= args.seg_blocks) {      // the second product of the sum
                        k -= args.seg_blocks * C::BK;
                        ma = &maps.a1;
                        mb = &maps.b1;
                    }
                }
                if constexpr (kKind == kWeights) {
                    if (it.mat > 0) ma = &maps.a1;
                    mb = it.mat == 0 ? &maps.b0 : it.mat == 1 ? &maps.b1 : &maps.b2;
                }
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt) {
                    const CUtensorMap* mam = gated(kKind) && mt == 1 ? &maps.a1 : ma;
                    if constexpr (C::kAMN) {
                        const int krow = kKind == kWeights ? it.row0_pad + k
                                                           : it.expert * args.a_rows + k;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d_pair(sa + mt * C::A_SUB + j * C::BK * 128, mam, fb, m + 64 * j, krow);
                    } else {
#pragma unroll
                        for (int j = 0; j < C::KSUB; ++j)
                            tma_load_2d_pair(sa + mt * C::A_SUB + j * 128 * 128, mam, fb, k + 64 * j,
                                             it.expert * args.a_rows + m);
                    }
                }
                if constexpr (C::kBMN) {
#pragma unroll
                    for (int j = 0; j < C::NB / 64; ++j)
                        tma_load_2d_pair(sb + j * C::BK * 128, mb, fb, it.n0 + (int)rank * C::NB + 64 * j,
                                         it.row0_pad + k);
                } else {
                    // the odd CTA holds the upper half of the N rows
                    const int brow = (args.padded ? it.row0_pad : it.row0) + (int)rank * (it.n >> 1);
#pragma unroll
                    for (int j = 0; j < C::KSUB; ++j)
                        tma_load_2d_pair(sb + j * C::NB * 128, mb, fb, k + 64 * j, brow);
                }
                ++fills;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && !*abort_flag) give_up();
        *fills_out = fills;
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---------------- MMA issuer (even CTA) ----------------
        int stage = 0;
        uint32_t phase = 0;
        int i = 0;
        bool ok = true;
        bool issued = false;
        for (int w = cluster; ok && w < total; w += n_clusters, ++i) {
            const Item it = item_of<kKind, C>(args, w);
            const int acc = i % C::BUFS;
            const uint32_t acc_phase = (uint32_t)((i / C::BUFS) & 1);
            if (!mbar_wait_for(tempty_bar(acc), acc_phase ^ 1u, args.wait_cycles, abort_flag)) {
                ok = false;
                break;
            }
            fence_after();
            const uint32_t d_tmem = tmem_base + (uint32_t)(acc * C::ACC_COLS);
            const uint32_t idesc = idesc_for<C::kAMN, C::kBMN>(it.n);
            for (int kb = 0; kb < it.k_blocks; ++kb) {
                if (!mbar_wait_for(full_bar(stage), phase, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                const int steps = kb == it.k_blocks - 1 ? it.k16_last : C::BK / 16;
#pragma unroll
                for (int kk = 0; kk < C::BK / 16; ++kk) {
                    if (kKind == kWeights && kk >= steps) break;
                    uint64_t bd;
                    if constexpr (C::kBMN) bd = mn_desc(sb + kk * 2048, C::BK * 128);
                    else bd = sw128_desc(sb + (kk / 4) * C::NB * 128) + (uint64_t)((kk % 4) * 2);
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        uint64_t ad;
                        if constexpr (C::kAMN) ad = mn_desc(sa + mt * C::A_SUB + kk * 2048, C::BK * 128);
                        else ad = sw128_desc(sa + mt * C::A_SUB + (kk / 4) * 128 * 128) + (uint64_t)((kk % 4) * 2);
                        mma_bf16_pair(d_tmem + (uint32_t)(mt * C::BN), ad, bd, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
                    }
                }
                issued = true;
                commit_pair_multicast(empty_bar(stage), 0x3);
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            commit_pair_multicast(tfull_bar(acc), 0x3);
        }
        if (!ok && !*abort_flag) give_up();
        // Every MMA has completed before TMEM is freed.
        if (issued) {
            commit_pair_multicast(done_bar, 0x1);
            (void)mbar_wait(done_bar, 0);
        }
    } else if (warp >= 4) {
        // ---------------- epilogue (both CTAs) ----------------
        const int quad = warp & 3;            // TMEM lanes 32*quad .. 32*quad+31
        const int half = (warp - 4) >> 2;     // which 32-column blocks
        const uint32_t tempty0 = mapa_shared(tempty_bar(0), 0);
        int i = 0;
        for (int w = cluster; w < total; w += n_clusters, ++i) {
            const Item it = item_of<kKind, C>(args, w);
            const int acc = i % C::BUFS;
            const uint32_t acc_phase = (uint32_t)((i / C::BUFS) & 1);
            bool ok = __all_sync(0xffffffffu, mbar_wait_for(tfull_bar(acc), acc_phase, args.wait_cycles, abort_flag));
            if constexpr (kKind == kGatedFp8) {
                // the four warps that exchange maxima go on together or not at all
                uint32_t all;
                asm volatile(
                    "{\n\t.reg .pred p, q;\n\t"
                    "setp.ne.u32 p, %1, 0;\n\t"
                    "barrier.cta.red.and.pred q, %2, 128, p;\n\t"
                    "selp.u32 %0, 1, 0, q;\n\t}"
                    : "=r"(all)
                    : "r"((uint32_t)ok), "r"(1 + half)
                    : "memory");
                ok = all != 0;
            }
            if (!ok) {
                if (!*abort_flag) give_up();
                break;
            }
            fence_after();
            const int f = it.m0 + (int)rank * 128 + quad * 32 + lane;
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * C::ACC_COLS);
#pragma unroll 1
            for (int c0 = 32 * half; c0 < it.n; c0 += 64) {
                uint32_t v[32];
                if constexpr (gated(kKind)) {
                    uint32_t u[32];
                    tmem_ld32(taddr + c0, v);
                    tmem_ld32(taddr + C::BN + c0, u);
                    tmem_ld_wait();
                    store_gated<kKind>(args, it, f, c0, lane, v, u,
                                       amax_all + half * 512 + ((c0 >> 6) & 1) * 256, quad, 1 + half);
                } else {
                    if (kKind == kWeights && it.rows == 0) {      // a group without rows: zeros
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[c] = 0;
                    } else {
                        tmem_ld32(taddr + c0, v);
                        tmem_ld_wait();
                    }
                    if constexpr (kKind == kRows || kKind == kInput) store_rows(args, it, f, c0, v);
                    else if constexpr (hidden(kKind)) store_hidden<kKind>(args, it, f, c0, lane, v);
                    else if constexpr (kKind == kWeights) store_weights(args, it, f, c0, v);
                    else store_product(args, it, f, c0, v);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_tmem(tempty0 + 8u * acc);
        }
    }

    fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' roles have stopped
    const bool aborted = *abort_flag || ld_shared_cluster(peer_abort) != 0;
    cluster_sync();
    if (aborted) {
        if (rank == 0 && threadIdx.x == 0)
            drain_pair<C::STAGES>(full_bar(0), *fills_out,
                                  (int)ld_shared_cluster(mapa_shared(smem_u32(fills_out), 1)),
                                  (uint32_t)C::STAGE_BYTES);
        cluster_sync();
    }
    if (warp == 2) {
        fence_after();
        tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
}

template <int kKind, int kNB>
cudaError_t launch(const Maps& maps, const TileArgs& args, int num_sms, cudaStream_t s) {
    using C = Cfg<kKind, kNB>;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = smem_limit_once(tile_gemm_kernel<kKind, kNB>, C::SMEM_BYTES, done);
    if (e != cudaSuccess) return e;
    int grid = 0;
    e = pair_grid<tile_gemm_kernel<kKind, kNB>, C::SMEM_BYTES, kThreads>(num_sms, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(tile_gemm_kernel<kKind, kNB>, dim3(grid), dim3(kThreads), C::SMEM_BYTES, s, maps, args);
}

}  // namespace tg
}  // namespace moe
