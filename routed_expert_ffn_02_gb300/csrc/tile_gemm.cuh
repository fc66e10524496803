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
// lane and a row per column; an epilogue warp turns 32 x 32 values around
// through shared memory (see "fragments and staging tiles").
//
// Three stages of 128 of K (64 KB per CTA), two accumulators in TMEM.  The gated
// products of the forward pass have two accumulators per item (gate and up share
// the rows' tile): with chunks of 256 rows these fill TMEM, and the epilogue is
// not hidden under the next item.
//
// What bounds it (GB300, 1.9 GHz unless the power cap is reached): an item of
// K = 4096 takes 19.3 us at N = 256 with its operands in L2 (17.9 for the MMAs
// alone, 13.8 for the copies alone), 15.8 at N = 176 and 13.2 at any N up to 128
// (the MMA's floor of about 100 cycles).  Shared memory carries 128 bytes a
// cycle then: half of it the MMA's operands, half the copies that bring them.
// Long runs of N = 256 reach 1.36 kW, the power cap, at 1.55-1.75 GHz: 1.6-1.7
// PFLOP/s, as the library's products do (measured 1.69 sustained).  Halving the
// copies of B (an experiment; multicast between pairs would save as much) gained
// 2-5%, fetching weights into L2 ahead cost 2-30%.
//
// Roles per CTA (persistent, one cluster per SM pair):
//   warp 0      TMA producer (one lane);
//   warp 1      MMA issuer (one lane, even CTA only);
//   warp 2      TMEM allocator;
//   warps 4-11  epilogue, two warps per 32 lanes of the accumulator, taking
//               its 32-column blocks in turn.
// Every mbarrier wait is bounded and drained as in gemm_tc.cu: on expiry a
// role records MOE_ERR_TIMEOUT, the cluster's CTAs stop, and copies and MMAs in
// flight are waited for before TMEM is freed.
#pragma once

#include <cuda.h>
#include <algorithm>

#include "act_dev.cuh"
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
constexpr int kEpiWarps = 8;         // 16 took 15% longer (16384 x 4096 results of K = 128)
constexpr int kTileFeatures = 256;   // features per item (both CTAs)
constexpr int kTileBytes = 32 * 64;  // a staging tile

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

// kSplit pairs of a cluster share an item: each takes a part of K, and the
// first adds the others' accumulators, which they store into its shared memory.
template <int kKind, int kNB, int kSplit = 1>
struct Cfg {
    static_assert(kSplit == 1 || (kKind == kProduct && kNB == 16));
    static constexpr int CTAS = 2 * kSplit;           // of a cluster
    // the other pairs' parts: [pair - 1][4 warps][32 values][32 lanes]
    static constexpr int PARTS_BYTES = (kSplit - 1) * 4 * 32 * 32 * 4;
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
    // what B's rows, and the K rows of a weight gradient's last block, are rounded up to
    static constexpr int BOX = NB < 32 ? NB : 32;
    static constexpr int STAGES =
        (192 * 1024 - PARTS_BYTES) / STAGE_BYTES < 8 ? (192 * 1024 - PARTS_BYTES) / STAGE_BYTES : 8;
    static constexpr int ACC_COLS = MT * BN;          // TMEM columns of one accumulator set
    static constexpr int BUFS = 2 * ACC_COLS <= 512 ? 2 : 1;
    static constexpr int TMEM_COLS = BUFS * ACC_COLS;
    // staging tiles of an epilogue warp (32 rows x 32 features, bf16; two hold
    // a tile of fp32)
    static constexpr int TILES = kKind == kGatedFp8 ? 1 : 2;
    static constexpr int STAGING_BYTES = kEpiWarps * TILES * kTileBytes;
    // block maxima of the 8-bit epilogue: [half][parity][gate, up][4 warps][32 rows]
    static constexpr int AMAX_BYTES = kKind == kGatedFp8 ? 2 * 2 * 2 * 4 * 32 * 4 : 0;
    static constexpr int SMEM_BYTES =
        STAGES * STAGE_BYTES + STAGING_BYTES + AMAX_BYTES + PARTS_BYTES + 1024 /*align*/ + 512 /*barriers*/;
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
    int k16_last;  // 16-deep steps of the last block (of whole K)
    int boxes;     // B's rows of one CTA, in boxes of BOX
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
        it.k16_last = kKind == kProduct ? a.k16_last : C::BK / 16;
        it.boxes = (it.n / 2 + C::BOX - 1) / C::BOX;
    }
    return it;
}

// Tensor maps, by kind:
//   gated     a0 = Wg, a1 = Wu, b[0] = x; o0 = h, o1 = gate, o2 = up
//   hidden    a0 = Wd, b[0] = d; o0 = w h, o1 = dg, o2 = du
//   input     a0 = Wg, a1 = Wu, b[0] = dg, b[1] = du; o0 = d_x
//   weights   a0 = w h, a1 = x, b = d, dg, du; o0 = dWd, o1 = dWg, o2 = dWu
//   others    a0 = W, b[0] = x; o0 = y
// Operands are seen as strips of 64 columns (make_tma_map_strips), so that one
// copy loads a stage's tile of A or of B: the producer's copies, about 110
// cycles each to issue, bounded every item with fewer than 256 rows when a
// stage took 8 (K = 4096: 17.6 us for any N from 96 to 192).  b[..][i] holds
// boxes of 32 (i + 1) rows, for chunks of so many rows (a CTA's half, rounded
// up); weights: [0] 32 and [3] 128 rows of K, of a and b.  flat_a and, as b[0],
// b[1]: 64-column boxes, zero beyond the last column, for a product's last block
// where K does not fill it (two copies a strip).
struct Maps {
    CUtensorMap a0, a1, tail_a0, tail_a1;
    CUtensorMap b[3][4];
    CUtensorMap flat_a;
    CUtensorMap o0, o1, o2;
};

// 2^(b - 127); byte 255 stands for NaN.
__device__ __forceinline__ float scale_value(uint32_t b) {
    return __uint_as_float(b == 0 ? 1u << 22 : b == 255 ? 0x7fc00000u : b << 23);
}
__device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// tma_load_2d_pair for a 3-D map.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// ---- fragments and staging tiles --------------------------------------------
//
// An epilogue warp takes 32 features x 32 rows at a time.  It reads them from
// TMEM in the layout of 8 x 8 matrix fragments: lane t holds, for feature
// 8 i + t / 4 and row 8 j + 2 (t mod 4) + s, value [i][j][s].  Rounded to bf16
// and packed by s, a fragment is what stmatrix/ldmatrix with .trans exchange
// with a shared tile of 32 rows x 32 features: 4 instructions instead of 32
// two-byte accesses.  From the tile, four lanes copy a row's 64 bytes to or
// from global memory in 16-byte vectors.  16-byte chunk c of row r lies at
// chunk c ^ (r / 2 mod 4) of the row, so that neither side meets bank
// conflicts.  (Loading the residual of a 16384 x 4096 x 4096 product two bytes
// per lane, 64 bytes per instruction, took 280 us more than its 295.)
struct Frag {
    float v[4][4][2];
};
struct Packed {
    uint32_t v[4][4];
};

__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&r)[2][4][2]) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q >> 1][j][q & 1] = __uint_as_float(v[4 * j + q]);
}
// 32 lanes x 32 columns at taddr; complete after tmem_ld_wait().
__device__ __forceinline__ void load_frag(uint32_t taddr, Frag& f) {
    tmem_ld_frag(taddr, *reinterpret_cast<float(*)[2][4][2]>(&f.v[0]));
    tmem_ld_frag(taddr + (16u << 16), *reinterpret_cast<float(*)[2][4][2]>(&f.v[2]));
}

__device__ __forceinline__ Packed pack(const Frag& f) {
    Packed p;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) p.v[i][j] = pack_bf16(f.v[i][j][0], f.v[i][j][1]);
    return p;
}

__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int row, int chunk) {
    return tile + (uint32_t)row * 64u + (uint32_t)((chunk ^ (row >> 1)) & 3) * 16u;
}
__device__ __forceinline__ void frag_to_tile(uint32_t tile, const Packed& p, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         tile_at(tile, 8 * j + (lane & 7), lane >> 3)),
                     "r"(p.v[0][j]), "r"(p.v[1][j]), "r"(p.v[2][j]), "r"(p.v[3][j])
                     : "memory");
}
__device__ __forceinline__ void tile_to_frag(uint32_t tile, Packed& p, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(p.v[0][j]), "=r"(p.v[1][j]), "=r"(p.v[2][j]), "=r"(p.v[3][j])
                     : "r"(tile_at(tile, 8 * j + (lane & 7), lane >> 3))
                     : "memory");
}
__device__ __forceinline__ uint4 tile_vec(uint32_t tile, int row, int chunk) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(tile_at(tile, row, chunk))
                 : "memory");
    return v;
}
__device__ __forceinline__ void tile_put(uint32_t tile, int row, int chunk, const uint4& v) {
    st_shared_v4(tile_at(tile, row, chunk), v.x, v.y, v.z, v.w);
}

// An epilogue warp's place and its ring of staging tiles.
struct Warp {
    int lane, quad;
    uint32_t tiles;       // its staging tiles
    int used;             // tiles handed out
    uint32_t* amax;       // 8-bit epilogue: this block's maxima [gate, up][4 warps][32 rows]
    int bar_id;
};
// The next tile of the ring, no longer read by the store that used it before.
// Every use ends with a commit, so the groups in flight count the tiles in use.
template <int kTiles>
__device__ __forceinline__ uint32_t next_tile(Warp& w) {
    if (w.lane == 0) bulk_wait_read<kTiles - 1>();
    __syncwarp();
    return w.tiles + (uint32_t)(w.used++ % kTiles) * kTileBytes;
}

// Where 32 x 32 blocks of an output go: a map for whole blocks, which the copy
// engine stores from the tile, and the address for a group's last rows, stored
// in 16-byte vectors by the warp (whole blocks stored that way take the same
// time with four loads and stores more each).
struct OutBlock {
    const CUtensorMap* map;
    int x, y;                  // column and row of the block
    __nv_bfloat16* p;          // the same as an address, rows of ld values
    int64_t ld;
    int rows;                  // rows of the block that are there
};
// Packed fragment -> output.
template <int kTiles>
__device__ __forceinline__ void store_packed(Warp& w, const Packed& p, const OutBlock& o) {
    const uint32_t tile = next_tile<kTiles>(w);
    frag_to_tile(tile, p, w.lane);
    if (o.rows >= 32) {
        fence_proxy_async_shared();
        __syncwarp();
        if (w.lane == 0) tma_store_2d(o.map, tile, o.x, o.y);
    } else {
        __syncwarp();
        __nv_bfloat16* to = o.p + (int64_t)(w.lane >> 2) * o.ld + (w.lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (w.lane >> 2);
            const uint4 v = tile_vec(tile, row, w.lane & 3);
            if (row < o.rows) *reinterpret_cast<uint4*>(to) = v;
            to += 8 * o.ld;
        }
    }
    if (w.lane == 0) bulk_commit();
}

// Rows of a bf16 tensor on their way into a tile: loaded ahead, put later.
struct RowVecs {
    uint4 v[4];
};
__device__ __forceinline__ void load_rows(RowVecs& r, const __nv_bfloat16* in, int64_t ld, int left,
                                          int lane) {
    const __nv_bfloat16* p = in + (int64_t)(lane >> 2) * ld + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[i] = make_uint4(0, 0, 0, 0);
        if (8 * i + (lane >> 2) < left) r.v[i] = *reinterpret_cast<const uint4*>(p);
        p += 8 * ld;
    }
}
__device__ __forceinline__ void put_rows(uint32_t tile, const RowVecs& r, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tile_put(tile, 8 * i + (lane >> 2), lane & 3, r.v[i]);
}
// The same for rows of e4m3 with a scale per 128 features (two lanes a row).
struct RowBytes {
    uint4 v[2];
    uint32_t scale;      // of rows lane / 2 and 16 + lane / 2, a byte each
};
__device__ __forceinline__ void load_rows(RowBytes& r, const uint8_t* in, const uint8_t* scales,
                                          int64_t ld, int left, int lane) {
    r.scale = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 16 * i + (lane >> 1);
        r.v[i] = make_uint4(0, 0, 0, 0);
        if (row < left) {
            r.v[i] = *reinterpret_cast<const uint4*>(in + (int64_t)row * ld + (lane & 1) * 16);
            r.scale |= (uint32_t)scales[(int64_t)row * (ld / 128)] << (8 * i);
        }
    }
}
__device__ __forceinline__ void put_rows(uint32_t tile, const RowBytes& r, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float s = scale_value((r.scale >> (8 * i)) & 0xffu);
        const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[q >> 1] >> (16 * (q & 1)))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            o[q] = pack_bf16(f.x * s, f.y * s);
        }
        const int row = 16 * i + (lane >> 1), c = (lane & 1) * 2;
        tile_put(tile, row, c, make_uint4(o[0], o[1], o[2], o[3]));
        tile_put(tile, row, c + 1, make_uint4(o[4], o[5], o[6], o[7]));
    }
}

// Sums over the 32 features of one value per row: v[j][s] are this lane's
// sums of row 8 j + 2 (t mod 4) + s.  Each lane gets the sum of one row, whose
// number is returned in *row.
__device__ __forceinline__ float feature_sums(float (&v)[4][2], int lane, int* row) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i >> 1][i & 1];
#pragma unroll
    for (int o = 16, n = 4; o >= 4; o >>= 1, n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? w[i + n] : w[i], send = up ? w[i] : w[i + n];
            w[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    // lane bit 4 chose the upper half of j, bit 3 the lower bit of j, bit 2 s
    *row = ((lane >> 4) & 1) * 16 + ((lane >> 3) & 1) * 8 + (lane & 3) * 2 + ((lane >> 2) & 1);
    return w[0];
}

// ---- epilogues: one warp's 32 features from f0, 32 rows from c0 ---------------

// Largest magnitudes (as integers, which order them alike) of row c0 + lane of
// the two projections over the CTA's 128 features: each lane takes its
// features', the eight lanes of a row theirs, and the four warps exchange
// theirs through shared memory.  NaN does not count, nor, with kFinite, do
// infinities.
template <bool kFinite>
__device__ __forceinline__ void block_maxima(const Frag& g, const Frag& u, const Warp& w, uint32_t* mg, uint32_t* mu) {
    const int lane = w.lane;
    uint32_t m[2][8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a = fmaxf(a, kFinite ? fp8::finite_abs(g.v[i][j][s]) : fabsf(g.v[i][j][s]));
                b = fmaxf(b, kFinite ? fp8::finite_abs(u.v[i][j][s]) : fabsf(u.v[i][j][s]));
            }
            m[0][2 * j + s] = __float_as_uint(a);
            m[1][2 * j + s] = __float_as_uint(b);
        }
#pragma unroll
    for (int o = 16, n = 4; o >= 4; o >>= 1, n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const uint32_t keep = up ? m[z][i + n] : m[z][i], send = up ? m[z][i] : m[z][i + n];
                m[z][i] = max(keep, __shfl_xor_sync(0xffffffffu, send, o));
            }
    }
    const int row = ((lane >> 4) & 1) * 16 + ((lane >> 3) & 1) * 8 + (lane & 3) * 2 + ((lane >> 2) & 1);
    if (kFinite) asm volatile("bar.sync %0, 128;" ::"r"(w.bar_id) : "memory");   // the first exchange has been read
    w.amax[w.quad * 32 + row] = m[0][0];
    w.amax[128 + w.quad * 32 + row] = m[1][0];
    asm volatile("bar.sync %0, 128;" ::"r"(w.bar_id) : "memory");
    *mg = *mu = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        *mg = max(*mg, w.amax[q * 32 + lane]);
        *mu = max(*mu, w.amax[128 + q * 32 + lane]);
    }
}

// h = silu(g) u, with g and u kept.
template <int kKind>
__device__ __forceinline__ void store_gated(const TileArgs& a, const Item& it, int f0, int c0,
                                            const Frag& g, const Frag& u, const Maps& maps, Warp& w) {
    const int left = it.rows - c0, lane = w.lane;
    const int64_t at = (int64_t)(it.row0 + c0) * a.ld + f0;
    constexpr int kTiles = kKind == kGated ? 2 : 1;
    const auto out = [&](const CUtensorMap& m, void* p) {
        return OutBlock{&m, f0, it.row0 + c0, static_cast<__nv_bfloat16*>(p) + at, a.ld, left};
    };
    Packed h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h.v[i][j] = pack_bf16(g.v[i][j][0] * sigmoid(g.v[i][j][0]) * u.v[i][j][0],
                                  g.v[i][j][1] * sigmoid(g.v[i][j][1]) * u.v[i][j][1]);
    if constexpr (kKind == kGated) {
        store_packed<kTiles>(w, h, out(maps.o0, a.out));
        store_packed<kTiles>(w, pack(g), out(maps.o1, a.gate));
        store_packed<kTiles>(w, pack(u), out(maps.o2, a.up));
    } else {
        // a block's scale covers 128 features
        uint32_t mg, mu;                                  // of row c0 + lane
        block_maxima<false>(g, u, w, &mg, &mu);
        // an infinity among them: the maxima of the finite values (rare; the
        // four warps see the same maxima, so they go this way together)
        const bool infinite = __any_sync(0xffffffffu, max(mg, mu) == 0x7f800000u);
        if (infinite) block_maxima<true>(g, u, w, &mg, &mu);
        const uint32_t sg = fp8::scale_byte(__uint_as_float(mg)),
                       su = fp8::scale_byte(__uint_as_float(mu));
        if (w.quad == 0 && lane < left) {
            const int64_t s = (int64_t)(it.row0 + c0 + lane) * (a.ld / 128) + (f0 >> 7);
            a.gate_scales[s] = (uint8_t)sg;
            a.up_scales[s] = (uint8_t)su;
        }
        const float ig = fp8::inverse_scale(sg), iu = fp8::inverse_scale(su);
        Packed q;      // per value a byte of the gate and one of the up projection
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t b[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int r = 8 * j + 2 * (lane & 3) + s;
                const float xg = __shfl_sync(0xffffffffu, ig, r), xu = __shfl_sync(0xffffffffu, iu, r);
                // (the conversion keeps NaN and would saturate infinities)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[s][i] = infinite ? fp8::pack_e4m3x2(fp8::scaled(g.v[i][j][s], xg), fp8::scaled(u.v[i][j][s], xu))
                                       : fp8::pack_e4m3x2(g.v[i][j][s] * xg, u.v[i][j][s] * xu);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) q.v[i][j] = b[0][i] | b[1][i] << 16;
        }
        store_packed<kTiles>(w, h, out(maps.o0, a.out));
        const uint32_t tile = next_tile<kTiles>(w);
        frag_to_tile(tile, q, lane);
        __syncwarp();
        // two lanes a row, 16 features each: the gate's bytes and the up's
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 16 * i + (lane >> 1), c = (lane & 1) * 2;
            const uint4 lo = tile_vec(tile, r, c), hi = tile_vec(tile, r, c + 1);
            if (r < left) {
                const int64_t to = at + (int64_t)r * a.ld + c * 8;
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.gate) + to) =
                    make_uint4(__byte_perm(lo.x, lo.y, 0x6420), __byte_perm(lo.z, lo.w, 0x6420),
                               __byte_perm(hi.x, hi.y, 0x6420), __byte_perm(hi.z, hi.w, 0x6420));
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.up) + to) =
                    make_uint4(__byte_perm(lo.x, lo.y, 0x7531), __byte_perm(lo.z, lo.w, 0x7531),
                               __byte_perm(hi.x, hi.y, 0x7531), __byte_perm(hi.z, hi.w, 0x7531));
            }
        }
        if (lane == 0) bulk_commit();
    }
}

// fp32 block: through a tile of 128-byte rows (16-byte chunk c of row r at
// chunk c ^ (r mod 8)) where whole rows can be stored by the copy engine, else
// straight from the fragment, eight lanes storing 32 bytes of a row.
__device__ __forceinline__ void store_f32(Warp& w, const Frag& f, const CUtensorMap* map, int x, int y, float* out,
                                          int64_t ld, int left, int feats) {
    const int lane = w.lane;
    if (map && left >= 32) {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int r = 8 * j + 2 * (lane & 3) + s, c = 2 * i + (lane >> 4);
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(w.tiles + r * 128 + ((c ^ r) & 7) * 16 + ((lane >> 2) & 3) * 4),
                                 "f"(f.v[i][j][s])
                                 : "memory");
                }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, w.tiles, x, y);
            bulk_commit();
            bulk_commit();      // two tiles of the ring
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = 8 * j + 2 * (lane & 3) + s;
            float* o = out + (int64_t)r * ld + (lane >> 2);
            if (r < left) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (8 * i + (lane >> 2) < feats) o[8 * i] = f.v[i][j][s];
            }
        }
}

// What a hidden block reads, loaded a block ahead.
template <int kKind>
struct KeptRows {
    RowVecs g, u;
    float w;            // the gate of row c0 + lane
};
template <>
struct KeptRows<kHiddenFp8> {
    RowBytes g, u;
    float w;
};
template <int kKind>
__device__ __forceinline__ void load_kept(KeptRows<kKind>& k, const TileArgs& a, const Item& it, int f0,
                                          int c0, int lane) {
    const int left = it.rows - c0;
    const int64_t at = (int64_t)(it.row0 + c0) * a.ld + f0;
    k.w = 1.f;
    if (a.gates && lane < left) {
        const int r = it.row0 + c0 + lane, slot = a.perm ? a.perm[r] : r;
        k.w = slot >= 0 && slot < a.rows ? a.gates[slot] : 0.f;
    }
    if constexpr (kKind == kHidden) {
        load_rows(k.g, static_cast<const __nv_bfloat16*>(a.gate) + at, a.ld, left, lane);
        load_rows(k.u, static_cast<const __nv_bfloat16*>(a.up) + at, a.ld, left, lane);
    } else if constexpr (kKind == kHiddenFp8) {
        const int64_t s = (int64_t)(it.row0 + c0) * (a.ld / 128) + (f0 >> 7);
        load_rows(k.g, static_cast<const uint8_t*>(a.gate) + at, a.gate_scales + s, a.ld, left, lane);
        load_rows(k.u, static_cast<const uint8_t*>(a.up) + at, a.up_scales + s, a.ld, left, lane);
    }
}

// With q = d Wd (this accumulator), s = sigmoid(g), w the row's gate:
//   h = g s u,  dh = w q,  du = dh g s,  dg = dh u (s + g s (1 - s)),
//   d_gate = sum_i q_i h_i  (a part of it here: this warp's 32 features).
// dg, du and w h are rounded to bf16, the operands of the next products.
template <int kKind>
__device__ __forceinline__ void store_hidden(const TileArgs& a, const Item& it, int f0, int c0,
                                             Frag& q, const Packed& kg, const Packed& ku, float w,
                                             const Maps& maps, Warp& wp) {
    const int left = it.rows - c0, pad = it.n - c0, lane = wp.lane;
    if (left < 32) {       // rows up to the next multiple of 16 become zero (g and u are already)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (8 * j + 2 * (lane & 3) + s >= left)
#pragma unroll
                    for (int i = 0; i < 4; ++i) q.v[i][j][s] = 0.f;
    }
    Packed dg, du, ho;
    float part[4][2] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float wr[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) wr[s] = __shfl_sync(0xffffffffu, w, 8 * j + 2 * (lane & 3) + s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 g2 = unpack(kg.v[i][j]), u2 = unpack(ku.v[i][j]);
            float og[2], ou[2], oh[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float g = s ? g2.y : g2.x, u = s ? u2.y : u2.x, qv = q.v[i][j][s];
                const float sg = sigmoid(g), gs = g * sg, h = gs * u, dh = wr[s] * qv;
                part[j][s] = fmaf(qv, h, part[j][s]);
                og[s] = dh * u * fmaf(gs, 1.f - sg, sg);
                ou[s] = dh * gs;
                oh[s] = wr[s] * h;
            }
            dg.v[i][j] = pack_bf16(og[0], og[1]);
            du.v[i][j] = pack_bf16(ou[0], ou[1]);
            ho.v[i][j] = pack_bf16(oh[0], oh[1]);
        }
    }
    const int64_t to = (int64_t)(it.row0_pad + c0) * a.ld + f0;
    const auto out = [&](const CUtensorMap& m, __nv_bfloat16* p) {
        return OutBlock{&m, f0, it.row0_pad + c0, p + to, a.ld, pad};
    };
    store_packed<2>(wp, dg, out(maps.o1, a.d_gate));
    store_packed<2>(wp, du, out(maps.o2, a.d_up));
    store_packed<2>(wp, ho, out(maps.o0, a.out));
    if (a.gate_parts) {
        int r;
        const float sum = feature_sums(part, lane, &r);
        if (r < left) a.gate_parts[(int64_t)(f0 >> 5) * a.rows + it.row0 + c0 + r] = sum;
    }
}

// 64 rows of a weight gradient from c0 (always whole), in one copy out of both
// staging tiles: half the fences, barriers and copies of 32-row blocks.
__device__ __forceinline__ void store_weights(const TileArgs& a, const Item& it, int f0, int c0,
                                              const Packed& lo, const Packed& hi, const Maps& maps, Warp& w) {
    if (w.lane == 0) bulk_wait_read<0>();
    __syncwarp();
    frag_to_tile(w.tiles, lo, w.lane);
    frag_to_tile(w.tiles + kTileBytes, hi, w.lane);
    fence_proxy_async_shared();
    __syncwarp();
    if (w.lane == 0) {
        const int rows = it.mat == 0 ? a.n_total : a.m_total;    // of an expert's matrix: H, I
        tma_store_2d(it.mat == 0 ? &maps.o0 : it.mat == 1 ? &maps.o1 : &maps.o2, w.tiles, f0,
                     it.expert * rows + it.n0 + c0);
        bulk_commit();
    }
}

__device__ __forceinline__ void activate(Frag& f, int act) {
    float* v = &f.v[0][0][0];
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];       // NaN stays
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) gelu2(v[i], v[i + 1]);
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= sigmoid(v[i]);
    }
}

// What a product block adds, loaded a block ahead: its residual in vectors
// where rows are 16-byte aligned (a.vec), else a feature per lane and a row per
// word (packing them here would wait for the loads).
union Residual {
    RowVecs vecs;
    uint32_t words[32];
};
__device__ __forceinline__ void load_residual(Residual& r, const TileArgs& a, const Item& it, int f0,
                                              int c0, int lane) {
    const int64_t at = (int64_t)(it.row0 + c0) * a.ld + f0;
    if (a.vec) {
        load_rows(r.vecs, a.residual + at, a.ld, f0 + (lane & 3) * 8 < a.m_total ? it.rows - c0 : 0, lane);
        return;
    }
    const int left = f0 + lane < a.m_total ? it.rows - c0 : 0;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.residual + at) + lane;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        r.words[i] = 0;
        if (i < left) r.words[i] = *p;
        p += a.ld;
    }
}
__device__ __forceinline__ void store_product(const TileArgs& a, const Item& it, int f0, int c0, Frag& v,
                                              const Residual& res, const Maps& maps, Warp& w) {
    const int left = it.rows - c0, lane = w.lane, feats = a.m_total - f0;
    const int64_t at = (int64_t)(it.row0 + c0) * a.ld + f0;
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = 8 * i + (lane >> 2);
            const float b = f < feats ? a.bias[(int64_t)it.expert * a.m_total + f0 + f] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v.v[i][j][0] += b;
                v.v[i][j][1] += b;
            }
        }
    }
    activate(v, a.act);
    if (a.residual) {
        const uint32_t tile = next_tile<2>(w);
        if (a.vec) {
            put_rows(tile, res.vecs, lane);
        } else {
#pragma unroll
            for (int r = 0; r < 32; ++r)
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(tile_at(tile, r, lane >> 3) + (lane & 7) * 2),
                             "h"((uint16_t)res.words[r])
                             : "memory");
        }
        __syncwarp();
        Packed p;
        tile_to_frag(tile, p, lane);
        if (lane == 0) bulk_commit();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = unpack(p.v[i][j]);
                v.v[i][j][0] += x.x;
                v.v[i][j][1] += x.y;
            }
    }
    if (a.out32) {
        store_f32(w, v, a.map_out ? &maps.o0 : nullptr, f0, it.row0 + c0, a.out32 + at, a.ld, left, feats);
        return;
    }
    if (a.map_out) {
        const int rows = left >= 32 ? 32 : (lane & 3) * 8 < feats ? left : 0;
        store_packed<2>(w, pack(v), OutBlock{&maps.o0, f0, it.row0 + c0, a.out + at, a.ld, rows});
        return;
    }
    const uint32_t tile = next_tile<2>(w);
    frag_to_tile(tile, pack(v), lane);
    __syncwarp();
    uint16_t x[32];      // all loads before the first store
#pragma unroll
    for (int r = 0; r < 32; ++r)
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x[r]) : "r"(tile_at(tile, r, lane >> 3) + (lane & 7) * 2) : "memory");
    uint16_t* to = reinterpret_cast<uint16_t*>(a.out + at) + lane;
    const int rows = lane < feats ? left : 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        if (r < rows) *to = x[r];
        to += a.ld;
    }
    if (lane == 0) bulk_commit();
}

// ---- the kernel ------------------------------------------------------------

// Waits for what is in flight after an abort, as drain_pair does; here a
// stage's bytes differ from item to item: bytes(cta, s) of CTA 0 or 1's last
// fill of stage s.
template <int kStages, typename Bytes>
__device__ __forceinline__ void drain_stages(uint32_t full0, int fills_even, int fills_odd, Bytes bytes) {
    for (int s = 0; s < kStages; ++s) {
        const uint32_t bar = full0 + 8u * s;
        const int re = rounds_filled<kStages>(fills_even, s) - 1, ro = rounds_filled<kStages>(fills_odd, s) - 1;
        if (re < 0 && ro < 0) continue;
        if (ro == re + 1) {
            if (re >= 0) (void)mbar_wait(bar, (uint32_t)(re & 1));
            mbar_expect_tx(bar, bytes(1, s));
            (void)mbar_wait(bar, (uint32_t)(ro & 1));
        } else if (re == ro + 1) {
            mbar_complete_tx(bar, bytes(0, s));
            (void)mbar_wait(bar, (uint32_t)(re & 1));
        } else {
            (void)mbar_wait(bar, (uint32_t)(re & 1));
        }
    }
}

template <int kKind, int kNB, int kSplit>
__global__ void __cluster_dims__(2 * kSplit, 1, 1) __launch_bounds__(kThreads, 1)
tile_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ TileArgs args) {
    using C = Cfg<kKind, kNB, kSplit>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    constexpr int kStagingAt = C::STAGES * C::STAGE_BYTES, kAmaxAt = kStagingAt + C::STAGING_BYTES,
                  kPartsAt = kAmaxAt + C::AMAX_BYTES, kBarsAt = kPartsAt + C::PARTS_BYTES;
    const uint32_t bars = base + kBarsAt;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
    auto tfull_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + 2 + b); };
    const uint32_t done_bar = bars + 8u * (2 * C::STAGES + 4);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + kBarsAt + 8 * (2 * C::STAGES + 5));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* fills_out = reinterpret_cast<int*>(tmem_holder + 2);
    uint32_t* stage_bytes = tmem_holder + 3;     // of each stage's last fill

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank();
    const uint32_t rank = cta & 1u, even = cta & ~1u;      // the CTA's place in its pair; the pair's even CTA
    const int part = (int)(cta >> 1);                      // the pair's part of K
    auto give_up = [&]() {
        for (uint32_t c = 0; c < C::CTAS; ++c) st_shared_cluster(mapa_shared(smem_u32(tmem_holder + 1), c), 1u);
        *abort_flag = 1;
        set_status(args.hdr, MOE_ERR_TIMEOUT);
    };
    const int cluster = (int)blockIdx.x / C::CTAS;
    const int n_clusters = (int)gridDim.x / C::CTAS;
    const uint16_t pair_mask = (uint16_t)(0x3u << even);

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
        if (kKind != kProduct || args.flat_from > 0) {     // else there are only flat maps
            prefetch_map(&maps.a0);
            prefetch_map(&maps.b[0][C::NB / C::BOX - 1]);
        }
        if (gated(kKind) || kKind == kInput || kKind == kWeights) prefetch_map(&maps.a1);
        if (kKind == kInput || kKind == kWeights) prefetch_map(&maps.b[1][C::NB / C::BOX - 1]);
        if (kKind == kWeights) prefetch_map(&maps.b[2][C::NB / C::BOX - 1]);
    }
    if (warp == 2) tmem_alloc_pair(smem_u32(tmem_holder), C::TMEM_COLS);
    fence_before();
    cluster_sync();
    fence_after();
    const uint32_t tmem_base = *tmem_holder;
    if (!args.early) grid_dep_wait();
    grid_dep_launch();

    int total;
    if constexpr (kKind == kWeights) total = args.E * 3 * args.n_mtiles * args.n_ntiles;
    else total = (args.chunks ? *args.n_chunks : args.dense_chunks) * args.n_mtiles;

    [[maybe_unused]] Frag mine;          // split items: this warp's accumulator
    [[maybe_unused]] bool have = false;

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        const uint32_t full0 = mapa_shared(full_bar(0), even);
        int stage = 0;
        uint32_t phase = 0;
        int fills = 0;
        bool ok = true;
        for (int w = cluster; ok && w < total; w += n_clusters) {
            const Item it = item_of<kKind, C>(args, w);
            const int m = it.m0 + (int)rank * 128;
            for (int kb = part * it.k_blocks / kSplit; kb < (part + 1) * it.k_blocks / kSplit; ++kb) {
                if (!mbar_wait_for(empty_bar(stage), phase ^ 1u, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                const uint32_t fb = full0 + 8u * stage;
                int k = kb * C::BK;
                if constexpr (kKind == kWeights) {
                    // K runs over the group's rows: the last block loads the boxes that hold some
                    const int krow = it.row0_pad + k, n = it.n0 + (int)rank * C::NB;
                    const bool tail = kb == it.k_blocks - 1 && it.k16_last <= (C::BK - 32) / 16;
                    const int boxes = tail ? (it.k16_last + 1) / 2 : 1;
                    const uint32_t bytes = tail ? (uint32_t)boxes * (32 * 128 * 4) : (uint32_t)C::STAGE_BYTES;
                    stage_bytes[stage] = bytes;
                    if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * bytes);
                    if (!tail) {
                        tma_load_3d_pair(sa, it.mat ? &maps.a1 : &maps.a0, fb, 0, krow, m / 64);
                        tma_load_3d_pair(sb, &maps.b[it.mat][3], fb, 0, krow, n / 64);
                    } else {
                        // (in 64-wide strips of 32 rows each, where the whole block's are)
                        for (int q = 0; q < boxes; ++q)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t to = j * C::BK * 128 + q * 32 * 128;
                                tma_load_3d_pair(sa + to, it.mat ? &maps.tail_a1 : &maps.tail_a0, fb, 0, krow + 32 * q, m / 64 + j);
                                tma_load_3d_pair(sb + to, &maps.b[it.mat][0], fb, 0, krow + 32 * q, n / 64 + j);
                            }
                    }
                } else {
                    // B: the rows of the chunk, rounded up to a box, no more; of a product's
                    // last block, the strips of K that there are
                    const bool flat = kKind == kProduct && kb >= args.flat_from;
                    const int strips = flat ? args.flat_strips : C::KSUB;
                    const uint32_t bytes = (uint32_t)((C::A_BYTES / C::KSUB + it.boxes * C::BOX * 128) * strips);
                    stage_bytes[stage] = bytes;
                    if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * bytes);
                    const CUtensorMap *ma = &maps.a0, *mb = &maps.b[0][it.boxes - 1];
                    if constexpr (kKind == kInput) {
                        if (kb >= args.seg_blocks) {      // the second product of the sum
                            k -= args.seg_blocks * C::BK;
                            ma = &maps.a1;
                            mb = &maps.b[1][it.boxes - 1];
                        }
                    }
                    // the odd CTA holds the upper half of the N rows
                    const int brow = (args.padded ? it.row0_pad : it.row0) + (int)rank * (it.n >> 1);
                    if (flat) {
                        for (int j = 0; j < strips; ++j) {
                            tma_load_2d_pair(sa + j * 128 * 128, &maps.flat_a, fb, k + 64 * j, it.expert * args.a_rows + m);
                            tma_load_2d_pair(sb + j * it.boxes * C::BOX * 128, &maps.b[1][it.boxes - 1], fb, k + 64 * j, brow);
                        }
                    } else {
#pragma unroll
                        for (int mt = 0; mt < C::MT; ++mt) {
                            const CUtensorMap* mam = gated(kKind) && mt == 1 ? &maps.a1 : ma;
                            if constexpr (C::kAMN)
                                tma_load_3d_pair(sa + mt * C::A_SUB, mam, fb, 0, it.expert * args.a_rows + k, m / 64);
                            else
                                tma_load_3d_pair(sa + mt * C::A_SUB, mam, fb, 0, it.expert * args.a_rows + m, k / 64);
                        }
                        tma_load_3d_pair(sb, mb, fb, 0, brow, k / 64);
                    }
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
            [[maybe_unused]] const uint32_t b_strip = (uint32_t)(it.boxes * C::BOX * 128);
            const int kb0 = part * it.k_blocks / kSplit;
            for (int kb = kb0; kb < (part + 1) * it.k_blocks / kSplit; ++kb) {
                if (!mbar_wait_for(full_bar(stage), phase, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                const auto step = [&](int kk) {
                    uint64_t bd;
                    if constexpr (C::kBMN) bd = mn_desc(sb + kk * 2048, C::BK * 128);
                    else bd = sw128_desc(sb + (kk / 4) * b_strip) + (uint64_t)((kk % 4) * 2);
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        uint64_t ad;
                        if constexpr (C::kAMN) ad = mn_desc(sa + mt * C::A_SUB + kk * 2048, C::BK * 128);
                        else ad = sw128_desc(sa + mt * C::A_SUB + (kk / 4) * 128 * 128) + (uint64_t)((kk % 4) * 2);
                        mma_bf16_pair(d_tmem + (uint32_t)(mt * C::BN), ad, bd, idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
                    }
                };
                if ((kKind == kWeights || kKind == kProduct) && kb == it.k_blocks - 1 && it.k16_last < C::BK / 16) {
#pragma unroll 1
                    for (int kk = 0; kk < it.k16_last; ++kk) step(kk);
                } else {
#pragma unroll
                    for (int kk = 0; kk < C::BK / 16; ++kk) step(kk);
                }
                issued = true;
                commit_pair_multicast(empty_bar(stage), pair_mask);
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            commit_pair_multicast(tfull_bar(acc), pair_mask);
        }
        if (!ok && !*abort_flag) give_up();
        // Every MMA has completed before TMEM is freed.
        if (issued) {
            commit_pair_multicast(done_bar, (uint16_t)(1u << cta));
            (void)mbar_wait(done_bar, 0);
        }
    } else if (warp >= 4) {
        // ---------------- epilogue (both CTAs) ----------------
        const int quad = warp & 3;            // TMEM lanes 32*quad .. 32*quad+31
        const int half = (warp - 4) >> 2;     // which 32-row blocks: every other
        uint32_t* amax = reinterpret_cast<uint32_t*>(base_ptr + kAmaxAt) + half * 512;
        Warp wp = {lane, quad, base + kStagingAt + (uint32_t)(warp - 4) * C::TILES * kTileBytes, 0, amax, 1 + half};
        const uint32_t tempty0 = mapa_shared(tempty_bar(0), even);
        int i = 0;
        for (int w = cluster; w < total; w += n_clusters, ++i) {
            const Item it = item_of<kKind, C>(args, w);
            const int acc = i % C::BUFS;
            const uint32_t acc_phase = (uint32_t)((i / C::BUFS) & 1);
            const int f0 = it.m0 + (int)rank * 128 + quad * 32;
            const bool live = kKind != kProduct || f0 < args.m_total;
            // what the first block reads does not wait for the products
            [[maybe_unused]] KeptRows<kKind> kept;
            [[maybe_unused]] Residual res;
            if constexpr (hidden(kKind)) load_kept<kKind>(kept, args, it, f0, 32 * half, lane);
            if constexpr (kKind == kProduct)
                if (kSplit == 1 && live && args.residual) load_residual(res, args, it, f0, 32 * half, lane);
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
                    : "r"((uint32_t)ok), "r"(wp.bar_id)
                    : "memory");
                ok = all != 0;
            }
            if (!ok) {
                if (!*abort_flag) give_up();
                break;
            }
            fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * C::ACC_COLS);
            const int n = live ? it.n : 0;
            if constexpr (kSplit > 1) {
                // at most 32 rows and one item: the first pair waits for the others' parts below
                if (half == 0) {
                    load_frag(taddr, mine);
                    tmem_ld_wait();
                    have = true;
                    if (part > 0) {
                        const uint32_t to = mapa_shared(base + kPartsAt + (uint32_t)((part - 1) * 4 + quad) * 4096u, rank);
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            st_shared_cluster(to + (uint32_t)(q * 32 + lane) * 4u, __float_as_uint((&mine.v[0][0][0])[q]));
                    }
                }
            } else if constexpr (kKind == kWeights) {
#pragma unroll 1
                for (int c0 = 64 * half; c0 < n; c0 += 128) {
                    Packed lo = {}, hi = {};
                    if (it.rows > 0) {                 // a group without rows: zeros
                        Frag v, u;
                        load_frag(taddr + c0, v);
                        load_frag(taddr + c0 + 32, u);
                        tmem_ld_wait();
                        lo = pack(v);
                        hi = pack(u);
                    }
                    store_weights(args, it, f0, c0, lo, hi, maps, wp);
                }
            } else
#pragma unroll 1
            for (int c0 = 32 * half; c0 < n; c0 += 64) {
                Frag v;
                if constexpr (gated(kKind)) {
                    Frag u;
                    load_frag(taddr + c0, v);
                    load_frag(taddr + C::BN + c0, u);
                    tmem_ld_wait();
                    wp.amax = amax + ((c0 >> 6) & 1) * 256;
                    store_gated<kKind>(args, it, f0, c0, v, u, maps, wp);
                } else if constexpr (hidden(kKind)) {
                    load_frag(taddr + c0, v);
                    Packed g, u;
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                    put_rows(wp.tiles, kept.g, lane);
                    put_rows(wp.tiles + kTileBytes, kept.u, lane);
                    __syncwarp();
                    tile_to_frag(wp.tiles, g, lane);
                    tile_to_frag(wp.tiles + kTileBytes, u, lane);
                    const float gate = kept.w;
                    if (c0 + 64 < n) load_kept<kKind>(kept, args, it, f0, c0 + 64, lane);
                    tmem_ld_wait();
                    store_hidden<kKind>(args, it, f0, c0, v, g, u, gate, maps, wp);
                } else {
                    load_frag(taddr + c0, v);
                    tmem_ld_wait();
                    if constexpr (kKind == kProduct) {
                        const Residual now = res;
                        if (args.residual && c0 + 64 < n)
                            load_residual(res, args, it, f0, c0 + 64, lane);
                        store_product(args, it, f0, c0, v, now, maps, wp);
                    } else {
                        const int64_t at = (int64_t)(it.row0 + c0) * args.ld + f0;
                        if (kKind == kInput && args.out32)        // a slot's part of the sum
                            store_f32(wp, v, &maps.o0, f0, it.row0 + c0, args.out32 + at, args.ld, it.rows - c0, 32);
                        else
                            store_packed<2>(wp, pack(v), OutBlock{&maps.o0, f0, it.row0 + c0, args.out + at, args.ld, it.rows - c0});
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_tmem(tempty0 + 8u * acc);
        }
        if (lane == 0) bulk_wait_all();   // the stores have completed before the CTA leaves
        __syncwarp();
    }

    fence_before();
    __syncthreads();
    cluster_sync();   // all CTAs' roles have stopped, and the parts of a split item are in place
    bool aborted = *abort_flag != 0;
    for (uint32_t c = 0; c < C::CTAS; ++c)
        aborted |= ld_shared_cluster(mapa_shared(smem_u32(tmem_holder + 1), c)) != 0;
    cluster_sync();
    if (aborted) {
        if (rank == 0 && threadIdx.x == 0)
            drain_stages<C::STAGES>(full_bar(0), *fills_out,
                                    (int)ld_shared_cluster(mapa_shared(smem_u32(fills_out), even + 1)),
                                    [&](uint32_t c, int s) {
                                        return ld_shared_cluster(mapa_shared(smem_u32(stage_bytes + s), even + c));
                                    });
        cluster_sync();
    }
    if constexpr (kSplit > 1) {
        if (!aborted && part == 0 && have) {
            const int quad = warp & 3;
            const Item it = item_of<kKind, C>(args, cluster);
            const int f0 = it.m0 + (int)rank * 128 + quad * 32;
            if (f0 < args.m_total) {
                const float* parts = reinterpret_cast<const float*>(base_ptr + kPartsAt) + quad * 1024 + lane;
#pragma unroll
                for (int p = 0; p < kSplit - 1; ++p)
#pragma unroll
                    for (int q = 0; q < 32; ++q) (&mine.v[0][0][0])[q] += parts[p * 4096 + q * 32];
                Warp wp = {lane, quad, base + kStagingAt + (uint32_t)(warp - 4) * C::TILES * kTileBytes, 0, nullptr, 0};
                Residual res;
                if (args.residual) load_residual(res, args, it, f0, 0, lane);
                store_product(args, it, f0, 0, mine, res, maps, wp);
                if (lane == 0) bulk_wait_all();
                __syncwarp();
            }
        }
    }
    if (warp == 2) {
        fence_after();
        tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
    if (args.early) grid_dep_wait();   // complete only after the kernel before
}

// Maps of the rows operand b (chunks of at most 2 * nb rows), ksub strips of K per stage.
inline cudaError_t row_maps(CUtensorMap (&b)[4], const __nv_bfloat16* p, int64_t rows, int cols, int nb, int ksub) {
    if (nb < 32) return make_tma_map_strips(&b[0], p, (uint64_t)rows, (uint64_t)cols, (uint32_t)nb, (uint32_t)ksub);
    for (int i = 0; i < nb / 32; ++i) {
        const cudaError_t e = make_tma_map_strips(&b[i], p, (uint64_t)rows, (uint64_t)cols, 32u * (i + 1), (uint32_t)ksub);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// No more CTAs than there can be items: a small launch leaves SMs to the next
// one, whose prologue then overlaps it.
template <int kKind, int kNB>
cudaError_t launch(const Maps& maps, TileArgs args, int num_sms, cudaStream_t s) {
    using C = Cfg<kKind, kNB>;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = smem_limit_once(tile_gemm_kernel<kKind, kNB, 1>, C::SMEM_BYTES, done);
    if (e != cudaSuccess) return e;
    int grid = 0;
    e = pair_grid<tile_gemm_kernel<kKind, kNB, 1>, C::SMEM_BYTES, kThreads>(num_sms, &grid);
    if (e != cudaSuccess) return e;
    int64_t items;
    if (kKind == kWeights) {
        items = (int64_t)args.E * 3 * args.n_mtiles * args.n_ntiles;
    } else if (args.chunks) {
        items = max_chunks(args.rows, args.E, C::BN) * args.n_mtiles;
    } else {
        args.chunk_rows = dense_chunk(args.rows, C::BN, args.n_mtiles, grid / 2);
        args.dense_chunks = (int)(((int64_t)args.rows + args.chunk_rows - 1) / args.chunk_rows);
        items = (int64_t)args.dense_chunks * args.n_mtiles;
    }
    grid = (int)std::min<int64_t>(grid, 2 * items);
    return launch_pdl(tile_gemm_kernel<kKind, kNB, 1>, dim3(grid), dim3(kThreads), C::SMEM_BYTES, s, maps, args);
}

// One dense product of at most 2 * kNB rows, each item split over kSplit pairs.
// *fits: every item's cluster can be resident at once (nothing is launched if
// not).
template <int kKind, int kNB, int kSplit>
cudaError_t launch_split(const Maps& maps, TileArgs args, int num_sms, cudaStream_t s, bool* fits) {
    using C = Cfg<kKind, kNB, kSplit>;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = smem_limit_once(tile_gemm_kernel<kKind, kNB, kSplit>, C::SMEM_BYTES, done);
    if (e != cudaSuccess) return e;
    int twice = 0;       // two for each resident cluster
    e = pair_grid<tile_gemm_kernel<kKind, kNB, kSplit>, C::SMEM_BYTES, kThreads>(num_sms / C::CTAS * C::CTAS, &twice);
    if (e != cudaSuccess) return e;
    *fits = 2 * args.n_mtiles <= twice;
    if (!*fits) return cudaSuccess;
    args.chunk_rows = C::BN;
    args.dense_chunks = 1;
    return launch_pdl(tile_gemm_kernel<kKind, kNB, kSplit>, dim3(C::CTAS * args.n_mtiles), dim3(kThreads),
                      C::SMEM_BYTES, s, maps, args);
}

}  // namespace tg
}  // namespace moe
