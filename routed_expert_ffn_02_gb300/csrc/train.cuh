// train.cuh -- what the translation units of the training passes and of the
// product with an epilogue share: the lists of their work, the arguments of
// the tile kernel (tile_gemm.cuh), and the launchers.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "moe_internal.cuh"

namespace moe {

// Rows [row0, row0 + rows) of the sorted rows, of one expert.  In the padded
// buffers each expert's rows start at a multiple of 16 and are followed by
// zero rows up to the next one, so that a product over an expert's rows can
// run in whole MMA steps of 16.
struct RowChunk {
    int32_t expert;
    int32_t row0;
    int32_t rows;
    int32_t row0_pad;
};
__host__ __device__ inline int64_t max_chunks(int64_t P, int E, int most) { return P / most + E; }
inline int64_t padded_rows(int64_t P, int E) { return (int64_t)align_up((size_t)P, 16) + 16 * (int64_t)E; }

// A group of c rows in chunks of at most `most` rows (a multiple of 16):
// ceil(c / most) of them, of equal size up to the rounding to 16.  Unsigned: a
// group of 2^31 - 129 rows and its number of chunks add up to more than 2^31.
__host__ __device__ inline int chunk_size(int c, int most) {
    const uint32_t n = ((uint32_t)c + (uint32_t)most - 1) / (uint32_t)most;
    return n == 0 ? 0 : (int)((((uint32_t)c + n - 1) / n + 15) & ~15u);
}
__host__ __device__ inline int chunk_count(int c, int size) {
    return size == 0 ? 0 : (int)(((uint32_t)c + (uint32_t)size - 1) / (uint32_t)size);
}

// Rows of one group's chunks, for n_mtiles feature tiles on `pairs` CTA pairs.
// An item costs about its rows, but no less than 128 (see kThinRows), and 16
// for its ends; the
// grid takes whole rounds of items.  8192 x 2048 over K = 4096 in chunks of 256
// is 256 items on 76 pairs, four rounds for 3.4; in chunks of 224 it is 3.9.
inline int dense_chunk(int rows, int most, int n_mtiles, int pairs) {
    int best = most;
    int64_t least = INT64_MAX;
    for (int size = most; size >= 16; size -= 16) {
        const int64_t items = ((int64_t)rows + size - 1) / size * n_mtiles;
        const int64_t cost = (items + pairs - 1) / pairs * ((size < 128 ? 128 : size) + 16);
        if (cost < least) {
            least = cost;
            best = size;
        }
    }
    return best;
}

struct TileArgs {
    WsHeader* hdr;
    const RowChunk* chunks;    // the chunks, or null: one group of `rows` rows
    const int32_t* n_chunks;
    const RowChunk* groups;    // weight gradients: each expert's rows, or null likewise
    int dense_chunks;          // without lists: chunks, and the rows of each; set by the launchers
    int chunk_rows;
    int rows;                  // sorted rows
    int E;
    int early;                 // reads nothing of the kernel before: starts as that one's CTAs leave
    int padded;                // B's rows are those of a padded buffer
    int n_mtiles, n_ntiles;    // 256-wide tiles of the features (weights: of I and of H)
    int m_total, n_total;      // product: features; weights: I and H
    int a_rows;                // rows of A per expert
    int k_blocks;
    int seg_blocks;            // input gradient: blocks of the first product
    int flat_from;             // product: the block that K does not fill, its strips of 64 and
    int flat_strips;           // steps of 16
    int k16_last;
    int64_t ld;                // features of an output row
    long long wait_cycles;
    // Buffers by kind (see the epilogues).
    __nv_bfloat16* out;
    float* out32;
    void *gate, *up;           // the kept projections
    uint8_t *gate_scales, *up_scales;
    __nv_bfloat16 *d_gate, *d_up;
    const float* gates;        // gates and the slot of each sorted row
    const int32_t* perm;
    float* gate_parts;         // [I / 32, rows]
    const float* bias;
    const __nv_bfloat16* residual;
    int act;
    int vec;                   // product: rows of y and of the residual are 16-byte aligned
    int map_out;               // product: rows of y can be stored by the copy engine; set by the launcher
};

// Lists of the offsets' groups (chunks of at most `most` rows); the offsets
// are forced to ascend inside [0, rows] (MOE_ERR_BAD_INDEX recorded where
// they do not, or do not start at 0 and end at rows).
struct RowLists {
    RowChunk* chunks;      // [max_chunks]
    RowChunk* groups;      // [E]
    int32_t* n_chunks;
    int32_t* ends;         // [2]: the first group's first row, the last group's end
};
cudaError_t launch_plan_rows(const int32_t* offsets, int rows, int E, int most, const RowLists& l,
                             WsHeader* hdr, cudaStream_t s);

// Forward: the lists, and xs[p] = x[perm[p] / k] for the sorted rows.
cudaError_t launch_forward_rows(const __nv_bfloat16* x, const int32_t* perm, int k, int H,
                                const int32_t* offsets, int P, int E, int most, __nv_bfloat16* xs,
                                const RowLists& l, WsHeader* hdr, int num_sms, cudaStream_t s);

// Backward: the lists, and the padded rows of x (its values, where x_scales
// says that it holds e4m3; x_rows null: left out, x is not read) and of d.
struct BackwardRows {
    const void* x;
    const uint8_t* x_scales;
    const __nv_bfloat16* d;
    const int32_t *perm, *inv_perm, *offsets;
    __nv_bfloat16 *x_rows, *d_rows;
    RowLists lists;
    WsHeader* hdr;
    int T, k, H, E, most;
};
cudaError_t launch_backward_rows(const BackwardRows& q, int num_sms, cudaStream_t s);

// d_x[t] = sum_j y[inv[t * k + j]] (y fp32 [P, H]; d_x null: left out), and
// d_gates[s] = sum over parts [n_parts, P] at position inv[s] (null: left out;
// inv null: position s).  Positions outside the groups (ends of the lists; null:
// [0, P)) count as zeros.
cudaError_t launch_finish(const float* y, __nv_bfloat16* d_x, const float* parts, int n_parts, float* d_gates,
                          const int32_t* inv, const int32_t* ends, int T, int k, int H, int num_sms, cudaStream_t s);

// bf16 values of rows of e4m3 with a scale per 128 of K (exact).
cudaError_t launch_dequantize_rows(const uint8_t* q, const uint8_t* scales, int64_t rows, int K,
                                   __nv_bfloat16* x, int num_sms, cudaStream_t s);

// 3-D bf16 tensor map over a row-major [rows, cols] matrix seen as strips of 64
// columns, [cols / 64][rows][64], 128-byte swizzle, zero fill outside (columns behind
// the last whole strip left out): box = box_strips strips x box_rows rows, so
// that one copy loads several of the 128-byte-wide tiles the MMA reads.
cudaError_t make_tma_map_strips(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows,
                                uint32_t box_strips);
// Map for storing tiles (box = 32 columns x box_rows) of bf16 (64-byte
// swizzle) or fp32 (128-byte swizzle).
cudaError_t make_tma_map_tile(CUtensorMap* m, const void* ptr, bool f32, uint64_t rows, uint64_t cols,
                              uint32_t box_rows = 32);

// Products on CTA pairs.  `a` carries the lists, sizes and epilogue buffers;
// the launchers add the operands.
// Rows of B per CTA (half of the most rows of a chunk) that are built: a pair's
// MMA takes about 100 cycles for any N up to 128 and 134 for 256, so chunks of
// up to 128 rows are the narrowest of use (they leave room for a fourth stage
// and for two pairs of accumulators in TMEM); 16 where K is split instead.
constexpr int kWideRows = 128, kThinRows = 64, kSplitRows = 16;
cudaError_t launch_train_gate_up(const __nv_bfloat16* x, int64_t x_rows, const __nv_bfloat16* Wg,
                                 const __nv_bfloat16* Wu, int H, int I, bool fp8, int nb,
                                 TileArgs a, int num_sms, cudaStream_t s);
cudaError_t launch_train_down(const __nv_bfloat16* h, int64_t h_rows, const __nv_bfloat16* Wd,
                              int H, int I, int nb, TileArgs a, int num_sms, cudaStream_t s);
cudaError_t launch_hidden_grad(const __nv_bfloat16* d, int64_t d_rows, const __nv_bfloat16* Wd,
                               int H, int I, bool fp8, int nb, int64_t out_rows, TileArgs a,
                               int num_sms, cudaStream_t s);
cudaError_t launch_input_grad(const __nv_bfloat16* dg, const __nv_bfloat16* du, int64_t rows,
                              const __nv_bfloat16* Wg, const __nv_bfloat16* Wu, int H, int I,
                              int nb, TileArgs a, int num_sms, cudaStream_t s);
cudaError_t launch_weight_grad(const __nv_bfloat16* h, const __nv_bfloat16* dg,
                               const __nv_bfloat16* du, int64_t rows, const __nv_bfloat16* x,
                               const __nv_bfloat16* d, int64_t xd_rows, int H, int I, TileArgs a,
                               int num_sms, cudaStream_t s);
cudaError_t launch_product(const __nv_bfloat16* x, int64_t rows, const __nv_bfloat16* W, int N,
                           int K, int nb, TileArgs a, int num_sms, cudaStream_t s);

// The dense product of at most kFewRows rows by streaming the weights.
constexpr int kFewRows = 3;
struct ProductEpilogue {
    const float* bias;
    const __nv_bfloat16* residual;
    __nv_bfloat16* out;        // or out32
    float* out32;
    int act;
};
cudaError_t launch_product_rows(const __nv_bfloat16* x, int rows, const __nv_bfloat16* W, int N, int K,
                                const ProductEpilogue& e, cudaStream_t s);

}  // namespace moe
