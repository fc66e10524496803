// train_bwd.cu -- the experts' backward pass on the tile kernel, from the
// gradient d of the layer's output at each row's token and the row's gate w:
//   hidden   q = d Wd; dg, du, w h and the parts of d_gate in its epilogue;
//   input    dx = dg Wg + du Wu, one accumulation over both products;
//   weights  dWd = d^T (w h), dWg = dg^T x, dWu = du^T x over each expert's rows.
// Taking the gate into the epilogue of the first product saves a pass over the
// rows and a rounding (d is read as it is, by token), and d_gate = q . h needs no
// y kept.  H = 4096, I = 2048, us: 8192 rows of one expert 98 / 144 / 240 (1.40,
// 1.91 and 1.72 PFLOP/s); 131072 rows of 384 experts (341 each) 1940 / 3450 /
// 6300, where memory moves 10.2, 16.1 and 23 GB (5.3, 4.7 and 3.7 TB/s).  With
// so few rows an item's K is short: the weights' items (22 MMAs) are bound by
// shared memory, whose 128 bytes a cycle also carry the results out (2.7 us an
// item; 2.1 with the stores left out, 1.9 without the epilogue).
#include "tile_gemm.cuh"

namespace moe {

cudaError_t launch_hidden_grad(const __nv_bfloat16* d, int64_t d_rows, const __nv_bfloat16* Wd,
                               int H, int I, bool fp8, int nb, int64_t out_rows, TileArgs a,
                               int num_sms, cudaStream_t s) {
    using C = tg::Cfg<tg::kHidden, kWideRows>;
    tg::Maps m = {};
    cudaError_t e;
    if ((e = make_tma_map_strips(&m.a0, Wd, (uint64_t)a.E * H, I, C::BK, 2)) != cudaSuccess) return e;
    if ((e = tg::row_maps(m.b[0], d, d_rows, H, nb, C::KSUB)) != cudaSuccess) return e;
    if ((e = make_tma_map_tile(&m.o0, a.out, false, out_rows, I)) != cudaSuccess) return e;
    if ((e = make_tma_map_tile(&m.o1, a.d_gate, false, out_rows, I)) != cudaSuccess) return e;
    if ((e = make_tma_map_tile(&m.o2, a.d_up, false, out_rows, I)) != cudaSuccess) return e;
    a.n_mtiles = I / 256;
    a.a_rows = H;
    a.ld = I;
    a.k_blocks = H / C::BK;
    if (nb == kWideRows)
        return fp8 ? tg::launch<tg::kHiddenFp8, kWideRows>(m, a, num_sms, s)
                   : tg::launch<tg::kHidden, kWideRows>(m, a, num_sms, s);
    return fp8 ? tg::launch<tg::kHiddenFp8, kThinRows>(m, a, num_sms, s)
               : tg::launch<tg::kHidden, kThinRows>(m, a, num_sms, s);
}

cudaError_t launch_input_grad(const __nv_bfloat16* dg, const __nv_bfloat16* du, int64_t rows,
                              const __nv_bfloat16* Wg, const __nv_bfloat16* Wu, int H, int I,
                              int nb, TileArgs a, int num_sms, cudaStream_t s) {
    using C = tg::Cfg<tg::kInput, kWideRows>;
    tg::Maps m = {};
    cudaError_t e;
    if ((e = make_tma_map_strips(&m.a0, Wg, (uint64_t)a.E * I, H, C::BK, 2)) != cudaSuccess) return e;
    if ((e = make_tma_map_strips(&m.a1, Wu, (uint64_t)a.E * I, H, C::BK, 2)) != cudaSuccess) return e;
    if ((e = tg::row_maps(m.b[0], dg, rows, I, nb, C::KSUB)) != cudaSuccess) return e;
    if ((e = tg::row_maps(m.b[1], du, rows, I, nb, C::KSUB)) != cudaSuccess) return e;
    e = a.out32 ? make_tma_map_tile(&m.o0, a.out32, true, a.rows, H) : make_tma_map_tile(&m.o0, a.out, false, a.rows, H);
    if (e != cudaSuccess) return e;
    a.n_mtiles = H / 256;
    a.a_rows = I;
    a.ld = H;
    a.seg_blocks = I / C::BK;
    a.k_blocks = 2 * a.seg_blocks;
    if (nb == kWideRows) return tg::launch<tg::kInput, kWideRows>(m, a, num_sms, s);
    return tg::launch<tg::kInput, kThinRows>(m, a, num_sms, s);
}

cudaError_t launch_weight_grad(const __nv_bfloat16* h, const __nv_bfloat16* dg,
                               const __nv_bfloat16* du, int64_t rows, const __nv_bfloat16* x,
                               const __nv_bfloat16* d, int64_t xd_rows, int H, int I, TileArgs a,
                               int num_sms, cudaStream_t s) {
    using C = tg::Cfg<tg::kWeights, kWideRows>;
    tg::Maps m = {};
    cudaError_t e;
    const struct {
        CUtensorMap *whole, *tail;      // 128 and 32 rows of K
        const __nv_bfloat16* p;
        int64_t rows;
        int cols;
    } operands[] = {{&m.a0, &m.tail_a0, h, rows, I},
                    {&m.a1, &m.tail_a1, x, xd_rows, H},
                    {&m.b[0][3], &m.b[0][0], d, xd_rows, H},
                    {&m.b[1][3], &m.b[1][0], dg, rows, I},
                    {&m.b[2][3], &m.b[2][0], du, rows, I}};
    for (const auto& q : operands) {
        if ((e = make_tma_map_strips(q.whole, q.p, q.rows, q.cols, C::BK, 2)) != cudaSuccess) return e;
        if ((e = make_tma_map_strips(q.tail, q.p, q.rows, q.cols, 32, 1)) != cudaSuccess) return e;
    }
    if ((e = make_tma_map_tile(&m.o0, a.out, false, (uint64_t)a.E * H, I, 64)) != cudaSuccess) return e;
    if ((e = make_tma_map_tile(&m.o1, a.d_gate, false, (uint64_t)a.E * I, H, 64)) != cudaSuccess) return e;
    if ((e = make_tma_map_tile(&m.o2, a.d_up, false, (uint64_t)a.E * I, H, 64)) != cudaSuccess) return e;
    a.n_mtiles = I / 256;
    a.n_ntiles = H / 256;
    a.m_total = I;
    a.n_total = H;
    return tg::launch<tg::kWeights, kWideRows>(m, a, num_sms, s);
}

}  // namespace moe
