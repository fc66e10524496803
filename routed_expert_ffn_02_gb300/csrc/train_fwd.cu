// train_fwd.cu -- the training forward pass of the experts on the tile kernel:
//   gate/up  h = bf16(silu(g) * u), g = x Wg^T and u = x Wu^T kept in bf16 or 8 bits;
//   down     y = h Wd^T.
// Both are bound by the tensor cores at the power cap.  8192 rows, H = 4096, I =
// 2048, one expert: gate/up 152 us (1.81 PFLOP/s; the items' epilogues, 6 of 38
// us, are not hidden), down 75 us (1.83); 65536 rows of 64 experts, 8-bit
// checkpoints: 1290 us (1.70) and 623 us (1.76).
#include "tile_gemm.cuh"

namespace moe {

cudaError_t launch_train_gate_up(const __nv_bfloat16* x, int64_t x_rows, const __nv_bfloat16* Wg,
                                 const __nv_bfloat16* Wu, int H, int I, bool fp8, int nb,
                                 TileArgs a, int num_sms, cudaStream_t s) {
    tg::Maps m = {};
    cudaError_t e;
    using C = tg::Cfg<tg::kGated, kWideRows>;
    if ((e = make_tma_map_strips(&m.a0, Wg, (uint64_t)a.E * I, H, 128, C::KSUB)) != cudaSuccess) return e;
    if ((e = make_tma_map_strips(&m.a1, Wu, (uint64_t)a.E * I, H, 128, C::KSUB)) != cudaSuccess) return e;
    if ((e = tg::row_maps(m.b[0], x, x_rows, H, nb, C::KSUB)) != cudaSuccess) return e;
    if ((e = make_tma_map_tile(&m.o0, a.out, false, x_rows, I)) != cudaSuccess) return e;
    if (!fp8) {
        if ((e = make_tma_map_tile(&m.o1, a.gate, false, x_rows, I)) != cudaSuccess) return e;
        if ((e = make_tma_map_tile(&m.o2, a.up, false, x_rows, I)) != cudaSuccess) return e;
    }
    a.n_mtiles = I / 256;
    a.a_rows = I;
    a.ld = I;
    a.k_blocks = H / C::BK;
    if (nb == kWideRows)
        return fp8 ? tg::launch<tg::kGatedFp8, kWideRows>(m, a, num_sms, s)
                   : tg::launch<tg::kGated, kWideRows>(m, a, num_sms, s);
    return fp8 ? tg::launch<tg::kGatedFp8, kThinRows>(m, a, num_sms, s)
               : tg::launch<tg::kGated, kThinRows>(m, a, num_sms, s);
}

cudaError_t launch_train_down(const __nv_bfloat16* h, int64_t h_rows, const __nv_bfloat16* Wd,
                              int H, int I, int nb, TileArgs a, int num_sms, cudaStream_t s) {
    tg::Maps m = {};
    cudaError_t e;
    using C = tg::Cfg<tg::kRows, kWideRows>;
    if ((e = make_tma_map_strips(&m.a0, Wd, (uint64_t)a.E * H, I, 128, C::KSUB)) != cudaSuccess) return e;
    if ((e = tg::row_maps(m.b[0], h, h_rows, I, nb, C::KSUB)) != cudaSuccess) return e;
    if ((e = make_tma_map_tile(&m.o0, a.out, false, h_rows, H)) != cudaSuccess) return e;
    a.n_mtiles = H / 256;
    a.a_rows = H;
    a.ld = H;
    a.k_blocks = I / C::BK;
    if (nb == kWideRows) return tg::launch<tg::kRows, kWideRows>(m, a, num_sms, s);
    return tg::launch<tg::kRows, kThinRows>(m, a, num_sms, s);
}

}  // namespace moe
