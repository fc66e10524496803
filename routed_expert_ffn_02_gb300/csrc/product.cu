// product.cu -- the grouped bf16 product with bias, activation and residual in
// its epilogue, on the tile kernel.  16384 x 4096 x 4096 with silu, bias and
// residual: 292 us (1.88 PFLOP/s; 338 us, 1.63, at the power cap), the library's
// plain product 272; the epilogue's share is the last round's.  Rows whose
// length in bytes is no multiple of 16 (odd N) are loaded and stored two or four
// bytes a lane.
#include "tile_gemm.cuh"

namespace moe {

cudaError_t launch_product(const __nv_bfloat16* x, int64_t rows, const __nv_bfloat16* W, int N,
                           int K, int nb, TileArgs a, int num_sms, cudaStream_t s) {
    using C = tg::Cfg<tg::kProduct, kWideRows>;
    tg::Maps m = {};
    cudaError_t e;
    a.k_blocks = (K + C::BK - 1) / C::BK;
    a.flat_from = K / C::BK;           // the block that K does not fill, if there is one
    // Few rows, few feature tiles: K is split so that more SMs stream weights.
    // Up to 32 rows times 4096 x 4096 took 17.4 us on 16 pairs, 32 blocks of K at
    // 0.41 us (a pair's MMAs of few rows take about 100 cycles each); split in
    // two, 11.0; 24 rows times 384 x 4096 16.8, split in four 7.6.
    const bool split = !a.chunks && a.rows <= 2 * kSplitRows && a.k_blocks >= 8;
    if (split) nb = kSplitRows;
    if (a.flat_from > 0) {
        if ((e = make_tma_map_strips(&m.a0, W, (uint64_t)a.E * N, K, 128, C::KSUB)) != cudaSuccess) return e;
        if ((e = tg::row_maps(m.b[0], x, rows, K, nb, C::KSUB)) != cudaSuccess) return e;
    }
    const int rest = K - a.flat_from * C::BK;
    a.flat_strips = (rest + 63) / 64;
    a.k16_last = rest ? (rest + 15) / 16 : C::BK / 16;
    if (rest) {
        if ((e = make_tma_map_bf16(&m.flat_a, W, (uint64_t)a.E * N, K, 128)) != cudaSuccess) return e;
        for (int i = 0; i < (nb < 32 ? 1 : nb / 32); ++i)
            if ((e = make_tma_map_bf16(&m.b[1][i], x, rows, K, nb < 32 ? nb : 32 * (i + 1))) != cudaSuccess) return e;
    }
    a.map_out = N % (a.out32 ? 4 : 8) == 0;
    if (a.map_out) {
        e = a.out32 ? make_tma_map_tile(&m.o0, a.out32, true, rows, N) : make_tma_map_tile(&m.o0, a.out, false, rows, N);
        if (e != cudaSuccess) return e;
    }
    a.n_mtiles = (N + 255) / 256;
    a.m_total = N;
    a.a_rows = N;
    a.ld = N;
    if (nb == kWideRows) return tg::launch<tg::kProduct, kWideRows>(m, a, num_sms, s);
    if (split) {
        bool fits = false;
        e = tg::launch_split<tg::kProduct, kSplitRows, 4>(m, a, num_sms, s, &fits);
        if (fits || e != cudaSuccess) return e;
        e = tg::launch_split<tg::kProduct, kSplitRows, 2>(m, a, num_sms, s, &fits);
        if (fits || e != cudaSuccess) return e;
        return tg::launch<tg::kProduct, kSplitRows>(m, a, num_sms, s);
    }
    return tg::launch<tg::kProduct, kThinRows>(m, a, num_sms, s);
}

}  // namespace moe
