// fp8_solo.cu -- one-CTA grouped products of 8-bit block-scaled operands:
// experts of at most 128 rows, one row tile each, and, in products of few rows
// (Fp8Args::with_pairs), the larger experts' 128-row tiles too.
//
//   plain:    y[rows, n0:n0+256] = bf16( A W_e[n0:n0+256]^T )
//   gate/up:  h[rows, n0:n0+128] = quantised( silu(A Wg_e^T) * (A Wu_e^T) ),
//             the gate and up rows of the same 128 columns back to back in
//             one N = 256 MMA; the 128 columns of a row are one block of 128.
//
// A is [rows, K] e4m3 with one scale byte per 128 of K, W [E, N, K] e4m3 with
// one per 128 x 128; the tensor core applies both (fp8.cuh).  Each weight byte
// is read from HBM once and used for one tile of rows, so the kernel is a
// weight stream bound by HBM; the MMAs take a third of the time.
//
// Persistent CTAs, one per SM, warp-specialised: warp 0 TMA producer (one
// lane), warp 1 MMA issuer (M = 128, N = 256, K = 32), warp 2 TMEM allocator,
// warp 3 scale producer, warps 4-7 epilogue.  A ring of 4 stages of 128 of K
// (16 KB of A, 32 KB of W) and a ring of 4 scale slots, each the scale words
// of 512 of K: 128 rows of A and 256 rows of W, written to shared memory by
// warp 3 and copied to TMEM by the MMA lane.  Slot i of the shared ring goes
// to slot i of the TMEM ring, and a slot is refilled only after the MMAs that
// read it have completed (its "empty" barrier), so no copy to TMEM overtakes
// an MMA.  The two accumulators overlap in TMEM as in the pair kernel
// (fp8_pair.cu): an item's epilogue runs under the next item's stream.
//
// Thin tiles (at most 32 rows).  A TMEM lane is a row of A and a warp reads
// only its own 32 lanes, so a few rows would leave the whole epilogue to one
// warp (its 128 SwiGLUs per lane took longer than the ring could bridge: a
// decode batch of 24 streamed at 75% of HBM, 94% in the down product that has
// none).  The 32 rows are therefore loaded into all four quarters of A: every
// warp finds them in its lanes and does a quarter of the columns.  Tiles of at
// most 8 rows load only 8 per quarter, which takes 12 of 48 KB off each stage.
//
// Every wait is bounded; on expiry the kernel records MOE_ERR_TIMEOUT, drains
// its own copies and MMAs, frees TMEM and returns.  The draining waits run in
// every launch (whichever role gave up, or none): each role's waits expire by
// themselves, so a role that ran to its end cannot know that another did not.
#include <cuda.h>

#include "fp8.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

using namespace ptx;
using namespace tc;
using fp8::kBlock;
using fp8::kGroupBlocks;
using fp8::kScaleBytes;
using fp8::kScaleCols;

constexpr int BM = kTileM;                      // 128 rows per tile
constexpr int BN = 256;                         // MMA N
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * kBlock;            // 16 KB
constexpr int B_BYTES = BN * kBlock;            // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int SLOTS = 4;                        // scale ring
constexpr int SLOT_BYTES = 3 * kScaleBytes;     // A, W rows 0-127, W rows 128-255
constexpr int SLOT_COLS = 3 * kScaleCols;
constexpr int TMEM_COLS = 512;
constexpr int SCALE_COL = TMEM_COLS - SLOTS * SLOT_COLS;   // 464
constexpr int ACC1_COL = SCALE_COL - BN;                   // 208: the accumulators overlap
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SLOTS * SLOT_BYTES + 1024 + 256;
constexpr uint32_t kIdesc = fp8::make_idesc(BM, BN);
static_assert(BN - ACC1_COL <= 64, "the overlap lies in the part that the epilogue reads first");

template <bool kGated>
__global__ void __launch_bounds__(256, 1)
fp8_solo_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                const __grid_constant__ CUtensorMap tmA8, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1, Fp8Args args) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    const uint32_t slots = base + STAGES * STAGE_BYTES;
    const uint32_t bars = slots + SLOTS * SLOT_BYTES;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (STAGES + s); };
    auto sfull_bar = [&](int s) { return bars + 8u * (2 * STAGES + s); };
    auto sempty_bar = [&](int s) { return bars + 8u * (2 * STAGES + SLOTS + s); };
    const uint32_t tfull_bar = bars + 8u * (2 * STAGES + 2 * SLOTS);
    const uint32_t drained_bar = tfull_bar + 8u;    // the overlap of an item has been read
    const uint32_t max_bar = tfull_bar + 16u;       // thin gate/up: four warps' maxima are in
    const uint32_t done_bar = tfull_bar + 24u;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + (done_bar + 8u - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    __shared__ float part_max[2][4][32];   // thin gate/up: a row's maximum, by warp; items
                                           // alternate, so a reader is never overwritten
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(sfull_bar(s), 1);
            mbar_init(sempty_bar(s), 1);
        }
        mbar_init(tfull_bar, 1);
        mbar_init(drained_bar, 4);
        mbar_init(max_bar, 4);
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&tmA);
        prefetch_map(&tmA32);
        prefetch_map(&tmA8);
        prefetch_map(&tmB0);
        if (kGated) prefetch_map(&tmB1);
    }
    if (warp == 2) tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem_base = *tmem_holder;
    const int k_blocks = args.k_blocks;

    // Everything above overlaps the previous kernel.  With early_weights the
    // tile lists were complete before that kernel started (see Fp8Args), so
    // they and the weights are read before the wait for it; reads go to L2,
    // past this SM's L1.
    if (!args.early_weights) {
        grid_dep_wait();
        grid_dep_launch();
    }
    auto list_tile = [](const FatTile* p) {
        const uint4 v = ld::u32x4_cg(p);
        return FatTile{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
    };
    const fp8::OneGroup grp = args.group ? fp8::one_group(args) : fp8::OneGroup{0, 0};
    const bool with_pairs = args.with_pairs && !args.group;
    const int n_pair = with_pairs ? ld::i32_cg(&args.hdr->n_fat_tiles) : 0;
    const int n_solo = args.group ? 0 : n_pair + ld::i32_cg(&args.hdr->n_solo);
    const int n_tiles = args.group ? (grp.n + BM - 1) / BM : n_solo + ld::i32_cg(&args.hdr->n_thin_mma);
    const int total = n_tiles * args.n_blocks_n;
    // (the second tile of an expert's last pair may be empty)
    auto tile_at = [&](int i) {
        if (args.group) return fp8::group_tile(grp, i);
        return list_tile(i < n_pair   ? args.tiles + i
                         : i < n_solo ? args.solo_tiles + (i - n_pair)
                                      : args.thin_tiles + (i - n_solo));
    };
    // Items go round-robin to the first `active` CTAs, as many as keep every
    // wave full (see the bf16 one-CTA GEMM).
    const int waves = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const int active = waves > 0 ? (total + waves - 1) / waves : 0;
    // A CTA without items takes no role; total_mine ends its loops at once.
    const int total_mine = (int)blockIdx.x < active ? total : 0;
    if (args.early_weights && (warp != 0 || total_mine == 0)) {
        grid_dep_wait();
        grid_dep_launch();
    }
    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer ----------------
        int stage = 0;
        uint32_t phase = 0;
        int pending[STAGES];
        for (int s = 0; s < STAGES; ++s) pending[s] = -1;
        bool ok = true;
        auto load_w = [&](uint32_t sb, uint32_t bar, int x, int y) {
            tma_load_2d(sb, &tmB0, bar, x, y);
            if (kGated) tma_load_2d(sb + B_BYTES / 2, &tmB1, bar, x, y);
        };
        auto load_a = [&](uint32_t sa, uint32_t bar, int x, const FatTile& ft) {
            if (ft.rows > kThinMaxTokens) {
                tma_load_2d(sa, &tmA, bar, x, ft.row0);
            } else {
                // the rest of a quarter keeps what it held: rows of D that are not read
                const CUtensorMap* map = ft.rows > 8 ? &tmA32 : &tmA8;
#pragma unroll
                for (int i = 0; i < 4; ++i) tma_load_2d(sa + i * (A_BYTES / 4), map, bar, x, ft.row0);
            }
        };
        auto stage_bytes = [](const FatTile& ft) {
            return (uint32_t)(B_BYTES + (ft.rows > 8 ? A_BYTES : 4 * 8 * kBlock));
        };
        // The first stages' weights do not depend on the previous kernel.  They
        // are those of the CTA's first item with rows: the loop below skips
        // empty tiles, so what is started here has to be what it runs first.
        int early = 0, early_end = 0;   // stages [early_end - early, early_end) lack their rows
        uint32_t early_rows = 0;        // bytes of them per stage
        if (args.early_weights && total_mine > 0) {
            FatTile ft = {};
            int t = blockIdx.x;
            for (; t < total_mine; t += active) {
                ft = tile_at(t / args.n_blocks_n);
                if (ft.rows > 0) break;
            }
            const int brow = ft.expert * args.n_rows + (t % args.n_blocks_n) * (kGated ? 128 : BN);
            const int stages = ft.rows > 0 ? min(STAGES, k_blocks) : 0;
            for (; early < stages; ++early) {
                mbar_expect_tx(full_bar(early), stage_bytes(ft));
                load_w(base + early * STAGE_BYTES + A_BYTES, full_bar(early), early * kBlock, brow);
            }
            early_end = early;
            early_rows = stage_bytes(ft) - B_BYTES;
            grid_dep_wait();
            grid_dep_launch();
            // the rows come from the previous kernel's ordinary stores
            fence_proxy_async_global();
        }
        for (int t = blockIdx.x; ok && t < total_mine; t += active) {
            const FatTile ft = tile_at(t / args.n_blocks_n);
            if (ft.rows == 0) continue;
            const int brow = ft.expert * args.n_rows + (t % args.n_blocks_n) * (kGated ? 128 : BN);
            for (int kb = 0; kb < k_blocks; ++kb) {
                if (!mbar_wait_for(empty_bar(stage), phase ^ 1u, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = base + stage * STAGE_BYTES;
                if (early > 0) {
                    --early;
                } else {
                    mbar_expect_tx(full_bar(stage), stage_bytes(ft));
                    load_w(sa + A_BYTES, full_bar(stage), kb * kBlock, brow);
                }
                load_a(sa, full_bar(stage), kb * kBlock, ft);
                pending[stage] = (int)phase;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok) {
            *abort_flag = 1;
            set_status(args.hdr, MOE_ERR_TIMEOUT);
            for (int s = early_end - early; s < early_end; ++s) {
                mbar_complete_tx(full_bar(s), early_rows);
                pending[s] = 0;
            }
        }
        // Every copy has landed before the CTA leaves.  Also where this loop
        // ran to its end: the MMA lane may have given up on the last stages.
        for (int s = 0; s < STAGES; ++s)
            if (pending[s] >= 0) (void)mbar_wait(full_bar(s), (uint32_t)pending[s]);
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMA issuer ----------------
        int stage = 0, slot = 0;
        uint32_t phase = 0, sphase = 0;
        int it = 0;
        bool ok = true;
        bool issued = false;
        for (int t = blockIdx.x; ok && t < total_mine; t += active) {
            if (with_pairs && tile_at(t / args.n_blocks_n).rows == 0) continue;
            // the previous item's epilogue has read the overlap (and with it,
            // being in order, all of this buffer's previous item)
            if (it > 0 && !mbar_wait_for(drained_bar, (uint32_t)((it - 1) & 1), args.wait_cycles,
                                         abort_flag)) {
                ok = false;
                break;
            }
            fence_after();
            const uint32_t d_tmem = tmem_base + (uint32_t)((it & 1) ? ACC1_COL : 0);
            for (int kb = 0; kb < k_blocks; ++kb) {
                const uint32_t sc = tmem_base + SCALE_COL + slot * SLOT_COLS;
                if (kb % kGroupBlocks == 0) {
                    if (!mbar_wait_for(sfull_bar(slot), sphase, args.wait_cycles, abort_flag)) {
                        ok = false;
                        break;
                    }
                    fence_after();
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        fp8::scale_copy(sc + i * kScaleCols,
                                        fp8::scale_desc(slots + slot * SLOT_BYTES + i * kScaleBytes));
                    issued = true;
                }
                if (!mbar_wait_for(full_bar(stage), phase, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t sa = base + stage * STAGE_BYTES;
                const uint64_t ad = sw128_desc(sa);
                const uint64_t bd = sw128_desc(sa + A_BYTES);
                const uint32_t idesc = fp8::with_scale_byte(kIdesc, kb % kGroupBlocks);
#pragma unroll
                for (int kk = 0; kk < kBlock / 32; ++kk)   // +32 bytes per K step
                    fp8::mma(d_tmem, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc, sc,
                             sc + kScaleCols, (kb > 0 || kk > 0) ? 1u : 0u);
                commit(empty_bar(stage));
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (kb % kGroupBlocks == kGroupBlocks - 1 || kb == k_blocks - 1) {
                    commit(sempty_bar(slot));
                    if (++slot == SLOTS) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
            }
            if (!ok) break;
            commit(tfull_bar);
            ++it;
        }
        if (!ok) {
            *abort_flag = 1;
            set_status(args.hdr, MOE_ERR_TIMEOUT);
        }
        // Every MMA has completed before TMEM is freed.  Also where this loop
        // ran to its end: the epilogue may have given up on the last tile.
        if (issued) {
            commit(done_bar);
            (void)mbar_wait(done_bar, 0);
        }
    } else if (warp == 3) {
        // ---------------- scale producer ----------------
        // Lane l holds rows l, l + 32, l + 64, l + 96 of the A tile; every
        // 128 rows of W share one word, so its 512 bytes repeat it.
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        const int groups = (k_blocks + kGroupBlocks - 1) / kGroupBlocks;
        for (int t = blockIdx.x; ok && t < total_mine; t += active) {
            const FatTile ft = tile_at(t / args.n_blocks_n);
            if (ft.rows == 0) continue;
            const int nt = t % args.n_blocks_n;
            const uint8_t* ra[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // rows past the tile's only scale rows of D that are not stored;
                // a thin tile's rows repeat in every quarter
                const int r = min(ft.row0 + lane + (ft.rows > kThinMaxTokens ? 32 * i : 0),
                                  args.rows - 1);
                ra[i] = args.a_scales + (int64_t)r * k_blocks;
            }
            const int64_t eb = (int64_t)ft.expert * (args.n_rows / kBlock);
            const int last = args.n_rows / kBlock - 1;   // N is a multiple of 128, not of 256
            const uint8_t* rb0 =
                args.b0_scales + (eb + (kGated ? nt : min(2 * nt, last))) * k_blocks;
            const uint8_t* rb1 =
                kGated ? args.b1_scales + (eb + nt) * k_blocks
                       : args.b0_scales + (eb + min(2 * nt + 1, last)) * k_blocks;
            for (int g = 0; g < groups; ++g) {
                uint32_t a[4];
                const uint32_t b0 = fp8::scale_word(rb0, g, k_blocks);
                const uint32_t b1 = fp8::scale_word(rb1, g, k_blocks);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = fp8::scale_word(ra[i], g, k_blocks);
                if (!__all_sync(0xffffffffu, mbar_wait_for(sempty_bar(slot), phase ^ 1u,
                                                           args.wait_cycles, abort_flag))) {
                    ok = false;
                    break;
                }
                const uint32_t dst = slots + slot * SLOT_BYTES + lane * 16u;
                st_shared_v4(dst, a[0], a[1], a[2], a[3]);
                st_shared_v4(dst + kScaleBytes, b0, b0, b0, b0);
                st_shared_v4(dst + 2 * kScaleBytes, b1, b1, b1, b1);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull_bar(slot));
                if (++slot == SLOTS) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            set_status(args.hdr, MOE_ERR_TIMEOUT);
        }
    } else if (warp >= 4) {
        // ---------------- epilogue ----------------
        const int ew = warp - 4;   // TMEM lanes 32*ew .. 32*ew+31
        int it = 0, n_thin = 0;
        for (int t = blockIdx.x; t < total_mine; t += active) {
            const FatTile ft = tile_at(t / args.n_blocks_n);
            if (ft.rows == 0) continue;
            // the whole warp decides together (tcgen05.ld below is warp-wide)
            if (!__all_sync(0xffffffffu, mbar_wait_for(tfull_bar, (uint32_t)(it & 1),
                                                       args.wait_cycles, abort_flag))) {
                *abort_flag = 1;
                set_status(args.hdr, MOE_ERR_TIMEOUT);
                break;
            }
            fence_after();
            const int nt = t % args.n_blocks_n;
            const int odd = it & 1;
            const bool thin = ft.rows <= kThinMaxTokens;
            const int row = thin ? lane : ew * 32 + lane;
            const bool valid = row < ft.rows;
            const int64_t out_row = (int64_t)ft.row0 + row;
            const uint32_t taddr =
                tmem_base + ((uint32_t)(ew * 32) << 16) + (uint32_t)(odd ? ACC1_COL : 0);
            auto drained = [&]() {   // the columns shared with the other buffer have been read
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(drained_bar);
                __syncwarp();   // converged for the warp-wide TMEM loads that follow
            };
            if (kGated && thin) {
                // 32 of the 128 columns per warp; the row's maximum over the four warps
                const int f = 32 * ew;
                uint32_t g[32], u[32];
                tmem_ld32(taddr + f, g);
                tmem_ld32(taddr + 128 + f, u);
                tmem_ld_wait();
                drained();
                float h[32];
                float m = 0.f;
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                    h[q] = fp8::swiglu(__uint_as_float(g[q]), __uint_as_float(u[q]));
                    m = fmaxf(m, fp8::finite_abs(h[q]));
                }
                float(*pm)[32] = part_max[n_thin & 1];
                pm[ew][lane] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(max_bar);
                if (!__all_sync(0xffffffffu, mbar_wait_for(max_bar, (uint32_t)(n_thin & 1),
                                                           args.wait_cycles, abort_flag))) {
                    *abort_flag = 1;
                    set_status(args.hdr, MOE_ERR_TIMEOUT);
                    break;
                }
                ++n_thin;
                m = fmaxf(fmaxf(pm[0][lane], pm[1][lane]), fmaxf(pm[2][lane], pm[3][lane]));
                const uint32_t sb = fp8::scale_byte(m);
                const float inv = fp8::inverse_scale(sb);
                if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(args.out_q + out_row * args.ld_out +
                                                          (int64_t)nt * kBlock + f);
                    dst[0] = fp8::quantize16(h, inv);
                    dst[1] = fp8::quantize16(h + 16, inv);
                    if (ew == 0)
                        args.out_scales[out_row * (args.ld_out / kBlock) + nt] = (uint8_t)sb;
                }
            } else if (kGated) {
                // first the 64 columns whose TMEM columns overlap: the upper
                // ones of buffer 0 (up columns 208-255), the lower of buffer 1
                const int first = odd ? 0 : 64;
                float h[kBlock];
                float m = 0.f;
#pragma unroll
                for (int c = 0; c < kBlock; c += 32) {
                    const int f = (first + c) & 127;
                    uint32_t g[32], u[32];
                    tmem_ld32(taddr + f, g);
                    tmem_ld32(taddr + 128 + f, u);
                    tmem_ld_wait();
                    if (c == 32) drained();
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        h[c + q] = fp8::swiglu(__uint_as_float(g[q]), __uint_as_float(u[q]));
                        m = fmaxf(m, fp8::finite_abs(h[c + q]));
                    }
                }
                const uint32_t sb = fp8::scale_byte(m);
                const float inv = fp8::inverse_scale(sb);
                if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(args.out_q + out_row * args.ld_out +
                                                          (int64_t)nt * kBlock);
#pragma unroll
                    for (int q = 0; q < 8; ++q)   // h is in the order read
                        dst[(first / 16 + q) & 7] = fp8::quantize16(h + 16 * q, inv);
                    args.out_scales[out_row * (args.ld_out / kBlock) + nt] = (uint8_t)sb;
                }
            } else {
                const int64_t at = out_row * args.ld_out + (int64_t)nt * BN;
                const int cols = (int)min((int64_t)BN, args.ld_out - (int64_t)nt * BN);
#pragma unroll 1
                for (int i = 0; i < (thin ? 1 : 4); ++i) {
                    // 64 columns at a time, the overlapping ones first; of a
                    // thin tile each warp does 64
                    const int c = thin ? 64 * ew : odd ? 64 * i : 64 * ((i + 3) & 3);
                    uint32_t d[64];
                    tmem_ld32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(d));
                    tmem_ld32(taddr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(d + 32));
                    tmem_ld_wait();
                    if (i == 0) drained();
                    if (valid && c < cols) {
                        if (args.out32) {
                            uint4* d4 = reinterpret_cast<uint4*>(args.out32 + at + c);
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                d4[q] = make_uint4(d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]);
                        } else {
                            uint4* d4 = reinterpret_cast<uint4*>(args.out + at + c);
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                uint32_t o[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    o[j] = pack_bf16(__uint_as_float(d[8 * q + 2 * j]),
                                                     __uint_as_float(d[8 * q + 2 * j + 1]));
                                d4[q] = make_uint4(o[0], o[1], o[2], o[3]);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            __syncwarp();
            ++it;
        }
    }

    fence_before();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <bool kGated>
cudaError_t set_smem_attr() {
    static std::atomic<int> done[kMaxDevices];
    return smem_limit_once(fp8_solo_kernel<kGated>, SMEM_BYTES, done);
}

template <bool kGated>
cudaError_t launch(const uint8_t* a, int64_t rows, const uint8_t* b0, const uint8_t* b1,
                   const Fp8Args& args, int E, int num_sms, cudaStream_t s) {
    const uint64_t K = (uint64_t)args.k_blocks * kBlock;
    CUtensorMap mA, mA32, mA8, mB0, mB1;
    cudaError_t e;
    if ((e = make_tma_map_u8(&mA, a, (uint64_t)rows, K, BM)) != cudaSuccess) return e;
    if ((e = make_tma_map_u8(&mA32, a, (uint64_t)rows, K, kThinMaxTokens)) != cudaSuccess) return e;
    if ((e = make_tma_map_u8(&mA8, a, (uint64_t)rows, K, 8)) != cudaSuccess) return e;
    const uint32_t box = kGated ? 128 : 256;
    if ((e = make_tma_map_u8(&mB0, b0, (uint64_t)E * args.n_rows, K, box)) != cudaSuccess) return e;
    if ((e = make_tma_map_u8(&mB1, b1, (uint64_t)E * args.n_rows, K, box)) != cudaSuccess) return e;
    if ((e = set_smem_attr<kGated>()) != cudaSuccess) return e;
    return launch_pdl(fp8_solo_kernel<kGated>, dim3(num_sms), dim3(256), SMEM_BYTES, s, mA, mA32,
                      mA8, mB0, mB1, args);
}

}  // namespace

cudaError_t launch_fp8_solo_gate_up(const uint8_t* a, int64_t rows, const uint8_t* b0,
                                    const uint8_t* b1, const Fp8Args& args, int E, int num_sms,
                                    cudaStream_t s) {
    return launch<true>(a, rows, b0, b1, args, E, num_sms, s);
}
cudaError_t launch_fp8_solo(const uint8_t* a, int64_t rows, const uint8_t* b, const Fp8Args& args,
                            int E, int num_sms, cudaStream_t s) {
    return launch<false>(a, rows, b, b, args, E, num_sms, s);
}

}  // namespace moe
