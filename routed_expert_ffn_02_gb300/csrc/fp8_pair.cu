// fp8_pair.cu -- grouped products of 8-bit block-scaled operands on CTA pairs
// (tcgen05 cta_group::2): experts of more than 128 rows.
//
// The same products as fp8_solo.cu on 256 x 256 output tiles: CTA r of a pair
// loads its own 128 rows of A (planner tile 2q + r) and half of the W tile
// (gate / up rows, or the first / second 128 of 256 rows), so an SM reads 32
// KB from L2 per 128 of K where a one-CTA 128 x 256 tile reads 48 KB.  The
// 8-bit MMA runs at twice the bf16 rate on half the bytes, so the copies per
// MMA cycle are those of the bf16 pair GEMM (gemm_tc.cu), whose layout this
// kernel takes: stages of 256 of K (two 128-byte swizzle atoms per operand,
// 64 KB per CTA, 3 stages), the even CTA's lane issuing the MMAs of both.
//
// Scales.  Warps 8-11 of each CTA write the scale words of 512 of K (the CTA's
// own 128 rows of A, all 256 rows of W) straight to TMEM, each warp its 32
// lanes (the hardware reads the words of a row from every quarter), into a
// ring of 4 slots that the MMAs' completion frees.  That keeps the tensor
// pipe to MMAs: with copies from shared memory on it (tcgen05.cp, three per
// 512 of K) 16384 x 4096 x 4096 took 200.6 us, with these stores 197.1.
//
// What bounds it: power.  16384 x 4096 x 4096 takes 184 us (2.99 PFLOP/s) with
// the chip at its 1.4 kW limit and 1.72 GHz; with operands of zeros, at 2.03
// GHz, 168.  Per tile of 4096 of K about 18,000 cycles of issue against 16,400
// of MMA, and about 1,000 from one tile to the next.
//
// TMEM.  Two 256-column accumulators and the 48 columns of scales do not fit
// in 512 columns, so the accumulators overlap: buffer 0 is columns [0, 256),
// buffer 1 [208, 464), the scales [464, 512).  The epilogue of a tile reads
// the half that holds the overlap first and then frees it, so the next tile's
// MMAs wait for a quarter to a half of an epilogue, not for all of it.
//
// Roles as in the bf16 pair GEMM: warp 0 TMA producer, warp 1 MMA issuer
// (even CTA), warp 2 TMEM allocator, warps 4-7 epilogue, warps 8-11 scales.
// Every wait is bounded; on expiry the role records MOE_ERR_TIMEOUT, both
// CTAs stop issuing, issued MMAs and copies are waited for, TMEM is freed.
#include <cuda.h>

#include "fp8.cuh"
#include "moe_internal.cuh"
#include "pair_dev.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

using namespace ptx;
using namespace tc;
using fp8::kBlock;
using fp8::kGroupBlocks;
using fp8::kScaleCols;

constexpr int BM = kTileM;                         // A rows per CTA (M = 256 per pair)
constexpr int BN = 256;                            // MMA N (each CTA holds half of W's rows)
constexpr int KSUB = 2;                            // blocks of 128 of K per stage
constexpr int STAGES = 3;
constexpr int A_BYTES = BM * kBlock * KSUB;        // 32 KB
constexpr int B_BYTES = (BN / 2) * kBlock * KSUB;  // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 384;
constexpr int SLOTS = 4;
constexpr int SLOT_COLS = 3 * kScaleCols;          // A, W rows 0-127, W rows 128-255
constexpr int TMEM_COLS = 512;
constexpr int SCALE_COL = TMEM_COLS - SLOTS * SLOT_COLS;   // 464
constexpr int ACC1_COL = SCALE_COL - BN;                   // 208
constexpr int OUT_BUF_BYTES = 32 * 128;            // one 32-row, 128-byte box per warp
constexpr int STAGING_BYTES = 4 * OUT_BUF_BYTES;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + 1024 + 256;
constexpr uint32_t kIdesc = fp8::make_idesc(2 * BM, BN);
constexpr uint16_t kPairMask = 0x3;
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");
static_assert(BN - ACC1_COL <= 64, "the overlap lies in the part that the epilogue reads first");

template <bool kGated>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1,
                const __grid_constant__ CUtensorMap tmOut, Fp8Args args) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    const uint32_t staging = base + STAGES * STAGE_BYTES;
    const uint32_t bars = staging + STAGING_BYTES;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (STAGES + s); };
    auto sfull_bar = [&](int s) { return bars + 8u * (2 * STAGES + s); };
    auto sempty_bar = [&](int s) { return bars + 8u * (2 * STAGES + SLOTS + s); };
    const uint32_t tfull_bar = bars + 8u * (2 * STAGES + 2 * SLOTS);
    const uint32_t drained_bar = tfull_bar + 8u;    // the overlap of a tile has been read
    const uint32_t done_bar = tfull_bar + 16u;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + (done_bar + 8u - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* fills_out = reinterpret_cast<int*>(tmem_holder + 2);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();        // 0: issues the MMAs
    const uint32_t peer_abort = mapa_shared(smem_u32(tmem_holder + 1), rank ^ 1u);
    auto give_up = [&]() {   // a role that gives up stops both CTAs of the pair
        *abort_flag = 1;
        st_shared_cluster(peer_abort, 1u);
        set_status(args.hdr, MOE_ERR_TIMEOUT);
    };
    const int cluster = (int)blockIdx.x >> 1;
    const int n_clusters = (int)gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);     // even CTA's producer + both CTAs' bytes
            mbar_init(empty_bar(s), 1);    // the pair's MMA commit
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(sfull_bar(s), 8);    // 4 scale warps x 2 CTAs
            mbar_init(sempty_bar(s), 1);
        }
        mbar_init(tfull_bar, 1);
        mbar_init(drained_bar, 8);         // 4 epilogue warps x 2 CTAs
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        *fills_out = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&tmA);
        prefetch_map(&tmB0);
        if (kGated) prefetch_map(&tmB1);
        prefetch_map(&tmOut);
    }
    if (warp == 2) tmem_alloc_pair(smem_u32(tmem_holder), TMEM_COLS);
    fence_before();
    cluster_sync();   // barriers of both CTAs initialised, TMEM allocated
    fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_dep_wait();      // everything above overlaps the previous kernel
    grid_dep_launch();

    const fp8::OneGroup grp = args.group ? fp8::one_group(args) : fp8::OneGroup{0, 0};
    const int n_pairs = args.group ? (grp.n + 2 * BM - 1) / (2 * BM) : ld::i32_cg(&args.hdr->n_fat_tiles) >> 1;
    const int total = n_pairs * args.n_blocks_n;
    const int k_blocks = args.k_blocks;
    const int k_stages = (k_blocks + KSUB - 1) / KSUB;
    auto tile_at = [&](int w) {
        const int i = 2 * (w / args.n_blocks_n) + (int)rank;
        return args.group ? fp8::group_tile(grp, i) : args.tiles[i];
    };

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        const CUtensorMap* tmB = (kGated && rank == 1) ? &tmB1 : &tmB0;
        const uint32_t full0 = mapa_shared(full_bar(0), 0);   // even CTA's barriers
        int stage = 0;
        uint32_t phase = 0;
        int fills = 0;
        bool ok = true;
        FatTile ft_next = {};       // loaded one item ahead (its latency is hidden)
        if (cluster < total) ft_next = tile_at(cluster);
        for (int w = cluster; ok && w < total; w += n_clusters) {
            const FatTile ft = ft_next;
            if (w + n_clusters < total) ft_next = tile_at(w + n_clusters);
            const int nt = w % args.n_blocks_n;
            const int brow = ft.expert * args.n_rows + nt * (kGated ? BM : BN) +
                             (kGated ? 0 : (int)rank * BM);
            for (int ks = 0; ks < k_stages; ++ks) {
                if (!mbar_wait_for(empty_bar(stage), phase ^ 1u, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = base + stage * STAGE_BYTES;
                const uint32_t fb = full0 + 8u * stage;
                if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * STAGE_BYTES);
#pragma unroll
                for (int a = 0; a < KSUB; ++a) {
                    // a block past K is filled with zeros and not multiplied
                    const int kx = (ks * KSUB + a) * kBlock;
                    tma_load_2d_pair(sa + a * (A_BYTES / KSUB), &tmA, fb, kx, ft.row0);
                    tma_load_2d_pair(sa + A_BYTES + a * (B_BYTES / KSUB), tmB, fb, kx, brow);
                }
                ++fills;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && !*abort_flag) give_up();
        *fills_out = fills;
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---------------- MMA issuer (even CTA) ----------------
        int stage = 0, slot = 0;
        uint32_t phase = 0, sphase = 0;
        int it = 0;
        bool ok = true;
        bool issued = false;
        for (int w = cluster; ok && w < total; w += n_clusters, ++it) {
            const uint32_t d_tmem = tmem_base + (uint32_t)((it & 1) ? ACC1_COL : 0);
            for (int ks = 0; ks < k_stages; ++ks) {
                const int kb0 = ks * KSUB;
                const uint32_t sc = tmem_base + SCALE_COL + slot * SLOT_COLS;
                // (the fence below orders the scale stores before the MMAs)
                if (kb0 % kGroupBlocks == 0 &&
                    !mbar_wait_for(sfull_bar(slot), sphase, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                if (!mbar_wait_for(full_bar(stage), phase, args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                // Last, so that a tile's first operands are known to be there:
                // the previous tile's epilogue has read the overlap (and with
                // it, being in order, all of this buffer's previous tile).
                if (ks == 0 && it > 0 &&
                    !mbar_wait_for(drained_bar, (uint32_t)((it - 1) & 1), args.wait_cycles, abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t sa = base + stage * STAGE_BYTES;
#pragma unroll
                for (int a = 0; a < KSUB; ++a) {
                    const int kb = kb0 + a;
                    if (kb >= k_blocks) break;
                    const uint64_t ad = sw128_desc(sa + a * (A_BYTES / KSUB));
                    const uint64_t bd = sw128_desc(sa + A_BYTES + a * (B_BYTES / KSUB));
                    const uint32_t idesc = fp8::with_scale_byte(kIdesc, kb % kGroupBlocks);
#pragma unroll
                    for (int kk = 0; kk < kBlock / 32; ++kk)   // +32 bytes per K step
                        fp8::mma_pair(d_tmem, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc,
                                      sc, sc + kScaleCols, (kb > 0 || kk > 0) ? 1u : 0u);
                }
                issued = true;
                commit_pair_multicast(empty_bar(stage), kPairMask);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (kb0 % kGroupBlocks == kGroupBlocks - KSUB || ks == k_stages - 1) {
                    commit_pair_multicast(sempty_bar(slot), kPairMask);
                    if (++slot == SLOTS) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
            }
            if (!ok) break;
            commit_pair_multicast(tfull_bar, kPairMask);
        }
        if (!ok && !*abort_flag) give_up();
        // Every MMA has completed before TMEM is freed.  Also where this loop
        // ran to its end: an epilogue may have given up on the last tile.
        if (issued) {
            commit_pair_multicast(done_bar, 0x1);
            (void)mbar_wait(done_bar, 0);
        }
    } else if (warp >= 8) {
        // ---------------- scale producers (both CTAs) ----------------
        // Lane l holds rows l, l + 32, l + 64, l + 96 of this CTA's A tile
        // (TMEM columns 0-3 of the slot); every 128 rows of W share one word.
        const uint32_t tscale = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + SCALE_COL;
        const uint32_t sfull0 = mapa_shared(sfull_bar(0), 0);
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        const int groups = (k_blocks + kGroupBlocks - 1) / kGroupBlocks;
        const int last = args.n_rows / kBlock - 1;   // N is a multiple of 128, not of 256
        for (int w = cluster; ok && w < total; w += n_clusters) {
            const FatTile ft = tile_at(w);
            const int nt = w % args.n_blocks_n;
            const uint8_t* ra[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // rows past the tile's only scale rows of D that are not stored
                const int r = min(ft.row0 + lane + 32 * i, args.rows - 1);
                ra[i] = args.a_scales + (int64_t)r * k_blocks;
            }
            const int64_t eb = (int64_t)ft.expert * (args.n_rows / kBlock);
            const uint8_t* rb0 =
                args.b0_scales + (eb + (kGated ? nt : min(2 * nt, last))) * k_blocks;
            const uint8_t* rb1 =
                kGated ? args.b1_scales + (eb + nt) * k_blocks
                       : args.b0_scales + (eb + min(2 * nt + 1, last)) * k_blocks;
            for (int g = 0; g < groups; ++g) {
                uint32_t a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = fp8::scale_word(ra[i], g, k_blocks);
                const uint32_t b0 = fp8::scale_word(rb0, g, k_blocks);
                const uint32_t b1 = fp8::scale_word(rb1, g, k_blocks);
                if (!__all_sync(0xffffffffu, mbar_wait_for(sempty_bar(slot), phase ^ 1u,
                                                           args.wait_cycles, abort_flag))) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t t = tscale + slot * SLOT_COLS;
                tmem_st4(t, a[0], a[1], a[2], a[3]);
                tmem_st4(t + kScaleCols, b0, b0, b0, b0);
                tmem_st4(t + 2 * kScaleCols, b1, b1, b1, b1);
                tmem_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_tmem(sfull0 + 8u * slot);
                if (++slot == SLOTS) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0 && !*abort_flag) give_up();
    } else if (warp >= 4 && warp < 8) {
        // ---------------- epilogue (both CTAs) ----------------
        const int ew = warp - 4;              // TMEM lanes 32*ew .. 32*ew+31
        const int row = ew * 32 + lane;
        const uint32_t buf = staging + (uint32_t)ew * OUT_BUF_BYTES;
        const uint32_t drained0 = mapa_shared(drained_bar, 0);
        bool stored = false;                  // a tensor store of this warp may read buf
        int it = 0;
        FatTile ft_next = {};
        if (cluster < total) ft_next = tile_at(cluster);
        // Row `lane` of a 32 x 128-byte box: 16-byte chunk j at chunk
        // j ^ (row mod 8) (128-byte swizzle), then one tensor store.
        auto store_box = [&](const uint32_t (&v)[32], int x, int y) {
            if (lane == 0 && stored) bulk_wait_read<0>();
            __syncwarp();
            const uint32_t rb = buf + (uint32_t)lane * 128u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                st_shared_v4(rb + ((uint32_t)(j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1],
                             v[4 * j + 2], v[4 * j + 3]);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(&tmOut, buf, x, y);
                bulk_commit();
            }
            __syncwarp();
            stored = true;
        };
        for (int w = cluster; w < total; w += n_clusters, ++it) {
            const FatTile ft = ft_next;
            if (w + n_clusters < total) ft_next = tile_at(w + n_clusters);
            const int nt = w % args.n_blocks_n;
            const bool valid = row < ft.rows;
            const bool whole = ew * 32 + 32 <= ft.rows;   // else each valid lane stores its row
            const int odd = it & 1;
            const int64_t out_row = (int64_t)ft.row0 + row;
            const uint32_t taddr =
                tmem_base + ((uint32_t)(ew * 32) << 16) + (uint32_t)(odd ? ACC1_COL : 0);
            // the 64 columns that hold those shared with the other buffer
            const uint32_t shared_cols = taddr + (odd ? 0u : (uint32_t)(BN - 64));
            // the whole warp decides together (tcgen05.ld below is warp-wide)
            if (!__all_sync(0xffffffffu, mbar_wait_for(tfull_bar, (uint32_t)(it & 1),
                                                       args.wait_cycles, abort_flag))) {
                if (!*abort_flag) give_up();
                break;
            }
            fence_after();
            // They are read before anything else: the next tile's MMAs wait for
            // this (2,500 cycles per tile, 197 us in place of 184, when the
            // epilogue did its first quarter first and released with cluster
            // scope).
            uint32_t early[64];
            tmem_ld32(shared_cols, *reinterpret_cast<uint32_t(*)[32]>(early));
            tmem_ld32(shared_cols + 32, *reinterpret_cast<uint32_t(*)[32]>(early + 32));
            tmem_ld_wait();
            auto drained = [&]() {   // the columns shared with the other buffer have been read
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_tmem(drained0);
                __syncwarp();   // converged for the warp-wide TMEM loads that follow
            };
            drained();
            if (kGated) {
                // The columns read are the up values of features 64-127 (buffer
                // 0) or the gate values of 0-63 (buffer 1).  Those 64 features
                // stay in registers until the row's maximum is known; the
                // other 64 are computed for the maximum and once more after
                // it, which keeps the kernel within 168 registers.
                const int first = odd ? 0 : 64;
                float h[64], x[32];
                float m = 0.f;
                auto features = [&](int f, float* dst) {
                    uint32_t g[32], u[32];
                    tmem_ld32(taddr + f, g);
                    tmem_ld32(taddr + 128 + f, u);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        dst[q] = fp8::swiglu(__uint_as_float(g[q]), __uint_as_float(u[q]));
                };
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(taddr + (odd ? 128 : 0) + first + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        h[c + q] = fp8::swiglu(__uint_as_float(odd ? early[c + q] : o[q]),
                                               __uint_as_float(odd ? o[q] : early[c + q]));
                }
#pragma unroll
                for (int q = 0; q < 64; ++q) m = fmaxf(m, fp8::finite_abs(h[q]));
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    features((first ^ 64) + c, x);
#pragma unroll
                    for (int q = 0; q < 32; ++q) m = fmaxf(m, fp8::finite_abs(x[q]));
                }
                const uint32_t sb = fp8::scale_byte(m);
                const float inv = fp8::inverse_scale(sb);
                uint32_t mine[16], rest[16];   // 64 features each, in the order read
                auto pack = [&](const float* p, uint32_t* o) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        o[q] = fp8::pack_e4m3x4(fp8::scaled(p[4 * q], inv), fp8::scaled(p[4 * q + 1], inv),
                                                fp8::scaled(p[4 * q + 2], inv), fp8::scaled(p[4 * q + 3], inv));
                };
                pack(h, mine);
                pack(h + 32, mine + 8);
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    features((first ^ 64) + c, x);
                    pack(x, rest + c / 4);
                }
                uint32_t v[32];
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    v[q] = odd ? mine[q] : rest[q];
                    v[16 + q] = odd ? rest[q] : mine[q];
                }
                if (whole) {
                    store_box(v, nt * kBlock, ft.row0 + ew * 32);
                } else if (valid) {
                    uint4* d4 = reinterpret_cast<uint4*>(args.out_q + out_row * args.ld_out +
                                                         (int64_t)nt * kBlock);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        d4[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
                if (valid) args.out_scales[out_row * (args.ld_out / kBlock) + nt] = (uint8_t)sb;
                __syncwarp();
            } else {
                const int cols = (int)min((int64_t)BN, args.ld_out - (int64_t)nt * BN);
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    // 64 columns at a time, the ones already read first
                    const int c = odd ? 64 * i : 64 * ((i + 3) & 3);
                    if (i > 0) {
                        tmem_ld32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(early));
                        tmem_ld32(taddr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(early + 32));
                        tmem_ld_wait();
                    }
                    uint32_t v[32];
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        v[q] = pack_bf16(__uint_as_float(early[2 * q]), __uint_as_float(early[2 * q + 1]));
                    if (c >= cols) continue;
                    if (whole) {
                        store_box(v, nt * BN + c, ft.row0 + ew * 32);
                    } else if (valid) {
                        uint4* d4 = reinterpret_cast<uint4*>(args.out + out_row * args.ld_out +
                                                             (int64_t)nt * BN + c);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            d4[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) bulk_wait_all();   // every tensor store completed
        __syncwarp();
    }

    fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' roles have stopped
    // Both CTAs read the same two flags here, so they agree on the drain.  The
    // barrier after it keeps a CTA from exiting while a slower warp of its
    // peer still reads its shared memory (a fault of the whole launch).
    const bool aborted = *abort_flag || ld_shared_cluster(peer_abort) != 0;
    cluster_sync();
    if (aborted) {
        if (rank == 0 && threadIdx.x == 0)
            drain_pair<STAGES>(full_bar(0), *fills_out,
                               (int)ld_shared_cluster(mapa_shared(smem_u32(fills_out), 1)),
                               (uint32_t)STAGE_BYTES);
        cluster_sync();
    }
    if (warp == 2) {
        fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

template <bool kGated>
cudaError_t set_smem_attr() {
    static std::atomic<int> done[kMaxDevices];
    return smem_limit_once(fp8_pair_kernel<kGated>, SMEM_BYTES, done);
}

template <bool kGated>
cudaError_t launch(const uint8_t* a, int64_t rows, const uint8_t* b0, const uint8_t* b1,
                   const Fp8Args& args, int E, int num_sms, cudaStream_t s) {
    const uint64_t K = (uint64_t)args.k_blocks * kBlock, n = (uint64_t)E * args.n_rows;
    CUtensorMap mA, mB0, mB1, mO;
    cudaError_t e;
    if ((e = make_tma_map_u8(&mA, a, (uint64_t)rows, K, BM)) != cudaSuccess) return e;
    if ((e = make_tma_map_u8(&mB0, b0, n, K, 128)) != cudaSuccess) return e;
    if ((e = make_tma_map_u8(&mB1, b1, n, K, 128)) != cudaSuccess) return e;
    e = kGated ? make_tma_map_u8(&mO, args.out_q, (uint64_t)rows, (uint64_t)args.ld_out, 32)
               : make_tma_map_bf16(&mO, args.out, (uint64_t)rows, (uint64_t)args.ld_out, 32);
    if (e != cudaSuccess) return e;
    if ((e = set_smem_attr<kGated>()) != cudaSuccess) return e;
    int grid = 0;
    if ((e = pair_grid<fp8_pair_kernel<kGated>, SMEM_BYTES, THREADS>(num_sms, &grid)) != cudaSuccess) return e;
    return launch_pdl(fp8_pair_kernel<kGated>, dim3(grid), dim3(THREADS), SMEM_BYTES, s, mA, mB0, mB1,
                      mO, args);
}

}  // namespace

cudaError_t launch_fp8_pair_gate_up(const uint8_t* a, int64_t rows, const uint8_t* b0,
                                    const uint8_t* b1, const Fp8Args& args, int E, int num_sms,
                                    cudaStream_t s) {
    return launch<true>(a, rows, b0, b1, args, E, num_sms, s);
}
cudaError_t launch_fp8_pair(const uint8_t* a, int64_t rows, const uint8_t* b, const Fp8Args& args,
                            int E, int num_sms, cudaStream_t s) {
    return launch<false>(a, rows, b, b, args, E, num_sms, s);
}

}  // namespace moe
