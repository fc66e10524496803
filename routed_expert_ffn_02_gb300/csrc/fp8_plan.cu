// fp8_plan.cu -- the tile lists of the 8-bit products from group offsets.
#include "ld_dev.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

// Tile lists over group offsets alone, checked: offset e becomes the largest
// of offsets 0..e, inside [0, rows], so the groups never overlap and the
// lists never hold more rows than exist.  A thread per group; one scan of the
// three list lengths packed into 64 bits (pair tiles, solo, thin) and of the
// running maximum, so the block is no wider than the groups need.
__global__ void __launch_bounds__(1024)
plan_groups_kernel(const int32_t* __restrict__ offsets, int rows, int E, Plan plan) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ int off[kMaxE + 1];
    __shared__ int warp_max[32];
    __shared__ unsigned long long warp_sum[32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int e = threadIdx.x;
    const int given = e < E ? ld::i32(offsets + e) : 0, end = ld::i32(offsets + E);
    int v = min(max(given, 0), rows);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, u);
    }
    if (lane == 31) warp_max[w] = v;
    __syncthreads();
    for (int i = 0; i < w; ++i) v = max(v, warp_max[i]);
    if (e < E) off[e] = v;
    if (e == E - 1) off[E] = max(v, min(max(end, 0), rows));
    if ((e < E && v != given) || (e == 0 && (given != 0 || end != rows)))
        set_status(plan.hdr, MOE_ERR_BAD_INDEX);
    __syncthreads();
    const int c = e < E ? off[e + 1] - off[e] : 0;
    const int tiles = c > kTileM ? 2 * ((c + 2 * kTileM - 1) / (2 * kTileM)) : 0;
    const bool solo = c > kThinMaxTokens && c <= kTileM, thin = c > 0 && c <= kThinMaxTokens;
    const unsigned long long mine =
        (unsigned long long)tiles | (unsigned long long)solo << 32 | (unsigned long long)thin << 48;
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum[w] = incl;
    __syncthreads();
    unsigned long long before = incl - mine, total = 0;
    for (int i = 0; i < warps; ++i) {
        if (i < w) before += warp_sum[i];
        total += warp_sum[i];
    }
    FatTile ft;
    ft.expert = e;
    ft.pad = 0;
    for (int i = 0; i < tiles; ++i) {
        ft.row0 = v + i * kTileM;
        ft.rows = max(0, min(kTileM, c - i * kTileM));
        plan.tiles[(uint32_t)before + i] = ft;
    }
    ft.row0 = v;
    ft.rows = c;
    if (solo) plan.solo_tiles[(before >> 32) & 0xffff] = ft;
    if (thin) plan.mma_tiles[before >> 48] = ft;
    if (e == 0) {
        plan.hdr->n_fat_tiles = (int)(uint32_t)total;
        plan.hdr->n_solo = (int)((total >> 32) & 0xffff);
        plan.hdr->n_thin_mma = (int)(total >> 48);
    }
}

}  // namespace

cudaError_t launch_plan_groups(const int32_t* offsets, int rows, int E, const Plan& plan,
                               cudaStream_t s) {
    return launch_pdl(plan_groups_kernel, dim3(1), dim3((E + 31) / 32 * 32), 0, s, offsets, rows, E,
                      plan);
}

}  // namespace moe
