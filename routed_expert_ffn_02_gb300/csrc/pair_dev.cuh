// pair_dev.cuh -- what the grouped GEMMs on CTA pairs share: draining a
// pair's copies after an abort, and the grid of resident pairs.
#pragma once

#include <algorithm>
#include <mutex>

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

// Stage rounds filled into stage s by a producer that filled `fills` stages
// in ring order.
template <int kStages>
__device__ __forceinline__ int rounds_filled(int fills, int s) {
    return fills > s ? (fills - s + kStages - 1) / kStages : 0;
}

// After an abort, run by one thread of the even CTA once both CTAs' roles
// have stopped (fills_even / fills_odd: the stages each CTA's producer
// filled).  Every round of a stage that either CTA filled completes on the
// even CTA's full barrier; the two producers differ by at most one round per
// stage (a round needs the previous one consumed, which needs both CTAs'
// bytes).  A round only the odd CTA filled is armed here for its bytes; a
// round only the even CTA filled is credited the odd CTA's missing bytes.
// Then each last round is waited for with the full bound, so every copy of
// both CTAs has landed.
template <int kStages>
__device__ __forceinline__ void drain_pair(uint32_t full0, int fills_even, int fills_odd,
                                           uint32_t stage_bytes) {
    for (int s = 0; s < kStages; ++s) {
        const uint32_t bar = full0 + 8u * s;
        const int re = rounds_filled<kStages>(fills_even, s) - 1, ro = rounds_filled<kStages>(fills_odd, s) - 1;
        if (re < 0 && ro < 0) continue;
        if (ro == re + 1) {
            if (re >= 0) (void)ptx::mbar_wait(bar, (uint32_t)(re & 1));
            ptx::mbar_expect_tx(bar, stage_bytes);
            (void)ptx::mbar_wait(bar, (uint32_t)(ro & 1));
        } else if (re == ro + 1) {
            ptx::mbar_complete_tx(bar, stage_bytes);
            (void)ptx::mbar_wait(bar, (uint32_t)(re & 1));
        } else {
            (void)ptx::mbar_wait(bar, (uint32_t)(re & 1));
        }
    }
}

// CTAs to launch: two per co-resident cluster (an SM pair whose partner is
// busy or absent cannot host a cluster, so this can be below the SM count).
template <auto kKernel, int kSmemBytes, int kThreads = 256>
cudaError_t pair_grid(int num_sms, int* grid) {
    constexpr int kMaxDev = kMaxDevices;
    static int cached[kMaxDev] = {};
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    if (!cached[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms & ~1), 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmemBytes;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, kKernel, &cfg);
        if (e != cudaSuccess) return e;
        if (clusters < 1) return cudaErrorInvalidConfiguration;
        cached[dev] = 2 * std::min(clusters, num_sms / 2);
    }
    *grid = cached[dev];
    return cudaSuccess;
}

}  // namespace moe
