// nv4_split.h -- how many CTAs of a cluster share a tile of a product by splitting its K (host).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "nv4_internal.h"

namespace nv4 {

constexpr uint32_t kMaxSplit = 8;                 // the portable cluster size

// Clusters of z CTAs of a kernel that run at once, one CTA per SM.  The device's units hold
// different numbers of SMs, so it is not SMs / z: on 148 SMs 74 clusters of 2, 33 of 4, 22 of 6 and
// 15 of 8.  Remembered in fits, [device][z], which belongs to the kernel.
template <class Kern>
static uint32_t clusters_at_once(Kern kern, int threads, size_t smem, uint32_t z, int (&fits)[64][kMaxSplit + 1], int dev)
{
    const bool known = dev >= 0 && dev < 64;
    if (known && fits[dev][z] > 0) return (uint32_t)fits[dev][z];
    int n = num_sms() / (int)z;
    if (z > 1u) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((uint32_t)n * z, 1, 1);
        cfg.blockDim = dim3((uint32_t)threads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = z;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int m = 0;
        if (cudaOccupancyMaxActiveClusters(&m, kern, &cfg) == cudaSuccess && m > 0) n = m < n ? m : n;
        else (void)cudaGetLastError();
    }
    if (n < 1) n = 1;
    if (known) fits[dev][z] = n;
    return (uint32_t)n;
}

// The split z with the least waves x (steps of a CTA + overhead), overhead being what a wave costs
// beside its steps, in steps; the smaller z where two are equal.  Every CTA keeps `least` steps.
// (By SMs / z alone 16 tiles went to clusters of 8, the last of them in a wave of its own.)
template <class Kern>
static uint32_t split_tiles(Kern kern, int threads, size_t smem, uint32_t tiles, uint32_t steps, uint32_t least,
                            uint32_t overhead, int (&fits)[64][kMaxSplit + 1], int dev)
{
    uint32_t best = 1u;
    uint64_t cost = ~0ull;
    for (uint32_t z = 1u; z <= kMaxSplit && (z == 1u || steps >= least * z); ++z) {
        const uint32_t n = clusters_at_once(kern, threads, smem, z, fits, dev);
        const uint64_t c = (uint64_t)((tiles + n - 1u) / n) * ((steps + z - 1u) / z + overhead);
        if (c < cost) {
            cost = c;
            best = z;
        }
    }
    return best;
}

}  // namespace nv4
