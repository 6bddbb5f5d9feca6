// w4a16.cu -- the weight-only linear layer: BF16 / FP16 rows times NVFP4 weights (sm_100a).
//
// [CAL] layer table (W4A16 layers keep their activations in 16 bits); [FLOW] 3.4 (the value of a
// code is e2m1 * s_b * s2).  y[t, n] = s2 * sum_k x[t, k] * (e2m1(q[n, k]) * e4m3(s[n, k/16])):
// the weight products are exact, the sum runs in FP32, s2 is applied to the sum.
//
// One CTA per SM; a cluster of z of them owns a contiguous range of weight rows (balanced to one
// row) and splits K, each CTA taking its chunks of it: staging the token rows costs a CTA
// T * K / z values, so z grows with T * K.  A CTA walks its rows in tiles of at most 16; its 16
// warps split the tiles and, within a tile, K (nv4_w4.cuh).  A weight byte is read once; the
// cluster's partial sums meet through distributed shared memory, added in rank order.
// Bound: one token pays its latencies (launch, staging, first loads, one reduction: 1 x 2048 x 2048
// 6.2 us alone, 4.2 between others); 5 x 2048 x 16384 takes 12.4 us for 18.9 MB (15 us from a cold L2,
// issue slots 40% busy): six steps per warp do not cover what a launch costs before and after them.
#include "nv4_async.cuh"
#include "nv4_internal.h"
#include "nv4_split.h"
#include "nv4_w4.cuh"

namespace nv4 {

namespace w4 {

struct LinearParams {
    const void* x;
    int64_t ldx;
    const uint8_t* q;
    const uint8_t* sc;
    const float* d_s2;
    void* out;
    int64_t ldd;
    uint32_t T, N, K;
    uint32_t z, xs_bytes, red_bytes;              // cluster size; shared memory of token rows, of warp sums
    uint32_t tile, ntile, wk;                     // rows per tile, tiles per cluster, warps per tile
    uint32_t* d_flags;
};

template <int kDt, int kOut, bool kVec, int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Rows rows;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
    uint4* xs = reinterpret_cast<uint4*>(smem + kRing);
    float* red = reinterpret_cast<float*>(smem + kRing + p.xs_bytes);          // [2][16 warps][16][8 NT]
    float* part = red + p.red_bytes / sizeof(float);                           // [rows][8 NT], z > 1
    constexpr uint32_t kTile = 16u * 8u * NT;
    const uint32_t rank = p.z > 1u ? cluster_ctarank() : 0u;
    const uint32_t clu = blockIdx.x / p.z, nclu = gridDim.x / p.z;
    const uint32_t r0 = (uint32_t)((uint64_t)clu * p.N / nclu);
    const uint32_t R = (uint32_t)((uint64_t)(clu + 1u) * p.N / nclu) - r0, ntile = p.ntile;
    const uint32_t all = (p.K + kChunk - 1u) / kChunk;
    const uint32_t ch0 = rank * all / p.z, nch = (rank + 1u) * all / p.z - ch0;
    const uint32_t kb = ch0 * kChunk, kn = min(p.K, kb + nch * kChunk) - kb;   // this CTA's K range
    const uint32_t wk = p.wk, groups = kWarps / wk;
    const uint32_t grp = warp / wk, wig = warp - grp * wk;
    const float s2 = *p.d_s2;
    const uint32_t my_tiles = grp < ntile ? (ntile - grp + groups - 1u) / groups : 0u;
    const uint32_t my_chunks = wig < nch ? (nch - wig + wk - 1u) / wk : 0u, steps = my_tiles * my_chunks;

    const uint32_t m = p.T;
    uint32_t lt = grp, lc = wig;                  // the step to load next
    Rows16 rw;
    bool moved = true;
    auto load = [&](uint8_t* slot) {
        if (moved) {
            const uint32_t a = r0 + lt * p.tile, n = min(p.tile, r0 + R - min(a, r0 + R));
            const size_t row = (size_t)(a + g) * (p.K / 2u), row8 = row + (size_t)8u * (p.K / 2u);
            rw.set(p.q + row, p.sc + row / 8u, p.q + row8, p.sc + row8 / 8u, g < n, g + 8u < n);
            moved = false;
        }
        load_chunk<kVec>(slot, rw, ch0 + lc, p.K);
        lc += wk;
        if (lc >= nch) {
            lc = wig;
            lt += groups;
            moved = true;
        }
    };
    Ring ring;
    ring.begin(smem + warp * (kDepth * kSlot), steps, load);
    const bool wide = stage_tokens<kDt>(xs, rows, m, kn, [&](uint32_t i) {
        return static_cast<const void*>(static_cast<const uint16_t*>(p.x) + (int64_t)i * p.ldx + kb);
    });
    Acc<NT> acc;
    clear<NT>(acc);
    NonFinite odd;                                // among the outputs before they are rounded
    uint32_t ut = grp, uc = wig, buf = 0u;        // the step to multiply next
    ring.run(load, [&](const uint8_t* slot) {
        const uint4* xc = xs + (size_t)uc * 32u * m;
        if (kDt == 0 && wide) mma_chunk<true, NT>(acc, slot, xc, m);
        else mma_chunk<false, NT>(acc, slot, xc, m);
        uc += wk;
        if (uc < nch) return;
        // the tile's end: the group adds its warps' sums, one (token, row) per thread
        put_part<NT>(red + (size_t)(buf * kWarps + warp) * kTile, acc, g, t);
        clear<NT>(acc);
        group_barrier(grp, wk);
        const uint32_t a = ut * p.tile, nr = a < R ? min(p.tile, R - a) : 0u;
        const float* first = red + (size_t)(buf * kWarps + grp * wk) * kTile;
        for (uint32_t i = wig * 32u + lane; i < 16u * m; i += 32u * wk) {
            const uint32_t r = i & 15u, tok = i >> 4;
            if (r >= nr) continue;
            const float s = sum_parts<kTile>(first + r * (8 * NT) + tok, wk);
            if (p.z > 1u) part[(size_t)(a + r) * (8 * NT) + tok] = s * rows.descale[tok];
            else {
                const float y = s * s2 * rows.descale[tok];
                odd.see(y);
                store_out<kOut>(p.out, (int64_t)tok * p.ldd + r0 + a + r, y);
            }
        }
        buf ^= 1u;
        uc = wig;
        ut += groups;
    });
    if (p.z > 1u) {
        cluster_sync();
        const uint32_t n = R * m, i1 = (uint32_t)((uint64_t)(rank + 1u) * n / p.z);
        for (uint32_t i = (uint32_t)((uint64_t)rank * n / p.z) + threadIdx.x; i < i1; i += kThreads) {
            const uint32_t tok = i / R, r = i - tok * R;
            float v[8], s = 0.0f;
#pragma unroll
            for (uint32_t q = 0; q < 8u; ++q) v[q] = q < p.z ? ld_dsmem_f32(part + (size_t)r * (8 * NT) + tok, q) : 0.0f;
#pragma unroll
            for (uint32_t q = 0; q < 8u; ++q) s += v[q];
            odd.see(s * s2);
            store_out<kOut>(p.out, (int64_t)tok * p.ldd + r0 + r, s * s2);
        }
        cluster_sync();                           // the others' sums have been read
    }
    const uint32_t flags = __reduce_or_sync(0xFFFFFFFFu, odd.flag());
    if (lane == 0u) flag_or(p.d_flags, flags);
}

template <int kDt, int kOut, bool kVec, int NT>
static cudaError_t run_linear(LinearParams p, cudaStream_t s)
{
    auto kern = linear_kernel<kDt, kOut, kVec, NT>;
    static bool ready[64] = {};
    static int fits[64][kMaxSplit + 1] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 64;
    if (!known || !ready[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmemW4);
        if (e != cudaSuccess) return e;
        if (known) ready[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.z;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.z > 1u ? 1 : 0;
    const uint32_t n = clusters_at_once(kern, kThreads, kMaxSmemW4, p.z, fits, dev);
    p.red_bytes = 2u * kWarps * 16u * 8u * NT * (uint32_t)sizeof(float);
    const size_t fixed = kRing + (size_t)p.xs_bytes + p.red_bytes;
    uint32_t nclu = p.N < n ? p.N : n;
    if (p.z > 1u) {                               // more clusters than run at once if their sums need it
        const uint32_t fit = (uint32_t)((kMaxSmemW4 - fixed) / (8u * NT * sizeof(float)));
        if ((p.N + fit - 1u) / fit > nclu) nclu = (p.N + fit - 1u) / fit;
    }
    const uint32_t most = (p.N + nclu - 1u) / nclu;
    p.ntile = (most + 15u) / 16u;
    p.tile = (most + p.ntile - 1u) / p.ntile;
    p.wk = split_of(p.ntile, (p.K + kChunk - 1u) / kChunk / p.z);
    const size_t smem = fixed + (p.z > 1u ? (size_t)most * 8u * NT * sizeof(float) : 0u);
    cfg.gridDim = dim3(nclu * p.z, 1, 1);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int kDt, int kOut>
static cudaError_t pick_linear(const LinearParams& p, bool vec, cudaStream_t s)
{
    if (vec) return p.T <= 8u ? run_linear<kDt, kOut, true, 1>(p, s) : run_linear<kDt, kOut, true, 2>(p, s);
    return p.T <= 8u ? run_linear<kDt, kOut, false, 1>(p, s) : run_linear<kDt, kOut, false, 2>(p, s);
}

struct Staging {
    uint32_t z, bytes;                            // cluster size, shared memory of a CTA's token rows
    bool fits;
};

static Staging staging_of(int64_t T, int64_t K)
{
    const uint32_t nch = (uint32_t)((K + kChunk - 1) / kChunk), t = (uint32_t)T;
    uint32_t z = 1u;
    // split K until a CTA stages 128 chunks of token rows, as long as it keeps two chunks (5 x 2048 x
    // 16384: 23.7 us unsplit, 11.4 us in clusters of 4; 4 x 2048 x 2048: 4.4 us unsplit, 5.4 split)
    while (z < 8u && t * nch > 128u * z && nch >= 4u * z) z *= 2u;
    const uint32_t bytes = t * ((nch + z - 1u) / z * 512u);
    // per 8 tokens: the warps' sums, twice, and a cluster's sums of at least 256 rows
    const size_t sums = (2u * kWarps * 128u + 2048u) * sizeof(float);
    return {z, bytes, kRing + (size_t)bytes + ((t + 7u) / 8u) * sums <= kMaxSmemW4};
}

}  // namespace w4

bool few_rows_w4a16(int64_t T, int64_t K) { return T <= kMaxFewRows && w4::staging_of(T, K).fits; }

cudaError_t launch_linear_w4a16(const void* x, int dt, int64_t T, int64_t K, int64_t ldx, const uint8_t* q,
                                const uint8_t* sc, const float* d_s2, int64_t N, int out_dt, void* out, int64_t ldd,
                                uint32_t* d_flags, cudaStream_t s)
{
    using namespace w4;
    const Staging st = staging_of(T, K);
    const LinearParams p{x, ldx, q, sc, d_s2, out, ldd, (uint32_t)T, (uint32_t)N, (uint32_t)K, st.z, st.bytes, 0u, 0u, 0u, 0u,
                         d_flags};
    const bool vec = K % 64 == 0;                                  // (the scales are 16-byte aligned)
    if (dt == 0)
        return out_dt == 0 ? pick_linear<0, 0>(p, vec, s)
                           : out_dt == 1 ? pick_linear<0, 1>(p, vec, s) : pick_linear<0, 2>(p, vec, s);
    return out_dt == 0 ? pick_linear<1, 0>(p, vec, s)
                       : out_dt == 1 ? pick_linear<1, 1>(p, vec, s) : pick_linear<1, 2>(p, vec, s);
}

}  // namespace nv4
