// gemm.cu -- NVFP4 x NVFP4 block-scaled GEMM on the 5th-generation tensor cores (sm_100a).
//
// [FP4] section 4.1 (block-scaled FP4 matrix multiply with tcgen05.mma and scale
// factors reorganized for it), [CAST] section 4 (W4A4: activations and weights both
// NVFP4).  D[m, n] = s2_A * s2_B * sum_k (e2m1(a_mk) * sA[m, k/16]) * (e2m1(b_nk) * sB[n, k/16]),
// i.e. the product of the two dequantized matrices, accumulated in FP32 and written
// as BF16 or FP32.
//
// Kernel structure: persistent, one CTA per SM walking the 128 x kBN output tiles
// t = blockIdx.x, + gridDim.x, ... (kBN = 256 when N allows, else 128); 448 threads:
//   * warp 8, one lane: producer.  Per stage of 256 K-elements it loads the A and B code
//     tiles (128 rows x 128 bytes each) with 2-D TMA into 128-byte-swizzled shared
//     memory, and the stage's scale-factor atoms (4 x 512 bytes per operand, already in
//     the MMA layout, see nv4_scales_to_mma_layout) with 1-D bulk copies, all completing
//     on the stage's mbarrier.  A 4-stage ring that runs across tiles: while the epilogue
//     drains one tile, the first stages of the next are already loading.  A stage is
//     reused once the MMAs that read it have completed (tcgen05.commit on "empty").
//   * warps 4-7: scale writers, one per 32-lane tensor-memory sub-partition.  The
//     block-scaled MMA reads a K-step's scale factors from every sub-partition, so each
//     writer stores the stage's atoms into its own 32 lanes with tcgen05.st (48 or 32
//     columns per stage into one of kSfBufs buffers) and arrives on "sf_full".  Moving the
//     scales with tcgen05.st from four warps, instead of twelve tcgen05.cp 32x128b.warpx4
//     copies per stage issued by the MMA thread, takes the copies out of the tensor pipe's
//     instruction stream (8192^3: 2.85 -> 4.03 PFLOP/s; the copies cost per instruction,
//     not per byte).
//   * warp 9: allocates the tensor memory (the 128 x kBN FP32 accumulator and the scale
//     buffers); all its lanes wait until the epilogue has read the previous tile's accumulator
//     ("acc_empty") and per stage for the codes and the scales; an elected one issues four
//     tcgen05.mma kind::mxf4nvf4 block16 (K = 64 each) with both operands read from shared
//     memory through matrix descriptors, commits "empty" and "sf_free", and commits
//     "acc_full" after the tile's last stage.
//   * warps 0-3 and 10-13: epilogue, two warps per 32-lane sub-partition, half the columns
//     each.  A warp reads its 32 rows x kBN/2 accumulator columns with tcgen05.ld (one row
//     per thread), multiplies by s2_A * s2_B and arrives on acc_empty; for BF16 the half
//     row is converted into registers first and stored only after the accumulator has been
//     released, so the stores overlap the next tile's MMAs, each 32 x 16 block transposed
//     through 1 KB of shared memory so that a store instruction writes 16 rows x 32
//     contiguous bytes instead of 32 rows x 16.
// The accumulator is single-buffered (a second 256-column one does not fit the 512 columns
// next to the scale buffers): the tensor pipe idles while the epilogue reads it.
//
// When M and N are multiples of 256 the product runs on CTA pairs instead (the kernel
// gemm_pair_kernel below: 256 x 256 tiles, the 2-SM MMA): 8192^3 +2%, 16384 x 16384 x
// 2048 +7%.  Its cross-CTA hand-offs use plain (CTA-scope) mbarrier waits and remote
// arrives: with cluster-scope acquire/release on them the same kernel ran 40% slower.
// The pair kernel also multiplies MXFP4 operands (kMx: kind::mxf4 block32, E8M0 scales, any M and N; 16384
// x 16384 x 2048 in 325 us, 3.4 PFLOP/s); products of few rows or few tiles are gemm_mx.cu's.
// Every mbarrier wait is bounded (kWaitLimitNs); on expiry the kernel sets
// NV4_FLAG_TIMEOUT, every role stops, the stores are skipped, copies in flight are
// drained and the tensor memory is released.
#include "nv4_async.cuh"
#include "nv4_common.cuh"
#include "nv4_internal.h"
#include "nv4_tcgen05.cuh"
#include "nv4_tensormap.h"

namespace nv4 {

namespace gemm {

using namespace tc;

constexpr int kBM = 128;
constexpr int kBK = 256;                          // FP4 elements per stage (128 bytes per row)
constexpr int kStages = 4;
constexpr int kSfBufs = 4;                        // scale-factor buffers in tensor memory
constexpr int kThreads = 448;                     // warps 0-3, 10-13 epilogue, 4-7 scale writers, 8 producer, 9 MMA issuer
constexpr int kProducer = 256, kIssuer = 288;     // the two single-thread roles

// Tile width kBN = 128 or 256 (one MMA of 128 x kBN x 64 per K-step).
template <int kBN>
struct Cfg {
    static constexpr uint32_t kATile = 128 * 128;                    // A codes per stage
    static constexpr uint32_t kBTile = kBN * 128;                    // B codes per stage
    static constexpr uint32_t kSfA = 4 * 512;                        // 4 K-steps x one 128-row atom
    static constexpr uint32_t kSfB = (kBN / 128) * 4 * 512;
    static constexpr uint32_t kStageTx = kATile + kBTile + kSfA + kSfB;
    static constexpr uint32_t kTmemCols = kBN == 128 ? 256 : 512;   // power of two >= accumulator + scales
    static constexpr uint32_t kSfBCols = 16 * (kBN / 128);           // B scale columns per buffer
    static constexpr uint32_t kSfCols = 16 + kSfBCols;               // one buffer: A (16 columns), then B
    static_assert(kBN + kSfBufs * kSfCols <= kTmemCols, "tensor memory");
    // Instruction descriptor of kind::mxf4nvf4: A and B E2M1 (format 1), K-major, scale
    // factors UE4M3 (bit 23 = 0), N >> 3 in bits 17-22, M >> 4 in bits 24-28, dense K = 64.
    static constexpr uint32_t kIdesc =
        (1u << 7) | (1u << 10) | ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
};

template <int kBN>
struct Smem {
    uint8_t a[kStages][Cfg<kBN>::kATile];         // 1024-byte aligned (128-byte swizzle atoms)
    uint8_t b[kStages][Cfg<kBN>::kBTile];
    uint8_t sfa[kStages][Cfg<kBN>::kSfA];
    uint8_t sfb[kStages][Cfg<kBN>::kSfB];
    uint8_t stg[8][1024];                         // per epilogue warp: 32 rows x 32 bytes, swizzled
    uint64_t full[kStages], empty[kStages], sf_full[kSfBufs], sf_free[kSfBufs], acc_full, acc_empty, drain;
    uint32_t tmem_base;
    uint32_t abort;                               // set by a wait that gave up
    uint32_t issued, consumed;                    // stages loaded / stages handed to the MMA
};

struct Params {
    CUtensorMap map_a, map_b;                     // codes [rows, K/2] bytes, 128 x 128-byte boxes
    const uint8_t* sfa;                           // scale atoms in the MMA layout
    const uint8_t* sfb;
    const float* d_s2a;
    const float* d_s2b;
    void* out;
    int64_t ldd;
    uint32_t n_tiles, k_stages, kt4;              // kt4 = K / 64: scale atoms per 128-row tile
    uint32_t tiles;                               // output tiles in all
    uint32_t* d_flags;
    uint32_t M, N, mt, nt;                        // MXFP4: sizes, 128-row atom tiles of A and of B
    uint32_t vec;                                 // MXFP4: ldd keeps 16-byte alignment
};

template <int kBN, int kOut>   // tile width 128 | 256; output 0 bf16, 2 fp32
__global__ void __launch_bounds__(kThreads, 1)
gemm_nvfp4_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<kBN>;
    extern __shared__ uint8_t smem_raw[];
    Smem<kBN>& sm = *reinterpret_cast<Smem<kBN>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t KS = p.k_stages;

    if (threadIdx.x == kProducer) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < kSfBufs; ++b) {
            mbar_init(&sm.sf_full[b], 4);                          // one arrival per scale-writer warp
            mbar_init(&sm.sf_free[b], 1);
        }
        mbar_init(&sm.acc_full, 1);
        mbar_init(&sm.acc_empty, 8);                               // one arrival per epilogue warp
        mbar_init(&sm.drain, 1);
        sm.abort = 0u;
        sm.issued = sm.consumed = 0u;
        mbar_init_fence();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_b)) : "memory");
    }
    if (warp == kIssuer / 32) tmem_alloc(&sm.tmem_base, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    uint32_t flags = 0u;
    auto aborted = [&]() { return *reinterpret_cast<volatile uint32_t*>(&sm.abort) != 0u; };

    if (warp == kProducer / 32) {
        if (lane == 0) {                                           // producer, running ahead across tiles
            uint32_t g = 0;
            for (uint32_t t = blockIdx.x; t < p.tiles && !aborted(); t += gridDim.x) {
                const uint32_t n_tile = t % p.n_tiles, m_tile = t / p.n_tiles;
                for (uint32_t ks = 0; ks < KS; ++ks, ++g) {
                    const uint32_t s = g % kStages;
                    if (g >= (uint32_t)kStages && !wait_bar(&sm.empty[s], ((g / kStages) - 1u) & 1u)) {
                        flags |= kFlagTimeout;
                        atomicOr(&sm.abort, 1u);
                    }
                    if (aborted()) break;
                    mbar_arrive_expect_tx(&sm.full[s], C::kStageTx);
                    tma_load_2d(sm.a[s], &p.map_a, &sm.full[s], (int)(ks * 128u), (int)(m_tile * kBM));
                    tma_load_2d(sm.b[s], &p.map_b, &sm.full[s], (int)(ks * 128u), (int)(n_tile * kBN));
                    bulk_load(sm.sfa[s], p.sfa + ((size_t)m_tile * p.kt4 + 4u * ks) * 512u, C::kSfA, &sm.full[s]);
#pragma unroll
                    for (uint32_t h = 0; h < (uint32_t)(kBN / 128); ++h)  // one run of 4 atoms per 128 rows
                        bulk_load(sm.sfb[s] + 2048u * h,
                                  p.sfb + ((size_t)(n_tile * (kBN / 128) + h) * p.kt4 + 4u * ks) * 512u, 2048u,
                                  &sm.full[s]);
                }
            }
            sm.issued = g;
        }
        __syncwarp();
    } else if (warp == kIssuer / 32) {
        // ---- MMA issuer
        const uint64_t da0 = smem_desc(smem_u32(sm.a[0]), 1u, 64u, 2u), db0 = smem_desc(smem_u32(sm.b[0]), 1u, 64u, 2u);
        uint32_t g = 0, i = 0, s = 0, ph = 0;                      // kStages == kSfBufs: stage s uses buffer s
        static_assert(kStages == kSfBufs, "stage and scale buffer advance together");
        bool ok = true;
        for (uint32_t t = blockIdx.x; ok && t < p.tiles; t += gridDim.x, ++i) {
            // the accumulator is free once the epilogue has read the previous tile
            if (i > 0) ok = wait_bar_warp(&sm.acc_empty, (i - 1u) & 1u);
            tc_fence_after();
            for (uint32_t ks = 0; ok && ks < KS; ++ks, ++g) {
                ok = wait_bar_warp(&sm.full[s], ph) && wait_bar_warp(&sm.sf_full[s], ph);
                if (!ok) break;
                tc_fence_after();
                // scale columns (written by the scale writers): A row r of K-step j at column
                // ta + 4j + r/32, B row n at tb + nb*j + n/32
                constexpr uint32_t nb = 4u * (kBN / 128);
                const uint32_t ta = tmem + kBN + C::kSfCols * s, tb = ta + 16u;
                const uint64_t da = da0 + (uint64_t)(s * (C::kATile / 16u)), db = db0 + (uint64_t)(s * (C::kBTile / 16u));
                if (elect_one()) {
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
                        mma_fp4<false, false>(tmem, da + 2u * j, db + 2u * j, C::kIdesc, ta + 4u * j, tb + nb * j,
                                              (ks | j) != 0u ? 1u : 0u);
                    tc_commit(&sm.empty[s]);                       // frees the stage when these MMAs finish
                    tc_commit(&sm.sf_free[s]);                     // and the scale buffer
                }
                __syncwarp();
                if (++s == (uint32_t)kStages) {
                    s = 0u;
                    ph ^= 1u;
                }
            }
            if (ok && elect_one()) tc_commit(&sm.acc_full);        // this tile's accumulator is complete
            __syncwarp();
        }
        if (!ok && lane == 0) {
            flags |= kFlagTimeout;
            atomicOr(&sm.abort, 1u);
        }
        if (lane == 0) sm.consumed = g;
        if (elect_one()) tc_commit(&sm.drain);                     // every tensor-core operation issued
        __syncwarp();
        if (!wait_bar_warp(&sm.drain, 0u)) flags |= kFlagTimeout;
    } else if (warp >= 4 && warp < 8) {
        // ---- scale writers, warps 4-7 (tensor-memory sub-partition q = warp % 4, lanes
        // 32q..32q+31).  The block-scaled MMA reads the scale factors of a K-step from the
        // lanes of every sub-partition: row r of a 512-byte atom (32 rows x 16 bytes, rows r,
        // r+32, r+64, r+96 of the operand, 4 scales each) goes to lane 32q + r of every q, as
        // four consecutive columns.  Per stage each writer loads row `lane` of the stage's
        // atoms from shared memory and stores them with tcgen05.st into buffer g % kSfBufs:
        // 16 A columns (K-step j at 4j) and 16 or 32 B columns (K-step j, half h at nb*j + 4h).
        // Every lane waits on the barriers itself; the decision to stop is warp-uniform.
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        constexpr uint32_t nb = 4u * (kBN / 128);
        uint32_t g = 0;
        bool quit = false;
        for (uint32_t t = blockIdx.x; t < p.tiles && !quit; t += gridDim.x) {
            for (uint32_t ks = 0; ks < KS; ++ks, ++g) {
                const uint32_t s = g % kStages, b = g % kSfBufs;
                bool ok = wait_bar(&sm.full[s], (g / kStages) & 1u);
                if (ok && g >= (uint32_t)kSfBufs) ok = wait_bar(&sm.sf_free[b], ((g / kSfBufs) - 1u) & 1u);
                const bool timed_out = __any_sync(0xFFFFFFFFu, !ok);
                quit = timed_out || __any_sync(0xFFFFFFFFu, aborted());
                if (quit) {
                    if (timed_out && lane == 0) { flags |= kFlagTimeout; atomicOr(&sm.abort, 1u); }
                    break;
                }
                tc_fence_after();
                uint32_t va[16], vb[4 * nb];
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4*>(sm.sfa[s] + 512u * j + 16u * lane);
                    va[4 * j] = x.x; va[4 * j + 1] = x.y; va[4 * j + 2] = x.z; va[4 * j + 3] = x.w;
#pragma unroll
                    for (uint32_t h = 0; h < (uint32_t)(kBN / 128); ++h) {
                        const uint4 y = *reinterpret_cast<const uint4*>(sm.sfb[s] + 2048u * h + 512u * j + 16u * lane);
                        const uint32_t c = nb * j + 4u * h;
                        vb[c] = y.x; vb[c + 1] = y.y; vb[c + 2] = y.z; vb[c + 3] = y.w;
                    }
                }
                const uint32_t ta = tmem + lanes + kBN + C::kSfCols * b;
                tmem_st<16>(ta, va);
                tmem_st<4 * nb>(ta + 16u, vb);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.sf_full[b]);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue warps 0-3 and 10-13: warp w reads accumulator lanes 32q..32q+31
        // (q = w % 4, one output row per thread), columns [h * kBN/2, (h + 1) * kBN/2) with
        // h = (w >= 10).  BF16: the half row is converted into registers, the accumulator is
        // released, and only then stored (overlapping the next tile's MMAs), each 32 x 16
        // block transposed through the warp's 1 KB of shared memory so that a store
        // instruction writes 16 rows x 32 contiguous bytes.  FP32: stored as read.
        const uint32_t q = (uint32_t)warp & 3u, h = warp >= 10 ? 1u : 0u;
        uint8_t* st = sm.stg[q + 4u * h];
        const float alpha = __fmul_rn(*p.d_s2a, *p.d_s2b);
        constexpr int kChunks = kBN / 64;                          // 32-column chunks per warp
        uint32_t i = 0;
        for (uint32_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++i) {
            const bool ok = !aborted() && wait_bar(&sm.acc_full, i & 1u);
            if (!ok) {
                if (!aborted()) { flags |= kFlagTimeout; atomicOr(&sm.abort, 1u); }
                break;
            }
            tc_fence_after();
            __syncwarp();
            const uint32_t n_tile = t % p.n_tiles, m_tile = t / p.n_tiles;
            const int64_t row0 = (int64_t)m_tile * kBM + 32 * q;  // this warp's first row
            const int64_t col0 = (int64_t)n_tile * kBN + (int64_t)h * (kBN / 2);
            const uint32_t taddr = tmem + ((32u * q) << 16) + h * (uint32_t)(kBN / 2);
            if constexpr (kOut == 2) {
#pragma unroll 1
                for (int cb = 0; cb < kChunks; ++cb) {
                    float v[32];
                    tmem_ld32(taddr + (uint32_t)(32 * cb), v);
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + (row0 + lane) * p.ldd + col0 + 32 * cb);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[k] = make_float4(__fmul_rn(v[4 * k], alpha), __fmul_rn(v[4 * k + 1], alpha),
                                           __fmul_rn(v[4 * k + 2], alpha), __fmul_rn(v[4 * k + 3], alpha));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_empty);
            } else {
                uint32_t w[16 * kChunks];
#pragma unroll
                for (int cb = 0; cb < kChunks; ++cb) {
                    float v[32];
                    tmem_ld32(taddr + (uint32_t)(32 * cb), v);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                            : "=r"(w[16 * cb + k])
                            : "f"(__fmul_rn(v[2 * k + 1], alpha)), "f"(__fmul_rn(v[2 * k], alpha)));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_empty);         // the accumulator is free
                // 16-byte piece p of staged row r at r * 32 + 16 * (p ^ ((r >> 2) & 1)):
                // conflict-free for the row-per-thread writes and the 16-rows-per-instruction reads
                const int pr = lane >> 1, pc = lane & 1;
#pragma unroll
                for (int c16 = 0; c16 < 2 * kChunks; ++c16) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4*>(st + 32 * lane + 16 * (k ^ ((lane >> 2) & 1))) =
                            make_uint4(w[8 * c16 + 4 * k], w[8 * c16 + 4 * k + 1], w[8 * c16 + 4 * k + 2],
                                       w[8 * c16 + 4 * k + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int rr = pr + 16 * k;
                        const uint4 x = *reinterpret_cast<const uint4*>(st + 32 * rr + 16 * (pc ^ ((rr >> 2) & 1)));
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (row0 + rr) * p.ldd + col0 + 16 * c16 +
                                                  8 * pc) = x;
                    }
                    __syncwarp();
                }
            }
        }
    }

    // ---- teardown: drain copies that were loaded but never consumed, free tensor memory
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == kProducer) {
        for (uint32_t g = sm.consumed; g < sm.issued; ++g)
            if (!wait_bar(&sm.full[g % kStages], (g / kStages) & 1u)) flags |= kFlagTimeout;
    }
    if (warp == kIssuer / 32) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    flags = __reduce_or_sync(0xFFFFFFFFu, flags);
    if (lane == 0) flag_or(p.d_flags, flags);
}

// ---------------------------------------------------------------- the CTA-pair kernel
// 256 x 256 output tiles computed by a pair of CTAs (a 2-CTA cluster) with the 2-SM MMA
// (tcgen05.mma.cta_group::2, M = 256): CTA r of the pair holds rows 128r..128r+127 of the
// tile's A and of its B in its own shared memory, the full N = 256 of B's scale atoms, and
// its 128 x 256 FP32 accumulator.  The pair's MMA reads each B half once and shares it, so
// per SM a stage moves 16 KB less B through shared memory (TMA write and MMA read) than
// the single-CTA 128 x 256 tile does for the same work.  Roles per CTA as in the kernel
// above (producer, scale writers, epilogue); warp 9 of rank 0 issues the pair's MMAs and
// warp 9 of rank 1 forwards "this stage's codes have landed and its scales are written"
// to it (a cluster-scope mbarrier arrive).  The MMA thread's commits arrive on the
// barriers of both CTAs (tcgen05.commit ... multicast::cluster, mask 0b11); rank 1's
// epilogue warps release the accumulator on rank 0's acc_empty.  No load is multicast.
constexpr int kStages2 = 5;
constexpr int kSfBufs2 = 5;                       // 256 + 5 x 48 = 496 tensor-memory columns

struct Smem2 {
    uint8_t a[kStages2][128 * 128];               // this CTA's 128 rows of A (1024-byte aligned)
    uint8_t b[kStages2][128 * 128];               // this CTA's 128 rows of B
    uint8_t sfa[kStages2][4 * 512];               // A scale atoms of this CTA's rows
    uint8_t sfb[kStages2][8 * 512];               // B scale atoms of all 256 rows
    uint8_t stg[8][1024];                         // epilogue transposes
    uint64_t full[kStages2], empty[kStages2], peer_ready[kStages2], sf_full[kSfBufs2], sf_free[kSfBufs2];
    uint64_t acc_full, acc_empty, drain;
    uint32_t tmem_base;
    uint32_t abort;
    uint32_t issued, consumed;
};

template <bool kMx, int kOut>
__global__ void __launch_bounds__(kThreads, 1)
gemm_pair_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<256>;
    constexpr int kStages = kStages2;
    constexpr uint32_t kAtoms = kMx ? 2u : 4u;                     // scale atoms per 128 rows and stage
    constexpr uint32_t kTx = 2u * 128u * 128u + 3u * kAtoms * 512u;
    // instruction descriptor: as Cfg<256>::kIdesc with M = 256 (the pair); E8M0 scales: bit 23
    constexpr uint32_t kIdesc2 = (1u << 7) | (1u << 10) | ((uint32_t)(256 >> 3) << 17) | (kMx ? 1u << 23 : 0u) |
                                 ((uint32_t)(256 >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    Smem2& sm = *reinterpret_cast<Smem2*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t KS = p.k_stages;
    const uint32_t rank = cluster_ctarank();
    const uint32_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == kProducer) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
            mbar_init(&sm.peer_ready[s], 1);
        }
        for (int b = 0; b < kSfBufs2; ++b) {
            mbar_init(&sm.sf_full[b], 8);                          // the writers of both CTAs
            mbar_init(&sm.sf_free[b], 1);
        }
        mbar_init(&sm.acc_full, 1);
        mbar_init(&sm.acc_empty, 16);                              // 8 epilogue warps in each CTA
        mbar_init(&sm.drain, 1);
        sm.abort = 0u;
        sm.issued = sm.consumed = 0u;
        mbar_init_fence();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_b)) : "memory");
    }
    if (warp == kIssuer / 32) tmem_alloc_pair(&sm.tmem_base, C::kTmemCols);
    tc_fence_before();
    cluster_sync();                                                // barriers of both CTAs initialised
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    uint32_t flags = 0u;
    auto aborted = [&]() { return *reinterpret_cast<volatile uint32_t*>(&sm.abort) != 0u; };
    auto give_up = [&]() { flags |= kFlagTimeout; atomicOr(&sm.abort, 1u); };

    if (warp == kProducer / 32) {
        if (lane == 0) {                                           // producer: this CTA's halves
            uint32_t g = 0;
            for (uint32_t t = pair; t < p.tiles && !aborted(); t += npairs) {
                const uint32_t n_tile = t % p.n_tiles, m_tile = t / p.n_tiles;
                const uint32_t mrow = 2u * m_tile + rank, nrow = 2u * n_tile + rank;   // 128-row tiles
                for (uint32_t ks = 0; ks < KS; ++ks, ++g) {
                    const uint32_t s = g % kStages;
                    if (g >= (uint32_t)kStages && !wait_bar(&sm.empty[s], ((g / kStages) - 1u) & 1u)) give_up();
                    if (aborted()) break;
                    mbar_arrive_expect_tx(&sm.full[s], kTx);
                    tma_load_2d(sm.a[s], &p.map_a, &sm.full[s], (int)(ks * 128u), (int)(mrow * 128u));
                    tma_load_2d(sm.b[s], &p.map_b, &sm.full[s], (int)(ks * 128u), (int)(nrow * 128u));
                    if constexpr (kMx) {
                        // 2 atoms of 128 K-elements; past an odd end the last one again (its codes
                        // are zeros there), past the last rows the last row tile (rows not stored)
                        const uint32_t a1 = min(2u * ks + 1u, p.kt4 - 1u);
                        const uint8_t* fa = p.sfa + (size_t)min(mrow, p.mt - 1u) * p.kt4 * 512u;
                        bulk_load(sm.sfa[s], fa + 2u * ks * 512u, 512u, &sm.full[s]);
                        bulk_load(sm.sfa[s] + 512u, fa + a1 * 512u, 512u, &sm.full[s]);
#pragma unroll
                        for (uint32_t h = 0; h < 2u; ++h) {
                            const uint8_t* fb = p.sfb + (size_t)min(2u * n_tile + h, p.nt - 1u) * p.kt4 * 512u;
                            bulk_load(sm.sfb[s] + 2048u * h, fb + 2u * ks * 512u, 512u, &sm.full[s]);
                            bulk_load(sm.sfb[s] + 2048u * h + 512u, fb + a1 * 512u, 512u, &sm.full[s]);
                        }
                    } else {
                        bulk_load(sm.sfa[s], p.sfa + ((size_t)mrow * p.kt4 + 4u * ks) * 512u, 2048u, &sm.full[s]);
#pragma unroll
                        for (uint32_t h = 0; h < 2u; ++h)
                            bulk_load(sm.sfb[s] + 2048u * h, p.sfb + ((size_t)(2u * n_tile + h) * p.kt4 + 4u * ks) * 512u,
                                      2048u, &sm.full[s]);
                    }
                }
            }
            sm.issued = g;
        }
        __syncwarp();
    } else if (warp == kIssuer / 32) {
        if (rank == 0) {                                           // the pair's MMA issuer
            const uint64_t da0 = smem_desc(smem_u32(sm.a[0]), 1u, 64u, 2u), db0 = smem_desc(smem_u32(sm.b[0]), 1u, 64u, 2u);
            uint32_t g = 0, i = 0, s = 0, ph = 0;                  // kStages2 == kSfBufs2: stage s uses buffer s
            static_assert(kStages2 == kSfBufs2, "stage and scale buffer advance together");
            bool ok = true;
            for (uint32_t t = pair; ok && t < p.tiles; t += npairs, ++i) {
                if (i > 0) ok = wait_bar_warp(&sm.acc_empty, (i - 1u) & 1u);
                tc_fence_after();
                for (uint32_t ks = 0; ok && ks < KS; ++ks, ++g) {
                    ok = wait_bar_warp(&sm.full[s], ph) && wait_bar_warp(&sm.sf_full[s], ph) &&
                         wait_bar_warp(&sm.peer_ready[s], ph);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t ta = tmem + 256u + C::kSfCols * s, tb = ta + 16u;
                    const uint64_t da = da0 + (uint64_t)(s * 1024u), db = db0 + (uint64_t)(s * 1024u);
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t j = 0; j < 4; ++j) {
                            // MXFP4: an atom's words serve two steps, the second from byte 2 on
                            const uint32_t at = kMx ? j >> 1 : j, id = kMx ? 2u * (j & 1u) : 0u;
                            mma_fp4<true, kMx>(tmem, da + 2u * j, db + 2u * j, kIdesc2 | (id << 29) | (id << 4), ta + 4u * at,
                                               tb + 8u * at, (ks | j) != 0u ? 1u : 0u);
                        }
                        tc_commit_pair(&sm.empty[s]);
                        tc_commit_pair(&sm.sf_free[s]);
                    }
                    __syncwarp();
                    if (++s == (uint32_t)kStages) {
                        s = 0u;
                        ph ^= 1u;
                    }
                }
                if (ok && elect_one()) tc_commit_pair(&sm.acc_full);
                __syncwarp();
            }
            if (!ok && lane == 0) give_up();
            if (lane == 0) sm.consumed = g;
            if (elect_one()) tc_commit_pair(&sm.drain);
            __syncwarp();
            if (!wait_bar_warp(&sm.drain, 0u)) flags |= kFlagTimeout;
        } else if (lane == 0) {                                    // rank 1: forwards its landed stages
            uint32_t g = 0;
            for (uint32_t t = pair; t < p.tiles && !aborted(); t += npairs) {
                for (uint32_t ks = 0; ks < KS; ++ks, ++g) {
                    const uint32_t s = g % kStages;
                    if (!wait_bar(&sm.full[s], (g / kStages) & 1u)) {
                        give_up();
                        break;
                    }
                    mbar_arrive_cluster(&sm.peer_ready[s], 0u);
                }
            }
            sm.consumed = g;
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ---- scale writers: as in the single-CTA kernel, this CTA's rows of A, all of B
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        uint32_t g = 0;
        bool quit = false;
        for (uint32_t t = pair; t < p.tiles && !quit; t += npairs) {
            for (uint32_t ks = 0; ks < KS; ++ks, ++g) {
                const uint32_t s = g % kStages, b = g % kSfBufs2;
                bool ok = wait_bar(&sm.full[s], (g / kStages) & 1u);
                if (ok && g >= (uint32_t)kSfBufs2) ok = wait_bar(&sm.sf_free[b], ((g / kSfBufs2) - 1u) & 1u);
                const bool timed_out = __any_sync(0xFFFFFFFFu, !ok);
                quit = timed_out || __any_sync(0xFFFFFFFFu, aborted());
                if (quit) {
                    if (timed_out && lane == 0) give_up();
                    break;
                }
                tc_fence_after();
                uint32_t va[4 * kAtoms], vb[8 * kAtoms];
#pragma unroll
                for (uint32_t j = 0; j < kAtoms; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4*>(sm.sfa[s] + 512u * j + 16u * lane);
                    va[4 * j] = x.x; va[4 * j + 1] = x.y; va[4 * j + 2] = x.z; va[4 * j + 3] = x.w;
#pragma unroll
                    for (uint32_t h = 0; h < 2u; ++h) {
                        const uint4 y = *reinterpret_cast<const uint4*>(sm.sfb[s] + 2048u * h + 512u * j + 16u * lane);
                        const uint32_t c = 8u * j + 4u * h;
                        vb[c] = y.x; vb[c + 1] = y.y; vb[c + 2] = y.z; vb[c + 3] = y.w;
                    }
                }
                const uint32_t ta = tmem + lanes + 256u + C::kSfCols * b;
                tmem_st<4 * kAtoms>(ta, va);
                tmem_st<8 * kAtoms>(ta + 16u, vb);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {                                   // on the MMA issuer's CTA
                    if (rank == 0) mbar_arrive(&sm.sf_full[b]);
                    else mbar_arrive_cluster(&sm.sf_full[b], 0u);
                }
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue warps 0-3 and 10-13, as in the single-CTA kernel; rows 128 * rank + ...
        const uint32_t q = (uint32_t)warp & 3u, h = warp >= 10 ? 1u : 0u;
        uint8_t* st = sm.stg[q + 4u * h];
        const float alpha = kMx ? 1.0f : __fmul_rn(*p.d_s2a, *p.d_s2b);
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(&sm.acc_empty);
                else mbar_arrive_cluster(&sm.acc_empty, 0u);
            }
        };
        uint32_t i = 0;
        for (uint32_t t = pair; t < p.tiles; t += npairs, ++i) {
            const bool ok = !aborted() && wait_bar(&sm.acc_full, i & 1u);
            if (!ok) {
                if (!aborted()) give_up();
                break;
            }
            tc_fence_after();
            __syncwarp();
            const uint32_t n_tile = t % p.n_tiles, m_tile = t / p.n_tiles;
            const int64_t row0 = (int64_t)m_tile * 256 + 128 * (int64_t)rank + 32 * q;
            const int64_t col0 = (int64_t)n_tile * 256 + (int64_t)h * 128;
            const uint32_t taddr = tmem + ((32u * q) << 16) + h * 128u;
            if constexpr (kOut == 2) {
#pragma unroll 1
                for (int cb = 0; cb < 4; ++cb) {
                    if (kMx && col0 + 32 * cb >= p.N) break;       // the warp's columns are the same
                    float v[32];
                    tmem_ld32(taddr + (uint32_t)(32 * cb), v);
                    if (kMx && (p.vec == 0u || col0 + 32 * cb + 32 > p.N)) {
                        // as for BF16 below: through shared memory, 4 rows x 8 columns a store
                        float* sf = reinterpret_cast<float*>(st);
#pragma unroll
                        for (int c8 = 0; c8 < 4; ++c8) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) sf[8 * lane + ((k + lane) & 7)] = v[8 * c8 + k];
                            __syncwarp();
                            const int c = lane & 7;
                            const int64_t col = col0 + 32 * cb + 8 * c8 + c;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int rr = 4 * k + (lane >> 3);
                                if (row0 + rr < p.M && col < p.N)
                                    static_cast<float*>(p.out)[(row0 + rr) * p.ldd + col] = sf[8 * rr + ((c + rr) & 7)];
                            }
                            __syncwarp();
                        }
                        continue;
                    }
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + (row0 + lane) * p.ldd + col0 + 32 * cb);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (kMx && row0 + lane >= p.M) continue;
                        o[k] = make_float4(__fmul_rn(v[4 * k], alpha), __fmul_rn(v[4 * k + 1], alpha),
                                           __fmul_rn(v[4 * k + 2], alpha), __fmul_rn(v[4 * k + 3], alpha));
                    }
                }
                release();
            } else {
                uint32_t w[64];
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    float v[32];
                    tmem_ld32(taddr + (uint32_t)(32 * cb), v);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                            : "=r"(w[16 * cb + k])
                            : "f"(__fmul_rn(v[2 * k + 1], alpha)), "f"(__fmul_rn(v[2 * k], alpha)));
                }
                release();
                const int pr = lane >> 1, pc = lane & 1;
#pragma unroll
                for (int c16 = 0; c16 < 8; ++c16) {
                    if (kMx && col0 + 16 * c16 >= p.N) break;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4*>(st + 32 * lane + 16 * (k ^ ((lane >> 2) & 1))) =
                            make_uint4(w[8 * c16 + 4 * k], w[8 * c16 + 4 * k + 1], w[8 * c16 + 4 * k + 2],
                                       w[8 * c16 + 4 * k + 3]);
                    __syncwarp();
                    if (kMx && (p.vec == 0u || col0 + 16 * c16 + 16 > p.N)) {
                        // rows of no 16-byte alignment, or the ragged end: 2 rows x 16 columns a store
                        const int c = lane & 15;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int rr = 2 * k + (lane >> 4);
                            const int64_t col = col0 + 16 * c16 + c;
                            if (row0 + rr < p.M && col < p.N)
                                static_cast<uint16_t*>(p.out)[(row0 + rr) * p.ldd + col] = *reinterpret_cast<const uint16_t*>(
                                    st + 32 * rr + 16 * ((c >> 3) ^ ((rr >> 2) & 1)) + 2 * (c & 7));
                        }
                        __syncwarp();
                        continue;
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int rr = pr + 16 * k;
                        const uint4 x = *reinterpret_cast<const uint4*>(st + 32 * rr + 16 * (pc ^ ((rr >> 2) & 1)));
                        if (kMx && row0 + rr >= p.M) continue;
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (row0 + rr) * p.ldd + col0 + 16 * c16 +
                                                  8 * pc) = x;
                    }
                    __syncwarp();
                }
            }
        }
    }

    // ---- teardown: this CTA's loads drained, then the pair's barrier (rank 0 reaches it
    // only after its MMAs, which read both CTAs' shared memory, have completed), then the
    // pair's tensor memory is released
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == kProducer) {
        for (uint32_t g = sm.consumed; g < sm.issued; ++g)
            if (!wait_bar(&sm.full[g % kStages], (g / kStages) & 1u)) flags |= kFlagTimeout;
    }
    tc_fence_before();
    cluster_sync();
    if (warp == kIssuer / 32) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::kTmemCols);
    }
    flags = __reduce_or_sync(0xFFFFFFFFu, flags);
    if (lane == 0) flag_or(p.d_flags, flags);
}

// Block scales [rows, kb] (row-major, kb = K/16) -> the MMA atom layout, one thread per
// 32-bit word (one row's 4 consecutive scales); padding rows and columns are zero.
__global__ void __launch_bounds__(256)
mma_scale_layout_kernel(const uint8_t* __restrict__ sc, uint32_t rows, uint32_t kb, uint32_t kt,
                        uint32_t total_words, uint32_t* __restrict__ out)
{
    for (uint32_t w = blockIdx.x * 256u + threadIdx.x; w < total_words; w += gridDim.x * 256u) {
        // word w = ((rt * kt) + g) * 128 + (r % 32) * 4 + (r % 128) / 32
        const uint32_t atom = w >> 7, in = w & 127u;
        const uint32_t rt = atom / kt, g = atom - rt * kt;
        const uint32_t r = rt * 128u + (in >> 2) + 32u * (in & 3u);
        uint32_t v = 0u;
        if (r < rows) {
            const uint8_t* src = sc + (size_t)r * kb + 4u * g;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                if (4u * g + j < kb) v |= (uint32_t)src[j] << (8u * j);
        }
        out[w] = v;
    }
}

}  // namespace gemm

namespace gemm {

// Persistent launch of the pair kernel: as many pairs as can be resident at once.
template <bool kMx, int kOut>
static cudaError_t run_pair(const Params& p, int dev, cudaStream_t s)
{
    static bool attr_set[64] = {};
    static int resident[64] = {};
    constexpr size_t smem = sizeof(Smem2) + 1024;
    static_assert(smem > kSmemOfOnePerSm, "one CTA per SM: see kSmemOfOnePerSm");
    auto kern = gemm_pair_kernel<kMx, kOut>;
    const bool known = dev >= 0 && dev < 64;
    if (!known || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (known) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int pairs_cap = known ? resident[dev] : 0;
    if (pairs_cap <= 0) {
        cfg.gridDim = dim3(2u * (uint32_t)(num_sms() / 2), 1, 1);
        if (cudaOccupancyMaxActiveClusters(&pairs_cap, kern, &cfg) != cudaSuccess || pairs_cap <= 0) {
            (void)cudaGetLastError();
            pairs_cap = num_sms() / 2;
        }
        if (known) resident[dev] = pairs_cap;
    }
    cfg.gridDim = dim3(2u * (p.tiles < (uint32_t)pairs_cap ? p.tiles : (uint32_t)pairs_cap), 1, 1);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gemm

size_t mma_scale_bytes(int64_t rows, int64_t kb)
{
    return (size_t)((rows + 127) / 128) * 128u * (size_t)((kb + 3) / 4) * 4u;
}

cudaError_t launch_mma_scale_layout(const uint8_t* sc, int64_t rows, int64_t kb, uint8_t* out, cudaStream_t s)
{
    const uint32_t kt = (uint32_t)((kb + 3) / 4);
    const uint32_t words = (uint32_t)(mma_scale_bytes(rows, kb) / 4u);
    int64_t need = ((int64_t)words + 255) / 256;
    const int64_t cap = (int64_t)num_sms() * 8;
    const int grid = (int)(need < cap ? (need > 0 ? need : 1) : cap);
    gemm::mma_scale_layout_kernel<<<grid, 256, 0, s>>>(sc, (uint32_t)rows, (uint32_t)kb, kt, words,
                                                       reinterpret_cast<uint32_t*>(out));
    return cudaGetLastError();
}

cudaError_t launch_gemm_nvfp4(const uint8_t* qa, const uint8_t* sfa, const float* d_s2a, const uint8_t* qb,
                              const uint8_t* sfb, const float* d_s2b, int64_t M, int64_t N, int64_t K, int out_dt,
                              void* out, int64_t ldd, uint32_t* d_flags, cudaStream_t s)
{
    using namespace gemm;
    Params p = {};
    static bool attr_set[4][64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int o = out_dt == 2 ? 1 : 0;
    if (M % 256 == 0 && N % 256 == 0) {
        // 256 x 256 tiles on CTA pairs (2-SM MMA)
        if (!code_map(&p.map_a, qa, M, K, 128u) || !code_map(&p.map_b, qb, N, K, 128u)) return cudaErrorInvalidValue;
        p.sfa = sfa;
        p.sfb = sfb;
        p.d_s2a = d_s2a;
        p.d_s2b = d_s2b;
        p.out = out;
        p.ldd = ldd;
        p.n_tiles = (uint32_t)(N / 256);
        p.k_stages = (uint32_t)(K / kBK);
        p.kt4 = (uint32_t)(K / 64);
        p.tiles = (uint32_t)((M / 256) * (N / 256));
        p.d_flags = d_flags;
        return o ? run_pair<false, 2>(p, dev, s) : run_pair<false, 0>(p, dev, s);
    }
    const bool wide = N % 256 == 0;
    const int bn = wide ? 256 : 128;
    if (!code_map(&p.map_a, qa, M, K, 128u) || !code_map(&p.map_b, qb, N, K, (uint32_t)bn)) return cudaErrorInvalidValue;
    p.sfa = sfa;
    p.sfb = sfb;
    p.d_s2a = d_s2a;
    p.d_s2b = d_s2b;
    p.out = out;
    p.ldd = ldd;
    p.n_tiles = (uint32_t)(N / bn);
    p.k_stages = (uint32_t)(K / kBK);
    p.kt4 = (uint32_t)(K / 64);
    p.tiles = (uint32_t)((M / kBM) * (N / bn));
    p.d_flags = d_flags;
    const size_t smem = (wide ? sizeof(Smem<256>) : sizeof(Smem<128>)) + 1024;
    const int v = 2 * (wide ? 1 : 0) + o;
    auto kern = wide ? (o ? gemm_nvfp4_kernel<256, 2> : gemm_nvfp4_kernel<256, 0>)
                     : (o ? gemm_nvfp4_kernel<128, 2> : gemm_nvfp4_kernel<128, 0>);
    if (dev < 0 || dev >= 64 || !attr_set[v][dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[v][dev] = true;
    }
    const unsigned grid = (unsigned)(p.tiles < (uint32_t)num_sms() ? p.tiles : (uint32_t)num_sms());
    kern<<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_gemm_mxfp4(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb, int64_t M,
                              int64_t N, int64_t K, int out_dt, void* out, int64_t ldd, bool dependent,
                              uint32_t* d_flags, cudaStream_t s)
{
    using namespace gemm;
    // few rows, or few tiles: the kernel of 128-row tiles, which splits K (gemm_mx.cu)
    if (M <= kMaxSmallRows || ((M + 127) / 128) * ((N + 127) / 128) <= num_sms()) return launch_gemm_mxfp4_small(qa, sfa, qb, sfb, M, N, K, out_dt, out, ldd, dependent, d_flags, s);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    Params p = {};
    if (!code_map(&p.map_a, qa, M, K, 128u) || !code_map(&p.map_b, qb, N, K, 128u)) return cudaErrorInvalidValue;
    p.sfa = sfa;
    p.sfb = sfb;
    p.out = out;
    p.ldd = ldd;
    p.n_tiles = (uint32_t)((N + 255) / 256);
    p.k_stages = (uint32_t)((K + kBK - 1) / kBK);
    p.kt4 = (uint32_t)((K + 127) / 128);
    p.tiles = (uint32_t)((M + 255) / 256) * p.n_tiles;
    p.d_flags = d_flags;
    p.M = (uint32_t)M;
    p.N = (uint32_t)N;
    p.mt = (uint32_t)((M + 127) / 128);
    p.nt = (uint32_t)((N + 127) / 128);
    p.vec = ldd % (out_dt == 2 ? 4 : 8) == 0 ? 1u : 0u;
    return out_dt == 2 ? run_pair<true, 2>(p, dev, s) : run_pair<true, 0>(p, dev, s);
}

}  // namespace nv4
