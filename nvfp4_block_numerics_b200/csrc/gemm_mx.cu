// gemm_mx.cu -- MXFP4 x MXFP4 product for few rows of A (decode batches) or few tiles, on the
// block-scaled tensor cores (sm_100a).  The form for many is the CTA-pair kernel of gemm.cu.
//
// [FP4] 1.2, 4.1.  D^T tile = B tile * A tile^T: 128 rows of B (the weights) are the MMA's M, up to
// kTok rows of A its N, so that the tensor cores' 128 rows are filled by the operand that has them.
// The bound is reading the weights once: N x K x 17/32 bytes.  One tile per cluster of z CTAs, each
// with its own part of K (nv4_split.h; 16 x 2048 x 16384: 14.0 us with z = 8 in two waves, 9.0
// with z = 6 in one); the partial sums meet
// through distributed shared memory, added in rank order.
//   * warp 0, one lane: TMA of the code tiles (256 K-elements per stage, 128-byte swizzle, zeros
//     outside) and bulk copies of the scale atoms.  The first stages' weights are requested before
//     the wait for the kernel in front (programmatic dependent launch), the rows of A after it.
//   * warp 1: owns the tensor memory; walks the stages with all lanes and issues four MMAs (K = 64)
//     per stage from an elected one.
//   * warps 4-7: move the scales into tensor memory (tcgen05.st, see gemm.cu), then read the
//     accumulator, one weight row per thread.
//   * warps 8-15, where x comes unquantized (the linear layer, up to 16 rows): quantize their CTA's
//     part of x into the stage, codes in the swizzled layout and scales as atoms, three stages ahead.
//     One launch instead of two, and no workspace.
// 16 x 16384 x 2048: 6.7 us, 9.1 with quantization (L2 holds the weights between calls; 14.6 us and 17.9
// MB from a cold one).  What bounds it there is eight stages behind a prologue and in front of a
// reduction: tensor pipe below 1%, issue slots 22%.
// Every mbarrier wait is bounded (kWaitLimitNs), as in gemm.cu.
#include <type_traits>

#include "nv4_internal.h"
#include "nv4_mxfp4.cuh"
#include "nv4_split.h"
#include "nv4_tcgen05.cuh"
#include "nv4_tensormap.h"

namespace nv4 {

namespace gemmx {

using namespace tc;

constexpr int kThreads = 256;                     // + those that quantize
constexpr int kQuant = 256;
constexpr int kStages = 6;
constexpr int kSfBufs = 4;                        // 16 columns each: 8 of the weights, 8 of the rows
constexpr uint32_t kSfCol = 128;                  // behind the accumulator
constexpr uint32_t kTmemCols = 256;

struct Params {
    CUtensorMap map_w, map_x;                     // codes [rows, K/2] bytes, boxes of 128 and kTok rows x 128 bytes
    const uint8_t* sfw;
    const uint8_t* sfx;
    void* out;
    int64_t ldd;
    uint32_t M, N, K, z, n_tiles, stages, kt;     // kt: scale atoms per row tile
    const void* x;                                // kIn >= 0: A as it came
    int64_t ldx;
    uint32_t* d_flags;
};

template <int kTok>
struct Smem {
    union {                                       // 1024-byte aligned
        uint8_t w[kStages][128 * 128];
        float part[kTok][128];                    // once the last product has read its weights
    };
    uint8_t x[kStages][kTok * 128];
    uint8_t sfw[kStages][1024];
    uint8_t sfx[kStages][1024];
    uint64_t full[kStages], empty[kStages], sf_full[kSfBufs], sf_free[kSfBufs], acc_full, drain;
    uint32_t tmem_base, abort, issued, consumed;
};

// kIn: -1 A quantized, else the type of x (0 BF16, 2 FP32).
template <int kTok, int kOut, int kIn>
__global__ void __launch_bounds__(kIn >= 0 ? kThreads + kQuant : kThreads, 1) gemm_mx_small_kernel(const __grid_constant__ Params p)
{
    // kind::mxf4: A and B E2M1, K-major, E8M0 scales (bit 23), N >> 3 in bits 17-22, M >> 4 in bits
    // 24-28; the two bytes of a scale word that a step uses in bits 4-5 (B) and 29-30 (A)
    constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(kTok >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
    constexpr uint32_t kTx = 128u * 128u + 1024u + (kIn >= 0 ? 0u : kTok * 128u + 1024u);
    constexpr uint32_t kBlock = kIn >= 0 ? kThreads + kQuant : kThreads;
    extern __shared__ uint8_t smem_raw[];
    Smem<kTok>& sm = *reinterpret_cast<Smem<kTok>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = p.z > 1u ? cluster_ctarank() : 0u, t = blockIdx.x / p.z;
    const uint32_t n_tile = t % p.n_tiles, m0 = (t / p.n_tiles) * kTok;
    const uint32_t ks0 = rank * p.stages / p.z, KS = (rank + 1u) * p.stages / p.z - ks0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], kIn >= 0 ? 1 + kQuant / 32 : 1);          // the copies, the quantizing warps
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < kSfBufs; ++b) {
            mbar_init(&sm.sf_full[b], 4);
            mbar_init(&sm.sf_free[b], 1);
        }
        mbar_init(&sm.acc_full, 1);
        mbar_init(&sm.drain, 1);
        sm.abort = sm.issued = sm.consumed = 0u;
        mbar_init_fence();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_w)) : "memory");
        if constexpr (kIn < 0)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_x)) : "memory");
    }
    if (warp == 1) tmem_alloc(&sm.tmem_base, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    uint32_t flags = 0u;
    auto aborted = [&]() { return *reinterpret_cast<volatile uint32_t*>(&sm.abort) != 0u; };
    auto give_up = [&]() { flags |= kFlagTimeout; atomicOr(&sm.abort, 1u); };

    if (warp == 0) {
        if (lane == 0) {
            auto weights = [&](uint32_t ks) {
                const uint32_t s = ks % kStages, a0 = 2u * (ks0 + ks);
                const uint8_t* f = p.sfw + (size_t)n_tile * p.kt * 512u;
                mbar_arrive_expect_tx(&sm.full[s], kTx);
                tma_load_2d(sm.w[s], &p.map_w, &sm.full[s], (int)((ks0 + ks) * 128u), (int)(n_tile * 128u));
                load_atoms(sm.sfw[s], f, a0, p.kt, &sm.full[s]);
            };
            auto rows = [&](uint32_t ks) {
                if constexpr (kIn >= 0) return;                    // the quantizing warps'
                const uint32_t s = ks % kStages, a0 = 2u * (ks0 + ks);
                const uint8_t* f = p.sfx + (size_t)(m0 / 128u) * p.kt * 512u;
                tma_load_2d(sm.x[s], &p.map_x, &sm.full[s], (int)((ks0 + ks) * 128u), (int)m0);
                load_atoms(sm.sfx[s], f, a0, p.kt, &sm.full[s]);
            };
            const uint32_t first = min(KS, (uint32_t)kStages);
            for (uint32_t ks = 0; ks < first; ++ks) weights(ks);
            if constexpr (kIn < 0) asm volatile("griddepcontrol.wait;" ::: "memory");     // A is complete
            for (uint32_t ks = 0; ks < first; ++ks) rows(ks);
            uint32_t ks = first;
            for (; ks < KS; ++ks) {
                if (!wait_bar(&sm.empty[ks % kStages], ((ks / kStages) - 1u) & 1u)) give_up();
                if (aborted()) break;
                weights(ks);
                rows(ks);
            }
            sm.issued = ks;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer
        const uint64_t dw0 = smem_desc(smem_u32(sm.w[0]), 1u, 64u, 2u), dx0 = smem_desc(smem_u32(sm.x[0]), 1u, 64u, 2u);
        uint32_t ks = 0;
        bool ok = true;
        for (; ks < KS; ++ks) {
            const uint32_t s = ks % kStages, b = ks % kSfBufs;
            ok = wait_bar_warp(&sm.full[s], (ks / kStages) & 1u) && wait_bar_warp(&sm.sf_full[b], (ks / kSfBufs) & 1u);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dw = dw0 + (uint64_t)(s * 1024u), dx = dx0 + (uint64_t)(s * (kTok * 8u));
            const uint32_t f0 = tmem + kSfCol + 16u * b;
            if (elect_one()) {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    const uint32_t id = 2u * (j & 1u);
                    mma_fp4<false, true>(tmem, dw + 2u * j, dx + 2u * j, kIdesc | (id << 29) | (id << 4), f0 + 4u * (j >> 1),
                                         f0 + 8u + 4u * (j >> 1), (ks | j) != 0u ? 1u : 0u);
                }
                tc_commit(&sm.empty[s]);
                tc_commit(&sm.sf_free[b]);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) give_up();
        if (lane == 0) sm.consumed = ks;
        if (elect_one()) {
            if (ok) tc_commit(&sm.acc_full);
            tc_commit(&sm.drain);
        }
        __syncwarp();
        if (!wait_bar_warp(&sm.drain, 0u)) flags |= kFlagTimeout;
    } else if (kIn >= 0 && warp >= 8) {
        // ---- x of one stage: M rows x 16 half blocks, two lanes to a block
        if constexpr (kIn >= 0) {
            const uint32_t tid = threadIdx.x - kThreads;
            const uint32_t kb = ks0 * 256u;
            constexpr uint32_t kPer = kTok * 16u / kQuant;         // half blocks per thread
            constexpr uint32_t kAhead = 3;                         // stages of x in registers
            float vs[kAhead][kPer][16];
            uint32_t abs_[kAhead][kPer];
            auto fetch = [&](float (&v)[kPer][16], uint32_t (&ab)[kPer], uint32_t ks) {
#pragma unroll
                for (uint32_t j = 0; j < kPer; ++j) {
                    const uint32_t i = tid + kQuant * j, r = i >> 4, k = kb + 256u * ks + 16u * (i & 15u);
                    ab[j] = 0u;
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[j][e] = 0.0f;
                    if (r < p.M - m0 && k < p.K && ks < KS) load16<kIn>(p.x, (int64_t)(m0 + r) * p.ldx + k, v[j], ab[j]);
                }
            };
            bool stop = false;
            auto stage = [&](float (&v)[kPer][16], uint32_t (&ab)[kPer], uint32_t ks) {
                const uint32_t s = ks % kStages;
                uint32_t code[kPer], c0[kPer], c1[kPer];
#pragma unroll
                for (uint32_t j = 0; j < kPer; ++j) {
                    ab[j] = max(ab[j], __shfl_xor_sync(0xFFFFFFFFu, ab[j], 1));
                    code[j] = mxfp4_encode16(v[j], ab[j], c0[j], c1[j]);
                    if (code[j] == 0xFFu) flags |= kFlagNonFinite;
                }
                fetch(v, ab, ks + kAhead);
                const bool ok = ks < (uint32_t)kStages || wait_bar(&sm.empty[s], ((ks / kStages) - 1u) & 1u);
                if (!__all_sync(0xFFFFFFFFu, ok) || __any_sync(0xFFFFFFFFu, aborted())) {
                    if (!ok && lane == 0) give_up();
                    stop = true;
                    return;
                }
#pragma unroll
                for (uint32_t j = 0; j < kPer; ++j) {
                    const uint32_t i = tid + kQuant * j, r = i >> 4, h = i & 15u;        // half block h of row r: block h / 2
                    *reinterpret_cast<uint2*>(sm.x[s] + 128u * r + 16u * ((h >> 1) ^ (r & 7u)) + 8u * (h & 1u)) =
                        make_uint2(c0[j], c1[j]);
                    if ((h & 1u) == 0u) sm.sfx[s][512u * (h >> 3) + 16u * r + ((h >> 1) & 3u)] = (uint8_t)code[j];
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.full[s]);
            };
#pragma unroll
            for (uint32_t a = 0; a < kAhead; ++a) fetch(vs[a], abs_[a], a);
            for (uint32_t ks = 0; ks < KS && !stop; ks += kAhead)
#pragma unroll
                for (uint32_t a = 0; a < kAhead; ++a)
                    if (ks + a < KS && !stop) stage(vs[a], abs_[a], ks + a);
            __syncwarp();
        }
    } else if (warp >= 4) {
        const uint32_t quad = (uint32_t)warp & 3u, lanes = (32u * quad) << 16;
        bool quit = false;
        for (uint32_t ks = 0; ks < KS; ++ks) {
            const uint32_t s = ks % kStages, b = ks % kSfBufs;
            bool ok = wait_bar(&sm.full[s], (ks / kStages) & 1u);
            if (ok && ks >= (uint32_t)kSfBufs) ok = wait_bar(&sm.sf_free[b], ((ks / kSfBufs) - 1u) & 1u);
            const bool timed_out = __any_sync(0xFFFFFFFFu, !ok);
            quit = timed_out || __any_sync(0xFFFFFFFFu, aborted());
            if (quit) {
                if (timed_out && lane == 0) give_up();
                break;
            }
            tc_fence_after();
            uint32_t v[16];
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
                const uint4 a = *reinterpret_cast<const uint4*>(sm.sfw[s] + 512u * j + 16u * lane);
                const uint4 c = *reinterpret_cast<const uint4*>(sm.sfx[s] + 512u * j + 16u * lane);
                v[4 * j] = a.x; v[4 * j + 1] = a.y; v[4 * j + 2] = a.z; v[4 * j + 3] = a.w;
                v[8 + 4 * j] = c.x; v[8 + 4 * j + 1] = c.y; v[8 + 4 * j + 2] = c.z; v[8 + 4 * j + 3] = c.w;
            }
            tmem_st<16>(tmem + lanes + kSfCol + 16u * b, v);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.sf_full[b]);
        }
        // the accumulator, transposed into shared memory: [row of A][128 weight rows]
        if (!quit) {
            const bool ok = wait_bar(&sm.acc_full, 0u);
            if (__any_sync(0xFFFFFFFFu, !ok)) {
                if (lane == 0) give_up();
            } else {
                tc_fence_after();
#pragma unroll 1
                for (uint32_t c = 0; c < (uint32_t)kTok; c += 16u) {
                    float v[16];
                    tmem_ld16(tmem + lanes + c, v);
#pragma unroll
                    for (uint32_t k = 0; k < 16; ++k) sm.part[c + k][32u * quad + lane] = v[k];
                }
            }
        }
        __syncwarp();
    }

    // ---- copies loaded but never multiplied, the cluster's sums, tensor memory
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0)
        for (uint32_t ks = sm.consumed; ks < sm.issued; ++ks)
            if (!wait_bar(&sm.full[ks % kStages], (ks / kStages) & 1u)) flags |= kFlagTimeout;
    if (p.z > 1u) cluster_sync();
    const uint32_t n0 = n_tile * 128u, rows = min(128u, p.N - n0), toks = min((uint32_t)kTok, p.M - m0);
    // four weight rows of a row of A per thread
    const uint32_t j1 = (rank + 1u) * toks * 32u / p.z;
    for (uint32_t i = rank * toks * 32u / p.z + threadIdx.x; i < j1; i += kBlock) {
        const uint32_t r = 4u * (i & 31u), tok = i >> 5;
        if (r >= rows) continue;
        const float* own = &sm.part[0][0] + 4u * i;
        const float4 v = p.z > 1u ? cluster_sum4(own, p.z) : *reinterpret_cast<const float4*>(own);
        // no sum is stored to which a CTA that gave up would have contributed (its word is read behind the
        // sums, in whose latency most of it hides: 0.1 of 6.4 us, 0.2 in front of them)
        if (p.z > 1u ? cluster_any(&sm.abort, p.z) : aborted()) continue;
        const float sum[4] = {v.x, v.y, v.z, v.w};
        const int64_t at = (int64_t)(m0 + tok) * p.ldd + n0 + r;
#pragma unroll
        for (uint32_t k = 0; k < 4u; ++k) {
            if (r + k >= rows) break;
            if constexpr (kOut == 2) {
                static_cast<float*>(p.out)[at + k] = sum[k];
            } else {
                uint16_t b;
                asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(sum[k]));
                static_cast<uint16_t*>(p.out)[at + k] = b;
            }
        }
    }
    if (p.z > 1u) cluster_sync();                                  // the others have read this CTA's sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    flags = __reduce_or_sync(0xFFFFFFFFu, flags);
    if (lane == 0) flag_or(p.d_flags, flags);
}

template <int kTok, int kOut, int kIn = -1>
static cudaError_t run(Params& p, uint32_t tiles, bool dependent, cudaStream_t s)
{
    static bool ready[64] = {};
    static int fits[64][kMaxSplit + 1] = {};
    auto kern = gemm_mx_small_kernel<kTok, kOut, kIn>;
    constexpr size_t smem = sizeof(Smem<kTok>) + 1024;
    static_assert(smem > kSmemOfOnePerSm, "one CTA per SM: see kSmemOfOnePerSm");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    constexpr int threads = kIn >= 0 ? kThreads + kQuant : kThreads;
    // a wave beside its stages (launch, first loads, the cluster's sums): some 4 stages' time
    p.z = split_tiles(kern, threads, smem, tiles, p.stages, 2u, 4u, fits, dev);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles * p.z, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (p.z > 1u) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = p.z;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

static bool fill(Params& p, const uint8_t* qw, const uint8_t* sfw, int64_t M, int64_t N, int64_t K, void* out, int64_t ldd,
                 uint32_t* d_flags)
{
    if (!code_map(&p.map_w, qw, N, K, 128u)) return false;
    p.sfw = sfw;
    p.out = out;
    p.ldd = ldd;
    p.M = (uint32_t)M;
    p.N = (uint32_t)N;
    p.K = (uint32_t)K;
    p.n_tiles = (uint32_t)((N + 127) / 128);
    p.stages = (uint32_t)((K + 255) / 256);
    p.kt = (uint32_t)((K + 127) / 128);
    p.d_flags = d_flags;
    return true;
}

}  // namespace gemmx

cudaError_t launch_gemm_mxfp4_small(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb, int64_t M,
                                    int64_t N, int64_t K, int out_dt, void* out, int64_t ldd, bool dependent,
                                    uint32_t* d_flags, cudaStream_t s)
{
    using namespace gemmx;
    Params p = {};
    const uint32_t tok = M <= 16 ? 16u : M <= 32 ? 32u : M <= 64 ? 64u : 128u;
    if (!fill(p, qb, sfb, M, N, K, out, ldd, d_flags) || !code_map(&p.map_x, qa, M, K, tok)) return cudaErrorInvalidValue;
    p.sfx = sfa;
    const uint32_t tiles = p.n_tiles * (uint32_t)((M + tok - 1) / tok);
    auto pick = [&](auto o) {
        constexpr int O = decltype(o)::value;
        if (tok == 16u) return run<16, O>(p, tiles, dependent, s);
        if (tok == 32u) return run<32, O>(p, tiles, dependent, s);
        if (tok == 64u) return run<64, O>(p, tiles, dependent, s);
        return run<128, O>(p, tiles, dependent, s);
    };
    return out_dt == 2 ? pick(std::integral_constant<int, 2>{}) : pick(std::integral_constant<int, 0>{});
}

cudaError_t launch_linear_mxfp4_small(const void* x, int in_dt, int64_t M, int64_t K, int64_t ldx, const uint8_t* qw,
                                      const uint8_t* sfw, int64_t N, int out_dt, void* out, int64_t ldd, uint32_t* d_flags,
                                      cudaStream_t s)
{
    using namespace gemmx;
    Params p = {};
    if (!fill(p, qw, sfw, M, N, K, out, ldd, d_flags)) return cudaErrorInvalidValue;
    p.x = x;
    p.ldx = ldx;
    if (in_dt == 0) return out_dt == 2 ? run<16, 2, 0>(p, p.n_tiles, false, s) : run<16, 0, 0>(p, p.n_tiles, false, s);
    return out_dt == 2 ? run<16, 2, 2>(p, p.n_tiles, false, s) : run<16, 0, 2>(p, p.n_tiles, false, s);
}

}  // namespace nv4
