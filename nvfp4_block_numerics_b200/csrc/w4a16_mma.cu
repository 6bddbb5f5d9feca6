// w4a16_mma.cu -- the weight-only linear layer for many rows, on the 5th-generation tensor cores
// (sm_100a): BF16 / FP16 rows times NVFP4 weights.
//
// [CAL] layer table (W4A16); the few-row form is in w4a16.cu.  out^T tile = W tile * x tile^T: the
// 128 weight rows of a tile are the MMA's M, kTok rows of x its N.  The MMA takes no FP4 beside
// 16-bit operands, so the codes are decoded on the way: e2m1 * e4m3 is exact in BF16 and FP16.
// The decoded operand goes to TENSOR memory, not to shared memory: tcgen05.mma reads its A operand
// from there, so a decoded byte is written once and read without shared memory, which the x tiles
// already keep busy (a 128 x 256 x 64 step moves 32 KB of x in and 32 KB out of it in 512 clocks).
//
// Persistent, one CTA per SM, 20 warps:
//   * warp 0, one lane: 2-D TMA of x, kTok rows x 64 K-elements per stage (128-byte swizzle, zeros
//     outside), a ring of kStages that runs across tiles.
//   * warp 1: owns the tensor memory; walks the stages with all lanes and issues four MMAs (K = 16)
//     per stage from an elected one.
//   * warps 4-11: decoders, two sets of four; a warp owns 32 weight rows (the tensor memory lanes
//     it may write) and takes every other 256-element chunk of K.  It fills a ring in shared memory
//     for itself with cp.async, eight lanes to a row's 128 bytes, across the ends of tiles; then
//     each lane decodes the codes of one row and writes 32 columns per stage (tcgen05.st).  (With
//     each lane loading its own row from global memory, 32 lines per instruction, the load path
//     set the pace: 895 clocks per stage, 245 us for 4096 x 16384 x 2048.)
//   * warps 12-19: epilogue, two warps per 32 lanes, half the columns each; 16-bit outputs leave
//     through a 2 KB transpose per warp so that a store covers 64 bytes of an output row.
// With few tiles a cluster of z CTAs shares one: each multiplies its part of K, the partial sums
// meet through distributed shared memory and are added in rank order.
// Bound: the tensor pipe and the decoders together (4096 x 16384 x 2048: 214 us back to back, 1.28 PFLOP/s, 79% of
// a BF16 library product at its burst rate, and 247 us, 1.11 PFLOP/s, among other passes with new inputs; tensor
// pipe 64%, issue slots 50%).  The decoders' rate per
// stage is the same whatever kTok is, so 17 rows cost nearly what 128 do (2880 x 2880: 9.9 and 12.5 us).
// Every mbarrier wait is bounded (kWaitLimitNs), as in gemm.cu.
#include <type_traits>

#include "nv4_cpasync.cuh"
#include "nv4_internal.h"
#include "nv4_split.h"
#include "nv4_tcgen05.cuh"
#include "nv4_tensormap.h"

namespace nv4 {

namespace w4mma {

using namespace tc;

constexpr int kThreads = 640;
constexpr int kABufs = 8;                         // decoded stages in tensor memory, 32 columns each
constexpr uint32_t kACol = 256;                   // behind the accumulator's columns
constexpr int kDepth = 2;                         // chunks of 256 K-elements in flight per decoder warp
constexpr uint32_t kSlot = 32u * 128u + 32u * 16u;          // codes and scales of 32 rows x 256
template <int kTok>
constexpr int kStages = kTok == 256 ? 4 : 6;      // stages of x

struct Params {
    CUtensorMap map_x;                            // x [T, K], boxes of kTok rows x 64 elements
    const uint8_t* q;
    const uint8_t* sc;
    const float* d_s2;
    void* out;
    int64_t ldd;
    uint32_t T, N, K, z, n_tiles, tiles, chunks;  // n_tiles: of 128 weight rows; chunks of 256 K-elements
    uint32_t vec;                                 // 16-byte stores of 16-bit outputs are aligned
    uint32_t* d_flags;
};

template <int kTok>
struct Smem {
    uint8_t x[kStages<kTok>][kTok * 128];         // 1024-byte aligned
    uint8_t ring[8][kDepth * kSlot];
    uint8_t stg[8][2048];
    uint64_t full[kStages<kTok>], empty[kStages<kTok>], a_full[kABufs], a_free[kABufs], acc_full, acc_empty, drain;
    uint32_t tmem_base, abort, issued, consumed;
};

// One K = 16 step, A in tensor memory.
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 "}" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// The 64 values as 32 words of two: FP16 by conversion and multiply, BF16 by converting those
// (at most 6 significant bits: exact both times).
template <int kDt>
__device__ __forceinline__ void decode64(uint32_t (&o)[32], const uint32_t (&q)[8], uint32_t s)
{
    uint32_t p[4];
    {
        uint32_t a, b;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(s & 0xFFFFu)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(s >> 16)));
        p[0] = __byte_perm(a, a, 0x1010);
        p[1] = __byte_perm(a, a, 0x3232);
        p[2] = __byte_perm(b, b, 0x1010);
        p[3] = __byte_perm(b, b, 0x3232);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        uint32_t h[4];
        cvt_e2m1x8_to_f16x8(q[u], h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t r;
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h[i]), "r"(p[u >> 1]));
            if constexpr (kDt == 0) {
                float lo, hi;
                f16x2_to_f32(r, lo, hi);
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
            }
            o[4 * u + i] = r;
        }
    }
}

template <int kOut>
__device__ __forceinline__ uint16_t to16(float v)
{
    uint16_t b;
    if constexpr (kOut == 0)
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
    else
        asm("cvt.rn.f16.f32 %0, %1;" : "=h"(b) : "f"(v));
    return b;
}

template <int kOut>
__device__ __forceinline__ void store1(void* out, int64_t at, float v)
{
    if constexpr (kOut == 2) static_cast<float*>(out)[at] = v;
    else static_cast<uint16_t*>(out)[at] = to16<kOut>(v);
}

template <int kTok, int kDt, int kOut, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) linear_mma_kernel(const __grid_constant__ Params p)
{
    // kind::f16: FP32 accumulator (bit 4), A and B types in bits 7 and 10 (0 FP16, 1 BF16), both
    // K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28
    constexpr int kStages = w4mma::kStages<kTok>;
    constexpr uint32_t kIdesc = (1u << 4) | (kDt == 0 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(kTok >> 3) << 17) |
                                ((128u >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    Smem<kTok>& sm = *reinterpret_cast<Smem<kTok>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* part = reinterpret_cast<float*>(&sm.x[0][0]);           // z > 1: [kTok][128], once the last product has read x
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = p.z > 1u ? cluster_ctarank() : 0u;
    const uint32_t clu = blockIdx.x / p.z, nclu = gridDim.x / p.z;
    const uint32_t ch0 = rank * p.chunks / p.z, NC = (rank + 1u) * p.chunks / p.z - ch0;   // this CTA's chunks of a tile
    const uint32_t KS = (min(p.K, (ch0 + NC) * 256u) - ch0 * 256u + 63u) / 64u;            // and stages of 64

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < kABufs; ++b) {
            mbar_init(&sm.a_full[b], 4);                           // the four warps of a decoder set
            mbar_init(&sm.a_free[b], 1);
        }
        mbar_init(&sm.acc_full, 1);
        mbar_init(&sm.acc_empty, 8);
        mbar_init(&sm.drain, 1);
        sm.abort = sm.issued = sm.consumed = 0u;
        mbar_init_fence();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_x)) : "memory");
    }
    if (warp == 1) tmem_alloc(&sm.tmem_base, 512u);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    uint32_t flags = 0u;
    NonFinite odd;                                                 // among the outputs before they are rounded
    auto aborted = [&]() { return *reinterpret_cast<volatile uint32_t*>(&sm.abort) != 0u; };
    auto give_up = [&]() { flags |= kFlagTimeout; atomicOr(&sm.abort, 1u); };

    if (warp == 0) {
        if (lane == 0) {                                           // producer of x
            uint32_t g = 0;
            for (uint32_t t = clu; t < p.tiles && !aborted(); t += nclu) {
                const int tok0 = (int)((t / p.n_tiles) * kTok);
                for (uint32_t ks = 0; ks < KS; ++ks, ++g) {
                    const uint32_t s = g % kStages;
                    if (g >= (uint32_t)kStages && !wait_bar(&sm.empty[s], ((g / kStages) - 1u) & 1u)) give_up();
                    if (aborted()) break;
                    mbar_arrive_expect_tx(&sm.full[s], kTok * 128u);
                    tma_load_2d(sm.x[s], &p.map_x, &sm.full[s], (int)(ch0 * 256u + ks * 64u), tok0);
                }
            }
            sm.issued = g;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer
        // two stages at a time, so that their four barriers are tried together (a tile may end on an
        // odd stage: the positions are counted over all tiles)
        const uint64_t desc0 = smem_desc(smem_u32(sm.x[0]), 1u, 64u, 2u);
        uint32_t g = 0u, i = 0u;
        bool ok = true;
        for (uint32_t t = clu; ok && t < p.tiles; t += nclu, ++i) {
            if (i > 0u) ok = wait_bar_warp(&sm.acc_empty, (i - 1u) & 1u);
            tc_fence_after();
            for (uint32_t ks = 0; ok && ks < KS;) {
                const uint32_t n = min(2u, KS - ks), g1 = g + 1u;
                uint64_t* const bar[4] = {&sm.full[g % kStages], &sm.a_full[g % kABufs], &sm.full[g1 % kStages],
                                          &sm.a_full[g1 % kABufs]};
                const uint32_t parity[4] = {(g / kStages) & 1u, (g / kABufs) & 1u, (g1 / kStages) & 1u, (g1 / kABufs) & 1u};
                ok = wait_bars_warp(bar, parity, 2u * n);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (uint32_t u = 0; u < 2; ++u) {
                    if (u == n) break;
                    const uint32_t s = (g + u) % kStages, b = (g + u) % kABufs;
                    const uint64_t desc = desc0 + (uint64_t)(s * (kTok * 8u));
                    const uint32_t a0 = tmem + kACol + 32u * b;
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t j = 0; j < 4; ++j)
                            mma_f16(tmem, a0 + 8u * j, desc + 2u * j, kIdesc, (ks | u | j) != 0u ? 1u : 0u);
                        tc_commit(&sm.empty[s]);
                        tc_commit(&sm.a_free[b]);
                    }
                    __syncwarp();
                }
                ks += n;
                g += n;
            }
            if (ok && elect_one()) tc_commit(&sm.acc_full);
            __syncwarp();
        }
        if (!ok && lane == 0) give_up();
        if (lane == 0) sm.consumed = g;
        if (elect_one()) tc_commit(&sm.drain);
        __syncwarp();
        if (!wait_bar_warp(&sm.drain, 0u)) flags |= kFlagTimeout;
    } else if (warp >= 4 && warp < 12) {
        // ---- decoders: set 0 the even, set 1 the odd chunks (counted over all tiles)
        const uint32_t quad = (uint32_t)warp & 3u, set = ((uint32_t)warp - 4u) >> 2, piece = (uint32_t)lane & 7u,
                       sub = (uint32_t)lane >> 3;
        uint8_t* ring = sm.ring[warp - 4];
        const size_t pitch = p.K / 2u, spitch = p.K / 16u;
        uint32_t lt = clu, lc = set, ut = clu, uc = set, base = 0u;            // (tile, chunk) to load, to decode; stages before
        auto settle = [&](uint32_t& t, uint32_t& c) {
            while (t < p.tiles && c >= NC) {
                c -= NC;
                t += nclu;
            }
        };
        auto load = [&](uint32_t at) {
            if (lt < p.tiles) {
                const uint32_t row0 = (lt % p.n_tiles) * 128u + 32u * quad, live = row0 < p.N ? min(32u, p.N - row0) : 0u;
                const uint32_t dst = smem_u32(ring) + at * kSlot, ks = (ch0 + lc) * 256u, k = ks + 32u * piece;
                const uint8_t* src = p.q + (size_t)(row0 + sub) * pitch + k / 2u;
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) {                 // rows sub + 4 i, 16-byte piece XOR row
                    const uint32_t r = sub + 4u * i, d = dst + 128u * r + 16u * (piece ^ (r & 7u));
                    if constexpr (kVec) {
                        const bool ok = r < live && k < p.K;
                        cp_async<16>(d, ok ? src : p.q, ok ? 16u : 0u);
                    } else {
#pragma unroll
                        for (uint32_t h = 0; h < 2; ++h) {
                            const bool ok = r < live && k + 16u * h < p.K;
                            cp_async<8>(d + 8u * h, ok ? src + 8u * h : p.q, ok ? 8u : 0u);
                        }
                    }
                    src += 4u * pitch;
                }
                const uint8_t* ss = p.sc + (size_t)(row0 + lane) * spitch + ks / 16u;
                const uint32_t sd = dst + 4096u + 16u * lane;
                const bool mine = (uint32_t)lane < live;
                if constexpr (kVec) {
#pragma unroll
                    for (uint32_t h = 0; h < 4; ++h) {
                        const bool ok = mine && ks + 64u * h < p.K;
                        cp_async<4>(sd + 4u * h, ok ? ss + 4u * h : p.sc, ok ? 4u : 0u);
                    }
                } else {
#pragma unroll
                    for (uint32_t h = 0; h < 4; ++h) {
                        uint32_t w = 0u;
#pragma unroll
                        for (uint32_t b = 0; b < 4; ++b)
                            if (mine && ks + 64u * h + 16u * b < p.K) w |= (uint32_t)__ldg(ss + 4u * h + b) << (8u * b);
                        *reinterpret_cast<uint32_t*>(ring + at * kSlot + 4096u + 16u * lane + 4u * h) = w;
                    }
                }
                lc += 2u;
                settle(lt, lc);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        settle(lt, lc);
        settle(ut, uc);
        base = (ut - clu) / nclu * KS;
        for (uint32_t i = 0; i < (uint32_t)kDepth; ++i) load(i);
        bool quit = false;
        for (uint32_t at = 0u; ut < p.tiles && !quit; at = at + 1u == (uint32_t)kDepth ? 0u : at + 1u) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            __syncwarp();
            const uint8_t* slot = ring + at * kSlot;
            const uint32_t ns = min(4u, KS - 4u * uc);
#pragma unroll 1
            for (uint32_t i = 0; i < ns; ++i) {
                const uint32_t g = base + 4u * uc + i, b = g % kABufs;
                const uint4 qa = *reinterpret_cast<const uint4*>(slot + 128u * lane + 16u * ((2u * i) ^ (lane & 7u)));
                const uint4 qb = *reinterpret_cast<const uint4*>(slot + 128u * lane + 16u * ((2u * i + 1u) ^ (lane & 7u)));
                const uint32_t q[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
                uint32_t o[32];
                decode64<kDt>(o, q, *reinterpret_cast<const uint32_t*>(slot + 4096u + 16u * lane + 4u * i));
                const bool ok = g < (uint32_t)kABufs || wait_bar(&sm.a_free[b], ((g / kABufs) - 1u) & 1u);
                const bool timed_out = __any_sync(0xFFFFFFFFu, !ok);
                quit = timed_out || __any_sync(0xFFFFFFFFu, aborted());
                if (quit) {
                    if (timed_out && lane == 0) give_up();
                    break;
                }
                tc_fence_after();
                tmem_st<32>(tmem + ((32u * quad) << 16) + kACol + 32u * b, o);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.a_full[b]);
            }
            __syncwarp();                                          // the slot has been read
            if (quit) break;
            load(at);
            uc += 2u;
            settle(ut, uc);
            base = (ut - clu) / nclu * KS;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
    } else if (warp >= 12) {
        // ---- epilogue: lanes 32 quad .. + 31 (one weight row per thread), columns (tokens) of half h
        const uint32_t quad = (uint32_t)warp & 3u, h = warp >= 16 ? 1u : 0u;
        uint8_t* st = sm.stg[warp - 12];
        const float s2 = *p.d_s2;
        constexpr uint32_t kCols = kTok / 2;
        uint32_t i = 0;
        for (uint32_t t = clu; t < p.tiles; t += nclu, ++i) {
            const bool ok = !aborted() && wait_bar(&sm.acc_full, i & 1u);
            if (!ok) {
                if (!aborted()) give_up();
                break;
            }
            tc_fence_after();
            __syncwarp();
            const uint32_t n0 = (t % p.n_tiles) * 128u + 32u * quad, tok0 = (t / p.n_tiles) * kTok + h * kCols;
            const uint32_t taddr = tmem + ((32u * quad) << 16) + h * kCols;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_empty);
            };
            if (p.z > 1u) {                                        // (one tile per cluster)
#pragma unroll 1
                for (uint32_t c = 0; c < kCols; c += 16u) {
                    float v[16];
                    tmem_ld16(taddr + c, v);
#pragma unroll
                    for (uint32_t k = 0; k < 16; ++k) part[(h * kCols + c + k) * 128u + 32u * quad + lane] = v[k];
                }
                release();
                continue;
            }
            if constexpr (kOut == 2) {
#pragma unroll 1
                for (uint32_t c = 0; c < kCols; c += 16u) {
                    float v[16];
                    tmem_ld16(taddr + c, v);
#pragma unroll
                    for (uint32_t k = 0; k < 16; ++k) {
                        odd.see(v[k] * s2);                        // (what lies outside the output is 0 s2, or NaN with all of it)
                        if (tok0 + c + k < p.T && n0 + lane < p.N)
                            static_cast<float*>(p.out)[(int64_t)(tok0 + c + k) * p.ldd + n0 + lane] = v[k] * s2;
                    }
                }
                release();
            } else {
                // converted into registers first: the accumulator is released before the stores
                uint32_t w[kCols / 2];
#pragma unroll
                for (uint32_t c = 0; c < kCols; c += 16u) {
                    float v[16];
                    tmem_ld16(taddr + c, v);
#pragma unroll
                    for (uint32_t k = 0; k < 16; ++k) odd.see(v[k] * s2);
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k)
                        w[c / 2 + k] = (uint32_t)to16<kOut>(v[2 * k] * s2) | (uint32_t)to16<kOut>(v[2 * k + 1] * s2) << 16;
                }
                release();
                const bool vec = p.vec != 0u && n0 + 32u <= p.N;
#pragma unroll
                for (uint32_t c = 0; c < kCols; c += 32u) {
                    constexpr uint32_t kBlk = kCols < 32u ? kCols : 32u;   // tokens per block
#pragma unroll
                    for (uint32_t k = 0; k < kBlk; ++k)            // [token][32 rows] of 16 bits
                        *reinterpret_cast<uint16_t*>(st + 64u * k + 2u * lane) = (uint16_t)(w[(c + k) / 2] >> (16u * (k & 1u)));
                    __syncwarp();
                    if (vec) {
#pragma unroll
                        for (uint32_t k = 0; k < kBlk / 8u; ++k) {
                            const uint32_t tok = 8u * k + ((uint32_t)lane >> 2), at = tok0 + c + tok;
                            const uint4 x = *reinterpret_cast<const uint4*>(st + 64u * tok + 16u * (lane & 3));
                            if (at < p.T)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (int64_t)at * p.ldd + n0 + 8u * (lane & 3)) = x;
                        }
                    } else {
                        for (uint32_t k = 0; k < kBlk; ++k)
                            if (tok0 + c + k < p.T && n0 + lane < p.N)
                                static_cast<uint16_t*>(p.out)[(int64_t)(tok0 + c + k) * p.ldd + n0 + lane] =
                                    *reinterpret_cast<const uint16_t*>(st + 64u * k + 2u * lane);
                    }
                    __syncwarp();
                }
            }
        }
    }

    // ---- teardown: copies loaded but never multiplied, the cluster's sums, tensor memory
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0)
        for (uint32_t g = sm.consumed; g < sm.issued; ++g)
            if (!wait_bar(&sm.full[g % kStages], (g / kStages) & 1u)) flags |= kFlagTimeout;
    if (p.z > 1u) {
        cluster_sync();
        const uint32_t n0 = (clu % p.n_tiles) * 128u, tok0 = (clu / p.n_tiles) * kTok;
        const float s2 = *p.d_s2;
        const uint32_t rows = min(128u, p.N - n0), toks = min((uint32_t)kTok, p.T - tok0);
        // four weight rows of a token per thread
        const uint32_t j1 = (rank + 1u) * toks / p.z;
        for (uint32_t i = (rank * toks / p.z) * 32u + threadIdx.x; i < j1 * 32u; i += kThreads) {
            const uint32_t r = 4u * (i & 31u), tok = i >> 5;
            if (r >= rows) continue;
            const float4 sum = cluster_sum4(part + 4u * i, p.z);
            const float o[4] = {sum.x * s2, sum.y * s2, sum.z * s2, sum.w * s2};
            if (cluster_any(&sm.abort, p.z)) continue;             // a CTA that gave up has no sums to add
#pragma unroll
            for (uint32_t k = 0; k < 4u; ++k)
                if (r + k < rows) {
                    odd.see(o[k]);
                    store1<kOut>(p.out, (int64_t)(tok0 + tok) * p.ldd + n0 + r + k, o[k]);
                }
        }
        cluster_sync();                                            // the others have read this CTA's sums
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512u);
    }
    flags = __reduce_or_sync(0xFFFFFFFFu, flags | odd.flag());
    if (lane == 0) flag_or(p.d_flags, flags);
}

static bool x_map(CUtensorMap* map, const void* x, int dt, int64_t T, int64_t K, int64_t ldx, uint32_t box_rows)
{
    auto enc = encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)T};
    const cuuint64_t strides[1] = {(cuuint64_t)ldx * 2u};
    const cuuint32_t box[2] = {64u, box_rows};
    const cuuint32_t es[2] = {1u, 1u};
    return enc(map, dt == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(x),
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kTok, int kDt, int kOut, bool kVec>
static cudaError_t run(Params& p, cudaStream_t s)
{
    static bool ready[64] = {};
    static int fits[64][kMaxSplit + 1] = {};
    auto kern = linear_mma_kernel<kTok, kDt, kOut, kVec>;
    static_assert(kTok == 256 || kStages<kTok> * 128 >= 512, "the partial sums take the place of x");
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
    const uint32_t sms = (uint32_t)num_sms();
    // every CTA keeps a chunk; a wave beside its chunks (launch, first loads, the cluster's sums): some
    // 3 chunks' time.  With more tiles than SMs a CTA walks several unsplit, the next one's loads under
    // the last one's stores (1000 x 2880 x 2880 on tiles of 128, 184 of them: 38 us, 52 in clusters of 2).  (The sums of
    // 256 token columns would leave nothing of x's stages to spare.)
    p.z = kTok <= 128 && p.tiles <= sms ? split_tiles(kern, kThreads, smem, p.tiles, p.chunks, 1u, 3u, fits, dev) : 1u;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.z > 1u ? p.tiles * p.z : p.tiles < sms ? p.tiles : sms, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.z;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.z > 1u ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int kTok>
static cudaError_t pick(Params& p, int dt, int out_dt, bool vec, cudaStream_t s)
{
    auto by_out = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (out_dt == 0) return vec ? run<kTok, D, 0, true>(p, s) : run<kTok, D, 0, false>(p, s);
        if (out_dt == 1) return vec ? run<kTok, D, 1, true>(p, s) : run<kTok, D, 1, false>(p, s);
        return vec ? run<kTok, D, 2, true>(p, s) : run<kTok, D, 2, false>(p, s);
    };
    return dt == 0 ? by_out(std::integral_constant<int, 0>{}) : by_out(std::integral_constant<int, 1>{});
}

}  // namespace w4mma

cudaError_t launch_linear_w4a16_mma(const void* x, int dt, int64_t T, int64_t K, int64_t ldx, const uint8_t* q,
                                    const uint8_t* sc, const float* d_s2, int64_t N, int out_dt, void* out, int64_t ldd,
                                    uint32_t* d_flags, cudaStream_t s)
{
    using namespace w4mma;
    Params p = {};
    p.q = q;
    p.sc = sc;
    p.d_s2 = d_s2;
    p.out = out;
    p.ldd = ldd;
    p.T = (uint32_t)T;
    p.N = (uint32_t)N;
    p.K = (uint32_t)K;
    p.n_tiles = (uint32_t)((N + 127) / 128);
    p.chunks = (uint32_t)((K + 255) / 256);
    p.vec = ldd % 8 == 0 ? 1u : 0u;
    p.d_flags = d_flags;
    const uint32_t sms = (uint32_t)num_sms();
    // the widest token tile that the rows fill, but 128 instead of 256 while those tiles fit the SMs at once (they
    // can split K then), or where they cost less: waves x (stages + a tile's end) + what a launch costs, in stages
    // of some 0.34 us, which hardly depend on the width.  128 / 256, us: 300 x 8192 x 8192 93.6 / 51.8, 1000 x
    // 2880 x 2880 37.3 / 26.0, 256 x 16384 x 2048 30.9 / 21.5, 600 x 4096 x 1024 17.0 / 13.9; 600 x 2880 x 2880
    // 21.7 / 25.6, 512 x 4096 x 4096 29.5 / 30.9, 800 x 5000 x 512 13.1 / 19.9.
    uint32_t tok = T <= 32 ? 32u : T <= 64 ? 64u : T <= 128 ? 128u : 256u;
    auto tiles = [&](uint32_t k) { return (uint64_t)p.n_tiles * (uint64_t)((T + k - 1) / k); };
    if (tok == 256u) {
        const uint64_t stages = (uint64_t)(K + 63) / 64, narrow = (tiles(128u) + sms - 1u) / sms, wide = (tiles(256u) + sms - 1u) / sms;
        if (narrow == 1u || narrow * (stages + 2u) + 20u <= wide * (stages + stages / 20u + 6u) + 28u) tok = 128u;
    }
    p.tiles = (uint32_t)tiles(tok);
    if (!x_map(&p.map_x, x, dt, T, K, ldx, tok)) return cudaErrorInvalidValue;
    const bool vec = K % 64 == 0;                                  // (16-byte aligned codes, 4-byte aligned scales)
    if (tok == 32u) return pick<32>(p, dt, out_dt, vec, s);
    if (tok == 64u) return pick<64>(p, dt, out_dt, vec, s);
    if (tok == 128u) return pick<128>(p, dt, out_dt, vec, s);
    return pick<256>(p, dt, out_dt, vec, s);
}

}  // namespace nv4
