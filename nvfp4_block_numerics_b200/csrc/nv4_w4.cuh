// nv4_w4.cuh -- the product of a few BF16 / FP16 rows with NVFP4 weights: what the weight-only
// linear layer and the mixture-of-experts kernels share.
//
// A warp multiplies 16 weight rows by up to 8 * NT token rows over K in chunks of 256, with
// mma.m16n8k16 (weights are the 16-row operand, tokens the 8-column one).  Lane (g, t) of the
// warp (g = lane / 4, t = lane % 4) holds 64 elements of a chunk of weight rows g and g + 8, 32
// consecutive ones of either half, and feeds them to 16 MMA steps of 4 elements: a dot product
// does not care which K-element sits in which MMA slot as long as both operands agree, so the
// codes need no shuffling.
//
// The weights stream through a ring in shared memory that each warp fills for itself with
// cp.async, kDepth chunks ahead, across the ends of tiles: no barrier, no register holds what is
// in flight, and the loop stays small (with the ring in registers, three chunks unrolled, every
// launch paid for fetching the code: 16 warps took 2600 clocks for their first chunks).
//
// e2m1 * e4m3 has at most 6 significant bits and lies on multiples of 2^-10 below 2688: exact
// in FP16, so a weight is decoded by one conversion (cvt.rn.f16x2.e2m1x2, two codes) and one
// multiply; measured in registers alone 15.8 T weights/s against the 11.6 T/s that HBM can
// deliver.  The same through BF16 (mask and shift, bf16x2 multiply) gives 9.4 T/s, below it.
// So the token rows are FP16 too.  FP16 rows are taken as they are.  BF16 rows are multiplied by
// 2^4 and converted, exact for magnitudes from 2^-21 to 2^12 (8 significant bits above the last
// FP16 bit, 2^-24).  If a call has others, its rows are read again, each with a power of two of
// its own (largest exponent to 2^14): exact for elements down to 2^-31 of the row's largest.  If
// a row spans more, or holds a NaN, an Inf or a BF16 subnormal, the call uses BF16 operands
// (kWide: the same codes, converted once more), which is exact for every input.
#pragma once

#include <cstdint>

#include "nv4_async.cuh"
#include "nv4_common.cuh"
#include "nv4_cpasync.cuh"
#include "nv4_internal.h"

namespace nv4 {
namespace w4 {

constexpr int kThreads = 512;                     // 16 warps, one CTA per SM
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kChunk = 256;                  // K-elements of one warp step
constexpr int kDepth = 3;                         // chunks of 16 rows in flight per warp
constexpr int kDepth32 = 2;                       // chunks of 2 x 16 rows
constexpr uint32_t kSlot = 16u * 128u + 16u * 16u;          // codes and scales of 16 rows x 256
constexpr uint32_t kRing = kWarps * kDepth * kSlot;         // bytes for all warps
constexpr uint32_t kRing32 = kWarps * kDepth32 * 2u * kSlot;

// Where this lane's share of a tile's rows g (a) and g + 8 (b) lies, and the bytes a copy of it
// has (0: no such row).  Set once per tile; chunk c is a constant offset away.
struct Rows16 {
    const uint8_t *qa, *qb, *sa, *sb;
    uint32_t na, nb;

    __device__ __forceinline__ void set(const uint8_t* q0, const uint8_t* s0, const uint8_t* q1, const uint8_t* s1, bool la,
                                        bool lb)
    {
        const uint32_t t = threadIdx.x & 3u;
        qa = q0 + 16u * t;
        qb = q1 + 16u * t;
        sa = s0 + 4u * t;
        sb = s1 + 4u * t;
        na = la ? 16u : 0u;
        nb = lb ? 16u : 0u;
    }
};

// Starts the loads of chunk c of 16 weight rows into a ring slot.  Slot: four 16-byte vectors per
// lane (row g halves 0 and 1, row g + 8 halves 0 and 1), then the scales, 16 bytes per row.
// kVec: K a multiple of 64 and 4-byte aligned scales; else 8 bytes of codes at a time, scales byte
// by byte through registers.
template <bool kVec>
__device__ __forceinline__ void load_chunk(uint8_t* slot, const Rows16& r, uint32_t c, uint32_t K)
{
    const uint32_t lane = threadIdx.x & 31u, t = lane & 3u;
    const uint32_t dst = smem_u32(slot) + 16u * lane, sdst = smem_u32(slot) + 2048u + 4u * lane;   // scales: row g, word t
    const uint8_t *qa = r.qa + c * 128u, *qb = r.qb + c * 128u, *sa = r.sa + c * 16u, *sb = r.sb + c * 16u;
    if (kVec && (c + 1u) * kChunk <= K) {
        cp_async<16>(dst, qa, r.na);
        cp_async<16>(dst + 512u, qa + 64u, r.na);
        cp_async<16>(dst + 1024u, qb, r.nb);
        cp_async<16>(dst + 1536u, qb + 64u, r.nb);
        cp_async<4>(sdst, sa, r.na >> 2);
        cp_async<4>(sdst + 128u, sb, r.nb >> 2);
        return;
    }
    const uint32_t ks = c * kChunk + 64u * t;
#pragma unroll
    for (uint32_t p = 0; p < 2; ++p) {
        const uint32_t k = c * kChunk + 128u * p + 32u * t;
        if constexpr (kVec) {
            cp_async<16>(dst + 512u * p, qa + 64u * p, k < K ? r.na : 0u);
            cp_async<16>(dst + 1024u + 512u * p, qb + 64u * p, k < K ? r.nb : 0u);
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
                cp_async<8>(dst + 512u * p + 8u * j, qa + 64u * p + 8u * j, k + 16u * j < K ? r.na >> 1 : 0u);
                cp_async<8>(dst + 1024u + 512u * p + 8u * j, qb + 64u * p + 8u * j, k + 16u * j < K ? r.nb >> 1 : 0u);
            }
        }
    }
    if constexpr (kVec) {
        cp_async<4>(sdst, sa, ks < K ? r.na >> 2 : 0u);
        cp_async<4>(sdst + 128u, sb, ks < K ? r.nb >> 2 : 0u);
    } else {
        uint32_t a = 0u, b = 0u;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            if (r.na != 0u && ks + 16u * j < K) a |= (uint32_t)__ldg(sa + j) << (8u * j);
            if (r.nb != 0u && ks + 16u * j < K) b |= (uint32_t)__ldg(sb + j) << (8u * j);
        }
        *reinterpret_cast<uint32_t*>(slot + 2048u + 4u * lane) = a;
        *reinterpret_cast<uint32_t*>(slot + 2048u + 128u + 4u * lane) = b;
    }
}

// Walks a warp's steps: load(slot) starts the next step's loads, use(slot) multiplies the next
// one.  begin() before the token rows are staged, run() after.
template <int kSlots, uint32_t kBytes>
struct RingOf {
    uint8_t* base;                                // this warp's slots
    uint32_t steps, issued;

    template <class Load>
    __device__ __forceinline__ void begin(uint8_t* b, uint32_t n, Load& load)
    {
        base = b;
        steps = n;
        issued = 0u;
        for (int i = 0; i < kSlots; ++i) {
            if (issued < steps) load(base + issued * kBytes);
            ++issued;
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }

    template <class Load, class Use>
    __device__ __forceinline__ void run(Load& load, Use use)
    {
        uint32_t at = 0u;
        for (uint32_t i = 0; i < steps; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
            __syncwarp();
            uint8_t* slot = base + at * kBytes;
            use(slot);
            __syncwarp();                         // the slot has been read
            if (issued < steps) load(slot);
            ++issued;
            asm volatile("cp.async.commit_group;" ::: "memory");
            at = at + 1u == (uint32_t)kSlots ? 0u : at + 1u;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
};
using Ring = RingOf<kDepth, kSlot>;
using Ring32 = RingOf<kDepth32, 2u * kSlot>;

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two FP16 values that BF16 holds exactly, as BF16.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h)
{
    float lo, hi;
    f16x2_to_f32(h, lo, hi);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two E4M3 scale bytes as FP16, each in both halves of a word.
__device__ __forceinline__ void scale_pair(uint16_t s, uint32_t (&p)[2])
{
    uint32_t a;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(s));
    p[0] = __byte_perm(a, a, 0x1010);
    p[1] = __byte_perm(a, a, 0x3232);
}

template <bool kWide>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if constexpr (kWide)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Independent accumulators per 8-token tile: an MMA waits for the one before it on the same
// accumulator, and with one chain of 16 per chunk that latency, not the decoding, set the pace
// (156 clocks per chunk and SM with one chain, T = 5, K = 16384).
template <int NT>
constexpr int kChains = NT == 1 ? 4 : 2;

template <int NT, int kCh>
using AccOf = float[kCh][NT][4];
template <int NT>
using Acc = float[kChains<NT>][NT][4];

// acc += 16 weight rows x token rows over half p of one chunk.  x(j, u): this lane's 16-byte vector of
// token 8 j + g, the 8 elements from 128 (u / 4) + 32 t + 8 (u % 4) of the chunk on.
template <bool kWide, int NT, int kCh, class X>
__device__ __forceinline__ void mma_half(AccOf<NT, kCh>& acc, const uint8_t* slot, uint32_t p, X x)
{
    const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
    const uint4 qa = *reinterpret_cast<const uint4*>(slot + 512u * p + 16u * lane);
    const uint4 qb = *reinterpret_cast<const uint4*>(slot + 1024u + 512u * p + 16u * lane);
    uint32_t s0[2], s1[2];
    scale_pair(*reinterpret_cast<const uint16_t*>(slot + 2048u + 16u * g + 8u * p + 2u * t), s0);
    scale_pair(*reinterpret_cast<const uint16_t*>(slot + 2048u + 128u + 16u * g + 8u * p + 2u * t), s1);
    const uint32_t wa[4] = {qa.x, qa.y, qa.z, qa.w}, wb[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u) {
        uint32_t a[4], b[4];
        cvt_e2m1x8_to_f16x8(wa[u], a);
        cvt_e2m1x8_to_f16x8(wb[u], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = mul_f16x2(a[i], s0[u >> 1]);
            b[i] = mul_f16x2(b[i], s1[u >> 1]);
            if constexpr (kWide) {
                a[i] = f16x2_to_bf16x2(a[i]);
                b[i] = f16x2_to_bf16x2(b[i]);
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < (uint32_t)NT; ++j) {
            const uint4 v = x(j, 4u * p + u);
            mma<kWide>(acc[(2u * u) % kCh][j], a[0], b[0], a[1], b[1], v.x, v.y);
            mma<kWide>(acc[(2u * u + 1u) % kCh][j], a[2], b[2], a[3], b[3], v.z, v.w);
        }
    }
}

template <bool kWide, int NT, int kCh, class X>
__device__ __forceinline__ void mma_step(AccOf<NT, kCh>& acc, const uint8_t* slot, X x)
{
#pragma unroll
    for (uint32_t p = 0; p < 2; ++p) mma_half<kWide, NT, kCh>(acc, slot, p, x);
}

// Token rows in shared memory, xs: the chunk's [8][m][4] vectors (u, token, t).  Columns past m
// are given token 0's values: nothing reads what they add up to.
template <bool kWide, int NT>
__device__ __forceinline__ void mma_chunk(Acc<NT>& acc, const uint8_t* slot, const uint4* xs, uint32_t m)
{
    const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
    const uint4* x0[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x0[j] = xs + (8u * j + g < m ? 8u * j + g : 0u) * 4u + t;
    mma_step<kWide, NT, kChains<NT>>(acc, slot, [&](uint32_t j, uint32_t u) { return x0[j][u * m * 4u]; });
}

// Up to 8 token rows in global memory against kHalves groups of 16 weight rows (slot, slot + kSlot),
// which share what is loaded of the tokens.  row: this lane's (column g's), chunk: where the step
// begins.  kWide: BF16 as the caller gave it, K elements.  Else FP16 in vector order, zero-padded to
// whole chunks: the 32 vectors of a chunk as [u][t], so that the four lanes of a column read 64
// consecutive bytes (in the natural order they touch four places 64 bytes apart, and L1 was what
// bounded the gate / up product of 48 tokens: 85% busy, 176 us).
template <bool kWide, int kHalves, int kCh>
__device__ __forceinline__ void mma_rows(AccOf<1, kCh> (&acc)[kHalves], const uint8_t* slot, const uint16_t* row, uint32_t chunk,
                                         uint32_t K)
{
    const uint32_t t = threadIdx.x & 3u;
    uint4 v[8];
#pragma unroll
    for (uint32_t u = 0; u < 8; ++u) {
        if constexpr (kWide) {
            const uint32_t at = chunk * kChunk + 128u * (u >> 2) + 32u * t + 8u * (u & 3u);
            v[u] = at < K ? *reinterpret_cast<const uint4*>(row + at) : make_uint4(0u, 0u, 0u, 0u);
        } else {
            v[u] = *reinterpret_cast<const uint4*>(row + chunk * kChunk + 32u * u + 8u * t);
        }
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
        mma_step<kWide, 1, kCh>(acc[h], slot + h * kSlot, [&](uint32_t, uint32_t u) { return v[u]; });
}

// Element offset, in a row in vector order, of the 8 values from 8 v on.
__device__ __forceinline__ uint32_t vec_offset(uint32_t v)
{
    const uint32_t l = v & 31u;
    return (v >> 5) * kChunk + (4u * (l >> 4) + (l & 3u)) * 32u + ((l & 15u) >> 2) * 8u;
}

__host__ __device__ inline uint32_t padded(uint32_t K) { return (K + kChunk - 1u) / kChunk * kChunk; }

// ---------------------------------------------------------------- token rows into shared memory
// Per token: exponent statistics and the factor that undoes its scaling.
struct Rows {
    uint32_t emax[kMaxFewRows], emin[kMaxFewRows];          // largest / smallest non-zero BF16 magnitude bits
    float descale[kMaxFewRows];
};

// 2^k for a biased exponent field, clamped to what FP32 holds from above (254) and, as the
// subnormal 2^-127, from below (0).
__device__ __forceinline__ float exp_field(int e)
{
    return e <= 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e > 254 ? 254 : e) << 23);
}

// Where the 8 values from 8 l on of chunk c of token i of m go.
__device__ __forceinline__ uint32_t vec_at(uint32_t c, uint32_t l, uint32_t m, uint32_t i)
{
    return ((c * 8u + 4u * (l >> 4) + (l & 3u)) * m + i) * 4u + ((l & 15u) >> 2);
}

// Converts m token rows (row(i): pointer to K values of the input type, 16-byte aligned) into
// xs, [chunk][8][m][4] vectors, zero-padded to whole chunks.  kDt 0: BF16, 1: FP16.  Returns
// (to every thread) whether the product has to use BF16 operands.  All threads take part; ends
// with a CTA barrier.  A warp takes one chunk of one token at a time.
template <int kDt, class RowPtr>
__device__ __forceinline__ bool stage_tokens(uint4* xs, Rows& rows, uint32_t m, uint32_t K, RowPtr row)
{
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t nch = (K + kChunk - 1u) / kChunk;
    auto fetch = [&](uint32_t i, uint32_t c) {
        const uint32_t k = c * kChunk + 8u * lane;
        return k < K ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row(i)) + k))
                     : make_uint4(0u, 0u, 0u, 0u);
    };
    auto put = [&](uint32_t i, uint32_t c, uint4 v, bool convert, float f) {
        if (convert) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                    : "=r"(w[j])
                    : "f"(__fmul_rn(bf16_hi(w[j]), f)), "f"(__fmul_rn(bf16_lo(w[j]), f)));
        }
        xs[vec_at(c, lane, m, i)] = v;
    };
    // magnitudes of 8 values: the largest, and the smallest non-zero one less one
    auto scan = [&](const uint4& v, uint32_t& hi, uint32_t& lo) {
        const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi = __vmaxu2(hi, w[j]);
            lo = __vminu2(lo, __vsub2(w[j], 0x00010001u));        // zero becomes 0xFFFF
        }
    };
    // warp w takes steps w, w + 16, ... of the m x nch (token, chunk) pairs, token outermost, four
    // loads at a time
    auto each = [&](auto&& body) {
        uint32_t i = 0u, c = warp;
        auto settle = [&]() {
            while (c >= nch && i < m) {
                c -= nch;
                ++i;
            }
        };
        settle();
        while (i < m) {
            uint32_t is[4], cs[4];
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                is[j] = i;
                cs[j] = c;
                v[j] = i < m ? fetch(i, c) : make_uint4(0u, 0u, 0u, 0u);
                c += kWarps;
                settle();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (is[j] < m) body(is[j], cs[j], v[j]);
        }
    };
    if (threadIdx.x < m) rows.descale[threadIdx.x] = kDt == 0 ? 0x1p-4f : 1.0f;
    if constexpr (kDt == 1) {
        each([&](uint32_t i, uint32_t c, const uint4& v) { put(i, c, v, false, 1.0f); });
        __syncthreads();
        return false;
    }
    uint32_t hi = 0u, lo = 0xFFFFFFFFu;
    each([&](uint32_t i, uint32_t c, const uint4& v) {
        scan(v, hi, lo);
        put(i, c, v, true, 0x1p4f);
    });
    // BF16 magnitudes 2^-21 = 0x3500 to below 2^12 = 0x4580, or zero
    if (__syncthreads_or(max(hi & 0xFFFFu, hi >> 16) >= 0x4580u || min(lo & 0xFFFFu, lo >> 16) + 1u < 0x3500u) == 0)
        return false;
    // rows by their own exponents
    if (threadIdx.x < m) {
        rows.emax[threadIdx.x] = 0u;
        rows.emin[threadIdx.x] = 0xFFFFu;
    }
    __syncthreads();
    each([&](uint32_t i, uint32_t, const uint4& v) {
        hi = 0u;
        lo = 0xFFFFFFFFu;
        scan(v, hi, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, max(hi & 0xFFFFu, hi >> 16));
        lo = __reduce_min_sync(0xFFFFFFFFu, min(lo & 0xFFFFu, lo >> 16));
        if (lane == 0) {
            atomicMax(&rows.emax[i], hi);
            atomicMin(&rows.emin[i], lo);
        }
    });
    __syncthreads();
    bool mine = false;
    if (threadIdx.x < m && rows.emax[threadIdx.x] != 0u) {
        const int e1 = (int)(rows.emax[threadIdx.x] >> 7), e0 = (int)((rows.emin[threadIdx.x] + 1u) >> 7);
        mine = e1 == 255 || e0 == 0 || e1 - e0 > 31 || e1 < 20;
    }
    const bool wide = __syncthreads_or(mine) != 0;
    if (threadIdx.x < m) {
        const int e1 = (int)(rows.emax[threadIdx.x] >> 7);
        rows.descale[threadIdx.x] = wide || e1 == 0 ? 1.0f : exp_field(e1 - 14);
    }
    each([&](uint32_t i, uint32_t c, const uint4& v) {
        const int e1 = (int)(rows.emax[i] >> 7);
        put(i, c, v, !wide, e1 == 0 ? 1.0f : exp_field(268 - e1));
    });
    __syncthreads();
    return wide;
}

// How many warps share a tile (its K range split between them): the power of two with the
// shortest longest warp for ntile tiles of nch chunks on 16 warps, a tile's end and its barrier
// counted as a quarter of a chunk's time.
__host__ __device__ __forceinline__ uint32_t split_of(uint32_t ntile, uint32_t nch)
{
    uint32_t best = 1u, cost = 0xFFFFFFFFu;
#pragma unroll
    for (uint32_t lg = 0u; lg <= 4u; ++lg) {
        const uint32_t wk = 1u << lg, groups = (uint32_t)kWarps >> lg;
        const uint32_t c = ((ntile + groups - 1u) >> (4u - lg)) * (((nch + wk - 1u) >> lg) * 8u + (lg > 0u ? 2u : 1u));
        if (c < cost && (lg == 0u || wk <= nch)) {
            cost = c;
            best = wk;
        }
    }
    return best;
}

// Barrier of the wk warps of a group (at most 8 groups of more than one warp: barriers 1-8).
__device__ __forceinline__ void group_barrier(uint32_t grp, uint32_t wk)
{
    if (wk == 1u) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1u + grp), "r"(32u * wk) : "memory");
}

// Adds wk partial sums, kTile apart, in warp order.
template <uint32_t kTile>
__device__ __forceinline__ float sum_parts(const float* first, uint32_t wk)
{
    float s = 0.0f;
#pragma unroll 4
    for (uint32_t w = 0; w < wk; ++w) s += first[(size_t)w * kTile];
    return s;
}

template <int NT, int kCh = kChains<NT>>
__device__ __forceinline__ void clear(AccOf<NT, kCh>& acc)
{
#pragma unroll
    for (int c = 0; c < kCh; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[c][j][0] = acc[c][j][1] = acc[c][j][2] = acc[c][j][3] = 0.0f;
}

// The chains' sum, in chain (0).
template <int NT, int kCh = kChains<NT>>
__device__ __forceinline__ void join(AccOf<NT, kCh>& acc)
{
#pragma unroll
    for (int c = kCh / 2; c > 0; c /= 2)
#pragma unroll
        for (int i = 0; i < c; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] += acc[i + c][j][v];
}

// A warp's 16 x 8 NT sums to its place in shared memory, [16][8 NT].
template <int NT, int kCh = kChains<NT>>
__device__ __forceinline__ void put_part(float* part, AccOf<NT, kCh>& chains, uint32_t g, uint32_t t)
{
    join<NT, kCh>(chains);
    const float (&acc)[NT][4] = chains[0];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        *reinterpret_cast<float2*>(part + g * (8 * NT) + 8 * j + 2 * t) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(part + (g + 8) * (8 * NT) + 8 * j + 2 * t) = make_float2(acc[j][2], acc[j][3]);
    }
}

// Programmatic dependent launch: wait for the kernel before (its writes are visible then); let
// the kernel behind start its own prologue.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <int kOut>
__device__ __forceinline__ void store_out(void* out, int64_t at, float v)
{
    if constexpr (kOut == 2) {
        static_cast<float*>(out)[at] = v;
    } else {
        uint16_t b;
        if constexpr (kOut == 0)
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
        else
            asm("cvt.rn.f16.f32 %0, %1;" : "=h"(b) : "f"(v));
        static_cast<uint16_t*>(out)[at] = b;
    }
}

}  // namespace w4
}  // namespace nv4
