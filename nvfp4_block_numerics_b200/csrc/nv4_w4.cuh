// nv4_w4.cuh -- the product of a few BF16 / FP16 rows with NVFP4 weights: what the weight-only
// linear layer and the mixture-of-experts kernels share.
//
// A warp multiplies 16 weight rows by up to 8 * NT token rows over K in chunks of 256, with
// mma.m16n8k16 (weights are the 16-row operand, tokens the 8-column one).  Lane (g, t) of the
// warp (g = lane / 4, t = lane % 4) holds 64 consecutive K-elements of weight rows g and g + 8,
// loaded straight from global memory (32 bytes of codes, 4 block scales each), and feeds them to
// 16 MMA steps of 4 elements: a dot product does not care which K-element sits in which MMA
// slot as long as both operands agree, so the codes need no shuffling and no shared memory.
// e2m1 * e4m3 has at most 6 significant bits and lies on multiples of 2^-10 below 2688: exact
// in FP16, so a weight is decoded by one conversion (cvt.rn.f16x2.e2m1x2, two codes) and one
// multiply; measured in registers alone 15.8 T weights/s against the 11.6 T/s that HBM can
// deliver.  The same through BF16 (mask and shift, bf16x2 multiply) gives 9.4 T/s, below it.
// So the token rows are FP16 too.  FP16 rows are taken as they are.  BF16 rows are scaled by a
// power of two per row (largest exponent to 2^14) and converted: exact for elements down to
// 2^-31 of the row's largest (8 significant bits above the last FP16 bit, 2^-24).  A row that
// spans more, or holds a NaN, an Inf or a BF16 subnormal, switches its whole pass to BF16
// operands (kWide: the same codes, converted once more), which is exact for every input.
#pragma once

#include <cstdint>

#include "nv4_common.cuh"

namespace nv4 {
namespace w4 {

constexpr int kThreads = 512;                     // 16 warps, one CTA per SM
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kChunk = 256;                  // K-elements of one warp step

struct Frag {
    uint32_t q0[8], q1[8];                        // 64 codes of row g, of row g + 8
    uint32_t s0, s1;                              // their 4 block scales (E4M3 bytes)
};

// 64 codes and 4 scales of one weight row from element k0 on; zeros where the row ends or is
// not live.  kVec: K a multiple of 64 and 32-byte aligned rows (one 32-byte load).
template <bool kVec>
__device__ __forceinline__ void load_row(uint32_t (&q)[8], uint32_t& s, const uint8_t* __restrict__ qrow,
                                         const uint8_t* __restrict__ srow, uint32_t k0, uint32_t K, bool live)
{
    if constexpr (kVec) {
        if (live && k0 < K) {
            asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]),
                           "=r"(q[7])
                         : "l"(qrow + (k0 >> 1)));
            s = __ldg(reinterpret_cast<const uint32_t*>(srow + (k0 >> 4)));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = 0u;
            s = 0u;
        }
    } else {
        s = 0u;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            uint2 v = make_uint2(0u, 0u);
            if (live && k0 + 16u * j < K) {
                v = __ldg(reinterpret_cast<const uint2*>(qrow + (k0 >> 1) + 8u * j));
                s |= (uint32_t)__ldg(srow + (k0 >> 4) + j) << (8u * j);
            }
            q[2 * j] = v.x;
            q[2 * j + 1] = v.y;
        }
    }
}

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

// Four E4M3 scale bytes as FP16, each in both halves of a word.
__device__ __forceinline__ void scale_pairs(uint32_t s, uint32_t (&p)[4])
{
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(s & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(s >> 16)));
    p[0] = __byte_perm(a, a, 0x1010);
    p[1] = __byte_perm(a, a, 0x3232);
    p[2] = __byte_perm(b, b, 0x1010);
    p[3] = __byte_perm(b, b, 0x3232);
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

// acc += 16 weight rows x m token rows over one chunk.  xs: the chunk's token values,
// [8][m][4] 16-byte vectors: vector (u, token, t) holds elements 64 t + 8 u .. + 7.
template <bool kWide, int NT>
__device__ __forceinline__ void mma_chunk(float (&acc)[NT][4], const Frag& f, const uint4* xs, uint32_t m,
                                          uint32_t g, uint32_t t)
{
    uint32_t p0[4], p1[4];
    scale_pairs(f.s0, p0);
    scale_pairs(f.s1, p1);
#pragma unroll
    for (uint32_t u = 0; u < 8; ++u) {
        uint32_t a[4], b[4];
        cvt_e2m1x8_to_f16x8(f.q0[u], a);
        cvt_e2m1x8_to_f16x8(f.q1[u], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = mul_f16x2(a[i], p0[u >> 1]);
            b[i] = mul_f16x2(b[i], p1[u >> 1]);
            if constexpr (kWide) {
                a[i] = f16x2_to_bf16x2(a[i]);
                b[i] = f16x2_to_bf16x2(b[i]);
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < (uint32_t)NT; ++j) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (8u * j + g < m) x = xs[(u * m + 8u * j + g) * 4u + t];
            mma<kWide>(acc[j], a[0], b[0], a[1], b[1], x.x, x.y);
            mma<kWide>(acc[j], a[2], b[2], a[3], b[3], x.z, x.w);
        }
    }
}

// ---------------------------------------------------------------- token rows into shared memory
// Per token of a pass: exponent statistics and the factor that undoes its scaling.
struct Rows {
    uint32_t emax[24], emin[24];                  // largest / smallest non-zero BF16 magnitude bits
    float descale[24];
};

// 2^k for a biased exponent field, clamped to what FP32 holds from above (254) and, as the
// subnormal 2^-127, from below (0).
__device__ __forceinline__ float exp_field(int e)
{
    return e <= 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e > 254 ? 254 : e) << 23);
}

// Converts m token rows (row(i): pointer to K values of the input type, 16-byte aligned) into
// xs, [chunk][8][m][4] vectors, zero-padded to whole chunks.  kDt 0: BF16, 1: FP16.  Returns
// (to every thread) whether the pass has to use BF16 operands.  All threads take part; ends
// with a CTA barrier.
template <int kDt, class RowPtr>
__device__ __forceinline__ bool stage_tokens(uint4* xs, Rows& rows, uint32_t m, uint32_t K, RowPtr row)
{
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t nch = (K + kChunk - 1u) / kChunk, n = m * nch;
    bool wide = false;
    if constexpr (kDt == 0) {
        if (threadIdx.x < m) {
            rows.emax[threadIdx.x] = 0u;
            rows.emin[threadIdx.x] = 0xFFFFu;
        }
        __syncthreads();
        for (uint32_t it = warp; it < n; it += kWarps) {
            const uint32_t i = it / nch, k = (it - i * nch) * kChunk + 8u * lane;
            uint32_t hi = 0u, lo = 0xFFFFFFFFu;
            if (k < K) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row(i)) + k));
                const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    hi = __vmaxu2(hi, w[j]);
                    lo = __vminu2(lo, __vsub2(w[j], 0x00010001u));    // zero becomes 0xFFFF
                }
            }
            hi = __reduce_max_sync(0xFFFFFFFFu, max(hi & 0xFFFFu, hi >> 16));
            lo = __reduce_min_sync(0xFFFFFFFFu, min(lo & 0xFFFFu, lo >> 16));
            if (lane == 0) {
                atomicMax(&rows.emax[i], hi);
                atomicMin(&rows.emin[i], lo);
            }
        }
        __syncthreads();
        bool mine = false;
        if (threadIdx.x < m && rows.emax[threadIdx.x] != 0u) {
            const int e1 = (int)(rows.emax[threadIdx.x] >> 7), e0 = (int)((rows.emin[threadIdx.x] + 1u) >> 7);
            mine = e1 == 255 || e0 == 0 || e1 - e0 > 31 || e1 < 20;
        }
        wide = __syncthreads_or(mine) != 0;
        if (threadIdx.x < m) {
            const int e1 = (int)(rows.emax[threadIdx.x] >> 7);
            rows.descale[threadIdx.x] = wide || e1 == 0 ? 1.0f : exp_field(e1 - 14);
        }
    } else {
        if (threadIdx.x < m) rows.descale[threadIdx.x] = 1.0f;
    }
    for (uint32_t it = warp; it < n; it += kWarps) {
        const uint32_t i = it / nch, c = it - i * nch, k = c * kChunk + 8u * lane;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (k < K) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row(i)) + k));
        if constexpr (kDt == 0) {
            if (!wide) {
                const int e1 = (int)(rows.emax[i] >> 7);
                const float f = e1 == 0 ? 1.0f : exp_field(268 - e1);
                uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                        : "=r"(w[j])
                        : "f"(__fmul_rn(bf16_hi(w[j]), f)), "f"(__fmul_rn(bf16_lo(w[j]), f)));
            }
        }
        xs[((c * 8u + (lane & 7u)) * m + i) * 4u + (lane >> 3)] = v;
    }
    __syncthreads();
    return wide;
}

// How many warps share a tile (its K range split between them): the power of two that gives
// the shortest longest warp for ntile tiles of nch chunks on 16 warps; the smaller one of equals
// (fewer partial sums to add).
__device__ __forceinline__ uint32_t split_of(uint32_t ntile, uint32_t nch)
{
    uint32_t best = 1u, cost = 0xFFFFFFFFu;
    for (uint32_t wk = 1u; wk <= (uint32_t)kWarps && (wk == 1u || wk <= nch); wk *= 2u) {
        const uint32_t groups = kWarps / wk;
        const uint32_t c = ((ntile + groups - 1u) / groups) * ((nch + wk - 1u) / wk);
        if (c < cost) {
            cost = c;
            best = wk;
        }
    }
    return best;
}

__device__ __forceinline__ void group_barrier(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

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
