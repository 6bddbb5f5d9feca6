// nv4_mxfp4.cuh -- what the kernels that quantize to MXFP4 share (the rule: variants.cu).
#pragma once

#include "nv4_common.cuh"

namespace nv4 {

template <int kIn>
__device__ __forceinline__ void load16(const void* x, int64_t off, float v[16], uint32_t& amax_bits)
{
    amax_bits = 0u;
    if constexpr (kIn == 0) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + off);
        const uint4 a = __ldcs(src), b = __ldcs(src + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        }
        amax_bits = max(m & 0xFFFFu, m >> 16) << 16;
    } else {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const float*>(x) + off);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 t = __ldcs(src + k);
            const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                amax_bits = max(amax_bits, w[j] & 0x7FFFFFFFu);
                v[4 * k + j] = __uint_as_float(w[j]);
            }
        }
    }
}

// floor(log2(a)) for a finite positive FP32 bit pattern (normal or subnormal).
__device__ __forceinline__ int floor_log2_bits(uint32_t b)
{
    const int e = (int)(b >> 23);
    return e != 0 ? e - 127 : -149 + (31 - __clz(b));
}

// 2^k as FP32 for k in [-149, 127] (exact).
__device__ __forceinline__ float pow2f(int k)
{
    return k >= -126 ? __uint_as_float((uint32_t)(k + 127) << 23) : __uint_as_float(1u << (k + 149));
}

// The E8M0 code of a block with the largest magnitude ab (FP32 bits; 0xFF for a NaN or Inf) and
// this lane's 16 codes of it.
__device__ __forceinline__ uint32_t mxfp4_encode16(const float (&v)[16], uint32_t ab, uint32_t& c0, uint32_t& c1)
{
    c0 = c1 = 0u;
    if (ab >= 0x7F800000u) return 0xFFu;
    const int e = ab == 0u ? -127 : max(floor_log2_bits(ab) - 2, -127);
    const float inv = pow2f(-e);                                   // normal: -e in [-125, 127]
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(v[i], inv);
    c0 = cvt_e2m1x8(y);
    c1 = cvt_e2m1x8(y + 8);
    return (uint32_t)(e + 127);
}

}  // namespace nv4
