// w4a16.cu -- the weight-only linear layer: BF16 / FP16 rows times NVFP4 weights (sm_100a).
//
// [CAL] layer table (W4A16 layers keep their activations in 16 bits); [FLOW] 3.4 (the value of a
// code is e2m1 * s_b * s2).  y[t, n] = s2 * sum_k x[t, k] * (e2m1(q[n, k]) * e4m3(s[n, k/16])):
// the weight products are exact, the sum runs in FP32, s2 is applied to the sum.
//
// One persistent CTA per SM owns a contiguous range of weight rows (balanced to one row) and
// walks it in tiles of at most 16 rows; its 16 warps split a tile's K range (nv4_w4.cuh), so a
// weight byte is read once per pass of up to 24 tokens.  Token rows are staged once per pass.
#include "nv4_internal.h"
#include <type_traits>

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
    uint32_t T, N, K, cap;                        // cap: tokens per pass
};

template <int kDt, int kOut, bool kVec, int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Rows rows;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
    const uint32_t nch = (p.K + kChunk - 1u) / kChunk;
    uint4* xs = reinterpret_cast<uint4*>(smem);
    float* red = reinterpret_cast<float*>(smem + (size_t)nch * 512u * p.cap);     // [2][16 warps][16][8 NT]
    constexpr uint32_t kTile = 16u * 8u * NT;
    const uint32_t r0 = (uint32_t)((uint64_t)blockIdx.x * p.N / gridDim.x);
    const uint32_t R = (uint32_t)((uint64_t)(blockIdx.x + 1u) * p.N / gridDim.x) - r0;
    const uint32_t ntile = (R + 15u) / 16u;
    const uint32_t wk = split_of(ntile, nch), groups = kWarps / wk;
    const uint32_t grp = warp / wk, wig = warp - grp * wk;
    const float s2 = *p.d_s2;

    auto load = [&](Frag& f, uint32_t tile, uint32_t c) {
        const uint32_t a = r0 + tile * R / ntile, b = r0 + (tile + 1u) * R / ntile;
        const uint32_t k0 = c * kChunk + 64u * t, ra = a + g, rb = a + 8u + g;
        load_row<kVec>(f.q0, f.s0, p.q + (size_t)ra * (p.K / 2u), p.sc + (size_t)ra * (p.K / 16u), k0, p.K, ra < b);
        load_row<kVec>(f.q1, f.s1, p.q + (size_t)rb * (p.K / 2u), p.sc + (size_t)rb * (p.K / 16u), k0, p.K, rb < b);
    };

    for (uint32_t p0 = 0; p0 < p.T; p0 += p.cap) {
        const uint32_t m = min(p.cap, p.T - p0);
        Frag cur;
        if (grp < ntile) load(cur, grp, wig);     // in flight while the tokens are staged
        if (p0 > 0) __syncthreads();              // the previous pass has read its tokens
        const bool wide = stage_tokens<kDt>(xs, rows, m, p.K, [&](uint32_t i) {
            return static_cast<const void*>(static_cast<const uint16_t*>(p.x) + (int64_t)(p0 + i) * p.ldx);
        });
        uint32_t buf = 0u;
        for (uint32_t tile = grp; tile < ntile; tile += groups, buf ^= 1u) {
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
            for (uint32_t c = wig; c < nch; c += wk) {
                Frag next;
                const bool more = c + wk < nch;
                if (more || tile + groups < ntile) load(next, more ? tile : tile + groups, more ? c + wk : wig);
                const uint4* xc = xs + (size_t)c * 32u * m;
                if (kDt == 0 && wide)
                    mma_chunk<true, NT>(acc, cur, xc, m, g, t);
                else
                    mma_chunk<false, NT>(acc, cur, xc, m, g, t);
                cur = next;
            }
            float* part = red + (size_t)(buf * kWarps + warp) * kTile;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                *reinterpret_cast<float2*>(part + g * (8 * NT) + 8 * j + 2 * t) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2*>(part + (g + 8) * (8 * NT) + 8 * j + 2 * t) = make_float2(acc[j][2], acc[j][3]);
            }
            if (wk == 1u) __syncwarp();
            else group_barrier(1u + grp, 32u * wk);           // at most 8 groups: barriers 1-8
            // the group adds its warps' partial sums, one (token, row) per thread, in warp order
            const uint32_t a = r0 + tile * R / ntile, nr = r0 + (tile + 1u) * R / ntile - a;
            const float* first = red + (size_t)(buf * kWarps + grp * wk) * kTile;
            for (uint32_t i = wig * 32u + lane; i < 16u * m; i += 32u * wk) {
                const uint32_t r = i & 15u, tok = i >> 4;
                if (r >= nr) continue;
                float s = 0.0f;
                for (uint32_t w = 0; w < wk; ++w) s += first[(size_t)w * kTile + r * (8 * NT) + tok];
                store_out<kOut>(p.out, (int64_t)(p0 + tok) * p.ldd + a + r, s * s2 * rows.descale[tok]);
            }
        }
    }
}

template <int kDt, int kOut, bool kVec>
static cudaError_t run_linear(const LinearParams& p, uint32_t nt, cudaStream_t s)
{
    auto kern = nt == 1 ? linear_kernel<kDt, kOut, kVec, 1>
                        : nt == 2 ? linear_kernel<kDt, kOut, kVec, 2> : linear_kernel<kDt, kOut, kVec, 3>;
    const size_t smem = (size_t)((p.K + kChunk - 1u) / kChunk) * 512u * p.cap + 2u * kWarps * 16u * 8u * nt * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const uint32_t sms = (uint32_t)num_sms();
    kern<<<p.N < sms ? p.N : sms, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace w4

cudaError_t launch_linear_w4a16(const void* x, int dt, int64_t T, int64_t K, int64_t ldx, const uint8_t* q,
                                const uint8_t* sc, const float* d_s2, int64_t N, int out_dt, void* out, int64_t ldd,
                                cudaStream_t s)
{
    using namespace w4;
    LinearParams p{x, ldx, q, sc, d_s2, out, ldd, (uint32_t)T, (uint32_t)N, (uint32_t)K, 0u};
    // tokens per pass: what shared memory holds beside the partial sums, 24 at most
    const uint32_t per_token = (uint32_t)((K + kChunk - 1) / kChunk) * 512u;
    uint32_t cap = (uint32_t)(T < 24 ? T : 24);
    while (cap > 1u && (size_t)cap * per_token + 2u * kWarps * 128u * ((cap + 7u) / 8u) * sizeof(float) > kMaxSmemW4) --cap;
    p.cap = cap;
    const uint32_t nt = (cap + 7u) / 8u;
    const bool vec = K % 64 == 0 && (reinterpret_cast<uintptr_t>(q) & 31u) == 0u && (reinterpret_cast<uintptr_t>(sc) & 3u) == 0u;
    auto pick = [&](auto dt_c) {
        constexpr int D = decltype(dt_c)::value;
        if (out_dt == 0) return vec ? run_linear<D, 0, true>(p, nt, s) : run_linear<D, 0, false>(p, nt, s);
        if (out_dt == 1) return vec ? run_linear<D, 1, true>(p, nt, s) : run_linear<D, 1, false>(p, nt, s);
        return vec ? run_linear<D, 2, true>(p, nt, s) : run_linear<D, 2, false>(p, nt, s);
    };
    return dt == 0 ? pick(std::integral_constant<int, 0>{}) : pick(std::integral_constant<int, 1>{});
}

}  // namespace nv4
