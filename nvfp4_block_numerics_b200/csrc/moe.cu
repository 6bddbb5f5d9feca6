// moe.cu -- a mixture-of-experts layer for a few tokens on NVFP4 expert weights (sm_100a).
//
// [DSPARK], [CAST] section 3 (routed experts w1 / w3 / w2 stored in NVFP4, w1 and w3 with a
// common scale_2); [CAL] layer table (expert layers W4A16).
//
//   route    logits[t, e] = sum_h x[t, h] wr[e, h]; p = softmax(logits); the k largest logits
//            (ties: the lower index); weight = p, or p / sum of the chosen p
//   experts  h = silu(gate_e x) * (up_e x);  y[t] = sum_j weight[t, j] * down_e h
//
// Four launches, each a programmatic dependent of the one before.  Gate / up fills an SM's register file and
// down most of it, so that on an SM their prologues (lists, first weights) begin once the kernel in front
// has left it, not under it; only the router's and the small kernels' CTAs share one.
//   * moe_route_kernel: a 16-CTA cluster per one or two tokens.  The products are exact and are summed in
//     FP64, so that the choice of experts is that of the exact logits unless two of them lie within the
//     sums' rounding (2^-53 of the sum of magnitudes, per addition).  For BF16 that takes FP64 products (formed
//     in FP32, which some leave, 48 tokens took 12.6 us instead of 16.2).  It also converts BF16 token rows to
//     FP16, each with a power of two of its own (moe_rows_kernel does where the experts are given).
//   * moe_up_kernel, one CTA per SM: the flat list (expert, i) of gate / up row pairs of the
//     chosen experts is cut into one contiguous range per CTA, walked in tiles of 16 pairs, two
//     MMA row groups of 8 gate rows and the same 8 up rows, so both halves of an h meet in one
//     thread.  h goes to the workspace in FP32.
//   * moe_hidden_kernel, one CTA per (expert, token) row of h: scales it by a power of two and
//     writes it as two FP16 values, h = hi + 2^-11 lo: 22 bits, a relative error of 2^-22 (one FP16
//     value, 2^-11, was a visible part of the outputs' error).
//   * moe_down_kernel, one CTA per SM: a CTA owns a range of output rows for all tokens and all
//     chosen experts, so the sum over a token's experts needs no other CTA and is in a fixed
//     order.  The row's scale, the expert's scale_2 and the routing weight are applied in FP32.
// The floor is reading the chosen experts' weights once from HBM; both products (nv4_w4.cuh) split
// their rows evenly over the SMs, to one row, and read the token rows through L1.  An expert with
// more than 8 tokens is multiplied in passes of 8.
// 64 experts of 1536 x 4096, 8 per token: 1 token 38.7 us on the device, 45 a call (85 MB; by itself, from a cold
// L2, router 9, gate / up 24, hidden 5, down 18), 48 tokens 257 us either way (680 MB; 16, 118, 5.5, 111).
// Bound, 48 tokens: decoding on the issue slots (54% gate / up, 43% down) and L1 (52%, 61%) at 3.9 and 2.1 TB/s
// (the second part of h costs down 27 of its 111 us); 1 token: four launches' latencies.
#include <cfloat>

#include "nv4_async.cuh"
#include "nv4_internal.h"
#include "nv4_w4.cuh"

namespace nv4 {

namespace moe {

using w4::kChunk;
using w4::kThreads;
using w4::kWarps;

constexpr uint32_t kPass = 8;                     // tokens of one expert multiplied at once

// ---------------------------------------------------------------- token rows
// The workspace: x as FP16 in vector order [T][H padded], what undoes each row's scaling
// (negative: the row is not held by FP16, see w4::stage_tokens), h in FP32 [rows][I], h in two FP16
// parts in vector order [rows][2][I padded], its scales.
struct Work {
    uint16_t* x16;
    float* xd;
    float* h;
    uint16_t* h16;
    float* hd;
};

__host__ __device__ inline size_t align256(size_t n) { return (n + 255u) & ~(size_t)255u; }

__host__ inline Work work_of(void* w, size_t T, size_t k, size_t H, size_t I, size_t* bytes)
{
    uint8_t* b = static_cast<uint8_t*>(w);
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t* r = b + at;
        at += align256(n);
        return r;
    };
    Work o;
    o.x16 = reinterpret_cast<uint16_t*>(take(T * w4::padded((uint32_t)H) * 2u));
    o.xd = reinterpret_cast<float*>(take(T * 4u));
    o.h = reinterpret_cast<float*>(take(T * k * I * 4u));
    o.h16 = reinterpret_cast<uint16_t*>(take(T * k * w4::padded((uint32_t)I) * 4u));
    o.hd = reinterpret_cast<float*>(take(T * k * 4u));
    *bytes = at;
    return o;
}

// The CTA's threads bring one row into vector order, a BF16 one (kDt 0) converted to FP16 with a
// power of two of its own.
template <int kDt>
__device__ __forceinline__ void convert_row(const uint16_t* x, uint32_t H, uint16_t* out, float* descale, uint32_t* red)
{
    const uint32_t tid = threadIdx.x, n = blockDim.x, warp = tid >> 5, lane = tid & 31u;
    float f = 1.0f;
    if constexpr (kDt == 0) {
        uint32_t hi = 0u, lo = 0xFFFFFFFFu;
        for (uint32_t k = 8u * tid; k < H; k += 8u * n) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + k));
            const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hi = __vmaxu2(hi, w[j]);
                lo = __vminu2(lo, __vsub2(w[j], 0x00010001u));    // zero becomes 0xFFFF
            }
        }
        hi = __reduce_max_sync(0xFFFFFFFFu, max(hi & 0xFFFFu, hi >> 16));
        lo = __reduce_min_sync(0xFFFFFFFFu, min(lo & 0xFFFFu, lo >> 16));
        if (lane == 0u) {
            red[warp] = hi;
            red[32u + warp] = lo;
        }
        __syncthreads();
        for (uint32_t w = 0; w < n / 32u; ++w) {
            hi = max(hi, red[w]);
            lo = min(lo, red[32u + w]);
        }
        const int e1 = (int)(hi >> 7), e0 = (int)((lo + 1u) >> 7);
        const bool wide = hi != 0u && (e1 == 255 || e0 == 0 || e1 - e0 > 31 || e1 < 20);
        f = hi == 0u || wide ? 1.0f : w4::exp_field(268 - e1);
        if (tid == 0u) *descale = wide ? -1.0f : hi == 0u ? 1.0f : w4::exp_field(e1 - 14);
    } else {
        if (tid == 0u) *descale = 1.0f;
    }
    for (uint32_t i = tid; i < w4::padded(H) / 8u; i += n) {
        uint4 v = 8u * i < H ? __ldg(reinterpret_cast<const uint4*>(x + 8u * i)) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        if constexpr (kDt == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                    : "=r"(w[j])
                    : "f"(__fmul_rn(bf16_hi(w[j]), f)), "f"(__fmul_rn(bf16_lo(w[j]), f)));
        }
        *reinterpret_cast<uint4*>(out + w4::vec_offset(i)) = v;
    }
}

template <int kDt>
__global__ void __launch_bounds__(512) moe_rows_kernel(const void* x, int64_t ldx, uint32_t H, Work w)
{
    __shared__ uint32_t red[64];
    w4::pdl_launch();
    convert_row<kDt>(static_cast<const uint16_t*>(x) + (int64_t)blockIdx.x * ldx, H,
                     w.x16 + (size_t)blockIdx.x * w4::padded(H), w.xd + blockIdx.x, red);
}

// ---------------------------------------------------------------- router
constexpr int kRouteThreads = 512;
constexpr uint32_t kRouteCtas = 16;               // one cluster
constexpr uint32_t kRouteTokens = 2;              // tokens per cluster at most
constexpr uint32_t kRouteParts = 4;               // warps that share a logit, each a quarter of H

struct RouteParams {
    const void* x;
    int64_t ldx;
    const void* wr;                               // [E, H]
    int32_t* ids;
    float* weights;
    uint32_t T, H, E, k, renorm;
    uint32_t* d_flags;
    Work work;                                    // x16: null, or where to put the rows as FP16
};

template <int kDt>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kDt == 0) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        } else {
            f16x2_to_f32(w[i], f[2 * i], f[2 * i + 1]);
        }
    }
}

// kTok: tokens of the cluster (1, or up to kRouteTokens).  CTA i of the cluster collects the
// logits of token i and chooses: an expert's place is the number of experts that rank above it,
// so no round waits for the one before.
template <int kDt, int kTok>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const __grid_constant__ RouteParams p)
{
    __shared__ double part[kMaxMoeExperts][kRouteParts];
    __shared__ double logit[kMaxMoeExperts];
    __shared__ double chosen[kMaxMoeTopK];
    __shared__ double sums[kRouteThreads / 32];
    const uint32_t tid = threadIdx.x, rank = cluster_ctarank(), warp = tid >> 5, lane = tid & 31u;
    constexpr uint32_t kRW = kRouteThreads / 32;
    const uint32_t t0 = (blockIdx.x / kRouteCtas) * kTok, nt = min((uint32_t)kTok, p.T - t0);
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + (int64_t)t0 * p.ldx;
    const uint16_t* wr = static_cast<const uint16_t*>(p.wr);
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");              // this CTA runs
    w4::pdl_launch();

    // unit (expert, quarter): vectors of 8 values lane + 32 * quarter, + 128, ...
    bool waited = false;
    for (uint32_t u = rank * kRW + warp; u < p.E * kRouteParts; u += kRouteCtas * kRW) {
        const uint32_t e = u / kRouteParts, q = u % kRouteParts;
        double s[kTok][4];
#pragma unroll
        for (int i = 0; i < kTok; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0;
#pragma unroll 4
        for (uint32_t h = 8u * (lane + 32u * q); h < p.H; h += 8u * 32u * kRouteParts) {
            float w[8];
            unpack8<kDt>(__ldg(reinterpret_cast<const uint4*>(wr + (size_t)e * p.H + h)), w);
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                if ((uint32_t)i < nt) {
                    float v[8];
                    unpack8<kDt>(__ldg(reinterpret_cast<const uint4*>(x + (int64_t)i * p.ldx + h)), v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        // exact products; those of FP16 fit FP32 (2^-48 to 2^32), with one conversion instead of two
                        if constexpr (kDt == 0) s[i][j & 3] = fma((double)v[j], (double)w[j], s[i][j & 3]);
                        else s[i][j & 3] += (double)__fmul_rn(v[j], w[j]);
                    }
                }
            }
        }
        if (!waited) {                                             // the other CTAs run: write to them
            asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            waited = true;
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            double v = (s[i][0] + s[i][1]) + (s[i][2] + s[i][3]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
            if (lane == 0 && (uint32_t)i < nt) {
                uint32_t remote;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(&part[e][q])), "r"((uint32_t)i));
                asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(v) : "memory");
            }
        }
    }
    if (!waited) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    __syncwarp();
    cluster_sync();
    if (p.work.x16 != nullptr && rank >= kRouteTokens && rank - kRouteTokens < nt) {
        __shared__ uint32_t red[64];
        const uint32_t i = rank - kRouteTokens;
        convert_row<kDt>(x + (int64_t)i * p.ldx, p.H, p.work.x16 + (size_t)(t0 + i) * w4::padded(p.H), p.work.xd + t0 + i, red);
    }
    if (rank >= nt) return;
    const size_t row = (size_t)(t0 + rank) * p.k;
    uint32_t flags = 0u;
    if (tid < p.E) {
        const double v = (part[tid][0] + part[tid][1]) + (part[tid][2] + part[tid][3]);
        if (!(fabs(v) <= DBL_MAX)) flags = kFlagNonFinite;
        logit[tid] = v >= -DBL_MAX ? v : -DBL_MAX;                 // NaN and -inf rank last
    }
    __syncthreads();
    // expert e by `per` threads, each comparing it with its share of the others
    uint32_t lg = 0u;                                              // log2(per), per * E <= 512
    while (lg < 4u && (p.E << (lg + 1u)) <= (uint32_t)kRouteThreads) ++lg;
    const uint32_t e = tid >> lg, per = 1u << lg;
    uint32_t above = 0u;
    if (e < p.E) {
        const double mine = logit[e];
#pragma unroll 4
        for (uint32_t o = tid & (per - 1u); o < p.E; o += per)
            above += logit[o] > mine || (logit[o] == mine && o < e) ? 1u : 0u;
    }
    for (uint32_t d = 1u; d < per; d <<= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, d);
    if (e < p.E && above < p.k && (tid & (per - 1u)) == 0u) {
        p.ids[row + above] = (int32_t)e;
        chosen[above] = logit[e];
    }
    __syncthreads();
    const double top = chosen[0];
    if (p.renorm == 0u) {
        double s = tid < p.E ? exp(logit[tid] - top) : 0.0;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        if (lane == 0) sums[warp] = s;
        __syncthreads();
    }
    if (warp == 0u) {
        const double pj = lane < p.k ? exp(chosen[lane] - top) : 0.0;
        double s = p.renorm != 0u ? pj : lane < kRW ? sums[lane] : 0.0;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        if (lane < p.k) p.weights[row + lane] = (float)(pj / s);
    }
    flags = __reduce_or_sync(0xFFFFFFFFu, flags);
    if (lane == 0) flag_or(p.d_flags, flags);
}

// ---------------------------------------------------------------- the chosen experts
struct Experts {
    const void* x;
    int64_t ldx;
    const int32_t* ids;                           // [T, k]; outside [0, E): no expert
    const float* weights;
    const uint8_t *gq, *gs, *uq, *us, *dq, *ds;   // codes and scales: gate, up [E, I, H], down [E, H, I]
    const float *g2, *u2, *d2;                    // [E]
    Work work;
    void* out;
    int64_t ldd;
    uint32_t T, k, E, H, I;
    uint32_t* d_flags;
};

// (What a kernel in front on the stream wrote is read with coherent loads: a CTA may have started
// before it was written.)
//
// Which tokens chose which expert, built by every CTA for itself: a bit per token and expert, so
// that a token that names an expert twice has it once, and the order is that of the tokens.
// Rows: the (expert, token) pairs in that order; row r of h belongs to token tok[r].  Sub-lists:
// up to 8 rows of one expert.
struct Lists {
    unsigned long long mask[kMaxMoeExperts];
    uint8_t tok[kMaxMoePairs];
    uint16_t expert[kMaxMoeExperts];              // chosen experts in ascending order
    uint16_t first[kMaxMoeExperts + 1];           // their first rows
    uint16_t sub[kMaxMoeExperts + 1];             // and first sub-lists
    uint16_t slot[kMaxMoeExperts];                // expert -> its place among the chosen
    uint32_t scan[kWarps];
    uint32_t n, subs;                             // chosen experts, sub-lists

    // the chosen expert that sub-list s belongs to
    __device__ __forceinline__ uint32_t find(uint32_t s) const
    {
        uint32_t a = 0u, b = n;                   // sub[a] <= s < sub[b]
        while (b - a > 1u) {
            const uint32_t m = (a + b) >> 1;
            if (sub[m] <= s) a = m;
            else b = m;
        }
        return a;
    }
};

__device__ __forceinline__ void build_lists(Lists& L, const Experts& p)
{
    const uint32_t P = p.T * p.k, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    if (tid < p.E) L.mask[tid] = 0ull;
    __syncthreads();
    for (uint32_t i = tid; i < P; i += kThreads) {
        const int32_t e = __ldcg(p.ids + i);
        if (e >= 0 && e < (int32_t)p.E) atomicOr(&L.mask[e], 1ull << (i / p.k));
    }
    __syncthreads();
    // exclusive scan over the experts of rows (at most 2048, bits 0-11), sub-lists (at most 768,
    // bits 12-21) and chosen experts (at most 512, bits 22-31) in one word
    unsigned long long mask = tid < p.E ? L.mask[tid] : 0ull;
    const uint32_t cnt = (uint32_t)__popcll(mask), mine = cnt + (((cnt + 7u) >> 3) << 12) + (cnt != 0u ? 1u << 22 : 0u);
    uint32_t a = mine;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, a, d);
        if (lane >= d) a += o;
    }
    if (lane == 31u) L.scan[warp] = a;
    __syncthreads();
    uint32_t total = 0u;
#pragma unroll
    for (uint32_t w = 0; w < (uint32_t)kWarps; ++w) {
        const uint32_t v = L.scan[w];
        if (w < warp) a += v;
        total += v;
    }
    a -= mine;
    const uint32_t slot = a >> 22, at = a & 0xFFFu;
    if (cnt != 0u) {
        L.expert[slot] = (uint16_t)tid;
        L.first[slot] = (uint16_t)at;
        L.sub[slot] = (uint16_t)((a >> 12) & 0x3FFu);
        L.slot[tid] = (uint16_t)slot;
        for (uint32_t i = 0; mask != 0ull; ++i, mask &= mask - 1ull) L.tok[at + i] = (uint8_t)(__ffsll((long long)mask) - 1);
    }
    if (tid == 0u) {
        L.n = total >> 22;
        L.subs = (total >> 12) & 0x3FFu;
        L.first[total >> 22] = (uint16_t)(total & 0xFFFu);
        L.sub[total >> 22] = (uint16_t)L.subs;
    }
    __syncthreads();
}

// A sum of scaled rows times what undoes the row's scale (a power of two) and times scale_2, the one below 1
// first: neither the sum times a large one nor the product of two small ones leaves FP32 where the result does not.
__device__ __forceinline__ float two_scales(float sum, float d, float s2) { return d < 1.0f ? sum * d * s2 : sum * s2 * d; }

// ---------------------------------------------------------------- gate, up, SwiGLU
constexpr uint32_t kMaxSegs = 8;

// A run of row pairs of one sub-list in a CTA's range, in tiles of th pairs from tile0 on; its
// tokens are rows f0 .. f0 + m - 1 of the lists.
struct Seg {
    uint32_t expert, f0, m, i0, n, th, tile0;
};

struct Segs {
    Seg s[kMaxSegs];
    uint32_t n, ntile, pairs;
};

template <bool kVec>
__global__ void __launch_bounds__(kThreads, 1) moe_up_kernel(const __grid_constant__ Experts p)
{
    extern __shared__ __align__(16) uint8_t smem[];                // the warps' rings
    __shared__ Lists L;
    __shared__ Segs S;
    __shared__ __align__(16) float red[kWarps][32 * 8];            // [half][gate 8, up 8][column]
    __shared__ float descale[kMaxMoeTokens];
    constexpr uint32_t kTile = 32u * 8u;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const uint32_t nch = (p.H + kChunk - 1u) / kChunk;
    w4::pdl_wait();                                                // ids are the router's
    w4::pdl_launch();
    // the rows in their FP16 form, unless some BF16 row has none: then all as they are
    const float d = tid < p.T ? p.work.xd[tid] : 1.0f;             // (in flight while the lists are built)
    build_lists(L, p);
    const bool wide = __syncthreads_or(d < 0.0f) != 0;
    if (tid < p.T) descale[tid] = wide ? 1.0f : d;                 // (read behind the barriers below)
    const uint16_t* x = wide ? static_cast<const uint16_t*>(p.x) : p.work.x16;
    const int64_t ldx = wide ? p.ldx : (int64_t)w4::padded(p.H);
    const uint32_t total = L.subs * p.I;                           // at most 768 x 2^15
    uint32_t at = (uint32_t)((uint64_t)blockIdx.x * total / gridDim.x);
    const uint32_t end = (uint32_t)((uint64_t)(blockIdx.x + 1u) * total / gridDim.x);
    while (at < end) {
        if (tid == 0u) {
            uint32_t n = 0u, nt = 0u, w = at, s = w / p.I, a = L.find(s);
            while (w < end && n < kMaxSegs) {
                Seg& sg = S.s[n];
                sg.expert = L.expert[a];
                sg.f0 = L.first[a] + (s - L.sub[a]) * kPass;
                sg.m = min(kPass, L.first[a + 1u] - sg.f0);
                sg.i0 = w - s * p.I;
                sg.n = min(p.I - sg.i0, end - w);
                const uint32_t tiles = (sg.n + 15u) / 16u;
                sg.th = (sg.n + tiles - 1u) / tiles;
                sg.tile0 = nt;
                nt += (sg.n + sg.th - 1u) / sg.th;
                w += sg.n;
                ++n;
                ++s;
                if (s >= L.sub[a + 1u]) ++a;
            }
            S.n = n;
            S.ntile = nt;
            S.pairs = w - at;
        }
        __syncthreads();
        const uint32_t wk = w4::split_of(S.ntile, nch), groups = kWarps / wk, grp = warp / wk, wig = warp - grp * wk;
        const uint32_t my_tiles = grp < S.ntile ? (S.ntile - grp + groups - 1u) / groups : 0u;
        const uint32_t steps = my_tiles * (wig < nch ? (nch - wig + wk - 1u) / wk : 0u);
        uint32_t lt = grp, lc = wig, ls = 0u;
        w4::Rows16 rw[2];
        bool moved = true;
        auto load = [&](uint8_t* slot) {
            if (moved) {
                while (ls + 1u < S.n && lt >= S.s[ls + 1u].tile0) ++ls;
                const Seg& sg = S.s[ls];
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    const uint32_t r = 8u * h + g, i = (lt - sg.tile0) * sg.th + r;
                    const bool live = r < sg.th && i < sg.n;
                    const size_t row = ((size_t)sg.expert * p.I + sg.i0 + i) * (p.H / 2u);
                    rw[h].set(p.gq + row, p.gs + row / 8u, p.uq + row, p.us + row / 8u, live, live);
                }
                moved = false;
            }
            w4::load_chunk<kVec>(slot, rw[0], lc, p.H);
            w4::load_chunk<kVec>(slot + w4::kSlot, rw[1], lc, p.H);
            lc += wk;
            if (lc >= nch) {
                lc = wig;
                lt += groups;
                moved = true;
            }
        };
        w4::Ring32 ring;
        ring.begin(smem + warp * (w4::kDepth32 * 2u * w4::kSlot), steps, load);
        w4::AccOf<1, 2> acc[2];
        w4::clear<1, 2>(acc[0]);
        w4::clear<1, 2>(acc[1]);
        uint32_t ut = grp, uc = wig, us = 0u;
        const uint16_t* xr = nullptr;                              // column g's token row
        ring.run(load, [&](const uint8_t* slot) {
            if (uc == wig) {
                while (us + 1u < S.n && ut >= S.s[us + 1u].tile0) ++us;
                xr = x + (int64_t)L.tok[S.s[us].f0 + min(g, S.s[us].m - 1u)] * ldx;
            }
            if (wide) w4::mma_rows<true, 2, 2>(acc, slot, xr, uc, p.H);
            else w4::mma_rows<false, 2, 2>(acc, slot, xr, uc, p.H);
            uc += wk;
            if (uc < nch) return;
            w4::group_barrier(grp, wk);                            // the last tile's sums have been read
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w4::put_part<1, 2>(red[warp] + 16 * 8 * h, acc[h], g, t);
                w4::clear<1, 2>(acc[h]);
            }
            w4::group_barrier(grp, wk);
            const Seg& sg = S.s[us];
            const uint32_t a = (ut - sg.tile0) * sg.th, nr = min(sg.th, sg.n - a);
            const float* first = red[grp * wk];
            const float s_gate = __ldg(p.g2 + sg.expert), s_up = __ldg(p.u2 + sg.expert);
            for (uint32_t i = wig * 32u + lane; i < 16u * sg.m; i += 32u * wk) {
                const uint32_t r = i & 15u, col = i >> 4, hr = sg.f0 + col, at_r = (r >> 3) * 128u + (r & 7u) * 8u + col;
                if (r >= nr) continue;
                const float ds = descale[L.tok[hr]];
                const float gv = two_scales(w4::sum_parts<kTile>(first + at_r, wk), ds, s_gate);
                const float uv = two_scales(w4::sum_parts<kTile>(first + at_r + 64u, wk), ds, s_up);
                p.work.h[(size_t)hr * p.I + sg.i0 + a + r] = gv / (1.0f + expf(-gv)) * uv;
            }
            uc = wig;
            ut += groups;
        });
        at += S.pairs;
        __syncthreads();                                           // S and the sums are free
    }
}

// ---------------------------------------------------------------- h to two FP16 parts
// One CTA per row (rows that no pair has are converted too, and read by nothing).  What hi leaves of
// a value is at most 2^-11 of it (and exact in FP32): lo, 2^11 times that, is within FP16's range
// again and rounds it by 2^-22 of the value, or by 2^-50 of the row's largest.  Nothing is left of an
// Inf or a NaN.
__global__ void __launch_bounds__(256) moe_hidden_kernel(const __grid_constant__ Experts p)
{
    __shared__ uint32_t red[8];
    w4::pdl_wait();
    w4::pdl_launch();
    const uint32_t tid = threadIdx.x;
    const float4* src = reinterpret_cast<const float4*>(p.work.h + (size_t)blockIdx.x * p.I);
    constexpr int kKeep = 2;                                       // 8 values each
    float4 keep[kKeep][2];
    uint32_t top = 0u;
    auto scan = [&](const float4& v) {
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
            if (b < 0x7F800000u) top = max(top, b);                // the largest finite magnitude
        }
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const uint32_t v = tid + 256u * i;
        keep[i][0] = keep[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (8u * v < p.I) {
            keep[i][0] = src[2u * v];
            keep[i][1] = src[2u * v + 1u];
        }
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        scan(keep[i][0]);
        scan(keep[i][1]);
    }
    for (uint32_t v = tid + 256u * kKeep; 8u * v < p.I; v += 256u) {
        scan(src[2u * v]);
        scan(src[2u * v + 1u]);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((tid & 31u) == 0u) red[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) top = max(top, red[w]);
    const int e1 = (int)(top >> 23), fe = top == 0u ? 127 : min(268 - e1, 254);     // factor 2^(fe - 127): largest to 2^14
    const float f = w4::exp_field(fe);
    if (tid == 0u) p.work.hd[blockIdx.x] = w4::exp_field(254 - fe);
    auto put = [&](uint32_t v, const float4& a, const float4& b) {
        const float z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t o[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float s[2] = {__fmul_rn(z[2 * j], f), __fmul_rn(z[2 * j + 1], f)}, h[2];
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(s[1]), "f"(s[0]));
            f16x2_to_f32(o[j], h[0], h[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) s[i] = fabsf(h[i]) <= FLT_MAX ? (s[i] - h[i]) * 0x1p11f : 0.0f;
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(l[j]) : "f"(s[1]), "f"(s[0]));
        }
        uint16_t* at = p.work.h16 + 2u * (size_t)blockIdx.x * w4::padded(p.I) + w4::vec_offset(v);
        *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(at + w4::padded(p.I)) = make_uint4(l[0], l[1], l[2], l[3]);
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (8u * (tid + 256u * i) < w4::padded(p.I)) put(tid + 256u * i, keep[i][0], keep[i][1]);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (uint32_t v = tid + 256u * kKeep; 8u * v < w4::padded(p.I); v += 256u)
        put(v, 8u * v < p.I ? src[2u * v] : zero, 8u * v < p.I ? src[2u * v + 1u] : zero);
}

// ---------------------------------------------------------------- down, weighted sum
template <int kOut, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) moe_down_kernel(const __grid_constant__ Experts p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Lists L;
    float* Yall = reinterpret_cast<float*>(smem + w4::kRing);      // [16 warps][T][16]
    // of a row of h: its scale, routing weight x expert scale, in the order of two_scales; as many as there are pairs, the
    // rest of the SM is L1's
    float2* coef = reinterpret_cast<float2*>(Yall + (size_t)kWarps * p.T * 16u);
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const uint32_t r0 = (uint32_t)((uint64_t)blockIdx.x * p.H / gridDim.x);
    const uint32_t R = (uint32_t)((uint64_t)(blockIdx.x + 1u) * p.H / gridDim.x) - r0;
    const uint32_t ntile = (R + 15u) / 16u, th = (R + ntile - 1u) / ntile;      // at most 16 tiles: H <= 256 x CTAs
    const uint32_t wpt = kWarps / ntile, tile = warp % ntile, widx = warp / ntile;
    const uint32_t ta = tile * th, tn = ta < R ? min(th, R - ta) : 0u;
    const bool works = widx < wpt;
    float* Y = Yall + (size_t)warp * p.T * 16u;
    for (uint32_t i = lane; i < p.T * 16u; i += 32u) Y[i] = 0.0f;
    const uint32_t nch = (p.I + kChunk - 1u) / kChunk;
    // ids and weights were written before the two kernels in front of this one began
    build_lists(L, p);
    for (uint32_t i = tid; i < p.T * p.k; i += kThreads) {
        const uint32_t tok = i / p.k, j0 = tok * p.k;
        const int32_t e = __ldcg(p.ids + i);
        if (e < 0 || e >= (int32_t)p.E) continue;
        float w = 0.0f;
        bool first = true;                                         // the token's first mention of the expert: all its weights
        for (uint32_t j = j0; j < j0 + p.k; ++j) {
            const bool same = __ldcg(p.ids + j) == e;
            if (same && j < i) first = false;
            if (same) w += __ldcg(p.weights + j);
        }
        if (first) coef[L.first[L.slot[e]] + __popcll(L.mask[e] & ((1ull << tok) - 1ull))].y = w * __ldg(p.d2 + e);
    }
    // this warp's run of the tile's (sub-list, chunk) steps
    const uint32_t n = L.subs * nch, s0 = works ? (uint32_t)((uint64_t)widx * n / wpt) : 0u;
    const uint32_t steps = works ? (uint32_t)((uint64_t)(widx + 1u) * n / wpt) - s0 : 0u;
    uint32_t us = s0 / nch, uc = s0 - us * nch, ua = steps != 0u ? L.find(us) : 0u;
    uint32_t ls = us, lc = uc, la = ua;
    size_t row = 0u;                                               // byte offset of this lane's codes (scales: an eighth)
    bool moved = true;
    auto load = [&](uint8_t* slot) {
        if (moved) {
            if (ls >= L.sub[la + 1u]) ++la;
            row = ((size_t)L.expert[la] * p.H + r0 + ta + g) * (p.I / 2u);
            moved = false;
        }
        const uint32_t eight = 8u * (p.I / 2u);
        w4::Rows16 rw;
        rw.set(p.dq + row, p.ds + row / 8u, p.dq + row + eight, p.ds + row / 8u + eight / 8u, g < tn, g + 8u < tn);
        w4::load_chunk<kVec>(slot, rw, lc, p.I);
        if (++lc == nch) {
            lc = 0u;
            ++ls;
            moved = true;
        }
    };
    w4::Ring ring;
    ring.begin(smem + warp * (w4::kDepth * w4::kSlot), steps, load);
    w4::pdl_wait();                                                // h is complete
    __syncthreads();                                               // coef
    for (uint32_t i = tid; i < (uint32_t)L.first[L.n]; i += kThreads) {
        const float d = p.work.hd[i], c = coef[i].y;
        coef[i] = d < 1.0f ? make_float2(d, c) : make_float2(c, d);
    }
    __syncthreads();
    w4::AccOf<2, 2> acc;                                           // [chain][part of h]
    w4::clear<2, 2>(acc);
    const uint32_t part = w4::padded(p.I);
    uint32_t left = steps, f0 = 0u, m = 0u;
    const uint16_t* xr = nullptr;
    bool fresh = true, paired = false;
    ring.run(load, [&](const uint8_t* slot) {
        if (fresh) {
            if (us >= L.sub[ua + 1u]) ++ua;
            f0 = L.first[ua] + (us - L.sub[ua]) * kPass;
            m = min(kPass, L.first[ua + 1u] - f0);
            // up to 4 rows: both parts of a row are columns of one MMA, 4 apart (8 tokens of 64 experts 129 us, with
            // two MMAs 140; 1 token 38.9, 40.2; 48 tokens 258, 262)
            paired = m <= 4u;
            const uint32_t col = paired ? g & 3u : g;
            xr = p.work.h16 + 2u * (size_t)(f0 + min(col, m - 1u)) * part + (paired && g >= 4u ? part : 0u);
            fresh = false;
        }
        if (paired) {
            w4::mma_rows<false, 1, 4>(reinterpret_cast<w4::AccOf<1, 4>(&)[1]>(acc), slot, xr, uc, p.I);
        } else {
            const uint16_t* at = xr + uc * kChunk + 8u * t;
#pragma unroll 1                                                   // (what a launch pays for fetching the code counts)
            for (uint32_t q = 0; q < 2; ++q, at += 128u) {
                uint4 x[2][4];
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j)
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) x[j][u] = *reinterpret_cast<const uint4*>(at + j * part + 32u * u);
                w4::mma_half<false, 2, 2>(acc, slot, q, [&](uint32_t j, uint32_t u) { return x[j][u & 3u]; });
            }
        }
        --left;
        if (++uc < nch && left != 0u) return;
        // the sub-list's end: its columns, each times its coefficient, into the warp's sums
        float v[4];                                                // rows g (columns 2 t, 2 t + 1) and g + 8
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const float a = acc[0][0][i] + acc[1][0][i], b = acc[0][1][i] + acc[1][1][i];
            const float lo = __shfl_xor_sync(0xFFFFFFFFu, a + b, 2);           // paired: four chains of columns 4 - 7
            v[i] = paired ? a + b + lo * 0x1p-11f : a + b * 0x1p-11f;
        }
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
            const uint32_t col = 2u * t + i;
            if (col < m) {
                float* y = Y + (size_t)L.tok[f0 + col] * 16u;
                const float2 c = coef[f0 + col];
                y[g] += v[i] * c.x * c.y;
                y[g + 8] += v[2 + i] * c.x * c.y;
            }
        }
        __syncwarp();
        w4::clear<2, 2>(acc);
        uc = 0u;
        ++us;
        fresh = true;
    });
    __syncthreads();
    // ---- the warps' sums of a tile, in warp order
    NonFinite odd;                                                 // among the outputs before they are rounded
    for (uint32_t i = tid; i < p.T * R; i += kThreads) {
        const uint32_t tok = i / R, r = i - tok * R, tl = r / th, in = r - tl * th;
        float v = 0.0f;
#pragma unroll 4
        for (uint32_t w = 0; w < wpt; ++w) v += Yall[((size_t)(w * ntile + tl) * p.T + tok) * 16u + in];
        odd.see(v);
        w4::store_out<kOut>(p.out, (int64_t)tok * p.ldd + r0 + r, v);
    }
    const uint32_t flags = __reduce_or_sync(0xFFFFFFFFu, odd.flag());
    if (lane == 0u) flag_or(p.d_flags, flags);
}

template <class Kern, class P>
static cudaError_t launch(Kern kern, const P& p, uint32_t grid, uint32_t threads, size_t smem, uint32_t cluster, bool dependent,
                          cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1u) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Once per kernel and device: its shared memory limit, and clusters of 16.
template <class Kern>
static cudaError_t prepare(Kern kern, bool (&ready)[64], int smem, bool cluster16)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && ready[dev]) return cudaSuccess;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && cluster16) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev >= 0 && dev < 64) ready[dev] = true;
    return e;
}

template <int kDt, int kTok>
static cudaError_t run_route(const RouteParams& p, cudaStream_t s)
{
    static bool ready[64] = {};
    const cudaError_t e = prepare(moe_route_kernel<kDt, kTok>, ready, 0, true);
    if (e != cudaSuccess) return e;
    return launch(moe_route_kernel<kDt, kTok>, p, (p.T + kTok - 1u) / kTok * kRouteCtas, kRouteThreads, 0, kRouteCtas, false, s);
}

template <bool kVec>
static cudaError_t run_up(const Experts& p, cudaStream_t s)
{
    static bool ready[64] = {};
    const cudaError_t e = prepare(moe_up_kernel<kVec>, ready, (int)w4::kRing32, false);
    if (e != cudaSuccess) return e;
    return launch(moe_up_kernel<kVec>, p, (uint32_t)num_sms(), kThreads, w4::kRing32, 1u, true, s);
}

template <int kOut, bool kVec>
static cudaError_t run_down(const Experts& p, cudaStream_t s)
{
    static bool ready[64] = {};
    const uint32_t sms = (uint32_t)num_sms(), grid = p.H < sms ? p.H : sms;
    if ((p.H + grid - 1u) / grid > 16u * kWarps) return cudaErrorInvalidValue;
    auto smem = [](size_t T, size_t pairs) { return w4::kRing + kWarps * T * 16u * sizeof(float) + pairs * sizeof(float2); };
    const cudaError_t e = prepare(moe_down_kernel<kOut, kVec>, ready, (int)smem((size_t)kMaxMoeTokens, (size_t)kMaxMoePairs), false);
    if (e != cudaSuccess) return e;
    return launch(moe_down_kernel<kOut, kVec>, p, grid, kThreads, smem(p.T, (size_t)p.T * p.k), 1u, true, s);
}

}  // namespace moe

size_t moe_work_bytes(int64_t T, int64_t k, int64_t H, int64_t I)
{
    size_t n = 0;
    (void)moe::work_of(nullptr, (size_t)T, (size_t)k, (size_t)H, (size_t)I, &n);
    return n;
}

cudaError_t launch_moe_route(const void* x, int dt, int64_t T, int64_t H, int64_t ldx, const void* wr, int64_t E,
                             int top_k, int renorm, int32_t* ids, float* weights, const MoeExpertsArgs* then,
                             uint32_t* d_flags, cudaStream_t s)
{
    using namespace moe;
    RouteParams p{x, ldx, wr, ids, weights, (uint32_t)T, (uint32_t)H, (uint32_t)E, (uint32_t)top_k, (uint32_t)renorm, d_flags, {}};
    size_t n;
    if (then != nullptr) p.work = work_of(then->work, (size_t)T, (size_t)top_k, (size_t)H, (size_t)then->I, &n);
    // a cluster per token while they all run at once (T = 8, 64 experts of 4096: 6.1 us, against 7.3 for 9
    // with two tokens each), then two, which read the router's weights half as often (T = 48: 16.2)
    if (T <= 8) return dt == 0 ? run_route<0, 1>(p, s) : run_route<1, 1>(p, s);
    return dt == 0 ? run_route<0, kRouteTokens>(p, s) : run_route<1, kRouteTokens>(p, s);
}

cudaError_t launch_moe_experts(const MoeExpertsArgs& a, bool routed, cudaStream_t s)
{
    using namespace moe;
    size_t n;
    const Experts p{a.x, a.ldx, a.ids, a.weights, a.gq, a.gs, a.uq, a.us, a.dq, a.ds, a.g2, a.u2, a.d2,
                    work_of(a.work, (size_t)a.T, (size_t)a.k, (size_t)a.H, (size_t)a.I, &n), a.out, a.ldd,
                    (uint32_t)a.T, (uint32_t)a.k, (uint32_t)a.E, (uint32_t)a.H, (uint32_t)a.I, a.d_flags};
    if (!routed) {
        if (a.dt == 0) moe_rows_kernel<0><<<(unsigned)a.T, 512, 0, s>>>(a.x, a.ldx, p.H, p.work);
        else moe_rows_kernel<1><<<(unsigned)a.T, 512, 0, s>>>(a.x, a.ldx, p.H, p.work);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const bool vu = a.H % 64 == 0, vd = a.I % 64 == 0;             // (the scales are 16-byte aligned)
    cudaError_t e = vu ? run_up<true>(p, s) : run_up<false>(p, s);  // behind the router or moe_rows_kernel
    if (e != cudaSuccess) return e;
    e = launch(moe_hidden_kernel, p, p.T * p.k, 256u, 0, 1u, true, s);
    if (e != cudaSuccess) return e;
    if (a.out_dt == 0) return vd ? run_down<0, true>(p, s) : run_down<0, false>(p, s);
    if (a.out_dt == 1) return vd ? run_down<1, true>(p, s) : run_down<1, false>(p, s);
    return vd ? run_down<2, true>(p, s) : run_down<2, false>(p, s);
}

}  // namespace nv4
