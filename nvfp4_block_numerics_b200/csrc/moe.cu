// moe.cu -- a mixture-of-experts layer for a few tokens on NVFP4 expert weights (sm_100a).
//
// [DSPARK], [CAST] section 3 (routed experts w1 / w3 / w2 stored in NVFP4, w1 and w3 with a
// common scale_2); [CAL] layer table (expert layers W4A16).
//
//   route    logits[t, e] = sum_h x[t, h] wr[e, h]; p = softmax(logits); the k largest logits
//            (ties: the lower index); weight = p, or p / sum of the chosen p
//   experts  h = silu(gate_e x) * (up_e x);  y[t] = sum_j weight[t, j] * down_e h
//
// Three launches.  moe_route_kernel: one 8-CTA cluster per few tokens.  The products of 16-bit
// values are exact in FP32 and are summed in FP64, so that the choice of experts is that of the
// exact logits whatever the summation order.  moe_up_kernel and moe_down_kernel: one CTA per SM,
// the product of nv4_w4.cuh on the experts that some token chose.  The bound is reading those
// experts' weights once from HBM, so both kernels split the rows of all chosen experts evenly
// over the SMs, to one row.
//   * up: the flat list (expert, i) of gate / up row pairs is cut into one contiguous range per
//     CTA, walked in tiles of 8 pairs: MMA rows 0-7 are gate rows, 8-15 the same up rows, so
//     both halves of an h meet in one thread.  h goes to the workspace in FP32.
//   * down: a CTA owns a range of output rows for all tokens and all chosen experts, so the sum
//     over a token's experts needs no other CTA and is in a fixed order.  h is scaled per
//     (token, expert) by a power of two and rounded to FP16 (11 bits: a relative error of 2^-11,
//     an eighth of the BF16 output's own rounding); its scale, the expert's scale_2 and the
//     routing weight are applied in FP32 to the accumulated product.
#include <cfloat>
#include <type_traits>

#include "nv4_async.cuh"
#include "nv4_internal.h"
#include "nv4_w4.cuh"

namespace nv4 {

namespace moe {

using w4::Frag;
using w4::kChunk;
using w4::kThreads;
using w4::kWarps;

constexpr uint32_t kPass = 24;                    // tokens of one expert multiplied at once

// ---------------------------------------------------------------- router
constexpr int kRouteThreads = 256;
constexpr uint32_t kRouteCtas = 8;                // one cluster
constexpr uint32_t kRouteTokens = 4;              // tokens per cluster

struct RouteParams {
    const void* x;
    int64_t ldx;
    const void* wr;                               // [E, H]
    int32_t* ids;
    float* weights;
    uint32_t T, H, E, k, renorm;
    uint32_t* d_flags;
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

template <int kDt>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(kRouteThreads)
moe_route_kernel(const __grid_constant__ RouteParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    double* logits = reinterpret_cast<double*>(smem);              // [kRouteTokens][E], in the cluster's rank 0
    const uint32_t rank = cluster_ctarank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    constexpr uint32_t kRW = kRouteThreads / 32;
    const uint32_t t0 = (blockIdx.x / kRouteCtas) * kRouteTokens, nt = min(kRouteTokens, p.T - t0);
    const uint16_t* x = static_cast<const uint16_t*>(p.x);
    const uint16_t* wr = static_cast<const uint16_t*>(p.wr);
    uint32_t flags = 0u;
    cluster_sync();                                                // rank 0 runs: its shared memory can be written

    for (uint32_t e = rank * kRW + warp; e < p.E; e += kRouteCtas * kRW) {
        double s[kRouteTokens];
#pragma unroll
        for (uint32_t i = 0; i < kRouteTokens; ++i) s[i] = 0.0;
        for (uint32_t h = 8u * lane; h < p.H; h += 256u) {
            float w[8];
            unpack8<kDt>(__ldg(reinterpret_cast<const uint4*>(wr + (size_t)e * p.H + h)), w);
#pragma unroll
            for (uint32_t i = 0; i < kRouteTokens; ++i) {
                if (i >= nt) break;
                float v[8];
                unpack8<kDt>(__ldg(reinterpret_cast<const uint4*>(x + (int64_t)(t0 + i) * p.ldx + h)), v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i] = fma((double)v[j], (double)w[j], s[i]);
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < kRouteTokens; ++i) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], d);
            if (lane == 0 && i < nt) {
                uint32_t remote;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(logits + i * p.E + e)), "r"(0u));
                asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(s[i]) : "memory");
            }
        }
    }
    cluster_sync();
    if (rank != 0u) return;
    // one warp per token: lane l holds experts l, l + 32, ...; k rounds of a warp argmax
    for (uint32_t i = warp; i < nt; i += kRW) {
        const double* lg = logits + i * p.E;
        double top = -DBL_MAX, sum = 0.0;
        bool bad = false;
        for (uint32_t e = lane; e < p.E; e += 32u) {
            bad |= !(fabs(lg[e]) <= DBL_MAX);
            top = fmax(top, lg[e]);                                // a NaN is passed over
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        if (bad) flags |= kFlagNonFinite;
        if (p.renorm == 0u) {
            for (uint32_t e = lane; e < p.E; e += 32u) sum += exp(lg[e] - top);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        }
        uint64_t taken = 0ull;                                     // this lane's experts, one bit each (E <= 512)
        int32_t my_id = 0;
        double my_p = 0.0;
        for (uint32_t j = 0; j < p.k; ++j) {
            double v = -DBL_MAX;
            uint32_t id = 0xFFFFFFFFu;
            for (uint32_t e = lane, b = 0; e < p.E; e += 32u, ++b) {
                if ((taken >> b) & 1ull) continue;
                const double c = lg[e] >= -DBL_MAX ? lg[e] : -DBL_MAX;     // NaN and -inf rank last
                if (id == 0xFFFFFFFFu || c > v) {
                    v = c;
                    id = e;
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const double ov = __shfl_xor_sync(0xFFFFFFFFu, v, d);
                const uint32_t oi = __shfl_xor_sync(0xFFFFFFFFu, id, d);
                if (oi != 0xFFFFFFFFu && (id == 0xFFFFFFFFu || ov > v || (ov == v && oi < id))) {
                    v = ov;
                    id = oi;
                }
            }
            if ((id & 31u) == lane) taken |= 1ull << (id >> 5);
            const double pj = exp(lg[id] - top);
            if (p.renorm != 0u) sum += pj;
            if (lane == j) {                                       // k <= 32
                my_id = (int32_t)id;
                my_p = pj;
            }
        }
        if (lane < p.k) {
            p.ids[(size_t)(t0 + i) * p.k + lane] = my_id;
            p.weights[(size_t)(t0 + i) * p.k + lane] = (float)(my_p / sum);
        }
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
    float* h;                                     // workspace [T * k, I]
    void* out;
    int64_t ldd;
    uint32_t T, k, E, H, I;
    uint32_t smem_rows;                           // bytes of shared memory for token rows
};

// Which tokens chose which expert, built by every CTA for itself.  A pair is t * k + j; a token
// that names an expert twice has it once, with both weights.
struct Lists {
    int32_t id[kMaxMoePairs];                     // the pair's expert, -1: none or named before
    uint16_t pair[kMaxMoePairs];                  // pairs by expert, in token order
    uint16_t expert[kMaxMoeExperts];              // chosen experts in ascending order
    uint16_t first[kMaxMoeExperts + 1];           // their first entry in pair[]
    uint32_t scan[2][kWarps];
    uint32_t n;                                   // chosen experts
};

__device__ __forceinline__ void build_lists(Lists& L, const Experts& p)
{
    const uint32_t P = p.T * p.k, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    for (uint32_t i = tid; i < P; i += kThreads) {
        const int32_t e = __ldg(p.ids + i);
        bool ok = e >= 0 && e < (int32_t)p.E;
        for (uint32_t j = i - i % p.k; j < i; ++j) ok = ok && __ldg(p.ids + j) != e;
        L.id[i] = ok ? e : -1;
    }
    __syncthreads();
    uint32_t cnt = 0u;
    if (tid < p.E)
        for (uint32_t i = 0; i < P; ++i) cnt += L.id[i] == (int32_t)tid ? 1u : 0u;
    // exclusive scans over the experts: chosen ones and their pairs
    uint32_t a = cnt != 0u ? 1u : 0u, b = cnt;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint32_t oa = __shfl_up_sync(0xFFFFFFFFu, a, d), ob = __shfl_up_sync(0xFFFFFFFFu, b, d);
        if (lane >= d) {
            a += oa;
            b += ob;
        }
    }
    if (lane == 31u) {
        L.scan[0][warp] = a;
        L.scan[1][warp] = b;
    }
    __syncthreads();
    uint32_t ba = 0u, bb = 0u, n = 0u, np = 0u;
    for (uint32_t w = 0; w < (uint32_t)kWarps; ++w) {
        if (w < warp) {
            ba += L.scan[0][w];
            bb += L.scan[1][w];
        }
        n += L.scan[0][w];
        np += L.scan[1][w];
    }
    if (cnt != 0u) {
        const uint32_t slot = ba + a - 1u;
        uint32_t at = bb + b - cnt;
        L.expert[slot] = (uint16_t)tid;
        L.first[slot] = (uint16_t)at;
        for (uint32_t i = 0; i < P; ++i)
            if (L.id[i] == (int32_t)tid) L.pair[at++] = (uint16_t)i;
    }
    if (tid == 0u) {
        L.n = n;
        L.first[n] = (uint16_t)np;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- gate, up, SwiGLU
// kNT: 8-token tiles of a pass (1 or 3).
template <int kDt, bool kVec, int NT>
__device__ __forceinline__ void up_pass(const Experts& p, const Lists& L, w4::Rows& rows, uint4* xs, float* red,
                                        uint32_t e, uint32_t f0, uint32_t m, uint32_t i0, uint32_t i1)
{
    constexpr uint32_t kTile = 16u * 8u * NT;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
    const uint32_t nch = (p.H + kChunk - 1u) / kChunk, R = i1 - i0, ntile = (R + 7u) / 8u;
    const uint32_t wk = w4::split_of(ntile, nch), groups = kWarps / wk, grp = warp / wk, wig = warp - grp * wk;
    const size_t mat = (size_t)e * p.I;
    auto load = [&](Frag& f, uint32_t tile, uint32_t c) {
        const uint32_t a = i0 + tile * R / ntile, b = i0 + (tile + 1u) * R / ntile, i = a + g;
        const uint32_t k0 = c * kChunk + 64u * t;
        const size_t q = (mat + i) * (p.H / 2u), s = (mat + i) * (p.H / 16u);
        w4::load_row<kVec>(f.q0, f.s0, p.gq + q, p.gs + s, k0, p.H, i < b);
        w4::load_row<kVec>(f.q1, f.s1, p.uq + q, p.us + s, k0, p.H, i < b);
    };
    Frag cur;
    if (grp < ntile) load(cur, grp, wig);
    __syncthreads();                                               // the previous pass has read its tokens
    const bool wide = w4::stage_tokens<kDt>(xs, rows, m, p.H, [&](uint32_t i) {
        return static_cast<const void*>(static_cast<const uint16_t*>(p.x) + (int64_t)(L.pair[f0 + i] / p.k) * p.ldx);
    });
    const float sg = p.g2[e], su = p.u2[e];
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
                w4::mma_chunk<true, NT>(acc, cur, xc, m, g, t);
            else
                w4::mma_chunk<false, NT>(acc, cur, xc, m, g, t);
            cur = next;
        }
        float* part = red + (size_t)(buf * kWarps + warp) * kTile;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            *reinterpret_cast<float2*>(part + g * (8 * NT) + 8 * j + 2 * t) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2*>(part + (g + 8) * (8 * NT) + 8 * j + 2 * t) = make_float2(acc[j][2], acc[j][3]);
        }
        if (wk == 1u) __syncwarp();
        else w4::group_barrier(1u + grp, 32u * wk);
        const uint32_t a = i0 + tile * R / ntile, nr = i0 + (tile + 1u) * R / ntile - a;
        const float* first = red + (size_t)(buf * kWarps + grp * wk) * kTile;
        for (uint32_t i = wig * 32u + lane; i < 8u * m; i += 32u * wk) {
            const uint32_t r = i & 7u, tok = i >> 3;
            if (r >= nr) continue;
            float sa = 0.0f, sb = 0.0f;
            for (uint32_t w = 0; w < wk; ++w) {
                sa += first[(size_t)w * kTile + r * (8 * NT) + tok];
                sb += first[(size_t)w * kTile + (r + 8u) * (8 * NT) + tok];
            }
            const float gv = sa * sg * rows.descale[tok], uv = sb * su * rows.descale[tok];
            p.h[(size_t)L.pair[f0 + tok] * p.I + a + r] = gv / (1.0f + expf(-gv)) * uv;
        }
    }
}

template <int kDt, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) moe_up_kernel(const __grid_constant__ Experts p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Lists L;
    __shared__ w4::Rows rows;
    uint4* xs = reinterpret_cast<uint4*>(smem);
    float* red = reinterpret_cast<float*>(smem + p.smem_rows);
    build_lists(L, p);
    const uint64_t total = (uint64_t)L.n * p.I;
    const uint64_t end = (blockIdx.x + 1u) * total / gridDim.x;
    const uint32_t cap = min(kPass, p.smem_rows / ((p.H + kChunk - 1u) / kChunk * 512u));
    for (uint64_t at = blockIdx.x * total / gridDim.x; at < end;) {
        const uint32_t a = (uint32_t)(at / p.I), i0 = (uint32_t)(at - (uint64_t)a * p.I);
        const uint32_t i1 = (uint32_t)min((uint64_t)p.I, end - (uint64_t)a * p.I);
        const uint32_t f0 = L.first[a], m_e = L.first[a + 1u] - f0;
        for (uint32_t q = 0; q < m_e; q += cap) {
            const uint32_t m = min(cap, m_e - q);
            if (m <= 8u) up_pass<kDt, kVec, 1>(p, L, rows, xs, red, L.expert[a], f0 + q, m, i0, i1);
            else up_pass<kDt, kVec, 3>(p, L, rows, xs, red, L.expert[a], f0 + q, m, i0, i1);
        }
        at = (uint64_t)a * p.I + i1;
    }
}

// ---------------------------------------------------------------- down, weighted sum
constexpr uint32_t kMaxSubs = 32;                 // (expert, up to kPass of its tokens) staged at once

struct Batch {
    uint16_t expert[kMaxSubs], first[kMaxSubs], m[kMaxSubs], row0[kMaxSubs];
    uint32_t n, rows, next_a, next_q;
};

// One sub-list's product: acc over chunks [c0, c1) of a 16-row tile, added into this warp's
// sums Y[token][16], each token's column times its coefficient.
template <bool kVec, int NT>
__device__ __forceinline__ void down_run(const Experts& p, const Lists& L, const float* coef, float* Y,
                                         const uint4* xs, uint32_t m, uint32_t f0, const uint8_t* q, const uint8_t* s,
                                         bool la, bool lb, uint32_t c0, uint32_t c1)
{
    const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    Frag cur, next;
    const size_t q8 = (size_t)8u * (p.I / 2u), s8 = (size_t)8u * (p.I / 16u);
    auto load = [&](Frag& f, uint32_t c) {
        const uint32_t k0 = c * kChunk + 64u * t;
        w4::load_row<kVec>(f.q0, f.s0, q, s, k0, p.I, la);
        w4::load_row<kVec>(f.q1, f.s1, q + q8, s + s8, k0, p.I, lb);
    };
    load(cur, c0);
    for (uint32_t c = c0; c < c1; ++c) {
        if (c + 1u < c1) load(next, c + 1u);
        w4::mma_chunk<false, NT>(acc, cur, xs + (size_t)c * 32u * m, m, g, t);
        cur = next;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
            const uint32_t col = 8u * j + 2u * t + i;
            if (col < m) {
                float* y = Y + (size_t)(L.pair[f0 + col] / p.k) * 16u;
                y[g] += acc[j][i] * coef[col];
                y[g + 8] += acc[j][2 + i] * coef[col];
            }
        }
    __syncwarp();
}

template <int kOut, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) moe_down_kernel(const __grid_constant__ Experts p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Lists L;
    __shared__ Batch B;
    __shared__ float coef[kMaxSubs * kPass];
    uint4* xs = reinterpret_cast<uint4*>(smem);
    float* Yall = reinterpret_cast<float*>(smem + p.smem_rows);    // [16 warps][T][16]
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2;
    build_lists(L, p);
    const uint32_t r0 = (uint32_t)((uint64_t)blockIdx.x * p.H / gridDim.x);
    const uint32_t R = (uint32_t)((uint64_t)(blockIdx.x + 1u) * p.H / gridDim.x) - r0;
    const uint32_t ntile = (R + 15u) / 16u;                        // at most 16: H <= 256 x CTAs
    const uint32_t wpt = kWarps / ntile, tile = warp % ntile, widx = warp / ntile;
    const bool works = widx < wpt;
    const uint32_t ta = r0 + tile * R / ntile, tb = r0 + (tile + 1u) * R / ntile;
    float* Y = Yall + (size_t)warp * p.T * 16u;
    for (uint32_t i = lane; i < p.T * 16u; i += 32u) Y[i] = 0.0f;
    const uint32_t nch = (p.I + kChunk - 1u) / kChunk, row_vecs = nch * 32u;
    const uint32_t cap_rows = min(kMaxSubs * kPass, p.smem_rows / (row_vecs * 16u)), cap = min(kPass, cap_rows);
    if (tid == 0u) B.next_a = B.next_q = 0u;

    for (;;) {
        __syncthreads();                                           // the previous batch has been used
        if (tid == 0u) {                                           // the next batch: whole sub-lists while they fit
            uint32_t n = 0u, rows = 0u, a = B.next_a, q = B.next_q;
            while (a < L.n && n < kMaxSubs) {
                const uint32_t m = min(cap, (uint32_t)L.first[a + 1u] - L.first[a] - q);
                if (rows + m > cap_rows) break;
                B.expert[n] = L.expert[a];
                B.first[n] = (uint16_t)(L.first[a] + q);
                B.m[n] = (uint16_t)m;
                B.row0[n] = (uint16_t)rows;
                rows += m;
                ++n;
                q += m;
                if (q == (uint32_t)L.first[a + 1u] - L.first[a]) {
                    ++a;
                    q = 0u;
                }
            }
            B.n = n;
            B.rows = rows;
            B.next_a = a;
            B.next_q = q;
        }
        __syncthreads();
        const uint32_t n = B.n;
        if (n == 0u) break;
        // ---- h rows: one warp per row; scaled by a power of two to FP16
        for (uint32_t r = warp; r < B.rows; r += kWarps) {
            uint32_t s = 0u;
            while (s + 1u < n && r >= B.row0[s + 1u]) ++s;
            const uint32_t i = r - B.row0[s], m = B.m[s], pr = L.pair[B.first[s] + i];
            const float4* src = reinterpret_cast<const float4*>(p.h + (size_t)pr * p.I);
            uint32_t top = 0u;
            for (uint32_t k = 4u * lane; k < p.I; k += 128u) {
                const float4 v = src[k >> 2];
                const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
                    if (b < 0x7F800000u) top = max(top, b);        // the largest finite one
                }
            }
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            const int e1 = (int)(top >> 23);
            const int fe = top == 0u ? 127 : min(268 - e1, 254);   // factor 2^(fe - 127)
            const float f = w4::exp_field(fe);
            uint4* dst = xs + (size_t)B.row0[s] * row_vecs;
            for (uint32_t v8 = lane; v8 < row_vecs; v8 += 32u) {
                const uint32_t c = v8 >> 5, l = v8 & 31u, k = c * kChunk + 8u * l;
                uint4 o = make_uint4(0u, 0u, 0u, 0u);
                if (k < p.I) {
                    const float4 u = src[k >> 2], v = src[(k >> 2) + 1u];
                    const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
                    uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                            : "=r"(ow[j])
                            : "f"(__fmul_rn(w[2 * j + 1], f)), "f"(__fmul_rn(w[2 * j], f)));
                }
                dst[((c * 8u + (l & 7u)) * m + i) * 4u + (l >> 3)] = o;
            }
            if (lane == 0u) {
                const uint32_t tok = pr / p.k;
                const int32_t e = L.id[pr];
                float w = 0.0f;                                    // a token's weights of this expert
                for (uint32_t j = 0; j < p.k; ++j)
                    if (__ldg(p.ids + tok * p.k + j) == e) w += __ldg(p.weights + tok * p.k + j);
                coef[r] = w * p.d2[e] * w4::exp_field(254 - fe);
            }
        }
        __syncthreads();
        // ---- products: (sub-list, chunk) steps in a contiguous run per warp
        if (works) {
            const uint32_t steps = n * nch, b = (widx + 1u) * steps / wpt;
            for (uint32_t at = widx * steps / wpt; at < b;) {
                const uint32_t s = at / nch, c0 = at - s * nch, c1 = min(nch, b - s * nch), m = B.m[s];
                const size_t row = (size_t)B.expert[s] * p.H + ta + g;
                const uint8_t* q = p.dq + row * (p.I / 2u);
                const uint8_t* sc = p.ds + row * (p.I / 16u);
                const uint4* xb = xs + (size_t)B.row0[s] * row_vecs;
                const bool la = ta + g < tb, lb = ta + g + 8u < tb;
                if (m <= 8u) down_run<kVec, 1>(p, L, coef + B.row0[s], Y, xb, m, B.first[s], q, sc, la, lb, c0, c1);
                else down_run<kVec, 3>(p, L, coef + B.row0[s], Y, xb, m, B.first[s], q, sc, la, lb, c0, c1);
                at = s * nch + c1;
            }
        }
    }
    // ---- the warps' sums of a tile, in warp order (the loop ended behind a CTA barrier)
    for (uint32_t i = tid; i < p.T * R; i += kThreads) {
        const uint32_t tok = i / R, r = i - tok * R;
        uint32_t tl = r * ntile / R;                               // the tile that holds row r
        while (r < tl * R / ntile) --tl;
        while (r >= (tl + 1u) * R / ntile) ++tl;
        const uint32_t in = r - tl * R / ntile;
        float v = 0.0f;
        for (uint32_t w = 0; w < wpt; ++w) v += Yall[((size_t)(w * ntile + tl) * p.T + tok) * 16u + in];
        w4::store_out<kOut>(p.out, (int64_t)tok * p.ldd + r0 + r, v);
    }
}

}  // namespace moe

cudaError_t launch_moe_route(const void* x, int dt, int64_t T, int64_t H, int64_t ldx, const void* wr, int64_t E,
                             int top_k, int renorm, int32_t* ids, float* weights, uint32_t* d_flags, cudaStream_t s)
{
    using namespace moe;
    RouteParams p{x, ldx, wr, ids, weights, (uint32_t)T, (uint32_t)H, (uint32_t)E, (uint32_t)top_k, (uint32_t)renorm, d_flags};
    const unsigned grid = (unsigned)((T + kRouteTokens - 1) / kRouteTokens) * kRouteCtas;
    const size_t smem = (size_t)kRouteTokens * E * sizeof(double);
    if (dt == 0) moe_route_kernel<0><<<grid, kRouteThreads, smem, s>>>(p);
    else moe_route_kernel<1><<<grid, kRouteThreads, smem, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_moe_experts(const MoeExpertsArgs& a, cudaStream_t s)
{
    using namespace moe;
    Experts p{a.x, a.ldx, a.ids, a.weights, a.gq, a.gs, a.uq, a.us, a.dq, a.ds, a.g2, a.u2, a.d2, a.h, a.out, a.ldd,
              (uint32_t)a.T, (uint32_t)a.k, (uint32_t)a.E, (uint32_t)a.H, (uint32_t)a.I, 0u};
    auto vec = [](const void* q, const void* sc) {
        return (reinterpret_cast<uintptr_t>(q) & 31u) == 0u && (reinterpret_cast<uintptr_t>(sc) & 3u) == 0u;
    };
    const uint32_t sms = (uint32_t)num_sms();
    {
        const uint32_t red = 2u * kWarps * 16u * kPass * (uint32_t)sizeof(float);
        p.smem_rows = (uint32_t)(kMaxSmemMoe - red) & ~511u;
        const bool v = a.H % 64 == 0 && vec(a.gq, a.gs) && vec(a.uq, a.us);
        auto kern = a.dt == 0 ? (v ? moe_up_kernel<0, true> : moe_up_kernel<0, false>)
                              : (v ? moe_up_kernel<1, true> : moe_up_kernel<1, false>);
        const size_t smem = (size_t)p.smem_rows + red;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        kern<<<sms, kThreads, smem, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const uint32_t grid = (uint32_t)a.H < sms ? (uint32_t)a.H : sms;
    if (((uint32_t)a.H + grid - 1u) / grid > 16u * kWarps) return cudaErrorInvalidValue;
    const uint32_t sums = kWarps * (uint32_t)a.T * 16u * (uint32_t)sizeof(float);
    p.smem_rows = (uint32_t)(kMaxSmemMoe - sums) & ~511u;
    const bool v = a.I % 64 == 0 && vec(a.dq, a.ds);
    auto kern = a.out_dt == 0 ? (v ? moe_down_kernel<0, true> : moe_down_kernel<0, false>)
                              : a.out_dt == 1 ? (v ? moe_down_kernel<1, true> : moe_down_kernel<1, false>)
                                              : (v ? moe_down_kernel<2, true> : moe_down_kernel<2, false>);
    const size_t smem = (size_t)p.smem_rows + sums;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace nv4
