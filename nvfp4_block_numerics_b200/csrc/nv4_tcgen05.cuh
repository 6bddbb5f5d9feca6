// nv4_tcgen05.cuh -- tensor-memory, descriptor and commit helpers of the tcgen05 kernels (sm_100a).
#pragma once

#include "nv4_async.cuh"

namespace nv4 {
namespace tc {

// A kernel whose CTAs hold tensor memory while they wait for the other CTAs of their cluster asks
// for more shared memory than half of an SM's 228 KB (less 1 KB per CTA): no two such CTAs, of one
// kernel or of two on different streams, then share an SM.  If they did, two clusters could each
// hold the tensor memory that a CTA of the other one waits to allocate.
constexpr size_t kSmemOfOnePerSm = (228u * 1024u) / 2u - 1024u;

// ---------------------------------------------------------------- PTX helpers
// As mbar_wait (false when the phase did not complete within kWaitLimitNs), with a time for which
// the hardware may suspend the thread.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity)
{
    const uint32_t addr = smem_u32(bar);
    auto tried = [&]() {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(addr), "r"(parity), "r"(20000u)
                     : "memory");
        return ok != 0u;
    };
    if (tried()) return true;
    const uint64_t t0 = global_ns();
    while (!tried())
        if (global_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

// Every lane of a warp waits; whether all of them saw the phase.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity)
{
    return __all_sync(0xFFFFFFFFu, wait_bar(bar, parity)) != 0;
}

// Every lane of a warp waits for n barriers (bar[i], parity[i]); all are tried at once before any is
// waited for: a try takes some 130 clocks to answer.
template <int kN>
__device__ __forceinline__ bool wait_bars_warp(uint64_t* const (&bar)[kN], const uint32_t (&parity)[kN], uint32_t n)
{
    bool seen[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) seen[i] = (uint32_t)i >= n || mbar_try_wait(bar[i], parity[i]);
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (!seen[i]) ok = ok && wait_bar(bar[i], parity[i]);
    return __all_sync(0xFFFFFFFFu, ok) != 0;
}

// One lane of the warp.  The issuing warps walk their stages with all lanes and issue under this:
// addresses and descriptors are then the same for the whole warp, as the instructions want them.
// (With the loop itself under a lane test the four MMAs and two commits of a stage took 550 clocks
// to issue, whatever their size.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0u;
}

// Shared-memory matrix descriptor (Blackwell format): start address, leading and
// stride byte offsets in 16-byte units, descriptor version 1 (bits 46-47) and the
// layout/swizzle mode in bits 61-63 (0 none, 2 = 128-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lbo & 0x3FFFu) << 16) |
           ((uint64_t)(sbo & 0x3FFFu) << 32) | (1ull << 46) | ((uint64_t)layout << 61);
}

__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// MXFP4 scale atoms a0 and a0 + 1 (128 K-elements each) of a row tile that has kt of them; past an
// odd end the last one again (the codes are zeros there).
__device__ __forceinline__ void load_atoms(uint8_t* dst, const uint8_t* atoms, uint32_t a0, uint32_t kt, uint64_t* bar)
{
    const uint8_t* src = atoms + (size_t)a0 * 512u;
    if (a0 + 1u < kt) {
        bulk_load(dst, src, 1024u, bar);
    } else {
        bulk_load(dst, src, 512u, bar);
        bulk_load(dst + 512u, src, 512u, bar);
    }
}

__device__ __forceinline__ void tmem_alloc(uint32_t* dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Writes n consecutive 32-bit tensor-memory columns of this warp's 32 lanes (one register
// per column and lane); the caller waits with tmem_st_wait before handing them on.
template <int n>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[n]);

template <>
__device__ __forceinline__ void tmem_st<8>(uint32_t taddr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                   "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
                   "r"(v[15])
                 : "memory");
}

template <>
__device__ __forceinline__ void tmem_st<32>(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                   "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
                   "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
                   "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]),
                   "r"(v[31])
                 : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One K = 64 step of the block-scaled FP4 MMA; the scale columns at sfa and sfb.  Pair: the
// 2-SM form.  kMx: E8M0 scales of 32 elements (two of a word's four bytes, chosen by the
// instruction descriptor), else E4M3 scales of 16 elements (all four).
template <bool kPair, bool kMx>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
#define NV4_MMA_FP4(form)                                                                              \
    asm volatile("{\n\t.reg .pred p;\n\t"                                                              \
                 "setp.ne.b32 p, %4, 0;\n\t"                                                           \
                 "tcgen05.mma." form " [%0], %1, %2, %3, [%5], [%6], p;\n\t"                           \
                 "}"                                                                                   \
                 ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) \
                 : "memory")
    if constexpr (kPair && kMx) NV4_MMA_FP4("cta_group::2.kind::mxf4.block_scale.block32");
    else if constexpr (kPair) NV4_MMA_FP4("cta_group::2.kind::mxf4nvf4.block_scale.block16");
    else if constexpr (kMx) NV4_MMA_FP4("cta_group::1.kind::mxf4.block_scale.block32");
    else NV4_MMA_FP4("cta_group::1.kind::mxf4nvf4.block_scale.block16");
#undef NV4_MMA_FP4
}

// Arrives on mbar once every tcgen05 operation issued so far by this thread completes.
__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// The sum, in rank order, of four floats at p (16-byte aligned) over the z CTAs of a cluster; z is at
// most 8.  Four at a time: read one by one, the sums of a 128 x 128 tile shared by two CTAs cost 32
// round trips (384 x 2048 x 2048: 13.6 us, against 9.3).
__device__ __forceinline__ float4 cluster_sum4(const float* p, uint32_t z)
{
    float4 v[8];
#pragma unroll
    for (uint32_t k = 0; k < 8u; ++k) {
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k < z) {
            uint32_t remote;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(k));
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[k].x), "=f"(v[k].y), "=f"(v[k].z), "=f"(v[k].w)
                         : "r"(remote)
                         : "memory");
        }
    }
    float4 s = v[0];
#pragma unroll
    for (uint32_t k = 1; k < 8u; ++k) {
        s.x += v[k].x;
        s.y += v[k].y;
        s.z += v[k].z;
        s.w += v[k].w;
    }
    return s;
}

// 32 consecutive FP32 accumulator columns of this warp's 32 lanes (one row per thread).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float v[32])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                   "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
                   "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
                   "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 columns, likewise.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Arrives on the barrier at bar's offset in both CTAs of the pair once every tcgen05
// operation issued so far by this thread completes.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3u)
                 : "memory");
}

}  // namespace tc
}  // namespace nv4
