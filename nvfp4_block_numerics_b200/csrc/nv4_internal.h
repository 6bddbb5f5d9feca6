// nv4_internal.h -- declarations shared by the kernel files and the C-ABI layer.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "nv4.h"

namespace nv4 {

// Division of 32-bit unsigned integers by a fixed divisor d >= 1 with one
// multiply-high, one add and one shift (T. Granlund and P. L. Montgomery,
// "Division by invariant integers using multiplication", PLDI 1994, round-up
// method): with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (mulhi(n, m) + n) >> s for every n < 2^32.
struct FastDiv {
    uint32_t d = 1, m = 1, s = 0;
    __host__ __device__ FastDiv() {}
    __host__ __device__ explicit FastDiv(uint32_t div) : d(div)
    {
        s = 0;
        while ((1ull << s) < div) ++s;
        m = (uint32_t)((((1ull << 32) * ((1ull << s) - div)) / div) + 1ull);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const
    {
        return (uint32_t)(((uint64_t)__umulhi(n, m) + n) >> s);
    }
};

int num_sms();

constexpr int kMaxHessianJobs = 128;
constexpr int kMaxSweepJobs = 192;
constexpr int kMaxCastJobs = 128;

// One tensor of a (batched) per-tensor amax, block quantization or dequantization call.
struct AmaxTask {
    const void* x;
    int64_t n;
    float* d_amax;
};
struct QuantTask {
    const void* x;
    int64_t rows, cols, ld;
    const float* d_amax;
    uint8_t* q;           // packed codes (code output) or null
    uint8_t* scales;
    void* out;            // fake quantize-dequantize output or null
    int64_t ld_out;
    float* d_s2;
};
struct DequantTask {
    const uint8_t* q;
    const uint8_t* scales;
    const float* d_s2;
    int64_t rows, cols;
    void* out;
};
constexpr int kMaxActJobs = 128;

cudaError_t launch_amax(const AmaxTask* tasks, int n, int dt, uint32_t* d_flags, cudaStream_t s);
// Second-level scales of empty tensors: d_out[i] = RN32(*d_amax[i] / divisor) for n pairs,
// NV4_FLAG_OVERFLOW where that is not finite (one small launch; nothing else is read).
cudaError_t launch_scale_only(const float* const* d_amax, float* const* d_out, int n, float divisor,
                              uint32_t* d_flags, cudaStream_t s);
cudaError_t launch_block_quant(const QuantTask* tasks, int n, int in_dt, int out_dt, uint32_t* d_flags,
                               cudaStream_t s);
cudaError_t launch_mxfp4_quant(const void* x, int in_dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* q,
                               uint8_t* e8m0, uint32_t* d_flags, cudaStream_t s);
cudaError_t launch_mxfp4_dequant(const uint8_t* q, const uint8_t* e8m0, int64_t rows, int64_t cols, int out_dt,
                                 void* out, cudaStream_t s);
cudaError_t launch_fp8_quant(const void* x, int in_dt, int64_t rows, int64_t cols, int64_t ld, const float* d_amax,
                             uint8_t* q, float* d_scale, uint32_t* d_flags, cudaStream_t s);
cudaError_t launch_fp8_dequant(const uint8_t* q, const float* d_scale, int64_t rows, int64_t cols, int out_dt,
                               void* out, cudaStream_t s);
cudaError_t launch_hadamard2(int mode, const void* w, int dt, int64_t rows, int64_t cols, int64_t ld, int n,
                             float* d_amax, uint8_t* q, uint8_t* sc, float* d_s2, float* out, uint32_t* d_flags,
                             cudaStream_t s);
cudaError_t launch_hadamard_quant(int mode, const void* x, int64_t rows, int64_t cols, int64_t ld, int n,
                                  float* d_amax, uint8_t* q, uint8_t* sc, float* d_s2, uint32_t* d_flags,
                                  cudaStream_t s);
cudaError_t launch_cluster_selftest(uint32_t bad, uint32_t* status, cudaStream_t s);
cudaError_t launch_wait_selftest(const uint32_t* flag, uint64_t limit_ns, uint32_t* status, cudaStream_t s);
size_t mma_scale_bytes(int64_t rows, int64_t kb);
cudaError_t launch_mma_scale_layout(const uint8_t* sc, int64_t rows, int64_t kb, uint8_t* out, cudaStream_t s);
cudaError_t launch_gemm_nvfp4(const uint8_t* qa, const uint8_t* sfa, const float* d_s2a, const uint8_t* qb,
                              const uint8_t* sfb, const float* d_s2b, int64_t M, int64_t N, int64_t K, int out_dt,
                              void* out, int64_t ldd, uint32_t* d_flags, cudaStream_t s);
// K of one linear_w4a16 / mixture-of-experts call at most: one token row in shared memory.
constexpr int64_t kMaxW4K = 65536;
constexpr size_t kMaxSmemW4 = 220u * 1024u;
// Rows up to which the weight-only linear layer runs on launch_linear_w4a16, above them on its _mma
// form.  16 rows on either (us): 2880 x 2880 8.8 / 9.9, 16384 x 2048 11.1 / 15.3, 8192 x 8192 23.4 /
// 27.5; a third column of 8 tokens would cost the former what the latter's 32 columns have free.
constexpr int64_t kMaxFewRows = 16;
// Whether a call runs on launch_linear_w4a16: few rows, and shared memory holds them (5 rows of 65536, 8
// of 32768; read in passes instead, each of which reads the weights again, 16 x 8192 x 65536 took 605 us,
// against 170; layers of a few hundred rows lose by it, 16 x 300 x 65536 37 us, against 48).
bool few_rows_w4a16(int64_t T, int64_t K);
cudaError_t launch_linear_w4a16(const void* x, int dt, int64_t T, int64_t K, int64_t ldx, const uint8_t* q,
                                const uint8_t* sc, const float* d_s2, int64_t N, int out_dt, void* out, int64_t ldd,
                                uint32_t* d_flags, cudaStream_t s);
cudaError_t launch_linear_w4a16_mma(const void* x, int dt, int64_t T, int64_t K, int64_t ldx, const uint8_t* q,
                                    const uint8_t* sc, const float* d_s2, int64_t N, int out_dt, void* out, int64_t ldd,
                                    uint32_t* d_flags, cudaStream_t s);
// Mixture-of-experts limits: tokens and (token, expert) pairs of a call, experts, experts per
// token, widths.
constexpr int64_t kMaxMoeTokens = 64, kMaxMoePairs = 2048, kMaxMoeExperts = 512, kMaxMoeTopK = 32;
constexpr int64_t kMaxMoeWidth = 32768;
struct MoeExpertsArgs {
    const void* x;
    int dt, out_dt;
    int64_t T, k, E, H, I, ldx, ldd;
    const int32_t* ids;
    const float* weights;
    const uint8_t *gq, *gs, *uq, *us, *dq, *ds;
    const float *g2, *u2, *d2;
    void* work;
    void* out;
    uint32_t* d_flags;
};
size_t moe_work_bytes(int64_t T, int64_t k, int64_t H, int64_t I);
cudaError_t launch_moe_route(const void* x, int dt, int64_t T, int64_t H, int64_t ldx, const void* wr, int64_t E,
                             int top_k, int renorm, int32_t* ids, float* weights, const MoeExpertsArgs* then,
                             uint32_t* d_flags, cudaStream_t s);
// routed: the call in front on the stream is launch_moe_route with these arguments as `then`.
cudaError_t launch_moe_experts(const MoeExpertsArgs& a, bool routed, cudaStream_t s);
cudaError_t launch_mxfp4_quant_mma(const void* x, int in_dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* q,
                                   uint8_t* sf, uint32_t* d_flags, cudaStream_t s);
// dependent: the call in front on the stream is launch_mxfp4_quant_mma, which wrote qa and sfa.
cudaError_t launch_gemm_mxfp4(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb, int64_t M,
                              int64_t N, int64_t K, int out_dt, void* out, int64_t ldd, bool dependent,
                              uint32_t* d_flags, cudaStream_t s);
cudaError_t launch_gemm_mxfp4_small(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb, int64_t M,
                                    int64_t N, int64_t K, int out_dt, void* out, int64_t ldd, bool dependent,
                                    uint32_t* d_flags, cudaStream_t s);
// Rows of A up to which launch_gemm_mxfp4 runs on launch_gemm_mxfp4_small (and above them while its
// 128 x 128 tiles fit the SMs at once), else on the CTA-pair kernel.  Either, in us: 128 x 2880 x 2880
// 8.5 / 15.7, 128 x 16384 x 2048 10.2 / 11.6, 128 x 8192 x 8192 14.9 / 25.9, 256 x 2048 x 16384 14.6 /
// 45, 1024 x 2048 x 2048 10.0 / 11.4; with more tiles than SMs 64 x 32768 x 4096 22.2 / 26.2, 64 x 65536
// x 4096 47.4 / 46.8, 128 x 65536 x 4096 55.0 / 48.2, 128 x 151936 x 1024 68 / 37.
constexpr int64_t kMaxSmallRows = 64;
// The linear layer for up to kMaxFusedRows rows: quantization and product in one kernel.  On the
// device it is level with two (16 x 16384 x 2048 9.3 us, 16 x 2880 x 2880 7.0); a call costs one launch
// less (1 x 2880 x 2880: 12.5 us a call, 17.5 with two).  Every tile quantizes the rows again, so past
// kMaxFusedWeights weights two kernels are faster, if there is a workspace for them (16 rows, fused / the
// product alone, to which the quantizer adds 3 us: 20000 x 512 8.5 / 7.3, 32768 x 1024 11.1 / 9.3, 8192 x
// 8192 15.5 / 11.0, 32768 x 4096 29.5 / 19.0, 65536 x 4096 64 / 41).
constexpr int64_t kMaxFusedWeights = (int64_t)1 << 25;
constexpr int64_t kMaxFusedRows = 16;
cudaError_t launch_linear_mxfp4_small(const void* x, int in_dt, int64_t M, int64_t K, int64_t ldx, const uint8_t* qw,
                                      const uint8_t* sfw, int64_t N, int out_dt, void* out, int64_t ldd, uint32_t* d_flags,
                                      cudaStream_t s);
cudaError_t launch_dequant(const DequantTask* tasks, int n, int out_dt, cudaStream_t s);
cudaError_t launch_hessian(const nv4_hessian_job* jobs, int n, uint32_t* d_flags, cudaStream_t s, int* bad_job);
cudaError_t launch_sweep(const nv4_sweep_job* jobs, int n, int dt, uint32_t* d_flags, cudaStream_t s);
cudaError_t launch_cast(const nv4_cast_job* jobs, int n, unsigned long long* d_counts, uint32_t* d_flags,
                        cudaStream_t s);
cudaError_t launch_selftest(uint32_t* d_out, cudaStream_t s);
cudaError_t launch_fma_probe(int packed, uint32_t blocks, uint32_t iters, float* sink, cudaStream_t s);

}  // namespace nv4
