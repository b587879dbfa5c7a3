// Internal declarations of the decoder-block operators (norm, linear, gated linear unit): the
// argument blocks of their kernels and the arithmetic that every engine's epilogue shares.
#pragma once

#include <atomic>

#include <cuda_fp8.h>

#include "gdn_internal.cuh"

namespace gdn {

// Activations.  `PRECISE` (fp32 outputs) takes the full-accuracy exponential and division; otherwise the
// result is rounded to bf16 (relative step 2^-8) and the fast ones (relative error below 2^-20 for the
// arguments where the result is not itself lost in that rounding) are enough.
template <bool PRECISE>
__device__ __forceinline__ float logistic(float z)
{
    if (PRECISE) return 1.f / (1.f + expf(-z));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-z)));
    return r;
}
constexpr float kGeluA = 1.5957691216057308f;            // 2 sqrt(2 / pi): 0.5 (1 + tanh u) = logistic(2 u)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

// The normal distribution function Phi(z) = erfc(-z / sqrt 2) / 2.  Not PRECISE: the Chebyshev fit of erfc in
// Press et al., Numerical Recipes, section 6.2 ("erfcc": fractional error below 1.2e-7 everywhere, so that the small
// tail keeps its digits), one division and one exponential without a branch; erff takes both of its branches in
// almost every warp.
template <bool PRECISE>
__device__ __forceinline__ float normal_cdf(float z)
{
    if (PRECISE) return 0.5f * erfcf(z * -0.70710678118654752f);
    const float x = fabsf(z) * 0.70710678118654752f;
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.5f, x, 1.f)));
    float p = 0.17087277f;
    p = fmaf(p, t, -0.82215223f);
    p = fmaf(p, t, 1.48851587f);
    p = fmaf(p, t, -1.13520398f);
    p = fmaf(p, t, 0.27886807f);
    p = fmaf(p, t, -0.18628806f);
    p = fmaf(p, t, 0.09678418f);
    p = fmaf(p, t, 0.37409196f);
    p = fmaf(p, t, 1.00002368f);
    p = fmaf(p, t, -1.26551223f);
    const float half = 0.5f * t * __expf(fmaf(-x, x, p));  // erfc(x) / 2
    return z < 0.f ? half : 1.f - half;
}

template <bool PRECISE, int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if (ACT == GDN_ACT_SILU) return z * logistic<PRECISE>(z);
    if (ACT == GDN_ACT_GELU) return z * normal_cdf<PRECISE>(z);
    if (ACT == GDN_ACT_GELU_TANH) return z * logistic<PRECISE>(z * (kGeluA + kGeluB * z * z));
    if (ACT == GDN_ACT_RELU) return z < 0.f ? 0.f : z;  // (keeps a NaN)
    if (ACT == GDN_ACT_SIGMOID) return logistic<PRECISE>(z);
    return z;
}
// value and derivative
template <bool PRECISE, int ACT>
__device__ __forceinline__ void act_both(float z, float &v, float &d)
{
    if (ACT == GDN_ACT_SILU) {
        const float p = logistic<PRECISE>(z);
        v = z * p;
        d = p * (1.f + z * (1.f - p));
    } else if (ACT == GDN_ACT_GELU) {
        const float c = normal_cdf<PRECISE>(z);
        const float e = PRECISE ? expf(-0.5f * z * z) : __expf(-0.5f * z * z);
        v = z * c;
        d = c + z * e * 0.3989422804014327f;  // 1 / sqrt(2 pi)
    } else if (ACT == GDN_ACT_GELU_TANH) {
        const float z2 = z * z, p = logistic<PRECISE>(z * (kGeluA + kGeluB * z2));
        v = z * p;
        d = p + v * (1.f - p) * (kGeluA + 3.f * kGeluB * z2);
    } else if (ACT == GDN_ACT_RELU) {
        v = z < 0.f ? 0.f : z;
        d = z > 0.f ? 1.f : 0.f;
    } else if (ACT == GDN_ACT_SIGMOID) {
        const float p = logistic<PRECISE>(z);
        v = p;
        d = p * (1.f - p);
    } else {
        v = z;
        d = 1.f;
    }
}
// f(an integral constant of the activation): the choice is made once, outside f's loops
template <int A> struct ActTag { static constexpr int value = A; };
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case GDN_ACT_SILU: f(ActTag<GDN_ACT_SILU>()); break;
    case GDN_ACT_GELU: f(ActTag<GDN_ACT_GELU>()); break;
    case GDN_ACT_GELU_TANH: f(ActTag<GDN_ACT_GELU_TANH>()); break;
    case GDN_ACT_RELU: f(ActTag<GDN_ACT_RELU>()); break;
    case GDN_ACT_SIGMOID: f(ActTag<GDN_ACT_SIGMOID>()); break;
    default: f(ActTag<GDN_ACT_NONE>());
    }
}

// What a product's epilogue does with z = sum_k A(m, k) B(n, k).
enum Epi : int {
    kEpiLinear = 0,    // out = act(sx_m sw_n z + bias_n) + extra_mn
    kEpiGated = 1,     // out = act(gate) up, gate / up from rows n and F + n of B
    kEpiDact = 2,      // out = extra_mn act'(z + bias_n); column sums of it over groups of rows into colpart
    kEpiGatedBwd = 3,  // out[m, n] = extra up act'(gate), out[m, F + n] = extra act(gate); out2 = act(gate) up
};

// One product with its epilogue.  A(m, k) is at a[m lda + k], or a[k lda + m] when a_t; B(n, k) at
// b[n ldb + k], or b[k ldb + n] when b_t.  Gated modes: B has 2 N rows, gate rows first.
struct GemmArgs {
    int64_t M, N, K;
    gdn_dtype in, out_dt;
    const void *a, *b;
    int64_t lda, ldb;
    int a_t, b_t;
    const float *x_scale, *w_scale;  // per row of A and of B, nullable (1)
    const float *bias;               // per column, nullable
    gdn_activation act;
    const void *extra;               // residual (nullable), dy or dh: [M][ld_extra], the output's type
    int64_t ld_extra;
    void *out;
    int64_t ldo;
    void *out2;                      // kEpiGatedBwd: the recomputed output [M][ldo2], nullable
    int64_t ldo2;
    float *colpart;                  // kEpiDact: column sums of groups of rows, [gemm_colparts][N], nullable
};

// bf16 and e4m3 operands whose rows start on 16-byte boundaries (tma_ok); output types as gdn_linear allows
cudaError_t launch_gemm_tc(const GemmArgs &g, Epi epi, cudaStream_t st);
bool tma_ok(const void *p, int64_t ld, int64_t rows, size_t esz);
// copies rows into a layout of `pitch` elements per row
cudaError_t launch_repack(const void *src, gdn_dtype t, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t pitch, cudaStream_t st);
gdn_status read_tc_status(cudaStream_t st);  // synchronises; clears
// the form for few rows (launch_gemm_tc chooses), its status word
cudaError_t launch_gemm_small(const GemmArgs &g, Epi epi, cudaStream_t st);
gdn_status read_small_status(cudaStream_t st);
// rows of partial column sums that a kEpiDact product writes
int64_t gemm_colparts(const GemmArgs &g, Epi epi);
int64_t gemm_small_colparts(const GemmArgs &g, Epi epi);
// a TMA map over `rows` rows of `cols` elements, boxes of 128 bytes x box_rows, 128-byte swizzle
bool make_operand_map(CUtensorMap *m, gdn_dtype t, const void *base, int64_t cols, int64_t rows, int64_t ld, int box_rows);

cudaError_t launch_gemm_simt(const GemmArgs &g, Epi epi, cudaStream_t st);

// out[n] = sum over `parts` rows of part[.][N] (a fixed order: the same sum every time)
cudaError_t launch_colsum_finish(const float *part, int64_t parts, int64_t N, float *out, cudaStream_t st);
// part[i][n] = sum of rows 32 i .. 32 i + 31 of x (M x N): `parts` of them must be ceil(M / 32)
cudaError_t launch_colsum_rows(const void *x, gdn_dtype dt, int64_t M, int64_t N, int64_t ld, float *part, cudaStream_t st);

struct NormArgs {
    int64_t M;
    int D;
    gdn_dtype dt, w_dt, out_dt;
    const void *x, *r;       // r nullable
    int64_t ldx, ldr;
    const void *w;           // [D], nullable (1)
    float eps;
    void *y;                 // [M][D], out_dt
    float *scale;            // e4m3: [M]
    void *h;                 // [M][D], nullable
    int normalise;           // 0: y = x (the quantiser alone)
};
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st);

struct NormBwdArgs {
    int64_t M;
    int D;
    gdn_dtype dt, w_dt;
    const void *dy, *h, *dh;  // dh nullable
    int64_t ld_dy, ld_h, ld_dh;
    const void *w;            // nullable
    float eps;
    void *dx;                 // [M][D]
    float *dw;                // [D], nullable
    float *part;              // workspace, norm_bwd_parts() rows of D
    float *rstd;              // workspace [M] (wide rows only)
};
int norm_bwd_parts(int64_t M, int D, gdn_dtype dt, int num_sms);  // rows of partial sums the launch writes
bool norm_bwd_wide(int D);  // rows too wide for one block's registers: the two-kernel form
cudaError_t launch_norm_bwd(const NormBwdArgs &a, int num_sms, cudaStream_t st);

// The library-managed workspace of (device, stream), grown to `need` bytes; and whether it holds them already.
gdn_status managed_workspace(size_t need, cudaStream_t stream, void **out, size_t *out_bytes);
bool managed_workspace_holds(size_t need, cudaStream_t stream);
int device_sm_count();  // of the current device (asked once per device)
// Whether this is the first call with `seen` on the current device; then the caller sets the kernel's attributes.
// (Two threads may both see a first call: setting an attribute twice is harmless.)
inline bool first_on_device(std::atomic<uint64_t> &seen)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return true;
    return !(seen.load(std::memory_order_relaxed) >> dev & 1);
}
inline void done_on_device(std::atomic<uint64_t> &seen)
{
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev <= 63) seen.fetch_or(1ull << dev, std::memory_order_relaxed);
}

// typed loads and stores
template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f<__nv_fp8_e4m3>(__nv_fp8_e4m3 v) { return (float)v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __nv_fp8_e4m3 from_f<__nv_fp8_e4m3>(float v)
{
    __nv_fp8_e4m3 q;
    q.__x = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
    return q;
}

}  // namespace gdn
