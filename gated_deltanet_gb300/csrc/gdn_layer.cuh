// Internal declarations of the decoder-block operators (norm, linear, gated linear unit): the
// argument blocks of their kernels and the arithmetic that every engine's epilogue shares.
//
// Figures in the comments at these kernels are of calls on the same tensors, twenty in a captured graph, unless they say
// otherwise: what fits L2 is read from there.
#pragma once

#include <atomic>

#include <cuda_fp8.h>

#include "gdn_internal.cuh"

namespace gdn {

// Activations.  `PRECISE` (fp32 outputs) takes the full-accuracy exponential and division; otherwise the
// result is rounded to bf16 (relative step 2^-8) and the fast ones are enough: the rounding of the exponent makes exp(-z) off by up to
// |z| 2^-23 of itself (2^-16.5 at |z| = 90), the approximate exponential and reciprocal by 2^-21.  A logistic function below the
// smallest normal fp32 number (z < -87.3) is flushed to 0, so that silu is 0 there where it is -1e-36 and less.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kF32Max = 3.40282347e38f, kBf16Max = 3.38953139e38f;
__device__ __forceinline__ float fast_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <bool PRECISE>
__device__ __forceinline__ float logistic(float z)
{
    return PRECISE ? 1.f / (1.f + expf(-z)) : fast_rcp(1.f + fast_exp2(-kLog2e * z));
}
// two fp32 lanes of one instruction
struct Pair {
    uint64_t r;
};
__device__ __forceinline__ Pair pair_of(float x, float y)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.r) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ void unpair(Pair p, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p.r)); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.r) : "l"(a.r), "l"(b.r), "l"(c.r));
    return d;
}
constexpr float kGeluA = 1.5957691216057308f;            // 2 sqrt(2 / pi): 0.5 (1 + tanh u) = logistic(2 u)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

// The normal distribution function Phi(z) = erfc(-z / sqrt 2) / 2 of two values, and exp(-z^2 / 2).  Not PRECISE:
// erfc(x) = t exp(-x^2 + P(t)) with t = 1 / (1 + x / 2), a published form (Press et al., Numerical Recipes), P here a fit of
// its own: the degree-9 minimax polynomial of log(exp(x^2) erfc(x) / t)
// over 0 < t <= 1 (iteratively reweighted least squares on 4000 Chebyshev nodes: off by 1.0e-7 of the value everywhere, so
// that the small tail keeps its digits); P and x^2 in units of log 2, the factor 1/2 in P's constant.  No branch (erff
// takes both of its own in almost every warp: the gradient through gelu took 114 us at 16384 x 2048 x 2048, 103 with
// this), two values to an instruction.
template <bool PRECISE>
__device__ __forceinline__ void normal_cdf(const float *z, float *phi, float *bell)
{
    if constexpr (PRECISE) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            phi[i] = 0.5f * erfcf(z[i] * -0.70710678118654752f);
            bell[i] = expf(-0.5f * z[i] * z[i]);
        }
    } else {
        float x[2], t[2], e[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            t[i] = fast_rcp(fmaf(fabsf(z[i]), 0.35355339059327376f, 1.f));
            x[i] = z[i] * 0.84932180028801907f;  // x^2: z^2 / 2 in units of log 2
        }
        const Pair tt = pair_of(t[0], t[1]);
        Pair p = pair_of(0.24143842f, 0.24143842f);
        constexpr float c[9] = {-1.16414727f, 2.10785656f, -1.59912835f, 0.38024972f, -0.26125970f, 0.13816426f, 0.53985201f, 1.44272232f, -2.82574812f};
#pragma unroll
        for (int k = 0; k < 9; ++k) p = fma2(p, tt, pair_of(c[k], c[k]));
        p = fma2(pair_of(-x[0], -x[1]), pair_of(x[0], x[1]), p);
        unpair(p, e[0], e[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float half = t[i] * fast_exp2(e[i]);  // erfc(|z| / sqrt 2) / 2
            phi[i] = z[i] < 0.f ? half : 1.f - half;
            bell[i] = fast_exp2(-x[i] * x[i]);
        }
    }
}

// the activation of two values
template <bool PRECISE, int ACT>
__device__ __forceinline__ void act_value(const float *z, float *v)
{
    if constexpr (ACT == GDN_ACT_GELU) {
        float phi[2], bell[2];
        normal_cdf<PRECISE>(z, phi, bell);
        v[0] = z[0] * phi[0];
        v[1] = z[1] * phi[1];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (ACT == GDN_ACT_SILU) v[i] = z[i] * logistic<PRECISE>(z[i]);
            else if (ACT == GDN_ACT_GELU_TANH) v[i] = z[i] * logistic<PRECISE>(z[i] * (kGeluA + kGeluB * z[i] * z[i]));
            else if (ACT == GDN_ACT_RELU) v[i] = z[i] < 0.f ? 0.f : z[i];  // (keeps a NaN)
            else if (ACT == GDN_ACT_SIGMOID) v[i] = logistic<PRECISE>(z[i]);
            else v[i] = z[i];
        }
    }
}
// values and derivatives
template <bool PRECISE, int ACT>
__device__ __forceinline__ void act_both(const float *z, float *v, float *d)
{
    if constexpr (ACT == GDN_ACT_GELU) {
        float phi[2], bell[2];
        normal_cdf<PRECISE>(z, phi, bell);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[i] = z[i] * phi[i];
            d[i] = fmaf(z[i] * 0.3989422804014327f, bell[i], phi[i]);  // 1 / sqrt(2 pi)
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (ACT == GDN_ACT_SILU) {
                const float p = logistic<PRECISE>(z[i]);
                v[i] = z[i] * p;
                d[i] = fmaf(v[i], 1.f - p, p);
            } else if (ACT == GDN_ACT_GELU_TANH) {
                const float z2 = z[i] * z[i], p = logistic<PRECISE>(z[i] * (kGeluA + kGeluB * z2));
                v[i] = z[i] * p;
                // (z^2 may pass fp32's range, where p is 0 or 1 and the product with it has to stay 0)
                d[i] = p + v[i] * (1.f - p) * fminf(kGeluA + 3.f * kGeluB * z2, kF32Max);
            } else if (ACT == GDN_ACT_RELU) {
                v[i] = z[i] < 0.f ? 0.f : z[i];
                d[i] = z[i] > 0.f ? 1.f : 0.f;
            } else if (ACT == GDN_ACT_SIGMOID) {
                // p (1 - p): for z > 0 the difference as exp(-z) p (1 - p itself has lost its digits from z of about 10 on)
                const float e = PRECISE ? expf(-z[i]) : fast_exp2(-kLog2e * z[i]), p = PRECISE ? 1.f / (1.f + e) : fast_rcp(1.f + e);
                v[i] = p;
                d[i] = p * (z[i] > 0.f ? e * p : 1.f - p);
            } else {
                v[i] = z[i];
                d[i] = 1.f;
            }
        }
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

// How long a device-side wait of the products may last.  The calling thread's switch for testing what happens then
// (gdn_layer_test_withhold): launches of kernel instances of their own, whose load warps load nothing and whose waits have a
// limit of 5 ms.  (As run-time arguments of every instance the switch and the limit cost a token's product 0.16 of 7.9 us.)
constexpr uint64_t kWaitLimitNs = 2000000000ull, kTestWaitLimitNs = 5000000ull;
bool &withhold_loads();

constexpr int64_t kFewRows = 128;  // bf16 and e4m3 rows to this many take the kernel of few rows

// One product with its epilogue.  A(m, k) is at a[m lda + k], or a[k lda + m] when a_t; B(n, k) at
// b[n ldb + k], or b[k ldb + n] when b_t.  Gated modes: B has 2 N rows, gate rows first.
struct GemmArgs {
    int64_t M, N, K;
    gdn_dtype in, out_dt;
    const void *a, *b;
    int64_t lda, ldb;
    int a_t, b_t;
    int64_t a_plane, b_plane;        // fp32 as three bf16 planes, this many elements apart (0: as it is)
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

// bf16 and e4m3 operands whose rows start on 16-byte boundaries (tma_ok), fp32 ones as planes; output types as
// gdn_linear allows
cudaError_t launch_gemm_tc(const GemmArgs &g, Epi epi, cudaStream_t st);
bool tma_ok(const void *p, int64_t ld, int64_t rows, size_t esz);
// fp32 rows into three planes of bf16 (`plane` elements apart, `pitch` elements per row)
cudaError_t launch_split(const float *src, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t pitch, int64_t plane, cudaStream_t st);
// copies rows into a layout of `pitch` elements per row
cudaError_t launch_copy_rows(const void *src, gdn_dtype t, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t ldd, cudaStream_t st);
gdn_status read_tc_status(cudaStream_t st);  // its status word: synchronises; clears
// the form for few rows (launch_gemm_tc chooses), and its status word
cudaError_t launch_gemm_small(const GemmArgs &g, Epi epi, cudaStream_t st);
gdn_status read_small_status(cudaStream_t st);
// rows of partial column sums that a kEpiDact product writes
int64_t gemm_colparts(const GemmArgs &g, Epi epi);
int64_t gemm_small_colparts(const GemmArgs &g, Epi epi);
// a TMA map over `rows` rows of `cols` elements (bf16, e4m3), boxes of 128 bytes x box_rows, 128-byte swizzle
bool make_operand_map(CUtensorMap *m, gdn_dtype t, const void *base, int64_t cols, int64_t rows, int64_t ld, int box_rows);

cudaError_t launch_gemm_simt(const GemmArgs &g, Epi epi, cudaStream_t st);
int64_t gemm_simt_colparts(const GemmArgs &g, Epi epi);

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

// Launches of these operators overlap their neighbours' ends: a kernel may be set up while the one before it in the
// stream still runs (programmatic stream serialisation), waits for it with grid_wait() before it touches global memory,
// and lets the next one be set up with grid_release().  A kernel that holds tensor memory releases only once it has it:
// a successor that got the columns first would wait for a kernel that waits for columns.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), unsigned grid_x, unsigned grid_y, int threads, size_t smem, int cluster, cudaStream_t st,
                              const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid_x, grid_y);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
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
