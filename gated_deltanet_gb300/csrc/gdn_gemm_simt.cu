// Products on the CUDA cores, with the epilogues of the decoder-block operators: fp32 inputs.
//
// A 64 x 64 tile of the output per CTA of 256 threads, 4 x 4 entries per thread, fp32 sums in the
// order of k; 16 values of k at a time through shared memory.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kT = 64, kKt = 16;

template <int EPI>
__global__ void __launch_bounds__(256) gemm_simt_kernel(GemmArgs g)
{
    constexpr bool kTwo = EPI == kEpiGated || EPI == kEpiGatedBwd;
    constexpr int kB = kTwo ? 2 : 1;
    __shared__ float sa[kKt][kT + 4], sb[kB][kKt][kT + 4];
    __shared__ float cs[16][kT];
    grid_release();
    grid_wait();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * kT, n0 = (int64_t)blockIdx.y * kT;  // (x has the larger limit)
    const float *A = (const float *)g.a, *B = (const float *)g.b;
    float acc[kB][4][4] = {};
    for (int64_t k0 = 0; k0 < g.K; k0 += kKt) {
        // consecutive threads along the operand's contiguous index
        for (int i = tid; i < kT * kKt; i += 256) {
            const int mi = g.a_t ? i & (kT - 1) : i / kKt, ki = g.a_t ? i / kT : i & (kKt - 1);
            const int64_t m = m0 + mi, k = k0 + ki;
            sa[ki][mi] = m < g.M && k < g.K ? A[g.a_t ? k * g.lda + m : m * g.lda + k] : 0.f;
            const int ni = g.b_t ? i & (kT - 1) : i / kKt, kj = g.b_t ? i / kT : i & (kKt - 1);
            const int64_t n = n0 + ni, kk = k0 + kj;
#pragma unroll
            for (int h = 0; h < kB; ++h) {
                const int64_t row = n + h * g.N;
                sb[h][kj][ni] = n < g.N && kk < g.K ? B[g.b_t ? kk * g.ldb + row : row * g.ldb + kk] : 0.f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKt; ++k) {
            const float4 a = *(const float4 *)&sa[k][4 * ty];
            const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int h = 0; h < kB; ++h) {
                const float4 b = *(const float4 *)&sb[h][k][4 * tx];
                const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(av[i], bv[j], acc[h][i][j]);
            }
        }
        __syncthreads();
    }
    float *out = (float *)g.out;
    const float *extra = (const float *)g.extra;
    float col[4] = {};
    with_act(g.act, [&](auto tag) {
        constexpr int ACT = decltype(tag)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + 4 * ty + i;
            if (m >= g.M) continue;
            float v[4], d[4];
            if (EPI == kEpiLinear || EPI == kEpiDact) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (g.bias && n0 + 4 * tx + j < g.N) acc[0][i][j] += g.bias[n0 + 4 * tx + j];
            }
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                if (EPI == kEpiLinear || EPI == kEpiGated) act_value<true, ACT>(&acc[0][i][j], v + j);
                else act_both<true, ACT>(&acc[0][i][j], v + j, d + j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + 4 * tx + j;
                if (n >= g.N) continue;
                const float u = acc[kB - 1][i][j];
                if (EPI == kEpiLinear) {
                    out[m * g.ldo + n] = extra ? v[j] + extra[m * g.ld_extra + n] : v[j];
                } else if (EPI == kEpiDact) {
                    const float dz = extra[m * g.ld_extra + n] * d[j];
                    out[m * g.ldo + n] = dz;
                    col[j] += dz;
                } else if (EPI == kEpiGated) {
                    out[m * g.ldo + n] = v[j] * u;
                } else {
                    const float dh = extra[m * g.ld_extra + n];
                    out[m * g.ldo + n] = dh * u * d[j];
                    out[m * g.ldo + g.N + n] = dh * v[j];
                    if (g.out2) ((float *)g.out2)[m * g.ldo2 + n] = v[j] * u;
                }
            }
        }
    });
    if (EPI == kEpiDact && g.colpart) {
        // this tile's column sums over its two groups of 32 rows
#pragma unroll
        for (int j = 0; j < 4; ++j) cs[ty][4 * tx + j] = col[j];
        __syncthreads();
        if (tid < 2 * kT) {
            const int half = tid / kT, c = tid % kT;
            float s = 0.f;
            for (int i = 0; i < 8; ++i) s += cs[8 * half + i][c];
            const int64_t p = m0 / 32 + half, n = n0 + c;
            if (n < g.N && p * 32 < g.M) g.colpart[p * g.N + n] = s;
        }
    }
}

// 32 columns per CTA, the parts dealt to 32 warps, whose sums meet in a fixed order
__global__ void __launch_bounds__(1024) colsum_finish_kernel(const float *part, int64_t parts, int64_t N, float *out)
{
    __shared__ float s[32][33];
    grid_release();
    grid_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t n = (int64_t)blockIdx.x * 32 + lane;
    float acc = 0.f;
    if (n < N) {
#pragma unroll 8
        for (int64_t p = w; p < parts; p += 32) acc += part[p * N + n];
    }
    s[w][lane] = acc;
    __syncthreads();
    // warp w sums column w of the tile
    acc = s[lane][w];
#pragma unroll
    for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (lane == 0 && (int64_t)blockIdx.x * 32 + w < N) out[(int64_t)blockIdx.x * 32 + w] = acc;
}

template <typename T>
__global__ void __launch_bounds__(128) colsum_rows_kernel(const T *x, int64_t M, int64_t N, int64_t ld, float *part)
{
    grid_release();
    grid_wait();
    const int64_t n = (int64_t)blockIdx.y * 128 + threadIdx.x, p = blockIdx.x;
    if (n >= N) return;
    float acc = 0.f;
    for (int64_t m = p * 32; m < M && m < p * 32 + 32; ++m) acc += to_f(x[m * ld + n]);
    part[p * N + n] = acc;
}

}  // namespace

cudaError_t launch_gemm_simt(const GemmArgs &g, Epi epi, cudaStream_t st)
{
    if (g.M <= 0 || g.N <= 0) return cudaSuccess;
    auto go = [&](auto *kern) {
        return launch_overlapped(kern, (unsigned)((g.M + kT - 1) / kT), (unsigned)((g.N + kT - 1) / kT), 256, 0, 0, st, g);
    };
    switch (epi) {
    case kEpiGated: return go(gemm_simt_kernel<kEpiGated>);
    case kEpiDact: return go(gemm_simt_kernel<kEpiDact>);
    case kEpiGatedBwd: return go(gemm_simt_kernel<kEpiGatedBwd>);
    default: return go(gemm_simt_kernel<kEpiLinear>);
    }
}

cudaError_t launch_colsum_finish(const float *part, int64_t parts, int64_t N, float *out, cudaStream_t st)
{
    if (N <= 0) return cudaSuccess;
    return launch_overlapped(colsum_finish_kernel, (unsigned)((N + 31) / 32), 1, 1024, 0, 0, st, part, parts, N, out);
}

cudaError_t launch_colsum_rows(const void *x, gdn_dtype dt, int64_t M, int64_t N, int64_t ld, float *part, cudaStream_t st)
{
    if (M <= 0 || N <= 0) return cudaSuccess;
    const unsigned gx = (unsigned)((M + 31) / 32), gy = (unsigned)((N + 127) / 128);
    if (dt == GDN_F32) return launch_overlapped(colsum_rows_kernel<float>, gx, gy, 128, 0, 0, st, (const float *)x, M, N, ld, part);
    return launch_overlapped(colsum_rows_kernel<__nv_bfloat16>, gx, gy, 128, 0, 0, st, (const __nv_bfloat16 *)x, M, N, ld, part);
}

}  // namespace gdn
