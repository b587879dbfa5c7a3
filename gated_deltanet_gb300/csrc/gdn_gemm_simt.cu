// Products of fp32 operands on the CUDA cores, with the epilogues of the decoder-block operators: few rows, which do not
// repay their splitting into bf16 planes for the tensor cores.
//
// A CTA of 256 threads owns a tile of 64 x 64 outputs, 4 x 4 entries per thread in packed pairs (one instruction, two fused
// multiply-adds), 32 values of k at a time through two buffers with the next ones on their way in registers.  The
// contraction is split over a cluster whose CTAs send their sums to the CTA that finishes the rows, in the order of the
// contraction, so that every SM has work.  A thread's columns are two groups half a tile apart, so that a gated tile holds
// gate and up columns of the same outputs in the same thread.  Bound: the latency of the loads (64 x 2048 x 2048:
// 28 us with the weights in L2, 29 from HBM; one row 26: the tile stays 64 rows); shared memory's 128 bytes a clock would be
// next.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kKt = 32, kMaxSplit = 8;
constexpr int kThreads = 256, T = 64, RM = 4, RG = 2, CN = 4, H = 2, kTy = 16;  // (rows and columns in two groups of two)
constexpr int kLd = T + 4, kRowStep = T / 2;
constexpr int E = T * kKt / kThreads, Q = E / 4;  // elements of each operand per thread and step, in fours
constexpr int kAcross = kThreads / kKt;

// four consecutive elements at p, zero from `left` on
__device__ __forceinline__ float4 load4(const float *p, bool row, int64_t left, bool vec)
{
    if (row && vec && left >= 4) return *(const float4 *)p;
    float4 v;
    v.x = row && left > 0 ? p[0] : 0.f;
    v.y = row && left > 1 ? p[1] : 0.f;
    v.z = row && left > 2 ? p[2] : 0.f;
    v.w = row && left > 3 ? p[3] : 0.f;
    return v;
}
__device__ __forceinline__ uint32_t peer_addr(const float *p, uint32_t cta)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(cta));
    return a;
}

template <int EPI>
__global__ void __launch_bounds__(kThreads, 2) gemm_simt_kernel(GemmArgs g, int mtiles, int split, int vec_a, int vec_b)
{
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    constexpr int kOutN = kGated ? T / 2 : T;        // output columns of a tile
    __shared__ __align__(16) float sa[2][kKt][kLd], sb[2][kKt][kLd];
    __shared__ float cs[EPI == kEpiDact ? kTy : 1][T];
    float *const red = &sa[0][0][0];  // [split][T / split][T], once the operands are dead: sums of the rows finished here
    static_assert(sizeof(sa) >= T * T * sizeof(float), "sums fit the operands' place");
    grid_release();
    grid_wait();
    const int tid = threadIdx.x, tx = (tid >> 5 & 1) * 8 + (tid & 7), ty = (tid >> 6) * 4 + (tid >> 3 & 3);
    const int rank = blockIdx.x % split;
    const int64_t tile = blockIdx.x / split;
    const int64_t m0 = tile % mtiles * T, n0 = tile / mtiles * kOutN;
    const float *A = (const float *)g.a, *B = (const float *)g.b;

    // This thread's elements of each operand's next values of k: consecutive along k of one row (K-major), or fours along
    // the rows at one k
    const int row = tid % T, koff = tid / T * E, kk = tid / kAcross, at = 4 * (tid % kAcross);
    float4 ra[Q], rb[Q];
    auto fetch = [&](int64_t k0) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (g.a_t) {
                const int64_t m = m0 + q * 4 * kAcross + at;
                ra[q] = load4(A + (k0 + kk) * g.lda + m, k0 + kk < g.K, g.M - m, vec_a);
            } else {
                const int64_t k = k0 + koff + 4 * q;
                ra[q] = load4(A + (m0 + row) * g.lda + k, m0 + row < g.M, g.K - k, vec_a);
            }
            if (g.b_t) {
                const int64_t n = n0 + q * 4 * kAcross + at;
                rb[q] = load4(B + (k0 + kk) * g.ldb + n, k0 + kk < g.K, g.N - n, vec_b);
            } else {
                const int64_t k = k0 + koff + 4 * q, n = n0 + (kGated ? row % kOutN : row);
                rb[q] = load4(B + (kGated && row >= kOutN ? g.N + n : n) * g.ldb + k, n < g.N, g.K - k, vec_b);
            }
        }
    };
    auto keep_one = [&](float (*dst)[kLd], const float4 *v, bool along) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (along) {
                *(float4 *)&dst[kk][q * 4 * kAcross + at] = v[q];
            } else {
                dst[koff + 4 * q][row] = v[q].x;
                dst[koff + 4 * q + 1][row] = v[q].y;
                dst[koff + 4 * q + 2][row] = v[q].z;
                dst[koff + 4 * q + 3][row] = v[q].w;
            }
        }
    };
    auto keep = [&](int buf) {
        keep_one(sa[buf], ra, g.a_t);
        keep_one(sb[buf], rb, g.b_t);
    };
    const int64_t kt = (g.K + kKt - 1) / kKt, kt0 = kt * rank / split, kt1 = kt * (rank + 1) / split;
    Pair acc[RM][H];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < H; ++j) acc[i][j].r = 0;
    if (kt0 < kt1) {
        fetch(kt0 * kKt);
        keep(0);
    }
    __syncthreads();
    for (int64_t t = kt0; t < kt1; ++t) {
        const int buf = (int)(t - kt0) & 1;
        if (t + 1 < kt1) fetch((t + 1) * kKt);
#pragma unroll
        for (int k = 0; k < kKt; ++k) {
            float a[RM];
            Pair b[H];
#pragma unroll
            for (int i = 0; i < RM; i += RG) {
                const float *p = &sa[buf][k][i / RG * kRowStep + RG * ty];
                *(float2 *)(a + i) = *(const float2 *)p;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float *p = &sb[buf][k][h * (T / 2) + H * tx];
                *(float2 *)(b + h) = *(const float2 *)p;
            }
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const Pair aa = pair_of(a[i], a[i]);
#pragma unroll
                for (int j = 0; j < H; ++j) acc[i][j] = fma2(aa, b[j], acc[i][j]);
            }
        }
        if (t + 1 < kt1) keep(buf ^ 1);
        __syncthreads();
    }

    // one pair of neighbouring outputs (m, n), (m, n + 1); returns dz in z (kEpiDact)
    float *out = (float *)g.out;
    const float *extra = (const float *)g.extra;
    auto finish = [&](auto tag, int64_t m, int64_t n, float *z, const float *u) {
        constexpr int ACT = decltype(tag)::value;
        float v[2], d[2];
        if (!kGated && g.bias) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (n + j < g.N) z[j] += g.bias[n + j];
        }
        if constexpr (EPI == kEpiLinear || EPI == kEpiGated) act_value<true, ACT>(z, v);
        else act_both<true, ACT>(z, v, d);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (m >= g.M || n + j >= g.N) {
                z[j] = 0.f;
                continue;
            }
            const int64_t c = n + j;
            if (EPI == kEpiLinear) {
                out[m * g.ldo + c] = extra ? v[j] + extra[m * g.ld_extra + c] : v[j];
            } else if (EPI == kEpiDact) {
                z[j] = extra[m * g.ld_extra + c] * d[j];
                out[m * g.ldo + c] = z[j];
            } else if (EPI == kEpiGated) {
                out[m * g.ldo + c] = v[j] * u[j];
            } else {
                const float dh = extra[m * g.ld_extra + c];
                out[m * g.ldo + c] = dh * u[j] * d[j];
                out[m * g.ldo + g.N + c] = dh * v[j];
                if (g.out2) ((float *)g.out2)[m * g.ldo2 + c] = v[j] * u[j];
            }
        }
    };
    auto row_of = [&](int i) { return i / RG * kRowStep + RG * ty + i % RG; };
    auto col_of = [&](int j) { return (j / H) * (T / 2) + H * tx + j % H; };
    int groups;  // row groups whose column sums lie in cs
    if (split == 1) {
        groups = kTy;
        float col[CN] = {};
        with_act(g.act, [&](auto tag) {
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const int64_t m = m0 + row_of(i);
                float z[CN];
#pragma unroll
                for (int j = 0; j < H; ++j) unpair(acc[i][j], z[2 * j], z[2 * j + 1]);
                if constexpr (kGated) {
#pragma unroll
                    for (int j = 0; j < H; j += 2) finish(tag, m, n0 + H * tx + j, z + j, z + H + j);
                } else {
#pragma unroll
                    for (int j = 0; j < CN; j += 2) {
                        finish(tag, m, n0 + col_of(j), z + j, z + j);
                        if (EPI == kEpiDact) {
                            col[j] += z[j];
                            col[j + 1] += z[j + 1];
                        }
                    }
                }
            }
        });
        if constexpr (EPI == kEpiDact) {
#pragma unroll
            for (int j = 0; j < CN; ++j) cs[ty][col_of(j)] = col[j];
        }
    } else {
        // partial sums to the CTAs that finish their rows, T / split each (whose operands are dead once all are here)
        const int per = T / split;
        asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            const int r = row_of(i);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                float x, y;
                unpair(acc[i][j], x, y);
                const uint32_t dst = peer_addr(red + (rank * per + r % per) * T + col_of(2 * j), r / per);
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(x), "f"(y) : "memory");
            }
        }
        asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
        constexpr int kPairs = kOutN / 2;
        groups = kThreads / kPairs;
        const int c = tid % kPairs * 2, grp = tid / kPairs;
        float col[2] = {};
        with_act(g.act, [&](auto tag) {
            for (int r = grp; r < per; r += kThreads / kPairs) {
                float z[2] = {}, u[2] = {};
                for (int s = 0; s < split; ++s) {
                    const float *p = red + (s * per + r) * T + c;
                    z[0] += p[0];
                    z[1] += p[1];
                    if (kGated) {
                        u[0] += p[T / 2];
                        u[1] += p[T / 2 + 1];
                    }
                }
                finish(tag, m0 + rank * per + r, n0 + c, z, u);
                col[0] += z[0];
                col[1] += z[1];
            }
        });
        if constexpr (EPI == kEpiDact) {
            cs[grp][c] = col[0];
            cs[grp][c + 1] = col[1];
        }
    }
    if constexpr (EPI == kEpiDact) {
        if (g.colpart) {
            __syncthreads();
            if (tid < T && n0 + tid < g.N) {
                float sum = 0.f;
                for (int i = 0; i < groups; ++i) sum += cs[i][tid];
                g.colpart[(tile % mtiles * split + rank) * g.N + n0 + tid] = sum;
            }
        }
    }
}

// tiles, and the contraction split for two CTAs on an SM
struct SimtPlan {
    int split, mtiles;
    int64_t tiles;
};
SimtPlan plan_simt(const GemmArgs &g, Epi epi)
{
    SimtPlan p;
    const int64_t sms = device_sm_count(), out_n = epi == kEpiGated || epi == kEpiGatedBwd ? T / 2 : T;
    p.mtiles = (int)((g.M + T - 1) / T);
    p.tiles = p.mtiles * ((g.N + out_n - 1) / out_n);
    p.split = 1;
    while (p.split < kMaxSplit && p.tiles * p.split * 2 <= 2 * sms && g.K / (p.split * 2) >= 2 * kKt) p.split *= 2;
    return p;
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
    const int64_t p = blockIdx.x;
    for (int64_t n = (int64_t)blockIdx.y * 128 + threadIdx.x; n < N; n += (int64_t)gridDim.y * 128) {
        float acc = 0.f;
        for (int64_t m = p * 32; m < M && m < p * 32 + 32; ++m) acc += to_f(x[m * ld + n]);
        part[p * N + n] = acc;
    }
}

}  // namespace

int64_t gemm_simt_colparts(const GemmArgs &g, Epi epi)
{
    const SimtPlan p = plan_simt(g, epi);
    return (int64_t)p.mtiles * p.split;
}

cudaError_t launch_gemm_simt(const GemmArgs &g, Epi epi, cudaStream_t st)
{
    if (g.M <= 0 || g.N <= 0) return cudaSuccess;
    const SimtPlan p = plan_simt(g, epi);
    auto on16 = [](const void *q, int64_t ld) { return ((uintptr_t)q & 15) == 0 && ld % 4 == 0; };
    auto go = [&](auto *kern) {
        return launch_overlapped(kern, (unsigned)(p.tiles * p.split), 1, kThreads, 0, p.split > 1 ? p.split : 0, st, g, p.mtiles, p.split,
                                 (int)on16(g.a, g.lda), (int)on16(g.b, g.ldb));
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
    const unsigned gx = (unsigned)((M + 31) / 32), gy = (unsigned)((N + 127) / 128 < 65535 ? (N + 127) / 128 : 65535);  // (a grid's most)
    if (dt == GDN_F32) return launch_overlapped(colsum_rows_kernel<float>, gx, gy, 128, 0, 0, st, (const float *)x, M, N, ld, part);
    return launch_overlapped(colsum_rows_kernel<__nv_bfloat16>, gx, gy, 128, 0, 0, st, (const __nv_bfloat16 *)x, M, N, ld, part);
}

}  // namespace gdn
