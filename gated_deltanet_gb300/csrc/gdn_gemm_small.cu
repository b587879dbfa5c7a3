// Products of few rows (decode, short batches) on the tensor cores: bound by reading the weights once.
//
// The roles of the operands are swapped: 128 rows of the weight are the M side of the instruction and up to
// NT rows of x its N side, so that one token costs an N = 16 instruction and not a padded 128 x 256 tile.  The
// contraction is split over a cluster of up to eight CTAs, which makes enough CTAs to keep every SM's
// loads in flight (N = 2048 alone is 16 tiles); their fp32 partial sums meet through distributed shared memory,
// each CTA of the cluster finishing its share of the rows of x, in a fixed order.  A CTA's shared memory is
// one long queue of 128-byte-wide weight boxes: most of what a CTA reads is requested at once.
#include <cstring>

#include <cudaTypedefs.h>

#include "gdn_layer.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

__device__ unsigned g_small_status;
constexpr unsigned long long kLimitNs = 2000000000ull;
constexpr int kThreads = 192;             // four epilogue warps, one that loads, one that issues
constexpr int kWBytes = 128 * 128;        // a stage's weights: 128 rows of 128 bytes
constexpr int kMaxStages = 12, kMaxSplit = 8;

struct SmallMaps {
    CUtensorMap w, x;
};
struct SmallParams {
    int64_t M, N;        // rows of x; output columns (gated: F)
    int kblocks, stages, split;
    int mtiles;
    const float *x_scale, *w_scale, *bias;
    int act;
    const void *extra;
    int64_t ld_extra;
    void *out;
    int64_t ldo;
    void *out2;
    int64_t ldo2;
    float *colpart;
};

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity)
{
    return mbar_wait(bar, parity, &g_small_status, kStatusTimeout, kLimitNs);
}
// a float at the same place in CTA `cta` of the cluster
__device__ __forceinline__ float peer_float(const float *p, uint32_t cta)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(cta));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
template <bool FP8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if (FP8)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc));
    else
        mma_ss(d, a, b, idesc, acc);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

// WT: the weight lies [contraction][features] (MN-major operand), else [features][contraction]
template <bool FP8, bool WT, int EPI, int NT, typename TO>
__global__ void __launch_bounds__(kThreads)
gemm_small_kernel(const __grid_constant__ SmallMaps maps, const SmallParams p)
{
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    constexpr bool kPrecise = sizeof(TO) == 4;
    constexpr int kOut = kGated ? 64 : 128;  // features of a tile
    constexpr int kStage = kWBytes + NT * 128;
    constexpr int kCols = NT < 32 ? 32 : NT;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
    __shared__ uint32_t tslot;
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *red = (float *)sm;  // [NT][128], once every stage is dead
    const int tid = threadIdx.x, warp = tid >> 5;
    const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
    const int mi = tile % p.mtiles, ni = tile / p.mtiles;
    const int64_t m0 = (int64_t)mi * NT, n0 = (int64_t)ni * kOut;
    const int kb0 = (int)((int64_t)p.kblocks * rank / p.split), kb1 = (int)((int64_t)p.kblocks * (rank + 1) / p.split);

    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc(&tslot, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tslot;
    bool ok = true;

    if (warp == 4) {
        int s = 0;
        uint32_t ph = 1;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!(ok = __all_sync(0xffffffffu, wait(&empty[s], ph)))) break;
            if (elect_one_sync()) {
                uint8_t *sw = sm + s * kStage, *sx = sw + kWBytes;
                const int k0 = kb * (FP8 ? 128 : 64);
                mbar_arrive_expect_tx(&full[s], kStage);
                if (kGated) {
                    tma_load_2d(sw, &maps.w, k0, (int)n0, &full[s]);
                    tma_load_2d(sw + 8192, &maps.w, k0, (int)(p.N + n0), &full[s]);
                } else if (WT) {
                    tma_load_2d(sw, &maps.w, (int)n0, k0, &full[s]);
                    tma_load_2d(sw + 8192, &maps.w, (int)n0 + 64, k0, &full[s]);
                } else {
                    tma_load_2d(sw, &maps.w, k0, (int)n0, &full[s]);
                }
                tma_load_2d(sx, &maps.x, k0, (int)m0, &full[s]);
            }
            __syncwarp();
            if (++s == p.stages) { s = 0; ph ^= 1; }
        }
    } else if (warp == 5) {
        constexpr uint32_t id = FP8 ? (1u << 4) | ((uint32_t)(NT >> 3) << 17) | (8u << 24) : idesc_bf16_f32(128, NT, WT, 0);
        int s = 0;
        uint32_t ph = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!(ok = __all_sync(0xffffffffu, wait(&full[s], ph)))) break;
            tc_fence_after();
            const uint32_t a = smem_u32(sm + s * kStage);
            const uint64_t da = sdesc_sw128(a, WT ? 8192 : 16, 1024), db = sdesc_sw128(a + kWBytes, 16, 1024);
            if (elect_one_sync()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mma<FP8>(tmem, da + j * (WT ? 128 : 2), db + j * 2, id, kb > kb0 || j);
                mma_commit(&empty[s]);
                if (kb + 1 == kb1) mma_commit(&done);
            }
            __syncwarp();
            if (++s == p.stages) { s = 0; ph ^= 1; }
        }
    } else {
        // this CTA's partial sums, [row of x][feature]
        ok = __all_sync(0xffffffffu, wait(&done, 0));
        if (ok) {
            tc_fence_after();
            const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
                if (m0 + c >= p.M) break;
                float v[16];
                tmem_ld16(tl + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) asm volatile("" : "+f"(v[j]));
#pragma unroll
                for (int j = 0; j < 16; ++j) red[(c + j) * 128 + tid] = v[j];
            }
            tc_fence_before();
        }
    }
    if (!ok) {
        // a wait ran out: give whatever is still in flight a millisecond to land before the memory is let go
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000) {}
    }
    __syncwarp();
    cluster_sync();
    if (warp < 4 && ok) {
        // rows rank, rank + split, ... of the tile: the partial sums in the order of the contraction, then the epilogue
        TO *out = (TO *)p.out;
        const TO *extra = (const TO *)p.extra;
        const int f = kGated ? tid & 63 : tid;
        const int64_t n = n0 + f;
        const int first = kGated ? rank + (tid >> 6) * p.split : rank, step = kGated ? 2 * p.split : p.split;
        const int rows = (int)(p.M - m0 < NT ? p.M - m0 : NT);
        const bool in = n < p.N;
        const float bias = !kGated && p.bias && in ? p.bias[n] : 0.f;
        const float wg = FP8 && p.w_scale && in ? p.w_scale[n] : 1.f;
        const float wu = FP8 && kGated && p.w_scale && in ? p.w_scale[p.N + n] : 1.f;
        float col = 0.f;
        with_act(p.act, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
            constexpr int U = 4;  // rows at a time, for loads in flight
            for (int t0 = first; t0 < rows; t0 += U * step) {
                float z[U] = {}, u[U] = {}, e[U] = {}, sx[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int t = t0 + i * step;
                    sx[i] = 1.f;
                    if (t >= rows) continue;
                    const int64_t m = m0 + t;
                    if (EPI != kEpiGated && extra && in) e[i] = to_f(extra[m * p.ld_extra + n]);
                    if (FP8 && p.x_scale) sx[i] = p.x_scale[m];
                    for (int c = 0; c < p.split; ++c) {
                        z[i] += peer_float(red + t * 128 + f, c);
                        if (kGated) u[i] += peer_float(red + t * 128 + 64 + f, c);
                    }
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int t = t0 + i * step;
                    if (t >= rows || !in) continue;
                    const int64_t m = m0 + t;
                    if (FP8 && p.w_scale) {
                        z[i] *= sx[i] * wg;
                        u[i] *= sx[i] * wu;
                    }
                    if (EPI == kEpiLinear) {
                        float y = act_value<kPrecise, ACT>(z[i] + bias);
                        out[m * p.ldo + n] = from_f<TO>(y + e[i]);
                    } else if (EPI == kEpiGated) {
                        out[m * p.ldo + n] = from_f<TO>(act_value<kPrecise, ACT>(z[i]) * u[i]);
                    } else if (EPI == kEpiDact) {
                        float v, d;
                        act_both<kPrecise, ACT>(z[i] + bias, v, d);
                        const float dz = e[i] * d;
                        out[m * p.ldo + n] = from_f<TO>(dz);
                        col += dz;
                    } else {
                        float v, d;
                        act_both<kPrecise, ACT>(z[i], v, d);
                        out[m * p.ldo + n] = from_f<TO>(e[i] * u[i] * d);
                        out[m * p.ldo + p.N + n] = from_f<TO>(e[i] * v);
                        if (p.out2) ((TO *)p.out2)[m * p.ldo2 + n] = from_f<TO>(v * u[i]);
                    }
                }
            }
        });
        if (EPI == kEpiDact && p.colpart && in) p.colpart[((int64_t)mi * p.split + rank) * p.N + n] = col;
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

size_t esz(gdn_dtype t) { return t == GDN_F32 ? 4 : t == GDN_BF16 ? 2 : 1; }

// How a product is cut: rows of x per tile, CTAs per contraction, CTAs resident per SM
struct SmallPlan {
    int nt, split, mtiles, stages;
    int64_t tiles;
    size_t smem;
};
SmallPlan plan_small(const GemmArgs &g, Epi epi)
{
    SmallPlan p{};
    const bool gated = epi == kEpiGated || epi == kEpiGatedBwd;
    p.nt = g.M <= 16 ? 16 : g.M <= 32 ? 32 : g.M <= 64 ? 64 : 128;
    p.mtiles = (int)((g.M + p.nt - 1) / p.nt);
    const int kb = (int)((g.K * (int64_t)esz(g.in) + 127) / 128);
    p.tiles = (g.N + (gated ? 63 : 127)) / (gated ? 64 : 128) * p.mtiles;
    // as many CTAs as two per SM hold; every CTA keeps at least two blocks of the contraction
    const int64_t slots = 2 * device_sm_count();
    int64_t split = slots / p.tiles;
    split = split > kMaxSplit ? kMaxSplit : split;
    split = split > kb / 2 ? kb / 2 : split;
    p.split = (int)(split < 1 ? 1 : split);
    const bool two = p.tiles * p.split > device_sm_count();
    const size_t stage = kWBytes + p.nt * 128, room = (two ? 110 : 222) * 1024;
    p.stages = (int)(room / stage);
    const int need = (kb + p.split - 1) / p.split;
    p.stages = p.stages > kMaxStages ? kMaxStages : p.stages;
    p.stages = p.stages > need ? need : p.stages;
    const size_t bytes = p.stages * stage, redb = (size_t)p.nt * 512;
    p.smem = 1024 + (bytes > redb ? bytes : redb);
    return p;
}

template <bool FP8, bool WT, int EPI, int NT, typename TO>
cudaError_t go(const GemmArgs &g, const SmallPlan &pl, cudaStream_t st)
{
    constexpr bool gated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    SmallMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const int64_t wrows = gated ? 2 * g.N : g.N;
    const bool w_ok = WT ? make_operand_map(&maps.w, g.in, g.b, g.N, g.K, g.ldb, 64)
                         : make_operand_map(&maps.w, g.in, g.b, g.K, wrows, g.ldb, gated ? 64 : 128);
    if (!w_ok || !make_operand_map(&maps.x, g.in, g.a, g.K, g.M, g.lda, NT)) return cudaErrorInvalidValue;
    SmallParams p{};
    p.M = g.M; p.N = g.N;
    p.kblocks = (int)((g.K * (int64_t)esz(g.in) + 127) / 128);
    p.stages = pl.stages; p.split = pl.split; p.mtiles = pl.mtiles;
    p.x_scale = g.x_scale; p.w_scale = g.w_scale; p.bias = g.bias; p.act = g.act;
    p.extra = g.extra; p.ld_extra = g.ld_extra;
    p.out = g.out; p.ldo = g.ldo; p.out2 = g.out2; p.ldo2 = g.ldo2;
    p.colpart = g.colpart;
    auto *kern = gemm_small_kernel<FP8, WT, EPI, NT, TO>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pl.tiles * pl.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)pl.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

template <bool FP8, bool WT, int EPI, typename TO>
cudaError_t pick(const GemmArgs &g, cudaStream_t st)
{
    const SmallPlan p = plan_small(g, (Epi)EPI);
    switch (p.nt) {
    case 16: return go<FP8, WT, EPI, 16, TO>(g, p, st);
    case 32: return go<FP8, WT, EPI, 32, TO>(g, p, st);
    case 64: return go<FP8, WT, EPI, 64, TO>(g, p, st);
    default: return go<FP8, WT, EPI, 128, TO>(g, p, st);
    }
}

}  // namespace

int64_t gemm_small_colparts(const GemmArgs &g, Epi epi)
{
    const SmallPlan p = plan_small(g, epi);
    return (int64_t)p.mtiles * p.split;
}

cudaError_t launch_gemm_small(const GemmArgs &g, Epi epi, cudaStream_t st)
{
    if (g.M <= 0 || g.N <= 0) return cudaSuccess;
    const bool f32 = g.out_dt == GDN_F32;
    if (g.in == GDN_E4M3) {
        if (epi == kEpiGated) return pick<true, false, kEpiGated, __nv_bfloat16>(g, st);
        return f32 ? pick<true, false, kEpiLinear, float>(g, st) : pick<true, false, kEpiLinear, __nv_bfloat16>(g, st);
    }
    switch (epi) {
    case kEpiGated: return pick<false, false, kEpiGated, __nv_bfloat16>(g, st);
    case kEpiGatedBwd: return pick<false, false, kEpiGatedBwd, __nv_bfloat16>(g, st);
    case kEpiDact: return pick<false, false, kEpiDact, __nv_bfloat16>(g, st);
    default: break;
    }
    if (g.b_t) return pick<false, true, kEpiLinear, __nv_bfloat16>(g, st);
    return f32 ? pick<false, false, kEpiLinear, float>(g, st) : pick<false, false, kEpiLinear, __nv_bfloat16>(g, st);
}

gdn_status read_small_status(cudaStream_t st)
{
    unsigned word = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, g_small_status, sizeof(word), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_small_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return word & kStatusTimeout ? GDN_ERR_TIMEOUT : GDN_OK;
}

}  // namespace gdn
