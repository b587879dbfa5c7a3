// Products of few rows (decode, short batches) on the tensor cores: they read the weights once, and are bound by that and by
// what a launch, a wait for the first weights and a meeting of the cluster take.
//
// The roles of the operands are swapped: 128 rows of the weight are the M side of the instruction and up to
// NT rows of x its N side, so that one token costs an N = 16 instruction and not a padded 128 x 256 tile.  The
// contraction is split over a cluster of up to eight CTAs, which makes enough CTAs to keep every SM's
// loads in flight (N = 2048 alone is 16 tiles).  Each CTA sends its fp32 partial sums to the CTAs of the cluster
// that finish the rows of x in turn (row t: CTA t mod split), which add them in the order of the
// contraction; sums are sent and not fetched, so that one meeting of the cluster is enough.  A CTA's shared
// memory is one queue of 128-byte-wide weight boxes, and two CTAs share an SM: most of what they read is
// requested at once.  Measured: 64 rows of 2048 by 11008 gated bf16 weights (45 MB) 12.6 us from HBM, 9.1 from L2 (x is
// staged again for each of its 86 weight tiles: 109 MB through L2); one row by 2048 x 5504 7.2 us from HBM, 5.5 from L2.
#include <atomic>
#include <cstring>

#include <cudaTypedefs.h>

#include "gdn_layer.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

__device__ unsigned g_small_status;
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
    int vec_out, vec_extra;  // rows of out (and out2), of extra allow groups of four elements
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    return mbar_wait(bar, parity, &g_small_status, kStatusTimeout, limit_ns);
}
// the shared memory of CTA `cta` of the cluster, at the place of p
__device__ __forceinline__ uint32_t peer_addr(const float *p, uint32_t cta)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(cta));
    return a;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
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

// WT: the weight lies [contraction][features] (MN-major operand), else [features][contraction].  WITHHOLD: the load warp loads
// nothing, so that every wait for operands runs out.
template <bool FP8, bool WT, int EPI, int NT, typename TO, bool WITHHOLD>
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
    __shared__ float cols[EPI == kEpiDact ? kThreads / 32 : 1][128];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *red = (float *)(sm + p.stages * kStage);  // [split][slots][128]: partial sums of the rows finished here
    const int slots = (NT + p.split - 1) / p.split;
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
    cluster_arrive();  // (waited for before the first store into another CTA)
    tc_fence_after();
    const uint32_t tmem = tslot;
    bool ok = true;
    constexpr uint64_t limit = WITHHOLD ? kTestWaitLimitNs : kWaitLimitNs;
    grid_release();
    grid_wait();

    if (warp == 4) {
        int s = 0;
        uint32_t ph = 1;
        for (int kb = WITHHOLD ? kb1 : kb0; kb < kb1; ++kb) {
            if (!(ok = __all_sync(0xffffffffu, wait(&empty[s], ph, limit)))) break;
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
        bool ready = false;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!ready && !(ok = __all_sync(0xffffffffu, wait(&full[s], ph, limit)))) break;
            tc_fence_after();
            uint64_t *const rel = &empty[s];
            const uint32_t a = smem_u32(sm + s * kStage);
            const uint64_t da = sdesc_sw128(a, WT ? 8192 : 16, 1024), db = sdesc_sw128(a + kWBytes, 16, 1024);
            if (++s == p.stages) { s = 0; ph ^= 1; }
            // the next block's state, asked for before this block's products are issued
            ready = __all_sync(0xffffffffu, mbar_test_wait(&full[s], ph));
            if (elect_one_sync()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mma<FP8>(tmem, da + j * (WT ? 128 : 2), db + j * 2, id, kb > kb0 || j);
                mma_commit(rel);
                if (kb + 1 == kb1) mma_commit(&done);
            }
            __syncwarp();
        }
    } else {
        ok = __all_sync(0xffffffffu, wait(&done, 0, limit));
        tc_fence_after();
    }
    if (!ok) {
        // a wait ran out: give whatever is still in flight a millisecond to land before the memory is let go
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000) {}
    }
    __syncwarp();
    cluster_wait();  // every CTA of the cluster runs
    if (warp < 4 && ok) {
        // partial sums to the CTAs that finish their rows: lane = feature, so 32 lanes store 128 bytes
        const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
        int owner = 0, slot = 0;
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
            if (m0 + c >= p.M) break;
            float v[16];
            tmem_ld16(tl + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) asm volatile("" : "+f"(v[j]));
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (m0 + c + j < p.M) peer_store(peer_addr(red + (rank * slots + slot) * 128 + tid, owner), v[j]);
                if (++owner == p.split) { owner = 0; ++slot; }
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (ok) {
        // rows rank, rank + split, ... of the tile: the partial sums in the order of the contraction, then the
        // epilogue; four features a thread, a row per 32 (gated: 16) threads
        constexpr int kPer = kOut / 4, kGroups = kThreads / kPer, kElem = (int)sizeof(TO);
        TO *out = (TO *)p.out;
        const TO *extra = (const TO *)p.extra;
        const int f = tid % kPer * 4, grp = tid / kPer;
        const int64_t n = n0 + f;
        const int rows = (int)(p.M - m0 < NT ? p.M - m0 : NT);
        const int mine = rows > rank ? (rows - rank + p.split - 1) / p.split : 0;  // rows finished here
        const int have = p.N - n >= 4 ? 4 : p.N > n ? (int)(p.N - n) : 0;          // features that exist
        // whole groups of four by one load or store, where every row allows it
        const bool vec_out = have == 4 && p.vec_out, vec_extra = have == 4 && p.vec_extra;
        float bias[4], wg[4], wu[4], col[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bias[j] = !kGated && p.bias && j < have ? p.bias[n + j] : 0.f;
            wg[j] = FP8 && p.w_scale && j < have ? p.w_scale[n + j] : 1.f;
            wu[j] = FP8 && kGated && p.w_scale && j < have ? p.w_scale[p.N + n + j] : 1.f;
        }
        auto put = [&](TO *dst, const float *v) {
            if (vec_out) {
                if constexpr (kElem == 2) *(uint2 *)dst = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                else *(float4 *)dst = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < have) dst[j] = from_f<TO>(v[j]);
            }
        };
        with_act(p.act, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
            for (int sl = grp; sl < mine; sl += kGroups) {
                const int64_t m = m0 + rank + (int64_t)sl * p.split;
                float e[4] = {};
                if (EPI != kEpiGated && extra) {
                    const TO *src = extra + m * p.ld_extra + n;
                    if (vec_extra) {
                        if constexpr (kElem == 2) {
                            const uint2 u = *(const uint2 *)src;
                            e[0] = __uint_as_float(u.x << 16); e[1] = __uint_as_float(u.x & 0xffff0000u);
                            e[2] = __uint_as_float(u.y << 16); e[3] = __uint_as_float(u.y & 0xffff0000u);
                        } else {
                            const float4 u = *(const float4 *)src;
                            e[0] = u.x; e[1] = u.y; e[2] = u.z; e[3] = u.w;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < have) e[j] = to_f(src[j]);
                    }
                }
                const float sx = FP8 && p.x_scale ? p.x_scale[m] : 1.f;
                float z[4] = {}, u[4] = {};
                for (int c = 0; c < p.split; ++c) {
                    const float *r = red + (c * slots + sl) * 128 + f;
                    const float4 a = *(const float4 *)r;
                    z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
                    if (kGated) {
                        const float4 b = *(const float4 *)(r + 64);
                        u[0] += b.x; u[1] += b.y; u[2] += b.z; u[3] += b.w;
                    }
                }
                float y[4], y2[4], a[4], d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (FP8 && p.w_scale) {
                        z[j] *= sx * wg[j];
                        u[j] *= sx * wu[j];
                    }
                    if (!kGated) z[j] += bias[j];
                }
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    if (EPI == kEpiLinear || EPI == kEpiGated) act_value<kPrecise, ACT>(z + j, a + j);
                    else act_both<kPrecise, ACT>(z + j, a + j, d + j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (EPI == kEpiLinear) {
                        y[j] = a[j] + e[j];
                    } else if (EPI == kEpiGated) {
                        y[j] = a[j] * u[j];
                    } else if (EPI == kEpiDact) {
                        y[j] = e[j] * d[j];
                        col[j] += y[j];
                    } else {
                        y[j] = e[j] * u[j] * d[j];
                        y2[j] = e[j] * a[j];
                        z[j] = a[j] * u[j];
                    }
                }
                put(out + m * p.ldo + n, y);
                if (EPI == kEpiGatedBwd) {
                    put(out + m * p.ldo + p.N + n, y2);
                    if (p.out2) put((TO *)p.out2 + m * p.ldo2 + n, z);
                }
            }
        });
        if (EPI == kEpiDact && p.colpart) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cols[grp][f + j] = col[j];
        }
    }
    if (EPI == kEpiDact && p.colpart) {
        __syncthreads();
        if (tid < 128 && n0 + tid < p.N) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) sum += cols[w][tid];
            p.colpart[((int64_t)mi * p.split + rank) * p.N + n0 + tid] = sum;
        }
    }
    if (warp == 5) {  // (the accumulators were read before the cluster met)
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

size_t esz(gdn_dtype t) { return t == GDN_BF16 ? 2 : 1; }  // of an operand

constexpr size_t kRoom = 110 * 1024;  // a CTA's shared memory: two on an SM

// How a product is cut: rows of x per tile, CTAs per contraction
struct SmallPlan {
    int nt, split, mtiles, stages;
    int64_t tiles;
    size_t smem;
};

// two CTAs of this size on an SM (without the carve-out the driver leaves room for one)
template <typename F>
cudaError_t allow_two(F *kern)
{
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRoom);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

// A kernel of the same block and shared memory that holds no tensor memory: the runtime answers one block per SM
// for every kernel that allocates tensor memory, whatever it holds, while the SM runs two of them.
__global__ void __launch_bounds__(kThreads) place_kernel() {}

// clusters of `split` CTAs of this size that the device runs at once (asked once per device)
int64_t clusters_at_once(int split)
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][kMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = 0;
    int n = known[dev][split].load(std::memory_order_relaxed);
    if (n) return n;
    auto *kern = place_kernel;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRoom;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (allow_two(kern) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = 2 * device_sm_count() / (split + 1);
    }
    known[dev][split].store(n, std::memory_order_relaxed);
    return n;
}

SmallPlan plan_small(const GemmArgs &g, Epi epi)
{
    SmallPlan p{};
    const bool gated = epi == kEpiGated || epi == kEpiGatedBwd;
    p.nt = g.M <= 16 ? 16 : g.M <= 32 ? 32 : 64;
    p.mtiles = (int)((g.M + p.nt - 1) / p.nt);
    const int kb = (int)((g.K * (int64_t)esz(g.in) + 127) / 128);
    p.tiles = (g.N + (gated ? 63 : 127)) / (gated ? 64 : 128) * p.mtiles;
    // The largest split whose clusters all run at once (a cluster that has to wait for a free place doubles the
    // time: N = 2048, K = 5504 took 13.7 us with the sixteenth cluster of eight left over, on one CTA per SM);
    // every CTA keeps at least two blocks of the contraction.
    p.split = kMaxSplit;
    while (p.split > 1 && (p.split > kb / 2 || clusters_at_once(p.split) < p.tiles)) --p.split;
    const size_t stage = kWBytes + p.nt * 128, red = (size_t)(p.nt + kMaxSplit) * 512;
    p.stages = (int)((kRoom - 1024 - red) / stage);
    const int need = (kb + p.split - 1) / p.split;
    p.stages = p.stages > kMaxStages ? kMaxStages : p.stages;
    p.stages = p.stages > need ? need : p.stages;
    p.smem = 1024 + p.stages * stage + red;
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
    auto four = [](const void *q, int64_t ld) { return ((uintptr_t)q & (4 * sizeof(TO) - 1)) == 0 && ld % 4 == 0; };
    p.vec_out = four(g.out, g.ldo) && (EPI != kEpiGatedBwd || (g.N % 4 == 0 && four(g.out2, g.ldo2)));
    p.vec_extra = four(g.extra, g.ld_extra);
    auto *kern = gemm_small_kernel<FP8, WT, EPI, NT, TO, false>;
    static std::atomic<uint64_t> seen;
    bool first = first_on_device(seen);
    if constexpr (!FP8 && !WT && EPI == kEpiLinear && NT == 16 && sizeof(TO) == 2) {
        if (withhold_loads()) {
            kern = gemm_small_kernel<FP8, WT, EPI, NT, TO, true>;
            first = true;
        }
    }
    if (first) {
        const cudaError_t e = allow_two(kern);
        if (e != cudaSuccess) return e;
        if (!withhold_loads()) done_on_device(seen);
    }
    return launch_overlapped(kern, (unsigned)(pl.tiles * pl.split), 1, kThreads, pl.smem, pl.split, st, maps, p);
}

template <bool FP8, bool WT, int EPI, typename TO>
cudaError_t pick(const GemmArgs &g, cudaStream_t st)
{
    const SmallPlan p = plan_small(g, (Epi)EPI);
    switch (p.nt) {
    case 16: return go<FP8, WT, EPI, 16, TO>(g, p, st);
    case 32: return go<FP8, WT, EPI, 32, TO>(g, p, st);
    default: return go<FP8, WT, EPI, 64, TO>(g, p, st);
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
