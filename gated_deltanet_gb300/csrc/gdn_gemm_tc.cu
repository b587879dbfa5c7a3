// Products of bf16 and e4m3 operands on the tensor cores, with the epilogues of the decoder-block
// operators.
//
// A pair of CTAs (a cluster of two, one per SM) owns a 256 x BN tile of accumulators: each CTA holds
// 128 rows of A and half of B's rows in its shared memory and one M = 256 tcgen05.mma reads both halves,
// so that every byte staged serves twice the products of a single CTA's tile (a single CTA's 128 x 256
// instruction with both operands in shared memory takes 161 cycles here for 128 cycles of work; the pair's
// reads half of B per SM).  Roles per CTA: eight epilogue warps, one thread that issues the TMA loads, one
// that issues the products (in the pair's first CTA only).  The accumulators are double-buffered in tensor
// memory, so a tile's epilogue runs under the next tile's products; a persistent grid walks the tiles in
// groups of eight row tiles, which keeps one group's operands in L2.
//
// Operands are loaded as 128-byte-swizzled boxes, either along k (K-major) or, for the products of the
// backward passes, along m / n as they lie in memory (MN-major): nothing is transposed.
#include <cstring>
#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>

#include "gdn_layer.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

__device__ unsigned g_tc_status;  // kStatusTimeout once a wait ran out
constexpr unsigned long long kLimitNs = 2000000000ull;

constexpr int kEpiWarps = 8, kThreads = 32 * (kEpiWarps + 2);
constexpr int kABytes = 128 * 128;       // a CTA's rows of A, 128 bytes of k (or 64 k rows of 2 x 64 m)
constexpr int kStageBuf = 32 * 128;      // one epilogue box: 32 rows of 128 bytes

// Shared memory of a CTA.  BN = 128: two 128-byte-wide blocks of k per stage, so that eight products and not four
// follow each wait (16384 x 2048 x 2048: 112 -> 87 us; with BN = 256, whose products take twice as long, it is flat).
// BOXES: epilogue boxes per warp; with two, the second box of extra values loads, and the first box of results
// leaves, beside the arithmetic.
template <int BN, int BOXES> struct Geo {
    static constexpr int kAtoms = BN == 256 ? 1 : 2;
    static constexpr int kB = BN / 2 * 128;
    static constexpr int kAtom = kABytes + kB;  // 128 bytes of k
    static constexpr int kStage = kAtoms * kAtom;
    static constexpr int kBoxBytes = kEpiWarps * BOXES * kStageBuf;
    static constexpr int kBars(int stages) { return 2 * stages + 4 + 2 * kEpiWarps; }
    static constexpr int kStages = (227 * 1024 - 1024 - kBoxBytes - 512) / kStage;
    static constexpr int kTmem = 2 * BN;  // two accumulators
    static constexpr int kSmem = 1024 + kStages * kStage + kBoxBytes + kBars(kStages) * 8 + 16;
};
static_assert(Geo<256, 1>::kStages == 6 && Geo<256, 2>::kStages == 5 && Geo<128, 1>::kStages == 4, "stages");
static_assert(Geo<256, 1>::kSmem <= 227 * 1024 && Geo<256, 2>::kSmem <= 227 * 1024 && Geo<128, 1>::kSmem <= 227 * 1024,
              "shared memory budget");

struct TcMaps {
    CUtensorMap a, b, out, up, extra;
};
struct TcParams {
    int64_t M, N;            // output rows; output columns (gated: F)
    int kblocks;             // stages of k
    int mt, nt;              // tiles of 256 rows, of BN accumulator columns
    int tma_out, tma_extra;                   // boxes of them by TMA (else element by element)
    int vec_w, vec_up, vec_bias, vec_out2;    // 16-byte accesses of them
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

// ------------------------------------------------------------------ pair primitives
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
// the address, in the first CTA of the pair, of a barrier at the same place
__device__ __forceinline__ uint32_t leader_addr(const void *p)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
__device__ __forceinline__ void remote_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// a wait for arrivals of both CTAs
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint64_t t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        const uint64_t t = globaltimer();
        if (!t0) t0 = t;
        if (t - t0 > kLimitNs) {
            atomicOr(&g_tc_status, kStatusTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_cta(uint64_t *bar, uint32_t parity)
{
    return mbar_wait(bar, parity, &g_tc_status, kStatusTimeout, kLimitNs);
}
__device__ __forceinline__ void pair_load(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
template <bool FP8>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if (FP8)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc));
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// arrives on the barrier at the same place in both CTAs once every product issued so far is done
__device__ __forceinline__ void pair_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// ------------------------------------------------------------------ epilogue boxes
template <typename TO> struct Box {
    static constexpr int kCols = 128 / (int)sizeof(TO);
    // byte offset of (row, column) in a 128-byte-swizzled box
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        const int b = c * (int)sizeof(TO);
        return (uint32_t)(r * 128 + ((((b >> 4) ^ (r & 7)) << 4) | (b & 15)));
    }
};
// Rows that TMA cannot address (a pitch or a base off 16 bytes): element by element, 32 columns at a time
template <typename TO>
__device__ __forceinline__ void box_in(uint8_t *buf, const void *src, int64_t ld, int64_t row0, int64_t col0, int64_t M, int64_t N, int lane)
{
    for (int r = 0; r < 32; ++r)
        for (int c = lane; c < Box<TO>::kCols; c += 32) {
            const bool in = row0 + r < M && col0 + c < N;
            *(TO *)(buf + Box<TO>::at(r, c)) = in ? ((const TO *)src)[(row0 + r) * ld + col0 + c] : from_f<TO>(0.f);
        }
    __syncwarp();
}
template <typename TO>
__device__ __forceinline__ void box_out(const uint8_t *buf, void *dst, int64_t ld, int64_t row0, int64_t col0, int64_t M, int64_t N, int lane)
{
    __syncwarp();
    for (int r = 0; r < 32; ++r)
        for (int c = lane; c < Box<TO>::kCols; c += 32)
            if (row0 + r < M && col0 + c < N) ((TO *)dst)[(row0 + r) * ld + col0 + c] = *(const TO *)(buf + Box<TO>::at(r, c));
    __syncwarp();
}
__device__ __forceinline__ float lo_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// 16 columns of a box row (group g of them), 16 bytes at a time
__device__ __forceinline__ void row_get(const uint8_t *buf, int r, int g, float *v, __nv_bfloat16)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint4 u = *(const uint4 *)(buf + r * 128 + (((2 * g + j) ^ (r & 7)) << 4));
        v[8 * j] = lo_bf16(u.x); v[8 * j + 1] = hi_bf16(u.x);
        v[8 * j + 2] = lo_bf16(u.y); v[8 * j + 3] = hi_bf16(u.y);
        v[8 * j + 4] = lo_bf16(u.z); v[8 * j + 5] = hi_bf16(u.z);
        v[8 * j + 6] = lo_bf16(u.w); v[8 * j + 7] = hi_bf16(u.w);
    }
}
__device__ __forceinline__ void row_get(const uint8_t *buf, int r, int g, float *v, float)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) *(float4 *)(v + 4 * j) = *(const float4 *)(buf + r * 128 + (((4 * g + j) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void row_put(uint8_t *buf, int r, int g, const float *v, __nv_bfloat16)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) *(uint4 *)(buf + r * 128 + (((2 * g + j) ^ (r & 7)) << 4)) = pack8(v + 8 * j);
}
__device__ __forceinline__ void row_put(uint8_t *buf, int r, int g, const float *v, float)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) *(float4 *)(buf + r * 128 + (((4 * g + j) ^ (r & 7)) << 4)) = *(const float4 *)(v + 4 * j);
}
// 16 values of a row of global memory from column c on (an output without a box of its own)
__device__ __forceinline__ void line_out(__nv_bfloat16 *dst, int64_t c, int64_t N, int vec, const float *v)
{
    if (vec && c + 16 <= N) {
        *(uint4 *)dst = pack8(v);
        *(uint4 *)(dst + 8) = pack8(v + 8);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c + j < N) dst[j] = __float2bfloat16_rn(v[j]);
    }
}
// 16 per-column values (the same for every row): by 16-byte loads where `vec` and all exist; 0 past the end
__device__ __forceinline__ void columns(const float *src, int64_t c, int64_t N, int vec, float *v)
{
    if (vec && c + 16 <= N) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *(float4 *)(v + 4 * j) = __ldg((const float4 *)(src + c) + j);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = c + j < N ? __ldg(src + c + j) : 0.f;
    }
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}
// keeps the uses of freshly loaded accumulators behind the wait for them
__device__ __forceinline__ void pin16(float *v)
{
#pragma unroll
    for (int j = 0; j < 16; ++j) asm volatile("" : "+f"(v[j]));
}

// Sum over the warp's 32 rows of each of 16 columns (one per register): halves of the columns change hands at every
// step, 16 shuffles in all; lanes 2 c and 2 c + 1 end with the sum of column c.
__device__ __forceinline__ float column_sums(float *v, int lane)
{
#pragma unroll
    for (int w = 8; w; w >>= 1) {
        const bool high = lane & (2 * w);
#pragma unroll
        for (int j = 0; j < w; ++j) {
            const float give = high ? v[j] : v[j + w], keep = high ? v[j + w] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * w);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

constexpr int kLinearBoxes = 1;
template <int N> struct Count { static constexpr int value = N; };

// LAYOUT 0: A and B K-major; 1: B MN-major; 2: both MN-major
template <bool FP8, int LAYOUT, int EPI, int BN, int BOXES, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_tc_kernel(const __grid_constant__ TcMaps maps, const TcParams p)
{
    using G = Geo<BN, BOXES>;
    constexpr int kAtoms = G::kAtoms;
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    constexpr bool kExtra = EPI != kEpiGated;
    constexpr bool kPrecise = sizeof(TO) == 4;
    constexpr int kOutN = kGated ? BN / 2 : BN;  // output columns of a tile
    static_assert(!kGated || BN == 256, "a gated tile is 128 gate and 128 up columns");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *boxes = sm + G::kStages * G::kStage;
    uint64_t *full = (uint64_t *)(boxes + G::kBoxBytes);
    uint64_t *empty = full + G::kStages, *tfull = empty + G::kStages, *tempty = tfull + 2, *ebar = tempty + 2;
    uint32_t *tslot = (uint32_t *)(ebar + 2 * kEpiWarps);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int tiles = p.mt * p.nt;

    if (tid == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * kEpiWarps);
        }
        for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(&ebar[i], 1);
        fence_mbar_init();
    }
    if (warp == kEpiWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(G::kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    // tile -> (row tile, column tile): groups of eight row tiles, column tiles within a group one after another
    auto place = [&](int t, int &m, int &n) {
        const int per = 8 * p.nt, g = t / per, w = t - g * per, rows = min(8, p.mt - 8 * g);
        m = 8 * g + w % rows;
        n = w / rows;
    };
    bool ok = true;

    if (warp == kEpiWarps) {
        // ---------------------------------------------------------------- loads
        uint32_t s = 0, ph = 1;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int mi, ni;
            place(t, mi, ni);
            const int m0 = mi * 256 + (int)rank * 128;
            const int n0 = kGated ? (rank ? (int)p.N : 0) + ni * kOutN : ni * BN + (int)rank * (BN / 2);
            for (int kb = 0; kb < p.kblocks; ++kb) {
                if (!(ok = __all_sync(0xffffffffu, wait_cta(&empty[s], ph)))) break;
                if (elect_one_sync()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * G::kStage);
                    const uint32_t bar = leader_addr(&full[s]);
#pragma unroll
                    for (int at = 0; at < kAtoms; ++at) {
                        uint8_t *sa = sm + s * G::kStage + at * G::kAtom, *sb = sa + kABytes;
                        const int k0 = (kb * kAtoms + at) * (FP8 ? 128 : 64);  // (past the end: zeros)
                        if (LAYOUT == 2) {
                            pair_load(sa, &maps.a, m0, k0, bar);
                            pair_load(sa + 8192, &maps.a, m0 + 64, k0, bar);
                        } else {
                            pair_load(sa, &maps.a, k0, m0, bar);
                        }
                        if (LAYOUT >= 1) {
#pragma unroll
                            for (int j = 0; j < BN / 128; ++j) pair_load(sb + 8192 * j, &maps.b, n0 + 64 * j, k0, bar);
                        } else {
                            pair_load(sb, &maps.b, k0, n0, bar);
                        }
                    }
                }
                __syncwarp();
                if (++s == G::kStages) { s = 0; ph ^= 1; }
            }
        }
        // the last products have read every stage before the CTAs of the pair may leave
        for (int i = 0; i < G::kStages && ok; ++i) {
            ok = __all_sync(0xffffffffu, wait_cta(&empty[s], ph));
            if (++s == G::kStages) { s = 0; ph ^= 1; }
        }
    } else if (warp == kEpiWarps + 1) {
        // ---------------------------------------------------------------- products
        if (rank == 0) {
            // (the whole warp follows the loop, so that its bookkeeping stays uniform; one elected lane issues)
            constexpr uint32_t id = FP8 ? (1u << 4) | ((uint32_t)(BN >> 3) << 17) | (16u << 24)
                                        : idesc_bf16_f32(256, BN, LAYOUT == 2, LAYOUT >= 1);
            constexpr uint32_t sa_step = LAYOUT == 2 ? 128 : 2, sb_step = LAYOUT >= 1 ? 128 : 2;
            const uint32_t base = smem_u32(sm);
            const uint64_t da0 = sdesc_sw128(base, LAYOUT == 2 ? 8192 : 16, 1024);
            const uint64_t db0 = sdesc_sw128(base + kABytes, LAYOUT >= 1 ? 8192 : 16, 1024);
            uint32_t s = 0, ph = 0, n = 0;
            for (int t = pair; t < tiles && ok; t += pairs, ++n) {
                const uint32_t acc = n & 1;
                if (!(ok = __all_sync(0xffffffffu, wait_cluster(&tempty[acc], ((n >> 1) & 1) ^ 1)))) break;
                tc_fence_after();
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!(ok = __all_sync(0xffffffffu, wait_cluster(&full[s], ph)))) break;
                    tc_fence_after();
                    const uint64_t da = da0 + s * (G::kStage >> 4), db = db0 + s * (G::kStage >> 4);
                    uint64_t *const rel = &empty[s];
                    if (++s == G::kStages) { s = 0; ph ^= 1; }
                    if (elect_one_sync()) {
#pragma unroll
                        for (int j = 0; j < 4 * kAtoms; ++j)
                            pair_mma<FP8>(tmem + acc * BN, da + (j >> 2) * (G::kAtom >> 4) + (j & 3) * sa_step,
                                          db + (j >> 2) * (G::kAtom >> 4) + (j & 3) * sb_step, id, (kb | j) != 0);
                        pair_commit(rel);
                        if (kb + 1 == p.kblocks) pair_commit(&tfull[acc]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        constexpr int kCols = Box<TO>::kCols;
        const int q = warp & 3, half = warp >> 2;
        constexpr int kChunks = kOutN / kCols / 2;  // boxes' worth of columns of this warp
        uint8_t *const boxes0 = boxes + warp * BOXES * kStageBuf;
        uint64_t *const eb = ebar + 2 * warp;
        uint32_t n = 0, eph = 0;  // (a phase bit per box)
        // every box but the `pending` latest is free again, for copies by either path
        auto boxes_free = [&](auto pending) {
            fence_proxy_async();
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(decltype(pending)::value) : "memory");
            __syncwarp();
        };
        for (int t = pair; t < tiles && ok; t += pairs, ++n) {
            int mi, ni;
            place(t, mi, ni);
            const int64_t row0 = (int64_t)mi * 256 + rank * 128 + q * 32, row = row0 + lane;
            const uint32_t acc = n & 1;
            const uint32_t tl = tmem + acc * BN + ((uint32_t)(q * 32) << 16);
            auto col_of = [&](int c) { return (int64_t)ni * kOutN + (half * kChunks + c) * kCols; };
            auto live = [&](int c) { return col_of(c) < p.N && row0 < p.M; };
            auto box_of = [&](int c) { return boxes0 + (c % BOXES) * kStageBuf; };
            // extra values (residual, dy, dh) of chunk c into its box
            auto fetch = [&](int c) {
                if (!kExtra || !p.extra || !live(c)) return;
                if (p.tma_extra) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&eb[c % BOXES], kStageBuf);
                        tma_load_2d(box_of(c), &maps.extra, (int)col_of(c), (int)row0, &eb[c % BOXES]);
                    }
                } else {
                    box_in<TO>(box_of(c), p.extra, p.ld_extra, row0, col_of(c), p.M, p.N, lane);
                }
            };
            // a finished box to its place: columns col0 ..., of an output with its own map
            auto store = [&](uint8_t *buf, const CUtensorMap *map, int tma, void *dst, int64_t ld, int64_t col0) {
                if (tma) {
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(map, buf, (int)col0, (int)row0);
                        tma_store_commit();
                    }
                } else {
                    box_out<TO>(buf, dst, ld, row0, col0, p.M, p.N, lane);
                }
            };
            boxes_free(Count<0>());
            for (int c = 0; c < BOXES && c < kChunks; ++c) fetch(c);  // under the tile's products
            const float sx = FP8 && p.x_scale && row < p.M ? p.x_scale[row] : 1.f;
            ok = wait_cluster(&tfull[acc], (n >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                const int64_t col0 = col_of(c);
                uint8_t *const buf = box_of(c);
                if (c >= BOXES) {
                    boxes_free(Count<BOXES - 1>());
                    fetch(c);
                }
                if (!live(c)) continue;
                if (kExtra && p.extra && p.tma_extra) {
                    ok = wait_cta(&eb[c % BOXES], (eph >> (c % BOXES)) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    eph ^= 1u << (c % BOXES);
                }
                // 16 columns at a time, in a loop that stays rolled: unrolled over a box, an activation's code left the
                // instruction cache at every pass (erf's gradient took 19 K cycles a tile, 2.5 times its arithmetic).
                // The next accumulators load under this group's arithmetic.
                constexpr int kGroups = kCols / 16;
                const int tc = (half * kChunks + c) * kCols;  // accumulator column
                float nv[16], nu[kGated ? 16 : 1];
                tmem_ld16(tl + tc, nv);
                if constexpr (kGated) tmem_ld16(tl + BN / 2 + tc, nu);
#pragma unroll 1
                for (int g = 0; g < kGroups; ++g) {
                    const int64_t cg = col0 + 16 * g;
                    float v[16], u[16], e[16];
                    if (kExtra && p.extra) row_get(buf, lane, g, e, TO());
                    tmem_ld_wait();
                    pin16(nv);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = nv[j];
                    if constexpr (kGated) {
                        pin16(nu);
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = nu[j];
                    }
                    if (g + 1 < kGroups) {
                        tmem_ld16(tl + tc + 16 * (g + 1), nv);
                        if constexpr (kGated) tmem_ld16(tl + BN / 2 + tc + 16 * (g + 1), nu);
                    }
                    if (FP8 && p.w_scale) {
                        float ws[16];
                        columns(p.w_scale, cg, p.N, p.vec_w, ws);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] *= sx * ws[j];
                        if constexpr (kGated) {
                            columns(p.w_scale + p.N, cg, p.N, p.vec_up, ws);
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] *= sx * ws[j];
                        }
                    }
                    if (!kGated && p.bias) {
                        float bs[16];
                        columns(p.bias, cg, p.N, p.vec_bias, bs);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] += bs[j];
                    }
                    if constexpr (EPI == kEpiLinear) {
                        if (p.act != GDN_ACT_NONE)
                            with_act(p.act, [&](auto tag) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = act_value<kPrecise, decltype(tag)::value>(v[j]);
                            });
                        if (p.extra) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] += e[j];
                        }
                    } else if constexpr (EPI == kEpiDact) {
                        const bool in = row < p.M;
                        with_act(p.act, [&](auto tag) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float a, d;
                                act_both<kPrecise, decltype(tag)::value>(v[j], a, d);
                                v[j] = in ? e[j] * d : 0.f;
                            }
                        });
                    } else if constexpr (EPI == kEpiGated) {
                        with_act(p.act, [&](auto tag) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = act_value<kPrecise, decltype(tag)::value>(v[j]) * u[j];
                        });
                    } else {
                        float h[16];
                        with_act(p.act, [&](auto tag) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float a, d;
                                act_both<kPrecise, decltype(tag)::value>(v[j], a, d);
                                h[j] = a * u[j];
                                v[j] = e[j] * u[j] * d;
                                u[j] = e[j] * a;
                            }
                        });
                        row_put(boxes0 + kStageBuf, lane, g, u, TO());  // (one chunk a tile: the second box is free)
                        if (p.out2 && row < p.M) line_out((__nv_bfloat16 *)p.out2 + row * p.ldo2 + cg, cg, p.N, p.vec_out2, h);
                    }
                    row_put(buf, lane, g, v, TO());
                    if (EPI == kEpiDact && p.colpart) {
                        const float sum = column_sums(v, lane);
                        const int64_t cc = cg + (lane >> 1);
                        if (!(lane & 1) && cc < p.N) p.colpart[(row0 >> 5) * p.N + cc] = sum;
                    }
                }
                store(buf, &maps.out, p.tma_out, p.out, p.ldo, col0);
                if constexpr (EPI == kEpiGatedBwd) {
                    static_assert(kChunks == 1 && BOXES == 2, "boxes of the two halves");
                    store(boxes0 + kStageBuf, &maps.up, p.tma_out, (TO *)p.out + p.N, p.ldo, col0);
                }
            }
            if (!ok) break;
            // the accumulators are read: hand them back to the issuer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive(leader_addr(&tempty[acc]));
        }
        if (lane == 0) tma_store_wait0();
    }
    if (!ok) {
        // a wait ran out: give whatever is still in flight a millisecond to land before the memory is let go
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000) {}
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == kEpiWarps + 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::kTmem));
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)p;
    });
    return fn;
}

size_t esz(gdn_dtype t) { return t == GDN_F32 ? 4 : t == GDN_BF16 ? 2 : 1; }

template <bool FP8, int LAYOUT, int EPI, int BN, int BOXES, typename TO>
cudaError_t go(const GemmArgs &g, cudaStream_t st)
{
    constexpr bool gated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    TcMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const int64_t brows = gated ? 2 * g.N : g.N;
    const bool a_ok = LAYOUT == 2 ? make_operand_map(&maps.a, g.in, g.a, g.M, g.K, g.lda, 64) : make_operand_map(&maps.a, g.in, g.a, g.K, g.M, g.lda, 128);
    const bool b_ok = LAYOUT >= 1 ? make_operand_map(&maps.b, g.in, g.b, brows, g.K, g.ldb, 64) : make_operand_map(&maps.b, g.in, g.b, g.K, brows, g.ldb, BN / 2);
    if (!a_ok || !b_ok) return cudaErrorInvalidValue;
    TcParams p{};
    p.M = g.M; p.N = g.N;
    const int per = Geo<BN, BOXES>::kAtoms * (FP8 ? 128 : 64);
    p.kblocks = (int)((g.K + per - 1) / per);
    p.mt = (int)((g.M + 255) / 256);
    p.nt = (int)((g.N + (gated ? BN / 2 : BN) - 1) / (gated ? BN / 2 : BN));
    p.x_scale = g.x_scale; p.w_scale = g.w_scale; p.bias = g.bias; p.act = g.act;
    p.extra = g.extra; p.ld_extra = g.ld_extra;
    p.out = g.out; p.ldo = g.ldo; p.out2 = g.out2; p.ldo2 = g.ldo2;
    p.colpart = g.colpart;
    const size_t eo = sizeof(TO);
    p.tma_out = tma_ok(g.out, g.ldo, g.M, eo) && (EPI != kEpiGatedBwd || (g.N * eo) % 16 == 0);
    if (p.tma_out && !make_operand_map(&maps.out, g.out_dt, g.out, g.N, g.M, g.ldo, 32)) return cudaErrorInvalidValue;
    if (p.tma_out && EPI == kEpiGatedBwd && !make_operand_map(&maps.up, g.out_dt, (const TO *)g.out + g.N, g.N, g.M, g.ldo, 32))
        return cudaErrorInvalidValue;
    p.tma_extra = g.extra && tma_ok(g.extra, g.ld_extra, g.M, eo);
    if (p.tma_extra && !make_operand_map(&maps.extra, g.out_dt, g.extra, g.N, g.M, g.ld_extra, 32)) return cudaErrorInvalidValue;
    auto on16 = [](const void *q) { return ((uintptr_t)q & 15) == 0; };
    p.vec_w = on16(g.w_scale);
    p.vec_up = g.w_scale && on16(g.w_scale + g.N);
    p.vec_bias = on16(g.bias);
    p.vec_out2 = tma_ok(g.out2, g.ldo2, 2, eo);

    auto *kern = gemm_tc_kernel<FP8, LAYOUT, EPI, BN, BOXES, TO>;
    static std::atomic<uint64_t> seen;
    if (first_on_device(seen)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<BN, BOXES>::kSmem);
        if (e != cudaSuccess) return e;
        done_on_device(seen);
    }
    const int64_t tiles = (int64_t)p.mt * p.nt;
    const int pairs = (int)(tiles < device_sm_count() / 2 ? tiles : device_sm_count() / 2);
    kern<<<2 * pairs, kThreads, Geo<BN, BOXES>::kSmem, st>>>(maps, p);
    return cudaGetLastError();
}

template <bool FP8, int LAYOUT, int EPI, typename TO>
cudaError_t pick(const GemmArgs &g, cudaStream_t st)
{
    if constexpr (EPI == kEpiGated || EPI == kEpiGatedBwd) {
        return go<FP8, LAYOUT, EPI, 256, EPI == kEpiGatedBwd ? 2 : 1, TO>(g, st);
    } else {
        // Whole rounds of tiles over the pairs of SMs decide: a round of 128-column tiles takes 0.58 of one of 256
        // columns (6.2 and 10.7 us at K = 2048: its products re-read A), but fills a ragged last round better.
        const int64_t pairs = device_sm_count() / 2, mt = (g.M + 255) / 256;
        const auto rounds = [&](int bn) { return (mt * ((g.N + bn - 1) / bn) + pairs - 1) / pairs; };
        if (0.58 * rounds(128) < rounds(256)) return go<FP8, LAYOUT, EPI, 128, 1, TO>(g, st);
        return go<FP8, LAYOUT, EPI, 256, EPI == kEpiDact ? 2 : kLinearBoxes, TO>(g, st);
    }
}

// Few rows: the weights' reading is the cost, and the pair's tiles would be padding.  (A weight gradient's rows are
// the weight's, and its contraction the batch.)
bool use_small(const GemmArgs &g) { return !g.a_t && g.M <= 128; }

template <typename T>
__global__ void __launch_bounds__(256) repack_kernel(const T *src, int64_t ld, int64_t rows, int64_t cols, T *dst, int64_t pitch)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256) dst[r * pitch + c] = src[r * ld + c];
}

}  // namespace

bool make_operand_map(CUtensorMap *m, gdn_dtype t, const void *base, int64_t cols, int64_t rows, int64_t ld, int box_rows)
{
    const auto enc = encoder();
    if (!enc) return false;
    const size_t e = esz(t);
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {rows > 1 ? (cuuint64_t)ld * e : ((cuuint64_t)cols * e + 15) / 16 * 16};
    cuuint32_t box[2] = {(cuuint32_t)(128 / e), (cuuint32_t)box_rows}, es[2] = {1, 1};
    const CUtensorMapDataType dt = t == GDN_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : t == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return enc(m, dt, 2, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tma_ok(const void *p, int64_t ld, int64_t rows, size_t e)
{
    return ((uintptr_t)p & 15) == 0 && (rows <= 1 || (size_t)ld * e % 16 == 0);
}

cudaError_t launch_repack(const void *src, gdn_dtype t, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t pitch, cudaStream_t st)
{
    const unsigned grid = (unsigned)(rows < 4096 ? rows : 4096);
    if (t == GDN_BF16) repack_kernel<<<grid, 256, 0, st>>>((const uint16_t *)src, ld, rows, cols, (uint16_t *)dst, pitch);
    else repack_kernel<<<grid, 256, 0, st>>>((const uint8_t *)src, ld, rows, cols, (uint8_t *)dst, pitch);
    return cudaGetLastError();
}

int64_t gemm_colparts(const GemmArgs &g, Epi epi)
{
    return g.in != GDN_F32 && use_small(g) ? gemm_small_colparts(g, epi) : (g.M + 31) / 32;
}

cudaError_t launch_gemm_tc(const GemmArgs &g, Epi epi, cudaStream_t st)
{
    if (g.M <= 0 || g.N <= 0) return cudaSuccess;
    if (use_small(g)) return launch_gemm_small(g, epi, st);
    const bool f32 = g.out_dt == GDN_F32;
    if (g.in == GDN_E4M3) {
        if (epi == kEpiGated) return pick<true, 0, kEpiGated, __nv_bfloat16>(g, st);
        return f32 ? pick<true, 0, kEpiLinear, float>(g, st) : pick<true, 0, kEpiLinear, __nv_bfloat16>(g, st);
    }
    switch (epi) {
    case kEpiGated: return pick<false, 0, kEpiGated, __nv_bfloat16>(g, st);
    case kEpiGatedBwd: return pick<false, 0, kEpiGatedBwd, __nv_bfloat16>(g, st);
    case kEpiDact: return pick<false, 0, kEpiDact, __nv_bfloat16>(g, st);
    default: break;
    }
    if (g.a_t) return pick<false, 2, kEpiLinear, __nv_bfloat16>(g, st);
    if (g.b_t) return pick<false, 1, kEpiLinear, __nv_bfloat16>(g, st);
    return f32 ? pick<false, 0, kEpiLinear, float>(g, st) : pick<false, 0, kEpiLinear, __nv_bfloat16>(g, st);
}

gdn_status read_tc_status(cudaStream_t st)
{
    unsigned word = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, g_tc_status, sizeof(word), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_tc_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return word & kStatusTimeout ? GDN_ERR_TIMEOUT : read_small_status(st);
}

}  // namespace gdn
