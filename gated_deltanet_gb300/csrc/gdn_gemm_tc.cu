// Products of bf16, e4m3 and (as three bf16 planes) fp32 operands on the tensor cores, with the epilogues of the
// decoder-block operators.
//
// A pair of CTAs (a cluster of two, one per SM) owns a 256 x BN tile of accumulators: each CTA holds
// 128 rows of A and half of B's rows in its shared memory and one M = 256 tcgen05.mma reads both halves,
// so that every byte staged serves twice the products of a single CTA's tile (a single CTA's 128 x 256
// instruction with both operands in shared memory takes 161 cycles here for 128 cycles of work; the pair's
// reads half of B per SM).  Roles per CTA: eight epilogue warps (each half of the columns of 32 rows), one
// that issues the TMA loads, one that issues the products (in the pair's first CTA only).  The accumulators are double-buffered in tensor
// memory, so a tile's epilogue runs under the next tile's products; a persistent grid walks the tiles in
// groups of eight row tiles, which keeps one group's operands in L2.
//
// Operands are loaded as 128-byte-swizzled boxes, either along k (K-major) or, for the products of the
// backward passes, along m / n as they lie in memory (MN-major): nothing is transposed.
//
// Bound: the tensor pipe (16384 x 2048 x 2048 in bf16: 72.6 us, 1.89 PFLOP/s, the pipe 80 % active; gated 8191 x 2048 x
// 5504: 89 %; 4096 x 2048 x 2048 in fp32: 158 us, 217 TFLOP/s); with short contractions (K = 256) the epilogue.
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

constexpr int kEpiWarps = 8, kThreads = 32 * (kEpiWarps + 2);
constexpr int kABytes = 128 * 128;       // a CTA's rows of A, 128 bytes of k (or 64 k rows of 2 x 64 m)

// What the operands are: bf16, e4m3, or fp32 as three bf16 planes each (x = x0 + x1 + x2, 8 bits of the significand
// apiece; launch_split).  Of the nine products of planes the six that reach fp32's last bits are taken: x0 w0, and x0 w1,
// x1 w0, x1 w1, x0 w2, x2 w0, which are 2^-8 of it and less.  The tensor cores truncate their running sums (2e-6 off after
// 128 additions, five times fp32's own rounding), so x0 w0 is summed over kChain stages at a time only and the epilogue
// adds those partial sums in registers; the others have an accumulator of their own, whose truncation is 2^-8 as large.
enum Kind : int { kBf16 = 0, kE4m3 = 1, kF32 = 2 };
constexpr int kChain = 2;
constexpr int kMaxSplit = 4;

// Shared memory of a CTA: operands, each epilogue warp's column vectors (scales and bias of its half of a tile; the
// tensors of the epilogue go between registers and global memory) and its 32 x 16 patch for rows off 16 bytes.  BN = 128: two
// 128-byte-wide blocks of k per stage, so that eight products and not four follow each wait (16384 x 2048 x 2048:
// 112 -> 87 us; with BN = 256, whose products take twice as long, it is flat).
template <int KIND, int BN, bool SPLIT> struct Geo {
    static constexpr int kAtoms = KIND == kF32 ? 3 : BN == 256 ? 1 : 2;  // (fp32: the planes of one block of k)
    static constexpr int kPerStage = KIND == kF32 ? 1 : kAtoms;          // blocks of k
    static constexpr int kB = BN / 2 * 128;
    static constexpr int kAtom = kABytes + kB;  // 128 bytes of k
    static constexpr int kStage = kAtoms * kAtom;
    static constexpr int kColBytes = kEpiWarps * (2 * 128 + 32 * 17) * 4;
    static constexpr int kParts = SPLIT ? kEpiWarps * 3 * 16 * 128 : 0;  // the other CTAs' sums of a split contraction
    static constexpr int kStages = (227 * 1024 - 1024 - kColBytes - kParts - 256) / kStage;
    static_assert(kStages == (KIND == kF32 ? 2 : BN == 256 ? 6 : SPLIT ? 3 : 4) && (KIND != kF32 || BN == 128), "stages");
    static constexpr int kBars = 2 * kStages + 4;
    static constexpr int kTmem = (KIND == kF32 ? 4 : 2) * BN;  // two accumulators (fp32: and two for the small products)
    static constexpr int kSmem = 1024 + kStages * kStage + kColBytes + kParts + kBars * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

struct TcMaps {
    CUtensorMap a[3], b[3];  // (planes; the first alone unless fp32)
};
struct TcParams {
    int64_t M, N;            // output rows; output columns (gated: F)
    int kblocks;             // stages of k
    int mt, nt;              // tiles of 256 rows, of BN accumulator columns
    int split;               // pairs that share a tile's contraction (SPLIT: 2 or 4)
    int vec_extra, vec_out, vec_out2;  // what their rows allow: accesses of 32 bytes (2), of 16 (1) or of elements
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
// the address, in CTA `cta` of the cluster, of what is at p here
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t cta)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(cta));
    return r;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Relaxed: it hands over tensor memory and nothing else.  The warp's reads of the accumulators are complete (tcgen05.wait::ld)
// and ordered before the arrival by tcgen05.fence::before_thread_sync (for the whole warp: __syncwarp, then one lane arrives);
// the issuer's tcgen05.fence::after_thread_sync, behind the wait that saw the arrival, orders its products after it.  Only tcgen05
// instructions reach tensor memory, and those two fences are what orders them between threads that meet in any way, so no
// release of ordinary memory is needed: column vectors and patch stay the warp's own.  A release would wait for the
// epilogue's global stores, 1400 cycles a tile.
__device__ __forceinline__ void remote_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// a wait for arrivals of both CTAs
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
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
        if (t - t0 > limit_ns) {
            atomicOr(&g_tc_status, kStatusTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_cta(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    return mbar_wait(bar, parity, &g_tc_status, kStatusTimeout, limit_ns);
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
// arrives on the barrier at the same place in both CTAs of the pair from `leader` on once every product issued so far is done
__device__ __forceinline__ void pair_commit(uint64_t *bar, uint32_t leader)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)(3u << leader))
        : "memory");
}

// ------------------------------------------------------------------ epilogue rows
// A thread has 16 columns of its row at a time: 32 (fp32: 64) bytes, whole sectors of memory, so they go straight
// between registers and global memory.  (Boxes in shared memory with TMA stores cost a pipeline stage or two, waits
// for their reuse, and were slower by 2 to 8 %.)
// `vec`: 2 where every row allows 32-byte accesses, 1 where it allows 16-byte ones, 0 for single elements.
__device__ __forceinline__ void load32(const void *p, uint32_t *lo, uint32_t *hi)
{
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(lo[0]), "=r"(lo[1]), "=r"(lo[2]), "=r"(lo[3]), "=r"(hi[0]), "=r"(hi[1]), "=r"(hi[2]), "=r"(hi[3])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store32(void *p, const uint4 &a, const uint4 &b)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x),
                 "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
template <typename TO> struct Line;
template <> struct Line<__nv_bfloat16> {
    uint4 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int vec)
    {
        if (vec == 2) {
            load32(p, &a.x, &b.x);
        } else {
            a = *(const uint4 *)p;
            b = *((const uint4 *)p + 1);
        }
    }
    __device__ __forceinline__ void set(int j, __nv_bfloat16 v)  // (j a constant)
    {
        uint32_t &w = j < 2 ? a.x : j < 4 ? a.y : j < 6 ? a.z : j < 8 ? a.w : j < 10 ? b.x : j < 12 ? b.y : j < 14 ? b.z : b.w;
        const uint32_t u = __bfloat16_as_ushort(v);
        w = j & 1 ? (w & 0xffffu) | (u << 16) : (w & 0xffff0000u) | u;
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *v) const
    {
        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
};
template <> struct Line<float> {
    float v_[16];
    __device__ __forceinline__ void load(const float *p, int)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) *(float4 *)(v_ + 4 * j) = *((const float4 *)p + j);
    }
    __device__ __forceinline__ void set(int j, float v) { v_[j] = v; }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int j = 0; j < 16; ++j) v_[j] = 0.f;
    }
    __device__ __forceinline__ void get(float *v) const
    {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = v_[j];
    }
};
// `p`: column c of this lane's row, of the 32 rows from row0 on; columns from N on and rows from M on read as zero and
// are not written.  A last group that ends before its 16 columns, and rows off 16 bytes (of small gated outputs,
// and the second half of a gated gradient's rows of odd width; other such tensors come by copies), pass through the warp's patch, so that half a warp
// reads or writes the 16 columns of a row together (lane by lane, every element was a sector of its own: 117 us for
// 8071 x 955 outputs with a residual against 81).
constexpr int kPatch = 17;  // floats per row of the patch: lanes that read down a column meet no bank twice
// (out of line: the fast path's loop has to stay small)
__device__ __noinline__ void patch_turn(float *v, int lane, float *patch)  // 16 values per lane: by rows of 16 -> by lanes
{
#pragma unroll
    for (int i = 0; i < 16; ++i) patch[(2 * i + (lane >> 4)) * kPatch + (lane & 15)] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = patch[lane * kPatch + i];
    __syncwarp();
}
template <typename TO>
__device__ __noinline__ void patch_out(const float *v, TO *first, int64_t ld, int rows, int cols, int lane, float *patch)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) patch[lane * kPatch + i] = v[i];
    __syncwarp();
    const int j = lane & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        if (r < rows && j < cols) first[r * ld + j] = from_f<TO>(patch[r * kPatch + j]);
    }
    __syncwarp();
}
template <typename TO>
__device__ __forceinline__ void line_in(Line<TO> &l, const TO *p, int64_t ld, int64_t row0, int lane, int64_t M, int64_t c, int64_t N, int vec)
{
    l.zero();
    if (vec && c + 16 <= N) {
        if (row0 + lane < M) l.load(p, vec);
        return;
    }
    const TO *first = p - lane * ld + (lane & 15);  // row0's; turned to this lane's row when it is used
    const bool col = c + (lane & 15) < N;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        if (col && row0 + r < M) l.set(i, first[r * ld]);
    }
}
template <typename TO>
__device__ __forceinline__ void line_get(const Line<TO> &l, float *v, int lane, int64_t c, int64_t N, int vec, float *patch)
{
    l.get(v);
    if (!(vec && c + 16 <= N)) {
        float w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = v[j];
        patch_turn(w, lane, patch);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = w[j];
    }
}
__device__ __forceinline__ void line_put(__nv_bfloat16 *p, const float *v, int vec)
{
    const uint4 a = pack8(v), b = pack8(v + 8);
    if (vec == 2) {
        store32(p, a, b);
    } else {
        *(uint4 *)p = a;
        *((uint4 *)p + 1) = b;
    }
}
__device__ __forceinline__ void line_put(float *p, const float *v, int)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) *((float4 *)p + j) = *(const float4 *)(v + 4 * j);
}
template <typename TO>
__device__ __forceinline__ void line_out(TO *p, int64_t ld, int64_t row0, int lane, int64_t M, int64_t c, int64_t N, int vec, const float *v,
                                         float *patch)
{
    if (vec && c + 16 <= N) {
        if (row0 + lane < M) line_put(p, v, vec);
        return;
    }
    float w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = v[j];
    patch_out<TO>(w, p - lane * ld, ld, (int)(M - row0 < 32 ? M - row0 : 32), (int)(N - c < 16 ? N - c : 16), lane, patch);
}
// Per-column values (scales, bias) of one half of a tile, `COUNT` from column c on: four (two) a lane, on their way in
// registers while the tile before is finished, then in the warp's shared memory; and 16 of them back.  0 past the end.
template <int COUNT> struct ColumnsAhead {
    float v[COUNT / 32];
    __device__ __forceinline__ void fetch(const float *src, int64_t c, int64_t N, int lane)
    {
#pragma unroll
        for (int i = 0; i < COUNT / 32; ++i) v[i] = c + 32 * i + lane < N ? __ldg(src + c + 32 * i + lane) : 0.f;
    }
    __device__ __forceinline__ void keep(float *dst, int lane) const
    {
#pragma unroll
        for (int i = 0; i < COUNT / 32; ++i) dst[32 * i + lane] = v[i];
    }
};
__device__ __forceinline__ void columns(const float *src, float *v)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) *(float4 *)(v + 4 * j) = *((const float4 *)src + j);
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

// LAYOUT 0: A and B K-major; 1: B MN-major; 2: both MN-major
//
// SPLIT: fewer tiles than pairs, so `split` pairs (a cluster) share a tile: each sums its part of the contraction, sends
// its sums of the columns that another pair finishes to that pair's shared memory (32 rows of a column to a store), and
// finishes its own share, the parts added in the order of the contraction.
//
// WITHHOLD: the load warps load nothing, so that every wait for operands runs out.
template <int KIND, int LAYOUT, int EPI, int BN, typename TO, bool SPLIT, bool WITHHOLD>
__global__ void __launch_bounds__(kThreads, 1)
gemm_tc_kernel(const __grid_constant__ TcMaps maps, const TcParams p)
{
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    constexpr bool kExtra = EPI != kEpiGated;
    constexpr bool kPrecise = sizeof(TO) == 4;
    constexpr int kOutN = kGated ? BN / 2 : BN;  // output columns of a tile
    constexpr bool FP8 = KIND == kE4m3, F32 = KIND == kF32;
    using G = Geo<KIND, BN, SPLIT>;
    constexpr int kAtoms = G::kAtoms;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *const cols = (float *)(sm + G::kStages * G::kStage);
    float *const parts = (float *)(sm + G::kStages * G::kStage + G::kColBytes);
    uint64_t *full = (uint64_t *)(sm + G::kStages * G::kStage + G::kColBytes + G::kParts);
    uint64_t *empty = full + G::kStages, *tfull = empty + G::kStages, *tempty = tfull + 2;
    uint32_t *tslot = (uint32_t *)(tempty + 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cluster_rank(), rank = crank & 1, leader = SPLIT ? crank & ~1u : 0;
    const int tiles = p.mt * p.nt;
    const int pairs = SPLIT ? tiles : gridDim.x >> 1, pair = SPLIT ? blockIdx.x / (2 * p.split) : blockIdx.x >> 1;
    const int share = SPLIT ? crank >> 1 : 0;  // its part of the contraction: blocks kb0 ..
    const int kb0 = SPLIT ? p.kblocks * share / p.split : 0;
    const int kblocks = SPLIT ? p.kblocks * (share + 1) / p.split - kb0 : p.kblocks;

    if (tid == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * kEpiWarps);
        }
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
    grid_release();
    grid_wait();

    // tile -> (row tile, column tile): groups of eight row tiles, column tiles within a group one after another
    auto place = [&](int t, int &m, int &n) {
        const int per = 8 * p.nt, g = t / per, w = t - g * per, rows = min(8, p.mt - 8 * g);
        m = 8 * g + w % rows;
        n = w / rows;
    };
    bool ok = true;
    constexpr uint64_t limit = WITHHOLD ? kTestWaitLimitNs : kWaitLimitNs;

    if (warp == kEpiWarps) {
        // ---------------------------------------------------------------- loads
        uint32_t s = 0, ph = 1;
        for (int t = WITHHOLD ? tiles : pair; t < tiles && ok; t += pairs) {
            int mi, ni;
            place(t, mi, ni);
            const int m0 = mi * 256 + (int)rank * 128;
            const int n0 = kGated ? (rank ? (int)p.N : 0) + ni * kOutN : ni * BN + (int)rank * (BN / 2);
            for (int kb = kb0; kb < kb0 + kblocks; ++kb) {
                if (!(ok = __all_sync(0xffffffffu, wait_cta(&empty[s], ph, limit)))) break;
                if (elect_one_sync()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * G::kStage);
                    const uint32_t bar = peer_addr(&full[s], leader);
#pragma unroll
                    for (int at = 0; at < kAtoms; ++at) {
                        uint8_t *sa = sm + s * G::kStage + at * G::kAtom, *sb = sa + kABytes;
                        const int k0 = (kb * G::kPerStage + (F32 ? 0 : at)) * (FP8 ? 128 : 64);  // (past the end: zeros)
                        const CUtensorMap *ma = &maps.a[F32 ? at : 0], *mb = &maps.b[F32 ? at : 0];
                        if (LAYOUT == 2) {
                            pair_load(sa, ma, m0, k0, bar);
                            pair_load(sa + 8192, ma, m0 + 64, k0, bar);
                        } else {
                            pair_load(sa, ma, k0, m0, bar);
                        }
                        if (LAYOUT >= 1) {
#pragma unroll
                            for (int j = 0; j < BN / 128; ++j) pair_load(sb + 8192 * j, mb, n0 + 64 * j, k0, bar);
                        } else {
                            pair_load(sb, mb, k0, n0, bar);
                        }
                    }
                }
                __syncwarp();
                if (++s == G::kStages) { s = 0; ph ^= 1; }
            }
        }
        // the last products have read every stage before the CTAs of the pair may leave
        for (int i = 0; i < G::kStages && ok; ++i) {
            ok = __all_sync(0xffffffffu, wait_cta(&empty[s], ph, limit));
            if (++s == G::kStages) { s = 0; ph ^= 1; }
        }
        if (SPLIT) cluster_sync();  // (the exchange of the parts)
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
            uint32_t s = 0, ph = 0, n = 0, parity = 0;
            for (int t = pair; t < tiles && ok; t += pairs, parity ^= 1) {
                const uint32_t small = tmem + (2 + parity) * BN;  // (fp32)
                for (int kb = 0, chain = 0; kb < kblocks; ++kb) {
                    const uint32_t acc = n & 1;
                    if (chain == 0) {
                        if (!(ok = __all_sync(0xffffffffu, wait_cluster(&tempty[acc], ((n >> 1) & 1) ^ 1, limit)))) break;
                        tc_fence_after();
                    }
                    if (!(ok = __all_sync(0xffffffffu, wait_cluster(&full[s], ph, limit)))) break;
                    tc_fence_after();
                    const uint64_t da = da0 + s * (G::kStage >> 4), db = db0 + s * (G::kStage >> 4);
                    uint64_t *const rel = &empty[s];
                    if (++s == G::kStages) { s = 0; ph ^= 1; }
                    const bool last = kb + 1 == kblocks || (F32 && chain + 1 == kChain);
                    if (elect_one_sync()) {
                        if constexpr (F32) {
                            constexpr int pa[5] = {0, 1, 1, 0, 2}, pb[5] = {1, 0, 1, 2, 0};
#pragma unroll
                            for (int i = 0; i < 5; ++i)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    pair_mma<false>(small, da + pa[i] * (G::kAtom >> 4) + j * sa_step, db + pb[i] * (G::kAtom >> 4) + j * sb_step, id,
                                                    (kb | i | j) != 0);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                pair_mma<false>(tmem + acc * BN, da + j * sa_step, db + j * sb_step, id, (chain | j) != 0);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4 * kAtoms; ++j)
                                pair_mma<FP8>(tmem + acc * BN, da + (j >> 2) * (G::kAtom >> 4) + (j & 3) * sa_step,
                                              db + (j >> 2) * (G::kAtom >> 4) + (j & 3) * sb_step, id, (kb | j) != 0);
                        }
                        pair_commit(rel, leader);
                        if (last) pair_commit(&tfull[acc], leader);
                    }
                    __syncwarp();
                    ++chain;
                    if (last) {
                        chain = 0;
                        ++n;
                    }
                }
            }
        }
        if (SPLIT) cluster_sync();
    } else {
        // ---------------------------------------------------------------- epilogue
        constexpr int kGroups = kOutN / 32;           // groups of 16 columns of this warp: half of the tile's
        const int q = warp & 3, half = warp >> 2;     // its 32 rows, its half
        const TO *const extra = (const TO *)p.extra;
        float *const cs = cols + warp * 256;          // scales (gate, up), bias
        float *const patch = cols + kEpiWarps * 256 + warp * 32 * kPatch;
        constexpr int kHalf = kOutN / 2;              // columns of this warp
        uint32_t n = 0, parity = 0;
        int64_t row0 = 0, col0 = 0;                   // of the tile at hand
        auto to_tile = [&](int t) {
            int mi, ni;
            place(t, mi, ni);
            row0 = (int64_t)mi * 256 + rank * 128 + q * 32;
            col0 = (int64_t)ni * kOutN + half * kHalf;
        };
        // What a tile's epilogue reads (its column vectors, its first group of residual, dy or dh) is asked for while the
        // tile before is finished, the other groups' values a group ahead.  (Two groups ahead: registers spill.)
        // the groups that this pair finishes: all, or its share
        const int per = SPLIT ? kGroups / p.split : kGroups, g_lo = share * per, g_hi = g_lo + per;
        Line<TO> ne;
        ColumnsAhead<kHalf> gate_scale, up_scale, bias_ahead;
        auto ask_extra = [&](int g) {
            const int64_t c = col0 + 16 * g;
            line_in(ne, extra + (row0 + lane) * p.ld_extra + c, p.ld_extra, row0, lane, p.M, c, p.N, p.vec_extra);
        };
        auto groups_here = [&] {
            const int64_t left = p.N - col0;  // columns of this warp's half that exist
            return row0 >= p.M || left <= 0 ? 0 : left < kGroups * 16 ? (int)((left + 15) / 16) : kGroups;
        };
        auto ask_tile = [&] {
            if (FP8 && p.w_scale) gate_scale.fetch(p.w_scale, col0, p.N, lane);
            if (FP8 && kGated && p.w_scale) up_scale.fetch(p.w_scale + p.N, col0, p.N, lane);
            if (!kGated && p.bias) bias_ahead.fetch(p.bias, col0, p.N, lane);
            if (kExtra && extra && groups_here() > g_lo) {
                ask_extra(g_lo);
                // the rest of the row into L2 (16054 x 256 x 8064 with a residual: 190 -> 173 us; flat where the products take longer)
                if (row0 + lane < p.M)
                    for (int c = 0; c < kHalf; c += 128 / (int)sizeof(TO))
                        if (col0 + c < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(extra + (row0 + lane) * p.ld_extra + col0 + c));
            }
        };
        // where the sums of group g from share `from` lie: the other shares' in their order, a column's 32 rows together
        constexpr int kVals = kGated ? 32 : 16;
        auto box = [&](int from, int g) {
            const int owner = g / per;
            return parts + (((warp * (p.split - 1) + (from < owner ? from : from - 1)) * per + g - owner * per) * kVals) * 32 + lane;
        };
        auto send = [&](int g, const float *v, const float *u) {
            const uint32_t dst = peer_addr(box(share, g), 2 * (g / per) + rank);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                peer_store(dst + 128 * j, v[j]);
                if constexpr (kGated) peer_store(dst + 128 * (16 + j), u[j]);
            }
        };
        auto join = [&](int g, float *v, float *u) {
            float sv[16], su[16];
            for (int from = 0; from < p.split; ++from) {
                const float *src = box(from, g);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float a = from == share ? v[j] : src[32 * j];
                    sv[j] = from ? sv[j] + a : a;
                    if constexpr (kGated) {
                        const float b = from == share ? u[j] : src[32 * (16 + j)];
                        su[j] = from ? su[j] + b : b;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                v[j] = sv[j];
                if constexpr (kGated) u[j] = su[j];
            }
        };
        if (pair < tiles) {
            to_tile(pair);
            ask_tile();
        }
        for (int t = pair; t < tiles && ok; t += pairs, parity ^= 1) {
            const int64_t row = row0 + lane;
            const bool in = row < p.M;
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * kHalf;
            const int groups = groups_here();
            const float sx = FP8 && p.x_scale && in ? p.x_scale[row] : 1.f;
            if (p.bias || (FP8 && p.w_scale)) {
                __syncwarp();  // (the last tile's are read)
                if (FP8 && p.w_scale) gate_scale.keep(cs, lane);
                if (FP8 && kGated && p.w_scale) up_scale.keep(cs + kHalf, lane);
                if (!kGated && p.bias) bias_ahead.keep(cs + 128, lane);
                __syncwarp();
            }
            // one group of 16 columns: from its sums to its outputs
            auto finish = [&](int g, float *v, float *u, const float *e) {
                const int64_t cg = col0 + 16 * g;
                if (FP8 && p.w_scale) {
                    float ws[16];
                    columns(cs + 16 * g, ws);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] *= sx * ws[j];
                    if constexpr (kGated) {
                        columns(cs + kHalf + 16 * g, ws);
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] *= sx * ws[j];
                    }
                }
                if (!kGated && p.bias) {
                    float bs[16];
                    columns(cs + 128 + 16 * g, bs);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] += bs[j];
                }
                TO *const dst = (TO *)p.out + row * p.ldo + cg;
                if constexpr (EPI == kEpiLinear) {
                    if (p.act != GDN_ACT_NONE)
                        with_act(p.act, [&](auto tag) {
#pragma unroll
                            for (int j = 0; j < 16; j += 2) act_value<kPrecise, decltype(tag)::value>(v + j, v + j);
                        });
                    if (extra) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] += e[j];
                    }
                } else if constexpr (EPI == kEpiDact) {
                    with_act(p.act, [&](auto tag) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float a[2], d[2];
                            act_both<kPrecise, decltype(tag)::value>(v + j, a, d);
                            v[j] = in ? e[j] * d[0] : 0.f;
                            v[j + 1] = in ? e[j + 1] * d[1] : 0.f;
                        }
                    });
                } else if constexpr (EPI == kEpiGated) {
                    with_act(p.act, [&](auto tag) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            act_value<kPrecise, decltype(tag)::value>(v + j, v + j);
                            v[j] *= u[j];
                            v[j + 1] *= u[j + 1];
                        }
                    });
                } else {
                    float h[16];
                    with_act(p.act, [&](auto tag) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float a[2], d[2];
                            act_both<kPrecise, decltype(tag)::value>(v + j, a, d);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                h[j + i] = a[i] * u[j + i];
                                v[j + i] = e[j + i] * u[j + i] * d[i];
                                u[j + i] = e[j + i] * a[i];
                            }
                        }
                    });
                    line_out(dst + p.N, p.ldo, row0, lane, p.M, cg, p.N, p.vec_out, u, patch);
                    if (p.out2) line_out((TO *)p.out2 + row * p.ldo2 + cg, p.ldo2, row0, lane, p.M, cg, p.N, p.vec_out2, h, patch);
                }
                line_out(dst, p.ldo, row0, lane, p.M, cg, p.N, p.vec_out, v, patch);
                if (EPI == kEpiDact && p.colpart) {
                    const float sum = column_sums(v, lane);
                    const int64_t cc = cg + (lane >> 1);
                    if (!(lane & 1) && cc < p.N) p.colpart[(row0 >> 5) * p.N + cc] = sum;
                }
            };
            auto extra_of = [&](int g, float *e) {  // (called for g = g_lo, g_lo + 1, ...)
                if (kExtra && extra) {
                    line_get(ne, e, lane, col0 + 16 * g, p.N, p.vec_extra, patch);
                    if (g + 1 < groups && g + 1 < g_hi) ask_extra(g + 1);
                }
            };
            // the next tile's, once the last group has taken its own
            auto ask_next = [&] {
                if (t + pairs < tiles) {
                    to_tile(t + pairs);
                    ask_tile();
                }
            };
            auto sums_ready = [&] {
                ok = __all_sync(0xffffffffu, wait_cluster(&tfull[n & 1], (n >> 1) & 1, limit));
                tc_fence_after();
                return ok;
            };
            // the accumulators are read: hand them back to the issuer
            auto sums_read = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) remote_arrive(peer_addr(&tempty[n & 1], leader));
                ++n;
            };
            if constexpr (F32) {
                float sv[kGroups][16], su[kGated ? kGroups : 1][16];
                // (an infinite or NaN leading sum stands: a small product of an infinity with a zero plane would spoil it)
                auto with_small = [](float sum, float small) { return fabsf(sum) <= kF32Max ? sum + small : sum; };
                enum Part { kFirst, kNext, kSmall };
                auto add = [&](uint32_t from, auto part) {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        if (g >= groups) continue;
                        float v[16], u[16];
                        tmem_ld16(from + 16 * g, v);
                        if constexpr (kGated) tmem_ld16(from + BN / 2 + 16 * g, u);
                        tmem_ld_wait();
                        pin16(v);
                        if constexpr (kGated) pin16(u);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            constexpr Part what = (Part)decltype(part)::value;
                            sv[g][j] = what == kFirst ? v[j] : what == kNext ? sv[g][j] + v[j] : with_small(sv[g][j], v[j]);
                            if constexpr (kGated) su[g][j] = what == kFirst ? u[j] : what == kNext ? su[g][j] + u[j] : with_small(su[g][j], u[j]);
                        }
                    }
                };
                for (int kb = 0; kb < kblocks; kb += kChain) {
                    if (!sums_ready()) break;
                    if (kb == 0) add(lanes + (n & 1) * BN, std::integral_constant<int, kFirst>());
                    else add(lanes + (n & 1) * BN, std::integral_constant<int, kNext>());
                    if (kb + kChain >= kblocks) add(lanes + (2 + parity) * BN, std::integral_constant<int, kSmall>());
                    sums_read();
                }
                if constexpr (SPLIT) {
                    if (ok) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g)
                            if (g < groups && (g < g_lo || g >= g_hi)) send(g, sv[g], su[kGated ? g : 0]);
                    }
                    cluster_sync();
                }
                if (!ok) break;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    if (g >= groups || (SPLIT && (g < g_lo || g >= g_hi))) continue;
                    float e[16];
                    extra_of(g, e);
                    if constexpr (SPLIT) join(g, sv[g], su[kGated ? g : 0]);
                    finish(g, sv[g], su[kGated ? g : 0], e);
                }
                ask_next();
            } else if constexpr (SPLIT) {
                const uint32_t tl = lanes;
                float v[16], u[16], e[16];
                auto sums = [&](int g) {
                    tmem_ld16(tl + 16 * g, v);
                    if constexpr (kGated) tmem_ld16(tl + BN / 2 + 16 * g, u);
                    tmem_ld_wait();
                    pin16(v);
                    if constexpr (kGated) pin16(u);
                };
                if (sums_ready()) {
#pragma unroll 1
                    for (int g = 0; g < groups; ++g) {
                        if (g >= g_lo && g < g_hi) continue;
                        sums(g);
                        send(g, v, u);
                    }
                }
                cluster_sync();
                if (!ok) break;
#pragma unroll 1
                for (int g = g_lo; g < groups && g < g_hi; ++g) {
                    extra_of(g, e);
                    sums(g);
                    join(g, v, u);
                    finish(g, v, u, e);
                }
            } else {
                const uint32_t tl = lanes + (n & 1) * BN;
                if (!sums_ready()) break;
                float nv[16], nu[kGated ? 16 : 1];
                if (groups) {
                    tmem_ld16(tl, nv);
                    if constexpr (kGated) tmem_ld16(tl + BN / 2, nu);
                }
                // (rolled: unrolled over a tile's columns, an activation's code left the instruction cache at every pass)
#pragma unroll 1
                for (int g = 0; g < groups; ++g) {
                    float v[16], u[16], e[16];
                    extra_of(g, e);
                    tmem_ld_wait();
                    pin16(nv);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = nv[j];
                    if constexpr (kGated) {
                        pin16(nu);
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = nu[j];
                    }
                    if (g + 1 < groups) {
                        tmem_ld16(tl + 16 * (g + 1), nv);
                        if constexpr (kGated) tmem_ld16(tl + BN / 2 + 16 * (g + 1), nu);
                    } else {
                        sums_read();  // (the last accumulators are in registers)
                    }
                    finish(g, v, u, e);
                }
                if (!groups) sums_read();
                ask_next();
            }
        }
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

size_t esz(gdn_dtype t) { return t == GDN_BF16 ? 2 : 1; }  // of an operand

template <int KIND, int LAYOUT, int EPI, int BN, typename TO, bool SPLIT = false>
cudaError_t go(const GemmArgs &g, cudaStream_t st, int split = 1)
{
    constexpr bool gated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    using G = Geo<KIND, BN, SPLIT>;
    TcMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const int64_t brows = gated ? 2 * g.N : g.N;
    const gdn_dtype in = KIND == kE4m3 ? GDN_E4M3 : GDN_BF16;
    for (int i = 0; i < (KIND == kF32 ? 3 : 1); ++i) {
        const void *a = (const char *)g.a + (KIND == kF32 ? 2 * i * g.a_plane : 0), *b = (const char *)g.b + (KIND == kF32 ? 2 * i * g.b_plane : 0);
        const bool a_ok = LAYOUT == 2 ? make_operand_map(&maps.a[i], in, a, g.M, g.K, g.lda, 64) : make_operand_map(&maps.a[i], in, a, g.K, g.M, g.lda, 128);
        const bool b_ok = LAYOUT >= 1 ? make_operand_map(&maps.b[i], in, b, brows, g.K, g.ldb, 64)
                                      : make_operand_map(&maps.b[i], in, b, g.K, brows, g.ldb, BN / 2);
        if (!a_ok || !b_ok) return cudaErrorInvalidValue;
    }
    TcParams p{};
    p.M = g.M; p.N = g.N;
    const int per = G::kPerStage * (KIND == kE4m3 ? 128 : 64);
    p.kblocks = (int)((g.K + per - 1) / per);
    p.mt = (int)((g.M + 255) / 256);
    p.nt = (int)((g.N + (gated ? BN / 2 : BN) - 1) / (gated ? BN / 2 : BN));
    p.x_scale = g.x_scale; p.w_scale = g.w_scale; p.bias = g.bias; p.act = g.act;
    p.extra = g.extra; p.ld_extra = g.ld_extra;
    p.out = g.out; p.ldo = g.ldo; p.out2 = g.out2; p.ldo2 = g.ldo2;
    p.colpart = g.colpart;
    p.split = split;
    const size_t eo = sizeof(TO);
    auto allows = [&](const void *q, int64_t ld, size_t also) {
        const size_t off = (uintptr_t)q | (g.M > 1 ? (size_t)ld * eo : 0) | also;
        return off % 32 == 0 ? 2 : off % 16 == 0 ? 1 : 0;
    };
    p.vec_out = allows(g.out, g.ldo, EPI == kEpiGatedBwd ? g.N * eo : 0);
    p.vec_extra = allows(g.extra, g.ld_extra, 0);
    p.vec_out2 = allows(g.out2, g.ldo2, 0);

    auto *kern = gemm_tc_kernel<KIND, LAYOUT, EPI, BN, TO, SPLIT, false>;
    static std::atomic<uint64_t> seen;
    bool first = first_on_device(seen);
    if constexpr (KIND != kE4m3 && LAYOUT == 0 && EPI == kEpiLinear && BN == 128 && sizeof(TO) == (KIND == kF32 ? 4 : 2)) {
        if (withhold_loads()) {
            kern = gemm_tc_kernel<KIND, LAYOUT, EPI, BN, TO, SPLIT, true>;
            first = true;
        }
    }
    if (first) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
        if (e != cudaSuccess) return e;
        if (!withhold_loads()) done_on_device(seen);
    }
    const int64_t tiles = (int64_t)p.mt * p.nt;
    const int pairs = SPLIT ? (int)tiles * split : (int)(tiles < device_sm_count() / 2 ? tiles : device_sm_count() / 2);
    return launch_overlapped(kern, 2 * pairs, 1, kThreads, G::kSmem, 2 * split, st, maps, p);
}

// (holds no tensor memory: the runtime answers one block per SM for a kernel that does, whatever else it asks for)
__global__ void __launch_bounds__(kThreads) place_kernel() {}

// clusters of 2 `split` CTAs, one to an SM, that the device runs at once (asked once per device)
int64_t clusters_at_once(int split)
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][kMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = 0;
    int n = known[dev][split].load(std::memory_order_relaxed);
    if (n) return n;
    constexpr int room = 200 * 1024;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2u * split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2u * split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = room;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, room) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, place_kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = device_sm_count() / (2 * split + 2);
    }
    known[dev][split].store(n, std::memory_order_relaxed);
    return n;
}

// Pairs that share a tile's contraction: as many as there is room for, while each keeps enough of it to repay the
// exchange of the sums (1.2 us for two, 2.0 us for four): six stages of bf16 or e4m3 (of 0.26 us; 256 x 2048 outputs:
// K = 1024 6.1 us alone and 6.3 as two, K = 2048 8.2 and 7.5, K = 5504 15.3 and 11.6; 256 x 512 x 8192 20.6, 13.9 as two,
// 10.1 as four); two of fp32 (six products each; 256 x 1024 x 512: 15.9, 13.7, 12.4 us); two of a gated tile.
template <int KIND>
int split_for(const GemmArgs &g, bool gated)
{
    const int64_t wide = gated ? 64 : 128, tiles = (g.M + 255) / 256 * ((g.N + wide - 1) / wide);
    const int per = Geo<KIND, 128, true>::kPerStage * (KIND == kE4m3 ? 128 : 64);
    const int64_t kb = (g.K + per - 1) / per, least = KIND == kF32 || gated ? 2 : 6;
    for (int split = gated ? 2 : kMaxSplit; split > 1; split /= 2)
        if (kb >= split * least && tiles <= clusters_at_once(split)) return split;
    return 1;
}

template <int KIND, int LAYOUT, int EPI, typename TO>
cudaError_t pick(const GemmArgs &g, cudaStream_t st)
{
    constexpr bool gated = EPI == kEpiGated || EPI == kEpiGatedBwd;
    const int split = split_for<KIND>(g, gated);
    if (split > 1) return go<KIND, LAYOUT, EPI, 128, TO, true>(g, st, split);
    if constexpr (KIND == kF32) {
        return go<KIND, LAYOUT, EPI, 128, TO>(g, st);
    } else {
        // Whole rounds of tiles over the pairs of SMs decide: a round of 128-column tiles takes 0.58 of one of 256
        // columns (6.2 and 10.7 us at K = 2048: its products re-read A), but fills a ragged last round better.
        const int64_t pairs = device_sm_count() / 2, mt = (g.M + 255) / 256;
        const auto rounds = [&](int64_t bn) { return (mt * ((g.N * (gated ? 2 : 1) + bn - 1) / bn) + pairs - 1) / pairs; };
        if (0.58 * rounds(128) < rounds(256)) return go<KIND, LAYOUT, EPI, 128, TO>(g, st);
        return go<KIND, LAYOUT, EPI, 256, TO>(g, st);
    }
}

// Few rows: the weights' reading is the cost, and the pair's tiles would be padding.  (A weight gradient's rows are
// the weight's, and its contraction the batch.)
bool use_small(const GemmArgs &g) { return !g.a_t && g.M <= kFewRows; }

// fp32 rows as three planes of bf16: each the rounding of what the ones before leave (exactly x from 2^-110 on; the planes of
// smaller values end at bf16's smallest, 2^-133), the first no larger than bf16's largest while x is finite; an infinity or NaN has zeros in the lower planes
__global__ void __launch_bounds__(256) split_kernel(const float *src, int64_t ld, int64_t rows, int64_t cols, __nv_bfloat16 *dst, int64_t pitch,
                                                    int64_t plane)
{
    grid_release();
    grid_wait();
    constexpr int kPairs = 8;
    const int64_t per_row = (cols + 64 * kPairs - 1) / (64 * kPairs), warps = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t u = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; u < rows * per_row; u += warps) {
        const int64_t r = u / per_row, c0 = (u - r * per_row) * (64 * kPairs) + (threadIdx.x & 31) * 2;
        float x[kPairs][2];
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) x[k][j] = c0 + 64 * k + j < cols ? src[r * ld + c0 + 64 * k + j] : 0.f;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            const int64_t c = c0 + 64 * k;
            if (c >= cols) break;
            const bool finite[2] = {fabsf(x[k][0]) <= kF32Max, fabsf(x[k][1]) <= kF32Max};
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                float y[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) y[j] = finite[j] ? fminf(fmaxf(x[k][j], -kBf16Max), kBf16Max) : i ? 0.f : x[k][j];
                const uint32_t w = pack_bf16(y[0], y[1]);
                *(uint32_t *)(dst + i * plane + r * pitch + c) = w;
                x[k][0] -= __uint_as_float(w << 16);
                x[k][1] -= __uint_as_float(w & 0xffff0000u);
            }
        }
    }
}

// Rows into another layout, element by element: a warp takes 32 x 16 consecutive elements of a row, all on their way at
// once (a block that walked a row four bytes a thread waited once per step: 16384 x 1001 x 1001 with a residual, four such
// copies, 108 us; 93 so).
template <typename T>
__global__ void __launch_bounds__(256) copy_rows_kernel(const T *src, int64_t ld, int64_t rows, int64_t cols, T *dst, int64_t ldd)
{
    constexpr int kEach = 16;
    grid_release();
    grid_wait();
    const int64_t per_row = (cols + 32 * kEach - 1) / (32 * kEach), warps = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t u = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; u < rows * per_row; u += warps) {
        const int64_t r = u / per_row, c = (u - r * per_row) * (32 * kEach) + (threadIdx.x & 31);
        T v[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] = c + 32 * i < cols ? src[r * ld + c + 32 * i] : T(0);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (c + 32 * i < cols) dst[r * ldd + c + 32 * i] = v[i];
    }
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
    const CUtensorMapDataType dt = t == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return enc(m, dt, 2, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tma_ok(const void *p, int64_t ld, int64_t rows, size_t e)
{
    return ((uintptr_t)p & 15) == 0 && (rows <= 1 || (size_t)ld * e % 16 == 0);
}

// one warp to 512 elements of a row, as many as run at once
unsigned blocks_of_rows(int64_t rows, int64_t cols)
{
    const int64_t blocks = (rows * ((cols + 511) / 512) + 7) / 8, most = 8 * device_sm_count();
    return (unsigned)(blocks < most ? blocks : most);
}

cudaError_t launch_split(const float *src, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t pitch, int64_t plane, cudaStream_t st)
{
    return launch_overlapped(split_kernel, blocks_of_rows(rows, cols), 1, 256, 0, 0, st, src, ld, rows, cols, (__nv_bfloat16 *)dst, pitch, plane);
}

cudaError_t launch_copy_rows(const void *src, gdn_dtype t, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t ldd, cudaStream_t st)
{
    const unsigned grid = blocks_of_rows(rows, cols);
    if (t == GDN_F32)
        return launch_overlapped(copy_rows_kernel<uint32_t>, grid, 1, 256, 0, 0, st, (const uint32_t *)src, ld, rows, cols, (uint32_t *)dst, ldd);
    if (t == GDN_BF16)
        return launch_overlapped(copy_rows_kernel<uint16_t>, grid, 1, 256, 0, 0, st, (const uint16_t *)src, ld, rows, cols, (uint16_t *)dst, ldd);
    return launch_overlapped(copy_rows_kernel<uint8_t>, grid, 1, 256, 0, 0, st, (const uint8_t *)src, ld, rows, cols, (uint8_t *)dst, ldd);
}

int64_t gemm_colparts(const GemmArgs &g, Epi epi)
{
    if (g.in == GDN_F32 && !g.a_plane) return gemm_simt_colparts(g, epi);
    return g.in != GDN_F32 && use_small(g) ? gemm_small_colparts(g, epi) : (g.M + 31) / 32;
}

cudaError_t launch_gemm_tc(const GemmArgs &g, Epi epi, cudaStream_t st)
{
    if (g.M <= 0 || g.N <= 0) return cudaSuccess;
    if (g.in == GDN_F32) {
        switch (epi) {
        case kEpiGated: return pick<kF32, 0, kEpiGated, float>(g, st);
        case kEpiGatedBwd: return pick<kF32, 0, kEpiGatedBwd, float>(g, st);
        case kEpiDact: return pick<kF32, 0, kEpiDact, float>(g, st);
        default: break;
        }
        return g.a_t ? pick<kF32, 2, kEpiLinear, float>(g, st) : g.b_t ? pick<kF32, 1, kEpiLinear, float>(g, st) : pick<kF32, 0, kEpiLinear, float>(g, st);
    }
    if (use_small(g)) return launch_gemm_small(g, epi, st);
    const bool f32 = g.out_dt == GDN_F32;
    if (g.in == GDN_E4M3) {
        if (epi == kEpiGated) return pick<kE4m3, 0, kEpiGated, __nv_bfloat16>(g, st);
        return f32 ? pick<kE4m3, 0, kEpiLinear, float>(g, st) : pick<kE4m3, 0, kEpiLinear, __nv_bfloat16>(g, st);
    }
    switch (epi) {
    case kEpiGated: return pick<kBf16, 0, kEpiGated, __nv_bfloat16>(g, st);
    case kEpiGatedBwd: return pick<kBf16, 0, kEpiGatedBwd, __nv_bfloat16>(g, st);
    case kEpiDact: return pick<kBf16, 0, kEpiDact, __nv_bfloat16>(g, st);
    default: break;
    }
    if (g.a_t) return pick<kBf16, 2, kEpiLinear, __nv_bfloat16>(g, st);
    if (g.b_t) return pick<kBf16, 1, kEpiLinear, __nv_bfloat16>(g, st);
    return f32 ? pick<kBf16, 0, kEpiLinear, float>(g, st) : pick<kBf16, 0, kEpiLinear, __nv_bfloat16>(g, st);
}

gdn_status read_tc_status(cudaStream_t st)
{
    unsigned word = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, g_tc_status, sizeof(word), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_tc_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return word & kStatusTimeout ? GDN_ERR_TIMEOUT : GDN_OK;
}

}  // namespace gdn
