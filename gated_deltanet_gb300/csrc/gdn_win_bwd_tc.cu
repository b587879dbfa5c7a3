// Gradients of attention with a sliding window and sinks on the tensor cores: bf16, heads of 64 or 128, rows on 16-byte boundaries.
//
//   P = exp2(c S - lse'),  dP = dO V^T,  Z = P (dP - delta):   dQ = scale Z K,  dK = scale Z^T Q,  dV = P^T dO
// with c = scale log2 e, lse' in base 2, delta = the row's dO . o.  Two kernels, each with the gradients it owns in tensor memory and
// the scores taken again (seven products of a tile of pairs in place of five, but no atomics: sums have a fixed order, and no fp32
// gradient passes through memory):
//   win_dq_kernel   128 queries of a head against the tiles of 128 keys that they see; also takes delta
//   win_dkv_kernel  128 keys of a key head against the tiles of 128 queries of its heads that see them, scores transposed (a lane is
//                   a key), so that P^T and Z^T are left operands in tensor memory as they come
// The far queries of sinks are dealt out to CTAs of their own, whose parts win_sinks_kernel adds up (WinSinks).
//
// 4 x 4096 tokens, 16 heads over 4 of 128, window 1024: 445 us: dQ 188, dK and dV 254 (680 TFLOP/s by the floor's five products).
//  - dQ: one CTA per SM walks tiles of queries (a CTA to each: 245 us at the time; starting one and filling its pipeline took 12000 cycles, the walk 24000).
//    Q and dO are left operands in tensor memory: 128 x 128 x 16 then takes 67 cycles, with both operands in shared memory 104, which is bound by
//    its 80 bytes a cycle.  A tile of keys takes 2480 cycles: its products 1610 alone, the copies of K and V take shared memory from them.
//  - dK, dV: no room for K and V beside four accumulators; a tile of queries takes 3000 cycles, its products 2740.
//  - Four groups of 128 lanes in place of two: no faster (the exponentials are 1024 cycles of a tile's either way), and 96 registers spill.
//
// Warps: 0-3 and 4-7 two groups of 128 lanes, each on half of a tile's columns, 8 loads, 9 products.
#include "gdn_mix.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kTile = 128, kBox = kTile * 128;
constexpr int kGroups = 2, kCols = kTile / kGroups, kLanes = 128 * kGroups, kLoads = 4 * kGroups, kProducts = kLoads + 1, kThreads = kLanes + 64;
constexpr uint32_t kTmem = 512;

__device__ unsigned g_win_bwd_status;

template <int D>
struct Geo {
    static constexpr int kBoxes = D / 64, kUnit = kBoxes * kBox, kRing = D == 128 ? 5 : 8;
    static constexpr int kA = 0, kB = kUnit, kRingAt = 2 * kUnit, kStats = kRingAt + kRing * kUnit, kBars = kStats + 1024, kItems = kBars + 256, kSmem = kItems + 128 + 1024;
};
enum Bar { kIn, kAB, kTaken, kSF, kSR, kPF, kPB, kZB, kDone, kFin, kLanded, kFull, kMostRing = 8, kEmpty = kFull + kMostRing, kNumBars = kEmpty + kMostRing };

struct Maps {
    CUtensorMap q, k, v, o, dout, dq, dk, dv;
};

__device__ __forceinline__ void init_bars(uint64_t *bar, int ring)
{
    mbar_init(&bar[kIn], 1);
    mbar_init(&bar[kAB], 4 * kGroups);
    mbar_init(&bar[kTaken], 1);
    mbar_init(&bar[kFin], 1);
    mbar_init(&bar[kSF], 1);
    mbar_init(&bar[kSR], 4 * kGroups);
    mbar_init(&bar[kPF], 1);
    mbar_init(&bar[kPB], 4 * kGroups);
    mbar_init(&bar[kZB], 4 * kGroups);
    mbar_init(&bar[kDone], 1);
    mbar_init(&bar[kLanded], 1);
    for (int i = 0; i < ring; ++i) {
        mbar_init(&bar[kFull + i], 1);
        mbar_init(&bar[kEmpty + i], 1);
    }
    fence_mbar_init();
}
// rows from `rows` on of a tile of BOXES boxes, by one warp
template <int BOXES>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int rows)
{
#pragma unroll
    for (int b = 0; b < BOXES; ++b)
        for (int e = rows * 8 + (threadIdx.x & 31); e < kTile * 8; e += 32) *(uint4 *)(tile + b * kBox + e * 16) = make_uint4(0, 0, 0, 0);
}
// D(128 x 128) = A(128 x D) B(128 x D)^T, both rows of d in shared memory
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b)
{
    const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(b, 16, 1024);
    constexpr uint32_t id = idesc_bf16_f32(128, 128, 0, 0);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t o = ((ks >> 2) * kBox + (ks & 3) * 32) >> 4;
        mma_ss(d, da + o, db + o, id, ks > 0);
    }
}
// The same with A's rows in tensor memory
template <int D>
__device__ __forceinline__ void mma_kept(uint32_t d, uint32_t a, uint32_t b)
{
    const uint64_t db = sdesc_sw128(b, 16, 1024);
    constexpr uint32_t id = idesc_bf16_f32(128, 128, 0, 0);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) mma_ts(d, a + ks * 8, db + (((ks >> 2) * kBox + (ks & 3) * 32) >> 4), id, ks > 0);
}
// D(128 x D) (+)= A(128 x 128) B(128 x D): A bf16 in tensor memory, each group's columns in the place of its scores, B's rows in shared memory
template <int D>
__device__ __forceinline__ void mma_sum(uint32_t d, uint32_t a, uint32_t b, bool fresh)
{
    const uint64_t db = sdesc_sw128(b, kBox, 1024);
    constexpr uint32_t id = idesc_bf16_f32(128, D, 0, 1);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_ts(d, a + ks / (kCols / 16) * kCols + ks % (kCols / 16) * 8, db + ks * 128, id, !fresh || ks > 0);
}
// the first rows of a tile in shared memory to [tokens][heads][D], by THREADS threads (r: which)
template <int D, int THREADS>
__device__ __forceinline__ void copy_rows(void *out, const uint8_t *tile, int64_t t0, int rows, int heads, int h, int r)
{
    for (int k = r; k < rows * (D / 8); k += THREADS) {
        const int row = k / (D / 8), e = k % (D / 8) * 8;
        *(uint4 *)((__nv_bfloat16 *)out + ((t0 + row) * heads + h) * D + e) = *(const uint4 *)(tile + (e >> 6) * kBox + sw128(row, e & 63));
    }
}

// ---------------------------------------------------------------- dQ (lane = query)
// A tile of queries of a head, and the tiles of keys that it sees: those of the sinks in front of its window, then the window's
struct Queries {
    int64_t at;            // of its first row in lse and delta
    int t0, rows, h, p0;   // first token, rows (0: no more tiles), head, position of the first row
    int k0, klen, hk;      // the sequence's first key and length, key head
    int lo, hi, first, nfirst, nt;
    int b, tb;             // batch and its token, as O is asked for
    __device__ __forceinline__ void set(const WinArgs &a, unsigned item)
    {
        h = (int)(item % (unsigned)a.H);
        hk = h / (a.H / a.HK);
        const Tile tl = tile_of(a.cu_q, a.N, a.Tq, kTile, item / (unsigned)a.H);
        const SeqRange sq = seq_range(a.cu_q, tl.n, a.Tq), sk = seq_range(a.cu_k, tl.n, a.Tk);
        const int i0 = tl.index * kTile;
        at = lse_at(a, tl.n, sq.bos, h) + i0;
        t0 = (int)(sq.bos + i0);
        b = a.cu_q ? 0 : tl.n;
        tb = t0 - b * a.Tq;
        rows = max(min(kTile, sq.len - i0), 0);
        p0 = i0 + sk.len - sq.len;
        k0 = (int)sk.bos;
        klen = sk.len;
        hi = min(max(p0 + rows, 0), klen);
        lo = hi == 0 ? 0 : min(max(p0 - a.window + 1, 0), hi);
        first = min(a.sinks, lo);
        nfirst = (first + kTile - 1) / kTile;
        nt = nfirst + (hi - lo + kTile - 1) / kTile;
    }
    __device__ __forceinline__ int key0(int t) const { return t < nfirst ? t * kTile : lo + (t - nfirst) * kTile; }
    __device__ __forceinline__ int columns(int t) const { return min(kTile, (t < nfirst ? first : hi) - key0(t)); }
    __device__ __forceinline__ bool ragged(int t) const { return key0(t) + kTile > klen; }
};
static_assert(sizeof(Queries) <= 64);

template <int D>
__global__ void __launch_bounds__(kThreads, 1) win_dq_kernel(const __grid_constant__ Maps maps, const WinArgs a, unsigned items, float *delta, uint64_t limit,
                                                             int withhold)
{
    using G = Geo<D>;
    constexpr uint32_t kS = 0, kP = 128, kQ = 256, kAQ = 384, kAG = 448;  // S, dP (Z in its place), dQ; Q and dO as left operands
    extern __shared__ uint8_t win_bwd_smem[];
    uint8_t *const sm = win_bwd_smem + (-smem_u32(win_bwd_smem) & 1023u);  // (an offset: a cast would lose that it is shared memory)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *bar = (uint64_t *)(sm + G::kBars);
    uint32_t *tslot = (uint32_t *)(bar + kNumBars);
    if (tid == 0) init_bars(bar, G::kRing);
    if (tid == 32) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.dout);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    if (warp == kLoads) tmem_alloc(tslot, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, base = smem_u32(sm);
    unsigned *const status = &g_win_bwd_status;
    auto wait = [&](int b, uint32_t parity) { return mbar_wait(&bar[b], parity, status, kStatusTimeout, limit); };
    auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    auto full = [&](int i) { return all(wait(kFull + i % G::kRing, (i / G::kRing) & 1)); };  // a tile of queries: O, K and V of each tile of keys, a place for dQ
    auto unit = [&](int i) { return G::kRingAt + (i % G::kRing) * G::kUnit; };

    // n counts this CTA's tiles of queries, i and first_unit the units, from and t the tiles of keys of all of them.  The loading warp finds
    // the tiles and hands them on with kIn, a tile without rows behind the last.
    Queries *const handed = (Queries *)(sm + G::kItems);
    bool ok = true;
    int n = 0, from = 0, first_unit = 0;
    Queries it;
    if (warp == kLoads) {
        // ---------------------------------------------------------------- loads
        ok = !withhold;
        int i = 0, mended = 0;
        for (unsigned item = blockIdx.x; ok; item += gridDim.x) {
            it.rows = 0;
            if (item < items) {
                it.set(a, item);
                if (it.rows == 0) continue;
            }
            if (n > 0 && !(ok = all(wait(kTaken, (n - 1) & 1)))) break;
            if (elect_one_sync()) {
                handed[n & 1] = it;
                if (it.rows == 0) {
                    mbar_arrive(&bar[kIn]);
                } else {
                    mbar_arrive_expect_tx(&bar[kIn], 2 * G::kUnit);
#pragma unroll
                    for (int b = 0; b < G::kBoxes; ++b) {
                        tma_load_3d(sm + G::kA + b * kBox, &maps.q, b * 64, it.h, it.t0, &bar[kIn]);
                        tma_load_3d(sm + G::kB + b * kBox, &maps.dout, b * 64, it.h, it.t0, &bar[kIn]);
                    }
                }
            }
            __syncwarp();
            ++n;
            if (it.rows == 0) break;
            for (int u = -1; u <= 2 * it.nt; ++u, ++i) {
                const int s = i % G::kRing, t = u >> 1;
                if (i >= G::kRing && !(ok = all(wait(kEmpty + s, (i / G::kRing - 1) & 1)))) break;
                if (u == 2 * it.nt) {  // (given to dQ as it is)
                    if (lane == 0) mbar_arrive(&bar[kFull + s]);
                    continue;
                }
                // K's rows behind the end are the next sequence's, and 0 x NaN is NaN: they are zeroed before the tile counts as full
                const bool mend = u >= 0 && !(u & 1) && it.ragged(t);
                uint64_t *const landing = &bar[mend ? (int)kLanded : kFull + s];
                if (elect_one_sync()) {
                    mbar_arrive_expect_tx(landing, G::kUnit);
#pragma unroll
                    for (int b = 0; b < G::kBoxes; ++b) {
                        if (u < 0) tma_load_4d(sm + unit(i) + b * kBox, &maps.o, b * 64, it.h, it.tb, it.b, landing);
                        else tma_load_3d(sm + unit(i) + b * kBox, u & 1 ? &maps.v : &maps.k, b * 64, it.hk, it.k0 + it.key0(t), landing);
                    }
                }
                __syncwarp();
                if (mend) {
                    if (!(ok = all(wait(kLanded, mended++ & 1)))) break;
                    zero_rows<G::kBoxes>(sm + unit(i), it.klen - it.key0(t));
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[kFull + s]);
                }
            }
        }
        // no copy outlives the CTA
        if (n > 0) wait(kIn, (n - 1) & 1);
        for (int k = max(0, i - G::kRing); k < i; ++k) wait(kFull + k % G::kRing, (k / G::kRing) & 1);
    } else if (warp == kProducts) {
        // ---------------------------------------------------------------- products: S(t+1), dQ(t), dP(t+1)
        auto key = [&](int t) { return first_unit + 1 + 2 * (t - from); };  // the unit of tile t's K; its V is the next
        auto scores = [&](int t) {
            tc_fence_after();
            if (elect_one_sync()) {
                mma_kept<D>(tmem + kS, tmem + kAQ, base + unit(key(t)));
                mma_commit(&bar[kSF]);
            }
            __syncwarp();
        };
        auto slopes = [&](int t) {
            tc_fence_after();
            if (elect_one_sync()) {
                mma_kept<D>(tmem + kP, tmem + kAG, base + unit(key(t) + 1));
                mma_commit(&bar[kPF]);
                mma_commit(&bar[kEmpty + (key(t) + 1) % G::kRing]);
            }
            __syncwarp();
        };
        for (;; ++n) {
            // (the groups have taken all of the last tile of queries' scores)
            if (!(ok = all(wait(kAB, n & 1)))) break;
            it = handed[n & 1];
            if (it.rows == 0) break;
            const int end = from + it.nt;
            if (it.nt > 0) {
                if (!(ok = full(key(from)))) break;
                scores(from);
                if (!(ok = full(key(from) + 1))) break;
                slopes(from);
            }
            for (int t = from; t < end; ++t) {
                if (t + 1 < end) {
                    if (!(ok = all(wait(kSR, t & 1)) && full(key(t + 1)))) break;
                    scores(t + 1);
                }
                if (!(ok = all(wait(kZB, t & 1)))) break;
                tc_fence_after();
                if (elect_one_sync()) {
                    mma_sum<D>(tmem + kQ, tmem + kP, base + unit(key(t)), t == from);
                    mma_commit(&bar[kEmpty + key(t) % G::kRing]);
                }
                __syncwarp();
                if (t + 1 < end) {
                    if (!(ok = full(key(t + 1) + 1))) break;
                    slopes(t + 1);
                }
            }
            if (!ok) break;
            if (elect_one_sync()) mma_commit(&bar[kDone]);
            __syncwarp();
            first_unit += 2 + 2 * it.nt;
            from = end;
        }
        if (elect_one_sync()) mma_commit(&bar[kFin]);  // every product has ended before the tensor memory goes
        __syncwarp();
        wait(kFin, 0);
    } else {
        const int x = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kS + kCols * x, tp = tmem + lanes + kP + kCols * x;
        const float c = a.scale * kLog2e;
        float *const part = (float *)(sm + G::kStats);
        bool stored = false;  // (thread 0: a store is on its way from a unit's place)
        int place = 0;
        // the next tile of queries: Q by one group, dO by the other, to tensor memory; delta by the other, which has the row of dO (what stands
        // behind the last row is not taken).  Before any product of the tile: they leave little of shared memory to others.
        auto take = [&]() {
            if (!(ok = bar_all(1, kLanes, warp != 0 || wait(kIn, n & 1)))) return;
            it = handed[n & 1];
            if (it.rows > 0) {
                if (!(ok = bar_all(1, kLanes, warp != 0 || wait(kFull + first_unit % G::kRing, (first_unit / G::kRing) & 1)))) return;
                const uint8_t *src = sm + (x == 0 ? G::kA : G::kB);
                uint32_t w[D / 2];
#pragma unroll
                for (int col = 0; col < D; col += 8) *(uint4 *)&w[col / 2] = *(const uint4 *)(src + (col >> 6) * kBox + sw128(r, col & 63));
#pragma unroll
                for (int col = 0; col < D; col += 32) tmem_st16(tmem + lanes + (x == 0 ? kAQ : kAG) + col / 2, w + col / 2);
                if (x != 0) {
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int col = 0; col < D; col += 8) {
                        const uint4 u = *(const uint4 *)(sm + unit(first_unit) + (col >> 6) * kBox + sw128(r, col & 63));
                        const uint32_t *pu = (const uint32_t *)&u, *pg = w + col / 2;
#pragma unroll
                        for (int k = 0; k < 4; ++k) sum[k] = fmaf(high_bf16(pu[k]), high_bf16(pg[k]), fmaf(low_bf16(pu[k]), low_bf16(pg[k]), sum[k]));
                    }
                    part[r] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kAB]);
        };
        take();
        while (ok && it.rows > 0) {
            const int p = it.p0 + r;
            float lse = r < it.rows ? a.lse[it.at + r] : INFINITY;
            bar_sync(1, kLanes);
            if (tid == 0) {  // (the next tile of queries may be loaded, and another unit in O's place and in the last dQ's)
                mbar_arrive(&bar[kTaken]);
                mbar_arrive(&bar[kEmpty + first_unit % G::kRing]);
                if (stored) {
                    tma_store_wait_read0();
                    mbar_arrive(&bar[kEmpty + place]);
                    stored = false;
                }
            }
            const float d = part[r];
            if (x == 0 && r < it.rows) delta[it.at + r] = d;
            lse = lse == -INFINITY ? INFINITY : lse * kLog2e;  // (a row that sees nothing: weights of zero)
            for (int t = 0; t < it.nt; ++t) {
                const int j0 = it.key0(t) + kCols * x, cols = it.columns(t) - kCols * x;
                if (!(ok = bar_all(1, kLanes, warp != 0 || wait(kSF, (from + t) & 1)))) break;
                tc_fence_after();
                float s[kCols];
#pragma unroll
                for (int q = 0; q < kCols; q += 32) tmem_ld32(ts + q, (uint32_t *)s + q);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kSR]);  // (the next tile's scores may come)
                const Pair cc = pair_of(c, c), minus = pair_of(-lse, -lse);
#pragma unroll
                for (int j = 0; j < kCols; j += 2) {
                    unpair(fma2(pair_of(s[j], s[j + 1]), cc, minus), s[j], s[j + 1]);
                    s[j] = ex2(s[j]);
                    s[j + 1] = ex2(s[j + 1]);
                }
                if (!(cols >= kCols && j0 + kCols - 1 <= it.p0 && (it.p0 + it.rows - 1 - j0 < a.window || j0 + kCols <= a.sinks))) {
                    const int end = min(cols, p - j0 + 1), begin = p - a.window + 1 - j0, sink = max(a.sinks - j0, 0);
                    if (__any_sync(0xffffffffu, end < kCols)) {
#pragma unroll
                        for (int j = 0; j < kCols; ++j) s[j] = j < end ? s[j] : 0.f;
                    }
                    if (__any_sync(0xffffffffu, sink < begin)) {
#pragma unroll
                        for (int j = 0; j < kCols; ++j) s[j] = (int)(j >= begin) | (int)(j < sink) ? s[j] : 0.f;
                    }
                }
                if (!(ok = bar_all(1, kLanes, warp != 0 || wait(kPF, (from + t) & 1)))) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < kCols; q += 32) {
                    float g[32];
                    uint32_t w[16];
                    tmem_ld32(tp + q, (uint32_t *)g);
                    tmem_ld_wait();
                    if (it.ragged(t)) {  // (dP is not finite where a key outside the sequence is not)
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = s[q + j] == 0.f ? 0.f : g[j];
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = pack_bf16(s[q + 2 * j] * (g[2 * j] - d), s[q + 2 * j + 1] * (g[2 * j + 1] - d));
                    tmem_st16(tp + q / 2, w);  // (over columns that are read already)
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kZB]);
            }
            from += it.nt;
            first_unit += 2 + 2 * it.nt;
            if (!ok || !(ok = bar_all(1, kLanes, warp != 0 || (wait(kDone, n & 1) && wait(kFull + (first_unit - 1) % G::kRing, ((first_unit - 1) / G::kRing) & 1)))))
                break;
            ++n;
            tc_fence_after();
            // the products go on with the next tile of queries while this one's gradient is stored
            const int t0 = it.t0, rows = it.rows, h = it.h, nt = it.nt;
            take();
            uint8_t *const tile = sm + unit(first_unit - 1);
#pragma unroll
            for (int q = 0; q < D / kGroups; q += 32) {
                const int col = x * (D / kGroups) + q;
                float o[32];
                if (nt > 0) {
                    tmem_ld32(tmem + lanes + kQ + col, (uint32_t *)o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = nt > 0 ? o[j] * a.scale : 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 8) *(uint4 *)(tile + (col >> 6) * kBox + sw128(r, (col & 63) + j)) = pack8(o + j);
            }
            fence_proxy_async();
            bar_sync(1, kLanes);
            place = (first_unit - 1) % G::kRing;
            if (rows == kTile) {
                if (tid == 0) {
#pragma unroll
                    for (int b = 0; b < G::kBoxes; ++b) tma_store_3d(&maps.dq, tile + b * kBox, b * 64, h, t0);
                    tma_store_commit();
                    stored = true;
                }
            } else {
                copy_rows<D, kLanes>(a.dq, tile, t0, rows, a.H, h, tid);
                bar_sync(1, kLanes);
                if (tid == 0) mbar_arrive(&bar[kEmpty + place]);
            }
        }
        if (tid == 0) tma_store_wait0();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kLoads) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

// ---------------------------------------------------------------- dK, dV (lane = key)
constexpr int kSinkRun = 1024;   // queries of a CTA that sums for a tile of sinks where the window does not reach
constexpr int kMostSinkTiles = 4;  // (more tiles of sinks share the work among them)

template <int D>
__global__ void __launch_bounds__(kThreads, 1) win_dkv_kernel(const __grid_constant__ Maps maps, const WinArgs a, const WinSinks sinks, int64_t key_tiles,
                                                              uint64_t limit, int withhold)
{
    using G = Geo<D>;
    constexpr uint32_t kS = 0, kP = 128, kV = 256, kK = 384;  // S^T (P^T in its place), dP^T (Z^T), dV, dK
    extern __shared__ uint8_t win_bwd_smem[];
    uint8_t *const sm = win_bwd_smem + (-smem_u32(win_bwd_smem) & 1023u);  // (an offset: a cast would lose that it is shared memory)
    const int hk = blockIdx.y, per = a.H / a.HK;
    const WinKeyTile kt(a, sinks, key_tiles, kTile, kSinkRun, blockIdx.x, hk);
    if (kt.cols <= 0) return;
    const SeqRange sq = kt.sq, sk = kt.sk;
    const int n = kt.n, j0 = kt.j0, cols = kt.cols, off = kt.off, begin = kt.begin, end = kt.end;
    float *const part = kt.part;
    const int tiles = begin < end ? (end - begin + kTile - 1) / kTile : 0, nt = tiles * per;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *bar = (uint64_t *)(sm + G::kBars);
    uint32_t *tslot = (uint32_t *)(bar + kNumBars);
    if (tid == 0) init_bars(bar, G::kRing);
    if (tid == 32) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.dout);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    if (warp == kLoads) tmem_alloc(tslot, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, base = smem_u32(sm);
    unsigned *const status = &g_win_bwd_status;
    auto wait = [&](int b, uint32_t parity) { return mbar_wait(&bar[b], parity, status, kStatusTimeout, limit); };
    auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    auto full = [&](int i) { return all(wait(kFull + i % G::kRing, (i / G::kRing) & 1)); };  // unit 2 t: Q, 2 t + 1: dO
    auto unit = [&](int i) { return G::kRingAt + (i % G::kRing) * G::kUnit; };
    auto query0 = [&](int t) { return begin + (t % tiles) * kTile; };
    auto head = [&](int t) { return hk * per + t / tiles; };
    auto ragged = [&](int t) { return query0(t) + kTile > sq.len; };

    if (warp == kLoads) {
        // ---------------------------------------------------------------- loads
        bool ok = !withhold;
        if (ok && elect_one_sync()) {
            mbar_arrive_expect_tx(&bar[kIn], 2 * G::kUnit);
#pragma unroll
            for (int b = 0; b < G::kBoxes; ++b) {
                tma_load_3d(sm + G::kA + b * kBox, &maps.k, b * 64, hk, (int)(sk.bos + j0), &bar[kIn]);
                tma_load_3d(sm + G::kB + b * kBox, &maps.v, b * 64, hk, (int)(sk.bos + j0), &bar[kIn]);
            }
        }
        __syncwarp();
        int i = 0, mended = 0;
        for (; i < 2 * nt && ok; ++i) {
            const int s = i % G::kRing, t = i >> 1;
            if (i >= G::kRing && !(ok = all(wait(kEmpty + s, (i / G::kRing - 1) & 1)))) break;
            // rows behind the end are the next sequence's, and 0 x NaN is NaN: they are zeroed before the tile counts as full
            const bool mend = ragged(t);
            uint64_t *const landing = &bar[mend ? (int)kLanded : kFull + s];
            if (elect_one_sync()) {
                mbar_arrive_expect_tx(landing, G::kUnit);
#pragma unroll
                for (int b = 0; b < G::kBoxes; ++b)
                    tma_load_3d(sm + unit(i) + b * kBox, i & 1 ? &maps.dout : &maps.q, b * 64, head(t), (int)(sq.bos + query0(t)), landing);
            }
            __syncwarp();
            if (mend) {
                if (!(ok = all(wait(kLanded, mended++ & 1)))) break;
                zero_rows<G::kBoxes>(sm + unit(i), sq.len - query0(t));
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kFull + s]);
            }
        }
        if (!withhold) wait(kIn, 0);
        for (int k = max(0, i - G::kRing); k < i; ++k) wait(kFull + k % G::kRing, (k / G::kRing) & 1);  // (no copy outlives the CTA)
    } else if (warp == kProducts) {
        // ---------------------------------------------------------------- products: dV(t), S(t+1), dK(t), dP(t+1)
        auto scores = [&](int t) {
            tc_fence_after();
            if (elect_one_sync()) {
                mma_rows<D>(tmem + kS, base + G::kA, base + unit(2 * t));
                mma_commit(&bar[kSF]);
            }
            __syncwarp();
        };
        auto slopes = [&](int t) {
            tc_fence_after();
            if (elect_one_sync()) {
                mma_rows<D>(tmem + kP, base + G::kB, base + unit(2 * t + 1));
                mma_commit(&bar[kPF]);
            }
            __syncwarp();
        };
        bool ok = all(wait(kIn, 0));
        if (ok && nt > 0 && (ok = full(0))) {
            scores(0);
            if ((ok = full(1))) slopes(0);
        }
        for (int t = 0; t < nt && ok; ++t) {
            if (!(ok = all(wait(kPB, t & 1)))) break;
            tc_fence_after();
            if (elect_one_sync()) {
                mma_sum<D>(tmem + kV, tmem + kS, base + unit(2 * t + 1), t == 0);
                mma_commit(&bar[kEmpty + (2 * t + 1) % G::kRing]);
            }
            __syncwarp();
            if (t + 1 < nt) {
                if (!(ok = full(2 * t + 2))) break;
                scores(t + 1);
            }
            if (!(ok = all(wait(kZB, t & 1)))) break;
            tc_fence_after();
            if (elect_one_sync()) {
                mma_sum<D>(tmem + kK, tmem + kP, base + unit(2 * t), t == 0);
                mma_commit(&bar[kEmpty + (2 * t) % G::kRing]);
            }
            __syncwarp();
            if (t + 1 < nt) {
                if (!(ok = full(2 * t + 3))) break;
                slopes(t + 1);
            }
        }
        if (elect_one_sync()) mma_commit(&bar[kDone]);
        __syncwarp();
        wait(kDone, 0);
    } else {
        const int x = warp >> 2, r = tid & 127, j = j0 + r;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kS + kCols * x, tp = tmem + lanes + kP + kCols * x;
        const float c = a.scale * kLog2e;
        float *const stats = (float *)(sm + G::kStats) + x * 2 * kCols;  // [lse, delta][the group's queries]
        // this thread's number of tile t: lse (the first half of a group) or delta (the second) of one of the group's queries
        auto stat = [&](int t) {
            const int i = query0(t) + kCols * x + (r & (kCols - 1));
            if (i >= end) return r < kCols ? INFINITY : 0.f;  // weights of zero
            const int64_t at = lse_at(a, n, sq.bos, head(t)) + i;
            if (r >= kCols) return a.delta[at];
            const float l = a.lse[at] * kLog2e;
            return l == -INFINITY ? INFINITY : l;
        };
        float next = nt > 0 ? stat(0) : 0.f;
        bool ok = true;
        for (int t = 0; t < nt; ++t) {
            const int i0 = query0(t) + kCols * x, q0 = i0 + off, rows = min(end - i0, kCols);  // (the group's queries)
            float *const ls = stats, *const dl = ls + kCols;
            // (each is read between one of the two barriers and the other)
            const float now = next;
            if (r < kCols) ls[r] = now;
            if (t + 1 < nt) next = stat(t + 1);
            if (!(ok = bar_all(1 + x, 128, (warp & 3) || wait(kSF, t & 1)))) break;  // (the group leaves together)
            if (r >= kCols) ls[r] = now;
            tc_fence_after();
            float s[kCols];
#pragma unroll
            for (int q = 0; q < kCols; q += 32) tmem_ld32(ts + q, (uint32_t *)s + q);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < kCols; k += 4) {
                const float4 l = *(const float4 *)(ls + k);
                s[k] = ex2(fmaf(s[k], c, -l.x));
                s[k + 1] = ex2(fmaf(s[k + 1], c, -l.y));
                s[k + 2] = ex2(fmaf(s[k + 2], c, -l.z));
                s[k + 3] = ex2(fmaf(s[k + 3], c, -l.w));
            }
            if (!(rows == kCols && j0 + kTile - 1 <= q0 && (q0 + kCols - 1 - j0 < a.window || j0 + kTile <= a.sinks))) {
                const int first = j - q0, last = j < a.sinks ? rows : (int)min((int64_t)rows, (int64_t)j + a.window - q0);
                if (__any_sync(0xffffffffu, first > 0)) {
#pragma unroll
                    for (int k = 0; k < kCols; ++k) s[k] = k >= first ? s[k] : 0.f;
                }
                if (__any_sync(0xffffffffu, last < kCols)) {
#pragma unroll
                    for (int k = 0; k < kCols; ++k) s[k] = k < last ? s[k] : 0.f;
                }
            }
#pragma unroll
            for (int q = 0; q < kCols; q += 32) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = pack_bf16(s[q + 2 * k], s[q + 2 * k + 1]);
                tmem_st16(ts + q / 2, w);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kPB]);
            if (!(ok = bar_all(1 + x, 128, (warp & 3) || wait(kPF, t & 1)))) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < kCols; q += 32) {
                float g[32];
                uint32_t w[16];
                tmem_ld32(tp + q, (uint32_t *)g);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 d = *(const float4 *)(dl + q + k);
                    const float *u = s + q + k;
                    w[k / 2] = pack_bf16(u[0] * (g[k] - d.x), u[1] * (g[k + 1] - d.y));
                    w[k / 2 + 1] = pack_bf16(u[2] * (g[k + 2] - d.z), u[3] * (g[k + 3] - d.w));
                }
                tmem_st16(tp + q / 2, w);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kZB]);
        }
        // ---------------------------------------------------------------- dV by the first group, dK by the second
        const bool key = x != 0;
        ok = bar_all(1 + x, 128, ((warp & 3) || wait(kDone, 0)) && ok);
        if (ok) {
            tc_fence_after();
            const float f = key ? a.scale : 1.f;
            uint8_t *tile = sm + (key ? G::kA : G::kB);  // (K's and V's last products are taken)
#pragma unroll
            for (int col = 0; col < D; col += 32) {
                float o[32];
                if (nt > 0) {
                    tmem_ld32(tmem + lanes + (key ? kK : kV) + col, (uint32_t *)o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = nt > 0 ? o[k] * f : 0.f;
                if (part) {
                    float *dst = part + ((int64_t)(1 - key) * kTile + r) * D + col;  // dK, then dV
#pragma unroll
                    for (int k = 0; k < 32; k += 4) *(float4 *)(dst + k) = *(const float4 *)&o[k];
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) *(uint4 *)(tile + (col >> 6) * kBox + sw128(r, (col & 63) + 8 * k)) = pack8(o + 8 * k);
                }
            }
            if (!part) {
                fence_proxy_async();
                bar_sync(1 + x, 128);
                if (cols < kTile) {
                    copy_rows<D, 128>(key ? a.dk : a.dv, tile, sk.bos + j0, cols, a.HK, hk, r);
                } else if (r == 0) {
#pragma unroll
                    for (int b = 0; b < G::kBoxes; ++b) tma_store_3d(key ? &maps.dk : &maps.dv, tile + b * kBox, b * 64, hk, (int)(sk.bos + j0));
                    tma_store_commit();
                    tma_store_wait0();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kLoads) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

// dK and dV of the tiles of sinks: their own part and the runs', in order
template <int D>
__global__ void __launch_bounds__(256) win_sinks_kernel(const WinArgs a, const WinSinks s)
{
    const int which = blockIdx.z, st = blockIdx.y % s.tiles, hk = blockIdx.y / s.tiles;
    const int n = win_sinks_at(a, s, blockIdx.x / (kTile * D / 1024)), e = (blockIdx.x % (kTile * D / 1024)) * 1024 + threadIdx.x * 4, r = st * kTile + e / D;
    if (n < 0) return;
    const SeqRange sk = seq_range(a.cu_k, n, a.Tk);
    if (r >= sk.len) return;
    const float4 x = win_sinks_sum<float4>(a, s, kTile, kSinkRun, n, hk, st, (int64_t)which * kTile * D + e);
    __nv_bfloat16 *dst = (__nv_bfloat16 *)(which ? a.dv : a.dk) + ((sk.bos + r) * a.HK + hk) * D + e % D;
    *(uint2 *)dst = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

template <int D>
cudaError_t launch(const WinArgs &a, int64_t tq, int64_t tk, float *delta, void *ws, cudaStream_t st)
{
    Maps maps;
    if (!heads_map(&maps.q, a.q, D, a.H, tq, a.ldq, kTile) || !heads_map(&maps.k, a.k, D, a.HK, tk, a.ldk, kTile) ||
        !heads_map(&maps.v, a.v, D, a.HK, tk, a.ldv, kTile) || !heads_map(&maps.dout, a.dout, D, a.H, tq, a.ld_dout, kTile) ||
        !strided_map(&maps.o, a.o, D, a.H, a.Tq, a.cu_q ? 1 : a.N, a.o_head, a.o_tok, a.o_seq, kTile) || !heads_map(&maps.dq, a.dq, D, a.H, tq, (int64_t)a.H * D, kTile) ||
        !heads_map(&maps.dk, a.dk, D, a.HK, tk, (int64_t)a.HK * D, kTile) ||
        !heads_map(&maps.dv, a.dv, D, a.HK, tk, (int64_t)a.HK * D, kTile))
        return cudaErrorInvalidValue;
    constexpr int smem = Geo<D>::kSmem;
    static std::atomic<uint64_t> seen;
    if (first_on_device(seen)) {
        cudaError_t e = cudaFuncSetAttribute(win_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(win_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        done_on_device(seen);
    }
    size_t bytes;
    const WinSinks s = win_sinks_plan(a, kTile, kSinkRun, kMostSinkTiles, ws, &bytes);
    const int64_t qt = mix_slots(a.cu_q != nullptr, a.N, a.Tq, kTile), kt = mix_slots(a.cu_k != nullptr, a.N, a.Tk, kTile);
    const int64_t ctas = kt + s.slots * s.tiles;
    if (qt * a.H > INT32_MAX || ctas > INT32_MAX || s.places * kTile * D / 1024 > INT32_MAX) return cudaErrorInvalidConfiguration;
    const int withhold = withhold_loads();
    const uint64_t limit = withhold ? kTestWaitLimitNs : kWaitLimitNs;
    win_dq_kernel<D><<<(unsigned)std::min<int64_t>(qt * a.H, device_sm_count()), kThreads, smem, st>>>(maps, a, (unsigned)(qt * a.H), delta, limit, withhold);
    win_dkv_kernel<D><<<dim3((unsigned)ctas, a.HK), kThreads, smem, st>>>(maps, a, s, kt, limit, withhold);
    if (s.tiles > 0) win_sinks_kernel<D><<<dim3((unsigned)(s.places * (kTile * D / 1024)), a.HK * s.tiles, 2), 256, 0, st>>>(a, s);
    return cudaGetLastError();
}

}  // namespace

bool win_bwd_tc_ok(const WinArgs &a, int64_t tq, int64_t tk)
{
    const int64_t strides[] = {a.H > 1 ? a.o_head : 8, a.Tq > 1 ? a.o_tok : 8, !a.cu_q && a.N > 1 ? a.o_seq : 8};
    for (int64_t s : strides)
        if (s < 8 || s % 8 || s >= (int64_t)1 << 38) return false;
    return win_tc_ok(a, tq, tk) && tma_ok(a.dout, a.ld_dout, tq, 2) && !(((uintptr_t)a.dq | (uintptr_t)a.dk | (uintptr_t)a.dv) & 15) &&
           a.HK * kMostSinkTiles <= 65535;
}

size_t win_bwd_tc_bytes(const WinArgs &a)
{
    size_t bytes;
    win_sinks_plan(a, kTile, kSinkRun, kMostSinkTiles, nullptr, &bytes);
    return bytes;
}

cudaError_t launch_win_bwd_tc(const WinArgs &a, int64_t tq, int64_t tk, float *delta, void *ws, cudaStream_t st)
{
    return a.D == 64 ? launch<64>(a, tq, tk, delta, ws, st) : launch<128>(a, tq, tk, delta, ws, st);
}

gdn_status read_win_bwd_status(cudaStream_t st)
{
    unsigned word = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, g_win_bwd_status, sizeof(word), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_win_bwd_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return word & kStatusTimeout ? GDN_ERR_TIMEOUT : GDN_OK;
}

}  // namespace gdn
