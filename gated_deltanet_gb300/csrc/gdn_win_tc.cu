// Attention with a sliding window and sinks on the tensor cores, forward: bf16, heads of 64 or 128, rows on 16-byte boundaries.
//
// One CTA takes two tiles A and B of 128 queries (two query heads of one key head where there are such, else neighbouring rows), walks
// the tiles of 128 keys that they see (the sinks, then the window from its first key on) and keeps two scores' tiles and two outputs in
// tensor memory: while the tensor cores work for one tile, the other's warps take their softmax.  Per tile of keys:
//   S = Q K^T,  P = exp2(c S - m) (bf16, in S's place),  O += P V            c = scale log2 e
// in one pass over the keys.  m is a row's maximum as it was last raised: O and the sum are brought to a new one only when a score
// passes the old by more than 8 (P then stays below 2^8, in fp32's and bf16's range; the rounding of P is relative), so that most
// tiles leave O alone (the one-pass softmax of Milakov and Gimelshein, 2018, in the later published form that puts small raises off).
//
// Warps: 0-7 and 8-15 softmax of A and B and their outputs (two threads to a row: with one a tile's softmax took 3800 cycles, one warp to
// a scheduler and side having nothing to hide its latencies behind), 16 loads (a ring of K and V tiles) and zeroes the V rows behind a
// sequence's end (they are the next sequence's, and 0 x NaN is NaN), 17 products.
// The products are issued S_A(t), PV_B(t-1), S_B(t), PV_A(t): S(t) is complete only when PV(t-1) is, which is why a softmax that sees
// its scores may also touch its O.
// 4 x 4096 tokens, 16 heads over 4 of 128, window 1024: 146 us, 822 TFLOP/s; of 64 138.  S with both operands in shared memory takes 104 cycles a
// product where the arithmetic takes 64, with P V (67 of 64) 84 us of the 146; the rest are a CTA's start and end and the softmax between its nine tiles.
#include "gdn_mix.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kTile = 128, kThreads = 640, kBox = kTile * 128;
constexpr uint32_t kS = 0, kO = 256, kTmem = 512;  // + 128 for tile B
constexpr float kRaise = 8.f;

__device__ unsigned g_win_status;

template <int D>
struct Geo {
    static constexpr int kBoxes = D / 64, kUnit = kBoxes * kBox;
    static constexpr int kRing = D == 128 ? 4 : 8;  // K and V tiles in flight
    static constexpr int kQ = 0, kKV = 2 * kUnit, kRed = kKV + kRing * kUnit, kBars = kRed + 2048, kSmem = kBars + 256 + 1024;
};
enum Bar { kQF, kSF = kQF + 2, kPB = kSF + 2, kDone = kPB + 2, kLanded = kDone + 2, kFin, kFull, kMostRing = 8, kEmpty = kFull + kMostRing, kNumBars = kEmpty + kMostRing };

struct Maps {
    CUtensorMap q, k, v, o;
};

// What one of the two tiles is
struct Side {
    int i0, rows, h, p0;  // first query, how many (0: none), head, position of the first
    int lo, hi;           // keys its rows may see beside the sinks
    __device__ bool needs(int j0, int sinks) const { return rows > 0 && j0 < hi && (j0 + kTile > lo || j0 < sinks); }
    __device__ bool whole(int j0, int cols, int window, int sinks) const
    {
        // of the 64 keys from j0 on
        return cols >= 64 && j0 + 63 <= p0 && (p0 + rows - 1 - j0 < window || j0 + 64 <= sinks);
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) win_tc_kernel(const __grid_constant__ Maps maps, const WinArgs a, int by_heads, uint64_t limit, int withhold)
{
    using G = Geo<D>;
    extern __shared__ uint8_t win_tc_smem[];
    uint8_t *const sm = win_tc_smem + (-smem_u32(win_tc_smem) & 1023u);  // (an offset: a cast would lose that it is shared memory)
    const Tile tl = tile_of(a.cu_q, a.N, a.Tq, by_heads ? kTile : 2 * kTile, blockIdx.x);
    const SeqRange sq = seq_range(a.cu_q, tl.n, a.Tq), sk = seq_range(a.cu_k, tl.n, a.Tk);
    const int h0 = by_heads ? 2 * blockIdx.y : blockIdx.y, hk = h0 / (a.H / a.HK), off = sk.len - sq.len;
    auto side_of = [&](int x) {
        Side s;
        s.i0 = by_heads ? tl.index * kTile : (2 * tl.index + x) * kTile;
        s.rows = min(kTile, sq.len - s.i0);
        s.h = by_heads ? h0 + x : h0;
        s.p0 = s.i0 + off;
        s.hi = min(max(s.p0 + s.rows, 0), sk.len);
        s.lo = min(max(s.p0 - a.window + 1, 0), s.hi);
        return s;
    };
    const Side A = side_of(0), B = side_of(1);
    if (A.rows <= 0) return;
    const int hi = B.rows > 0 ? max(A.hi, B.hi) : A.hi, lo = A.lo;
    const int first = min(a.sinks, lo), nfirst = (first + kTile - 1) / kTile, nt = nfirst + (hi - lo + kTile - 1) / kTile;
    auto key0 = [&](int t) { return t < nfirst ? t * kTile : lo + (t - nfirst) * kTile; };
    auto columns = [&](int t) { return min(kTile, (t < nfirst ? first : hi) - key0(t)); };
    auto ragged = [&](int t) { return key0(t) + kTile > sk.len; };  // rows of the next sequence in it

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *bar = (uint64_t *)(sm + G::kBars);
    uint32_t *tslot = (uint32_t *)(bar + kNumBars);
    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bar[kQF + x], 1);
            mbar_init(&bar[kSF + x], 1);
            mbar_init(&bar[kPB + x], 8);
            mbar_init(&bar[kDone + x], 1);
        }
        mbar_init(&bar[kLanded], 1);
        mbar_init(&bar[kFin], 1);
        for (int i = 0; i < G::kRing; ++i) {
            mbar_init(&bar[kFull + i], 1);
            mbar_init(&bar[kEmpty + i], 1);
        }
        fence_mbar_init();
    }
    if (tid == 32) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    if (warp == 16) tmem_alloc(tslot, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, base = smem_u32(sm);
    unsigned *const status = &g_win_status;
    auto wait = [&](int b, uint32_t parity) { return mbar_wait(&bar[b], parity, status, kStatusTimeout, limit); };
    auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    // unit i of the ring: K of tile i / 2, or its V
    auto full = [&](int i) { return all(wait(kFull + i % G::kRing, (i / G::kRing) & 1)); };

    if (warp == 16) {
        // ---------------------------------------------------------------- loads
        bool ok = !withhold;
        auto queries = [&](int x) {
            if (elect_one_sync()) {
                mbar_arrive_expect_tx(&bar[kQF + x], G::kUnit);
#pragma unroll
                for (int b = 0; b < G::kBoxes; ++b)
                    tma_load_3d(sm + G::kQ + x * G::kUnit + b * kBox, &maps.q, b * 64, x ? B.h : A.h, (int)(sq.bos + (x ? B.i0 : A.i0)), &bar[kQF + x]);
            }
            __syncwarp();
        };
        // (without keys nothing waits for B's queries: they would land on its outputs)
        const bool both = ok && B.rows > 0 && nt > 0;
        if (ok) queries(0);
        int i = 0, mended = 0;
        for (; i < 2 * nt && ok; ++i) {
            const int s = i % G::kRing;
            if (i >= G::kRing && !(ok = all(wait(kEmpty + s, (i / G::kRing - 1) & 1)))) break;
            // V's rows behind the end are the next sequence's, and 0 x NaN is NaN: they are zeroed before the tile counts as full
            const bool mend = (i & 1) && ragged(i >> 1);
            uint64_t *const landing = &bar[mend ? (int)kLanded : kFull + s];
            if (elect_one_sync()) {
                mbar_arrive_expect_tx(landing, G::kUnit);
#pragma unroll
                for (int b = 0; b < G::kBoxes; ++b)
                    tma_load_3d(sm + G::kKV + s * G::kUnit + b * kBox, i & 1 ? &maps.v : &maps.k, b * 64, hk, (int)(sk.bos + key0(i >> 1)), landing);
            }
            __syncwarp();
            if (both && i == 0) queries(1);  // (behind what the first scores wait for)
            if (mend) {
                if (!(ok = all(wait(kLanded, mended++ & 1)))) break;
                uint8_t *v = sm + G::kKV + s * G::kUnit;
#pragma unroll
                for (int b = 0; b < G::kBoxes; ++b)
                    for (int e = (sk.len - key0(i >> 1)) * 8 + lane; e < kTile * 8; e += 32) *(uint4 *)(v + b * kBox + e * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kFull + s]);
            }
        }
        if (!withhold) wait(kQF, 0);
        if (both) wait(kQF + 1, 0);
        for (int k = max(0, i - G::kRing); k < i; ++k) wait(kFull + k % G::kRing, (k / G::kRing) & 1);  // (no copy outlives the CTA)
    } else if (warp == 17) {
        // ---------------------------------------------------------------- products
        const uint32_t idS = idesc_bf16_f32(128, 128, 0, 0), idO = idesc_bf16_f32(128, D, 0, 1);
        auto unit = [&](int i) { return base + G::kKV + (i % G::kRing) * G::kUnit; };
        auto scores = [&](int x, int t) {
            const uint64_t dq = sdesc_sw128(base + G::kQ + x * G::kUnit, 16, 1024), dk = sdesc_sw128(unit(2 * t), 16, 1024);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t o = ((ks >> 2) * kBox + (ks & 3) * 32) >> 4;
                mma_ss(tmem + kS + 128 * x, dq + o, dk + o, idS, ks > 0);
            }
            mma_commit(&bar[kSF + x]);
        };
        auto output = [&](int x, int t, bool fresh) {
            const uint64_t dv = sdesc_sw128(unit(2 * t + 1), kBox, 1024);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks) mma_ts(tmem + kO + 128 * x, tmem + kS + 128 * x + (ks >> 2) * 64 + (ks & 3) * 8, dv + ks * 128, idO, !fresh || ks > 0);
        };
        bool ok = all(wait(kQF, 0));
        int done[2] = {0, 0}, late = -1;  // late: the tile whose PV_B is still to come
        auto second = [&]() {  // PV_B(late)
            ok = all(wait(kPB + 1, done[1] & 1));
            if (!ok) return;
            tc_fence_after();
            if (elect_one_sync()) {
                output(1, late, done[1] == 0);
                mma_commit(&bar[kEmpty + (2 * late + 1) % G::kRing]);
            }
            __syncwarp();
            ++done[1];
            late = -1;
        };
        for (int t = 0; t < nt && ok; ++t) {
            const int j0 = key0(t);
            const bool needA = A.needs(j0, a.sinks), needB = B.needs(j0, a.sinks);
            if (!(ok = full(2 * t))) break;
            tc_fence_after();
            if (needA && elect_one_sync()) scores(0, t);
            __syncwarp();
            if (late >= 0) second();
            if (!ok) break;
            if (t == 0 && B.rows > 0 && !(ok = all(wait(kQF + 1, 0)))) break;
            if (elect_one_sync()) {
                if (needB) scores(1, t);
                mma_commit(&bar[kEmpty + (2 * t) % G::kRing]);
            }
            __syncwarp();
            if (!(ok = full(2 * t + 1))) break;
            if (needA) {
                if (!(ok = all(wait(kPB, done[0] & 1)))) break;
                tc_fence_after();
                if (elect_one_sync()) output(0, t, done[0] == 0);
                __syncwarp();
                ++done[0];
            }
            if (needB) late = t;
            else {
                if (elect_one_sync()) mma_commit(&bar[kEmpty + (2 * t + 1) % G::kRing]);
                __syncwarp();
            }
        }
        if (elect_one_sync()) mma_commit(&bar[kDone]);
        __syncwarp();
        if (ok && late >= 0) second();
        if (elect_one_sync()) {
            mma_commit(&bar[kDone + 1]);
            mma_commit(&bar[kFin]);  // every product has ended before the tensor memory goes
        }
        __syncwarp();
        wait(kFin, 0);
    } else if (warp < 16) {
        // ---------------------------------------------------------------- softmax (thread = half a row: 64 of a tile's keys)
        const int x = warp >> 3, half = warp >> 2 & 1, r = tid & 127, bar_id = 1 + x;
        const bool leads = (warp & 7) == 0;  // (one warp of a side polls, the others meet it: polls take instructions from those who work)
        const Side s = side_of(x);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, ts = tmem + lanes + kS + 128 * x, to = tmem + lanes + kO + 128 * x + half * (D / 2);
        const float c = a.scale * kLog2e;
        const int p = s.p0 + r;
        float *const red = (float *)(sm + G::kRed) + x * 256;  // [half][row]: the halves' maxima, last their sums
        float m = -INFINITY, l = 0.f;
        int done = 0;
        bool ok = true;
        for (int t = 0; t < nt; ++t) {
            const int j0 = key0(t) + 64 * half, cols = columns(t) - 64 * half;
            if (!s.needs(key0(t), a.sinks)) continue;
            if (!(ok = bar_all(bar_id, 256, !leads || wait(kSF + x, done & 1)))) break;
            tc_fence_after();
            float z[64];
            tmem_ld32(ts + 64 * half, (uint32_t *)z);
            tmem_ld32(ts + 64 * half + 32, (uint32_t *)z + 32);
            tmem_ld_wait();
            if (!s.whole(j0, cols, a.window, a.sinks)) {
                const int end = min(cols, p - j0 + 1), begin = p - a.window + 1 - j0, sink = max(a.sinks - j0, 0);
                if (__any_sync(0xffffffffu, end < 64)) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) z[j] = j < end ? z[j] : -INFINITY;
                }
                if (__any_sync(0xffffffffu, sink < begin)) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) z[j] = (int)(j >= begin) | (int)(j < sink) ? z[j] : -INFINITY;
                }
            }
            float top[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                top[q] = z[q];
#pragma unroll
                for (int j = 4 + q; j < 64; j += 4) top[q] = fmaxf(top[q], z[j]);
            }
            float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            mx *= c;
            if (bar_any(bar_id, 256, mx > m + kRaise)) {
                red[half * 128 + r] = mx;
                bar_sync(bar_id, 256);
                mx = fmaxf(mx, red[(half ^ 1) * 128 + r]);
                bar_sync(bar_id, 256);  // (the place is written again)
                const float raised = fmaxf(m, mx), f = m == -INFINITY ? 0.f : ex2(m - raised);
                l *= f;
                m = raised;
                if (done > 0) {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        float o[16];
                        tmem_ld16(to + 16 * q, (uint32_t *)o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= f;
                        tmem_st16(to + 16 * q, (const uint32_t *)o);
                    }
                }
            }
            const float mm = m == -INFINITY ? 0.f : m;
            const Pair cc = pair_of(c, c), minus = pair_of(-mm, -mm), one = pair_of(1.f, 1.f);
            Pair sum[2] = {pair_of(0.f, 0.f), pair_of(0.f, 0.f)};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float u, v;
                    unpair(fma2(pair_of(z[32 * q + 2 * j], z[32 * q + 2 * j + 1]), cc, minus), u, v);
                    u = ex2(u);
                    v = ex2(v);
                    sum[j & 1] = fma2(pair_of(u, v), one, sum[j & 1]);
                    w[j] = pack_bf16(u, v);
                }
                tmem_st16(ts + 64 * half + 16 * q, w);  // (in the place of this half's scores)
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kPB + x]);
            float u[4];
            unpair(sum[0], u[0], u[1]);
            unpair(sum[1], u[2], u[3]);
            l += (u[0] + u[1]) + (u[2] + u[3]);
            ++done;
        }
        // ---------------------------------------------------------------- outputs (thread = half a row)
        ok = bar_all(bar_id, 256, (!leads || wait(kDone + x, 0)) && ok);
        if (ok && s.rows > 0) {
            tc_fence_after();
            red[half * 128 + r] = l;
            bar_sync(bar_id, 256);
            l += red[(half ^ 1) * 128 + r];
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint8_t *tile = sm + G::kQ + x * G::kUnit;  // (the last scores are taken)
#pragma unroll
            for (int q = 0; q < D / 64; ++q) {
                const int col = half * (D / 2) + 32 * q;
                float o[32];
                if (done > 0) {
                    tmem_ld32(to + 32 * q, (uint32_t *)o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = done > 0 && l != 0.f ? o[j] * inv : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) *(uint4 *)(tile + (col >> 6) * kBox + sw128(r, (col & 63) + 8 * j)) = pack8(o + 8 * j);
            }
            if (half == 0 && a.lse && r < s.rows)
                a.lse[lse_at(a, tl.n, sq.bos, s.h) + s.i0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            fence_proxy_async();
            bar_sync(bar_id, 256);
            const int64_t t0 = sq.bos + s.i0;
            if (s.rows == kTile) {
                if (half == 0 && r == 0) {
#pragma unroll
                    for (int b = 0; b < G::kBoxes; ++b) tma_store_3d(&maps.o, tile + b * kBox, b * 64, s.h, (int)t0);
                    tma_store_commit();
                    tma_store_wait0();
                }
            } else {
                for (int k = half * 128 + r; k < s.rows * (D / 8); k += 256) {
                    const int row = k / (D / 8), e = k % (D / 8) * 8;
                    *(uint4 *)((__nv_bfloat16 *)a.o + ((t0 + row) * a.H + s.h) * D + e) = *(const uint4 *)(tile + (e >> 6) * kBox + sw128(row, e & 63));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

template <int D>
cudaError_t launch(const WinArgs &a, int64_t tq, int64_t tk, cudaStream_t st)
{
    Maps maps;
    if (!heads_map(&maps.q, a.q, D, a.H, tq, a.ldq, kTile) || !heads_map(&maps.k, a.k, D, a.HK, tk, a.ldk, kTile) ||
        !heads_map(&maps.v, a.v, D, a.HK, tk, a.ldv, kTile) || !heads_map(&maps.o, a.o, D, a.H, tq, (int64_t)a.H * D, kTile))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> seen;
    if (first_on_device(seen)) {
        const cudaError_t e = cudaFuncSetAttribute(win_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
        if (e != cudaSuccess) return e;
        done_on_device(seen);
    }
    const int by_heads = (a.H / a.HK) % 2 == 0;
    const int64_t tiles = mix_slots(a.cu_q != nullptr, a.N, a.Tq, by_heads ? kTile : 2 * kTile);
    if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
    const int withhold = withhold_loads();
    win_tc_kernel<D><<<dim3((unsigned)tiles, by_heads ? a.H / 2 : a.H), kThreads, Geo<D>::kSmem, st>>>(maps, a, by_heads, withhold ? kTestWaitLimitNs : kWaitLimitNs, withhold);
    return cudaGetLastError();
}

}  // namespace

bool win_tc_ok(const WinArgs &a, int64_t tq, int64_t tk)
{
    // (a scale that is not positive would turn the order of the scores)
    return (a.D == 64 || a.D == 128) && a.scale > 0.f && tq > 0 && tk > 0 && tq <= INT32_MAX - kTile && tk <= INT32_MAX - kTile &&
           tma_ok(a.q, a.ldq, tq, 2) && tma_ok(a.k, a.ldk, tk, 2) && tma_ok(a.v, a.ldv, tk, 2) && !((uintptr_t)a.o & 15);
}

cudaError_t launch_win_tc(const WinArgs &a, int64_t tq, int64_t tk, cudaStream_t st)
{
    return a.D == 64 ? launch<64>(a, tq, tk, st) : launch<128>(a, tq, tk, st);
}

gdn_status read_win_status(cudaStream_t st)
{
    unsigned word = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, g_win_status, sizeof(word), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_win_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return word & kStatusTimeout ? GDN_ERR_TIMEOUT : GDN_OK;
}

}  // namespace gdn
