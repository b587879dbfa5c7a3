// Linear attention with a decay for each head on the tensor cores: bf16, heads of 64 or 128 (K = V), rows on 16-byte boundaries.
//
// One CTA per (sequence or segment of one, value head, 64 columns of c) walks chunks of 128 tokens; the state X (D x 64, fp32)
// stays in tensor memory, or in registers.  Per chunk of n tokens, forward in time, every product a tcgen05 MMA with M = 128:
//   Z = a b^T                   (128 x 128)   Z_ij <- cs l^(i-j) Z_ij for j <= i, rounded to bf16 where it lies
//   O1 = a X,  O2 = Z c         (128 x 64)    out_i = os (l^(i+1) O1_i + O2_i)
//   X <- l^n X + b^T C          (D x 64)      C_j = cs l^(n-1-j) c_j as the sum of two or three bf16 values
// Against time the same with the powers counted from the chunk's other end.
// X enters O1 rounded to bf16, and b and c go in as they are.  C:
//  - Where a pass returns X (RETURNED; fp32) C goes into it as three bf16 values, 24 bits, and X is summed in registers: the accumulators begin at
//    zero in each chunk, because the tensor cores cut off what a small product has below a large sum, chunk after chunk.  X is then off by 1e-7
//    to 3e-7 of its 2-norm, as plain fp32 sums are.
//  - Where only outputs in bf16 (or the fp32 parts of bf16 gradients) see X, C goes in as hi + lo, 16 bits of it, and X is the accumulators' sum, which
//    leaves X 2.4e-6 of its 2-norm off, a 700th of the rounding with which it enters O1.
//
// Bound by shared memory: it gives the products about 80 bytes a cycle, so that one of 128 x 128 x 16 with both operands there takes
// 104 cycles (64 for the arithmetic), 128 x 64 x 16 takes 76, with its left operand in tensor memory 46, and it serves the copies and
// the warps beside them.  A chunk's products are 2640 cycles alone and about 3700 so; a chunk takes 4100.  Hence: hi and lo lie next to
// each other and go in as one right operand of 128 columns (X is the sum of two accumulators); outputs go from registers to memory.
// The third part is 608 cycles of products more and takes one of c's three stages.
// 4 x 4096 tokens of 16 heads of 128 80 us, 94 with the states returned (92 with X in the accumulators, whose sums leave slow decays 1.3e-6 off).
// A whole head to a CTA has the cheaper products (N = 128, X transposed, C in tensor memory) but half the CTAs and most of its
// CUDA-core work on the chain from chunk to chunk: 138 us where this took 80.
//
// Warps: 0 loads (TMA: two stages of a and b, three (two) of c, which is done with later; zeroes the rows behind a sequence's end, which are
// the next one's: 0 x NaN is NaN), 1 issues the products, 4-7 turn Z, 8-15 round and decay X, 16-19 write out, 20-27 scale and split c.
// One warp of a role polls a barrier and the others wait for it at a named one, which takes no instructions (polled by every waiting
// warp, 10 000 of a chunk's 24 500 instructions were polls).  Order of the products: X(m+1), O1(m), Z(m+1), O2(m); X is read, rounded
// and decayed, and c split, while the last three run.
#include <cudaTypedefs.h>

#include "gdn_mix.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kC = 128, kCols = 64, kThreads = 896, kStages = 2, kStagesC = 3, kBox = kC * 128;
// tensor-memory columns: Z (two buffers), the outputs, the state's two accumulators
constexpr uint32_t kZ = 0, kO1 = 256, kO2 = 320, kX = 384, kTmem = 512;

__device__ unsigned g_lin_status;

template <int D>
struct Geo {
    static constexpr int kBoxes = D / 64;
    static constexpr int kA = 0, kB = kBoxes * kBox, kStage = 2 * kBoxes * kBox;  // a and b; c in a ring of its own
    static constexpr int kCs = kStages * kStage, kXs = kCs + kStagesC * kBox, kParts = kXs + kBox, kBars = kParts + 2 * kBox, kSmem = kBars + 256 + 1024;
};
enum Bar { kFull, kEmpty = kFull + kStages, kFullC = kEmpty + kStages, kEmptyC = kFullC + kStagesC, kZF = kEmptyC + kStagesC, kZB = kZF + 2, kLanded = kZB + 2, kXB, kCB, kXF, kO1F, kOF, kOE, kFin, kNumBars };

struct Maps {
    CUtensorMap a[3], b[3], c[3];
};

constexpr float kAgain = 1.6f, kLaunches = 8.f;  // a split's walk in walks, its further launches in chunks (lin_tc_plan)

inline bool several(const LinArgs &a) { return a.cu && a.N > 1; }

struct Split {
    float *held;    // [passes][states][HV][D][D]: what a segment adds to the state, then the state that enters it; null: one segment each
    int tokens;     // of a segment (a multiple of kC)
    int64_t states;
    const int *chosen;  // packed: a multiple of `tokens` that lin_choose_kernel took, and whether a sequence is longer; nullable
    __device__ int segment() const { return chosen ? *chosen : tokens; }
    __device__ bool none() const { return chosen && !chosen[1]; }  // no sequence is cut
};

// A CTA's part of a sequence, in the order of processing
struct Part {
    SeqRange s;
    int chunks, m0, nm, seg;  // of the sequence; the first one's place, how many; which segment
    // (held: slots are those of the segments' states)
    __device__ Part(const LinArgs &a, bool split, bool held, int tokens, int64_t slot, int &n)
    {
        const Tile t = !split ? Tile{(int)slot, 0} : held ? cut_of(a.cu, a.N, a.T, tokens, slot) : tile_of(a.cu, a.N, a.T, tokens, slot);
        n = t.n;
        s = seq_range(a.cu, n, a.T);
        seg = t.index;
        chunks = (s.len + kC - 1) / kC;
        // (packed sequences of at most a segment's length stay whole)
        const int per = split ? tokens / kC : chunks;
        m0 = (int)min((int64_t)seg * per, (int64_t)chunks);
        nm = min(per, chunks - m0);
    }
    __device__ int chunk(int m, bool reverse) const { return reverse ? chunks - 1 - m0 - m : m0 + m; }
    __device__ int rows(int c) const { return min(kC, s.len - c * kC); }
};

// STATE: only what the segment adds to the state, from zero.  RETURNED: a pass returns its state (x1)
template <int D, bool STATE, bool RETURNED>
__global__ void __launch_bounds__(kThreads, 1) lin_tc_kernel(const __grid_constant__ Maps maps, const LinArgs args, const Split split, uint64_t limit, int withhold)
{
    using G = Geo<D>;
    constexpr int nct = D / kCols;
    extern __shared__ uint8_t lin_tc_smem[];
    uint8_t *const sm = lin_tc_smem + (-smem_u32(lin_tc_smem) & 1023u);
    // (the column halves and the passes of a head next to each other: they read the same tensors)
    const int c0 = (int)(blockIdx.x % nct) * kCols, pi = (int)(blockIdx.x / nct % args.passes);
    const LinPass &p = args.pass[pi];
    const unsigned rest = blockIdx.x / (nct * args.passes);
    const int hv = (int)(rest % args.HV);
    const int64_t slot = rest / args.HV;
    if (STATE && split.none()) return;
    int n;
    const Part part(args, split.held, STATE, split.segment(), slot, n);
    const bool rev = p.reverse;
    const bool last_seg = part.m0 + part.nm == part.chunks;
    const int nm = part.nm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float g = args.decay ? args.decay[hv] : 0.f, g2 = g * kRcpLn2;
    const int64_t xbase = ((int64_t)n * args.HV + hv) * D * D;
    auto xat = [&](int r, int c) { return xbase + (p.x_t ? (int64_t)(c0 + c) * D + r : (int64_t)r * D + c0 + c); };
    const int64_t at = split.held && part.nm < part.chunks ? (int64_t)pi * split.states + cut_state0(args.cu, n, args.T, split.segment()) + part.seg : 0;
    float *const mine = split.held && part.nm < part.chunks ? split.held + (at * args.HV + hv) * D * D + c0 : nullptr;

    if (nm <= 0) {
        // nothing to walk: a sequence without tokens hands its state on
        if (!STATE && part.chunks == 0 && part.seg == 0 && p.x1)
            for (int i = tid; i < D * kCols; i += kThreads) p.x1[xat(i / kCols, i % kCols)] = p.x0 ? p.x0[xat(i / kCols, i % kCols)] : 0.f;
        return;
    }
    if (STATE && last_seg) return;  // nothing follows it

    uint64_t *bar = (uint64_t *)(sm + G::kBars);
    uint32_t *tslot = (uint32_t *)(bar + kNumBars);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[kFull + i], 1);
            mbar_init(&bar[kEmpty + i], 1);
            mbar_init(&bar[kZF + i], 1);
            mbar_init(&bar[kZB + i], 4);
        }
        for (int i = 0; i < kStagesC; ++i) {
            mbar_init(&bar[kFullC + i], 1);
            mbar_init(&bar[kEmptyC + i], 1);
        }
        mbar_init(&bar[kLanded], 1);
        mbar_init(&bar[kXB], 8);
        mbar_init(&bar[kCB], 8);
        mbar_init(&bar[kXF], 1);
        mbar_init(&bar[kO1F], 1);
        mbar_init(&bar[kOF], 1);
        mbar_init(&bar[kOE], 4);
        mbar_init(&bar[kFin], 1);
        fence_mbar_init();
    }
    if (tid == 32) {
        prefetch_map(&maps.b[pi]);
        prefetch_map(&maps.a[pi]);
        prefetch_map(&maps.c[pi]);
    }
    if (warp == 3) tmem_alloc(tslot, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t base = smem_u32(sm);
    unsigned *const status = &g_lin_status;
    auto wait = [&](int b, uint32_t parity) { return mbar_wait(&bar[b], parity, status, kStatusTimeout, limit); };
    auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    // what goes into a state that is returned takes C's third part, which has the last of c's stages
    const bool third = RETURNED && p.x1 && (STATE || last_seg);
    const int ring = third ? kStagesC - 1 : kStagesC;
    constexpr int kThird = G::kCs + (kStagesC - 1) * kBox;
    auto loaded = [&](int m) { return all(wait(kFull + m % kStages, (m / kStages) & 1)); };    // a and b
    // c's stage of a chunk, and how often it has come round
    struct {
        int s = 0, round = 0;
        __device__ __forceinline__ void next(int ring)
        {
            if (++s == ring) s = 0, ++round;
        }
    } at_c;
    auto loaded_c = [&]() { return all(wait(kFullC + at_c.s, at_c.round & 1)); };

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        // (a and b are done with earlier than c, by most of a chunk's time)
        bool ok = !withhold;
        int m = 0;
        for (; m < nm && ok; ++m) {
            const int s = m % kStages, c = part.chunk(m, rev), rows = part.rows(c), t0 = (int)(part.s.bos + (int64_t)c * kC);
            uint8_t *const st = sm + s * G::kStage;
            auto zero_tail = [&](uint8_t *at, int boxes) {
                for (int b = 0; b < boxes; ++b)
                    for (int e = rows * 8 + lane; e < kC * 8; e += 32) *(uint4 *)(at + b * kBox + e * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
                __syncwarp();
            };
            if (m >= kStages && !(ok = all(wait(kEmpty + s, (m / kStages - 1) & 1)))) break;
            uint64_t *landing = &bar[rows < kC ? (int)kLanded : kFull + s];
            if (elect_one_sync()) {
                mbar_arrive_expect_tx(landing, (STATE ? 1 : 2) * G::kBoxes * kBox);
#pragma unroll
                for (int i = 0; i < G::kBoxes; ++i) {
                    tma_load_3d(st + G::kB + i * kBox, &maps.b[pi], i * 64, hv / p.rb, t0, landing);
                    if (!STATE) tma_load_3d(st + G::kA + i * kBox, &maps.a[pi], i * 64, hv / p.ra, t0, landing);
                }
            }
            __syncwarp();
            if (rows < kC) {  // (one chunk of a sequence at most)
                if (!(ok = all(wait(kLanded, 0)))) break;
                zero_tail(st + G::kB, G::kBoxes);
                if (lane == 0) mbar_arrive(&bar[kFull + s]);
            }
            const int sc = at_c.s;
            if (at_c.round > 0 && !(ok = all(wait(kEmptyC + sc, (at_c.round - 1) & 1)))) break;
            at_c.next(ring);
            landing = &bar[rows < kC ? (int)kLanded : kFullC + sc];
            if (elect_one_sync()) {
                mbar_arrive_expect_tx(landing, kBox);
                tma_load_3d(sm + G::kCs + sc * kBox, &maps.c[pi], c0, hv / p.rc, t0, landing);
            }
            __syncwarp();
            if (rows < kC) {
                if (!(ok = all(wait(kLanded, 1)))) break;
                zero_tail(sm + G::kCs + sc * kBox, 1);
                if (lane == 0) mbar_arrive(&bar[kFullC + sc]);
            }
        }
        // no copy outlives the CTA
        for (int i = max(0, m - kStages); i < m; ++i) wait(kFull + i % kStages, (i / kStages) & 1);
        for (int i = max(0, m - ring); i < m; ++i) wait(kFullC + i % ring, (i / ring) & 1);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products
        const uint32_t idZ = idesc_bf16_f32(128, 128, 0, 0), idO = idesc_bf16_f32(128, kCols, 0, 1), idX = idesc_bf16_f32(128, 2 * kCols, 1, 1), idX3 = idesc_bf16_f32(128, kCols, 1, 1);
        const uint64_t dX = sdesc_sw128(base + G::kXs, kBox, 1024), dC = sdesc_sw128(base + G::kParts, kBox, 1024), dC3 = sdesc_sw128(base + kThird, kBox, 1024);
        auto scores = [&](int m) {
            const uint32_t st = base + (m % kStages) * G::kStage, z = tmem + kZ + (m & 1) * 128;
            const uint64_t da = sdesc_sw128(st + G::kA, 16, 1024), db = sdesc_sw128(st + G::kB, 16, 1024);
            tc_fence_after();
            if (elect_one_sync()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = ((ks >> 2) * kBox + (ks & 3) * 32) >> 4;
                    mma_ss(z, da + o, db + o, idZ, ks > 0);
                }
                mma_commit(&bar[kZF + (m & 1)]);
            }
            __syncwarp();
        };
        bool ok = loaded(0);
        if (!STATE && ok) scores(0);
        for (int m = 0; m < nm && ok; ++m, at_c.next(ring)) {
            const uint32_t st = base + (m % kStages) * G::kStage;
            if (STATE && !(ok = loaded(m))) break;
            if (!(ok = all(wait(kXB, m & 1) && wait(kCB, m & 1)))) break;
            tc_fence_after();
            if (elect_one_sync()) {
                const uint64_t db = sdesc_sw128(st + G::kB, kBox, 1024);
#pragma unroll
                for (int ks = 0; ks < kC / 16; ++ks) mma_ss(tmem + kX, db + ks * 128, dC + ks * 128, idX, !RETURNED || ks > 0);
                if (third) {
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks) mma_ss(tmem + kX + kCols, db + ks * 128, dC3 + ks * 128, idX3, 1u);
                }
                mma_commit(&bar[kXF]);
                if (STATE) {
                    mma_commit(&bar[kEmpty + m % kStages]);
                    mma_commit(&bar[kEmptyC + at_c.s]);
                }
            }
            __syncwarp();
            if (!STATE) {
                if (m > 0 && !(ok = all(wait(kOE, (m - 1) & 1)))) break;  // the last outputs have been read
                const uint64_t da = sdesc_sw128(st + G::kA, 16, 1024), dc = sdesc_sw128(base + G::kCs + at_c.s * kBox, kBox, 1024);
                tc_fence_after();
                if (elect_one_sync()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) mma_ss(tmem + kO1, da + (((ks >> 2) * kBox + (ks & 3) * 32) >> 4), dX + ks * 128, idO, ks > 0);
                    mma_commit(&bar[kO1F]);
                    mma_commit(&bar[kEmpty + m % kStages]);
                }
                __syncwarp();
                if (m + 1 < nm) {
                    if (!(ok = loaded(m + 1))) break;
                    scores(m + 1);
                }
                if (!(ok = all(wait(kZB + (m & 1), (m >> 1) & 1)) && loaded_c())) break;
                tc_fence_after();
                if (elect_one_sync()) {
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks) mma_ts(tmem + kO2, tmem + kZ + (m & 1) * 128 + ks * 8, dc + ks * 128, idO, ks > 0);
                    mma_commit(&bar[kOF]);
                    mma_commit(&bar[kEmptyC + at_c.s]);
                }
                __syncwarp();
            }
        }
        if (elect_one_sync()) mma_commit(&bar[kFin]);  // every product has ended before the tensor memory goes
        __syncwarp();
        wait(kFin, 0);
    } else if (warp >= 4 && warp < 8) {
        // ---------------------------------------------------------------- Z (thread = row)
        if (!STATE) {
            const int i = tid - 128, w = warp - 4;
            const float l1 = decay_pow(g2, 1), l2 = decay_pow(g2, 2);
            for (int m = 0; m < nm; ++m) {
                if (!bar_all(1, 128, w != 0 || wait(kZF + (m & 1), (m >> 1) & 1))) break;
                tc_fence_after();
                const uint32_t z = tmem + lanes + kZ + (m & 1) * 128;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[32], u[16];
                    if (rev ? q < w : q > w) {  // (all of it on the side that does not count)
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = 0u;
                    } else {
                        tmem_ld32(z + 32 * q, v);
                        tmem_ld_wait();
                        float *const x = (float *)v;
                        // cs l^|i - j| from the column next to the row's own side on, one more l at every step (no table in shared
                        // memory, which the products keep busy)
                        if (q == w) {
                            float f = 0.f;
                            if (rev) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    f = j == lane ? p.cs : f * l1;
                                    x[j] = j < lane ? 0.f : x[j] * f;
                                }
                            } else {
#pragma unroll
                                for (int j = 31; j >= 0; --j) {
                                    f = j == lane ? p.cs : f * l1;
                                    x[j] = j > lane ? 0.f : x[j] * f;
                                }
                            }
                        } else {
                            float f = p.cs * decay_pow(g2, rev ? 32 * q - i : i - 32 * q - 31), f1 = f * l1;
                            if (rev) {
#pragma unroll
                                for (int j = 0; j < 32; j += 2) {
                                    x[j] *= f;
                                    x[j + 1] *= f1;
                                    f *= l2;
                                    f1 *= l2;
                                }
                            } else {
#pragma unroll
                                for (int j = 31; j > 0; j -= 2) {
                                    x[j] *= f;
                                    x[j - 1] *= f1;
                                    f *= l2;
                                    f1 *= l2;
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
                    }
                    tmem_st16(z + 16 * q, u);  // (over columns that are read already)
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kZB + (m & 1)]);
            }
        }
    } else if (warp >= 8 && warp < 16) {
        // ---------------------------------------------------------------- the state (thread = 32 columns of a row of X)
        const int r = tid & 127, c1 = warp >= 12 ? 32 : 0;
        const bool real = r < D;
        const uint32_t xt = tmem + lanes + kX + c1;
        float x[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = 0.f;
        if (!STATE && real) {
            if (mine) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) *(float4 *)&x[c] = *(const float4 *)(mine + (int64_t)r * D + c1 + c);
            } else if (p.x0) {
#pragma unroll
                for (int c = 0; c < 32; ++c) x[c] = p.x0[xat(r, c1 + c)];
            }
        }
        // the sum of the two accumulators; RETURNED: beside what the registers hold of the state
        auto read = [&]() {
            tc_fence_after();
            if constexpr (RETURNED) {
#pragma unroll
                for (int q = 0; q < 32; q += 16) {
                    float y[16], z[16];
                    tmem_ld16(xt + q, (uint32_t *)y);
                    tmem_ld16(xt + kCols + q, (uint32_t *)z);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[q + k] += y[k] + z[k];
                }
            } else {
                float y[32];
                tmem_ld32(xt, (uint32_t *)x);
                tmem_ld32(xt + kCols, (uint32_t *)y);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] += y[k];
            }
        };
        bool ok = true;
        for (int m = 0; m < nm; ++m) {
            const int rows = part.rows(part.chunk(m, rev)), late = rev && part.m0 + m == 0;
            const Decayed down(g, rows - late);
            if (m > 0) {
                if (!(ok = bar_all(2, 256, warp != 8 || wait(kXF, (m - 1) & 1)))) break;
                read();
            }
            if constexpr (!RETURNED) {
                const uint32_t none[32] = {};
                tmem_st32(xt + kCols, none);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float y[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] = down(x[16 * q + k]);
                    tmem_st16(xt + 16 * q, (const uint32_t *)y);
                }
            }
            if (!STATE) {
                if (m > 0 && !(ok = bar_all(2, 256, warp != 8 || wait(kO1F, (m - 1) & 1)))) break;  // the last copy has been read
                if (real) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) *(uint4 *)(sm + G::kXs + sw128(r, c1 + i)) = pack8(x + i);
                }
                fence_proxy_async();
            }
            if constexpr (!RETURNED) tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kXB]);
            if constexpr (RETURNED) {
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = down(x[k]);
            }
        }
        if (ok && (STATE || (p.x1 && last_seg)) && bar_all(2, 256, warp != 8 || wait(kXF, (nm - 1) & 1))) {
            read();
            const Decayed down(g, rev && !STATE ? 1 : 0);
            if (real) {
                if (STATE) {
#pragma unroll
                    for (int c = 0; c < 32; c += 4) *(float4 *)(mine + (int64_t)r * D + c1 + c) = *(const float4 *)&x[c];
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) p.x1[xat(r, c1 + c)] = down(x[c]);
                }
            }
        }
    } else if (warp >= 16 && warp < 20) {
        // ---------------------------------------------------------------- outputs (thread = row)
        if (!STATE) {
            const int i = tid & 127;
            const bool wide = ((uintptr_t)p.out & 31) == 0;
            for (int m = 0; m < nm; ++m) {
                const int c = part.chunk(m, rev), rows = part.rows(c), late = rev && part.m0 + m == 0;
                const float f = p.os * decay_pow(g2, rev ? max(rows - i - late, 0) : i + 1);
                const uint32_t o1 = tmem + lanes + kO1, o2 = tmem + lanes + kO2;
                const int64_t at = ((part.s.bos + (int64_t)c * kC + i) * args.HV + hv) * D + c0;
                if (!bar_all(3, 128, warp != 16 || wait(kOF, m & 1))) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float u[32], v[32];
                    tmem_ld32(o2 + 32 * q, (uint32_t *)u);
                    tmem_ld32(o1 + 32 * q, (uint32_t *)v);
                    tmem_ld_wait();
                    if (q == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[kOE]);
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) u[k] = fmaf(f, v[k], p.os * u[k]);
                    if (i < rows) {
                        if (p.out_f32) {
                            float *dst = (float *)p.out + at + 32 * q;
#pragma unroll
                            for (int k = 0; k < 32; k += 4) *(float4 *)(dst + k) = *(const float4 *)&u[k];
                        } else {
                            __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out + at + 32 * q;
#pragma unroll
                            for (int k = 0; k < 32; k += 16) {
                                const uint4 y = pack8(u + k), z = pack8(u + k + 8);
                                if (wide) {  // (a whole sector by one thread)
                                    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + k), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w),
                                                 "r"(z.x), "r"(z.y), "r"(z.z), "r"(z.w)
                                                 : "memory");
                                } else {
                                    *(uint4 *)(dst + k) = y;
                                    *(uint4 *)(dst + k + 8) = z;
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp >= 20) {
        // ---------------------------------------------------------------- C in parts (thread = 32 columns of a row)
        const int j = tid & 127, i0 = warp >= 24 ? 4 : 0;
        for (int m = 0; m < nm; ++m, at_c.next(ring)) {
            const int rows = part.rows(part.chunk(m, rev));
            const float f = j < rows ? p.cs * decay_pow(g2, rev ? j : rows - 1 - j) : 0.f;
            const uint8_t *const src = sm + G::kCs + at_c.s * kBox;
            uint8_t *const dst = sm + G::kParts;
            if (!bar_all(4, 256, warp != 20 || loaded_c())) break;
            uint4 hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 raw = *(const uint4 *)(src + sw128(j, 8 * (i0 + i)));
                const uint32_t *w = (const uint32_t *)&raw;
                uint32_t *ph = (uint32_t *)&hi[i], *pl = (uint32_t *)&lo[i];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float u = f * low_bf16(w[k]), v = f * high_bf16(w[k]);
                    ph[k] = pack_bf16(u, v);
                    pl[k] = pack_bf16(u - low_bf16(ph[k]), v - high_bf16(ph[k]));
                }
            }
            if (m > 0 && !bar_all(4, 256, warp != 20 || wait(kXF, (m - 1) & 1))) break;  // the products have read the last chunk's
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                *(uint4 *)(dst + sw128(j, 8 * (i0 + i))) = hi[i];
                *(uint4 *)(dst + kBox + sw128(j, 8 * (i0 + i))) = lo[i];
            }
            if (third) {  // (what the two leave, from c again: it stays until the products have been issued)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 raw = *(const uint4 *)(src + sw128(j, 8 * (i0 + i)));
                    const uint32_t *w = (const uint32_t *)&raw, *ph = (const uint32_t *)&hi[i], *pl = (const uint32_t *)&lo[i];
                    uint32_t left[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        left[k] = pack_bf16(f * low_bf16(w[k]) - low_bf16(ph[k]) - low_bf16(pl[k]), f * high_bf16(w[k]) - high_bf16(ph[k]) - high_bf16(pl[k]));
                    *(uint4 *)(sm + kThird + sw128(j, 8 * (i0 + i))) = make_uint4(left[0], left[1], left[2], left[3]);
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kCB]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

// What the segments add to the state -> the state that enters each (in place): four elements to a thread, a block of 1024 to a piece of a (cut
// sequence, head) pair.  Eight segments are asked for at once (one after the other, 19 segments took 64 us).
template <int D>
__global__ void __launch_bounds__(256) lin_join_kernel(const LinArgs args, const Split split)
{
    if (split.none()) return;
    constexpr int kPieces = D * D / 1024;
    const LinPass &p = args.pass[blockIdx.y];
    const int which = (int)(blockIdx.x / kPieces), at = (int)(blockIdx.x % kPieces) * 1024 + 4 * threadIdx.x, tokens = split.segment();
    const int place = which / args.HV, hv = which - place * args.HV;
    auto first_at = [&](int n) { return long_place(args.cu, n, args.T, tokens); };
    const int n = args.cu ? last_from_warp(args.N, place, first_at) : place;
    const SeqRange s = seq_range(args.cu, n, args.T);
    const int segs = (s.len + tokens - 1) / tokens;
    if (segs <= 1 || first_at(n) != place) return;  // (whole)
    const int64_t slot0 = cut_state0(args.cu, n, args.T, tokens), pair = (int64_t)n * args.HV + hv;
    const float g = args.decay ? args.decay[hv] : 0.f;
    // tokens of a segment in the order of processing: against time the first has the sequence's odd end
    const int odd = (s.len + kC - 1) / kC * kC - s.len;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = p.x0 ? p.x0[pair * D * D + (p.x_t ? ((at + e) % D) * D + at / D : at + e)] : 0.f;
    const int64_t step = (int64_t)args.HV * D * D;
    float *buf = split.held + (((int64_t)blockIdx.y * split.states + slot0) * args.HV + hv) * D * D + at;
    const Decayed first(g, tokens - (p.reverse ? odd + 1 : 0)), rest(g, tokens);
    for (int i = 0; i < segs; i += 8) {
        float4 add[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) add[k] = i + k + 1 < segs ? *(const float4 *)(buf + (i + k) * step) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < segs) {
                *(float4 *)(buf + (i + k) * step) = make_float4(x[0], x[1], x[2], x[3]);
                const float *y = (const float *)&add[k];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = (i + k == 0 ? first(x[e]) : rest(x[e])) + y[e];
            }
    }
}

// The segment of a packed batch, from its lengths: a multiple of the plan's, or none.  A warp takes one: the longest piece, or the SMs' share of
// all pieces and half a piece for the ragged end, in chunks, as in lin_tc_plan.  (In place of the
// plan's own segment, which fits one sequence of all tokens: 30 random cuts of 32768 tokens, 8 heads of 128, 172 -> 121 us, gradients 424 -> 295;
// one call more to wait for where little is to choose: two sequences of 8191 tokens 51 -> 57.)
__device__ constexpr int kMultiples[16] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 40, 48, 0};
__global__ void __launch_bounds__(512) lin_choose_kernel(const LinArgs args, int tokens, float share, int *chosen)
{
    __shared__ float time[16];
    __shared__ int cuts[16];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t per = kMultiples[w] ? (int64_t)kMultiples[w] * (tokens / kC) : INT32_MAX;
    float work = 0.f;
    int longest = 0;
    bool twice = false;
    for (int n = lane; n < args.N; n += 32) {
        const int chunks = (seq_range(args.cu, n, args.T).len + kC - 1) / kC;
        if (chunks == 0) continue;
        const bool cut = chunks > per;
        work += cut ? kAgain * (float)(chunks + 2 * ((chunks + per - 1) / per)) : (float)(chunks + 2);
        longest = max(longest, (int)min((int64_t)chunks, per));
        twice |= cut;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        work += __shfl_xor_sync(0xffffffffu, work, o);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    }
    twice = __any_sync(0xffffffffu, twice);
    if (lane == 0) cuts[w] = twice, time[w] = fmaxf((twice ? kAgain : 1.f) * (float)(longest + 2), work * share + 0.5f * (float)longest) + (twice ? kLaunches : 0.f);
    __syncthreads();
    if (threadIdx.x == 0) {
        int best = 15;  // (none, where another is not faster)
        for (int i = 0; i < 15; ++i)
            if (time[i] < time[best]) best = i;
        const int64_t seg = kMultiples[best] ? (int64_t)kMultiples[best] * tokens : INT32_MAX / kC * kC;
        chosen[1] = cuts[best];
        *chosen = (int)min(seg, (int64_t)(args.T + kC - 1) / kC * kC);  // (a sequence of all tokens is not longer)
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)p;
    }();
    return fn;
}

template <int D>
cudaError_t launch(const LinArgs &a, void *ws, int64_t tokens, cudaStream_t st)
{
    Maps maps;
    for (int i = 0; i < a.passes; ++i) {
        const LinPass &p = a.pass[i];
        if (!heads_map(&maps.a[i], p.a, D, a.HV / p.ra, tokens, p.lda, kC) || !heads_map(&maps.b[i], p.b, D, a.HV / p.rb, tokens, p.ldb, kC) ||
            !heads_map(&maps.c[i], p.c, D, a.HV / p.rc, tokens, p.ldc, kC))
            return cudaErrorInvalidValue;
    }
    const LinPlan plan = lin_tc_plan(a, D);
    Split split{};
    split.states = plan.states;
    split.tokens = plan.tokens;
    split.held = plan.bytes ? (float *)ws : nullptr;
    int *const chosen = split.held && several(a) ? (int *)((char *)ws + plan.bytes - kChosenBytes) : nullptr;
    split.chosen = chosen;
    static std::atomic<uint64_t> seen;
    if (first_on_device(seen)) {
        for (auto kern : {lin_tc_kernel<D, false, false>, lin_tc_kernel<D, true, false>, lin_tc_kernel<D, false, true>, lin_tc_kernel<D, true, true>}) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
            if (e != cudaSuccess) return e;
        }
        done_on_device(seen);
    }
    bool returned = false;
    for (int i = 0; i < a.passes; ++i) returned = returned || a.pass[i].x1;
    auto sums = returned ? lin_tc_kernel<D, true, true> : lin_tc_kernel<D, true, false>, walk = returned ? lin_tc_kernel<D, false, true> : lin_tc_kernel<D, false, false>;
    const int64_t each = (int64_t)a.HV * (D / kCols) * a.passes, joined = plan.places * a.HV * D * D / 1024;
    if (plan.slots * each > INT32_MAX || plan.states * each > INT32_MAX || joined > INT32_MAX) return cudaErrorInvalidConfiguration;
    const int withhold = withhold_loads();
    const uint64_t limit = withhold ? kTestWaitLimitNs : kWaitLimitNs;
    if (chosen) lin_choose_kernel<<<1, 512, 0, st>>>(a, plan.tokens, (float)each / (float)device_sm_count(), chosen);
    if (split.held) {
        sums<<<(unsigned)(plan.states * each), kThreads, Geo<D>::kSmem, st>>>(maps, a, split, limit, withhold);
        lin_join_kernel<D><<<dim3((unsigned)joined, a.passes), 256, 0, st>>>(a, split);
    }
    walk<<<(unsigned)(plan.slots * each), kThreads, Geo<D>::kSmem, st>>>(maps, a, split, limit, withhold);
    return cudaGetLastError();
}

}  // namespace

bool heads_map(CUtensorMap *m, const void *base, int D, int heads, int64_t tokens, int64_t ld, int box_rows)
{
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, tokens > 1 ? (cuuint64_t)ld * 2 : (cuuint64_t)heads * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool strided_map(CUtensorMap *m, const void *base, int D, int heads, int T, int batch, int64_t head, int64_t tok, int64_t seq, int box_rows)
{
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)batch};
    auto bytes = [&](int64_t stride, int64_t size) { return (cuuint64_t)(size > 1 ? stride : D) * 2; };  // (of one there is no next)
    const cuuint64_t strides[3] = {bytes(head, heads), bytes(tok, T), bytes(seq, batch)};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

LinPlan lin_tc_plan(const LinArgs &a, int D)
{
    // A split walks its chunks twice (the second time with outputs), so it pays only where (sequence, head) pairs leave SMs idle: the
    // time of a plan is taken as rounds of CTAs times chunks of a segment and two more to begin and end one, a walk without outputs as 0.6 of
    // one with them (measured: 80 us and 122 at 65536 tokens of 8 heads) and the further launches as 8 chunks.  The lengths of packed
    // sequences are not known here: the segment is what one sequence of all tokens would be cut into, and lin_choose_kernel takes a multiple of it.
    const int64_t each = std::max(1, (a.T + kC - 1) / kC), ctas = (int64_t)(a.cu ? 1 : a.N) * a.HV * (D / kCols) * a.passes, sms = device_sm_count();
    int64_t best = 1;
    double least = 1e30;
    for (int64_t s = 1; s <= std::min<int64_t>(64, (each + 3) / 4); ++s) {
        const int64_t per = (each + s - 1) / s;
        const double t = (double)((ctas * s + sms - 1) / sms) * (double)(per + 2) * (s > 1 ? (double)kAgain : 1.0) + (s > 1 ? (double)kLaunches : 0.0);
        if (t < least) least = t, best = s;
    }
    LinPlan p{};
    if (best == 1) {
        p.slots = a.N;
        return p;
    }
    p.tokens = (int)((each + best - 1) / best) * kC;
    p.slots = mix_slots(a.cu != nullptr, a.N, a.T, p.tokens);
    p.states = cut_states(a.cu != nullptr, a.N, a.T, p.tokens);
    p.places = long_places(a.cu != nullptr, a.N, a.T, p.tokens);
    p.bytes = (size_t)a.passes * p.states * a.HV * D * D * sizeof(float) + (several(a) ? kChosenBytes : 0);
    return p;
}

bool lin_tc_ok(const LinArgs &a, int64_t tokens)
{
    const int D = a.pass[0].da;
    if ((D != 64 && D != 128) || a.T < 1 || tokens > INT32_MAX - kC) return false;
    for (int i = 0; i < a.passes; ++i) {
        const LinPass &p = a.pass[i];
        if (p.da != D || p.dc != D) return false;
        if (!tma_ok(p.a, p.lda, tokens, 2) || !tma_ok(p.b, p.ldb, tokens, 2) || !tma_ok(p.c, p.ldc, tokens, 2) || ((uintptr_t)p.out & 15)) return false;
    }
    return true;
}

cudaError_t launch_lin_tc(const LinArgs &a, void *ws, int64_t tokens, cudaStream_t st)
{
    return a.pass[0].da == 64 ? launch<64>(a, ws, tokens, st) : launch<128>(a, ws, tokens, st);
}

gdn_status read_lin_status(cudaStream_t st)
{
    unsigned word = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, g_lin_status, sizeof(word), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_lin_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return word & kStatusTimeout ? GDN_ERR_TIMEOUT : GDN_OK;
}

}  // namespace gdn
