// Linear attention with a decay for each head on the tensor cores: bf16, heads of 64 or 128 (K = V), rows on 16-byte boundaries.
//
// One CTA per (sequence or segment of one, value head, 64 columns of c) walks chunks of 128 tokens; the state X (D x 64, fp32)
// stays in tensor memory.  Per chunk of n tokens, forward in time, every product a tcgen05 MMA with M = 128:
//   Z  = a b^T                       (128 x 128)     Z_ij -> cs l^(i-j) Z_ij for j <= i, rounded to bf16 where it lies
//   O1 = a X,  O2 = Z c              (128 x 64)      out_i = os (l^(i+1) O1_i + O2_i)
//   X <- l^n X + b^T C               (D x 64)        C_j = cs l^(n-1-j) c_j as the sum of two bf16 values
// X enters O1 rounded to bf16; the state itself takes C as hi + lo (16 bits of it; one bf16 alone would put 2^-9 into a state that
// is returned in fp32), and b and c as they are.  Against time the same with the powers counted from the chunk's other end.
//
// Warps: 0 loads (TMA, two stages of a, b and c's columns), 1 issues the products, 4-7 turn Z, 8-11 round and decay X, 12-15 write
// out, 16-19 scale c.  The chain from chunk to chunk is X's: product, read, round, decay, write back.
#include <cudaTypedefs.h>

#include "gdn_mix.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kC = 128, kCols = 64, kThreads = 640, kStages = 2, kBox = kC * 128;
constexpr uint32_t kZ = 0, kO1 = 256, kO2 = 320, kX = 384, kTmem = 512;  // tensor-memory columns (Z: two buffers)

__device__ unsigned g_lin_status;

template <int D>
struct Geo {
    static constexpr int kBoxes = D / 64;
    static constexpr int kA = 0, kB = kBoxes * kBox, kCc = 2 * kBoxes * kBox, kStage = (2 * kBoxes + 1) * kBox;
    static constexpr int kXs = kStages * kStage, kHi = kXs + kBox, kLo = kHi + kBox, kOut = kLo + kBox, kTab = kOut + kBox, kBars = kTab + 1024;
    static constexpr int kSmem = kBars + 256 + 1024;
};
enum Bar { kFull, kEmpty = kFull + kStages, kZF = kEmpty + kStages, kZB = kZF + 2, kXB = kZB + 2, kCB, kXF, kOF, kOE, kFix, kFin, kNumBars };

struct Maps {
    CUtensorMap a[3], b[3], c[3], out[3];
};

struct Split {
    float *states;  // [passes][slots][HV][D][D]: what a segment adds to the state, then the state that enters it; null: one segment each
    int tokens;     // of a segment (a multiple of kC)
    int64_t slots;
};

// A CTA's part of a sequence, in the order of processing
struct Part {
    SeqRange s;
    int chunks, m0, nm, seg;  // of the sequence; the first one's place, how many; which segment
    __device__ Part(const LinArgs &a, const Split &sp, int64_t slot, int &n)
    {
        const Tile t = sp.states ? tile_of(a.cu, a.N, a.T, sp.tokens, slot) : Tile{(int)slot, 0};
        n = t.n;
        s = seq_range(a.cu, n, a.T);
        seg = t.index;
        chunks = (s.len + kC - 1) / kC;
        const int per = sp.states ? sp.tokens / kC : chunks;
        m0 = (int)min((int64_t)seg * per, (int64_t)chunks);
        nm = min(per, chunks - m0);
    }
    __device__ int chunk(int m, bool reverse) const { return reverse ? chunks - 1 - m0 - m : m0 + m; }
    __device__ int rows(int c) const { return min(kC, s.len - c * kC); }
};

// STATE: only what the segment adds to the state, from zero
template <int D, bool STATE>
__global__ void __launch_bounds__(kThreads, 1) lin_tc_kernel(const __grid_constant__ Maps maps, const LinArgs args, const Split split, uint64_t limit, int withhold)
{
    using G = Geo<D>;
    constexpr int nct = D / kCols;
    extern __shared__ uint8_t lin_tc_smem[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)lin_tc_smem + 1023) & ~(uintptr_t)1023);
    const LinPass &p = args.pass[blockIdx.y];
    const int ct = (int)(blockIdx.x % nct), hv = (int)(blockIdx.x / nct % args.HV), c0 = ct * kCols;
    const int64_t slot = blockIdx.x / ((unsigned)nct * args.HV);
    int n;
    const Part part(args, split, slot, n);
    const bool rev = p.reverse;
    const bool last_seg = part.m0 + part.nm == part.chunks;
    const int nm = part.nm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float g = args.decay ? args.decay[hv] : 0.f, g2 = g * kRcpLn2;
    const int64_t xbase = ((int64_t)n * args.HV + hv) * D * D;
    auto xat = [&](int r, int c) { return xbase + (p.x_t ? (int64_t)(c0 + c) * D + r : (int64_t)r * D + c0 + c); };
    float *const mine = split.states ? split.states + (((int64_t)blockIdx.y * split.slots + slot) * args.HV + hv) * D * D + c0 : nullptr;

    if (nm <= 0) {
        // nothing to walk: a sequence without tokens hands its state on
        if (!STATE && part.chunks == 0 && part.seg == 0 && p.x1)
            for (int i = tid; i < D * kCols; i += kThreads) p.x1[xat(i / kCols, i % kCols)] = p.x0 ? p.x0[xat(i / kCols, i % kCols)] : 0.f;
        return;
    }
    if (STATE && last_seg) return;  // nothing follows it

    uint64_t *bar = (uint64_t *)(sm + G::kBars);
    uint32_t *tslot = (uint32_t *)(bar + kNumBars);
    float *tab = (float *)(sm + G::kTab);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar[kFull + i], 1);
            mbar_init(&bar[kEmpty + i], 1);
            mbar_init(&bar[kZF + i], 1);
            mbar_init(&bar[kZB + i], 4);
        }
        mbar_init(&bar[kXB], 4);
        mbar_init(&bar[kCB], 4);
        mbar_init(&bar[kXF], 1);
        mbar_init(&bar[kOF], 1);
        mbar_init(&bar[kOE], 4);
        mbar_init(&bar[kFix], 4);
        mbar_init(&bar[kFin], 1);
        fence_mbar_init();
    }
    if (tid < 256) {  // tab[127 + i - j]: cs l^|i - j| on the side that counts, else 0
        const int d = rev ? 127 - tid : tid - 127;
        tab[tid] = d >= 0 ? p.cs * decay_pow(g2, d) : 0.f;
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
    // the sequence's last chunk, where it is not full: its place here (or none)
    const int ragged = part.s.len % kC == 0 ? -1 : rev ? (part.m0 == 0 ? 0 : -1) : (last_seg ? nm - 1 : -1);
    auto loaded = [&](int m) { return wait(kFull + m % kStages, (m / kStages) & 1) && (m != ragged || wait(kFix, 0)); };

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        bool ok = !withhold;
        int m = 0;
        for (; m < nm && ok; ++m) {
            const int s = m % kStages;
            if (m >= kStages && !(ok = all(wait(kEmpty + s, (m / kStages - 1) & 1)))) break;
            if (elect_one_sync()) {
                uint8_t *st = sm + s * G::kStage;
                const int t0 = (int)(part.s.bos + (int64_t)part.chunk(m, rev) * kC);
                mbar_arrive_expect_tx(&bar[kFull + s], STATE ? (G::kBoxes + 1) * kBox : G::kStage);
#pragma unroll
                for (int i = 0; i < G::kBoxes; ++i) {
                    tma_load_3d(st + G::kB + i * kBox, &maps.b[blockIdx.y], i * 64, hv / p.rb, t0, &bar[kFull + s]);
                    if (!STATE) tma_load_3d(st + G::kA + i * kBox, &maps.a[blockIdx.y], i * 64, hv / p.ra, t0, &bar[kFull + s]);
                }
                tma_load_3d(st + G::kCc, &maps.c[blockIdx.y], c0, hv / p.rc, t0, &bar[kFull + s]);
            }
            __syncwarp();
        }
        for (int i = max(0, m - kStages); i < m; ++i) wait(kFull + i % kStages, (i / kStages) & 1);  // (no copy outlives the CTA)
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products
        const uint32_t idZ = idesc_bf16_f32(128, 128, 0, 0), idMN = idesc_bf16_f32(128, kCols, 0, 1), idX = idesc_bf16_f32(128, kCols, 1, 1);
        const uint64_t dX = sdesc_sw128(base + G::kXs, kBox, 1024), dHi = sdesc_sw128(base + G::kHi, kBox, 1024), dLo = sdesc_sw128(base + G::kLo, kBox, 1024);
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
        bool ok = all(loaded(0));
        if (!STATE && ok) scores(0);
        for (int m = 0; m < nm && ok; ++m) {
            const uint32_t st = base + (m % kStages) * G::kStage;
            if (!(ok = all(wait(kXB, m & 1)))) break;
            if (!STATE) {
                if (m > 0 && !(ok = all(wait(kOE, (m - 1) & 1)))) break;
                const uint64_t da = sdesc_sw128(st + G::kA, 16, 1024);
                tc_fence_after();
                if (elect_one_sync()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) mma_ss(tmem + kO1, da + (((ks >> 2) * kBox + (ks & 3) * 32) >> 4), dX + ks * 128, idMN, ks > 0);
                }
                __syncwarp();
            } else if (!(ok = all(loaded(m)))) {
                break;
            }
            if (!(ok = all(wait(kCB, m & 1)))) break;
            tc_fence_after();
            if (elect_one_sync()) {
                const uint64_t db = sdesc_sw128(st + G::kB, kBox, 1024);
#pragma unroll
                for (int ks = 0; ks < kC / 16; ++ks) mma_ss(tmem + kX, db + ks * 128, dHi + ks * 128, idX, 1u);
#pragma unroll
                for (int ks = 0; ks < kC / 16; ++ks) mma_ss(tmem + kX, db + ks * 128, dLo + ks * 128, idX, 1u);
                mma_commit(&bar[kXF]);
                if (STATE) mma_commit(&bar[kEmpty + m % kStages]);
            }
            __syncwarp();
            if (!STATE) {
                if (m + 1 < nm) {
                    if (!(ok = all(loaded(m + 1)))) break;
                    scores(m + 1);
                }
                if (!(ok = all(wait(kZB + (m & 1), (m >> 1) & 1)))) break;
                const uint64_t dc = sdesc_sw128(st + G::kCc, kBox, 1024);
                tc_fence_after();
                if (elect_one_sync()) {
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks) mma_ts(tmem + kO2, tmem + kZ + (m & 1) * 128 + ks * 8, dc + ks * 128, idMN, ks > 0);
                    mma_commit(&bar[kOF]);
                    mma_commit(&bar[kEmpty + m % kStages]);
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
            const int i = tid - 128;
            for (int m = 0; m < nm; ++m) {
                if (!all(wait(kZF + (m & 1), (m >> 1) & 1))) break;
                tc_fence_after();
                const uint32_t z = tmem + lanes + kZ + (m & 1) * 128;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[32], w[16];
                    tmem_ld32(z + 32 * q, v);
                    tmem_ld_wait();
                    const float *f = tab + 127 + i - 32 * q;
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = pack_bf16(__uint_as_float(v[2 * j]) * f[-2 * j], __uint_as_float(v[2 * j + 1]) * f[-2 * j - 1]);
                    tmem_st16(z + 16 * q, w);  // (over columns that are read already)
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kZB + (m & 1)]);
            }
        }
    } else if (warp >= 8 && warp < 12) {
        // ---------------------------------------------------------------- the state (thread = row of X)
        const int r = tid - 256;
        const uint32_t xt = tmem + lanes + kX;
        float x[kCols];
        if (r < D) {
            if (!STATE && mine) {
#pragma unroll
                for (int c = 0; c < kCols; c += 4) *(float4 *)&x[c] = *(const float4 *)(mine + (int64_t)r * D + c);
            } else if (!STATE && p.x0) {
#pragma unroll
                for (int c = 0; c < kCols; ++c) x[c] = p.x0[xat(r, c)];
            } else {
#pragma unroll
                for (int c = 0; c < kCols; ++c) x[c] = 0.f;
            }
        } else {
#pragma unroll
            for (int c = 0; c < kCols; ++c) x[c] = 0.f;
        }
        auto read = [&]() {
            tc_fence_after();
            tmem_ld32(xt, (uint32_t *)x);
            tmem_ld32(xt + 32, (uint32_t *)x + 32);
            tmem_ld_wait();
        };
        bool ok = true;
        for (int m = 0; m < nm; ++m) {
            const int c = part.chunk(m, rev);
            const Decayed down(g, part.rows(c) - (rev && part.m0 + m == 0));
            if (m > 0) {
                if (!(ok = all(wait(kXF, (m - 1) & 1)))) break;
                read();
            }
            if (!STATE && r < D) {
#pragma unroll
                for (int i = 0; i < kCols / 8; ++i) *(uint4 *)(sm + G::kXs + sw128(r, 8 * i)) = pack8(x + 8 * i);
            }
#pragma unroll
            for (int i = 0; i < kCols; ++i) x[i] = down(x[i]);
            tmem_st32(xt, (const uint32_t *)x);
            tmem_st32(xt + 32, (const uint32_t *)x + 32);
            tmem_st_wait();
            tc_fence_before();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kXB]);
        }
        if (ok && (STATE || (p.x1 && last_seg)) && all(wait(kXF, (nm - 1) & 1))) {
            read();
            const Decayed down(g, rev && !STATE ? 1 : 0);
            if (r < D) {
                if (STATE) {
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) *(float4 *)(mine + (int64_t)r * D + c) = *(const float4 *)&x[c];
                } else {
#pragma unroll
                    for (int c = 0; c < kCols; ++c) p.x1[xat(r, c)] = down(x[c]);
                }
            }
        }
    } else if (warp >= 12 && warp < 16) {
        // ---------------------------------------------------------------- outputs (thread = row)
        if (!STATE) {
            const int i = tid - 384;
            const uint32_t o1 = tmem + lanes + kO1, o2 = tmem + lanes + kO2;
            uint8_t *const tile = sm + G::kOut;
            for (int m = 0; m < nm; ++m) {
                const int c = part.chunk(m, rev), rows = part.rows(c);
                const int late = rev && part.m0 + m == 0;
                const float f = p.os * decay_pow(g2, rev ? max(rows - i - late, 0) : i + 1);
                const int64_t t0 = part.s.bos + (int64_t)c * kC;
                const bool ok = wait(kOF, m & 1);
                if (tid == 384) tma_store_wait_read0();
                if (!bar_all(1, 128, ok)) break;  // (together: the others would wait for a warp that gave up)
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float u[32], w[32];
                    tmem_ld32(o1 + 32 * q, (uint32_t *)u);
                    tmem_ld32(o2 + 32 * q, (uint32_t *)w);
                    tmem_ld_wait();
                    if (q == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[kOE]);
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) u[k] = fmaf(f, u[k], p.os * w[k]);
                    if (p.out_f32) {
                        if (i < rows) {
                            float *dst = (float *)p.out + ((t0 + i) * args.HV + hv) * D + c0 + 32 * q;
#pragma unroll
                            for (int k = 0; k < 32; k += 4) *(float4 *)(dst + k) = *(const float4 *)&u[k];
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) *(uint4 *)(tile + sw128(i, 32 * q + 8 * k)) = pack8(u + 8 * k);
                    }
                }
                if (!p.out_f32) {
                    if (rows == kC) fence_proxy_async();
                    bar_sync(1, 128);
                    if (rows == kC) {
                        if (tid == 384) {
                            tma_store_3d(&maps.out[blockIdx.y], tile, c0, hv, (int)t0);
                            tma_store_commit();
                        }
                    } else {
                        for (int k = i; k < rows * 8; k += 128)
                            *(uint4 *)((__nv_bfloat16 *)p.out + ((t0 + (k >> 3)) * args.HV + hv) * D + c0 + 8 * (k & 7)) =
                                *(const uint4 *)(tile + sw128(k >> 3, 8 * (k & 7)));
                    }
                }
            }
            if (tid == 384) tma_store_wait0();
        }
    } else if (warp >= 16) {
        // ---------------------------------------------------------------- C: c's rows scaled (thread = row)
        const int j = tid - 512;
        for (int m = 0; m < nm; ++m) {
            const int rows = part.rows(part.chunk(m, rev));
            uint8_t *const stage = sm + (m % kStages) * G::kStage, *const src = stage + G::kCc;
            if (!all(wait(kFull + m % kStages, (m / kStages) & 1))) break;
            if (m == ragged) {  // the rows behind the end are the next sequence's, and 0 x NaN is NaN
                if (j >= rows) {
#pragma unroll
                    for (int b = 0; b <= G::kBoxes; ++b)
#pragma unroll
                        for (int i = 0; i < 8; ++i) *(uint4 *)(stage + G::kB + b * kBox + j * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kFix]);
            }
            const float f = j < rows ? p.cs * decay_pow(g2, rev ? j : rows - 1 - j) : 0.f;
            uint4 hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 raw = *(const uint4 *)(src + sw128(j, 8 * i));
                const uint32_t *w = (const uint32_t *)&raw;
                uint32_t *ph = (uint32_t *)&hi[i], *pl = (uint32_t *)&lo[i];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float u = f * __uint_as_float(w[k] << 16), v = f * __uint_as_float(w[k] & 0xffff0000u);
                    ph[k] = pack_bf16(u, v);
                    pl[k] = pack_bf16(u - __uint_as_float(ph[k] << 16), v - __uint_as_float(ph[k] & 0xffff0000u));
                }
            }
            if (m > 0 && !all(wait(kXF, (m - 1) & 1))) break;  // the products have read the last chunk's
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                *(uint4 *)(sm + G::kHi + sw128(j, 8 * i)) = hi[i];
                *(uint4 *)(sm + G::kLo + sw128(j, 8 * i)) = lo[i];
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

// What the segments add to the state -> the state that enters each (in place), one thread per element
template <int D>
__global__ void lin_join_kernel(const LinArgs args, const Split split)
{
    const LinPass &p = args.pass[blockIdx.y];
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t pair = e / (D * D);
    const int at = (int)(e % (D * D)), n = (int)(pair / args.HV), hv = (int)(pair % args.HV);
    if (n >= args.N) return;
    const SeqRange s = seq_range(args.cu, n, args.T);
    const int64_t slot0 = args.cu ? clamp64(args.cu[n], 0, args.T) / split.tokens + n : (int64_t)n * ((args.T + split.tokens - 1) / split.tokens);
    const float g = args.decay ? args.decay[hv] : 0.f;
    const int segs = (s.len + split.tokens - 1) / split.tokens;
    // tokens of a segment in the order of processing: against time the first has the sequence's odd end
    const int odd = (s.len + kC - 1) / kC * kC - s.len;
    float x = p.x0 ? p.x0[pair * D * D + (p.x_t ? (at % D) * D + at / D : at)] : 0.f;
    float *buf = split.states + (((int64_t)blockIdx.y * split.slots + slot0) * args.HV + hv) * D * D + at;
    const Decayed first(g, split.tokens - (p.reverse ? odd + 1 : 0)), rest(g, split.tokens);
    for (int i = 0; i < segs; ++i, buf += (int64_t)args.HV * D * D) {
        const float add = i + 1 < segs ? *buf : 0.f;
        *buf = x;
        x = (i == 0 ? first(x) : rest(x)) + add;
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
        if (!p.out_f32 && !heads_map(&maps.out[i], p.out, D, a.HV, tokens, (int64_t)a.HV * D, kC)) return cudaErrorInvalidValue;
    }
    const LinPlan plan = lin_tc_plan(a, D);
    Split split{};
    split.slots = plan.slots;
    split.tokens = plan.tokens;
    split.states = plan.bytes ? (float *)ws : nullptr;
    static std::atomic<uint64_t> seen;
    if (first_on_device(seen)) {
        cudaError_t e = cudaFuncSetAttribute(lin_tc_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(lin_tc_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
        if (e != cudaSuccess) return e;
        done_on_device(seen);
    }
    const int64_t ctas = plan.slots * a.HV * (D / kCols), elements = (int64_t)a.N * a.HV * D * D;
    if (ctas > INT32_MAX || elements / 256 > INT32_MAX) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas, a.passes);
    const int withhold = withhold_loads();
    const uint64_t limit = withhold ? kTestWaitLimitNs : kWaitLimitNs;
    if (split.states) {
        lin_tc_kernel<D, true><<<grid, kThreads, Geo<D>::kSmem, st>>>(maps, a, split, limit, withhold);
        lin_join_kernel<D><<<dim3((unsigned)((elements + 255) / 256), a.passes), 256, 0, st>>>(a, split);
    }
    lin_tc_kernel<D, false><<<grid, kThreads, Geo<D>::kSmem, st>>>(maps, a, split, limit, withhold);
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

LinPlan lin_tc_plan(const LinArgs &a, int D)
{
    // A split walks its chunks twice (the second time with outputs), so it pays only where (sequence, head) pairs leave SMs
    // idle: the time of a plan is taken as rounds of CTAs times chunks of a segment, a chunk of the first walk as 0.6 of one.
    const int64_t total = a.cu ? (a.T + kC - 1) / kC : (int64_t)a.N * ((a.T + kC - 1) / kC);  // chunks, and per sequence (packed: on average)
    const int64_t each = std::max<int64_t>(1, (total + a.N - 1) / a.N), ctas = (int64_t)a.N * a.HV * (D / kCols) * a.passes, sms = device_sm_count();
    int64_t best = 1;
    double least = 1e30;
    for (int64_t s = 1; s <= std::min<int64_t>(64, (each + 3) / 4); ++s) {
        const int64_t per = (each + s - 1) / s;
        const double t = (double)((ctas * s + sms - 1) / sms) * (double)per * (s > 1 ? 1.6 : 1.0) + (s > 1 ? 8.0 : 0.0);
        if (t < least) least = t, best = s;
    }
    LinPlan p{};
    if (best == 1) {
        p.slots = a.N;
        return p;
    }
    p.tokens = (int)((each + best - 1) / best) * kC;
    p.slots = mix_slots(a.cu != nullptr, a.N, a.T, p.tokens);
    p.bytes = (size_t)a.passes * p.slots * a.HV * D * D * sizeof(float);
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
