// Internal declarations of the token mixers beside the gated delta rule: linear attention with a decay for each head, and
// softmax attention with a sliding window and first tokens that stay visible.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

// ---------------------------------------------------------------- sequences
// Where sequence n stands among `total` tokens: packed by cu (n + 1 offsets) or one of equal length T.  Offsets are clamped to
// the tensor, so that a malformed table can give wrong results but no access outside.
struct SeqRange {
    int64_t bos;
    int len;
};
__host__ __device__ inline int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }
__device__ __forceinline__ SeqRange seq_range(const int64_t *cu, int n, int T)
{
    if (!cu) return {(int64_t)n * T, T};
    const int64_t b = clamp64(cu[n], 0, T), e = clamp64(cu[n + 1], b, T);
    return {b, (int)(e - b)};
}
// Tiles of `tile` tokens of all sequences in one grid dimension.  Equal lengths: ceil(T / tile) each.  Packed: sequence n has the
// slots from floor(cu[n] / tile) + n on, so that no two share one and total / tile + N + 1 slots are enough; some stay empty.
__host__ __device__ inline int64_t mix_slots(bool packed, int N, int T, int tile)
{
    return packed ? (int64_t)T / tile + N + 1 : (int64_t)N * ((T + tile - 1) / tile);
}
struct Tile {
    int n, index;  // sequence, tile within it
};
// the last n below N with start(n) <= at, or 0 (start does not fall)
template <typename F>
__device__ __forceinline__ int last_from(int N, int64_t at, F start)
{
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start(mid) <= at) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
// The same by a whole warp, 32 of them at a time: where every warp of many CTAs looks a sequence up (each step of the other waits for memory:
// the join of the sinks' gradients of 200 sequences took 130 us more with it)
template <typename F>
__device__ __forceinline__ int last_from_warp(int N, int64_t at, F start)
{
    const int lane = threadIdx.x & 31;
    int lo = 0;
    for (int left = N; left > 1;) {
        const int step = (left + 31) / 32, i = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, i == 0 || (i < left && start(lo + i) <= at));
        const int k = 31 - __clz(below);
        lo += k * step;
        left = min(step, left - k * step);
    }
    return lo;
}
// tile i of sequence n; i outside what a sequence can have: one that is behind every end
__device__ __forceinline__ Tile tile_at(int n, int64_t i, int tile)
{
    const int64_t past = max(INT32_MAX / tile - 1, 1);
    return {n, (int)(i < 0 || i > past ? past : i)};
}
__device__ __forceinline__ Tile tile_of(const int64_t *cu, int N, int T, int tile, int64_t slot)
{
    if (!cu) {
        const unsigned per = (unsigned)(T + tile - 1) / tile, n = (unsigned)slot / per;  // (slots of equal lengths are grid indices: 31 bits)
        return {(int)n, (int)((unsigned)slot - n * per)};
    }
    auto first = [&](int n) { return (int64_t)((unsigned)clamp64(cu[n], 0, T) / (unsigned)tile) + n; };
    const int n = last_from(N, slot, first);
    return tile_at(n, slot - first(n), tile);  // (slots in front of the first sequence are empty too)
}
// Places for the sequences of `least` tokens or more alone: sequence n has min(n, floor(cu[n] / least)), so that no two of them share one and
// floor(T / least) are enough whatever N is.  (Shorter ones' places are others' or nobody's.)  Equal lengths: n.
__host__ __device__ inline int64_t long_places(bool packed, int N, int T, int least)
{
    return !packed ? (T >= least ? N : 0) : T / least < N ? T / least : N;
}
__device__ __forceinline__ int64_t long_place(const int64_t *cu, int n, int T, int least)
{
    if (!cu) return n;
    return min((int)((unsigned)clamp64(cu[n], 0, T) / (unsigned)least), n);
}
// The sequences that are cut, those longer than `tokens`, hold their segments' states one behind the other: sequence n from
// floor(cu[n] / tokens) + its place on (a sequence of more than `tokens` has at most floor(len / tokens) + 1 segments).
__host__ __device__ inline int64_t cut_states(bool packed, int N, int T, int tokens)
{
    return packed ? T / tokens + long_places(packed, N, T, tokens) : (int64_t)N * ((T + tokens - 1) / tokens);
}
__device__ __forceinline__ int64_t cut_state0(const int64_t *cu, int n, int T, int tokens)
{
    return cu ? (int64_t)((unsigned)clamp64(cu[n], 0, T) / (unsigned)tokens) + long_place(cu, n, T, tokens) : (int64_t)n * ((T + tokens - 1) / tokens);
}
// The segment whose state is the at-th (of a sequence that is not cut, or behind its end, where there is none)
__device__ __forceinline__ Tile cut_of(const int64_t *cu, int N, int T, int tokens, int64_t at)
{
    if (!cu) return tile_of(cu, N, T, tokens, at);
    auto first = [&](int n) { return cut_state0(cu, n, T, tokens); };
    const int n = last_from(N, at, first);
    return tile_at(n, at - first(n), tokens);
}

// ---------------------------------------------------------------- linear attention
// One pass of linear attention over every (sequence, value head), in time or against it.  With l = exp(decay), n tokens:
//   out_i = os (cs sum_{j <= i} l^(i-j) (a_i . b_j) c_j + l^(i+1) a_i X0)
//   X1    = cs sum_j l^(n-1-j) b_j c_j^T + l^n X0                                X [da][dc]
// against time: j >= i, l^(j-i), and X0 enters one step later (l^(n-1-i)); X1 = cs sum_j l^j b_j c_j^T + l^(n-1) X0, times l when
// it is written.  The forward is (q, k, v); with dO the gradients are dq = (dO, v, k) in time and dk = (v, dO, q),
// dv = (k, q, dO) against it: the state's gradient R_t = l R_{t+1} + scale q_t dO_t^T runs backward.
struct LinPass {
    const void *a, *b, *c;   // [tokens][heads][da], [..][da], [..][dc]
    int64_t lda, ldb, ldc;   // elements from a token to the next
    int ra, rb, rc;          // value heads that share a head of a, b, c
    void *out;               // [tokens][HV][dc], the inputs' type or (out_f32) fp32; nullable
    const float *x0;         // [N][HV][da][dc], or (x_t) [N][HV][dc][da]; nullable (zero)
    float *x1;               // the same layout, nullable
    float cs, os;
    int da, dc, out_f32, x_t, reverse;
};
struct LinArgs {
    LinPass pass[3];
    int passes;              // 1, or 3 (the gradients)
    const float *decay;      // [HV], nullable (0)
    const int64_t *cu;
    int T, N, HV;            // packed: T = all tokens
    unsigned *status;
};
// bf16, all sizes 64 or all 128, rows on 16-byte boundaries: on the tensor cores.  A plan splits sequences into segments where there
// are few; then `bytes` of workspace.
struct LinPlan {
    size_t bytes;            // of workspace, the last kChosenBytes of them for packed sequences' segment where that is chosen on the device
    int64_t slots;           // (sequence, segment) pairs, some of them empty
    int64_t states, places;  // segments' states held, and sequences that are cut, at most
    int tokens;              // of a segment
};
constexpr size_t kChosenBytes = 256;
LinPlan lin_simt_plan(const LinArgs &a);
cudaError_t launch_lin_simt(const LinArgs &a, gdn_dtype dt, void *ws, cudaStream_t st);
bool lin_tc_ok(const LinArgs &a, int64_t tokens);
LinPlan lin_tc_plan(const LinArgs &a, int D);
cudaError_t launch_lin_tc(const LinArgs &a, void *ws, int64_t tokens, cudaStream_t st);
gdn_status read_lin_status(cudaStream_t st);
// a TMA map over bf16 [tokens][heads][D], `ld` elements from a token to the next: boxes of 64 elements x 1 head x box_rows tokens
bool heads_map(CUtensorMap *m, const void *base, int D, int heads, int64_t tokens, int64_t ld, int box_rows);
// the same over [batch][T][heads][D] by strides (multiples of 8 elements): boxes of a sequence's tokens, zeros behind its end
bool strided_map(CUtensorMap *m, const void *base, int D, int heads, int T, int batch, int64_t head, int64_t tok, int64_t seq, int box_rows);
// dq and dk of heads that r value heads share: out[t][h][d] = sum over i of part[t][h r + i][d], in order (`part`: dq's, then dk's)
cudaError_t launch_lin_heads(const float *part, const LinArgs &a, int64_t tokens, int H, int r, int D, void *dq, void *dk, gdn_dtype dt, cudaStream_t st);

struct LinStepArgs {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *decay, *h0;
    const int64_t *cu;
    void *o;
    float *ht;
    int T, N, H, HV, K, V;
    float scale;
};
cudaError_t launch_lin_step(const LinStepArgs &a, gdn_dtype dt, cudaStream_t st);

// l^x of a log-decay in base 2 and a count of steps; l^0 = 1 for every decay, minus infinity too
__device__ __forceinline__ float decay_pow(float g2, int x) { return x == 0 ? 1.f : exp2f(g2 * (float)x); }
// The state after x steps, l^x X.  Near 1 as X + X (l^x - 1): l^x itself, rounded, would lose the digits of 1 - l^x chunk after chunk.
struct Decayed {
    float f;
    bool near;
    __device__ __forceinline__ Decayed(float g, int x)
    {
        const float d = x == 0 ? 0.f : g * (float)x;
        near = d > -0.5f;
        f = near ? expm1f(d) : expf(d);
    }
    __device__ __forceinline__ float operator()(float X) const { return fmaf(X, f, near ? X : 0.f); }
};

// ---------------------------------------------------------------- window attention
// Query i of a sequence with Lq queries and Lk keys stands at position p = i + Lk - Lq and sees key j when
// j <= p and (p - j < window or j < sinks).
struct WinArgs {
    const void *q, *k, *v;      // [tokens][heads][D]
    int64_t ldq, ldk, ldv;
    const int64_t *cu_q, *cu_k;  // both or none
    int Tq, Tk, N, H, HK, D;
    int window, sinks;          // clamped to [1, Tk] and [0, Tk]
    float scale;
    void *o;                    // [tokens][H][D]
    float *lse;                 // [B][H][Tq] (packed: [H][Tq]), nullable
    int64_t o_seq, o_tok, o_head;  // o's strides in elements (gradients: as the caller has it)
    // gradients
    const void *dout;
    int64_t ld_dout;
    const float *delta;         // rows' sums of dO o, laid out as lse
    void *dq, *dk, *dv;
    unsigned *status;
};
__host__ __device__ inline int64_t lse_at(const WinArgs &a, int n, int64_t bos, int h)
{
    // element of row `bos` (the first of sequence n) and head h
    return a.cu_q ? (int64_t)h * a.Tq + bos : ((int64_t)n * a.H + h) * a.Tq;
}
// Keys that are sinks are seen by every query behind them.  Where the window does not reach, the queries of a tile of sinks are dealt out
// to CTAs of their own, `run` queries each, whose fp32 parts of dK and dV a join adds to the tile's in order: one CTA for all of them would
// walk the whole sequence while the others see a window.  Sequences of fewer than `least` keys, whose sinks have few far queries, stay with their
// tiles' CTAs and have no place here, so that the parts are at most 2 + sinks / run times what dK and dV would take in fp32, however many sequences
// there are.  Few: none behind the tiles of sinks, or half a run where key tiles fill the GPU four times over and a CTA's longer walk costs less
// than the parts' way through memory (bf16, 8 heads over 4 of 128, 4 sinks, dealt out and not: 200 x 300 tokens, window 128 661 us and 501; one
// sequence of 1660, window 1024 103 and 123).
struct WinSinks {
    float *own, *parts;     // [places][HK][tiles][2][tile][D] of the tiles' own CTAs, [slots][HK][tiles][2][tile][D] of the runs
    int tiles;              // tiles of sinks whose far queries are dealt out; 0: none
    int least;
    int64_t places, slots;  // of sequences that are dealt out, of their runs
    __device__ __forceinline__ bool deals(const SeqRange &sq, const SeqRange &sk) const { return tiles > 0 && sq.len > 0 && sk.len >= least; }
    __device__ __forceinline__ int64_t place(const WinArgs &a, int n) const { return long_place(a.cu_k, n, a.Tk, least); }
    // the first run of a sequence that is dealt out
    __device__ __forceinline__ int64_t slot0(const WinArgs &a, int n, int run) const
    {
        return a.cu_q ? (int64_t)((unsigned)clamp64(a.cu_q[n], 0, a.Tq) / (unsigned)run) + place(a, n) : (int64_t)n * ((a.Tq + run - 1) / run);
    }
};
inline WinSinks win_sinks_plan(const WinArgs &a, int tile, int run, int most, void *ws, size_t *bytes)
{
    WinSinks s{};
    const int tiles = (a.sinks + tile - 1) / tile;
    *bytes = 0;
    if (a.window >= a.Tk || tiles > most || tiles == 0) return s;
    const bool packed = a.cu_q != nullptr;
    const bool full = (packed ? 1 : (int64_t)a.N) * a.Tk / tile * a.HK >= 4 * (int64_t)device_sm_count();
    s.least = a.window + tiles * tile + (full ? run / 2 : 0);
    s.places = long_places(packed, a.N, a.Tk, s.least);
    if (s.places == 0) return s;
    s.tiles = tiles;
    s.slots = packed ? a.Tq / run + s.places : (int64_t)a.N * ((a.Tq + run - 1) / run);
    const int64_t each = (int64_t)a.HK * tiles * 2 * tile * a.D;
    s.own = (float *)ws;
    s.parts = s.own + s.places * each;
    *bytes = (size_t)(s.places + s.slots) * each * sizeof(float);
    return s;
}
// What a CTA of dK and dV sums: a tile of keys against queries begin .. end of each head
struct WinKeyTile {
    SeqRange sq, sk;
    int n, j0, cols, off, begin, end;
    float *part;  // fp32 [2][tile][D] (dK, dV) in place of the gradients; null: these
    __device__ __forceinline__ WinKeyTile(const WinArgs &a, const WinSinks &s, int64_t key_tiles, int tile, int run, int64_t item, int hk)
    {
        const bool far = item >= key_tiles;  // a run of queries against a tile of sinks
        if (far) item -= key_tiles;
        const int64_t slot = far ? item / s.tiles : 0;
        Tile tl;
        if (far && a.cu_q) {
            auto first = [&](int n) { return s.slot0(a, n, run); };
            const int last = last_from_warp(a.N, slot, first);
            tl = tile_at(last, slot - first(last), run);
        } else {
            tl = far ? tile_of(nullptr, a.N, a.Tq, run, slot) : tile_of(a.cu_k, a.N, a.Tk, tile, item);
        }
        n = tl.n;
        sq = seq_range(a.cu_q, n, a.Tq);
        sk = seq_range(a.cu_k, n, a.Tk);
        const int st = far ? (int)(item % s.tiles) : tl.index;
        j0 = st * tile;
        cols = min(tile, sk.len - j0);
        off = sk.len - sq.len;
        begin = max(0, j0 - off);
        end = (int)clamp64((int64_t)j0 + cols - 1 + a.window - off, 0, sq.len);  // the last (exclusive) that sees a key through the window
        const bool dealt = !far && st < s.tiles && s.deals(sq, sk);
        if (far) {
            begin = max(max(begin, end), tl.index * run);
            end = (int)min((int64_t)sq.len, (int64_t)(tl.index + 1) * run);
            if (begin >= end || !s.deals(sq, sk)) cols = 0;  // (nothing to do)
        } else if (!dealt && j0 < a.sinks) {
            end = sq.len;
        }
        const int64_t size = (int64_t)2 * tile * a.D;
        part = far ? s.parts + ((slot * a.HK + hk) * s.tiles + st) * size : dealt ? s.own + ((s.place(a, n) * a.HK + hk) * s.tiles + st) * size : nullptr;
    }
};
__device__ __forceinline__ float added(float x, float y) { return x + y; }
__device__ __forceinline__ float4 added(float4 x, float4 y) { return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); }
// The sequence that is dealt out at a place, or -1 (by whole warps)
__device__ __forceinline__ int win_sinks_at(const WinArgs &a, const WinSinks &s, int64_t place)
{
    auto first = [&](int n) { return s.place(a, n); };
    const int n = a.cu_q ? last_from_warp(a.N, place, first) : (int)place;
    return first(n) == place && s.deals(seq_range(a.cu_q, n, a.Tq), seq_range(a.cu_k, n, a.Tk)) ? n : -1;
}
// what stands at `at` in the parts [2][tile][D] of a tile of sinks, added up in order (F: one element, or four)
template <typename F>
__device__ __forceinline__ F win_sinks_sum(const WinArgs &a, const WinSinks &s, int tile, int run, int n, int hk, int st, int64_t at)
{
    const SeqRange sq = seq_range(a.cu_q, n, a.Tq), sk = seq_range(a.cu_k, n, a.Tk);
    const int j0 = st * tile, cols = min(tile, sk.len - j0), off = sk.len - sq.len;
    const int from = max(max(0, j0 - off), (int)clamp64((int64_t)j0 + cols - 1 + a.window - off, 0, sq.len));  // the first query of a run
    const int64_t slot0 = s.slot0(a, n, run), size = (int64_t)2 * tile * a.D;
    F x = *(const F *)(s.own + ((s.place(a, n) * a.HK + hk) * s.tiles + st) * size + at);
    for (int i = from / run; from < sq.len && i * run < sq.len; ++i) x = added(x, *(const F *)(s.parts + (((slot0 + i) * a.HK + hk) * s.tiles + st) * size + at));
    return x;
}
__device__ __forceinline__ bool win_sees(int p, int j, int window, int sinks) { return j <= p && (p - j < window || j < sinks); }
cudaError_t launch_win_simt(const WinArgs &a, gdn_dtype dt, cudaStream_t st);
// bf16 heads of 64 or 128, rows on 16-byte boundaries, a positive scale: on the tensor cores (tq, tk: all tokens)
bool win_tc_ok(const WinArgs &a, int64_t tq, int64_t tk);
cudaError_t launch_win_tc(const WinArgs &a, int64_t tq, int64_t tk, cudaStream_t st);
gdn_status read_win_status(cudaStream_t st);
bool win_bwd_tc_ok(const WinArgs &a, int64_t tq, int64_t tk);
size_t win_bwd_tc_bytes(const WinArgs &a);  // of workspace, beside delta (which the call fills)
cudaError_t launch_win_bwd_tc(const WinArgs &a, int64_t tq, int64_t tk, float *delta, void *ws, cudaStream_t st);
gdn_status read_win_bwd_status(cudaStream_t st);
cudaError_t launch_win_delta(const WinArgs &a, gdn_dtype dt, float *delta, cudaStream_t st);
cudaError_t launch_win_dq_simt(const WinArgs &a, gdn_dtype dt, cudaStream_t st);
size_t win_dkv_simt_bytes(const WinArgs &a);  // of workspace, beside delta
cudaError_t launch_win_dkv_simt(const WinArgs &a, gdn_dtype dt, void *ws, cudaStream_t st);

struct WinStepArgs {
    const void *q;              // [N][T][H][D], token stride ldq
    int64_t ldq;
    const void *k, *v;          // [N][S][HK][D] by strides
    int64_t k_seq, k_tok, k_head, v_seq, v_tok, v_head;
    const void *lengths;        // [N] int32 or int64
    int lengths_64;
    int N, T, S, H, HK, D, window, sinks;
    float scale;
    void *o;                    // [N][T][H][D]
};
cudaError_t launch_win_step(const WinStepArgs &a, gdn_dtype dt, cudaStream_t st);

}  // namespace gdn
