// Attention with a sliding window and sinks on the CUDA cores, forward and gradients: every type, any head size up to 256, any
// alignment.  (bf16 heads of 64 and 128 on 16-byte boundaries take the tensor cores.)
//
// 16 x 16 threads over tiles of TILE queries by TILE keys in fp32, rows ty + 16 r and columns tx + 16 c of the scores per thread,
// operands read 16 bytes at a time along the contraction.  The forward keeps a running maximum and sum per row (one pass over the
// keys); the gradients recompute p = exp(scale s - lse).  dK and dV sum over every query head of a key head in the CTA that owns the
// key tile, in a fixed order and without atomics.  Bound by a tile's chain (loads, products through shared memory) where tiles are few, else by
// reads of shared memory: 2 x 4096 tokens, 4 heads of 64, window 256, fp32: 152 us, gradients 423.
#include "gdn_mix.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -INFINITY;
constexpr int kSinkRun = 256, kMostSinks = 512;  // queries of a run, and sinks up to which they are dealt out (WinSinks)

// TILE rows of D columns as fp32, zeros behind `rows` and D, at a stride of DP + 4
template <typename T, int TILE, int DP>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int64_t ld, int rows, int D)
{
    for (int i = threadIdx.x; i < TILE * DP; i += kThreads) {
        const int r = i / DP, c = i % DP;
        dst[r * (DP + 4) + c] = r < rows && c < D ? to_f<T>(src[(int64_t)r * ld + c]) : 0.f;
    }
}

// z[r][c] = sum_k A[ty + 16 r][k] B[tx + 16 c][k]
template <int RT, int DP>
__device__ __forceinline__ void dot_tile(float (*z)[RT], const float *A, const float *B, int D)
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) z[i][j] = 0.f;
    for (int k = 0; k < D; k += 4) {
        float4 u[RT], v[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            u[i] = *(const float4 *)&A[(ty + 16 * i) * (DP + 4) + k];
            v[i] = *(const float4 *)&B[(tx + 16 * i) * (DP + 4) + k];
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) z[i][j] += u[i].x * v[j].x + u[i].y * v[j].y + u[i].z * v[j].z + u[i].w * v[j].w;
    }
}

// acc[r][4 m + e] += sum_j P[ty + 16 r][j] V[j][64 m + 4 tx + e]   (P at a stride of TILE + 4)
template <int RT, int TILE, int DP>
__device__ __forceinline__ void mul_tile(float (*acc)[DP / 16], const float *P, const float *V)
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int j = 0; j < TILE; j += 4) {
        float p[RT][4];
#pragma unroll
        for (int i = 0; i < RT; ++i) *(float4 *)p[i] = *(const float4 *)&P[(ty + 16 * i) * (TILE + 4) + j];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int m = 0; m < DP / 64; ++m) {
                const float4 v = *(const float4 *)&V[(j + k) * (DP + 4) + 64 * m + 4 * tx];
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    acc[i][4 * m] += p[i][k] * v.x;
                    acc[i][4 * m + 1] += p[i][k] * v.y;
                    acc[i][4 * m + 2] += p[i][k] * v.z;
                    acc[i][4 * m + 3] += p[i][k] * v.w;
                }
            }
    }
}

// rows ty + 16 r of acc to dst (token stride ld)
template <typename T, int RT, int DP>
__device__ __forceinline__ void store_tile(T *dst, int64_t ld, const float (*acc)[DP / 16], int rows, int D)
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) {
            const int r = ty + 16 * i, c = 64 * (e >> 2) + 4 * tx + (e & 3);
            if (r < rows && c < D) dst[(int64_t)r * ld + c] = from_f<T>(acc[i][e]);
        }
}

__device__ __forceinline__ float row_max(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The keys that queries at positions p0 .. p1 (inclusive) may see: [0, first) of the sinks, then [lo, hi)
struct Keys {
    int first, lo, hi;
};
__device__ __forceinline__ Keys keys_of(int p0, int p1, int window, int sinks)
{
    Keys k;
    k.hi = max(p1 + 1, 0);
    k.lo = min(max(p0 - window + 1, 0), k.hi);
    k.first = min(sinks, k.lo);
    return k;
}

template <typename T, int TILE, int DP>
__global__ void __launch_bounds__(kThreads) win_fwd_kernel(const WinArgs a)
{
    constexpr int RT = TILE / 16;
    extern __shared__ float4 win_smem[];
    float *Q = (float *)win_smem, *KV = Q + TILE * (DP + 4), *P = KV + TILE * (DP + 4);
    const Tile tl = tile_of(a.cu_q, a.N, a.Tq, TILE, blockIdx.x);
    const SeqRange sq = seq_range(a.cu_q, tl.n, a.Tq), sk = seq_range(a.cu_k, tl.n, a.Tk);
    const int i0 = tl.index * TILE, rows = min(TILE, sq.len - i0), h = blockIdx.y, hk = h / (a.H / a.HK);
    if (rows <= 0) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, p0 = i0 + sk.len - sq.len;
    const float c = a.scale * kLog2e;
    load_tile<T, TILE, DP>(Q, (const T *)a.q + (sq.bos + i0) * a.ldq + (int64_t)h * a.D, a.ldq, rows, a.D);

    float acc[RT][DP / 16] = {}, top[RT], total[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) top[i] = kNegInf, total[i] = 0.f;
    const Keys ks = keys_of(p0, p0 + rows - 1, a.window, a.sinks);
    const int nfirst = (ks.first + TILE - 1) / TILE, ntiles = nfirst + (ks.hi - ks.lo + TILE - 1) / TILE;
    for (int t = 0; t < ntiles; ++t) {
        const int j0 = t < nfirst ? t * TILE : ks.lo + (t - nfirst) * TILE, end = t < nfirst ? ks.first : ks.hi;
        const int cols = min(TILE, end - j0);
        __syncthreads();
        load_tile<T, TILE, DP>(KV, (const T *)a.k + (sk.bos + j0) * a.ldk + (int64_t)hk * a.D, a.ldk, cols, a.D);
        __syncthreads();
        float z[RT][RT];
        dot_tile<RT, DP>(z, Q, KV, a.D);
        __syncthreads();
        load_tile<T, TILE, DP>(KV, (const T *)a.v + (sk.bos + j0) * a.ldv + (int64_t)hk * a.D, a.ldv, cols, a.D);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = ty + 16 * i;
            float m = top[i];
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int k = tx + 16 * j;
                z[i][j] = k < cols && win_sees(p0 + r, j0 + k, a.window, a.sinks) ? z[i][j] * c : kNegInf;
                m = fmaxf(m, z[i][j]);
            }
            m = row_max(m);
            const float base = m == kNegInf ? 0.f : m, fix = exp2f(top[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const float e = exp2f(z[i][j] - base);
                sum += e;
                P[r * (TILE + 4) + tx + 16 * j] = e;
            }
            total[i] = total[i] * fix + row_sum(sum);
            top[i] = m;
#pragma unroll
            for (int e = 0; e < DP / 16; ++e) acc[i][e] *= fix;
        }
        __syncthreads();
        mul_tile<RT, TILE, DP>(acc, P, KV);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const float inv = total[i] > 0.f ? 1.f / total[i] : total[i] == 0.f ? 0.f : total[i];  // (a NaN stays)
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) acc[i][e] *= inv;
        if (a.lse && tx == 0 && ty + 16 * i < rows)
            a.lse[lse_at(a, tl.n, sq.bos, h) + i0 + ty + 16 * i] = total[i] == 0.f ? kNegInf : (top[i] + log2f(total[i])) * 0.69314718055994531f;
    }
    store_tile<T, RT, DP>((T *)a.o + ((sq.bos + i0) * a.H + h) * a.D, (int64_t)a.H * a.D, acc, rows, a.D);
}

// delta = sum over the head of dO o, one warp per (token, head)
template <typename T>
__global__ void __launch_bounds__(kThreads) win_delta_kernel(const WinArgs a, float *delta, int64_t rows)
{
    const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    if (w >= rows) return;
    const int lane = threadIdx.x & 31, h = (int)(w % a.H);
    const int64_t t = w / a.H;
    const int64_t n = a.cu_q ? 0 : t / a.Tq, i = t - n * a.Tq;
    const T *x = (const T *)a.dout + t * a.ld_dout + (int64_t)h * a.D, *y = (const T *)a.o + n * a.o_seq + i * a.o_tok + h * a.o_head;
    float s = 0.f;
    for (int d = lane; d < a.D; d += 32) s = fmaf(to_f<T>(x[d]), to_f<T>(y[d]), s);
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) delta[lse_at(a, (int)n, 0, h) + i] = s;
}

template <typename T, int TILE, int DP>
__global__ void __launch_bounds__(kThreads) win_dq_kernel(const WinArgs a)
{
    constexpr int RT = TILE / 16, ROW = TILE * (DP + 4);
    extern __shared__ float4 win_smem[];
    float *Q = (float *)win_smem, *G = Q + ROW, *K = G + ROW, *V = K + ROW, *P = V + ROW;
    const Tile tl = tile_of(a.cu_q, a.N, a.Tq, TILE, blockIdx.x);
    const SeqRange sq = seq_range(a.cu_q, tl.n, a.Tq), sk = seq_range(a.cu_k, tl.n, a.Tk);
    const int i0 = tl.index * TILE, rows = min(TILE, sq.len - i0), h = blockIdx.y, hk = h / (a.H / a.HK);
    if (rows <= 0) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, p0 = i0 + sk.len - sq.len;
    load_tile<T, TILE, DP>(Q, (const T *)a.q + (sq.bos + i0) * a.ldq + (int64_t)h * a.D, a.ldq, rows, a.D);
    load_tile<T, TILE, DP>(G, (const T *)a.dout + (sq.bos + i0) * a.ld_dout + (int64_t)h * a.D, a.ld_dout, rows, a.D);
    float lse[RT], delta[RT], acc[RT][DP / 16] = {};
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = ty + 16 * i;
        const int64_t at = lse_at(a, tl.n, sq.bos, h) + i0 + r;
        lse[i] = r < rows ? a.lse[at] * kLog2e : 0.f;
        delta[i] = r < rows ? a.delta[at] : 0.f;
    }
    const Keys ks = keys_of(p0, p0 + rows - 1, a.window, a.sinks);
    const int nfirst = (ks.first + TILE - 1) / TILE, ntiles = nfirst + (ks.hi - ks.lo + TILE - 1) / TILE;
    for (int t = 0; t < ntiles; ++t) {
        const int j0 = t < nfirst ? t * TILE : ks.lo + (t - nfirst) * TILE, end = t < nfirst ? ks.first : ks.hi;
        const int cols = min(TILE, end - j0);
        __syncthreads();
        load_tile<T, TILE, DP>(K, (const T *)a.k + (sk.bos + j0) * a.ldk + (int64_t)hk * a.D, a.ldk, cols, a.D);
        load_tile<T, TILE, DP>(V, (const T *)a.v + (sk.bos + j0) * a.ldv + (int64_t)hk * a.D, a.ldv, cols, a.D);
        __syncthreads();
        float z[RT][RT], dp[RT][RT];
        dot_tile<RT, DP>(z, Q, K, a.D);
        dot_tile<RT, DP>(dp, G, V, a.D);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int r = ty + 16 * i, k = tx + 16 * j;
                const bool seen = r < rows && k < cols && win_sees(p0 + r, j0 + k, a.window, a.sinks);
                P[r * (TILE + 4) + k] = seen ? exp2f(z[i][j] * (a.scale * kLog2e) - lse[i]) * (dp[i][j] - delta[i]) * a.scale : 0.f;
            }
        __syncthreads();
        mul_tile<RT, TILE, DP>(acc, P, K);
    }
    store_tile<T, RT, DP>((T *)a.dq + ((sq.bos + i0) * a.H + h) * a.D, (int64_t)a.H * a.D, acc, rows, a.D);
}

template <typename T, int TILE, int DP>
__global__ void __launch_bounds__(kThreads) win_dkv_kernel(const WinArgs a, const WinSinks sinks, int64_t key_tiles)
{
    constexpr int RT = TILE / 16, ROW = TILE * (DP + 4);
    extern __shared__ float4 win_smem[];
    float *K = (float *)win_smem, *V = K + ROW, *Q = V + ROW, *G = Q + ROW, *P = G + ROW, *Z = P + TILE * (TILE + 4);
    const int hk = blockIdx.y, G_ = a.H / a.HK;
    const WinKeyTile kt(a, sinks, key_tiles, TILE, kSinkRun, blockIdx.x, hk);
    if (kt.cols <= 0) return;
    const SeqRange sq = kt.sq, sk = kt.sk;
    const int n = kt.n, j0 = kt.j0, cols = kt.cols, off = kt.off, begin = kt.begin, end = kt.end;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_tile<T, TILE, DP>(K, (const T *)a.k + (sk.bos + j0) * a.ldk + (int64_t)hk * a.D, a.ldk, cols, a.D);
    load_tile<T, TILE, DP>(V, (const T *)a.v + (sk.bos + j0) * a.ldv + (int64_t)hk * a.D, a.ldv, cols, a.D);
    float dk[RT][DP / 16] = {}, dv[RT][DP / 16] = {};
    for (int g = 0; g < G_; ++g) {
        const int h = hk * G_ + g;
        for (int i0 = begin; i0 < end; i0 += TILE) {
            const int rows = min(TILE, end - i0);
            __syncthreads();
            load_tile<T, TILE, DP>(Q, (const T *)a.q + (sq.bos + i0) * a.ldq + (int64_t)h * a.D, a.ldq, rows, a.D);
            load_tile<T, TILE, DP>(G, (const T *)a.dout + (sq.bos + i0) * a.ld_dout + (int64_t)h * a.D, a.ld_dout, rows, a.D);
            __syncthreads();
            float z[RT][RT], dp[RT][RT];  // [key][query]
            dot_tile<RT, DP>(z, K, Q, a.D);
            dot_tile<RT, DP>(dp, V, G, a.D);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int i = tx + 16 * j;
                const int64_t at = lse_at(a, n, sq.bos, h) + i0 + i;
                const float lse = i < rows ? a.lse[at] * kLog2e : 0.f, delta = i < rows ? a.delta[at] : 0.f;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int k = ty + 16 * r;
                    const bool seen = i < rows && k < cols && win_sees(i0 + i + off, j0 + k, a.window, a.sinks);
                    const float p = seen ? exp2f(z[r][j] * (a.scale * kLog2e) - lse) : 0.f;
                    P[k * (TILE + 4) + i] = p;
                    Z[k * (TILE + 4) + i] = seen ? p * (dp[r][j] - delta) * a.scale : 0.f;
                }
            }
            __syncthreads();
            mul_tile<RT, TILE, DP>(dv, P, G);
            mul_tile<RT, TILE, DP>(dk, Z, Q);
        }
    }
    if (kt.part) {
        store_tile<float, RT, DP>(kt.part, a.D, dk, cols, a.D);
        store_tile<float, RT, DP>(kt.part + TILE * a.D, a.D, dv, cols, a.D);
        return;
    }
    store_tile<T, RT, DP>((T *)a.dk + ((sk.bos + j0) * a.HK + hk) * a.D, (int64_t)a.HK * a.D, dk, cols, a.D);
    store_tile<T, RT, DP>((T *)a.dv + ((sk.bos + j0) * a.HK + hk) * a.D, (int64_t)a.HK * a.D, dv, cols, a.D);
}

// dK and dV of the tiles of sinks: their own part and the runs', in order
template <typename T, int TILE>
__global__ void __launch_bounds__(kThreads) win_sinks_kernel(const WinArgs a, const WinSinks s, int64_t count)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= count) return;  // (a warp has one tile: they are multiples of 64)
    const int size = 2 * TILE * a.D, at = (int)(i % size), which = at / (TILE * a.D), e = at % (TILE * a.D), r0 = e / a.D;
    const int64_t tile = i / size;
    const int st = (int)(tile % s.tiles), hk = (int)(tile / s.tiles % a.HK), n = win_sinks_at(a, s, tile / s.tiles / a.HK), r = st * TILE + r0;
    if (n < 0) return;
    const SeqRange sk = seq_range(a.cu_k, n, a.Tk);
    if (r >= sk.len) return;
    ((T *)(which ? a.dv : a.dk))[((sk.bos + r) * a.HK + hk) * a.D + e % a.D] = from_f<T>(win_sinks_sum<float>(a, s, TILE, kSinkRun, n, hk, st, at));
}

template <typename K>
cudaError_t prepare(K kern, size_t smem, std::atomic<uint64_t> &seen)
{
    if (!first_on_device(seen)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) done_on_device(seen);
    return e;
}
// the forward or dQ: a CTA to a tile of queries of a head
template <typename T, int TILE, int DP>
cudaError_t launch_rows(const WinArgs &a, bool dq, cudaStream_t st)
{
    auto kern = dq ? win_dq_kernel<T, TILE, DP> : win_fwd_kernel<T, TILE, DP>;
    const size_t smem = (dq ? 4 : 2) * TILE * (DP + 4) * 4 + TILE * (TILE + 4) * 4;
    static std::atomic<uint64_t> seen[2];
    const cudaError_t e = prepare(kern, smem, seen[dq]);
    if (e != cudaSuccess) return e;
    const int64_t tiles = mix_slots(a.cu_q != nullptr, a.N, a.Tq, TILE);
    if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (tiles == 0) return cudaSuccess;
    kern<<<dim3((unsigned)tiles, a.H), kThreads, smem, st>>>(a);
    return cudaGetLastError();
}
template <typename T, int TILE, int DP>
cudaError_t launch_keys(const WinArgs &a, void *ws, cudaStream_t st)
{
    auto kern = win_dkv_kernel<T, TILE, DP>;
    const size_t smem = 4 * TILE * (DP + 4) * 4 + 2 * TILE * (TILE + 4) * 4;
    static std::atomic<uint64_t> seen;
    const cudaError_t e = prepare(kern, smem, seen);
    if (e != cudaSuccess) return e;
    size_t bytes;
    const WinSinks s = win_sinks_plan(a, TILE, kSinkRun, kMostSinks / TILE, ws, &bytes);
    const int64_t tiles = mix_slots(a.cu_k != nullptr, a.N, a.Tk, TILE), ctas = tiles + s.slots * s.tiles;
    const int64_t count = s.places * a.HK * s.tiles * 2 * TILE * a.D, blocks = (count + kThreads - 1) / kThreads;
    if (ctas > INT32_MAX || blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (tiles == 0) return cudaSuccess;
    kern<<<dim3((unsigned)ctas, a.HK), kThreads, smem, st>>>(a, s, tiles);
    if (s.tiles > 0) win_sinks_kernel<T, TILE><<<(unsigned)blocks, kThreads, 0, st>>>(a, s, count);
    return cudaGetLastError();
}
// Tiles of 64 (each key and query is read half as often), or of 32 where 64 would leave SMs without a tile, where much of a tile of 64 lies
// outside the window, and for heads whose tiles of 64 do not fit.  fp32, 64 and 32:
//   gradients, window 100, 2048 tokens of 4 heads over 2 of 64 (128 tiles of queries, 64 of keys): 182 us, 145; 300 tokens of 2 heads of 40: 90, 70
//   11502 tokens of 8 heads over 4 of 64: window 35 219, 176, gradients 766, 621; window 128 283, 252, gradients 887, 842
//   2 x 2048 tokens, 4 heads of 64, window 256: 94, 104, gradients 258, 272
//   8 heads of 128, window 128, 4 x 2048 tokens: 346, 412, gradients 1532, 1251
int tile_for(const WinArgs &a, const int64_t *cu, int T, int heads, bool forward)
{
    const bool narrow = a.window <= 128 && (!forward || a.D <= 64);
    return a.D > 128 || narrow || mix_slots(cu != nullptr, a.N, T, 64) * heads < device_sm_count() ? 32 : 64;
}
int key_tile(const WinArgs &a) { return tile_for(a, a.cu_k, a.Tk, a.HK, false); }
template <typename T>
cudaError_t launch_rows_of(const WinArgs &a, bool dq, cudaStream_t st)
{
    if (a.D > 128) return launch_rows<T, 32, 256>(a, dq, st);
    if (tile_for(a, a.cu_q, a.Tq, a.H, !dq) == 32) return a.D <= 64 ? launch_rows<T, 32, 64>(a, dq, st) : launch_rows<T, 32, 128>(a, dq, st);
    return a.D <= 64 ? launch_rows<T, 64, 64>(a, dq, st) : launch_rows<T, 64, 128>(a, dq, st);
}
template <typename T>
cudaError_t launch_keys_of(const WinArgs &a, void *ws, cudaStream_t st)
{
    if (a.D > 128) return launch_keys<T, 32, 256>(a, ws, st);
    if (key_tile(a) == 32) return a.D <= 64 ? launch_keys<T, 32, 64>(a, ws, st) : launch_keys<T, 32, 128>(a, ws, st);
    return a.D <= 64 ? launch_keys<T, 64, 64>(a, ws, st) : launch_keys<T, 64, 128>(a, ws, st);
}
cudaError_t launch_any(const WinArgs &a, gdn_dtype dt, bool dq, cudaStream_t st)
{
    return dt == GDN_F32 ? launch_rows_of<float>(a, dq, st) : launch_rows_of<__nv_bfloat16>(a, dq, st);
}

}  // namespace

cudaError_t launch_win_simt(const WinArgs &a, gdn_dtype dt, cudaStream_t st) { return launch_any(a, dt, false, st); }
cudaError_t launch_win_dq_simt(const WinArgs &a, gdn_dtype dt, cudaStream_t st) { return launch_any(a, dt, true, st); }
cudaError_t launch_win_dkv_simt(const WinArgs &a, gdn_dtype dt, void *ws, cudaStream_t st)
{
    return dt == GDN_F32 ? launch_keys_of<float>(a, ws, st) : launch_keys_of<__nv_bfloat16>(a, ws, st);
}
size_t win_dkv_simt_bytes(const WinArgs &a)
{
    size_t bytes;
    const int tile = key_tile(a);
    win_sinks_plan(a, tile, kSinkRun, kMostSinks / tile, nullptr, &bytes);
    return bytes;
}

cudaError_t launch_win_delta(const WinArgs &a, gdn_dtype dt, float *delta, cudaStream_t st)
{
    const int64_t rows = (a.cu_q ? (int64_t)a.Tq : (int64_t)a.N * a.Tq) * a.H, blocks = (rows * 32 + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (dt == GDN_F32) win_delta_kernel<float><<<(unsigned)blocks, kThreads, 0, st>>>(a, delta, rows);
    else win_delta_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, st>>>(a, delta, rows);
    return cudaGetLastError();
}

}  // namespace gdn
