// Attention of a few new tokens over a cache, with a sliding window and sinks (decoding).
//
// Bound by the window's keys and values, which are read once for all query heads of a key head: a CTA takes up to `R` rows (a row: a
// new token's query head) of one key head and one share of the keys they see.  The shares of an item are the CTAs of a cluster: each
// keeps its running maximum, sum and output, and at the end they add up one another's through distributed shared memory, so that a
// call is one launch and needs no workspace.
//   step_mma_kernel   bf16 heads of 64 and 128 on 16-byte boundaries, R = 16: each of four warps walks its own tiles of 16 keys, which
//                     arrive by cp.async (16 bytes a lane) some tiles ahead, S = Q K^T and O += P V by mma.sync (a tile of 128 queries
//                     for tcgen05 would be mostly empty; the keys' bytes bound the call all the same)
//   step_any_kernel   everything else, R = 8: tiles of 32 keys through shared memory, fp32 on the CUDA cores.  Bound by a tile's chain (loads,
//                     barrier, products, barrier; no tile is loaded ahead): the arithmetic of fp32 heads of 128 below is 30 us of 593
// 64 sequences, window 4096, 16 heads over 4: bf16 heads of 128 103 us, 5.2 TB/s; of 64 79; of 96 443; fp32 of 128 593 (read element by element
// 830, 876).  One sequence, window 1024: 10.2 us, launch and latency.
#include "gdn_mix.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kThreads = 128, kMostShares = 8;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// a float in the same place of another CTA's shared memory
__device__ __forceinline__ float peer_float(const float *p, uint32_t rank)
{
    uint32_t at;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ void cp_async16(uint32_t smem, const void *gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}

// What a CTA works on
struct Item {
    int n, hk, row0, rows;   // rows row0 .. of the T x (H / HK) of this key head
    int len, group;
    int first, lo, count;    // keys seen by any of its rows: [0, first) and `count` - first from lo on
    __device__ Item(const WinStepArgs &a, int64_t item, int R)
    {
        group = a.H / a.HK;
        const int all = a.T * group, tiles = (all + R - 1) / R;
        row0 = (int)(item % tiles) * R;
        rows = min(R, all - row0);
        hk = (int)(item / tiles % a.HK);
        n = (int)(item / ((int64_t)tiles * a.HK));
        len = (int)clamp64(a.lengths_64 ? ((const int64_t *)a.lengths)[n] : ((const int *)a.lengths)[n], 0, a.S);
        const int p0 = len - a.T + row0 / group, p1 = len - a.T + (row0 + rows - 1) / group, hi = max(p1 + 1, 0);
        lo = min(max(p0 - a.window + 1, 0), hi);
        first = min(a.sinks, lo);
        count = first + hi - lo;
    }
    __device__ int key(int i) const { return i < first ? i : lo + i - first; }
    __device__ int position(const WinStepArgs &a, int r) const { return len - a.T + (row0 + r) / group; }
    // element of row r in q (strided) or o
    __device__ int64_t at(const WinStepArgs &a, int r, int64_t ld) const
    {
        const int row = row0 + r, t = row / group, g = row - t * group;
        return ((int64_t)n * a.T + t) * ld + (int64_t)(hk * group + g) * a.D;
    }
};

// The cluster's rows: parts O [R][D + 4], top [R], total [R] of each CTA (maxima in units of log 2, O and total relative to them)
template <typename T, int R>
__device__ __forceinline__ void join_shares(const WinStepArgs &a, const Item &it, const float *O, const float *top, const float *total, int stride)
{
    const uint32_t n = cluster_size(), me = cluster_rank();
    if (n > 1) cluster_sync();
    else __syncthreads();
    for (int i = (int)me * kThreads + threadIdx.x; i < it.rows * a.D; i += (int)n * kThreads) {
        const int r = i / a.D, d = i - r * a.D;
        float m = -INFINITY, sum = 0.f, o = 0.f;
        for (uint32_t c = 0; c < n; ++c) m = fmaxf(m, n > 1 ? peer_float(top + r, c) : top[r]);
        const float base = m == -INFINITY ? 0.f : m;
        for (uint32_t c = 0; c < n; ++c) {
            const float w = exp2f((n > 1 ? peer_float(top + r, c) : top[r]) - base);
            sum = fmaf(w, n > 1 ? peer_float(total + r, c) : total[r], sum);
            o = fmaf(w, n > 1 ? peer_float(O + r * stride + d, c) : O[r * stride + d], o);
        }
        ((T *)a.o)[it.at(a, r, (int64_t)a.H * a.D) + d] = from_f<T>(sum == 0.f ? 0.f : o / sum);
    }
    if (n > 1) cluster_sync();  // (the others read this CTA's shared memory)
}

// ---------------------------------------------------------------- bf16 by mma.sync
constexpr int kKeys = 16;

template <int D>
struct StepGeo {
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kTile = kKeys * D * 2, kStage = 2 * kTile, kWarp = kStages * kStage;
    static constexpr int kRows = 16, kStride = D + 4;
    static constexpr int kParts = 4 * kRows * kStride * 4;  // four warps' outputs, over the dead stages
    static constexpr int kSmem = (4 * kWarp > kParts ? 4 * kWarp : kParts) + 4 * kRows * 2 * 4;
};
// byte of 16-byte piece c of row r in a tile of D elements a row
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4)); }

template <int D>
__global__ void __launch_bounds__(kThreads) step_mma_kernel(const WinStepArgs a)
{
    using G = StepGeo<D>;
    extern __shared__ __align__(128) uint8_t step_smem[];
    const uint32_t shares = cluster_size(), share = cluster_rank();
    const Item it(a, blockIdx.x / shares, 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 3, row = lane >> 2;
    const __nv_bfloat16 *K = (const __nv_bfloat16 *)a.k + it.n * a.k_seq + it.hk * a.k_head, *V = (const __nv_bfloat16 *)a.v + it.n * a.v_seq + it.hk * a.v_head;
    const int tiles = (it.count + kKeys - 1) / kKeys, t0 = (int)((int64_t)tiles * share / shares), t1 = (int)((int64_t)tiles * (share + 1) / shares);
    const uint32_t mine = smem_u32(step_smem) + warp * G::kWarp;

    auto load = [&](int t, int s) {  // keys and values of tile t, the last key again where there are fewer
        const uint32_t at = mine + s * G::kStage;
#pragma unroll
        for (int i = 0; i < kKeys * D / 8 / 32; ++i) {
            const int e = i * 32 + lane, r = e / (D / 8), c = e % (D / 8);
            const int64_t j = it.key(min(t * kKeys + r, it.count - 1));
            cp_async16(at + piece<D>(r, c), K + j * a.k_tok + c * 8);
            cp_async16(at + G::kTile + piece<D>(r, c), V + j * a.v_tok + c * 8);
        }
    };
#pragma unroll
    for (int s = 0; s < G::kStages - 1; ++s) {
        if (t0 + warp + 4 * s < t1) load(t0 + warp + 4 * s, s);
        cp_async_commit();
    }
    // Q as left operands: rows `row` and `row` + 8, elements 16 k + 2 quad and + 8
    uint32_t q[D / 16][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = row + 8 * h;
        const __nv_bfloat16 *src = (const __nv_bfloat16 *)a.q + (r < it.rows ? it.at(a, r, a.ldq) : 0);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) q[k][h + 2 * e] = r < it.rows ? *(const uint32_t *)(src + 16 * k + 8 * e + 2 * quad) : 0u;
    }
    const float c = a.scale * kLog2e;
    const int p[2] = {it.position(a, min(row, it.rows - 1)), it.position(a, min(row + 8, it.rows - 1))};
    float top[2] = {-INFINITY, -INFINITY}, total[2] = {0.f, 0.f}, o[D / 8][4] = {};
    int s = 0;
    for (int t = t0 + warp; t < t1; t += 4) {
        const int ahead = t + 4 * (G::kStages - 1), free = s == 0 ? G::kStages - 1 : s - 1;
        if (ahead < t1) load(ahead, free);
        cp_async_commit();
        cp_async_wait<G::kStages - 1>();
        __syncwarp();
        const uint32_t kt = mine + s * G::kStage, vt = kt + G::kTile;
        float z[2][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            // matrices: keys 0-7 and 8-15, elements 16 k .. + 7 and + 8 .. + 15
            uint32_t b[4];
            ldsm_x4(b, kt + piece<D>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
            mma_bf16_16816(z[0], q[k][0], q[k][1], q[k][2], q[k][3], b[0], b[1]);
            mma_bf16_16816(z[1], q[k][0], q[k][1], q[k][2], q[k][3], b[2], b[3]);
        }
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float m = top[h];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = t * kKeys + 8 * g + 2 * quad + e, j = it.key(i);
                    float &x = z[g][2 * h + e];
                    x = i < it.count && win_sees(p[h], j, a.window, a.sinks) ? x * c : -INFINITY;
                    m = fmaxf(m, x);
                }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float base = m == -INFINITY ? 0.f : m, fix = exp2f(top[h] - base);
            top[h] = m;
            total[h] *= fix;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                o[d][2 * h] *= fix;
                o[d][2 * h + 1] *= fix;
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float u = exp2f(z[g][2 * h] - base), v = exp2f(z[g][2 * h + 1] - base);
                total[h] += u + v;
                w[h + 2 * g] = pack_bf16(u, v);
            }
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            // matrices: keys 0-7 and 8-15, elements 16 d .. + 7, then + 8 .. + 15, transposed
            uint32_t b[4];
            const uint32_t at = vt + piece<D>(lane & 15, 2 * d + (lane >> 4));
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                         : "r"(at)
                         : "memory");
            mma_bf16_16816(o[2 * d], w[0], w[1], w[2], w[3], b[0], b[1]);
            mma_bf16_16816(o[2 * d + 1], w[0], w[1], w[2], w[3], b[2], b[3]);
        }
        __syncwarp();  // (the stage is loaded again next time round)
        s = s + 1 == G::kStages ? 0 : s + 1;
    }
    cp_async_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        total[h] += __shfl_xor_sync(0xffffffffu, total[h], 1);
        total[h] += __shfl_xor_sync(0xffffffffu, total[h], 2);
    }
    // the four warps' parts: maxima first, then the outputs relative to the rows' maximum, added up in order
    float *const O = (float *)step_smem, *const stat = (float *)(step_smem + G::kSmem - 4 * G::kRows * 2 * 4);  // [warp][top, total][row]
    if (quad == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            stat[warp * 32 + row + 8 * h] = top[h];
            stat[warp * 32 + 16 + row + 8 * h] = total[h];
        }
    }
    __syncthreads();
    float best[2], fix[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        best[h] = -INFINITY;
        for (int v = 0; v < 4; ++v) best[h] = fmaxf(best[h], stat[v * 32 + row + 8 * h]);
        fix[h] = exp2f(top[h] - (best[h] == -INFINITY ? 0.f : best[h]));
    }
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
            *(float2 *)(O + (warp * G::kRows + row + 8 * h) * G::kStride + 8 * d + 2 * quad) = make_float2(o[d][2 * h] * fix[h], o[d][2 * h + 1] * fix[h]);
    __syncthreads();
    for (int i = tid; i < G::kRows * D; i += kThreads) {
        const int at = i / D * G::kStride + i % D;
        float x = O[at];
        for (int v = 1; v < 4; ++v) x += O[v * G::kRows * G::kStride + at];
        O[at] = x;
    }
    float sum = 0.f, m = -INFINITY;
    if (tid < G::kRows) {
        for (int v = 0; v < 4; ++v) m = fmaxf(m, stat[v * 32 + tid]);
        for (int v = 0; v < 4; ++v) sum = fmaf(exp2f(stat[v * 32 + tid] - (m == -INFINITY ? 0.f : m)), stat[v * 32 + 16 + tid], sum);
    }
    __syncthreads();
    if (tid < G::kRows) {
        stat[tid] = m;
        stat[16 + tid] = sum;
    }
    join_shares<__nv_bfloat16, G::kRows>(a, it, O, stat, stat + 16, G::kStride);
}

// ---------------------------------------------------------------- any type and size, on the CUDA cores
constexpr int kAnyRows = 8, kAnyKeys = 32;

// E elements of 16 bytes as fp32
template <typename T>
__device__ __forceinline__ void spread(float *dst, uint4 x)
{
    if constexpr (sizeof(T) == 4) {
        *(uint4 *)dst = x;
    } else {
        *(float4 *)dst = make_float4(low_bf16(x.x), high_bf16(x.x), low_bf16(x.y), high_bf16(x.y));
        *(float4 *)(dst + 4) = make_float4(low_bf16(x.z), high_bf16(x.z), low_bf16(x.w), high_bf16(x.w));
    }
}

// WIDE: the cache's rows are on 16 bytes and a multiple of them long
template <typename T, int DP, bool WIDE>
__global__ void __launch_bounds__(kThreads) step_any_kernel(const WinStepArgs a)
{
    constexpr int kStride = DP + 4, kCols = (DP + kThreads - 1) / kThreads;
    extern __shared__ float4 step_any_smem[];
    float *const K = (float *)step_any_smem, *const V = K + kAnyKeys * kStride, *const Q = V + kAnyKeys * kStride, *const O = Q + kAnyRows * kStride;
    float *const P = O + kAnyRows * kStride, *const stat = P + kAnyRows * kAnyKeys;  // P [row][key]; stat: top, total, factor of each row
    const uint32_t shares = cluster_size(), share = cluster_rank();
    const Item it(a, blockIdx.x / shares, kAnyRows);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T *Kg = (const T *)a.k + it.n * a.k_seq + it.hk * a.k_head, *Vg = (const T *)a.v + it.n * a.v_seq + it.hk * a.v_head;
    for (int i = tid; i < kAnyRows * DP; i += kThreads) {
        const int r = i / DP, d = i % DP;
        Q[r * kStride + d] = r < it.rows && d < a.D ? to_f<T>(((const T *)a.q)[it.at(a, r, a.ldq) + d]) : 0.f;
    }
    if (tid < kAnyRows) {
        stat[tid] = -INFINITY;
        stat[kAnyRows + tid] = 0.f;
    }
    const int tiles = (it.count + kAnyKeys - 1) / kAnyKeys, t0 = (int)((int64_t)tiles * share / shares), t1 = (int)((int64_t)tiles * (share + 1) / shares);
    const float c = a.scale * kLog2e;
    float acc[kCols][kAnyRows] = {};
    for (int t = t0; t < t1; ++t) {
        const int keys = min(kAnyKeys, it.count - t * kAnyKeys);
        __syncthreads();
        if constexpr (WIDE) {  // (all of a thread's loads in flight: element by element a tile waited four times)
            constexpr int E = 16 / sizeof(T), kPer = DP / E, kAll = kAnyKeys * kPer / kThreads, kBatch = kAll < 8 ? kAll : 8;
#pragma unroll 1
            for (int b = 0; b < kAll; b += kBatch) {
                uint4 k[kBatch], v[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = tid + (b + u) * kThreads, r = i / kPer, d = i % kPer * E;
                    const bool in = r < keys && d < a.D;
                    const int64_t j = it.key(t * kAnyKeys + (in ? r : 0));
                    k[u] = in ? *(const uint4 *)(Kg + j * a.k_tok + d) : make_uint4(0, 0, 0, 0);
                    v[u] = in ? *(const uint4 *)(Vg + j * a.v_tok + d) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = tid + (b + u) * kThreads, r = i / kPer, d = i % kPer * E;
                    spread<T>(K + r * kStride + d, k[u]);
                    spread<T>(V + r * kStride + d, v[u]);
                }
            }
        } else {
#pragma unroll 8
            for (int i = tid; i < kAnyKeys * DP; i += kThreads) {
                const int r = i / DP, d = i % DP;
                const bool in = r < keys && d < a.D;
                const int64_t j = it.key(t * kAnyKeys + (in ? r : 0));
                K[r * kStride + d] = in ? to_f<T>(Kg[j * a.k_tok + d]) : 0.f;
                V[r * kStride + d] = in ? to_f<T>(Vg[j * a.v_tok + d]) : 0.f;
            }
        }
        __syncthreads();
        {  // rows warp and warp + 4, key lane
            float z[2] = {};
            for (int d = 0; d < a.D; d += 4) {
                const float4 k = *(const float4 *)(K + lane * kStride + d);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 q = *(const float4 *)(Q + (warp + 4 * h) * kStride + d);
                    z[h] += q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
                }
            }
            const int j = it.key(t * kAnyKeys + min(lane, keys - 1));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = warp + 4 * h;
                const float x = lane < keys && r < it.rows && win_sees(it.position(a, min(r, it.rows - 1)), j, a.window, a.sinks) ? z[h] * c : -INFINITY;
                float m = x;
#pragma unroll
                for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
                m = fmaxf(m, stat[r]);
                const float base = m == -INFINITY ? 0.f : m, e = exp2f(x - base);
                float sum = e;
#pragma unroll
                for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
                P[r * kAnyKeys + lane] = e;
                __syncwarp();
                if (lane == 0) {
                    const float fix = exp2f(stat[r] - base);
                    stat[2 * kAnyRows + r] = fix;
                    stat[kAnyRows + r] = fmaf(stat[kAnyRows + r], fix, sum);
                    stat[r] = m;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kCols; ++u) {
            const int d = tid + u * kThreads;
            if (d >= DP) continue;
#pragma unroll
            for (int r = 0; r < kAnyRows; ++r) acc[u][r] *= stat[2 * kAnyRows + r];
            for (int k = 0; k < kAnyKeys; k += 4) {
                const float v[4] = {V[k * kStride + d], V[(k + 1) * kStride + d], V[(k + 2) * kStride + d], V[(k + 3) * kStride + d]};
#pragma unroll
                for (int r = 0; r < kAnyRows; ++r) {
                    const float4 p = *(const float4 *)(P + r * kAnyKeys + k);
                    acc[u][r] += p.x * v[0] + p.y * v[1] + p.z * v[2] + p.w * v[3];
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kCols; ++u) {
        const int d = tid + u * kThreads;
        if (d < DP)
            for (int r = 0; r < kAnyRows; ++r) O[r * kStride + d] = acc[u][r];
    }
    join_shares<T, kAnyRows>(a, it, O, stat, stat + kAnyRows, kStride);
}

// CTAs that share an item: enough to fill the GPU some times over (the rounds' last one is then short), none without work
int shares_of(const WinStepArgs &a, int64_t items, int keys_each)
{
    const int64_t most = std::min<int64_t>(a.S, (int64_t)a.window + a.sinks + a.T);
    int n = 1;
    while (n < kMostShares && items * n < 4 * (int64_t)device_sm_count() && most >= (int64_t)2 * n * keys_each) n *= 2;
    return n;
}

template <typename K>
cudaError_t launch(K kern, const WinStepArgs &a, int R, int keys_each, size_t smem, std::atomic<uint64_t> &seen, cudaStream_t st)
{
    if (first_on_device(seen)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        done_on_device(seen);
    }
    const int64_t rows = (int64_t)a.T * (a.H / a.HK), items = (int64_t)a.N * a.HK * ((rows + R - 1) / R);
    const int shares = shares_of(a, items, keys_each);
    if (items * shares > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * shares));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)shares;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}
template <typename T, int DP>
cudaError_t launch_any(const WinStepArgs &a, cudaStream_t st)
{
    constexpr int E = 16 / sizeof(T);
    static std::atomic<uint64_t> seen[2];
    const size_t smem = 4 * ((2 * kAnyKeys + 2 * kAnyRows) * (DP + 4) + kAnyRows * kAnyKeys + 3 * kAnyRows);
    const int64_t strides = a.k_seq | a.k_tok | a.k_head | a.v_seq | a.v_tok | a.v_head;
    const bool wide = strides % E == 0 && a.D % E == 0 && !(((uintptr_t)a.k | (uintptr_t)a.v) & 15);
    return wide ? launch(step_any_kernel<T, DP, true>, a, kAnyRows, kAnyKeys, smem, seen[1], st)
                : launch(step_any_kernel<T, DP, false>, a, kAnyRows, kAnyKeys, smem, seen[0], st);
}
template <typename T>
cudaError_t launch_any(const WinStepArgs &a, cudaStream_t st)
{
    return a.D <= 64 ? launch_any<T, 64>(a, st) : a.D <= 128 ? launch_any<T, 128>(a, st) : launch_any<T, 256>(a, st);
}

}  // namespace

cudaError_t launch_win_step(const WinStepArgs &a, gdn_dtype dt, cudaStream_t st)
{
    if (dt == GDN_F32) return launch_any<float>(a, st);
    const int64_t strides = a.k_seq | a.k_tok | a.k_head | a.v_seq | a.v_tok | a.v_head;
    if ((a.D == 64 || a.D == 128) && strides % 8 == 0 && !(((uintptr_t)a.k | (uintptr_t)a.v) & 15) && !((uintptr_t)a.q & 3) && a.ldq % 2 == 0) {
        static std::atomic<uint64_t> seen[2];
        return a.D == 64 ? launch(step_mma_kernel<64>, a, 16, 4 * kKeys, StepGeo<64>::kSmem, seen[0], st)
                         : launch(step_mma_kernel<128>, a, 16, 4 * kKeys, StepGeo<128>::kSmem, seen[1], st);
    }
    return launch_any<__nv_bfloat16>(a, st);
}

}  // namespace gdn
