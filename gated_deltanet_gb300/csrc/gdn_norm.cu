// Root-mean-square norm of rows with the residual's addition, in bf16 / fp32 or e4m3 with a scale per
// row, and its gradients:
//
//   h = x + r;   n = sqrt(mean(h^2) + eps);   y = w h / n
//   e4m3:  s = max(max|y| / 448, 2^-126),  q = y / s
//   dx = dh + (w dy - h mean(w dy h) / n^2) / n,   dw = sum over rows of dy h / n
//
// Bound: HBM.  Each input is read once and each output written once: a row stays in the registers of the
// threads that share it while its sums meet, by shuffles and, for rows
// shared by several warps, one exchange through shared memory.  max|y| is taken as max|w h| / n, so that
// both statistics of a quantised row meet in the same exchange.  A block walks rows a grid apart with the
// next rows already on their way; the weights stay in registers.  Measured, 16384 rows of 2048 in bf16: norm with the
// residual 43.9 us, 6.1 TB/s; gradients 53.7 us, 5.0 TB/s at 70 % of all issue slots.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kRowThreads = 512;     // threads of a block, at most
constexpr int kMaxGroups = 4;        // groups of 16 bytes of a row per thread, at most
constexpr int kMaxSingles = 16;      // single elements of a row per thread, at most
constexpr int kWide = 8192;          // wider rows take the looping kernels (512 threads hold this much either way)
constexpr float kE4m3Max = 448.f, kScaleMin = 1.17549435e-38f;  // 2^-126: the smallest normal scale

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The scale of a row from max|w h| and 1 / n; NaN for a row that holds an infinity (inf - inf) or a NaN
__device__ __forceinline__ float row_scale(float most, float rn) { return max_nan(most * rn / kE4m3Max, kScaleMin) + (most - most); }

// VEC elements (16 bytes, or one element) as they are in memory
template <typename T, int VEC> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *(const uint4 *)p; }
    __device__ __forceinline__ void to(float *f) const
    {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};
template <> struct Raw<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = *(const float4 *)p; }
    __device__ __forceinline__ void to(float *f) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <typename T> struct Raw<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void to(float *f) const { f[0] = to_f(v); }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&p;
}
__device__ __forceinline__ uint32_t pack4_e4m3(const float *f)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
template <int VEC> __device__ __forceinline__ void put(__nv_bfloat16 *p, const float *f)
{
    if constexpr (VEC == 8) *(uint4 *)p = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    else *p = __float2bfloat16_rn(f[0]);
}
template <int VEC> __device__ __forceinline__ void put(float *p, const float *f)
{
    if constexpr (VEC == 4) *(float4 *)p = make_float4(f[0], f[1], f[2], f[3]);
    else *p = f[0];
}
template <int VEC> __device__ __forceinline__ void put(__nv_fp8_e4m3 *p, const float *f)
{
    if constexpr (VEC == 8) *(uint2 *)p = make_uint2(pack4_e4m3(f), pack4_e4m3(f + 4));
    else if constexpr (VEC == 4) *(uint32_t *)p = pack4_e4m3(f);
    else *p = from_f<__nv_fp8_e4m3>(f[0]);
}

__device__ __forceinline__ float weight_at(const void *w, gdn_dtype dt, int64_t i)
{
    if (!w) return 1.f;
    return dt == GDN_F32 ? ((const float *)w)[i] : __bfloat162float(((const __nv_bfloat16 *)w)[i]);
}

// What meets beside a row's sum of squares: nothing, another sum, or a maximum
enum Second : int { kNone, kSum, kMax };
// (sum of a, sum or maximum of b) over the tpr threads of a row; every one of them gets both.  `buf` is this
// row's half of a double buffer, so one barrier per row is enough.
template <int SECOND>
__device__ __forceinline__ float2 row_reduce(float a, float b, int tpr, float2 *buf)
{
    auto meet = [&](float o) { return SECOND == kMax ? max_nan(b, o) : b + o; };
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        if (off < tpr) {
            a += __shfl_xor_sync(0xffffffffu, a, off);
            if (SECOND != kNone) b = meet(__shfl_xor_sync(0xffffffffu, b, off));
        }
    }
    if (tpr > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = tpr >> 5, w0 = warp / nw * nw;
        if (lane == 0) buf[warp] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane < nw ? buf[w0 + lane] : make_float2(0.f, 0.f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int off = 8; off; off >>= 1) {
            if (off < nw) {
                a += __shfl_xor_sync(0xffffffffu, a, off);
                if (SECOND != kNone) b = meet(__shfl_xor_sync(0xffffffffu, b, off));
            }
        }
        a = __shfl_sync(0xffffffffu, a, 0);
        if (SECOND != kNone) b = __shfl_sync(0xffffffffu, b, 0);
    }
    return make_float2(a, b);
}

__device__ __forceinline__ void copy16(void *smem, const void *g)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The rows ahead of the one a thread works on.  16-byte groups come by asynchronous copies into slots of the
// thread's own (no other thread reads them, so a thread only waits for its own copies), kAhead rows deep: the
// copies in flight, not registers or resident blocks, cover the memory's latency.  Single elements (rows off 16
// bytes) are loaded into registers, one row ahead, zero where the row has none: what is done with them needs no
// condition and no branch (16384 rows of 1001: 36.7 us with a branch for each, 21.9 so; backward 64.2 and 56.7).
template <typename T, int VEC, int VPT, int TENSORS>
struct RowsAhead {
    static constexpr bool kAsync = VEC > 1;
    static constexpr int kAhead = !kAsync ? 1 : VPT == 1 ? 4 : VPT == 2 ? 3 : 2;
    static size_t bytes(int threads) { return kAsync ? (size_t)kAhead * TENSORS * VPT * threads * 16 : 0; }

    uint4 *slots;  // [kAhead][TENSORS][VPT][threads]
    const T *src[TENSORS];
    int64_t ld[TENSORS];
    int64_t step, M;
    int t, tpr, nv;
    Raw<T, VEC> held[kAsync ? 1 : TENSORS][kAsync ? 1 : VPT];

    __device__ __forceinline__ uint4 *slot(int stage, int k, int i) const
    {
        return slots + ((stage * TENSORS + k) * VPT + i) * blockDim.x + threadIdx.x;
    }
    __device__ __forceinline__ void fetch(int64_t row, int stage)
    {
        if constexpr (!kAsync) {
#pragma unroll
            for (int k = 0; k < TENSORS; ++k) {
                if (!src[k]) continue;
                const T *p = src[k] + row * ld[k] + t;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    held[k][i].v = from_f<T>(0.f);
                    if (t + i * tpr < nv && row < M) held[k][i].load(p + i * tpr);
                }
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * tpr;
            if (v < nv && row < M)
#pragma unroll
                for (int k = 0; k < TENSORS; ++k) {
                    if (!src[k]) continue;
                    copy16(slot(stage, k, i), src[k] + row * ld[k] + (int64_t)v * VEC);
                }
        }
        copies_done();
    }
    __device__ __forceinline__ void start(int64_t row)
    {
        for (int s = 0; s < (kAsync ? kAhead - 1 : 1); ++s) fetch(row + s * step, s);
    }
    // this thread's elements of tensor k of the row of round `it` (they are there: call after ready())
    __device__ __forceinline__ void ready()
    {
        if constexpr (kAsync) copies_wait<kAhead - 2>();
    }
    __device__ __forceinline__ void get(int it, int k, int i, float *f) const
    {
        if constexpr (kAsync) {
            Raw<T, VEC> r;
            r.v = *(const decltype(r.v) *)slot(it % kAhead, k, i);
            r.to(f);
        } else {
            held[k][i].to(f);
        }
    }
    // ask for the row that comes kAhead - 1 rounds later (single elements: the next one)
    __device__ __forceinline__ void next(int64_t row, int it)
    {
        if constexpr (kAsync) fetch(row + (kAhead - 1) * step, (it + kAhead - 1) % kAhead);
        else fetch(row + step, 0);
    }
};

// tpr threads (a power of two) per row, VPT groups of VEC elements each
template <typename T, typename TO, int VEC, int VPT>
__global__ void __launch_bounds__(kRowThreads) norm_kernel(NormArgs a, int tpr)
{
    __shared__ float2 red[2][kRowThreads / 32];
    grid_release();
    grid_wait();
    const int t = threadIdx.x & (tpr - 1), rpb = blockDim.x / tpr, nv = a.D / VEC;
    const int64_t step = (int64_t)gridDim.x * rpb;
    const T *x = (const T *)a.x, *r = (const T *)a.r;
    extern __shared__ uint4 ahead_slots[];
    RowsAhead<T, VEC, VPT, 2> in;
    in.slots = ahead_slots;
    in.src[0] = x; in.src[1] = r;
    in.ld[0] = a.ldx; in.ld[1] = a.ldr;
    in.step = step; in.M = a.M; in.t = t; in.tpr = tpr; in.nv = nv;
    int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
    in.start(row);
    float w[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (t + i * tpr) * VEC + j;
            w[i][j] = c < a.D ? weight_at(a.w, a.w_dt, c) : 0.f;
        }
    // every thread of a block runs the same number of rounds (they meet in the reduction)
    const int rounds = (int)((a.M - (int64_t)blockIdx.x * rpb + step - 1) / step);
    for (int it = 0; it < rounds; ++it, row += step) {
        float h[VPT][VEC];
        float ss = 0.f, mx = 0.f;
        in.ready();
        if constexpr (VEC == 1) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) in.get(it, 0, i, h[i]);
            if (r) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float q;
                    in.get(it, 1, i, &q);
                    h[i][0] += q;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if constexpr (VEC > 1) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) h[i][j] = 0.f;
            }
            if (VEC > 1 && t + i * tpr < nv && row < a.M) {
                in.get(it, 0, i, h[i]);
                if (r) {
                    float q[VEC];
                    in.get(it, 1, i, q);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) h[i][j] += q[j];
                }
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                ss = fmaf(h[i][j], h[i][j], ss);
                if (sizeof(TO) == 1) mx = max_nan(mx, fabsf(h[i][j] * w[i][j]));
            }
        }
        const int64_t cur = row;
        in.next(row, it);
        const float2 s = row_reduce<sizeof(TO) == 1 ? kMax : kNone>(ss, mx, tpr, red[it & 1]);
        const float rn = a.normalise ? 1.f / sqrtf(s.x / (float)a.D + a.eps) : 1.f;
        float inv = 1.f;
        if (sizeof(TO) == 1) {
            const float sc = row_scale(s.y, rn);
            inv = 1.f / sc;
            if (t == 0 && cur < a.M) a.scale[cur] = sc;
        }
        if (cur >= a.M) continue;
        if constexpr (VEC == 1) {
            T *const hp = (T *)a.h + cur * a.D + t;
            TO *const yp = (TO *)a.y + cur * a.D + t;
            if (a.h) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (t + i * tpr < nv) hp[i * tpr] = from_f<T>(h[i][0]);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float y = h[i][0] * rn * w[i][0];
                if (sizeof(TO) == 1) y *= inv;
                if (t + i * tpr < nv) yp[i * tpr] = from_f<TO>(y);
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * tpr;
            if (v >= nv) continue;
            if (a.h) put<VEC>((T *)a.h + cur * a.D + (int64_t)v * VEC, h[i]);
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                y[j] = h[i][j] * rn * w[i][j];
                if (sizeof(TO) == 1) y[j] *= inv;
            }
            put<VEC>((TO *)a.y + cur * a.D + (int64_t)v * VEC, y);
        }
    }
}

// Rows of any width: one block per row, read twice (the second time from the caches)
template <typename T, typename TO>
__global__ void __launch_bounds__(kRowThreads) norm_wide_kernel(NormArgs a)
{
    __shared__ float2 red[2][kRowThreads / 32];
    grid_release();
    grid_wait();
    const T *x = (const T *)a.x, *r = (const T *)a.r;
    int it = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, ++it) {
        auto at = [&](int c) {
            const float v = to_f(x[row * a.ldx + c]);
            return r ? v + to_f(r[row * a.ldr + c]) : v;
        };
        float ss = 0.f, mx = 0.f;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float h = at(c);
            ss = fmaf(h, h, ss);
            if (sizeof(TO) == 1) mx = max_nan(mx, fabsf(h * weight_at(a.w, a.w_dt, c)));
        }
        const float2 s = row_reduce<sizeof(TO) == 1 ? kMax : kNone>(ss, mx, blockDim.x, red[it & 1]);
        const float rn = a.normalise ? 1.f / sqrtf(s.x / (float)a.D + a.eps) : 1.f;
        float inv = 1.f;
        if (sizeof(TO) == 1) {
            const float sc = row_scale(s.y, rn);
            inv = 1.f / sc;
            if (threadIdx.x == 0) a.scale[row] = sc;
        }
        // (h may be r itself: it is written only here, by the thread that reads the same element)
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float h = at(c);
            if (a.h) ((T *)a.h)[row * a.D + c] = from_f<T>(h);
            float y = h * rn * weight_at(a.w, a.w_dt, c);
            if (sizeof(TO) == 1) y *= inv;
            ((TO *)a.y)[row * a.D + c] = from_f<TO>(y);
        }
    }
}

// The gradients of one row from (sum h^2, sum w dy h):  n = sqrt(mean h^2 + eps),
// dx = dh + (w dy - h mean(w dy h) / n^2) / n; the block's rows add dy h / n to dw in registers
template <typename T, int VEC, int VPT>
__global__ void __launch_bounds__(kRowThreads) norm_bwd_kernel(NormBwdArgs a, int tpr)
{
    __shared__ float2 red[2][kRowThreads / 32];
    grid_release();
    grid_wait();
    extern __shared__ uint4 ahead_slots[];
    const int t = threadIdx.x & (tpr - 1), rpb = blockDim.x / tpr, nv = a.D / VEC;
    const int64_t step = (int64_t)gridDim.x * rpb;
    const T *gy = (const T *)a.dy, *gh = (const T *)a.h, *gd = (const T *)a.dh;
    RowsAhead<T, VEC, VPT, 3> in;
    in.slots = ahead_slots;
    in.src[0] = gy; in.src[1] = gh; in.src[2] = gd;
    in.ld[0] = a.ld_dy; in.ld[1] = a.ld_h; in.ld[2] = a.ld_dh;
    in.step = step; in.M = a.M; in.t = t; in.tpr = tpr; in.nv = nv;
    int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
    in.start(row);
    float w[VPT][VEC], dw[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (t + i * tpr) * VEC + j;
            w[i][j] = c < a.D ? weight_at(a.w, a.w_dt, c) : 0.f;
            dw[i][j] = 0.f;
        }
    const int rounds = (int)((a.M - (int64_t)blockIdx.x * rpb + step - 1) / step);
    for (int it = 0; it < rounds; ++it, row += step) {
        // (the row's elements are read from their slots twice: held in registers they would cost occupancy)
        constexpr bool kTwice = RowsAhead<T, VEC, VPT, 3>::kAsync;
        float hk[kTwice ? 1 : VPT][VEC], dyk[kTwice ? 1 : VPT][VEC], dhk[kTwice ? 1 : VPT][VEC];
        float ss = 0.f, sd = 0.f;
        in.ready();
        const bool live = row < a.M;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (kTwice && !(t + i * tpr < nv && live)) continue;
            float h[VEC], dy[VEC];
            in.get(it, 0, i, dy);
            in.get(it, 1, i, h);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                ss = fmaf(h[j], h[j], ss);
                sd = fmaf(w[i][j] * dy[j], h[j], sd);
            }
            if constexpr (!kTwice) {
                hk[i][0] = h[0];
                dyk[i][0] = dy[0];
                dhk[i][0] = 0.f;
            }
        }
        if (!kTwice && gd) {
#pragma unroll
            for (int i = 0; i < (kTwice ? 0 : VPT); ++i) in.get(it, 2, i, dhk[i]);
        }
        const int64_t cur = row;
        if constexpr (!kTwice) in.next(row, it);
        const float2 s = row_reduce<kSum>(ss, sd, tpr, red[it & 1]);
        // (threads without a row have zeros, which with eps = 0 would give an infinite 1 / n and NaN in dw)
        const float rn = kTwice || live ? 1.f / sqrtf(s.x / (float)a.D + a.eps) : 0.f;
        const float c = s.y / (float)a.D * rn * rn * rn;  // dx = dh + w dy / n - h c
        T *const dxp = (T *)a.dx + cur * a.D + t;         // (single elements)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * tpr;
            if (kTwice && !(v < nv && live)) continue;
            float h[VEC], dy[VEC], dx[VEC];
            if constexpr (kTwice) {
                in.get(it, 0, i, dy);
                in.get(it, 1, i, h);
                if (gd) {
                    in.get(it, 2, i, dx);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) dx[j] = 0.f;
                }
            } else {
                dy[0] = dyk[i][0];
                h[0] = hk[i][0];
                dx[0] = dhk[i][0];
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = dy[j] * rn;
                dx[j] = fmaf(-h[j], c, fmaf(w[i][j], g, dx[j]));
                dw[i][j] = fmaf(g, h[j], dw[i][j]);
            }
            if constexpr (kTwice) put<VEC>((T *)a.dx + cur * a.D + (int64_t)v * VEC, dx);
            else if (v < nv && live) dxp[i * tpr] = from_f<T>(dx[0]);
        }
        if constexpr (kTwice) in.next(row, it);
    }
    if (!a.dw) return;
    if (rpb == 1) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (t + i * tpr < nv)
#pragma unroll
                for (int j = 0; j < VEC; ++j) a.part[(int64_t)blockIdx.x * a.D + (t + i * tpr) * VEC + j] = dw[i][j];
        return;
    }
    // several rows per block: their sums meet in the slots, [rows per block][D]
    float *dws = (float *)ahead_slots;
    const int grp = threadIdx.x / tpr;
    if constexpr (RowsAhead<T, VEC, VPT, 3>::kAsync) copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (t + i * tpr < nv)
#pragma unroll
            for (int j = 0; j < VEC; ++j) dws[grp * a.D + (t + i * tpr) * VEC + j] = dw[i][j];
    __syncthreads();
    for (int cidx = threadIdx.x; cidx < a.D; cidx += blockDim.x) {
        float s = 0.f;
        for (int q = 0; q < rpb; ++q) s += dws[q * a.D + cidx];
        a.part[(int64_t)blockIdx.x * a.D + cidx] = s;
    }
}

// Wide rows: dx and (where dw needs it) 1 / n of every row, either alone where its pointer is null; dw by columns
template <typename T>
__global__ void __launch_bounds__(kRowThreads) norm_bwd_wide_kernel(NormBwdArgs a)
{
    __shared__ float2 red[2][kRowThreads / 32];
    grid_release();
    grid_wait();
    const T *gy = (const T *)a.dy, *gh = (const T *)a.h, *gd = (const T *)a.dh;
    int it = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, ++it) {
        float ss = 0.f, sd = 0.f;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float h = to_f(gh[row * a.ld_h + c]);
            ss = fmaf(h, h, ss);
            sd = fmaf(weight_at(a.w, a.w_dt, c) * to_f(gy[row * a.ld_dy + c]), h, sd);
        }
        const float2 s = row_reduce<kSum>(ss, sd, blockDim.x, red[it & 1]);
        const float rn = 1.f / sqrtf(s.x / (float)a.D + a.eps);
        const float k = s.y / (float)a.D * rn * rn;
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rn;
        if (!a.dx) continue;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float h = to_f(gh[row * a.ld_h + c]);
            float dx = (weight_at(a.w, a.w_dt, c) * to_f(gy[row * a.ld_dy + c]) - h * k) * rn;
            if (gd) dx += to_f(gd[row * a.ld_dh + c]);
            ((T *)a.dx)[row * a.D + c] = from_f<T>(dx);
        }
    }
}
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_wide_kernel(NormBwdArgs a)
{
    grid_release();
    grid_wait();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.D) return;
    const T *gy = (const T *)a.dy, *gh = (const T *)a.h;
    float s = 0.f;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y)
        s = fmaf(to_f(gy[row * a.ld_dy + c]), to_f(gh[row * a.ld_h + c]) * a.rstd[row], s);
    a.part[(int64_t)blockIdx.y * a.D + c] = s;
}

bool aligned16(const void *p, int64_t ld, int esz) { return ((uintptr_t)p & 15) == 0 && (ld * esz) % 16 == 0; }

// Groups (16 bytes, or single elements) of a row per thread, threads per row, the block.  The statistics' exchange
// costs a thread about as many instructions as twenty elements do, and with one group a thread the kernels are
// bound by instructions before they are by memory (16384 rows of 2048 in bf16: norm 33.0 us at 75 % of all issue
// slots, 28.4 with four groups; backward 67.5 us, 59.0 with four and 53.9 with two, whose weight sums leave registers
// for more threads), so a thread takes up to four (backward: two) as long as every SM has 512 threads; few
// rows are spread over as many threads as they have groups.
struct RowPlan {
    int vec, vpt, tpr, threads;
};
RowPlan plan_rows(int64_t M, int D, int esz, bool vec_ok, bool backward, int num_sms)
{
    RowPlan p;
    p.vec = vec_ok ? 16 / esz : 1;
    const int nv = (D + p.vec - 1) / p.vec, least = vec_ok ? 1 : 4;
    const int most = vec_ok ? (backward ? 2 : kMaxGroups) : backward ? least : kMaxSingles;
    auto threads_of = [&](int vpt) {
        int t = 1;
        while (t * vpt < nv) t *= 2;
        return t;
    };
    p.vpt = most;
    while (threads_of(p.vpt) > kRowThreads) p.vpt *= vec_ok ? 2 : 4;  // (the backward's most, where it does not hold a row)
    while (p.vpt > least && threads_of(p.vpt / (vec_ok ? 2 : 4)) <= kRowThreads && M * threads_of(p.vpt) < (int64_t)num_sms * 512)
        p.vpt /= vec_ok ? 2 : 4;
    p.tpr = threads_of(p.vpt);
    // (backward: two rows of 2048 a block, whose dw meet before they are written)
    const int block = backward ? 256 : 128;
    p.threads = p.tpr < block ? block : p.tpr;
    return p;
}

int64_t norm_blocks(int64_t M, const RowPlan &p, int num_sms)
{
    const int64_t need = (M + p.threads / p.tpr - 1) / (p.threads / p.tpr);
    // what the registers (and the rows ahead in shared memory) leave room for
    const int room = p.vec > 1 ? (p.vpt == 1 ? 1024 : p.vpt == 2 ? 768 : 512) : p.vpt == 4 ? 1024 : 512;
    const int64_t most = (int64_t)num_sms * (room > p.threads ? room / p.threads : 1);
    return need < most ? need : most;
}

// launches with the dynamic shared memory allowed once per device
template <typename F, typename A>
cudaError_t launch_rows(F *kern, std::atomic<uint64_t> &seen, const A &a, unsigned grid, const RowPlan &p, size_t bytes, cudaStream_t st)
{
    if (bytes > 40 * 1024 && first_on_device(seen)) {  // (beside the static 256 bytes)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) return e;
        done_on_device(seen);
    }
    return launch_overlapped(kern, grid, 1, p.threads, bytes, 0, st, a, p.tpr);
}
template <typename T, typename TO, int VEC, int VPT>
cudaError_t norm_rows(const NormArgs &a, const RowPlan &p, unsigned grid, cudaStream_t st)
{
    static std::atomic<uint64_t> seen;
    return launch_rows(norm_kernel<T, TO, VEC, VPT>, seen, a, grid, p, RowsAhead<T, VEC, VPT, 2>::bytes(p.threads), st);
}
template <typename T, int VEC, int VPT>
cudaError_t norm_bwd_rows(const NormBwdArgs &a, const RowPlan &p, unsigned grid, cudaStream_t st)
{
    static std::atomic<uint64_t> seen;
    const size_t ring = RowsAhead<T, VEC, VPT, 3>::bytes(p.threads);
    const size_t sums = p.threads > p.tpr ? (size_t)(p.threads / p.tpr) * a.D * sizeof(float) : 0;
    return launch_rows(norm_bwd_kernel<T, VEC, VPT>, seen, a, grid, p, ring > sums ? ring : sums, st);
}

template <typename T, typename TO>
cudaError_t norm_go(const NormArgs &a, cudaStream_t st)
{
    constexpr int V = 16 / (int)sizeof(T);
    const int sms = device_sm_count();
    if (a.D > kWide) {
        const int64_t most = (int64_t)sms * 4;
        return launch_overlapped(norm_wide_kernel<T, TO>, (unsigned)(a.M < most ? a.M : most), 1, kRowThreads, 0, 0, st, a);
    }
    const bool ok = a.D % V == 0 && aligned16(a.x, a.ldx, sizeof(T)) && (!a.r || aligned16(a.r, a.ldr, sizeof(T))) &&
                    ((uintptr_t)a.y & 15) == 0 && ((uintptr_t)a.h & 15) == 0;
    const RowPlan p = plan_rows(a.M, a.D, sizeof(T), ok, false, sms);
    const unsigned grid = (unsigned)norm_blocks(a.M, p, sms);
    if (p.vec == 1) return p.vpt == 4 ? norm_rows<T, TO, 1, 4>(a, p, grid, st) : norm_rows<T, TO, 1, kMaxSingles>(a, p, grid, st);
    if (p.vpt == 1) return norm_rows<T, TO, V, 1>(a, p, grid, st);
    if (p.vpt == 2) return norm_rows<T, TO, V, 2>(a, p, grid, st);
    return norm_rows<T, TO, V, kMaxGroups>(a, p, grid, st);
}

bool bwd_vec(const NormBwdArgs &a, int esz)
{
    return a.D % (16 / esz) == 0 && aligned16(a.dy, a.ld_dy, esz) && aligned16(a.h, a.ld_h, esz) &&
           (!a.dh || aligned16(a.dh, a.ld_dh, esz)) && ((uintptr_t)a.dx & 15) == 0;
}

constexpr int kWideParts = 64;

// Whether dx lies over rows that the sums of dw read too
bool dx_over_inputs(const NormBwdArgs &a, size_t esz)
{
    const auto over = [&](const void *p, int64_t ld) {
        const uintptr_t d = (uintptr_t)a.dx, q = (uintptr_t)p;
        return d < q + ((a.M - 1) * ld + a.D) * esz && q < d + (size_t)a.M * a.D * esz;
    };
    return over(a.dy, a.ld_dy) || over(a.h, a.ld_h);
}

template <typename T>
cudaError_t norm_bwd_go(const NormBwdArgs &a, int sms, cudaStream_t st)
{
    constexpr int V = 16 / (int)sizeof(T);
    int64_t parts;
    cudaError_t e = cudaSuccess;
    if (norm_bwd_wide(a.D)) {
        // dw reads dy and h once more, with 1 / n of the rows: after the pass that has it and writes dx, but before dx where
        // dx takes the place of dy (by one more pass over the rows for 1 / n alone)
        const int64_t most = (int64_t)sms * 4;
        const bool first = a.dw && dx_over_inputs(a, sizeof(T));
        NormBwdArgs rows = a;
        if (first) rows.dx = nullptr;
        const auto walk = [&] {
            return launch_overlapped(norm_bwd_wide_kernel<T>, (unsigned)(a.M < most ? a.M : most), 1, kRowThreads, 0, 0, st, rows);
        };
        e = walk();
        parts = a.M < kWideParts ? a.M : kWideParts;
        if (a.dw && e == cudaSuccess)
            e = launch_overlapped(norm_dw_wide_kernel<T>, (unsigned)((a.D + 255) / 256), (unsigned)parts, 256, 0, 0, st, a);
        if (first && e == cudaSuccess) {
            rows.dx = a.dx;
            rows.rstd = nullptr;
            e = walk();
        }
    } else {
        const RowPlan p = plan_rows(a.M, a.D, sizeof(T), bwd_vec(a, sizeof(T)), true, sms);
        const unsigned grid = (unsigned)norm_blocks(a.M, p, sms);
        parts = grid;
        if (p.vec == 1) {
            if (p.vpt == 4) e = norm_bwd_rows<T, 1, 4>(a, p, grid, st);
            else e = norm_bwd_rows<T, 1, kMaxSingles>(a, p, grid, st);
        } else if (p.vpt == 1) {
            e = norm_bwd_rows<T, V, 1>(a, p, grid, st);
        } else if (p.vpt == 2) {
            e = norm_bwd_rows<T, V, 2>(a, p, grid, st);
        } else {
            e = norm_bwd_rows<T, V, kMaxGroups>(a, p, grid, st);
        }
    }
    if (e != cudaSuccess || !a.dw) return e;
    return launch_colsum_finish(a.part, parts, a.D, a.dw, st);
}

}  // namespace

bool norm_bwd_wide(int D) { return D > kWide; }

int norm_bwd_parts(int64_t M, int D, gdn_dtype dt, int num_sms)
{
    if (norm_bwd_wide(D)) return (int)(M < kWideParts ? M : kWideParts);
    // the larger of the vector and the single-element form (alignment is not known here)
    const int esz = dt == GDN_F32 ? 4 : 2;
    int64_t parts = norm_blocks(M, plan_rows(M, D, esz, false, true, num_sms), num_sms);
    if (D % (16 / esz) == 0) {
        const int64_t q = norm_blocks(M, plan_rows(M, D, esz, true, true, num_sms), num_sms);
        parts = q > parts ? q : parts;
    }
    return (int)parts;
}

cudaError_t launch_norm(const NormArgs &a, cudaStream_t st)
{
    if (a.M <= 0) return cudaSuccess;
    if (a.dt == GDN_F32) return a.out_dt == GDN_E4M3 ? norm_go<float, __nv_fp8_e4m3>(a, st) : norm_go<float, float>(a, st);
    return a.out_dt == GDN_E4M3 ? norm_go<__nv_bfloat16, __nv_fp8_e4m3>(a, st) : norm_go<__nv_bfloat16, __nv_bfloat16>(a, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, int num_sms, cudaStream_t st)
{
    if (a.M <= 0) return a.dw ? cudaMemsetAsync(a.dw, 0, a.D * sizeof(float), st) : cudaSuccess;
    return a.dt == GDN_F32 ? norm_bwd_go<float>(a, num_sms, st) : norm_bwd_go<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace gdn
