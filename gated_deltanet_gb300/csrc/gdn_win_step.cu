// Attention of a few new tokens over a cache, with a sliding window and sinks: simple form.
// One CTA per (sequence, key head, new token, query head of the group).
#include "gdn_mix.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads) win_step_kernel(const WinStepArgs a)
{
    __shared__ float q[256], e[kThreads], red[kThreads / 32];
    const int G = a.H / a.HK, tid = threadIdx.x;
    const int h = (int)(blockIdx.x % a.H), t = (int)(blockIdx.x / a.H % a.T), n = (int)(blockIdx.x / ((int64_t)a.H * a.T)), hk = h / G;
    int64_t len = a.lengths_64 ? ((const int64_t *)a.lengths)[n] : ((const int *)a.lengths)[n];
    len = clamp64(len, 0, a.S);
    const int p = (int)len - a.T + t;
    for (int d = tid; d < a.D; d += kThreads) q[d] = to_f<T>(((const T *)a.q)[((int64_t)n * a.T + t) * a.ldq + (int64_t)h * a.D + d]);
    const T *K = (const T *)a.k + n * a.k_seq + hk * a.k_head, *V = (const T *)a.v + n * a.v_seq + hk * a.v_head;
    const int hi = max(p + 1, 0), lo = min(max(p - a.window + 1, 0), hi), first = min(a.sinks, lo), count = first + hi - lo;
    float top = -INFINITY, total = 0.f, acc[2] = {};
    for (int b = 0; b < count; b += kThreads) {
        __syncthreads();
        const int i = b + tid, j = i < first ? i : lo + i - first;
        float z = -INFINITY;
        if (i < count) {
            z = 0.f;
            for (int d = 0; d < a.D; ++d) z = fmaf(q[d], to_f<T>(K[(int64_t)j * a.k_tok + d]), z);
            z *= a.scale * kLog2e;
        }
        float m = z;
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        m = top;
        for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, red[w]);
        const float base = m == -INFINITY ? 0.f : m, fix = exp2f(top - base);
        e[tid] = exp2f(z - base);
        __syncthreads();
        total *= fix;
        acc[0] *= fix;
        acc[1] *= fix;
        const int cols = min(kThreads, count - b);
        for (int k = 0; k < cols; ++k) {
            const int j2 = b + k < first ? b + k : lo + b + k - first;
            total += e[k];
            for (int u = 0; u < 2; ++u)
                if (tid + u * kThreads < a.D) acc[u] = fmaf(e[k], to_f<T>(V[(int64_t)j2 * a.v_tok + tid + u * kThreads]), acc[u]);
        }
        top = m;
    }
    for (int u = 0; u < 2; ++u) {
        const int d = tid + u * kThreads;
        if (d < a.D) ((T *)a.o)[(((int64_t)n * a.T + t) * a.H + h) * a.D + d] = from_f<T>(total == 0.f ? 0.f : acc[u] / total);
    }
}

}  // namespace

cudaError_t launch_win_step(const WinStepArgs &a, gdn_dtype dt, cudaStream_t st)
{
    const int64_t blocks = (int64_t)a.N * a.T * a.H;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (dt == GDN_F32) win_step_kernel<float><<<(unsigned)blocks, kThreads, 0, st>>>(a);
    else win_step_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
