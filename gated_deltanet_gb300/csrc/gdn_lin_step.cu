// Linear attention with a decay for each head, token by token (decoding, short continuations):
//   S <- l S + k_t v_t^T,  o_t = scale S^T q_t
//
// It has the state's traffic, 8 K V bytes per (sequence, value head), for a token or a few.  One CTA of 256 threads holds
// 64 columns of the state in registers for all tokens of its sequence: thread (row group y, column quad x) has rows y + 16 i and
// four columns, so that a row is read as 256 consecutive bytes and all of a thread's loads (8 of 16 bytes at K = 128) are in
// flight together.  Per token the read-out is a sum over the thread's rows, a shuffle between the warp's two row groups and a sum
// over eight warps in shared memory.  ht may be h0 itself: every element is read and written by the same thread.
// 64 sequences, 16 heads of 128 x 128: 27.7 us, 4.9 TB/s, of which DRAM sees two thirds in the launch and is 46 % busy: bound by three CTAs an
// SM (74 registers) that load, compute and store with nothing to cover one's stores by the next one's loads.  One sequence of 8 heads: 5.7.
#include "gdn_mix.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kCols = 64, kMaxD = 256;

template <typename T, int ROWS, bool VEC>
__global__ void __launch_bounds__(kThreads) lin_step_kernel(const LinStepArgs a)
{
    const int nct = (a.V + kCols - 1) / kCols;
    const int ct = (int)(blockIdx.x % nct), hv = (int)(blockIdx.x / nct % a.HV), n = (int)(blockIdx.x / ((unsigned)nct * a.HV));
    const int h = hv / (a.HV / a.H);
    const int tid = threadIdx.x, x = tid & 15, y = tid >> 4, warp = tid >> 5, lane = tid & 31;
    const int c0 = ct * kCols + 4 * x;
    const SeqRange s = seq_range(a.cu, n, a.T);
    const int64_t base = ((int64_t)n * a.HV + hv) * a.K * a.V;
    __shared__ float qk[2][2][kMaxD];  // [token parity][q, k]
    __shared__ float part[2][8][kCols];

    float S[ROWS][4];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = y + 16 * i;
        if constexpr (VEC) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a.h0 && r < a.K && c0 < a.V) f = *(const float4 *)(a.h0 + base + (int64_t)r * a.V + c0);
            S[i][0] = f.x; S[i][1] = f.y; S[i][2] = f.z; S[i][3] = f.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) S[i][k] = a.h0 && r < a.K && c0 + k < a.V ? a.h0[base + (int64_t)r * a.V + c0 + k] : 0.f;
        }
    }
    const Decayed down(a.decay ? a.decay[hv] : 0.f, 1);
    auto stage = [&](int t) {  // q and k of token t
        const int64_t row = s.bos + t;
        for (int i = tid; i < 2 * a.K; i += kThreads) {
            const int d = i < a.K ? i : i - a.K;
            qk[t & 1][i >= a.K][d] = i < a.K ? to_f<T>(((const T *)a.q)[row * a.ldq + (int64_t)h * a.K + d])
                                             : to_f<T>(((const T *)a.k)[row * a.ldk + (int64_t)h * a.K + d]);
        }
    };
    auto value = [&](int t, float *v) {
        const T *p = (const T *)a.v + (s.bos + t) * a.ldv + (int64_t)hv * a.V + c0;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = c0 + k < a.V ? to_f<T>(p[k]) : 0.f;
    };
    float v[4] = {};
    if (s.len > 0) {
        stage(0);
        value(0, v);
    }
    __syncthreads();
    for (int t = 0; t < s.len; ++t) {
        float vn[4] = {};
        if (t + 1 < s.len) {
            stage(t + 1);
            value(t + 1, vn);
        }
        float o[4] = {};
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = y + 16 * i;
            if (r < a.K) {
                const float q = qk[t & 1][0][r], k = qk[t & 1][1][r];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    S[i][j] = fmaf(k, v[j], down(S[i][j]));
                    o[j] = fmaf(q, S[i][j], o[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += __shfl_xor_sync(0xffffffffu, o[j], 16);
        if (lane < 16) *(float4 *)&part[t & 1][warp][4 * x] = make_float4(o[0], o[1], o[2], o[3]);
        __syncthreads();  // (also: the next token's q and k are there; the buffers of this parity are read before its next write)
        if (tid < kCols && ct * kCols + tid < a.V) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) sum += part[t & 1][w][tid];
            ((T *)a.o)[((s.bos + t) * a.HV + hv) * a.V + ct * kCols + tid] = from_f<T>(a.scale * sum);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = vn[j];
    }
    if (a.ht) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = y + 16 * i;
            if constexpr (VEC) {
                if (r < a.K && c0 < a.V) *(float4 *)(a.ht + base + (int64_t)r * a.V + c0) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r < a.K && c0 + k < a.V) a.ht[base + (int64_t)r * a.V + c0 + k] = S[i][k];
            }
        }
    }
}

template <typename T>
cudaError_t launch(const LinStepArgs &a, cudaStream_t st)
{
    const int64_t blocks = (int64_t)a.N * a.HV * ((a.V + kCols - 1) / kCols);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const bool vec = a.V % 4 == 0 && !(((uintptr_t)a.h0 | (uintptr_t)a.ht) & 15);
    auto kern = a.K <= 64 ? (vec ? lin_step_kernel<T, 4, true> : lin_step_kernel<T, 4, false>)
              : a.K <= 128 ? (vec ? lin_step_kernel<T, 8, true> : lin_step_kernel<T, 8, false>)
                           : (vec ? lin_step_kernel<T, 16, true> : lin_step_kernel<T, 16, false>);
    kern<<<(unsigned)blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_step(const LinStepArgs &a, gdn_dtype dt, cudaStream_t st)
{
    return dt == GDN_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace gdn
