// Linear attention with a decay for each head on the CUDA cores: every type, any head size up to 256.
//
// One CTA per (sequence, value head, 32 columns of c) walks the sequence in chunks of 32 tokens with the state X in registers
// (its owners add to it) and in shared memory (everyone reads it).  Per chunk, in fp32:
//   P_ij = cs l^|i-j| (a_i . b_j),  out = os (P c + diag(l^(i+1)) a X),  X <- l^n X + b^T diag(cs l^(n-1-j)) c
// (against time the powers count from the chunk's other end).  16 x 16 threads hold 2 x 2 outputs each and read operands 16 bytes
// at a time along the contraction.  Bound by a chunk's chain (loads, three products, 8 to 12 us) where CTAs are few, for which sequences are
// cut into segments (lin_simt_plan), else by reads of shared memory: 4 x 4096 tokens of 16 heads of 128 in fp32 2.2 ms, 7.8 TFLOP/s by the
// operator's 4 K V a token and head, 12.7 by what is done here (every 32 columns take a chunk's P again).
#include "gdn_mix.cuh"

namespace gdn {
namespace {

constexpr int kC = 32, kBV = 32, kThreads = 256, kMaxD = 256;
constexpr int kCS = kBV + 4;

template <typename T>
__device__ __forceinline__ void load_rows(float *dst, int stride, const T *src, int64_t ld, int rows, int cols, int width)
{
    // kC rows of `width` (a multiple of 4) columns, zeros behind `rows` and `cols`
    for (int i = threadIdx.x; i < kC * width; i += kThreads) {
        const int r = i / width, c = i - r * width;
        dst[r * stride + c] = r < rows && c < cols ? to_f<T>(src[(int64_t)r * ld + c]) : 0.f;
    }
}

struct Split {
    float *held;    // [passes][states][HV][da][dc]: what a segment adds to the state, then the state that enters it; null: one segment each
    int tokens;     // of a segment (a multiple of kC)
    int64_t slots, states;
    size_t pass;    // elements of a pass
    const int *chosen;  // several packed sequences: the segment that lin_choose_kernel took (`tokens` at least), and whether a sequence is longer
    __device__ int segment() const { return chosen ? *chosen : tokens; }
    __device__ bool none() const { return chosen && !chosen[1]; }  // no sequence is cut
};

// W: a, b columns at most.  STATE: only what a segment adds to the state, from zero.
template <typename T, int W, bool STATE>
__global__ void __launch_bounds__(kThreads) lin_simt_kernel(const LinArgs args, const Split split)
{
    extern __shared__ float4 lin_smem[];
    const LinPass &p = args.pass[blockIdx.y];
    const int nct = (p.dc + kBV - 1) / kBV;
    if (blockIdx.x >= (STATE ? split.states : split.slots) * args.HV * nct || (STATE && split.none())) return;
    const int ct = (int)(blockIdx.x % nct), hv = (int)(blockIdx.x / nct % args.HV);
    const int64_t slot = blockIdx.x / ((int64_t)nct * args.HV);
    const int tokens = split.segment();
    const Tile tl = !split.held ? Tile{(int)slot, 0} : STATE ? cut_of(args.cu, args.N, args.T, tokens, slot) : tile_of(args.cu, args.N, args.T, tokens, slot);
    const int n = tl.n;
    const SeqRange s = seq_range(args.cu, n, args.T);
    // the segment, in the order of processing
    const int chunks = (s.len + kC - 1) / kC, per = split.held ? tokens / kC : chunks;
    const int m0 = (int)min((int64_t)tl.index * per, (int64_t)chunks), m1 = (int)min((int64_t)m0 + per, (int64_t)chunks);
    const bool last = m1 == chunks, cut = chunks > per;
    if (STATE ? !cut || last : tl.index > 0 && m0 >= m1) return;
    const int da = p.da, w = (da + 3) & ~3, st = w + 4, c0 = ct * kBV, cols = min(kBV, p.dc - c0);
    float *A = (float *)lin_smem, *B = A + kC * st, *C = B + kC * st, *P = C + kC * kCS, *X = P + kC * kCS;  // X [w][kCS]
    __shared__ float pw[kC + 1];  // l^i
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int xq = tid & 7, xr = tid >> 3;  // the state's owner: columns 4 xq .., rows xr + 32 i
    const float g = args.decay ? args.decay[hv] : 0.f;
    if (tid <= kC) pw[tid] = decay_pow(g * kRcpLn2, tid);
    const int64_t xbase = ((int64_t)n * args.HV + hv) * da * p.dc;
    auto xat = [&](int r, int c) { return xbase + (p.x_t ? (int64_t)(c0 + c) * da + r : (int64_t)r * p.dc + c0 + c); };
    const int64_t at = cut ? cut_state0(args.cu, n, args.T, tokens) + tl.index : 0;
    float *const mine = cut ? split.held + blockIdx.y * split.pass + (at * args.HV + hv) * da * p.dc + c0 : nullptr;

    float x[W / 32][4];
#pragma unroll
    for (int i = 0; i < W / 32; ++i) {
        const int r = xr + 32 * i;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[i][k] = STATE || r >= da || 4 * xq + k >= cols ? 0.f : mine ? mine[(int64_t)r * p.dc + 4 * xq + k] : p.x0 ? p.x0[xat(r, 4 * xq + k)] : 0.f;
            if (r < w) X[r * kCS + 4 * xq + k] = x[i][k];
        }
    }
    const bool out = !STATE && p.out;
    for (int m = m0; m < m1; ++m) {
        const int c = p.reverse ? chunks - 1 - m : m;
        const int64_t t0 = s.bos + (int64_t)c * kC;
        const int rows = min(kC, s.len - c * kC);
        const int late = p.reverse && m == 0;  // X0 enters one step later
        __syncthreads();
        if (!STATE) load_rows<T>(A, st, (const T *)p.a + t0 * p.lda + (int64_t)(hv / p.ra) * da, p.lda, rows, da, w);
        load_rows<T>(B, st, (const T *)p.b + t0 * p.ldb + (int64_t)(hv / p.rb) * da, p.ldb, rows, da, w);
        load_rows<T>(C, kCS, (const T *)p.c + t0 * p.ldc + (int64_t)(hv / p.rc) * p.dc + c0, p.ldc, rows, cols, kBV);
        __syncthreads();
        float o[2][2] = {};
        if (out) {
            float z[2][2] = {};
            for (int k = 0; k < w; k += 4) {
                float4 u[2], v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    u[i] = *(const float4 *)&A[(ty + 16 * i) * st + k];
                    v[i] = *(const float4 *)&B[(tx + 16 * i) * st + k];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        z[i][j] += u[i].x * v[j].x + u[i].y * v[j].y + u[i].z * v[j].z + u[i].w * v[j].w;
                        o[i][j] += u[i].x * X[k * kCS + tx + 16 * j] + u[i].y * X[(k + 1) * kCS + tx + 16 * j] +
                                   u[i].z * X[(k + 2) * kCS + tx + 16 * j] + u[i].w * X[(k + 3) * kCS + tx + 16 * j];
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = ty + 16 * i, q = tx + 16 * j, gap = p.reverse ? q - r : r - q;
                    P[r * kCS + q] = gap >= 0 ? z[i][j] * (p.cs * pw[gap]) : 0.f;
                    o[i][j] *= pw[p.reverse ? max(rows - r - late, 0) : r + 1];
                }
        }
        if (!STATE) __syncthreads();
        if (out) {
#pragma unroll 4
            for (int j = 0; j < kC; ++j) {
                const float u0 = P[ty * kCS + j], u1 = P[(ty + 16) * kCS + j], v0 = C[j * kCS + tx], v1 = C[j * kCS + tx + 16];
                o[0][0] += u0 * v0;
                o[0][1] += u0 * v1;
                o[1][0] += u1 * v0;
                o[1][1] += u1 * v1;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = ty + 16 * i, q = tx + 16 * j;
                    if (r < rows && q < cols) {
                        const int64_t at = ((t0 + r) * args.HV + hv) * p.dc + c0 + q;
                        if (p.out_f32) ((float *)p.out)[at] = p.os * o[i][j];
                        else ((T *)p.out)[at] = from_f<T>(p.os * o[i][j]);
                    }
                }
        }
        const Decayed down(g, rows - late);
#pragma unroll
        for (int i = 0; i < W / 32; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][k] = down(x[i][k]);
        for (int j = 0; j < rows; ++j) {
            const float f = p.cs * pw[p.reverse ? j : rows - 1 - j];
            const float4 v = *(const float4 *)&C[j * kCS + 4 * xq];
#pragma unroll
            for (int i = 0; i < W / 32; ++i) {
                const int r = xr + 32 * i;
                if (r < w) {
                    const float b = f * B[j * st + r];
                    x[i][0] += b * v.x;
                    x[i][1] += b * v.y;
                    x[i][2] += b * v.z;
                    x[i][3] += b * v.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < W / 32; ++i) {
            const int r = xr + 32 * i;
            if (!STATE && r < w) *(float4 *)&X[r * kCS + 4 * xq] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        }
    }
    if (STATE) {
#pragma unroll
        for (int i = 0; i < W / 32; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = xr + 32 * i;
                if (r < da && 4 * xq + k < cols) mine[(int64_t)r * p.dc + 4 * xq + k] = x[i][k];
            }
    } else if (p.x1 && last) {
        const Decayed down(g, p.reverse && chunks > 0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < W / 32; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = xr + 32 * i;
                if (r < da && 4 * xq + k < cols) p.x1[xat(r, 4 * xq + k)] = down(x[i][k]);
            }
    }
}

// What the segments add to the state -> the state that enters each (in place), an element to a thread
__global__ void __launch_bounds__(kThreads) lin_join_kernel(const LinArgs args, const Split split)
{
    if (split.none()) return;
    const LinPass &p = args.pass[blockIdx.y];
    const int size = p.da * p.dc, tokens = split.segment();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, which = i / size, place = which / args.HV;
    if (place >= long_places(args.cu != nullptr, args.N, args.T, tokens)) return;
    const int at = (int)(i - which * size), hv = (int)(which - place * args.HV);
    auto first_at = [&](int n) { return long_place(args.cu, n, args.T, tokens); };
    const int n = args.cu ? last_from(args.N, place, first_at) : (int)place;
    const SeqRange s = seq_range(args.cu, n, args.T);
    const int segs = (s.len + tokens - 1) / tokens;
    if (segs <= 1 || first_at(n) != place) return;  // (whole)
    const int64_t slot0 = cut_state0(args.cu, n, args.T, tokens), pair = (int64_t)n * args.HV + hv;
    const float g = args.decay ? args.decay[hv] : 0.f;
    // tokens of a segment in the order of processing: against time the first has the sequence's odd end, and X0 enters one step later
    const int odd = (s.len + kC - 1) / kC * kC - s.len;
    const Decayed first(g, tokens - (p.reverse ? odd + 1 : 0)), rest(g, tokens);
    float x = p.x0 ? p.x0[pair * size + (p.x_t ? at % p.dc * p.da + at / p.dc : at)] : 0.f;
    float *buf = split.held + blockIdx.y * split.pass + (slot0 * args.HV + hv) * size + at;
    for (int k = 0; k < segs; ++k) {
        float *const here = buf + k * (int64_t)args.HV * size;
        const float add = k + 1 < segs ? *here : 0.f;
        *here = x;
        x = (k == 0 ? first(x) : rest(x)) + add;
    }
}

// The segment of several packed sequences, from their lengths: lin_simt_plan's rule with the longest one's chunks, and as many sequences as that
// makes of all chunks, in the place of one sequence of all tokens
__global__ void __launch_bounds__(kThreads) lin_choose_kernel(const LinArgs args, int tokens, int64_t ctas, int64_t room, int *chosen)
{
    __shared__ long long all[kThreads / 32];
    __shared__ int most[kThreads / 32];
    long long sum = 0;
    int longest = 0;
    for (int n = threadIdx.x; n < args.N; n += kThreads) {
        const int chunks = (seq_range(args.cu, n, args.T).len + kC - 1) / kC;
        sum += chunks;
        longest = max(longest, chunks);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    }
    if ((threadIdx.x & 31) == 0) all[threadIdx.x >> 5] = sum, most[threadIdx.x >> 5] = longest;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) {
            sum += all[w];
            longest = max(longest, most[w]);
        }
        const int64_t segs = min(room * longest / max(ctas * (int64_t)sum, (int64_t)1), (int64_t)longest / 4);
        // (not shorter than the plan's, whose grid and states it goes by)
        const int each = max(segs < 3 ? longest : (int)((longest + segs - 1) / segs), tokens / kC);
        chosen[0] = each * kC;
        chosen[1] = longest > each;
    }
}

// dq and dk (blockIdx.y) of shared heads, W elements to a thread
template <typename T, int W>
__global__ void lin_heads_kernel(const float *part, const int64_t *cu, int N, int64_t tokens, int H, int r, int D, T *dq, T *dk)
{
    // (rows outside every sequence have no parts)
    const int64_t per = (int64_t)H * D, lo = cu ? clamp64(cu[0], 0, tokens) * per : 0, hi = cu ? clamp64(cu[N], 0, tokens) * per : tokens * per;
    T *const out = blockIdx.y ? dk : dq;
    part += blockIdx.y * tokens * per * r;
    for (int64_t i = lo + W * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x); i < hi; i += W * (int64_t)gridDim.x * blockDim.x) {
        const int64_t head = i / D;
        const float *p = part + (head * r) * D + (i - head * D);
        float s[W];
#pragma unroll
        for (int e = 0; e < W; ++e) s[e] = 0.f;
        for (int k = 0; k < r; ++k) {
            float x[W];
            if constexpr (W == 4) *(float4 *)x = *(const float4 *)(p + (int64_t)k * D);
            else x[0] = p[(int64_t)k * D];
#pragma unroll
            for (int e = 0; e < W; ++e) s[e] += x[e];
        }
        if constexpr (W == 4 && sizeof(T) == 2) {
            __nv_bfloat162 y[2] = {__floats2bfloat162_rn(s[0], s[1]), __floats2bfloat162_rn(s[2], s[3])};
            *(uint2 *)(out + i) = *(const uint2 *)y;
        } else if constexpr (W == 4) {
            *(float4 *)(out + i) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            out[i] = from_f<T>(s[0]);
        }
    }
}

template <typename T>
cudaError_t heads(const float *part, const LinArgs &a, int64_t tokens, int H, int r, int D, void *dq, void *dk, cudaStream_t st)
{
    const int64_t n = tokens * H * D;
    if (n == 0) return cudaSuccess;
    const bool four = D % 4 == 0 && !(((uintptr_t)dq | (uintptr_t)dk) & 15);
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 1023) / 1024, 152 * 8);
    auto kern = four ? lin_heads_kernel<T, 4> : lin_heads_kernel<T, 1>;
    kern<<<dim3(blocks, 2), 256, 0, st>>>(part, a.cu, a.N, tokens, H, r, D, (T *)dq, (T *)dk);
    return cudaGetLastError();
}

// CTAs that walk a sequence, or a segment of one
int64_t ctas_of(const LinArgs &a)
{
    int64_t ctas = 0;
    for (int i = 0; i < a.passes; ++i) ctas += (int64_t)a.HV * ((a.pass[i].dc + kBV - 1) / kBV);
    return ctas;
}
// the segments that each of n sequences of `chunks` chunks is cut into (lin_simt_plan); fewer than three: none
int64_t segments(const LinArgs &a, int64_t n, int64_t chunks) { return std::min<int64_t>(4 * device_sm_count() / std::max<int64_t>(n * ctas_of(a), 1), chunks / 4); }
// whether several packed sequences' segment is chosen on the device: where as many of one length would not be cut
bool chooses(const LinArgs &a) { return a.cu && a.N > 1 && segments(a, a.N, (a.T + kC - 1) / kC / a.N) < 3; }

}  // namespace

LinPlan lin_simt_plan(const LinArgs &a)
{
    // A split walks twice (the second time with outputs), so only as many segments as bring four CTAs to an SM, of four chunks at least, and
    // none where that is two.  The lengths of packed sequences are not known here: the segment is what one sequence of all tokens is cut into,
    // shorter ones stay whole.  Where as many sequences of one length would not be cut, lin_choose_kernel takes a longer segment, or none (8 x 8192
    // tokens of 8 heads of 128, packed: 6007 us by the plan's segment, 4365; the call costs 6).  fp32, whole and cut: 2048 tokens of 8 heads of 64
    // 608 us and 100, gradients 553 and 182; 4 x 2048 of 8 heads of 128 (four segments) 907 and 735; 4 x 4096 of 16 heads of 128 (two) 2181 and
    // 2835; 300 tokens of 4 heads of 32, gradients (two) 64 and 70.
    int64_t size = 0;
    for (int i = 0; i < a.passes; ++i) size = std::max(size, (int64_t)a.pass[i].da * a.pass[i].dc);
    const int64_t each = (a.T + kC - 1) / kC, segs = segments(a, a.cu ? 1 : a.N, each);
    LinPlan p{};
    p.slots = a.N;
    if (segs < 3) return p;
    p.tokens = (int)((each + segs - 1) / segs) * kC;
    p.slots = mix_slots(a.cu != nullptr, a.N, a.T, p.tokens);
    p.states = cut_states(a.cu != nullptr, a.N, a.T, p.tokens);
    p.places = long_places(a.cu != nullptr, a.N, a.T, p.tokens);
    p.bytes = (size_t)a.passes * p.states * a.HV * size * sizeof(float);
    p.bytes = ((p.bytes + 255) & ~(size_t)255) + (chooses(a) ? kChosenBytes : 0);
    return p;
}

namespace {

template <typename T, int W>
cudaError_t launch(const LinArgs &a, void *ws, cudaStream_t st)
{
    const LinPlan plan = lin_simt_plan(a);
    int64_t most = 0, summed = 0, joined = 0;
    size_t smem = 0;
    Split split{};
    split.held = plan.bytes ? (float *)ws : nullptr;
    split.tokens = plan.tokens;
    split.slots = plan.slots;
    split.states = plan.states;
    size_t held = plan.bytes;
    if (plan.bytes && chooses(a)) {
        held -= kChosenBytes;
        split.chosen = (const int *)((const char *)ws + held);
    }
    split.pass = held / sizeof(float) / a.passes;
    for (int i = 0; i < a.passes; ++i) {
        const LinPass &p = a.pass[i];
        most = std::max(most, plan.slots * a.HV * ((p.dc + kBV - 1) / kBV));
        summed = std::max(summed, plan.states * a.HV * ((p.dc + kBV - 1) / kBV));
        joined = std::max(joined, (plan.places * a.HV * p.da * p.dc + kThreads - 1) / kThreads);
        const size_t w = (p.da + 3) & ~3;
        smem = std::max(smem, 4 * (2 * kC * (w + 4) + 2 * kC * kCS + w * kCS));
    }
    if (most > INT32_MAX || summed > INT32_MAX || joined > INT32_MAX) return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> seen;
    if (first_on_device(seen)) {
        const int bytes = 4 * (2 * kC * (W + 4) + 2 * kC * kCS + W * kCS);
        cudaError_t e = cudaFuncSetAttribute(lin_simt_kernel<T, W, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(lin_simt_kernel<T, W, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        done_on_device(seen);
    }
    if (split.chosen) lin_choose_kernel<<<1, kThreads, 0, st>>>(a, plan.tokens, ctas_of(a), 4 * device_sm_count(), const_cast<int *>(split.chosen));
    if (split.held) {
        lin_simt_kernel<T, W, true><<<dim3((unsigned)summed, a.passes), kThreads, smem, st>>>(a, split);
        lin_join_kernel<<<dim3((unsigned)joined, a.passes), kThreads, 0, st>>>(a, split);
    }
    lin_simt_kernel<T, W, false><<<dim3((unsigned)most, a.passes), kThreads, smem, st>>>(a, split);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_of(const LinArgs &a, void *ws, cudaStream_t st)
{
    int da = 0;
    for (int i = 0; i < a.passes; ++i) da = std::max(da, a.pass[i].da);
    return da <= 64 ? launch<T, 64>(a, ws, st) : da <= 128 ? launch<T, 128>(a, ws, st) : launch<T, kMaxD>(a, ws, st);
}

}  // namespace

cudaError_t launch_lin_simt(const LinArgs &a, gdn_dtype dt, void *ws, cudaStream_t st)
{
    return dt == GDN_F32 ? launch_of<float>(a, ws, st) : launch_of<__nv_bfloat16>(a, ws, st);
}

cudaError_t launch_lin_heads(const float *part, const LinArgs &a, int64_t tokens, int H, int r, int D, void *dq, void *dk, gdn_dtype dt, cudaStream_t st)
{
    return dt == GDN_F32 ? heads<float>(part, a, tokens, H, r, D, dq, dk, st) : heads<__nv_bfloat16>(part, a, tokens, H, r, D, dq, dk, st);
}

}  // namespace gdn
