/*
 * gdn.h -- C ABI of the GB300 gated delta-rule chunked-prefill forward.
 *
 * The operation (per sequence n, value head h; key/query head h / (HV/H)):
 *
 *   S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *   o_t = scale * S_t^T q_t,        S_0 = h0[n,h] (or 0),  ht[n,h] = S_T
 *
 * with alpha_t = exp(g_t) for a scalar gate (FlashQLA blog, "Further
 * optimisation via gate decay", the recurrence; "Key problems in FLA's GDN
 * chunked prefill", the chunk form) or alpha_t,d = exp(gk_t,d) for a
 * per-key-channel gate ("KDA source walkthrough", chunk_kda_fwd and the gk
 * branch of chunk_gated_delta_rule_fwd_h).  It is evaluated chunkwise
 * (chunk size C = 64): gate cumsum, gated strictly-lower K K^T, its
 * unit-lower-triangular inverse, the WY form, the serial inter-chunk state
 * scan and the output, optionally split over sequence segments on one GPU
 * (FlashQLA blog, "A balanced solution": the S* / M correction, and "Further
 * optimisation via gate decay": the gate-driven warmup).
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers (except in gdn_chunk_fwd_host),
 *    contiguous (row-major, last index fastest) and owned by the caller.
 *  - Shapes (FlashQLA blog, "Usage"; GDN-in-FLA notes, forward signature):
 *      q, k   [B, T, H,  K]    qkv_dtype
 *      v      [B, T, HV, V]    qkv_dtype
 *      o      [B, T, HV, V]    qkv_dtype (written)
 *      g      [B, T, HV]       fp32, natural-log gate (gate_kind SCALAR)
 *      gk     [B, T, HV, K]    fp32, natural-log gate (gate_kind CHANNEL)
 *      beta   [B, T, HV]       fp32
 *      h0     [N, HV, K, V]    fp32, nullable (= zero initial state)
 *      ht     [N, HV, K, V]    fp32, nullable (final state not written)
 *      cu_seqlens [N+1]        int64 token offsets, nullable.  When given the
 *                              input is packed: B must be 1, T is the total
 *                              token count and sequence n spans tokens
 *                              [cu[n], cu[n+1]) ("Flash Linear Attention"
 *                              page, sec. 2, varlen: FlashAttention semantics).
 *                              Without it N = B and each batch row is one
 *                              sequence of T tokens.
 *  - State layout is [K][V] row-major (FLA's default, not state_v_first).
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and the call returns without synchronising.  Argument errors
 *    are reported before anything is enqueued; errors found on the device
 *    (a bounded wait that ran out, a failed plan check) are recorded in the
 *    workspace status word, read with gdn_read_device_status().
 *  - Nothing aborts the process and no entry point calls exit().
 */
#ifndef GDN_GB300_H
#define GDN_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *gdn_stream_t; /* identical to cudaStream_t */

typedef enum {
    GDN_F32 = 0,
    GDN_BF16 = 1,
    GDN_E4M3 = 2 /* 8-bit floating point, 4 exponent and 3 mantissa bits (the decoder-block
                    operators only: gdn_rms_norm, gdn_linear, gdn_gated_linear)           */
} gdn_dtype;

typedef enum { GDN_GATE_SCALAR = 0, GDN_GATE_CHANNEL = 1 } gdn_gate_kind;

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID = -1,     /* null pointer, negative or inconsistent size       */
    GDN_ERR_UNSUPPORTED = -2, /* valid but not implemented (e.g. chunk_size != 64) */
    GDN_ERR_CUDA = -3,        /* a CUDA runtime call or launch failed              */
    GDN_ERR_TIMEOUT = -4,     /* a bounded device wait ran out (device status)     */
    GDN_ERR_NOMEM = -5,       /* library-managed workspace could not be allocated  */
    GDN_ERR_WORKSPACE = -6    /* caller workspace smaller than gdn_workspace_size  */
} gdn_status;

typedef struct {
    int B, T, H, HV, K, V;   /* varlen: B == 1 and T == total tokens               */
    gdn_dtype qkv_dtype;     /* q, k, v and o share it; g/beta/h0/ht are fp32      */
    gdn_gate_kind gate_kind; /* SCALAR: g [B,T,HV];  CHANNEL: gk [B,T,HV,K]        */
    int num_seqs;            /* N: B, or len(cu_seqlens) - 1 for packed input       */
} gdn_shape;

/* How a long sequence is split over the GPU (FlashQLA blog, in-GPU CP). */
typedef enum {
    GDN_CP_AUTO = 0,   /* planner decides (split only when (seq, head) pairs are few) */
    GDN_CP_OFF = 1,    /* one serial scan per (sequence, head)                        */
    GDN_CP_EXACT = 2,  /* segments start from S* = 0, M = I; serial S* / M combine
                          (per-channel gates: on the SIMT engine)                    */
    GDN_CP_WARMUP = 3  /* segments re-derive their start state from zero over a
                          warmup window sized from the gate statistics (per-channel
                          gates: each token's slowest channel bounds its decay; AUTO
                          picks it for them on the TC engine only when the (sequence,
                          head) pairs fill at most a quarter of the SMs)             */
} gdn_cp_mode;

typedef enum {
    GDN_ENGINE_AUTO = 0, /* tensor-core engine where supported, else SIMT            */
    GDN_ENGINE_SIMT = 1, /* fp32 CUDA-core engine (any supported shape, fp32 inputs) */
    GDN_ENGINE_TC = 2,   /* tcgen05/TMEM engine: bf16, K = V = 128, scalar or
                            per-channel gate, q/k/v/o (and gk) 16-byte aligned; a
                            call that asks for it on other inputs gets
                            GDN_ERR_INVALID                                       */
    GDN_ENGINE_RECURRENT = 3 /* token by token, no chunks ("Flash Linear Attention"
                            page, sec. 8, fused_recurrent, C = 1): for decode and
                            short continuations; any supported shape; no split.
                            AUTO selects it when no sequence is longer than 16
                            tokens (T, or max_seq_len for packed input).          */
} gdn_engine;

typedef struct {
    gdn_cp_mode cp_mode;
    int segment_chunks;    /* chunks per segment when split (0 = planner's choice)  */
    gdn_engine engine;
    int keys_unit_norm;    /* caller asserts ||k_t||_2 <= 1 and 0 <= beta_t <= 2, so
                              every transition has spectral norm <= its decay; lets
                              AUTO choose the warmup split (qk_l2norm together with
                              beta_logits implies it)                               */
    float warmup_log2_eps; /* warmup stops once the window's decay <= 2^this (0 = -24) */
    int max_seq_len;       /* packed input: bound on one sequence's length, used to
                              size the split grid (0 = T)                             */
    void *const *launch_events; /* optional, caller-owned CUDA events (cudaEvent_t):
                              event i is recorded on the stream right before the
                              call's i-th kernel launch and event `kernels` (see
                              gdn_plan) right after the last one, so consecutive
                              events time each kernel.  NULL: nothing recorded.   */
    int n_launch_events;   /* length of launch_events; extra marks are skipped      */
    int wait_limit_us;     /* wall-clock limit of every device-side wait of the
                              tensor-core kernels, in microseconds (0 = 2 s).  A
                              wait that runs out records GDN_ERR_TIMEOUT in the
                              device status and the kernel ends early.            */
    int test_withhold_first_arrival; /* testing the timeout path only: nonzero makes
                              the tensor-core scan's load warp withhold its "chunk
                              loaded" signal for the first chunk of every CTA, so
                              every role's wait runs out (bounded by
                              wait_limit_us), the device status reads
                              GDN_ERR_TIMEOUT and o / ht are left undefined.  No
                              effect on the SIMT engine.                          */
    /* Input activations done inside the kernels ("Flash Linear Attention" page,
     * sec. 10: the KDA inference backend takes raw tensors and fuses the gate,
     * the L2 norm and sigma(beta); "KDA source walkthrough",
     * kda_gate_chunk_cumsum, for the gate).  All zero: inputs used as given.   */
    const float *gate_A_log;   /* [HV], device; non-NULL: g_or_gk holds the raw
                              gate input x and the log-decay is
                              -exp(A_log[h]) * softplus(x + dt_bias), or with
                              gate_lower_bound < 0:
                              gate_lower_bound * sigmoid(exp(A_log[h]) (x + dt_bias)) */
    const float *gate_dt_bias; /* [HV] (scalar gate) or [HV][K] (per-channel), device,
                              nullable (zero)                                       */
    float gate_lower_bound;    /* < 0 selects the bounded form above; 0: softplus form */
    int beta_logits;           /* beta holds logits: the kernels use sigmoid(beta)     */
    int qk_l2norm;             /* q and k are scaled to unit L2 norm per (token, head)
                              inside the kernels: x / max(||x||_2, 1e-12)            */
    int state_v_first;         /* h0 and ht are [N, HV, V, K] instead of [N, HV, K, V]
                              (the transposed state layout; the library transposes
                              them around the call through its workspace)           */
} gdn_options;

/* Fill `opt` with the defaults (AUTO everywhere, no assertions).  No
 * counterpart in the pages (library infrastructure). */
void gdn_default_options(gdn_options *opt);

/* Human-readable name of a status code (static string, never NULL).  No
 * counterpart in the pages. */
const char *gdn_status_string(gdn_status st);

/* Library version: major * 10000 + minor * 100 + patch.  No counterpart in
 * the pages. */
int gdn_version(void);

/*
 * Bytes of device workspace gdn_chunk_fwd_ws needs for this problem and
 * options (at least 256: the first 256 bytes hold the device status word).
 * Returns 0 if the arguments are invalid or unsupported.  No counterpart in
 * the pages (the pages' kernels allocate their intermediates themselves).
 */
size_t gdn_workspace_size(const gdn_shape *s, int chunk_size, const gdn_options *opt);

/*
 * The forward pass of the problem statement (FlashQLA blog, "Usage":
 * chunk_gated_delta_rule(q, k, v, g, beta, scale, initial_state,
 * output_final_state, cu_seqlens) -> (o, final_state)) with a caller-provided
 * workspace (`workspace`, at least
 * gdn_workspace_size bytes, 256-byte aligned, device memory).  The
 * workspace must not be used by another call that can run concurrently.
 * Returns GDN_OK once all work is enqueued on `stream`.
 */
gdn_status gdn_chunk_fwd_ws(const gdn_shape *s,
                            const void *q, const void *k, const void *v,
                            const float *g_or_gk, const float *beta, float scale,
                            const float *h0, const int64_t *cu_seqlens, int chunk_size,
                            void *o, float *ht, const gdn_options *opt,
                            void *workspace, size_t ws_bytes, gdn_stream_t stream);

/*
 * The forward pass of the problem statement (FlashQLA blog, "Usage"; the
 * GDN-in-FLA notes, forward signature; "KDA source walkthrough",
 * chunk_kda_fwd for the per-channel gate) -- the plain entry point -- with
 * default options and a library-managed workspace,
 * cached per (device, stream) and grown stream-ordered (cudaMallocAsync on
 * `stream`) when a call needs more; while `stream` is being captured, by
 * memory beside the graph (cudaMalloc).  A workspace that a captured call
 * used is never freed: the graph may be replayed at any time that no other
 * call uses it.  Arguments as in gdn_chunk_fwd_ws.
 */
gdn_status gdn_chunk_fwd(const gdn_shape *s,
                         const void *q, const void *k, const void *v,
                         const float *g_or_gk, const float *beta, float scale,
                         const float *h0, const int64_t *cu_seqlens, int chunk_size,
                         void *o, float *ht, gdn_stream_t stream);

/* As gdn_chunk_fwd with explicit options (NULL = defaults): the split mode
 * and warmup threshold follow the FlashQLA blog, "A balanced solution" and
 * "Further optimisation via gate decay". */
gdn_status gdn_chunk_fwd_ex(const gdn_shape *s,
                            const void *q, const void *k, const void *v,
                            const float *g_or_gk, const float *beta, float scale,
                            const float *h0, const int64_t *cu_seqlens, int chunk_size,
                            void *o, float *ht, const gdn_options *opt, gdn_stream_t stream);

/*
 * The forward pass of the problem statement (FlashQLA blog, "Usage") as an
 * end-to-end call on HOST buffers (pageable or pinned): copies the inputs to
 * a library-owned device arena, runs gdn_chunk_fwd_ex, copies o (and ht when
 * non-NULL) back, and synchronises `stream` before returning.  The call is
 * cut into up to four groups of whole sequences (contiguous token ranges of
 * every tensor); group i runs on `stream` while group i+1's inputs are copied
 * in and group i-1's outputs copied out, each direction on a library-owned
 * stream of the current device.  `cu_seqlens` is a host array here too and is
 * checked on the host (cu[0] == 0, nondecreasing, cu[N] == T).  Same shapes
 * as above.
 */
gdn_status gdn_chunk_fwd_host(const gdn_shape *s,
                              const void *q, const void *k, const void *v,
                              const float *g_or_gk, const float *beta, float scale,
                              const float *h0, const int64_t *cu_seqlens, int chunk_size,
                              void *o, float *ht, const gdn_options *opt,
                              gdn_stream_t stream);

/*
 * No counterpart in the pages (the bounded device waits are this library's).
 * Synchronise `stream`, return the status the device recorded in the
 * workspace since the last read, and clear it.  `workspace` is the buffer
 * given to gdn_chunk_fwd_ws, or NULL for the library-managed workspace of
 * (current device, stream).
 */
gdn_status gdn_read_device_status(void *workspace, gdn_stream_t stream);

/*
 * The forward pass without any allocation (no counterpart in the paper; an
 * interface for callers that cannot allocate device memory when they run the
 * forward: code running inside a memory pool it does not own, runtimes that
 * forbid cudaMalloc on their hot path because it synchronises the device, or
 * embeddings that reserved all device memory up front).  Arguments as in
 * gdn_chunk_fwd_ex; the caller still provides every input and output.
 *
 * Scratch (the device status word and the chunk-parallel split's tables)
 * lives in one fixed 4 MiB device array owned by the library, which every
 * GPU that loads the library holds until the process exits.  A plan that
 * needs more scratch than that (gdn_workspace_size > 4 MiB, e.g. the exact
 * split over many segments) is rejected with GDN_ERR_WORKSPACE before
 * anything is enqueued; choose GDN_CP_OFF or GDN_CP_WARMUP, or use
 * gdn_chunk_fwd_ws with a larger workspace.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress with that device current); make that first call
 * before any stream capture.  Every call uses the same array, which keeps
 * the previous call's contents: calls that can overlap on the GPU -- on
 * different streams, or from different threads -- race on it and must be
 * serialised by the caller.  No cudaMalloc, cudaFree or other allocating
 * routine is called.  Argument errors return the same codes as
 * gdn_chunk_fwd_ex and enqueue nothing.  Errors found on the device (a wait
 * that ran out, a failed plan check, the warmup split's key-norm check) are
 * collected in the array's status word until gdn_read_noalloc_status reads
 * and clears it.
 */
gdn_status gdn_chunk_fwd_noalloc(const gdn_shape *s,
                                 const void *q, const void *k, const void *v,
                                 const float *g_or_gk, const float *beta, float scale,
                                 const float *h0, const int64_t *cu_seqlens, int chunk_size,
                                 void *o, float *ht, const gdn_options *opt, gdn_stream_t stream);

/*
 * The device status of gdn_chunk_fwd_noalloc calls on the current device (no
 * counterpart in the paper): synchronises `stream`, returns the status word of
 * the fixed array as gdn_read_device_status does for a workspace (GDN_OK,
 * GDN_ERR_TIMEOUT or GDN_ERR_INVALID) and clears it.  Allocates nothing.
 */
gdn_status gdn_read_noalloc_status(gdn_stream_t stream);

/*
 * Decode / continuation of the problem statement ("Flash Linear Attention"
 * page, sec. 8: fused_recurrent, the C = 1 form the layer selects for short
 * queries): the same operation and arguments as gdn_chunk_fwd (no chunk
 * size), evaluated token by token on the recurrent engine.  `ht` may be the
 * same buffer as `h0`: the state cache is then updated in place.  Suited to
 * a few tokens per sequence (decode steps continuing from a prefill's final
 * state); longer sequences are faster on gdn_chunk_fwd.
 */
gdn_status gdn_recurrent_fwd(const gdn_shape *s,
                             const void *q, const void *k, const void *v,
                             const float *g_or_gk, const float *beta, float scale,
                             const float *h0, const int64_t *cu_seqlens,
                             void *o, float *ht, gdn_stream_t stream);

/*
 * Backward pass of the chunked forward (GDN-in-FLA notes, backward: the gradients
 * dq, dk, dv, db, dg, dh0 of chunk_gated_delta_rule_bwd, Steps 1-7; "Flash Linear
 * Attention" page, sec. 7: the state gradient scanned in reverse time, the chunk
 * states recomputed).  Given the same inputs as gdn_chunk_fwd (scalar gate) and
 * `dout` [B,T,HV,V] (the dtype of v), the gradient of the loss with respect to o,
 * and `dht` [N,HV,K,V] fp32 (nullable: zero), the gradient with respect to the
 * final state, writes fp32
 *     dq, dk [B,T,H,K]   (with HV > H: summed over the value heads of each head)
 *     dv     [B,T,HV,V]
 *     dbeta  [B,T,HV]
 *     dg     [B,T,HV]    (natural-log gate, as g)
 *     dh0    [N,HV,K,V]  (nullable: not written)
 * The caller owns every buffer; the library-managed workspace of `stream` holds
 * the recomputed states (4 K V bytes per chunk and value head) and a gate buffer.
 * q, k, v, dout, dq and dk must be 16-byte aligned (rows are read by 16-byte loads,
 * four columns of dq and dk added by one 16-byte atomic).
 * Errors: GDN_ERR_INVALID (arguments, a null required pointer, a misaligned one),
 * GDN_ERR_UNSUPPORTED (per-channel gates, chunk_size != 64, K not 32/64/128),
 * GDN_ERR_NOMEM, GDN_ERR_CUDA; nothing is enqueued on an argument error.
 * Asynchronous on `stream`.
 */
gdn_status gdn_chunk_bwd(const gdn_shape *s,
                         const void *q, const void *k, const void *v,
                         const float *g, const float *beta, float scale,
                         const float *h0, const void *dout, const float *dht,
                         const int64_t *cu_seqlens, int chunk_size,
                         float *dq, float *dk, float *dv, float *dbeta, float *dg,
                         float *dh0, gdn_stream_t stream);

/*
 * Context parallel across devices, step 1 (FlashQLA blog, "Key problems in
 * FLA's GDN chunked prefill": the S* / M pre-process; "KDA source
 * walkthrough", the cp_context pre-process of chunk_kda_fwd): the summary of
 * every sequence of this (local) input as one piece of a longer sequence.
 * For sequence n and value head h, with S_end the state after the piece from
 * a start state S_0:  S_end = S*[n,h] + M[n,h] S_0.  Written as
 * summary[N, HV, K, V + K] fp32: row d holds S*[d, 0..V-1] then M[d, 0..K-1].
 * q is not needed.  Arguments otherwise as gdn_chunk_fwd_ex (no h0, no
 * outputs); the split options are ignored (one piece per sequence).
 */
gdn_status gdn_chunk_summary(const gdn_shape *s,
                             const void *k, const void *v,
                             const float *g_or_gk, const float *beta,
                             const int64_t *cu_seqlens, int chunk_size,
                             float *summary, const gdn_options *opt, gdn_stream_t stream);

/*
 * Context parallel, step 2 (same passages): the start state of every piece
 * from the summaries of the pieces before it.  summaries [ranks][pairs][K][V+K]
 * (as gdn_chunk_summary writes them, piece r of each of `pairs` (sequence,
 * head) pairs, gathered in piece order), h0 [pairs][K][V] (nullable: zero),
 * starts [ranks][pairs][K][V]:  starts[0] = h0,
 * starts[r+1] = S*_r + M_r starts[r].  K in {32, 64, 128}; pairs <= 65535.
 * Device pointers; asynchronous on `stream`.
 */
gdn_status gdn_chain_states(int ranks, int pairs, int K, int V, const float *summaries,
                            const float *h0, float *starts, gdn_stream_t stream);

/* ------------------------------------------------------------------------
 * The operators that stand around the gated delta rule in a decoder block:
 * the norm before it, the projections into and out of it, the feed-forward
 * block after it.  (No counterpart in the pages; their conventions are those
 * above: device pointers, work enqueued on `stream`, argument errors before
 * anything is enqueued.)
 *
 *  - Matrices are row-major with consecutive elements in a row; inputs take a
 *    row stride in elements (at least the row's length), outputs are
 *    contiguous unless they have a stride.  Any length, any alignment to the
 *    element: matrices whose rows do not start on 16-byte boundaries pass by
 *    padded copies in the workspace, and fp32 operands of more than 64 rows
 *    by their bf16 planes (six bytes an element).
 *  - Outputs lie over no input and no other output, unless said at the field
 *    (gdn_linear and gdn_gated_linear refuse a y that does, GDN_ERR_INVALID).
 *  - `workspace`: device memory of at least the size that the operator's
 *    _workspace_size call gives for the same arguments, 256-byte aligned, not
 *    used by another call that can run concurrently.  NULL: the
 *    library-managed workspace of (device, stream), which is not allowed to
 *    grow while the stream is being captured (GDN_ERR_NOMEM then).  A buffer
 *    that a captured call used is never freed, also where the workspace grows
 *    later; replays of the graph use it, so that they must not run
 *    concurrently with other calls on the library-managed workspace of the
 *    captured stream, nor with other graphs captured there (a workspace of
 *    the graph's own avoids that).  A size of 0 needs none.
 *  - A device-side wait that ran out (2 s) is recorded per device; the next
 *    gdn_read_layer_status reads and clears it.
 *  - Zero rows are allowed: outputs without rows are left alone, the
 *    gradients of weights and biases are then zero.
 */
typedef struct {
    int64_t rows;         /* M */
    int width;            /* D >= 1 */
    gdn_dtype dtype;      /* x, residual, h, dy, dh, dx: GDN_F32 or GDN_BF16           */
    gdn_dtype w_dtype;    /* weight: GDN_F32 or GDN_BF16                               */
    gdn_dtype out_dtype;  /* y: `dtype`, or GDN_E4M3 with one scale per row            */
    float eps;            /* >= 0 */
    const void *x;        /* [M][D], row stride ldx (backward: h)                      */
    int64_t ldx;
    const void *residual; /* [M][D], row stride ld_residual; nullable                  */
    int64_t ld_residual;
    const void *weight;   /* [D]; nullable (all one)                                   */
    void *y;              /* [M][D]                                                    */
    float *scale;         /* [M], out_dtype GDN_E4M3: y stands for scale[m] * y[m][d]  */
    void *h;              /* [M][D], x + residual rounded to dtype; may be residual or
                             x itself (same rows); nullable                            */
    const void *dy;       /* backward: [M][D], row stride ld_dy                        */
    int64_t ld_dy;
    const void *dh;       /* backward: the gradient that reaches h past the norm,
                             [M][D], row stride ld_dh; nullable (zero)                 */
    int64_t ld_dh;
    void *dx;             /* backward: [M][D], may be dy or dh itself (same rows)      */
    float *dweight;       /* backward: [D]; nullable                                   */
} gdn_norm_args;

/*
 * Root-mean-square norm of rows with the residual's addition in front:
 *     h = x + residual,  n = sqrt(mean(h^2) + eps),  y = weight h / n
 * in fp32 from the unrounded h, rounded once.  With out_dtype GDN_E4M3:
 *     scale = max(max|y| / 448, 2^-126),  y = e4m3(y / scale), saturating
 * (a row that holds a NaN or an infinity gets a NaN scale).
 */
gdn_status gdn_rms_norm(const gdn_norm_args *a, gdn_stream_t stream);

/* One scale per row and e4m3 values of x as it stands: gdn_rms_norm without
 * the norm, residual and weight (x, y, scale of `a`; NaN scales as there). */
gdn_status gdn_quantize_rows(const gdn_norm_args *a, gdn_stream_t stream);

/*
 * Gradients of gdn_rms_norm (bf16 / fp32 output) from h = x + residual:
 *     dx = dh + (weight dy - h mean(weight dy h) / n^2) / n
 * (the gradient of x and of residual), dweight = sum over rows of dy h / n,
 * summed in a fixed order.
 */
size_t gdn_rms_norm_bwd_workspace_size(const gdn_norm_args *a);
gdn_status gdn_rms_norm_bwd(const gdn_norm_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

typedef enum {
    GDN_ACT_NONE = 0,
    GDN_ACT_SILU = 1,      /* z / (1 + exp(-z))                                        */
    GDN_ACT_GELU = 2,      /* z (1 + erf(z / sqrt 2)) / 2                              */
    GDN_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2        */
    GDN_ACT_RELU = 4,
    GDN_ACT_SIGMOID = 5
} gdn_activation;

typedef struct {
    int64_t rows;         /* M, at most 2^31 - 256                                     */
    int out_features;     /* N (gated linear unit: F, the width of one half)           */
    int in_features;      /* K >= 1 */
    gdn_dtype dtype;      /* x and w: GDN_F32, GDN_BF16 or (forward only) GDN_E4M3     */
    gdn_dtype out_dtype;  /* y and residual: GDN_F32 or GDN_BF16 (fp32 inputs: GDN_F32;
                             gated and backward: `dtype`, GDN_BF16 for GDN_E4M3)       */
    gdn_activation act;
    const void *x;        /* [M][K], row stride ldx                                    */
    int64_t ldx;
    const void *w;        /* [N][K] (gated: [2F][K], the gate's rows first), stride ldw */
    int64_t ldw;
    const float *x_scale; /* [M] and [N] (gated: [2F]): the scales of GDN_E4M3 inputs  */
    const float *w_scale; /*   (both or none; none: 1)                                 */
    const float *bias;    /* [N], nullable (gated: none)                               */
    const void *residual; /* [M][N], row stride ld_residual; nullable                  */
    int64_t ld_residual;
    void *y;              /* [M][N] (gated: [M][F]), row stride ldy; may be residual
                             itself.  Gated backward: the recomputed output, nullable  */
    int64_t ldy;
    const void *dy;       /* backward: [M][N] (gated: [M][F]), row stride ld_dy        */
    int64_t ld_dy;
    void *dx;             /* backward: [M][K], nullable                                */
    void *dw;             /* backward: as w, contiguous, nullable                      */
    float *dbias;         /* backward: [N], nullable                                   */
} gdn_linear_args;

/*
 * Linear layer with its epilogue:
 *     y = act(x_scale_m w_scale_n (x w^T) + bias) + residual
 * Products are summed in fp32 and the epilogue runs on those sums; y is
 * rounded once.  bf16 and e4m3 inputs run on the tensor cores.  fp32 inputs
 * run on the CUDA cores up to 64 rows and on the tensor cores above, every
 * value as the sum of three bf16 values (the last bits of fp32 included);
 * infinities and NaN come through as a plain fp32 sum has them.
 */
size_t gdn_linear_workspace_size(const gdn_linear_args *a);
gdn_status gdn_linear(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

/*
 * Gradients of gdn_linear (F32 or BF16; the residual's is dy): with
 * z = x w^T + bias recomputed where there is an activation,
 *     dz = dy act'(z),  dx = dz w,  dw = dz^T x,  dbias = sum over rows of dz
 * dz is rounded to `dtype` between the products (an operand of the tensor
 * cores); dbias is summed from the unrounded values, in a fixed order.
 */
size_t gdn_linear_bwd_workspace_size(const gdn_linear_args *a);
gdn_status gdn_linear_bwd(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

/*
 * Gated linear unit, both projections and their product in one kernel:
 *     y = act(x w_gate^T) * (x w_up^T),   w = [w_gate; w_up]
 */
size_t gdn_gated_linear_workspace_size(const gdn_linear_args *a);
gdn_status gdn_gated_linear(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

/*
 * Gradients of gdn_gated_linear (F32 or BF16) from x, w and dy alone: the
 * projections are recomputed (nothing of the forward is kept), with
 *     dgate = dy up act'(gate),  dup = dy act(gate)
 * rounded to `dtype` between the products, dx = dgate w_gate + dup w_up and
 * dw = [dgate dup]^T x.  `y`, when given, receives the recomputed output.
 */
size_t gdn_gated_linear_bwd_workspace_size(const gdn_linear_args *a);
gdn_status gdn_gated_linear_bwd(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

/* Synchronise `stream`, return what device-side waits of the operators above
 * recorded on the current device since the last read (GDN_OK or
 * GDN_ERR_TIMEOUT) and clear it. */
gdn_status gdn_read_layer_status(gdn_stream_t stream);

/* Testing the timeout path only: while `on` is not 0, gdn_linear calls of the
 * calling thread launch instances of its kernels that load no operands, so
 * that the waits for them run out after 5 ms, gdn_read_layer_status reports
 * GDN_ERR_TIMEOUT and the outputs are undefined.  There are such instances
 * for bf16 to bf16 and fp32 products in tiles of 128 columns and for bf16
 * ones of up to 16 rows; other products run as ever.  The token mixers'
 * tensor-core kernels below load nothing either. */
void gdn_layer_test_withhold(int on);

/* ------------------------------------------------------------------------
 * Token mixers beside the gated delta rule: linear attention with a decay for
 * each head, and softmax attention with a sliding window and a few first
 * tokens that stay visible (sinks); their forms for single tokens and their
 * gradients.  (No counterpart in the pages.)
 *
 *  - Layouts are the delta rule's: [B][T][heads][size], heads that share a
 *    key head are neighbours (value head h reads key head h / (HV / H), query
 *    head h key head h / (H / HK)), packed input by cu_seqlens (B = 1, T all
 *    tokens).  Inputs take the distance from a token to the next in elements
 *    (a slice of a fused projection): heads and elements of a token are
 *    consecutive, the batch is T tokens apart.  Outputs are contiguous and
 *    lie over no input, unless said at the field.
 *  - Any alignment to the element.  bf16 heads of 64 or 128 (linear attention:
 *    K = V) on 16-byte boundaries run on the tensor cores, everything else on
 *    the CUDA cores.  Head sizes up to 256.
 *  - Offsets in cu_seqlens are clamped to the tensor; tokens outside every
 *    sequence are neither read nor written.
 *  - Workspaces as for the decoder-block operators above (and
 *    gdn_read_layer_status for device-side waits that ran out).
 *  - Inputs are finite: a NaN or an infinity reaches, besides the outputs that
 *    depend on it, others of the same sequence and tile of tokens (a product
 *    with a weight of zero is NaN); it reaches no other sequence.
 */
typedef struct {
    int B, T, H, HV, K, V;  /* packed: B = 1, T all tokens; K, V <= 256                  */
    int num_seqs;           /* N: B, or len(cu_seqlens) - 1                              */
    gdn_dtype dtype;        /* q, k, v, o, dout, dq, dk, dv: GDN_F32 or GDN_BF16         */
    float scale;
    const void *q, *k, *v;  /* [B][T][H][K], [B][T][H][K], [B][T][HV][V]                 */
    int64_t ldq, ldk, ldv;  /* elements from a token to the next                         */
    const float *decay;     /* [HV], natural logarithm (<= 0); nullable (no decay)       */
    const float *h0;        /* [N][HV][K][V], nullable (zero)                            */
    const int64_t *cu_seqlens;
    void *o;                /* [B][T][HV][V]                                             */
    float *ht;              /* [N][HV][K][V], nullable.  gdn_linear_attn_recurrent: may
                               be h0 itself (the state updated in place)                 */
    const void *dout;       /* backward: [B][T][HV][V]                                   */
    int64_t ld_dout;
    const float *dht;       /* backward: [N][HV][K][V], nullable (zero)                  */
    void *dq, *dk, *dv;     /* backward: as q, k, v, contiguous                          */
    float *dh0;             /* backward: [N][HV][K][V], nullable                         */
} gdn_linear_attn_args;

/*
 * Linear attention with a decay for each value head:
 *     S_t = exp(decay) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
 *     S_0 = h0,  ht = S_T
 * in chunks of tokens: within a chunk the decayed products of q and k, between
 * chunks the state, in fp32.  On the tensor cores the decayed products and the
 * state are rounded to bf16 as operands of the output; what is added to the
 * state (exp(decay (n - 1 - j)) v_j, k_j as it is) is split into bf16 parts: into
 * three where ht is asked for, which is then good to fp32 (3e-7 of its 2-norm),
 * into two (16 bits) where o alone takes the state.  So o may differ by its
 * rounding between a call with ht and one without.
 * The decay is a constant of the layer: no gradient is computed for it.
 */
size_t gdn_linear_attn_workspace_size(const gdn_linear_attn_args *a);
gdn_status gdn_linear_attn(const gdn_linear_attn_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

/* The same token by token, for decoding and short continuations (fp32
 * throughout; suited to a few tokens per sequence). */
gdn_status gdn_linear_attn_recurrent(const gdn_linear_attn_args *a, gdn_stream_t stream);

/*
 * Gradients of gdn_linear_attn from its inputs, dout and dht.  With
 * R_t = exp(decay) R_{t+1} + scale q_t dout_t^T, dht joining at the last token:
 *     dq_t = scale S_t dout_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,
 *     dh0 = exp(decay) R_1
 * (key heads that several value heads share: the sum of theirs, in fp32, in a
 * fixed order).  On the tensor cores R is split as the state is, for dh0 into
 * three parts.
 */
size_t gdn_linear_attn_bwd_workspace_size(const gdn_linear_attn_args *a);
gdn_status gdn_linear_attn_bwd(const gdn_linear_attn_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

typedef struct {
    int B, Tq, Tk, H, HK, D;  /* packed: B = 1, Tq and Tk all tokens; D <= 256           */
    int num_seqs;
    gdn_dtype dtype;          /* q, k, v, o and the gradients: GDN_F32 or GDN_BF16       */
    int window;               /* >= 1: keys a query sees, its own among them             */
    int sinks;                /* >= 0: first keys of the sequence that stay visible      */
    float scale;
    const void *q, *k, *v;    /* [B][Tq][H][D], [B][Tk][HK][D] twice                     */
    int64_t ldq, ldk, ldv;
    const int64_t *cu_seqlens_q, *cu_seqlens_k; /* [N + 1] both, or none                 */
    void *o;                  /* [B][Tq][H][D] (backward: an input)                      */
    float *lse;               /* [B][H][Tq], nullable (backward: an input)               */
    const void *dout;         /* backward: [B][Tq][H][D]                                 */
    int64_t ld_dout;
    void *dq, *dk, *dv;       /* backward: as q, k, v, contiguous                        */
    int64_t o_seq, o_tok, o_head; /* backward: o's strides in elements (consecutive in a
                                 head), as [B][H][Tq][D] has them; all zero: contiguous  */
} gdn_window_attn_args;

/*
 * Causal softmax attention with a sliding window and sinks.  Query i of a
 * sequence of Lq queries and Lk keys stands at p = i + Lk - Lq and sees key j
 * when j <= p and (p - j < window or j < sinks):
 *     o_i = sum_j softmax_j(scale q_i . k_j) v_j
 *     lse_i = log sum_j exp(scale q_i . k_j)
 * A row that sees nothing (p < 0) gives zeros and lse = -infinity.  Scores,
 * statistics and sums in fp32; on the tensor cores the weights exp(..) are
 * rounded to bf16 as operands.
 */
size_t gdn_window_attn_workspace_size(const gdn_window_attn_args *a);
gdn_status gdn_window_attn(const gdn_window_attn_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

/*
 * Gradients of gdn_window_attn from its inputs, o, lse and dout: with
 * p = exp(scale s - lse), delta = dout . o and dz = p (dout v^T - delta) scale,
 *     dq = dz k,  dk = dz^T q,  dv = p^T dout
 * (summed over the query heads of a key head in fp32, in a fixed order).
 */
size_t gdn_window_attn_bwd_workspace_size(const gdn_window_attn_args *a);
gdn_status gdn_window_attn_bwd(const gdn_window_attn_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

typedef struct {
    int N, T, S, H, HK, D;    /* sequences, new tokens each, cache slots each            */
    gdn_dtype dtype;
    int window, sinks;        /* as gdn_window_attn_args                                 */
    float scale;
    const void *q;            /* [N][T][H][D]                                            */
    int64_t ldq;
    const void *k, *v;        /* [N][S][HK][D], any strides, consecutive elements        */
    int64_t k_seq, k_tok, k_head, v_seq, v_tok, v_head; /* strides in elements           */
    const void *lengths;      /* [N]: slots filled, the new tokens among them            */
    int lengths_64;           /* lengths are int64 (else int32)                          */
    void *o;                  /* [N][T][H][D]                                            */
} gdn_window_decode_args;

/*
 * gdn_window_attn for a few new tokens over a cache: new token t of sequence n
 * stands at position lengths[n] - T + t.  Slots from lengths[n] on and slots
 * outside the window and the sinks are not read.  Lengths are clamped to
 * [0, S]; a row that sees nothing gives zeros.
 */
size_t gdn_window_attn_decode_workspace_size(const gdn_window_decode_args *a);
gdn_status gdn_window_attn_decode(const gdn_window_decode_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream);

/* Plan summary (host only, no GPU needed) -- what a call would launch: the
 * engine and the in-GPU split (FlashQLA blog, "A balanced solution", the CP
 * enable rule, re-derived for this GPU's SM count). */
typedef struct {
    gdn_engine engine;    /* engine the call would use                    */
    gdn_cp_mode cp_mode;  /* OFF, EXACT or WARMUP after AUTO is resolved   */
    int segment_chunks;   /* chunks per segment (huge when OFF)            */
    int segments;         /* segments per sequence (grid bound)            */
    int value_tiles;      /* CTAs per (sequence, head, segment)            */
    int kernels;          /* kernel launches per call                      */
    size_t workspace_bytes;
} gdn_plan_info;

gdn_status gdn_plan(const gdn_shape *s, int chunk_size, const gdn_options *opt,
                    int num_sms, gdn_plan_info *out);

#ifdef __cplusplus
}
#endif

#endif /* GDN_GB300_H */
