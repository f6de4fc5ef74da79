/*
 * streamkl.h -- C ABI of libstreamkl: the fused attention KL divergence on
 * one GB300 (sm_103a) GPU.
 *
 * Method: "StreamKL: Fast and Memory-Efficient KL Divergence for Boosting
 * Attention Distillation" (gist.science/paper/2606.20005, technical summary).
 * For every query row i of every (batch b, head h):
 *
 *     S_t = scale * Q_t K_t^T        t = 1 (teacher), 2 (student)
 *     P_t = softmax(S_t) over the keys row i may see
 *     KL[i] = sum_j P1[i,j] * (log P1[i,j] - log P2[i,j])        (Problem Statement)
 *
 * computed without ever holding an Nq x Nk matrix: the forward streams key
 * tiles through five running scalars per row (Methodology 1, "Online
 * Formulation") and saves only KL, LSE1, LSE2; the backward regenerates
 * P_t = exp(S_t - LSE_t) tile by tile (Methodology 2, "Recomputation
 * Strategy").  Small query counts split the key range across CTAs and merge
 * the partial states (Methodology 3, "Split-K Variant").
 *
 * Conventions shared by every entry point
 *  - Q1, K1, Q2, K2 are bf16 device tensors laid out [B, H, N, d] with d
 *    contiguous (K1, K2 have H_kv heads when keys are shared across a group
 *    of query heads); the element strides of the B, H and N axes are given in
 *    streamkl_shape and must be multiples of 8 elements (16 bytes).  Q1 and
 *    Q2 share one set of strides, K1 and K2 another.  Base pointers must be
 *    16-byte aligned.  d must be 64 or 128.
 *  - KL, LSE1, LSE2 and g are float32 [B, H, Nq], contiguous.  dQ is
 *    [B, H, Nq, d] and dK [B, H_kv, Nk, d], contiguous, float32 (or bf16 on
 *    request); with shared keys dK sums the gradients of every query head of
 *    the group.
 *  - Logarithms are natural.  LSE_t[i] = log sum_j exp(S_t[i,j]) includes the
 *    softmax scale.
 *  - causal != 0 aligns the mask bottom-right: row i sees keys
 *    j <= i + (Nk - Nq).  It requires Nq <= Nk, so no row is empty.
 *  - scale <= 0 (or NaN) selects the default d^-1/2.
 *  - The caller owns every buffer, inputs, outputs and workspace alike.  The
 *    library allocates no device memory, keeps no state between calls and
 *    runs everything asynchronously on the caller's stream.  Arguments are
 *    validated before anything is launched; on an error nothing is launched
 *    and no output is touched.
 *  - streamkl_fwd, streamkl_bwd and streamkl_bwd_joint only enqueue
 *    asynchronous work (kernels and a memset) on the caller's stream: with
 *    buffers allocated beforehand, a sequence of them can be captured into a
 *    CUDA graph and replayed.
 *  - Workspace: the first 256 bytes hold a device error word that kernels set
 *    (they never clear it) when a bounded wait inside them gives up.  Zero the
 *    workspace once when it is allocated; streamkl_workspace_status reads and
 *    clears the word.  A workspace must not be shared by calls that may run
 *    at the same time on different streams.
 */
#ifndef STREAMKL_H
#define STREAMKL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define STREAMKL_API __attribute__((visibility("default")))
#else
#define STREAMKL_API
#endif

/* Same object as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* streamkl_stream_t;

typedef enum {
    STREAMKL_OK = 0,
    STREAMKL_ERR_INVALID_ARG = 1, /* null pointer, bad size, misalignment, bad setting */
    STREAMKL_ERR_UNSUPPORTED = 2, /* valid but not implemented here (e.g. d not 64/128) */
    STREAMKL_ERR_WORKSPACE = 3,   /* workspace missing or smaller than the size query said */
    STREAMKL_ERR_CUDA = 4,        /* a CUDA runtime/driver call or launch failed */
    STREAMKL_ERR_TIMEOUT = 5      /* a kernel's bounded wait gave up (device error word) */
} streamkl_status;

typedef struct {
    int32_t B, H, Nq, Nk, d;
    int64_t q_stride_b, q_stride_h, q_stride_n; /* element strides of Q1 and Q2 */
    int64_t k_stride_b, k_stride_h, k_stride_n; /* element strides of K1 and K2 */
    int32_t H_kv; /* key heads: 0 (or H) = one per query head; otherwise H_kv divides H and
                     query head h uses key head h / (H / H_kv) (keys shared by a group) */
} streamkl_shape;

/* Optional knobs; pass NULL for the defaults. */
typedef struct {
    int32_t num_splits;    /* forward and key-split backward: 0 = automatic,        */
                           /*   n >= 1 forces n key-range splits                    */
    int32_t bwd_mode;      /* backward: 0 = automatic, 1 = fused (atomic dQ),        */
                           /*           2 = separate dQ and dK kernels,               */
                           /*           3 = key-split (needs Nq * H / H_kv <= 16)     */
    int64_t wait_limit_ns; /* limit of every in-kernel wait; 0 = default (2 s)      */
    int32_t debug_flags;   /* 0 in normal use; see STREAMKL_DEBUG_*                  */
    int32_t grad_bf16;     /* backward: 0 = float32 dQ/dK, 1 = bf16 dQ/dK            */
} streamkl_options;

/* Test aid for the bounded waits: the first CTA of the main kernel waits on a
 * barrier that nothing arrives on.  The wait gives up after wait_limit_ns,
 * the kernel records STREAMKL_ERR_TIMEOUT in the workspace error word and
 * returns; the outputs of that call are undefined. */
#define STREAMKL_DEBUG_INJECT_STALL 1

/* What a call will launch for a given shape (filled by the plan queries). */
typedef struct {
    int32_t path;       /* 0 = tile forward, 1 = decode (Nq <= 16, causal or not) forward,
                           2 = fused backward, 3 = separate-kernel backward,
                           4 = key-split backward (at most 16 query rows per key head;
                               the automatic choice there),
                           5 = joint backward (both sides, streamkl_bwd_joint) */
    int32_t num_splits; /* key splits of the forward (1 = no combine step) or of the
                           key-split backward */
    int32_t num_ctas;   /* CTAs of the main kernel                          */
    int32_t launches;   /* kernels launched per call                        */
    size_t workspace_bytes;
} streamkl_plan;

/* Plan of streamkl_fwd for this shape on the current device.  Needs a CUDA
 * device (the split count depends on its SM count).  Errors: INVALID_ARG,
 * UNSUPPORTED, CUDA. */
STREAMKL_API streamkl_status streamkl_fwd_plan(const streamkl_shape* shape, int causal, const streamkl_options* opt,
                                  streamkl_plan* plan);

/* Forward (Methodology 1 and 3).  Writes KL, LSE1, LSE2 for every row.
 * workspace must hold at least streamkl_fwd_plan(...).workspace_bytes bytes
 * (256 for the status word plus 20 bytes per row and split when the key
 * range is split).  Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
STREAMKL_API streamkl_status streamkl_fwd(const streamkl_shape* shape, const void* Q1, const void* K1, const void* Q2,
                             const void* K2, float scale, int causal, float* KL, float* LSE1, float* LSE2,
                             void* workspace, size_t workspace_bytes, const streamkl_options* opt,
                             streamkl_stream_t stream);

/* Plan of streamkl_bwd (fused vs separate kernels, workspace). */
STREAMKL_API streamkl_status streamkl_bwd_plan(const streamkl_shape* shape, int setting, int causal,
                                  const streamkl_options* opt, streamkl_plan* plan);

/* Backward (Methodology 2).  Gradient of sum_i g[i] * KL[i] with respect to
 * the trainable side:
 *   setting 1 (teacher fixed): dQ = dL/dQ2, dK = dL/dK2, dS2 = g (P2 - P1)
 *   setting 2 (student fixed): dQ = dL/dQ1, dK = dL/dK1,
 *                              dS1 = g P1 ((S1 - LSE1) - (S2 - LSE2) - KL)
 * and dQ = scale * dS K, dK = scale * dS^T Q.  KL, LSE1, LSE2 are the
 * forward's outputs for the same inputs.  dQ and dK are overwritten; they are
 * float32 unless opt->grad_bf16 selects bf16 (the fused mode then also needs
 * 4 bytes per dQ element of workspace to accumulate in float32).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
STREAMKL_API streamkl_status streamkl_bwd(const streamkl_shape* shape, int setting, const float* g, const void* Q1,
                             const void* K1, const void* Q2, const void* K2, const float* KL, const float* LSE1,
                             const float* LSE2, float scale, int causal, void* dQ, void* dK, void* workspace,
                             size_t workspace_bytes, const streamkl_options* opt, streamkl_stream_t stream);

/* Joint backward (Methodology 2, both settings at once): the gradient of
 * sum_i g[i] * KL[i] with respect to all four inputs, where the teacher's
 * gradients differentiate through P1 with P2 held fixed (setting 2) and the
 * student's through P2 with P1 held fixed (setting 1):
 *   dQ1 = scale * dS1 K1,  dK1 = scale * dS1^T Q1,  dS1 = g P1 ((S1 - LSE1) - (S2 - LSE2) - KL)
 *   dQ2 = scale * dS2 K2,  dK2 = scale * dS2^T Q2,  dS2 = g (P2 - P1)
 * Results equal streamkl_bwd with setting 2 (dQ1, dK1) and setting 1 (dQ2,
 * dK2), but the scores are regenerated once per kernel for both: a query-tile
 * kernel accumulates dQ1 and dQ2, a key-tile kernel dK1 and dK2, each output
 * written once (no atomics: the results are deterministic).  Layouts, dtypes
 * (opt->grad_bf16) and shared keys as for streamkl_bwd; dQ1/dQ2 are
 * [B, H, Nq, d], dK1/dK2 [B, H_kv, Nk, d].  opt->bwd_mode must be 0 and
 * num_splits is ignored.  The workspace holds the 256-byte error word only
 * (streamkl_bwd_joint_plan: path 5, 2 launches).  For at most 16 query rows
 * per key head (decode shapes) two streamkl_bwd calls, which take the
 * key-split kernel there, are faster.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
STREAMKL_API streamkl_status streamkl_bwd_joint_plan(const streamkl_shape* shape, int causal,
                                                     const streamkl_options* opt, streamkl_plan* plan);
STREAMKL_API streamkl_status streamkl_bwd_joint(const streamkl_shape* shape, const float* g, const void* Q1,
                                                const void* K1, const void* Q2, const void* K2, const float* KL,
                                                const float* LSE1, const float* LSE2, float scale, int causal,
                                                void* dQ1, void* dK1, void* dQ2, void* dK2, void* workspace,
                                                size_t workspace_bytes, const streamkl_options* opt,
                                                streamkl_stream_t stream);

/* Workspace sizes alone, with the default options (opt == NULL): the
 * workspace_bytes field of streamkl_fwd_plan / streamkl_bwd_plan.  They return
 * 0 when the shape, causal flag or setting is invalid or no CUDA device is
 * current (a valid call always needs at least the 256-byte status word).
 * Options that change the size (forced splits, bf16 gradients) need the plan
 * queries. */
STREAMKL_API size_t streamkl_fwd_workspace_bytes(const streamkl_shape* shape, int causal);
STREAMKL_API size_t streamkl_bwd_workspace_bytes(const streamkl_shape* shape, int setting, int causal);

/* Size of the library's own built-in scratch buffer used by streamkl_fwd_noalloc. */
#define STREAMKL_NOALLOC_SCRATCH_BYTES (8u << 20)

/* Forward for callers that cannot allocate device memory themselves -- for
 * example a host program or plugin that is handed tensor pointers by a
 * runtime that owns all device memory and offers it no allocator, or a
 * caller that must not allocate once its memory plan is fixed.  This entry
 * point has no counterpart in the paper; it is streamkl_fwd with the
 * workspace replaced by a fixed buffer that lives inside the library.
 *
 * Same arguments, outputs and validation as streamkl_fwd, minus the
 * workspace.  Neither this call nor anything it launches allocates device
 * memory: the scratch (the device error word plus the Split-K partial
 * states) is a file-scope device array of STREAMKL_NOALLOC_SCRATCH_BYTES
 * bytes that every GPU which loads the library holds until the process
 * exits.  A shape whose plan needs more scratch than that (20 bytes per
 * query row and key split, plus 256) returns STREAMKL_ERR_WORKSPACE and
 * launches nothing.  Every call looks up the array's device address on the
 * current device (a table lookup, no allocation); the first call on a device
 * also loads the library's device code there, so make that first call before
 * any stream capture.  All calls share the one array, so calls that may
 * overlap on the GPU (different streams, or different host threads) race on
 * it and must be serialised by the caller.
 *
 * A bounded wait inside the kernels that gives up (see wait_limit_ns) does
 * not change the return value, which only covers validation and launch: the
 * rows that the giving-up CTA owned come back as NaN, and the scratch's
 * device error word is set.  Read it with streamkl_noalloc_status after the
 * call and before the next one, which clears the word when it starts.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
STREAMKL_API streamkl_status streamkl_fwd_noalloc(const streamkl_shape* shape, const void* Q1, const void* K1,
                                                  const void* Q2, const void* K2, float scale, int causal, float* KL,
                                                  float* LSE1, float* LSE2, const streamkl_options* opt,
                                                  streamkl_stream_t stream);

/* streamkl_workspace_status for the built-in scratch of streamkl_fwd_noalloc
 * on the current device: synchronises `stream`, reads the device error word
 * into *device_error (if not NULL), clears it, and returns
 * STREAMKL_ERR_TIMEOUT if it was set, STREAMKL_OK otherwise (CUDA on a failed
 * copy).  Allocates nothing. */
STREAMKL_API streamkl_status streamkl_noalloc_status(streamkl_stream_t stream, uint32_t* device_error);

/* ---------------------------------------------------------------------------
 * Divergence of two attentions with modified scores.
 *
 * The divergence above with, per side t,
 *
 *     S_t = cap_t tanh(scale z_t / cap_t) - slopes_t[h] |i + offset[b] - j|
 *
 * for z_t = <q_t, k_t> of query row i and key j (cap_t = 0: scale z_t; slopes_t
 * NULL: no bias), and with the keys of each row restricted to a range:
 *
 *     begin[b, i] <= j < end[b, i],  and when causal  j <= i + offset[b].
 *
 * offset[b] is the key position of query row 0 (NULL: Nk - Nq, the bottom-right
 * alignment).  The ranges express causal, document, sliding-window and prefix
 * masks, padded batches and caches of unequal lengths, for both sides alike.
 *
 *  - begin, end: int32 [B, Nq], contiguous; NULL: 0 and Nk.  Values outside
 *    [0, Nk] are clamped.  offset: int32 [B].  slopes1, slopes2: float32 [H].
 *    All on the device.
 *  - A row that sees no key has KL = 0, LSE1 = LSE2 = -inf and zero gradients;
 *    a key that no row sees gets zero gradients; causal with Nq > Nk is allowed.
 *  - What a row does not see has no effect on its outputs and gradients, NaN
 *    and infinities included.  A visible one (or a product that overflows
 *    float32) makes the row NaN, capped or not.
 *  - A capped side needs 1e-5 <= scale / cap <= 1e5 (UNSUPPORTED otherwise).
 *  - The backward is the fused one (dQ added up in float32 in no fixed order, dK
 *    the same on every run); opt->bwd_mode must be 0; opt->num_splits sets the
 *    CTAs that share the query rows of a key tile (0 = automatic).  Its gradients include the slope of the cap,
 *    1 - tanh^2.  begin, end, offset, slopes, caps and scale as in the forward.
 *    bf16 gradients are the float32 ones, rounded once.
 *  - After a bounded wait has given up (the workspace's error word says so), the
 *    rows of KL and LSE, of dK and of dQ that lack anything are NaN.
 *  - Layouts, strides, dtypes, shared keys, workspace and streams as above.
 * ------------------------------------------------------------------------- */
typedef struct {
    float cap1, cap2;       /* the teacher's and the student's; 0 = none */
    const float* slopes1;
    const float* slopes2;
    const int32_t* begin;
    const int32_t* end;
    const int32_t* offset;
} streamkl_score;

/* score == NULL: plain scores, every key visible (up to causal).  Paths of the
 * plans: 0 tile forward, 1 decode forward (Nq <= 16), 2 fused backward.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
STREAMKL_API streamkl_status streamkl_score_fwd_plan(const streamkl_shape* shape, const streamkl_options* opt,
                                                     streamkl_plan* plan);
STREAMKL_API streamkl_status streamkl_score_fwd(const streamkl_shape* shape, const streamkl_score* score,
                                                const void* Q1, const void* K1, const void* Q2, const void* K2,
                                                float scale, int causal, float* KL, float* LSE1, float* LSE2,
                                                void* workspace, size_t workspace_bytes, const streamkl_options* opt,
                                                streamkl_stream_t stream);
STREAMKL_API streamkl_status streamkl_score_bwd_plan(const streamkl_shape* shape, int setting,
                                                     const streamkl_options* opt, streamkl_plan* plan);
STREAMKL_API streamkl_status streamkl_score_bwd(const streamkl_shape* shape, const streamkl_score* score, int setting,
                                                const float* g, const void* Q1, const void* K1, const void* Q2,
                                                const void* K2, const float* KL, const float* LSE1, const float* LSE2,
                                                float scale, int causal, void* dQ, void* dK, void* workspace,
                                                size_t workspace_bytes, const streamkl_options* opt,
                                                streamkl_stream_t stream);

/* Key ranges (begin, end, offset of streamkl_score) from the usual masks.  Query
 * row i < q_lengths[b] stands at key position p = i + offset[b], offset[b] =
 * k_lengths[b] - q_lengths[b] (lengths NULL: Nq, Nk; clamped to them; B up to
 * 65535 and Nq up to 2^31 - 256, UNSUPPORTED beyond); later
 * rows see nothing.  It sees the keys j < k_lengths[b] with
 *   causal:      j <= p;
 *   window > 0:  p - window < j < p + window;
 *   prefix [B]:  j <= p or j < prefix[b] (with causal; not with window or docs:
 *                UNSUPPORTED, the visible keys would not be one range);
 *   docs:        j in the document of p; num_bounds nondecreasing bounds, [num_bounds]
 *                or with docs_per_batch [B, num_bounds], document m being keys
 *                docs[m] <= j < docs[m + 1] (rows outside every document see nothing).
 * begin, end: int32 [B, Nq]; offset: int32 [B]; written by one launch.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
STREAMKL_API streamkl_status streamkl_key_ranges(int32_t B, int32_t Nq, int32_t Nk, int causal, int32_t window,
                                                 const int32_t* q_lengths, const int32_t* k_lengths,
                                                 const int32_t* prefix, const int32_t* docs, int32_t num_bounds,
                                                 int32_t docs_per_batch, int32_t* begin, int32_t* end, int32_t* offset,
                                                 streamkl_stream_t stream);

/* ---------------------------------------------------------------------------
 * Norm of query and key heads with the position rotation, and its gradient.
 *
 * The step before the divergence: for every head x (d values) of q and k
 *
 *     r = (mean(x^2) + eps)^(-1/2),   y = R(position) (r x * w)
 *
 * where R turns the first `rot` values of the head as pairs, (e, e + rot/2)
 * or, interleaved, (2e, 2e + 1), by the angle of the position and pair e:
 * (a, b) -> (a cos - b sin, b cos + a sin).  One launch covers q and k.
 *
 *  - q [B, Hq, N, d] and k [B, Hk, N, d] are bf16 with d contiguous, read
 *    through element strides (multiples of 8; 0 repeats along an axis), so
 *    that views of one packed projection need no copy; d is 64 or 128, rot a
 *    multiple of 8 up to d (0: norm only).  y is bf16 with strides of its
 *    own (e.g. rows of a cache); yq may be q and yk may be k.
 *  - wq, wk: [d], float32 or bf16 (weight_bf16), or NULL for weights of one.
 *  - table: float32 [table_rows, rot/2, 2], cosine and sine of each position
 *    and pair (streamkl_rope_table makes one).  positions: [B, N], int32 or
 *    int64 (pos_int64), contiguous, or NULL for start + n.  A row whose
 *    position is outside the table gets NaN in the rotated values (and in
 *    its gradients, and so in dwq / dwk).
 *  - N = 0 is allowed: nothing is written but zeros to dwq and dwk.
 *  - Statistics and sums are float32; every output is rounded once.
 * ------------------------------------------------------------------------- */
typedef struct {
    int64_t b, h, n; /* element strides of the B, H and N axes */
} streamkl_strides;

typedef struct {
    int32_t B, Hq, Hk, N, d, rot;
    int32_t interleaved; /* 0: pairs (e, e + rot/2), 1: pairs (2e, 2e + 1) */
    int32_t weight_bf16; /* wq, wk (and dwq, dwk): 0 = float32, 1 = bf16    */
    int32_t grad_bf16;   /* dyq, dyk of the backward: 0 = float32, 1 = bf16 */
    int32_t pos_int64;   /* positions: 0 = int32, 1 = int64                 */
    float eps;
    int64_t table_rows;
    int64_t start;           /* first position when positions is NULL */
    streamkl_strides q, k;   /* q and k */
    streamkl_strides yq, yk; /* yq and yk, or in the backward dyq and dyk */
    streamkl_strides dq, dk; /* backward only: dq and dk */
} streamkl_norm_rope;

/* Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
STREAMKL_API streamkl_status streamkl_norm_rope_fwd(const streamkl_norm_rope* desc, const void* q, const void* k,
                                                    const void* wq, const void* wk, const float* table,
                                                    const void* positions, void* yq, void* yk,
                                                    streamkl_stream_t stream);

/* Gradient of sum(dyq * yq) + sum(dyk * yk): dq, dk (bf16, strided) and
 * dwq, dwk ([d], the weights' type; NULL to skip one).  dq may be dyq and dk
 * may be dyk when those are bf16 with the same strides.  The sums run in a
 * fixed order: equal inputs give equal bits.  workspace as for the other
 * calls; its size is streamkl_norm_rope_workspace_bytes, which returns 0 for
 * an invalid description or when no CUDA device is current.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
STREAMKL_API size_t streamkl_norm_rope_workspace_bytes(const streamkl_norm_rope* desc);
STREAMKL_API streamkl_status streamkl_norm_rope_bwd(const streamkl_norm_rope* desc, const void* dyq, const void* dyk,
                                                    const void* q, const void* k, const void* wq, const void* wk,
                                                    const float* table, const void* positions, void* dq, void* dk,
                                                    void* dwq, void* dwk, void* workspace, size_t workspace_bytes,
                                                    streamkl_stream_t stream);

/* The same with positions on several axes (time, height and width of a patch):
 * positions is [axes, B, N] (not NULL), and pair e of a head is turned by the
 * token's position on axis axis_of[e], e < rot / 2 (axes up to 4), through the
 * table's row of that position.  Errors as above; INVALID_ARG for axes NULL. */
typedef struct {
    int32_t axes;
    uint8_t axis_of[64];
} streamkl_rope_axes;

STREAMKL_API streamkl_status streamkl_norm_rope_axes_fwd(const streamkl_norm_rope* desc, const streamkl_rope_axes* axes,
                                                         const void* q, const void* k, const void* wq, const void* wk,
                                                         const float* table, const void* positions, void* yq, void* yk,
                                                         streamkl_stream_t stream);
STREAMKL_API streamkl_status streamkl_norm_rope_axes_bwd(const streamkl_norm_rope* desc, const streamkl_rope_axes* axes,
                                                         const void* dyq, const void* dyk, const void* q, const void* k,
                                                         const void* wq, const void* wk, const float* table,
                                                         const void* positions, void* dq, void* dk, void* dwq, void* dwk,
                                                         void* workspace, size_t workspace_bytes,
                                                         streamkl_stream_t stream);

/* table[n][e] = (cos, sin) of n * inv_freq[e] for n < rows, e < half, from
 * angles in float64 (at position 10^6 a float32 angle is off by 0.03).
 * inv_freq: device float64 [half].  Errors: INVALID_ARG, CUDA. */
STREAMKL_API streamkl_status streamkl_rope_table(const double* inv_freq, int64_t rows, int32_t half, float* table,
                                                 streamkl_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention over whole prompts, and its gradients.
 *
 * For every query row i of every (batch b, head h), over the keys j of its
 * range (begin[b, i] <= j < end[b, i]; NULL: 0 and Nk; with causal != 0 also
 * j <= i + offset[b], NULL: Nk - Nq):
 *
 *     S = scale * Q K^T,  LSE[i] = log sum_j exp(S[i,j]),
 *     O[i] = sum_j exp(S[i,j] - LSE[i]) V[j]
 *
 *  - Q, O, dO [B, H, Nq, d] and K, V [B, H_kv, Nk, d] are bf16 with d
 *    contiguous (64 or 128) and strides of their own, multiples of 8 elements,
 *    that keep rows apart; H_kv divides H, and query head h uses key head
 *    h / (H / H_kv).  Base pointers are 16-byte aligned.
 *  - A row that sees no key has O = 0 and LSE = -inf, and no effect on any
 *    gradient.  What a row does not see (NaN and infinities included) has no
 *    effect on it; a row that sees a NaN or an infinite value of V gets NaN or an
 *    infinity in O, at least where that value counts and at most in the whole row.
 *    LSE has no values in it.
 *  - rest (NULL or bf16 [B, H, Nq, d], contiguous): what the rounding of O to
 *    bf16 left, for the backward's row sums of dO * O.
 *  - Probabilities enter the product with V rounded to bf16, with rest as two
 *    bf16 terms; sums, maxima and outputs are float32 until their one rounding.
 *  - Scores are float32: a probability is off by up to about 2^-22 max |S|, and
 *    rows with scores beyond 2^28 may be NaN.
 *  - Equal inputs give equal bits.  A give-up of a bounded wait leaves NaN in
 *    the rows that it left unfinished.
 *  - workspace may be NULL for a forward whose plan has 256 bytes (one split):
 *    nothing but the error word would stand there.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------- */
typedef struct {
    int32_t B, H, H_kv, Nq, Nk, d;
    streamkl_strides q, k, v, o;
    streamkl_strides d_o; /* backward only: dO */
} streamkl_attn;

STREAMKL_API streamkl_status streamkl_attn_fwd_plan(const streamkl_attn* desc, const streamkl_options* opt,
                                                    streamkl_plan* plan);
STREAMKL_API streamkl_status streamkl_attn_fwd(const streamkl_attn* desc, const void* Q, const void* K, const void* V,
                                               const int32_t* begin, const int32_t* end, const int32_t* offset,
                                               float scale, int causal, void* O, void* rest, float* LSE,
                                               void* workspace, size_t workspace_bytes, const streamkl_options* opt,
                                               streamkl_stream_t stream);

/* Gradients of sum(dO * O): dQ [B, H, Nq, d], dK, dV [B, H_kv, Nk, d], bf16 and
 * contiguous, sums in float32 rounded once; dK and dV sum over the query heads
 * of a key head.  O, rest and LSE are the forward's for the same inputs; without
 * rest (NULL) the row sums of dO * O carry O's rounding, which shows in dQ where
 * keys have much in common.  dQ is added up in no fixed order; dK and dV are the
 * same on every run.  Tokens that are not finite reach the gradients as in the
 * formulas (a visible key that scores -inf has P = dS = 0, and dQ = 0 * -inf where
 * it is infinite), but for those of dO: they make all features of dV NaN. */
STREAMKL_API streamkl_status streamkl_attn_bwd_plan(const streamkl_attn* desc, const streamkl_options* opt,
                                                    streamkl_plan* plan);
STREAMKL_API streamkl_status streamkl_attn_bwd(const streamkl_attn* desc, const void* dO, const void* Q, const void* K,
                                               const void* V, const void* O, const void* rest, const float* LSE,
                                               const int32_t* begin, const int32_t* end, const int32_t* offset,
                                               float scale, int causal, void* dQ, void* dK, void* dV, void* workspace,
                                               size_t workspace_bytes, const streamkl_options* opt,
                                               streamkl_stream_t stream);

/* ---------------------------------------------------------------------------
 * A paged cache of keys and values in 8 bits, and attention over it.
 *
 * k, v [pages, H_kv, T, d] are e4m3 bytes, contiguous, 16-byte aligned; T is 16,
 * 32, 64 or 128 and d is 64 or 128.  k_scale, v_scale [pages, H_kv] are float32,
 * positive and normal: a stored value stands for itself times its page's and
 * head's scale.  Token j of sequence b stands in row j % T of page
 * table[b][j / T]; table is int32 [B, M], lengths int32 [B] (tokens held before
 * the call of append, in all for the others; below 0 counts as 0).  A page may be
 * listed by several sequences as long as none of them appends to it.
 *
 * append writes counts[b] (int32 [B], clamped to 0 .. N; NULL: N) new tokens of
 * new_k, new_v [B, H_kv, N, d] (bf16) behind each sequence's lengths[b].  A page's
 * scale becomes the smallest 2^e, e >= -100, with every finite value of its new
 * tokens within 448 2^e, and no less than it was when the page held tokens
 * of the sequence before; those are then rounded to the new scale.  NaN and
 * infinities are stored as NaN.  Rows of the page behind the new tokens stay as
 * they are.  Tokens behind the table, or of a page outside [0, pages), are not
 * written.  A page that a call appends to is listed once, by one sequence.
 *
 * read gathers the first N tokens of each sequence as bf16 [B, H_kv, N, d]: zeros
 * behind lengths[b], NaN for pages that are not there.
 *
 * attn_cache8: softmax attention of the last N tokens (1 to 16) of each sequence,
 * Q [B, H, N, d] bf16, row i seeing keys j < lengths[b] - N + 1 + i; query head h
 * uses key head h / (H / H_kv).  O is bf16 [B, H, N, d], LSE float32 [B, H, N]; a
 * row that sees no key has O = 0 and LSE = -inf; a row that sees a page that is
 * not there, or a sequence longer than its table, is NaN, and so are rows that a
 * give-up of a bounded wait left unfinished.  opt->num_splits: CTAs that share out
 * the keys of all sequences (0 = automatic).  workspace may be NULL where the plan
 * has 256 bytes.  Equal inputs give equal bits.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------- */
typedef struct {
    int32_t pages, H_kv, T, d;
    int32_t B, M;
    int32_t H;          /* attn_cache8: query heads */
    int32_t N;          /* tokens of x and y */
    streamkl_strides x; /* new_k, out_k, or Q: element strides, multiples of 8 */
    streamkl_strides y; /* new_v, out_v, or O */
} streamkl_cache8;

STREAMKL_API streamkl_status streamkl_cache8_append(const streamkl_cache8* desc, void* k, void* v, float* k_scale,
                                                    float* v_scale, const int32_t* table, const int32_t* lengths,
                                                    const void* new_k, const void* new_v, const int32_t* counts,
                                                    streamkl_stream_t stream);
STREAMKL_API streamkl_status streamkl_cache8_read(const streamkl_cache8* desc, const void* k, const void* v,
                                                  const float* k_scale, const float* v_scale, const int32_t* table,
                                                  const int32_t* lengths, void* out_k, void* out_v,
                                                  streamkl_stream_t stream);
STREAMKL_API streamkl_status streamkl_attn_cache8_plan(const streamkl_cache8* desc, const streamkl_options* opt,
                                                       streamkl_plan* plan);
STREAMKL_API streamkl_status streamkl_attn_cache8(const streamkl_cache8* desc, const void* Q, const void* k, const void* v,
                                                  const float* k_scale, const float* v_scale, const int32_t* table,
                                                  const int32_t* lengths, float scale, void* O, float* LSE,
                                                  void* workspace, size_t workspace_bytes, const streamkl_options* opt,
                                                  streamkl_stream_t stream);

/* Synchronises `stream`, reads the workspace's device error word into
 * *device_error (if not NULL), clears it, and returns STREAMKL_ERR_TIMEOUT if
 * it was set, STREAMKL_OK otherwise (or CUDA on a failed copy). */
STREAMKL_API streamkl_status streamkl_workspace_status(void* workspace, streamkl_stream_t stream, uint32_t* device_error);

/* Static description of a status code; never NULL. */
STREAMKL_API const char* streamkl_status_string(streamkl_status status);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
STREAMKL_API int streamkl_version(void);

#ifdef __cplusplus
}
#endif

#endif /* STREAMKL_H */
