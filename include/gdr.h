/*
 * gdr.h -- C ABI of libgdr: Gated DeltaNet (GDN) chunked prefill, forward and
 * backward, on one NVIDIA GB300 (sm_103a).
 *
 * The operation (FlashQLA pages; problem statement of the GDN chunked-prefill
 * kernels): for every sequence n and value head h, with qk-head
 * hq = h / (Hv / Hq) (grouped heads, page 1 high-level API shapes),
 *
 *     S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,   a_t = exp(g_t),
 *     o_t = scale * S_t^T q_t,          S_0 = h0[n, h] (zeros when absent),
 *
 * evaluated chunk by chunk with 64-token chunks.  The calls mirror the
 * low-level entry points of page 1 ("usage and requirements"):
 *     forward  (q, k, v, g, beta, scale, h0, cu_seqlens) -> (o, final_state, A, h)
 *     backward (q, k, v, g, beta, A, do, dht, scale, h0, cu_seqlens)
 *                                                   -> (dq, dk, dv, dbeta, dg, dh0)
 * The cumulated gate g that the Python forward of the pages also returns is
 * not exported; the backward recomputes it from the raw g.
 *
 * Conventions shared by every call
 * --------------------------------
 * Layouts: row-major, innermost dimension last, contiguous, no padding:
 *   q, k, dq, dk        [B, T, Hq, K]
 *   v, o, do, dv        [B, T, Hv, V]
 *   g, beta, dg, dbeta  [B, T, Hv]          (fp32)
 *   A                   [B, T, Hv, 64]      (fp32; row r of its chunk's A at token r)
 *   h                   [NT, Hv, K, V]      (fp32; h[i] = state before chunk i)
 *   h0, final_state, dht, dh0   [N, Hv, K, V]   (fp32)
 * N = B for a fixed-length batch; for varlen (n_seqs > 0) B must be 1, the
 * sequences are packed along T and N = n_seqs.  Chunks restart at every
 * sequence start; NT (gdr_num_chunks) counts chunks over all sequences in order.
 * g is the per-token log-gate (<= 0 in the intended use: a_t in (0, 1]);
 * beta is the write strength as passed (already squashed by the caller).
 *
 * Sizes: K in {64, 128, 192}, V in {64, 128, 192, 256}; Hq >= 1; Hv a
 * multiple of Hq; T >= 1.  The tensor-core path takes bf16 inputs with
 * K = V = 128; every other size and fp32 inputs run on the CUDA cores.
 * Varlen sequences may have length 0 (their final state is h0).
 *
 * Ownership: the caller allocates every buffer, including the workspace
 * (sized by gdr_*_workspace_size).  The library allocates nothing, keeps no
 * state between calls and never writes its inputs.
 *
 * Execution: every call only enqueues work on `stream` (a cudaStream_t; NULL
 * is the legacy default stream) and returns; nothing synchronises.  Buffers
 * must stay valid until that work completes.  Calls on one workspace must not
 * overlap in time.
 *
 * Errors: every call returns GDR_OK (0) or one of the codes below; on an
 * argument error nothing is launched.  gdr_last_error() gives a message for
 * the calling thread's last failure.  Device-side problems (a bounded wait
 * that ran out, a violated index check in debug mode) are recorded in a device
 * status word and reported by gdr_check_status().
 */
#ifndef GDR_H
#define GDR_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define GDR_API __attribute__((visibility("default")))
#else
#define GDR_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* element types of gdr_buf */
#define GDR_BF16 0
#define GDR_F32 1

/* return codes */
#define GDR_OK 0
#define GDR_ERR_ARG 1       /* null or invalid argument */
#define GDR_ERR_SHAPE 2     /* unsupported sizes: K, V outside the sets above, Hv % Hq != 0, ... */
#define GDR_ERR_DTYPE 3     /* unsupported or mismatched element type */
#define GDR_ERR_ALIGN 4     /* a pointer not 16-byte aligned */
#define GDR_ERR_WORKSPACE 5 /* workspace missing or too small */
#define GDR_ERR_CUDA 6      /* a CUDA runtime call or launch failed */
#define GDR_ERR_TIMEOUT 7   /* a device-side bounded wait ran out (from gdr_check_status) */
#define GDR_ERR_DEVICE 8    /* a device-side index check failed (debug_checks) */

/* paths (gdr_opts.path) */
#define GDR_PATH_AUTO 0     /* tensor-core path where supported, else the CUDA-core path */
#define GDR_PATH_SIMT 1     /* fp32 CUDA-core kernels (any dtype, K,V in {64,128}) */
#define GDR_PATH_TC 2       /* tcgen05 tensor-core kernels (bf16, K = V = 128) */

/* A device buffer and its element type (GDR_BF16 or GDR_F32). */
typedef struct {
    void *ptr;
    int dtype;
} gdr_buf;

/* Problem sizes. */
typedef struct {
    int B, T, Hq, Hv, K, V;
    int n_seqs;                      /* 0: fixed-length batch; > 0: varlen, B must be 1 */
    const int32_t *cu_seqlens;       /* varlen: device array [n_seqs + 1], 0 .. T */
    const int32_t *cu_seqlens_host;  /* varlen: host copy of the same values */
} gdr_shape;

/* Options.  A zeroed struct (or NULL) selects every default. */
typedef struct {
    int cp_segments;        /* intra-card context parallelism: 0 auto, 1 off,
                               n > 1 = split the longest sequence into n segments */
    int path;               /* GDR_PATH_* */
    int debug_checks;       /* 1: kernels check every index against its extent */
    long long timeout_spins;/* cap on device-side barrier polls (0: default) */
    /* Optional per-kernel timing with caller-owned CUDA events (cudaEvent_t,
     * created by the caller).  When `events` is not NULL the call records
     * events[2i] on `stream` just before its i-th kernel launch and
     * events[2i+1] just after it, for i < max_events / 2, and stores a static
     * name of that kernel in names[i] (names may be NULL).  n_launched (may be
     * NULL) receives the number of kernels the call launched. */
    void **events;
    const char **names;
    int max_events;
    int *n_launched;
    /* Warm-up starts of context-parallel segments (FlashQLA pages: page 1,
     * "balanced solution", and page 3, "sliding-window warmup": a segment's
     * start state is approximated by scanning the few chunks before it from
     * zero).  Here it replaces the exact summary and combine for a v-head only
     * when, for every segment of every sequence, the bound on the start
     * state's error, prod_t a_t max(1, |1 - b_t |k_t|^2|) over the warm-up
     * window, is below 1e-6 (or the window reaches the sequence start, where
     * the warm-up is exact).  0 (default): 8 warm-up chunks where the plan's
     * segments are at least 32 chunks long, else the exact split; -1: always
     * the exact split; n > 0: n warm-up chunks.  Tensor-core path, forward and
     * the backward's state recompute; the reverse scan is always exact. */
    int cp_warmup;
} gdr_opts;

/* Number of 64-token chunks over all sequences (the NT of h).  -1 on bad shape. */
GDR_API long long gdr_num_chunks(const gdr_shape *shape);

/* How a call with these sizes, input dtype and options would run.  The
 * intra-card context-parallel split follows the pages' cost reasoning (page 1,
 * "two fused kernels and automatic CP": the per-segment steps cost about the
 * segment length, the combine about the number of segments), re-fitted to the
 * SM count of the current device (152 when no device is visible). */
typedef struct {
    int path;             /* GDR_PATH_SIMT or GDR_PATH_TC */
    long long n_chunks;   /* as gdr_num_chunks */
    int n_segments;       /* segments over all sequences; equal to the number of
                             sequences when no sequence is split */
    int seg_len;          /* chunks per segment (a sequence's last may be shorter) */
    int cp_warmup;        /* warm-up chunks at segment starts (0: exact split only) */
} gdr_plan;

/* Fills *out for a forward or backward call with inputs of element type
 * `in_dtype` (GDR_BF16 or GDR_F32).  Host-side only: touches no device memory
 * and launches nothing.  Returns GDR_OK or the error gdr_fwd would return for
 * these sizes, dtype and options. */
GDR_API int gdr_get_plan(const gdr_shape *shape, int in_dtype, const gdr_opts *opts, gdr_plan *out);

/* Workspace bytes needed by gdr_fwd / gdr_bwd for this shape and options.
 * Returns 0 and sets the last error on an invalid shape. */
GDR_API size_t gdr_fwd_workspace_size(const gdr_shape *shape, const gdr_opts *opts);
GDR_API size_t gdr_bwd_workspace_size(const gdr_shape *shape, const gdr_opts *opts);

/*
 * Forward.  Inputs: q, k, v (same dtype, GDR_BF16 or GDR_F32), g, beta (fp32),
 * scale, h0 (nullable: zero initial state).  Outputs: o (GDR_BF16 or GDR_F32,
 * independent of the input dtype), final_state (nullable), A (nullable; needed
 * later by gdr_bwd), h (nullable).  `workspace` must be 256-byte aligned and
 * hold gdr_fwd_workspace_size() bytes.
 */
GDR_API int gdr_fwd(const gdr_shape *shape, gdr_buf q, gdr_buf k, gdr_buf v, const float *g,
            const float *beta, float scale, const float *h0, gdr_buf o, float *final_state,
            float *A, float *h, void *workspace, size_t workspace_bytes, const gdr_opts *opts,
            void *stream);

/*
 * Backward of gdr_fwd's (o, final_state) with respect to (q, k, v, beta, g, h0).
 * Inputs: the forward's inputs, A as written by gdr_fwd, do (dtype of q),
 * dht (nullable: zero gradient of final_state), h0 (nullable).  Outputs:
 * dq, dk, dv (dtype of q), dbeta, dg (fp32), dh0 (nullable).
 * dbeta is the gradient with respect to beta as passed; dg with respect to
 * the raw per-token log-gate g.
 */
GDR_API int gdr_bwd(const gdr_shape *shape, gdr_buf q, gdr_buf k, gdr_buf v, const float *g,
            const float *beta, const float *A, gdr_buf do_, const float *dht, float scale,
            const float *h0, gdr_buf dq, gdr_buf dk, gdr_buf dv, float *dbeta, float *dg,
            float *dh0, void *workspace, size_t workspace_bytes, const gdr_opts *opts,
            void *stream);

/*
 * gdr_fwd without a workspace, for callers that cannot allocate device memory
 * (a plugin inside a host program that owns all device memory and offers no
 * allocator, or a path that must not call cudaMalloc because it may
 * synchronise the device).  The pages have no counterpart; this is a library
 * convenience.  Arguments and results are those of gdr_fwd, minus the
 * workspace: the call uses a fixed 64 MiB array compiled into the library,
 * which every GPU that loads the library keeps until the process exits.
 * Problems whose forward workspace, for the plan of the inputs' own dtype,
 * exceeds 64 MiB are rejected with GDR_ERR_WORKSPACE before anything is
 * launched; invalid arguments get gdr_fwd's error codes.  The first call on
 * each device looks the array's device address up (cudaGetSymbolAddress) and
 * keeps it for the life of the process; make that first call before any
 * stream capture, and make no call on a device after a cudaDeviceReset() of
 * it (the kept address is then stale).  All calls share the one array: calls
 * whose work overlaps on the GPU (different streams, or another thread) race
 * and corrupt each other's results, so serialise them.  Nothing carried over
 * from an earlier call is read.  The call itself allocates nothing.
 */
GDR_API int gdr_fwd_noalloc(const gdr_shape *shape, gdr_buf q, gdr_buf k, gdr_buf v, const float *g,
                            const float *beta, float scale, const float *h0, gdr_buf o, float *final_state,
                            float *A, float *h, const gdr_opts *opts, void *stream);

/*
 * Layer operators around a recurrent mixer
 * ----------------------------------------
 * What a layer runs before and after its token mixer, mixers with a diagonal
 * transition, and the delta rule for one token: the short causal convolution,
 * the selective state space scan, the gated linear recurrence, the
 * root-mean-square norm of a residual stream (in 8 bits with scales, or in the
 * input's type), the norm after a block with its gate and the stream, and the
 * product of 8-bit activations with 8-bit weights.  Ownership, execution and errors are as above.  Element
 * types: `dtype` is GDR_BF16 or GDR_F32 for the activations of a call;
 * parameters, recurrent states and their gradients are fp32 throughout.
 * Activations are [B, T, ...] with a contiguous innermost part and free
 * strides (in elements) between tokens (`*_row`) and batch rows (`*_batch`),
 * so that slices of one projection's output are read in place; what a call
 * writes is contiguous.  Packed sequences: `cu_seqlens` (device, int32,
 * [n_seqs + 1], rising from 0 to T) with B = 1, else null and n_seqs = B
 * sequences of T tokens.  No host copy of the bounds is needed: a call whose
 * bounds do not rise from 0 to T reads and writes nothing outside its
 * tensors, its results are unspecified, and gdr_check_status reports
 * GDR_ERR_DEVICE.
 */

/* Short causal convolution along the tokens, depthwise:
 *     pre_t = bias + sum_j weight[:, j] x_{t - W + 1 + j},   y_t = silu(pre_t) (or pre_t),
 * where the inputs before a sequence are its initial state (zeros when null).
 * State: the last W - 1 inputs of a sequence, oldest first, in `dtype`. */
typedef struct {
    const void *x;              /* [B, T, D], x_row, x_batch */
    const float *weight, *bias; /* [D, W], [D] (nullable) */
    const void *h0;             /* [n_seqs, W - 1, D], nullable */
    const int32_t *cu_seqlens;
    long long B, T, D, n_seqs, x_row, x_batch;
    int W, dtype, silu;         /* W in {2, 3, 4}; silu: 1 with, 0 without the activation */
    void *y;                    /* [B, T, D] (forward) */
    void *ht;                   /* [n_seqs, W - 1, D], nullable (forward) */
    /* backward: gradients of y (contiguous), of ht (nullable); of x, weight, bias, h0 (the last two nullable) */
    const void *dy, *dht;
    void *dx;
    float *dweight, *dbias;
    void *dh0;
    void *workspace;            /* gdr_conv_bwd_workspace_size bytes, 16-byte aligned */
    size_t workspace_bytes;
} gdr_conv_args;
GDR_API int gdr_conv_fwd(const gdr_conv_args *args, void *stream);
GDR_API size_t gdr_conv_bwd_workspace_size(long long B, long long T, long long D, int W);
GDR_API int gdr_conv_bwd(const gdr_conv_args *args, void *stream);

/* One token for each of `rows` sequences.  Row r uses and updates state slot
 * slots[r] (null: slot r).  A negative slot marks an idle row: its y is zero
 * and no state changes.  A slot past n_slots is treated the same and reported
 * by gdr_check_status (GDR_ERR_DEVICE).  A slot may appear once. */
typedef struct {
    const void *x;              /* [rows, D], x_row */
    const float *weight, *bias;
    void *state;                /* [n_slots, W - 1, D] */
    const int32_t *slots;       /* [rows], nullable */
    long long rows, D, n_slots, x_row;
    int W, dtype, silu;
    void *y;                    /* [rows, D] */
} gdr_conv_step_args;
GDR_API int gdr_conv_step(const gdr_conv_step_args *args, void *stream);

/* Selective state space scan.  For every sequence and channel d of group
 * g = d / (D / G), with s_t = softplus(dt_t + dt_bias) (or dt_t + dt_bias):
 *     h_t = e^{s_t A} h_{t-1} + s_t x_t B_t,   u_t = C_t . h_t + skip x_t,   y_t = u_t silu(z_t) (or u_t).
 * `states` (nullable) keeps h before every GDR_SSM_STRIDE-th token of every
 * batch row for the backward.  A, h0, ht, states, dht and dh0 are 16-byte
 * aligned. */
#define GDR_SSM_STRIDE 16
typedef struct {
    const void *x, *dt, *z;     /* [B, T, D]; z nullable */
    const void *Bm, *Cm;        /* [B, T, G, N], G and N contiguous */
    const float *A, *skip, *dt_bias; /* [D, N], [D] (nullable), [D] (nullable) */
    const float *h0;            /* [n_seqs, D, N], nullable */
    const int32_t *cu_seqlens;
    long long B, T, D, G, n_seqs;
    long long x_row, x_batch, dt_row, dt_batch, z_row, z_batch, b_row, b_batch, c_row, c_batch;
    int N, dtype, softplus;     /* N in {8, 16, 32, 64}; softplus: 1 with, 0 without */
    void *y;                    /* [B, T, D] (forward) */
    float *ht;                  /* [n_seqs, D, N], nullable (forward) */
    float *states;              /* [B, ceil(T / 16), D, N]: written by the forward, read by the backward */
    /* backward */
    const void *dy;             /* [B, T, D] contiguous */
    const float *dht;           /* nullable */
    void *dx, *ddt, *dz;        /* [B, T, D]; dz iff z */
    void *dB, *dC;              /* [B, T, G, N] */
    float *dA, *dskip, *ddt_bias; /* dskip iff skip, ddt_bias iff dt_bias */
    float *dh0;                 /* nullable */
    /* gdr_ssm_*_workspace_size bytes, 16-byte aligned (may be null when 0).  The backward's holds each channel
     * tile's part of dB and dC, 8 N bytes a token for every 512 / N channels of a group: at D = 4096 and one group
     * 16 KiB a token for N = 16, 256 KiB for N = 64. */
    void *workspace;
    size_t workspace_bytes;
} gdr_ssm_args;
GDR_API size_t gdr_ssm_fwd_workspace_size(const gdr_ssm_args *args);
GDR_API int gdr_ssm_fwd(const gdr_ssm_args *args, void *stream);
GDR_API size_t gdr_ssm_bwd_workspace_size(const gdr_ssm_args *args);
GDR_API int gdr_ssm_bwd(const gdr_ssm_args *args, void *stream);

/* One token for each of `rows` sequences; slots as in gdr_conv_step.  A and
 * state are 16-byte aligned. */
typedef struct {
    const void *x, *dt, *z;     /* [rows, D]; z nullable */
    const void *Bm, *Cm;        /* [rows, G, N] */
    const float *A, *skip, *dt_bias;
    float *state;               /* [n_slots, D, N] */
    const int32_t *slots;
    long long rows, D, G, n_slots, x_row, dt_row, z_row, b_row, c_row;
    int N, dtype, softplus;
    void *y;                    /* [rows, D] */
} gdr_ssm_step_args;
GDR_API int gdr_ssm_step(const gdr_ssm_step_args *args, void *stream);

/* Gated linear recurrence, one state a channel.  For every sequence and
 * channel, with s = decay_scale softplus(decay):
 *     a_t = e^{-s sigmoid(decay_gate_t)},
 *     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(input_gate_t) x_t,   y_t = h_t silu(z_t) (or h_t).
 * `states` (nullable) keeps h before every 48th token of every batch row for
 * the backward. */
#define GDR_LINEAR_STRIDE 48
typedef struct {
    const void *x, *input_gate, *decay_gate, *z; /* [B, T, D]; z nullable */
    const float *decay;         /* [D] */
    const float *h0;            /* [n_seqs, D], nullable */
    const int32_t *cu_seqlens;
    long long B, T, D, n_seqs;
    long long x_row, x_batch, i_row, i_batch, r_row, r_batch, z_row, z_batch; /* i: input_gate, r: decay_gate */
    float decay_scale;          /* positive */
    int dtype;
    void *y;                    /* [B, T, D] (forward) */
    float *ht;                  /* [n_seqs, D], nullable (forward) */
    float *states;              /* [B, ceil(T / 48), D]: written by the forward, read by the backward */
    /* backward */
    const void *dy;             /* [B, T, D] contiguous */
    const float *dht;           /* nullable */
    void *dx, *di, *dr, *dz;    /* [B, T, D]: of x, input_gate, decay_gate, z; dz iff z */
    float *ddecay;
    float *dh0;                 /* nullable */
    void *workspace;            /* gdr_linear_*_workspace_size bytes, 16-byte aligned (may be null when 0) */
    size_t workspace_bytes;
} gdr_linear_args;
GDR_API size_t gdr_linear_fwd_workspace_size(long long B, long long T, long long D);
GDR_API int gdr_linear_fwd(const gdr_linear_args *args, void *stream);
GDR_API size_t gdr_linear_bwd_workspace_size(long long B, long long T, long long D);
GDR_API int gdr_linear_bwd(const gdr_linear_args *args, void *stream);

/* One token for each of `rows` sequences; slots as in gdr_conv_step. */
typedef struct {
    const void *x, *input_gate, *decay_gate, *z; /* [rows, D]; z nullable */
    const float *decay;
    float *state;               /* [n_slots, D] */
    const int32_t *slots;
    long long rows, D, n_slots, x_row, i_row, r_row, z_row;
    float decay_scale;
    int dtype;
    void *y;                    /* [rows, D] */
} gdr_linear_step_args;
GDR_API int gdr_linear_step(const gdr_linear_step_args *args, void *stream);

/* One token for each of `rows` sequences through the gated delta rule (gdr_fwd's
 * recurrence and state), with h the state of a row's slot and qk-head
 * hq = hv / (Hv / Hq):
 *     h <- e^g h,   w = beta (v - h^T k),   h <- h + k w^T,   o = scale h^T q.
 * K in {64, 128, 192}, V in {64, 128, 192, 256}; slots as in gdr_conv_step.
 * state is 16-byte aligned. */
typedef struct {
    const void *q, *k, *v;      /* [rows, Hq, K] twice, [rows, Hv, V]; heads contiguous */
    const float *g, *beta;      /* [rows, Hv] */
    float *state;               /* [n_slots, Hv, K, V] */
    const int32_t *slots;       /* [rows], nullable */
    long long rows, Hq, Hv, n_slots, q_row, k_row, v_row;
    int K, V;
    float scale;
    int dtype;
    void *o;                    /* [rows, Hv, V] */
} gdr_delta_step_args;
GDR_API int gdr_delta_step(const gdr_delta_step_args *args, void *stream);

/* Root-mean-square norm of a residual stream:
 *     r = x + residual (rounded to `dtype`; r = x when residual is null),
 *     y = r rsqrt(mean(r^2) + eps) weight.
 * Output y in `dtype`, or (q not null) in 8 bits (e4m3): for each row and
 * block of 128 channels scale = max(max|y|, 1e-30) / 448 and q = y / scale,
 * y not rounded in between.  Scales lie block by block, [ceil(D / 128), M], the
 * order in which gdr_fp8_matmul reads them. */
typedef struct {
    const void *x, *residual;   /* [M, D], x_row, r_row; residual nullable */
    const float *weight;        /* [D] */
    long long M, D, x_row, r_row;
    float eps;
    int dtype;
    void *sum;                  /* [M, D] r; iff residual */
    void *y;                    /* [M, D], or null with q */
    void *q;                    /* [M, D] e4m3, or null with y */
    float *scales;              /* iff q */
} gdr_norm_args;
GDR_API int gdr_norm_fwd(const gdr_norm_args *args, void *stream);

/* Its gradient: dr (the gradient of x and of residual alike) from dy and dsum
 * (nullable), and dweight.  All [M, D] contiguous; `r` is the forward's sum
 * (or x). */
typedef struct {
    const void *r, *dy, *dsum;
    const float *weight;
    long long M, D;
    float eps;
    int dtype;
    void *dr;
    float *dweight;
    void *workspace;            /* gdr_norm_bwd_workspace_size bytes, 16-byte aligned */
    size_t workspace_bytes;
} gdr_norm_bwd_args;
GDR_API size_t gdr_norm_bwd_workspace_size(long long M, long long D);
GDR_API int gdr_norm_bwd(const gdr_norm_bwd_args *args, void *stream);

/* The norm after a block, with the block's gate, the residual stream and the
 * norm before the next block, each but the first optional:
 *     u = x rsqrt(mean(x^2) + eps) weight silu(gate),
 *     r = residual + scale u   (scale u without residual),
 *     y = r rsqrt(mean(r^2) + eps) next_weight   (r before it is rounded to `dtype`).
 * `stats` (nullable) keeps the two reciprocal roots of every row for the backward. */
typedef struct {
    /* [M, D]; gate and residual nullable.  Row m lies at (m / inner) *_outer + (m % inner) *_row: `inner` heads of a
     * token, each a row (1: rows *_outer apart). */
    const void *x, *gate, *residual;
    const float *weight, *next_weight; /* [D]; next_weight nullable */
    long long M, D, inner, x_row, x_outer, gate_row, gate_outer, residual_row, residual_outer;
    float scale, eps;
    int dtype;
    void *r;                    /* [M, D] */
    void *y;                    /* [M, D]; iff next_weight */
    float *stats;               /* [M, 2]: written by the forward, read by the backward */
    /* backward: gradients of r (nullable) and y (nullable); of x, gate, residual, weight, next_weight.  Without
     * next_weight the gradient of residual is that of r, and dresidual is null. */
    const void *dr, *dy;        /* [M, D] contiguous */
    void *dx, *dgate, *dresidual; /* dgate iff gate; dresidual iff residual and next_weight */
    float *dweight, *dnext_weight; /* dnext_weight iff next_weight */
    void *workspace;            /* gdr_block_norm_bwd_workspace_size bytes, 16-byte aligned */
    size_t workspace_bytes;
} gdr_block_norm_args;
GDR_API int gdr_block_norm_fwd(const gdr_block_norm_args *args, void *stream);
GDR_API size_t gdr_block_norm_bwd_workspace_size(long long M, long long D);
GDR_API int gdr_block_norm_bwd(const gdr_block_norm_args *args, void *stream);

/* out[m, n] = sum_kb a_scales[kb, m] b_scales[n / 128, kb] sum_{k in block kb} a[m, k] b[n, k]:
 * e4m3 operands, blocks of 128 along k (the last may be short), sums in fp32.
 * N at least 1, K a positive multiple of 16; a, b and out 16-byte aligned. */
typedef struct {
    const void *a, *b;          /* [M, K], [N, K] e4m3 */
    const float *a_scales, *b_scales; /* [ceil(K / 128), M], [ceil(N / 128), ceil(K / 128)] */
    long long M, N, K;
    int out_dtype;              /* GDR_BF16 or GDR_F32 */
    void *out;                  /* [M, N] */
} gdr_fp8_args;
GDR_API int gdr_fp8_matmul(const gdr_fp8_args *args, void *stream);

/* Synchronises `stream`, then reads and clears the device status word:
 * GDR_OK, GDR_ERR_TIMEOUT, GDR_ERR_DEVICE, or GDR_ERR_CUDA. */
GDR_API int gdr_check_status(void *stream);

/* Message of the calling thread's last failure ("" if none). */
GDR_API const char *gdr_last_error(void);

/* Library version, e.g. "gdr 0.1.0 sm_103a". */
GDR_API const char *gdr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */
