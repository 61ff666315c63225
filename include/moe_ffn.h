/*
 * moe_ffn.h - C ABI of the GB300 (sm_103a) DeepSeek-V4 routed-MoE FFN block with
 * hyper-connections.
 *
 * The block is the FFN sublayer of docs.rs "hf2q 0.1.3 src/inference/models/deepseek4/
 * ffn_forward.rs", function forward_ffn_rows: for `rows` tokens of one layer it maps the
 * hyper-connection state f32 [rows, hc, hidden] to a new state of the same shape through
 *   hc prelude   rms_norm_no_scale_f32 -> raw_matmul "HC FFN function" -> hc_split_sinkhorn
 *                -> hc_pre -> rms_norm (ffn_norm)
 *   router       raw_matmul "MoE gate" -> score route (layer >= hash_layer_count) or hash
 *                route (layer < hash_layer_count) -> sanitize indices
 *   experts      routed + shared gate/up projections -> SwiGLU -> down projections
 *                -> weighted reduce (routed slots weighted, shared added)
 *   hc post      hc_post (post * ffn_output + comb * state)
 * Every stage runs in this library's CUDA kernels; there is no host or CPU fallback.
 *
 * Conventions where the page leaves the arithmetic open (each fixed here, not by the page):
 *   - mixes split as [pre (hc) | post (hc) | comb (hc*hc, row-major i*hc+j)]; segment s is
 *     multiplied by hc_scale[s] and then hc_base is added; pre = sigmoid, post = 2*sigmoid;
 *     comb = Sinkhorn(exp(a - rowmax)), `sinkhorn_iters` sweeps of row then column
 *     normalisation, no epsilon;
 *   - hc_post: out[i] = post[i] * ffn_output + sum_j comb[i][j] * state[j];
 *   - score route: s = sigmoid(logit); top_k experts by s + exp_probs_b, slots in descending
 *     order of that value, exact ties to the lower expert index; weights s / sum(s) over the
 *     chosen experts (no extra scaling factor);
 *   - hash route: experts = tid2eid[token] in table order; weights sigmoid(logit) normalised
 *     over the slots whose expert is valid;
 *   - sanitize: an index outside [0, experts) is replaced by 0 for the projections, and the
 *     weighted reduce gives that slot no weight;
 *   - SwiGLU: silu(gate) * up, no clamp, no bias.
 *
 * Memory: all tensor arguments are DEVICE pointers owned by the caller, row-major and
 * contiguous.  bf16 arguments are passed as uint16_t bit patterns.
 */
#ifndef MOE_FFN_H
#define MOE_FFN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes (negative = error, the call did nothing on the device). */
#define MOE_FFN_OK 0
#define MOE_FFN_ERR_NULL_PTR (-1)          /* a required pointer is NULL */
#define MOE_FFN_ERR_BAD_CONFIG (-2)        /* config outside the supported shapes (see below) */
#define MOE_FFN_ERR_LAYER_RANGE (-3)       /* layer >= n_layers (the page's first guard) */
#define MOE_FFN_ERR_ROWS_ZERO (-4)         /* rows == 0 ("requires at least one token row") */
#define MOE_FFN_ERR_ROWS_RANGE (-5)        /* rows < 0, rows > max_rows, or rows*top_k overflows */
#define MOE_FFN_ERR_NO_ROUTING_SOURCE (-6) /* score layer without exp_probs_b, hash layer without tid2eid */
#define MOE_FFN_ERR_ALIAS (-7)             /* out_state overlaps state */
#define MOE_FFN_ERR_CUDA (-8)              /* a CUDA runtime/driver call failed; see moe_ffn_last_error */
#define MOE_FFN_ERR_NO_MEMORY (-9)         /* device or host allocation failed */
#define MOE_FFN_ERR_UNSUPPORTED (-10)      /* no sm_103 device */
#define MOE_FFN_ERR_ALIGNMENT (-11)        /* a pointer is not 16-byte aligned */
#define MOE_FFN_ERR_NO_WEIGHTS (-12)       /* forward on a layer whose weights were not given */

/* Device-side status bits (moe_ffn_status returns their OR since the previous call). */
#define MOE_FFN_DEV_TOKEN_RANGE 0x1   /* hash layer: token id outside [0, vocab); its slots masked */
#define MOE_FFN_DEV_ROUTE_RANGE 0x2   /* a routed expert index outside [0, experts); slot masked */
#define MOE_FFN_DEV_NONFINITE 0x4     /* a router logit, a SwiGLU output or an expert's output was NaN or infinite */
#define MOE_FFN_DEV_TIMEOUT 0x8       /* a bounded wait inside a kernel gave up (kernel returned) */

/* Shapes and constants of the block (the page's cfg fields).  Supported:
 *   1 <= hc <= 4;  128 <= hidden <= 4096, hidden % 128 == 0;  128 <= inter <= 2048, inter % 128 == 0;  shared_inter == inter;
 *   16 <= experts <= 512, experts % 16 == 0;  1 <= top_k <= 8, top_k <= experts;
 *   hash_layer_count <= n_layers;  1 <= max_rows <= 65536;  vocab >= 1;  sinkhorn_iters >= 0. */
typedef struct moe_ffn_config {
  int32_t hidden;            /* hidden_size (4096) */
  int32_t hc;                /* hyper_connection_count (4) */
  int32_t experts;           /* num_experts (256) */
  int32_t top_k;             /* num_experts_per_tok (6) */
  int32_t inter;             /* expert_intermediate_size (2048) */
  int32_t shared_inter;      /* shared expert intermediate size (= inter) */
  int32_t vocab;             /* vocab_size: token ids must lie in [0, vocab) on hash layers */
  int32_t n_layers;          /* num_hidden_layers */
  int32_t hash_layer_count;  /* layers below this use hash routing */
  int32_t max_rows;          /* largest `rows` a forward will be given; sizes the scratch */
  int32_t sinkhorn_iters;    /* Sinkhorn sweeps (20) */
  float rms_eps;             /* rms_norm_eps (1e-6) */
} moe_ffn_config;

/* Weights of one layer: DEVICE pointers, caller-owned, 16-byte aligned, valid for the life of
 * the handle.  A layer whose pointers are all NULL has no weights; forward on it fails.  The six
 * expert matrices may be NULL together (and only together): the layer's experts then come later
 * in MXFP8 (moe_ffn_set_mxfp8_experts), and a forward before that fails with NO_WEIGHTS. */
typedef struct moe_ffn_layer_weights {
  const uint16_t *hc_fn;       /* bf16 [(2+hc)*hc, hc*hidden]  hc_ffn_fn */
  const float *hc_base;        /* f32 [(2+hc)*hc]              hc_ffn_base */
  const float *hc_scale;       /* f32 [3]                      hc_ffn_scale */
  const float *ffn_norm;       /* f32 [hidden]                 ffn_norm */
  const uint16_t *gate;        /* bf16 [experts, hidden]       ffn_gate_inp (router) */
  const float *exp_probs_b;    /* f32 [experts]; required on score layers, else may be NULL */
  const int32_t *tid2eid;      /* i32 [vocab, top_k]; required on hash layers, else may be NULL */
  const uint16_t *gate_exps;   /* bf16 [experts, inter, hidden] */
  const uint16_t *up_exps;     /* bf16 [experts, inter, hidden] */
  const uint16_t *down_exps;   /* bf16 [experts, hidden, inter] */
  const uint16_t *gate_sh;     /* bf16 [shared_inter, hidden] */
  const uint16_t *up_sh;       /* bf16 [shared_inter, hidden] */
  const uint16_t *down_sh;     /* bf16 [hidden, shared_inter] */
} moe_ffn_layer_weights;

typedef struct moe_ffn_handle moe_ffn_handle;

/* Creates a handle on the current CUDA device.  Validates the config (BAD_CONFIG) and, for every
 * layer with weights, the routing source its layer type needs (NO_ROUTING_SOURCE) and pointer
 * alignment (ALIGNMENT).  Allocates the scratch for max_rows; the weights are read in place (no
 * copies: the tensor-core kernels take the bf16 matrices as they are).  Synchronous.  On failure
 * *out is NULL and nothing stays allocated. */
int moe_ffn_init(const moe_ffn_config *cfg, const moe_ffn_layer_weights *layers, moe_ffn_handle **out);

/* Enqueues the block for `rows` tokens of `layer` on `stream` (a cudaStream_t; NULL = legacy
 * default stream) and returns without waiting.
 *   state      f32 [rows, hc, hidden]  input hyper-connection state (read only)
 *   token_ids  i32 [rows]              token ids (read on hash layers only; may be NULL on score layers)
 *   out_state  f32 [rows, hc, hidden]  output state; must not overlap state
 * Returns MOE_FFN_OK or a negative code from the host-side checks (nothing enqueued then).
 * Rows <= 4 take the weight-streaming decode path; larger batches the tensor-core grouped-GEMM
 * path.  Forwards on one handle share its scratch: enqueue them on one stream (or order them),
 * never concurrently.  Data-dependent problems (a token id out of range, an expert index out of
 * range, a non-finite logit) do not fail the call: they set device status bits, masked slots
 * contribute nothing, and moe_ffn_status reports them. */
int moe_ffn_forward(moe_ffn_handle *h, const float *state, const int32_t *token_ids, int32_t rows,
                    int32_t layer, float *out_state, void *stream);

/* Several layers in one submission: enqueues the blocks of layers first_layer .. first_layer +
 * n_layers - 1 for the same `rows` tokens on `stream`, each taking the state the previous one made:
 * state -> layer first_layer -> ... -> out_state.  A decode step's loop over layers is its unit of
 * submission (docs.rs "hf2q 0.1.10 .../deepseek4/decode_cohort.rs", forward_verifier_decode_cohort:
 * two layers per command buffer, a B=4 step encoded as four rows=1 passes per layer); here each
 * layer is one launch for all rows and the whole chain is one CUDA graph.  The chain runs FFN
 * blocks back to back; the attention sublayer a model puts between them is the caller's (every
 * entry point of this library can be captured into the caller's own graph, which is how a step
 * with attention is batched).
 * The first call for a given (state, token_ids, rows, first_layer, n_layers, out_state) captures
 * the chain into a CUDA graph that the handle owns (the 8 most recently used are kept); later calls
 * with the same arguments launch it, reading whatever the buffers then hold.  The intermediate
 * states live in a handle-owned f32 [max_rows, hc, hidden] buffer, allocated by the first call with
 * n_layers > 1.  So make the first call of each argument set outside any stream capture, and not
 * while another thread captures in global mode.  Per-kernel stage timing does not apply.
 * Returns the codes of moe_ffn_forward, checked for every layer of the chain (LAYER_RANGE also when
 * n_layers < 1 or the chain passes the last layer), NO_MEMORY or CUDA; nothing is enqueued on an
 * error. */
int moe_ffn_forward_layers(moe_ffn_handle *h, const float *state, const int32_t *token_ids, int32_t rows,
                           int32_t first_layer, int32_t n_layers, float *out_state, void *stream);

/* The same block on HOST buffers: copies state [rows, hc, hidden] and token_ids [rows] (may be NULL
 * on score layers) from host memory into library-owned device buffers, runs moe_ffn_forward on
 * `stream`, copies the new state back into out_state (host), and waits for the stream.  Pinned
 * (page-locked) host memory gives the fastest copies.  Same return codes as moe_ffn_forward, plus
 * MOE_FFN_ERR_CUDA when a copy fails. */
int moe_ffn_forward_host(moe_ffn_handle *h, const float *state, const int32_t *token_ids, int32_t rows,
                         int32_t layer, float *out_state, void *stream);

/* Waits for the stream of the last forward and returns the OR of device status bits set since the
 * previous moe_ffn_status call (>= 0, then cleared), or MOE_FFN_ERR_CUDA. */
int moe_ffn_status(moe_ffn_handle *h);

/* Copies to host memory an intermediate of the last forward (after waiting for it), for stage-by-
 * stage checks.  `which` selects the buffer; `bytes` must equal its size for the last `rows`:
 *   0 pre f32 [rows, hc]      1 post f32 [rows, hc]      2 comb f32 [rows, hc, hc]
 *   3 ffn_norm f32 [rows, hidden]   4 logits f32 [rows, experts]
 *   5 indices i32 [rows, top_k]     6 route weights f32 [rows, top_k]
 *   7 safe indices u32 [rows, top_k] 8 ffn_output f32 [rows, hidden]
 * Returns MOE_FFN_OK, MOE_FFN_ERR_BAD_CONFIG for an unknown `which` or a size mismatch, or
 * MOE_FFN_ERR_CUDA. */
int moe_ffn_debug_copy(moe_ffn_handle *h, int32_t which, void *host_dst, size_t bytes);

/* Per-kernel timing (off by default).  While enabled, each forward records a CUDA event on its
 * stream before its first kernel and after every kernel; this adds a few microseconds per forward. */
int moe_ffn_set_stage_timing(moe_ffn_handle *h, int32_t enable);

/* After a forward made with stage timing on: waits for it and writes the duration (ms) of each of
 * its kernels, in launch order, to ms[i] and the kernel's name (a static string) to names[i] (names
 * may be NULL).  Returns the number of kernels written (at most max_stages), 0 when nothing was
 * timed, or a negative code. */
int moe_ffn_stage_times(moe_ffn_handle *h, float *ms, const char **names, int32_t max_stages);

/* Allocation-free HC split: the first stage of the block (HC RMSNorm, mix GEMV with hc_fn, split
 * into pre/post and the Sinkhorn comb, the same kernel and conventions as moe_ffn_forward) for
 * callers that cannot allocate device memory at call time: serving or real-time loops that forbid
 * allocation after start-up (cudaMalloc may synchronise the device), or hosts whose memory pool
 * owns the whole GPU, where cudaMalloc fails.  The pages have no counterpart of this entry point;
 * it exists for such callers.
 *   state    f32 [rows, hc, hidden] (device, 16-byte aligned)    hc_fn bf16 [(2+hc)*hc, hc*hidden]
 *   hc_scale f32 [3], hc_base f32 [(2+hc)*hc]                    (device)
 *   pre, post f32 [rows, hc]; comb f32 [rows, hc, hc]            (device outputs)
 * No handle and no allocation: the scratch is a fixed 1 MiB array inside the library (held by every
 * GPU that loads the library until exit), shared by all calls; each call clears the part that
 * must start at zero (one cudaMemsetAsync on the array) before its kernel.  Limits: 1 <= rows <=
 * 4096 and rows * (partial sums of the chosen split) must fit the 1 MiB; larger inputs return
 * MOE_FFN_ERR_ROWS_RANGE with a message in moe_ffn_last_error(NULL).  The first call on each device
 * looks the array's address up (and may load the module onto that device): make it before any
 * stream capture.  Calls whose kernels overlap on the GPU race on the shared scratch: order them on
 * one stream.  Returns MOE_FFN_OK or a negative code.  A CUDA error already pending from earlier
 * work is reported as MOE_FFN_ERR_CUDA before anything is enqueued; every other negative code
 * except a failed kernel launch also means nothing was enqueued (a failed launch comes after the
 * memset). */
int moe_ffn_hc_split_noalloc(const float *state, const uint16_t *hc_fn, const float *hc_scale,
                             const float *hc_base, int32_t rows, int32_t hc, int32_t hidden,
                             int32_t sinkhorn_iters, float rms_eps, float *pre, float *post, float *comb,
                             void *stream);

/* ---- The hyper-connection prelude and post of a sublayer ------------------------------------
 * Every sublayer of a layer wraps its body in the same hyper-connection stages: the attention
 * sublayer (docs.rs "hf2q 0.1.3 src/inference/models/deepseek4/attention_forward.rs", with the "HC
 * attention function" and attn_norm) as the FFN sublayer (ffn_forward.rs, with the "HC FFN
 * function" and ffn_norm).  Before the body: RMSNorm of the flattened state (no weight), the mix
 * GEMV with the sublayer's hc_fn, split + Sinkhorn into pre/post/comb (the conventions above),
 * hc_pre (x = sum_h pre[h] * state[h]) and the sublayer's RMSNorm of x.  After the body: hc_post
 * folds the body's output f back into the state.  The FFN sublayer's HC weights come with
 * moe_ffn_init; the attention sublayer's are registered with moe_ffn_set_attn_hc. */
#define MOE_FFN_SUBLAYER_ATTN 0
#define MOE_FFN_SUBLAYER_FFN 1

/* HC weights of one sublayer: DEVICE pointers, caller-owned, 16-byte aligned. */
typedef struct moe_ffn_hc_weights {
  const uint16_t *hc_fn;   /* bf16 [(2+hc)*hc, hc*hidden]  hc_attn_fn */
  const float *hc_base;    /* f32 [(2+hc)*hc]              hc_attn_base */
  const float *hc_scale;   /* f32 [3]                      hc_attn_scale */
  const float *norm;       /* f32 [hidden]                 attn_norm */
} moe_ffn_hc_weights;

/* Registers the attention sublayer's HC weights for `layer`; they must stay valid for the life of
 * the handle, and a later call for the same layer replaces them (hc_fn is read in place, also by
 * the tensor-core mix of the many-row path).  Synchronous.  Returns MOE_FFN_OK,
 * LAYER_RANGE, NULL_PTR, ALIGNMENT, NO_MEMORY or CUDA. */
int moe_ffn_set_attn_hc(moe_ffn_handle *h, int32_t layer, const moe_ffn_hc_weights *w);

/* Enqueues the HC prelude of `sublayer` (MOE_FFN_SUBLAYER_ATTN or _FFN) of `layer` for `rows`
 * tokens on `stream` and returns without waiting.
 *   state   f32 [rows, hc, hidden]  the state entering the sublayer (read only)
 *   x_norm  f32 [rows, hidden]      out: the body's input, RMSNorm(hc_pre(state, pre)) * norm
 *   pre     f32 [rows, hc]          out; may be NULL
 *   post    f32 [rows, hc]          out, for moe_ffn_hc_post
 *   comb    f32 [rows, hc, hc]      out, for moe_ffn_hc_post (row-major i*hc + j)
 * state and x_norm must be 16-byte aligned; no output may overlap state.  Uses the handle's scratch
 * like moe_ffn_forward (order the calls on one stream).  Returns MOE_FFN_OK, LAYER_RANGE, ROWS_ZERO,
 * ROWS_RANGE, NULL_PTR, ALIGNMENT, ALIAS, BAD_CONFIG (unknown sublayer), NO_WEIGHTS (the sublayer's
 * HC weights are not there) or CUDA; nothing is enqueued on an error. */
int moe_ffn_hc_pre(moe_ffn_handle *h, int32_t layer, int32_t sublayer, const float *state, int32_t rows,
                   float *x_norm, float *pre, float *post, float *comb, void *stream);

/* Enqueues hc_post: out_state[r, i, d] = post[r, i] * f[r, d] + sum_j comb[r, i, j] * state[r, j, d].
 *   f          f32 [rows, hidden]      the sublayer body's output
 *   state      f32 [rows, hc, hidden]  the state given to moe_ffn_hc_pre
 *   post, comb f32 [rows, hc], [rows, hc, hc] from moe_ffn_hc_pre
 *   out_state  f32 [rows, hc, hidden]  must not overlap any input
 * f, state and out_state must be 16-byte aligned.  Needs no scratch.  Returns MOE_FFN_OK,
 * ROWS_ZERO, ROWS_RANGE, NULL_PTR, ALIGNMENT, ALIAS or CUDA. */
int moe_ffn_hc_post(moe_ffn_handle *h, const float *f, const float *state, const float *post, const float *comb,
                    int32_t rows, float *out_state, void *stream);

/* ---- Quantised expert weights -----------------------------------------------------------------
 * The page consumes the expert matrices as raw GGUF types without naming a format; the quantised
 * mode here reads them as MXFP8 (OCP Microscaling): E4M3 codes (1 sign, 4 exponent bits with bias
 * 7, 3 mantissa bits; no infinities) in the bf16 matrices' layouts, and one E8M0 scale (2^(s-127))
 * per 32 consecutive elements of a row, so element k of a row is value(code) * 2^(scale[k/32] - 127).
 * The rest of the block is unchanged.  Rows <= 4 stream the codes and scales (about half the bytes
 * of bf16).  At four rows the decode kernel turns each tile into exact f16 weights in tensor memory
 * for the tensor cores (the batch rows go in as three f16 planes: values of magnitude 2^32 and
 * above come out infinite); that needs every scale of the layer within 22 binades of its largest
 * and no NaN code or scale, and a layer outside that, or one to three rows, decodes on the
 * CUDA-core kernel instead.  Larger batches run the tensor-core path on a bf16 expansion made at
 * registration, exact wherever code x scale is a normal bf16. */
typedef struct moe_ffn_mxfp8_experts {
  const uint8_t *gate_exps, *gate_exps_scale;  /* E4M3 [experts, inter, hidden], E8M0 [experts, inter, hidden/32] */
  const uint8_t *up_exps, *up_exps_scale;      /* the same layouts */
  const uint8_t *down_exps, *down_exps_scale;  /* E4M3 [experts, hidden, inter], E8M0 [experts, hidden, inter/32] */
  const uint8_t *gate_sh, *gate_sh_scale;      /* E4M3 [shared_inter, hidden], E8M0 [shared_inter, hidden/32] */
  const uint8_t *up_sh, *up_sh_scale;          /* the same layouts */
  const uint8_t *down_sh, *down_sh_scale;      /* E4M3 [hidden, shared_inter], E8M0 [hidden, shared_inter/32] */
} moe_ffn_mxfp8_experts;

/* Makes `layer` run on these MXFP8 experts (DEVICE pointers, caller-owned, 16-byte aligned, valid
 * for the life of the handle), in place of any bf16 experts given at init; a later call replaces
 * them.  The layer must have its other weights from moe_ffn_init.  Reads every code and scale once
 * on the device (NaN codes, the range of the scales).  On a handle with max_rows > 4 this also fills the bf16 expansion the
 * tensor-core path reads (allocating it on first use).  Synchronous.  Returns MOE_FFN_OK, LAYER_RANGE, NO_WEIGHTS, NULL_PTR, ALIGNMENT, NO_MEMORY or CUDA. */
int moe_ffn_set_mxfp8_experts(moe_ffn_handle *h, int32_t layer, const moe_ffn_mxfp8_experts *w);

/* Test hook: failure detection without a GPU fault.  Every wait inside the kernels is bounded; on
 * expiry a kernel sets MOE_FFN_DEV_TIMEOUT, stops its work, waits (bounded) for its own copies and
 * tensor-core operations in flight, frees its tensor memory and returns, leaving the handle usable.
 * This call makes one such wait run out on purpose, on the handle's later forwards:
 *   which = MOE_FFN_INJECT_DECODE_WAIT: rows <= 4, the decode kernel's final phase first waits for
 *           a count that nothing reaches;
 *   which = MOE_FFN_INJECT_GEMM_WAIT:   rows > 4, CTA 0 of the gate/up GEMM first waits on an
 *           mbarrier that nothing arrives at;
 *   which = MOE_FFN_INJECT_NONE:        no injected wait (the default).
 * wait_limit_us bounds every in-kernel wait of those forwards (0: the kernels' defaults, 1-2 s).
 * Outputs of a forward with an injected wait are not meaningful; its status carries the timeout bit.
 * Returns MOE_FFN_OK, NULL_PTR or BAD_CONFIG.  Nothing in the pages corresponds to it. */
#define MOE_FFN_INJECT_NONE 0
#define MOE_FFN_INJECT_DECODE_WAIT 1
#define MOE_FFN_INJECT_GEMM_WAIT 2
int moe_ffn_set_fault_injection(moe_ffn_handle *h, int32_t which, uint32_t wait_limit_us);

/* ---- The dense feed-forward sublayer on a plain residual stream --------------------------------
 * The same sublayer without hyper-connections and without routing: a dense layer, a shared expert
 * on its own, a draft head's layer.  These entry points take no handle.  Tensor arguments are
 * device pointers of the current device, rows contiguous, consecutive rows `ld_*` elements apart
 * (ld >= the row's length; column ranges of one tensor do not overlap).  Calls enqueue on `stream` and return without waiting; each call that
 * needs scratch takes it as `workspace`, which must not be in use by another call meanwhile (give
 * graphs that may run together workspaces of their own).  They can be captured into CUDA graphs.
 * All sums are in f32 and no atomics are used: the same call gives the same bits.  On an error
 * nothing is enqueued, except that a failed launch may leave earlier kernels of the call enqueued;
 * the message is moe_ffn_last_error(NULL) on the calling thread.  A failure that CUDA recovers from
 * (a capture that became invalid, memory for a kernel's code) is reported by this call only. */
#define MOE_FFN_F32 0
#define MOE_FFN_BF16 1
#define MOE_FFN_F16 2

#define MOE_FFN_GATE_NONE 0
#define MOE_FFN_GATE_VECTOR 1 /* [ceil(rows / rows_per_gate), hidden], contiguous: one vector for each rows_per_gate rows */
#define MOE_FFN_GATE_TOKEN 2  /* [rows]: one value for each row */

/* The norms before and after a block, fused with its gate and residual scale:
 *   n = f * rsqrt(mean(f^2) + eps) * norm_f      (n = f when norm_f is NULL)
 *   out = state + residual_scale * gate * n      (rounded to stream_type as it is stored)
 *   y = out * rsqrt(mean(out^2) + eps) * norm_next
 * With f NULL there is no block before: y is the norm of state, out is not written. */
typedef struct moe_ffn_block_norm_args {
  int32_t rows, hidden;         /* 1 <= hidden <= 8192, rows at most 2^30, rows times any ld at most 2^60 */
  int32_t stream_type;          /* type of state and out: MOE_FFN_F32 or block_type */
  int32_t block_type;           /* type of f and y */
  int32_t gate_type;            /* MOE_FFN_F32 or block_type */
  int32_t gate_kind, rows_per_gate;
  float residual_scale, eps;
  const void *state; int64_t ld_state;  /* [rows, hidden] */
  const void *f; int64_t ld_f;          /* [rows, hidden], or NULL */
  const void *gate;
  const float *norm_f, *norm_next;      /* [hidden], either may be NULL; norm_next exactly when y is */
  void *out; int64_t ld_out;            /* may be state itself (same ld); no other overlap */
  void *y; int64_t ld_y;
} moe_ffn_block_norm_args;

/* Returns MOE_FFN_OK, NULL_PTR, ROWS_ZERO, ROWS_RANGE, BAD_CONFIG (hidden, types, gate, ld),
 * ALIGNMENT (a pointer not aligned to its type), ALIAS, UNSUPPORTED or CUDA. */
int moe_ffn_block_norm(const moe_ffn_block_norm_args *a, void *stream);

/* Gradients of block_norm.  `a` holds the call's arguments with `state` the stream AFTER the block
 * (what the forward call wrote to out; with f NULL, its state); a->out and a->y are not read.
 * d_state is the gradient that goes on to the stream before the block. */
typedef struct moe_ffn_block_norm_grads {
  const void *d_out; int64_t ld_d_out;  /* stream_type; NULL: zero */
  const void *d_y; int64_t ld_d_y;      /* block_type; given exactly when norm_next is */
  void *d_state; int64_t ld_d_state;    /* stream_type; may be d_out itself (same ld) */
  void *d_f; int64_t ld_d_f;            /* block_type; given exactly when f is */
  void *d_gate;                         /* gate_type, the gate's layout; may be NULL */
  float *d_norm_f, *d_norm_next;        /* [hidden]; may be NULL */
  void *workspace; size_t workspace_bytes; /* at least moe_ffn_block_norm_workspace, 32-byte aligned */
} moe_ffn_block_norm_grads;

/* The codes of moe_ffn_block_norm, and NO_MEMORY when the workspace is too small. */
int moe_ffn_block_norm_backward(const moe_ffn_block_norm_args *a, const moe_ffn_block_norm_grads *g, void *stream);

/* Bytes of workspace that block_norm_backward needs for these arguments (pointers are only compared
 * with NULL); negative: an error code. */
int64_t moe_ffn_block_norm_workspace(const moe_ffn_block_norm_args *a, const moe_ffn_block_norm_grads *g);

/* The gated feed-forward block:  g = x w_gate^T,  u = x w_up^T,  y = (act(g) * u) w_down^T.
 * Both projections, the activation and the product are one kernel, the down projection another
 * (a few rows: weight-streaming kernels).  Operands are bf16 or f16, sums f32; act(g) * u is
 * rounded to the operand type before the down projection.
 * Backward, from the saved g and u (rounded to the type):  dh = d_y w_down;  dg = dh * u * act'(g);
 *   du = dh * act(g);  d_x = dg w_gate + du w_up;  d_w_gate = dg^T x;  d_w_up = du^T x;
 *   d_w_down = d_y^T (act(g) * u);  dg, du and act(g) * u are rounded to the type as operands. */
#define MOE_FFN_ACT_SILU 0
#define MOE_FFN_ACT_GELU 1 /* 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */

typedef struct moe_ffn_gated_args {
  int32_t rows, hidden, inter;  /* hidden and inter multiples of 8, at most 65536; rows at most 2^24 */
  int32_t type;                 /* MOE_FFN_BF16 or MOE_FFN_F16: every tensor below */
  int32_t activation;
  const void *x; int64_t ld_x;  /* [rows, hidden] */
  const void *w_gate, *w_up;    /* [inter, hidden], contiguous */
  const void *w_down;           /* [hidden, inter], contiguous */
  void *y; int64_t ld_y;        /* forward: [rows, hidden] */
  void *gate, *up;              /* [rows, inter], contiguous: forward writes g and u (or both NULL), backward reads them */
  const void *d_y; int64_t ld_d_y;            /* backward: [rows, hidden] */
  void *d_x; int64_t ld_d_x;                  /* backward: [rows, hidden], or NULL */
  void *d_w_gate, *d_w_up, *d_w_down;         /* backward: the weights' layouts; all three or none */
  void *workspace; size_t workspace_bytes;    /* at least moe_ffn_gated_workspace */
} moe_ffn_gated_args;

/* Every pointer 16-byte aligned, every ld a multiple of 8.  Returns MOE_FFN_OK, NULL_PTR, ROWS_ZERO,
 * ROWS_RANGE, BAD_CONFIG (sizes, type, activation, ld), ALIGNMENT, ALIAS (an output or the workspace
 * overlaps another tensor), NO_MEMORY (workspace too small), UNSUPPORTED or CUDA. */
int moe_ffn_gated_forward(const moe_ffn_gated_args *a, void *stream);
int moe_ffn_gated_backward(const moe_ffn_gated_args *a, void *stream);

/* Bytes of workspace that the forward (backward = 0) or backward call needs; negative: an error code. */
int64_t moe_ffn_gated_workspace(const moe_ffn_gated_args *a, int32_t backward);

/* Matrix product in 8-bit floating point with a scale for each block of 128:
 *   out[i, j] = sum_b a_scale[i, b] * b_scale[j / 128, b] * sum over k in block b of a[i, k] * b[j, k]
 * with blocks of 128 along k, the last of which may be shorter.  Sums are f32; scales may be any f32 values, and
 * their product may leave f32's range where the block's result does not.  (The MXFP8 experts
 * above have a power-of-two scale for each 32 elements instead.) */
#define MOE_FFN_E4M3 0
#define MOE_FFN_E5M2 1

typedef struct moe_ffn_fp8_matmul_args {
  int32_t rows, n, k;            /* k a multiple of 16, at most 2^20; n at most 2^20; rows at most 2^24 */
  int32_t a_type, b_type;        /* MOE_FFN_E4M3 or MOE_FFN_E5M2 */
  int32_t out_type;              /* MOE_FFN_F32, _BF16 or _F16 */
  const void *a; int64_t ld_a;   /* codes [rows, k]; 16-byte aligned, ld a multiple of 16 */
  const float *a_scale;          /* [rows, ceil(k / 128)], contiguous */
  const void *b; int64_t ld_b;   /* codes [n, k]; 16-byte aligned, ld a multiple of 16 */
  const float *b_scale;          /* [ceil(n / 128), ceil(k / 128)], contiguous */
  void *out; int64_t ld_out;     /* [rows, n], any ld >= n; overlaps no input */
} moe_ffn_fp8_matmul_args;

/* Returns MOE_FFN_OK, NULL_PTR, ROWS_ZERO, ROWS_RANGE, BAD_CONFIG, ALIGNMENT, ALIAS, UNSUPPORTED or
 * CUDA. */
int moe_ffn_fp8_matmul(const moe_ffn_fp8_matmul_args *a, void *stream);

/* Makes such an operand: a block is block_rows (1 or 128) rows x 128 columns, those at the ends may be
 * smaller.  scale = (largest magnitude of the block) / (largest finite code: 448 or 57344), 1 for a
 * block of zeros, at least 2^-126; with pow2 rounded up to a power of two.  code = x / scale, the quotient
 * in f32, rounded to nearest even.  (The f32 quotient of a value below 2^-100 may be off by a last place.)
 * A block with a NaN has the scale NaN, one with an infinity the scale infinity, and
 * products with either are not finite. */
typedef struct moe_ffn_fp8_quantise_args {
  int32_t rows, k;               /* k at most 2^20, rows at most 2^24 */
  int32_t type;                  /* of x: MOE_FFN_F32, _BF16 or _F16 */
  int32_t code_type;             /* MOE_FFN_E4M3 or MOE_FFN_E5M2 */
  int32_t block_rows, pow2;
  const void *x; int64_t ld_x;   /* [rows, k] */
  void *codes; int64_t ld_codes; /* [rows, k] */
  float *scales;                 /* [ceil(rows / block_rows), ceil(k / 128)], contiguous */
} moe_ffn_fp8_quantise_args;

/* The codes of moe_ffn_fp8_matmul. */
int moe_ffn_fp8_quantise(const moe_ffn_fp8_quantise_args *a, void *stream);

/* Where block_norm_fp8 and gated_quantise write codes and scales: as fp8_quantise makes them with block_rows 1. */
typedef struct moe_ffn_fp8_out {
  int32_t code_type, pow2;       /* MOE_FFN_E4M3 or MOE_FFN_E5M2 */
  void *codes; int64_t ld_codes; /* [rows, columns] */
  float *scales;                 /* [rows, ceil(columns / 128)], contiguous */
} moe_ffn_fp8_out;

/* block_norm with y as an operand of the FP8 product: the f32 values out * rsqrt(mean(out^2) + eps) * norm_next,
 * quantised without being rounded to block_type first.  norm_next is given and y NULL; block_type is f's type (any
 * with f NULL, which writes no out).  The codes of moe_ffn_block_norm. */
int moe_ffn_block_norm_fp8(const moe_ffn_block_norm_args *a, const moe_ffn_fp8_out *o, void *stream);

/* The gated block's product as an operand of its second FP8 product: act(gate) * up in f32, quantised.
 * gate and up may be column ranges of one tensor, as one product of both projections leaves them. */
typedef struct moe_ffn_gated_quantise_args {
  int32_t rows, columns;         /* columns at most 2^20, rows at most 2^24 */
  int32_t type;                  /* of gate and up: MOE_FFN_BF16 or _F16 */
  int32_t activation;
  const void *gate; int64_t ld_gate;  /* [rows, columns] */
  const void *up; int64_t ld_up;
} moe_ffn_gated_quantise_args;

/* The codes of moe_ffn_fp8_matmul. */
int moe_ffn_gated_quantise(const moe_ffn_gated_quantise_args *a, const moe_ffn_fp8_out *o, void *stream);

/* Weights in 4 bits with a scale for each group of columns:
 *   w[j, k] = (code[j, k] - zero[j, k / group]) * scale[j, k / group]
 * Codes 0..15 lie two to a byte, the even column in the low half.  Without zero points zero is 8. */
typedef struct moe_ffn_int4_weights_args {
  int32_t n, k;                  /* n at most 2^24, k a multiple of 32, at most 2^20 */
  int32_t group;                 /* 32, 64 or 128; the last group of a row may be shorter */
  int32_t scale_type;            /* MOE_FFN_BF16 or _F16 */
  uint8_t *codes;                /* [n, k / 2], contiguous, 16-byte aligned, as the next two */
  void *scales;                  /* [n, ceil(k / group)] */
  uint8_t *zeros;                /* [n, ceil(k / group)], the low four bits of each, or NULL */
} moe_ffn_int4_weights_args;

/* Makes such weights of w [n, k] (type MOE_FFN_F32, _BF16 or _F16; aligned to eight values, ld a multiple of 8).
 * Without zeros: scale = max|w| / 7 of the group, code = 8 + w / scale within 1..15.  With zeros:
 * scale = (max(w, 0) - min(w, 0)) / 15, zero = -min(w, 0) / scale, code = zero + w / scale within 0..15.
 * Quotients are f32, rounded to nearest even; they are by the scale as it is stored, which is 1 for a group of zeros and
 * at least scale_type's smallest normal value.  A group with a NaN or an infinity, or whose scale leaves scale_type, has
 * the scale infinity, and products with it are not finite. */
int moe_ffn_int4_quantise(const moe_ffn_int4_weights_args *a, const void *w, int32_t type, int64_t ld_w, void *stream);

/* The values of such weights, rounded to scale_type: out [n, k], 16-byte aligned, ld a multiple of 8.  For prompts, whose
 * products the 16-bit entry points make. */
int moe_ffn_int4_widen(const moe_ffn_int4_weights_args *a, void *out, int64_t ld_out, void *stream);

/* Product of a few rows with such weights: out[i, j] = sum over k of x[i, k] * w[j, k].  Each group's products are summed
 * in f32 and multiplied by its scale there.  Made for up to 32 rows; more are taken 32 at a time.
 * Where the call needs a workspace, x goes through it as a row's values over a power of two in FP8 planes: exact down to
 * 2^-14 of the row's largest magnitude, below that off by at most 2^-22 of it (f16: 2^-16 and 2^-27); magnitudes below
 * 2^-119 count as that in this, and sums are taken over that power of two before they are multiplied by scales, which
 * have to leave them in f32's range (as scales between 2^-100 and 2^100 do).
 * A row with a NaN or an infinity gives no finite result: NaN where the call needs a workspace, the products' infinities and
 * NaN where it needs none. */
typedef struct moe_ffn_int4_matmul_args {
  int32_t rows, n, k;            /* rows at most 2^16; n and k as above */
  int32_t type;                  /* of x, scales and out: MOE_FFN_BF16 or _F16 */
  int32_t group;
  const void *x; int64_t ld_x;   /* [rows, k]; 16-byte aligned, ld a multiple of 8 */
  const uint8_t *codes;          /* as above */
  const void *scales;
  const uint8_t *zeros;
  void *out; int64_t ld_out;     /* [rows, n], any ld >= n; overlaps no input */
  void *workspace; size_t workspace_bytes;  /* at least moe_ffn_int4_matmul_workspace, 256-byte aligned */
} moe_ffn_int4_matmul_args;

/* Bytes of workspace that the call needs (pointers are not read), 0 for none; negative: an error code. */
int64_t moe_ffn_int4_matmul_workspace(const moe_ffn_int4_matmul_args *a);

/* These three return MOE_FFN_OK, NULL_PTR, ROWS_ZERO, ROWS_RANGE, BAD_CONFIG, ALIGNMENT, ALIAS, UNSUPPORTED or CUDA,
 * int4_matmul NO_MEMORY too when the workspace is too small. */
int moe_ffn_int4_matmul(const moe_ffn_int4_matmul_args *a, void *stream);

/* A whole mixture-of-experts layer on a plain residual stream, for a few tokens:
 *   l = x router^T;  s = sigmoid(l) or softmax(l) over the experts
 *   the top_k experts by s + bias (in f32; without a bias by l), slots in descending order, exact ties to the lower index,
 *   NaN after everything else
 *   weight = route_scale * s, or with normalise route_scale * s / (sum of the chosen s)
 *   y = sum over the slots of weight * E(x) + sum over the shared experts of S(x), each a gated block
 *       E(x) = (act(x gate^T) * (x up^T)) down^T
 * weight * act(g) * u (a shared expert's without a weight) goes into the down projection as two numbers of the operand type:
 * 16 significant bits (f16: 22, but no more than 2^-36, and its range).
 * With bits 4 x goes through planes as int4_matmul's does, and the hidden values from f32 into three: off by at most 2^-14 of
 * a value, or 2^-27 of the largest of all of the token's experts.
 * A token that is not finite, or whose hidden values are not, gives results that are not (with bits 4 NaN); the others do
 * not see it.  An infinity or a NaN of an expert's matrix (with bits 4: scale) reaches the tokens that have chosen it alone. */
#define MOE_FFN_SCORE_SIGMOID 0
#define MOE_FFN_SCORE_SOFTMAX 1

typedef struct moe_ffn_matrices {  /* the matrices of one projection, [count, n, k], contiguous, 16-byte aligned */
  const void *w;                   /* bits 16: values; bits 4: codes as above */
  const void *scales;              /* bits 4 */
  const uint8_t *zeros;            /* bits 4: given for all projections, or for none */
} moe_ffn_matrices;

typedef struct moe_ffn_routed_args {
  int32_t rows, hidden, inter;     /* rows at most 32; hidden and inter multiples of 8 (bits 4: 32), at most 65536 */
  int32_t experts, top_k, shared;  /* at most 512, 8 (and experts) and 8 */
  int32_t type;                    /* MOE_FFN_BF16 or _F16: x, y, 16-bit weights, scales */
  int32_t router_type;             /* MOE_FFN_F32 or type */
  int32_t bits, group;             /* 16, or 4 with group 32, 64 or 128 */
  int32_t score, normalise, activation;
  float route_scale;
  const void *x; int64_t ld_x;     /* [rows, hidden]; 16-byte aligned, ld a multiple of 8 */
  const void *router;              /* [experts, hidden], contiguous, aligned to eight values */
  const float *bias;               /* [experts], or NULL */
  moe_ffn_matrices gate, up, down;                       /* [experts, inter, hidden] twice, [experts, hidden, inter] */
  moe_ffn_matrices shared_gate, shared_up, shared_down;  /* the same of the shared experts; all NULL with shared 0 */
  void *y; int64_t ld_y;           /* [rows, hidden], any ld >= hidden */
  int32_t *indices;                /* [rows, top_k], or NULL */
  float *weights;                  /* [rows, top_k], or NULL */
  void *workspace; size_t workspace_bytes;  /* at least moe_ffn_routed_workspace, 16-byte aligned */
} moe_ffn_routed_args;

/* The codes of moe_ffn_int4_matmul, and NO_MEMORY when the workspace is too small. */
int moe_ffn_routed_forward(const moe_ffn_routed_args *a, void *stream);

/* Bytes of workspace that the call needs; negative: an error code. */
int64_t moe_ffn_routed_workspace(const moe_ffn_routed_args *a);

/* Device status bits (MOE_FFN_DEV_TIMEOUT) that the kernels of the calls without a handle set on the current device
 * since the previous call, after waiting for `stream` (which must not be under capture); then cleared.
 * Each set of bits is reported to one caller.  Or a negative code. */
int moe_ffn_dense_status(void *stream);

/* Test hook for failure detection, as moe_ffn_set_fault_injection: with enable != 0, CTA 0 of each
 * tensor-core kernel of these calls that the process launches from now on first waits for
 * something that never comes, and wait_limit_us (0: 2 s) bounds every wait. */
int moe_ffn_dense_fault_injection(int32_t enable, uint32_t wait_limit_us);

/* Test hook: the tiles that a call with these sizes (contiguous rows) takes on a GPU of num_sms SMs, three
 * numbers for each of its tensor-core launches in order: the product (0 gate and up, 1 down, 2 hidden gradient,
 * 3 gradients, 4 FP8), the tile's columns, and how CTAs share it (0 one CTA, 1 a pair, 2 a cluster that shares
 * k).  Returns the number of launches, at most 3, 0 where the weight-streaming kernels serve the call, or a
 * negative code.  n and k: inter and hidden of the gated block. */
#define MOE_FFN_TILES_FORWARD 0
#define MOE_FFN_TILES_BACKWARD 1
#define MOE_FFN_TILES_BACKWARD_X 2
#define MOE_FFN_TILES_BACKWARD_WEIGHTS 3
#define MOE_FFN_TILES_FP8 4
int moe_ffn_dense_tiles(int32_t call, int32_t rows, int32_t n, int32_t k, int32_t num_sms, int32_t *tiles);

/* Text of the last error on this handle, or, when h is NULL, of the last failed call made without
 * a handle (init, the allocation-free split, a NULL handle) on the calling thread: that message
 * is kept per thread, so threads that fail at the same time do not overwrite each other's text.
 * The pointer stays valid until the same handle (or, for NULL, the same thread) fails again. */
const char *moe_ffn_last_error(const moe_ffn_handle *h);

/* Waits for outstanding work, frees everything the handle owns.  NULL is ignored. */
void moe_ffn_destroy(moe_ffn_handle *h);

#ifdef __cplusplus
}
#endif
#endif /* MOE_FFN_H */
