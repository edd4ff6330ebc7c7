/*
 * recon_chunk_ttt_b200 — C ABI of the ZipMap global large-chunk TTT layer on
 * B200 (sm_100a).
 *
 * The layer (kimjy99, "[논문리뷰] ZipMap: Linear-Time Stateful 3D
 * Reconstruction via Test-Time Training", section 2 "Feature Backbone"):
 *
 *   f_W(x) = W2 [ SiLU(W1 x) ⊙ (W3 x) ]                          (Eq. 1)
 *   L_i    = -f_W(k_i)^T v_i                                      (Eq. 2)
 *   g      = ∇_W Σ_i η_i L_i     (over every token of the chunk)   (Eq. 3)
 *   Ŵ      = ‖W‖ · (W - g) / ‖W - g‖   (L2 renormalisation, the update
 *                                       equations after Eq. 3)
 *   o_i    = f_Ŵ(q_i)            (apply, to image or ray-map queries)
 *
 * and, for streaming (section 3 "Streaming Reconstruction"), the same update
 * with the tokens of one frame at a time, the state carried across calls.
 * The renormalisation axis is row-wise (each row of W1, W3 of length d, each
 * row of W2 of length hidden, rescaled to its pre-update norm); "frobenius"
 * (one norm per matrix per head) and "off" are switches.
 *
 * Newton–Schulz (same section, the update after Eq. 3: Δ ← NewtonSchulz(g),
 * following the Muon optimizer; then Ŵ = ‖W‖ · (W − Δ)/‖W − Δ‖) is a switch,
 * ns_steps (0 = off, the layer above).  The page gives neither the polynomial
 * nor the step count; with ns_steps = k > 0 each of g1, g2, g3 of each head is
 * replaced by k steps of Muon's quintic iteration on X0 = g/‖g‖_F:
 *   X ← a X + (b A + c A²) X,  A = X Xᵀ,  (a, b, c) = (3.4445, −4.7750, 2.0315),
 * worked on the wide (d × hidden) orientation; g = 0 gives Δ = 0.  In
 * BF16_TC mode its GEMMs run on the tensor cores with each fp32 operand split
 * into two bf16 parts (hi + lo, three products), the iterate kept in fp32.
 *
 * Conventions shared by every entry point
 *  - All pointers except `cfg` are DEVICE pointers on the current CUDA device,
 *    owned by the caller; the library allocates no device memory and keeps no
 *    state between calls apart from one device error word per device and the
 *    optional tracing totals (ttt_trace_enable).
 *  - Every call is asynchronous on `stream` (NULL = the legacy default
 *    stream); arguments are validated on the host before anything is
 *    enqueued, so an error status means nothing was launched.
 *  - The update, reduce/renorm and apply kernels are launched as
 *    programmatic dependents (CUDA programmatic dependent launch): each
 *    waits for the complete, visible results of the work ahead of it on the
 *    stream before reading anything, and lets the next kernel on the stream
 *    start its launch early.  A caller's kernel that follows on the same
 *    stream and is itself launched with programmatic stream serialization
 *    must wait for its dependency (cudaGridDependencySynchronize) before
 *    reading this library's outputs; any other following work is ordered
 *    as usual.
 *  - Layouts are dense, row-major, per head h = 0..H-1:
 *        W1, W3 : float [H][hidden][d]      W2 : float [H][d][hidden]
 *        K, V, Q: [n][H*d] token-major, bf16 (precision BF16_TC) or
 *                 float (precision FP32_CHECK); head h is columns h*d..h*d+d-1
 *        eta    : float [n][H]
 *        O      : [m][H*d], bf16 (BF16_TC) or float (FP32_CHECK)
 *        shadow : bf16 copies of Ŵ for the tensor-core apply, in the same
 *                 layout as W1, W3, W2 (W1 block, then W3, then W2);
 *                 ttt_shadow_bytes() bytes.
 *  - Device pointers must be 16-byte aligned (tensor-memory-access rule), where
 *    an entry point does not say less.
 *  - Supported shapes: (d, hidden) = (64, 128) or (256, 512), heads >= 1
 *    (linear mode: (64, 64) or (256, 256)).
 *  - n = 0 or eta = 0 gives Ŵ = W.  Outputs may alias the weight inputs
 *    (in-place update); K, V, Q, eta and O must not alias outputs.
 *  - Results are deterministic run to run (fixed-order reductions, no
 *    atomics in any sum).
 */
#ifndef RECON_CHUNK_TTT_H
#define RECON_CHUNK_TTT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* ttt_stream_t;

typedef enum {
  TTT_OK = 0,
  TTT_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad enum   */
  TTT_ERR_UNSUPPORTED_SHAPE = 2, /* (d, hidden) not supported               */
  TTT_ERR_ALIGNMENT = 3,         /* a pointer is not 16-byte aligned        */
  TTT_ERR_WORKSPACE = 4,         /* workspace missing or too small          */
  TTT_ERR_CUDA = 5,              /* a CUDA runtime call failed              */
  TTT_ERR_DEVICE = 6             /* a kernel gave up a bounded wait         */
} ttt_status;

/* Fast-weight form.  TTT_MLP_SWIGLU: the layer above.  TTT_MLP_LINEAR:
 * f_W(k) = W k with one d x d matrix per head (67656.sbs reading notes,
 * section "为什么它像 attention（线性情形的直观推导）"), for which one step has
 * the closed form Ŵ = W + Σ_i η_i v_i k_i^T (before the renormalisation) and
 * the read o = Ŵ q is an un-normalised linear attention.  In linear mode
 * hidden must equal d, ns_steps must be 0, W is passed as W1 ([H][d][d],
 * row = output), W2 and W3 (and W2_out, W3_out) are unused and may be NULL,
 * the shadow holds the one bf16 matrix (H * d * d * 2 bytes) and partials
 * are [H][1][d*d] holding Σ η v k^T (= -g).  Its two contractions run on
 * CUDA cores with fp32 arithmetic in both precisions (BF16_TC reads bf16
 * tokens and the bf16 shadow and writes bf16 outputs); it is a reference
 * mode for that closed form, not the benchmarked layer. */
enum { TTT_MLP_SWIGLU = 0, TTT_MLP_LINEAR = 1 };
enum { TTT_RENORM_OFF = 0, TTT_RENORM_ROW = 1, TTT_RENORM_FROB = 2 };
enum { TTT_PREC_BF16_TC = 0, TTT_PREC_FP32_CHECK = 1 };
enum { TTT_MAX_NS_STEPS = 32 };

typedef struct {
  int32_t heads;     /* H, number of independent fast-weight MLPs          */
  int32_t d;         /* head dimension (64 or 256)                         */
  int32_t hidden;    /* fast-weight hidden width (128 or 512)              */
  int32_t mlp;       /* TTT_MLP_SWIGLU or TTT_MLP_LINEAR                   */
  int32_t renorm;    /* TTT_RENORM_*                                       */
  int32_t ns_steps;  /* Newton–Schulz steps on g: 0 (off) .. TTT_MAX_NS_STEPS */
  int32_t precision; /* TTT_PREC_BF16_TC: bf16 tensor-core operands, fp32
                        accumulation; TTT_PREC_FP32_CHECK: fp32 CUDA-core
                        arithmetic throughout                              */
} ttt_config;

/* Human-readable name of a status code (static string). */
const char* ttt_status_string(ttt_status s);

/* Bytes of device workspace ttt_update / ttt_stream_step need for n tokens
 * (0 if the config is invalid). */
size_t ttt_update_workspace_bytes(const ttt_config* cfg, int64_t n_tokens);

/* Bytes of the bf16 weight shadow (3 * H * d * hidden * 2; linear mode
 * H * d * d * 2). */
size_t ttt_shadow_bytes(const ttt_config* cfg);

/* Number of token splits S the update of n tokens reduces: the gradient is
 * accumulated as S fp32 partials over contiguous token ranges (a function of
 * cfg and n only), summed in increasing split order before the
 * renormalisation.  The workspace holds them.  0 if the config is invalid. */
int32_t ttt_update_splits(const ttt_config* cfg, int64_t n_tokens);

/*
 * One TTT update of all heads (Eq. 1–3 and the renormalisation above):
 *   g = ∇_W Σ_{i<n} η_i (−f_W(k_i)^T v_i),  Ŵ = renorm(W − Δ),
 *   Δ = g (ns_steps = 0) or NewtonSchulz(g) (ns_steps > 0).
 * Inputs W1, W2, W3 (fp32), K, V, eta for n >= 0 tokens.  Writes Ŵ to
 * W1_out, W2_out, W3_out (fp32, may equal the inputs) and, when `shadow` is
 * not NULL, bf16 copies of Ŵ to `shadow` for ttt_apply.
 * `workspace` must hold ttt_update_workspace_bytes(cfg, n) bytes (it may be
 * NULL when that is 0); its contents need no initialisation.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, WORKSPACE, CUDA.
 */
ttt_status ttt_update(const ttt_config* cfg,
                      const float* W1, const float* W2, const float* W3,
                      const void* K, const void* V, const float* eta, int64_t n,
                      float* W1_out, float* W2_out, float* W3_out, void* shadow,
                      void* workspace, size_t workspace_bytes, ttt_stream_t stream);

/*
 * Apply (read) the fast weights to m >= 0 queries: O[i] = f_Ŵ(Q[i]) per head
 * (section 2 of the review: o'_i = f_Ŵ(q_i); ray-map target queries use the
 * same call).  BF16_TC reads `shadow` (bf16 Ŵ, from ttt_update or
 * ttt_pack_shadow) and ignores W1..W3 (may be NULL); FP32_CHECK reads W1..W3
 * and ignores `shadow`.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, CUDA.
 */
ttt_status ttt_apply(const ttt_config* cfg,
                     const float* W1, const float* W2, const float* W3,
                     const void* shadow, const void* Q, int64_t m, void* O,
                     ttt_stream_t stream);

/* Write bf16 copies of W1, W2, W3 into `shadow` (for ttt_apply on weights
 * that did not come out of ttt_update). */
ttt_status ttt_pack_shadow(const ttt_config* cfg,
                           const float* W1, const float* W2, const float* W3,
                           void* shadow, ttt_stream_t stream);

/*
 * One streaming step (section 3 of the review, the per-frame TTTUpdate):
 * updates the state W1, W2, W3 IN PLACE with the n tokens of one frame, then
 * applies the new state to that frame's m queries, writing O.  `shadow` is
 * required for BF16_TC (it receives the bf16 copy of the new state) and may
 * be NULL for FP32_CHECK.  Workspace as for ttt_update(cfg, n).
 */
ttt_status ttt_stream_step(const ttt_config* cfg,
                           float* W1, float* W2, float* W3, void* shadow,
                           const void* K, const void* V, const float* eta, int64_t n,
                           const void* Q, int64_t m, void* O,
                           void* workspace, size_t workspace_bytes, ttt_stream_t stream);

/*
 * Synchronise `stream`, then read and clear this device's error word.  A
 * kernel that gives up a bounded wait (it never spins without a limit) sets
 * the word and returns early; such a call's outputs are undefined.
 * Returns TTT_OK, TTT_ERR_DEVICE (and *code = the kernel's reason, if code
 * is not NULL) or TTT_ERR_CUDA.
 */
ttt_status ttt_check_device_error(ttt_stream_t stream, int32_t* code);

/*
 * Failure-detection self-test (no counterpart on the pages): launches one
 * block whose thread waits, through the same bounded mbarrier wait the
 * kernels use, on a barrier nothing completes.  After limit_cycles SM cycles
 * (1 .. 2^31) the wait gives up, writes TTT_DEVICE_ERR_SELFTEST into the
 * device error word and the kernel returns; the next ttt_check_device_error
 * then returns TTT_ERR_DEVICE with that code, and the context stays usable.
 * Nothing traps or hangs.
 */
enum { TTT_DEVICE_ERR_SELFTEST = 7 };
ttt_status ttt_selftest_wait_timeout(int64_t limit_cycles, ttt_stream_t stream);

/*
 * Gated output unit (kimjy99 review, section 2 "Feature Backbone", the last
 * equation): o = RMSNorm(o') ⊙ SiLU(W_g o'), applied per head to the layer
 * output o' (e.g. ttt_apply's O).  The page does not say whether the unit
 * spans heads; heads being independent here, it is read per head:
 *   RMSNorm(x) = x / sqrt(mean_j x_j² + TTT_GATE_EPS)   (no learned gain)
 *   W_g: [H][d][d], row = output; bf16 (BF16_TC) or float (FP32_CHECK)
 *   O_prime, O: [m][H*d], the token type of the precision; O may equal
 *   O_prime (in place).
 * BF16_TC: W_g o' on the tensor cores (fp32 accumulation), RMS and gate in
 * fp32, o rounded to bf16.
 */
#define TTT_GATE_EPS 1e-6f
ttt_status ttt_gate(const ttt_config* cfg, const void* Wg, const void* O_prime, int64_t m,
                    void* O, ttt_stream_t stream);

/*
 * Token-sharded update across ranks (one chunk's tokens split over several
 * GPUs; the pages describe one GPU, this is the data-parallel form of the
 * same sum).  Eq. 3's g is a sum over tokens, so each rank reduces its own
 * tokens to a partial and the ranks exchange partials (an all-gather, e.g.
 * NCCL over NVLink, done by the caller); every rank then forms the same Ŵ.
 *
 * ttt_update_partial: the gradient partial of this rank's n tokens (weights
 *   W, tokens K, V, eta as in ttt_update) into `partial`, fp32, layout
 *   [H][3][hidden*d]: block 0 = g1 ([hidden][d]), block 1 = g3 ([hidden][d]),
 *   block 2 = −g2 ([d][hidden]); ttt_partial_floats(cfg) floats.  Partials add
 *   elementwise.  Workspace: ttt_update_workspace_bytes(cfg, n).  n = 0 gives
 *   zeros.
 * ttt_update_finish: Ŵ from `ranks` partials stored one after another
 *   ([ranks][H][3][hidden*d]), summed in rank order in fp64 (so the result
 *   does not depend on which rank computes it, and all ranks agree bitwise),
 *   then NewtonSchulz (cfg.ns_steps > 0) and the renormalisation as in
 *   ttt_update, against the pre-update W.  Outputs and shadow as in
 *   ttt_update (may alias W).  Workspace: ttt_finish_workspace_bytes(cfg).
 */
size_t ttt_partial_floats(const ttt_config* cfg);
size_t ttt_finish_workspace_bytes(const ttt_config* cfg);
ttt_status ttt_update_partial(const ttt_config* cfg, const float* W1, const float* W2,
                              const float* W3, const void* K, const void* V, const float* eta,
                              int64_t n, float* partial, void* workspace, size_t workspace_bytes,
                              ttt_stream_t stream);
ttt_status ttt_update_finish(const ttt_config* cfg, const float* W1, const float* W2,
                             const float* W3, const float* partials, int32_t ranks,
                             float* W1_out, float* W2_out, float* W3_out, void* shadow,
                             void* workspace, size_t workspace_bytes, ttt_stream_t stream);

/*
 * LaCT chunked orderings (mhpn.cn survey of TTSA3R / LaCT / ZipMap / LoGeR,
 * part "二、LaCT", "3应用场景"): the n tokens are cut into consecutive chunks of
 * `chunk` tokens (the last one shorter), and chunk i = tokens
 * [i*chunk, min(n, (i+1)*chunk)) is processed in order:
 *   TTT_ORDER_UPDATE_THEN_APPLY (block-causal): W <- U(W; chunk i) if the
 *       chunk updates, then O[chunk i] = f_W(Q[chunk i]);
 *   TTT_ORDER_APPLY_THEN_UPDATE (shifted block-causal): O[chunk i] =
 *       f_W(Q[chunk i]) with the state before the chunk, then W <- U(W; chunk i)
 *       if the chunk updates.
 * U is the update of ttt_update (with cfg's renorm and ns_steps), in place.
 * `update_mask` is a HOST array of ceil(n/chunk) bytes (nonzero = the chunk
 * updates) or NULL (every chunk updates); updating only chosen chunks gives the
 * cross-chunk causal pattern.  One chunk with APPLY_THEN_UPDATE is LaCT's
 * fully bidirectional pattern; one chunk with UPDATE_THEN_APPLY is the ZipMap
 * layer, and frame-sized chunks its streaming recurrence.
 *  - Arguments as in ttt_stream_step, with Q and O for the same n tokens
 *    (each token has a query): K, V, Q [n][H*d], eta [n][H], O [n][H*d].
 *  - BF16_TC: `shadow` is required; when the first operation is an apply it
 *    is first packed from W (the caller's contents do not matter).
 *    FP32_CHECK: `shadow` may be NULL.
 *  - chunk >= 1 and chunk * heads a multiple of 4 (every chunk's eta rows
 *    then start 16-byte aligned); workspace: ttt_update_workspace_bytes(cfg,
 *    min(chunk, n)).  Every argument is checked before anything is enqueued.
 */
enum { TTT_ORDER_UPDATE_THEN_APPLY = 0, TTT_ORDER_APPLY_THEN_UPDATE = 1 };
ttt_status ttt_chunked(const ttt_config* cfg, float* W1, float* W2, float* W3, void* shadow,
                       const void* K, const void* V, const float* eta, const void* Q,
                       int64_t n, int64_t chunk, int32_t order, const uint8_t* update_mask,
                       void* O, void* workspace, size_t workspace_bytes, ttt_stream_t stream);

/*
 * Allocation-free streaming step (the pages have no counterpart: this is a
 * deployment aid).  Same arguments and result as ttt_stream_step() minus the
 * workspace: the scratch is a fixed TTT_STATIC_SCRATCH_BYTES device array
 * inside the library, for callers that cannot allocate device memory when a
 * frame arrives (fixed memory budgets, allocator owned by another runtime, no
 * cudaMalloc after start-up).  The call allocates nothing.
 *  - Returns TTT_ERR_WORKSPACE, before launching anything, when
 *    ttt_update_workspace_bytes(cfg, n) exceeds TTT_STATIC_SCRATCH_BYTES.
 *    The limit depends on the configuration.  BF16_TC keeps the update's
 *    intermediates on chip, so its workspace stops growing with n: with 4
 *    heads of d = 256, hidden 512 every n fits (25.2 MB with ns_steps = 0,
 *    69.3 MB with ns_steps > 0); for every n, up to 31 such heads fit with
 *    ns_steps = 0 and 6 with ns_steps > 0.  FP32_CHECK keeps per-token
 *    intermediates: 4 heads of d = 256 fit up to 3,836 tokens per call with
 *    ns_steps = 0 and 2,044 with ns_steps > 0 (one 518 x 518 frame is 1,374
 *    tokens).
 *  - Every GPU that loads the library may hold the array until exit.
 *  - All calls on a device share the array and it keeps the last call's
 *    contents (nothing in it has to start at zero); calls that can overlap on
 *    the GPU race on it and must be serialised by the caller.
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress) and caches it with the id of the device's current
 *    context; a call after the context changed (cudaDeviceReset, or the
 *    primary context released and created again) looks it up anew.  Make
 *    such a call (the first on each device, and the first after a reset)
 *    before any stream capture.
 */
#define TTT_STATIC_SCRATCH_BYTES ((size_t)96 << 20)
ttt_status ttt_stream_step_static(const ttt_config* cfg,
                                  float* W1, float* W2, float* W3, void* shadow,
                                  const void* K, const void* V, const float* eta, int64_t n,
                                  const void* Q, int64_t m, void* O, ttt_stream_t stream);

/*
 * Gated delta rule: the causal sibling of the linear fast weights (mlp =
 * TTT_MLP_LINEAR).  The state S of a head has the linear mode's layout
 * (float [d][d], row = output); token after token it fades and is corrected
 * towards the token's value at the token's key, then read:
 *   S' = exp(log_decay_t) S,  u = beta_t (v_t - S' k_t),  S <- S' + u k_t^T,
 *   o_t = scale * S q_t.
 * (One gradient step of 1/2 |S' k - v|^2 with step beta; the keys and queries
 * are taken as they are: normalise them before the call where that is wanted.)
 *
 * ttt_delta_config: `heads` state heads; `qk_heads` heads of Q and K, a
 *   divisor of `heads` (state head h reads Q/K head h / (heads / qk_heads));
 *   d = 64, 128 or 256; scale finite.
 * ttt_delta_tokens: n tokens, packed.  Q, K: rows of qk_heads*d, V: rows of
 *   heads*d values of the precision's token type, consecutive rows ldq, ldk,
 *   ldv elements apart (at least the row; a multiple of 16 bytes), so they may
 *   be columns of one projection's output.  log_decay (<= 0; -inf forgets
 *   everything) and beta: float [n][heads], dense.  With `offsets` (device
 *   int64 [seqs + 1], non-decreasing, within 0..n) sequence i is the tokens
 *   offsets[i] .. offsets[i+1]-1; NULL: one sequence of all n tokens (seqs
 *   must be 1).  Sequences may be empty.  Rows of O (and of the token
 *   gradients) that belong to no sequence are left as they are.  Offsets that
 *   decrease or leave 0..n are clamped and reported in the device error word
 *   (TTT_DEVICE_ERR_OFFSETS); the outputs are then undefined.
 *   n up to 2^30; up to 65,535 sequences or requests; up to 4,096 heads.
 *   log_decay, beta, their gradients and slots: 4-byte aligned; offsets: 8.
 *   Rows of no sequence may hold anything; an infinity or NaN in a sequence
 *   reaches, besides all tokens behind it, up to 63 tokens before it.
 *
 * ttt_delta_chunk: all tokens of every sequence.  S_in: float
 *   [seqs][heads][d][d] or NULL (zeros); S_out: the states after the last
 *   tokens, or NULL; it may be S_in (in place).  An empty sequence hands its
 *   state on.  O: [n][heads*d] dense, token type.
 *   BF16_TC: chunks of 64 tokens on the tensor cores, the state and every sum
 *   in fp32.  For the states, operands that are not bf16 by nature go in as
 *   three bf16 parts, 24 bits.  For O, which is bf16 in the end, the state and
 *   the tokens' corrections u go in as two parts and the tokens' weights of
 *   each other as one: O is off by up to 2.4e-3 of itself (root mean square;
 *   its own rounding is 1.6e-3).  Short sequences, and FP32_CHECK (a check
 *   mode): token by token in fp32 on CUDA cores.
 * ttt_delta_step: one token for each of tok->n requests (tok->seqs = n,
 *   tok->offsets = NULL) on a pool of `pool` states float
 *   [pool][heads][d][d]: request i works on S[slots[i]] (slots: device int32
 *   [n]; NULL: slot i, and pool >= n).  S_out receives the states of the
 *   slots that were named and no others; it may be S (in place).  A slot that
 *   appears several times takes its tokens in the order of i.  A slot outside
 *   0..pool-1 (-1: padding) touches no state and its row of O is zero.
 * ttt_delta_backward: gradients of sum(dO . O) + sum(dS_out . S_out) for the
 *   tokens and S_in of ttt_delta_chunk.  dO: [n][heads*d] dense, token type;
 *   dS_out: float [seqs][heads][d][d] or NULL (zeros).  Writes dQ, dK
 *   ([n][qk_heads*d], summed over the heads that share them), dV
 *   ([n][heads*d]), token type, dense; dlog_decay, dbeta: float [n][heads];
 *   dS_in: float [seqs][heads][d][d] or NULL; it may be dS_out (in place).
 *   Nothing is kept from the forward call: it is recomputed in the workspace.
 *   dlog_decay of a token is exp(log_decay) times a product of the states on
 *   both sides of it, and 0 where nothing of the state is left.  BF16_TC:
 *   where log_decay >= -6 a running sum over the tokens behind it, whose fp32
 *   terms' rounding (some 1e-6 of them) it keeps; below -6 formed by itself from
 *   bf16 copies of the states (2e-3 of the products).  dbeta, dS_in and what
 *   dV is rounded from come as the states do, in 24 bits.  dQ and dK come from
 *   bf16 copies of the states before and their gradients behind each chunk, of dV
 *   and of one of the two weights of the tokens, two parts of the other and of u:
 *   off by 1.7e-3 to 2.4e-3 of themselves (1.6e-3 their own rounding).
 *
 * Outputs alias no input except where said.  Workspace bytes:
 * ttt_delta_workspace_bytes(cfg, n, seqs, backward); 0 where a call needs none
 * (short ones) and for an invalid config.  Nothing in it has to start at zero
 * or outlives the call.  Results are the same from run to run.
 */
typedef struct {
  int32_t heads;
  int32_t qk_heads;
  int32_t d;
  int32_t precision; /* TTT_PREC_* : type of Q, K, V, O and their gradients */
  float scale;       /* factor of the read, e.g. 1/sqrt(d) */
} ttt_delta_config;

typedef struct {
  const void* Q;
  const void* K;
  const void* V;
  const float* log_decay;
  const float* beta;
  int64_t ldq, ldk, ldv; /* elements between rows */
  int64_t n;
  const int64_t* offsets; /* device, or NULL */
  int64_t seqs;
} ttt_delta_tokens;

enum { TTT_DEVICE_ERR_OFFSETS = 8 };

size_t ttt_delta_workspace_bytes(const ttt_delta_config* cfg, int64_t n, int64_t seqs,
                                 int32_t backward);
ttt_status ttt_delta_chunk(const ttt_delta_config* cfg, const ttt_delta_tokens* tok,
                           const float* S_in, float* S_out, void* O, void* workspace,
                           size_t workspace_bytes, ttt_stream_t stream);
ttt_status ttt_delta_step(const ttt_delta_config* cfg, const ttt_delta_tokens* tok,
                          const int32_t* slots, int64_t pool, const float* S, float* S_out,
                          void* O, ttt_stream_t stream);
ttt_status ttt_delta_backward(const ttt_delta_config* cfg, const ttt_delta_tokens* tok,
                              const float* S_in, const void* dO, const float* dS_out, void* dQ,
                              void* dK, void* dV, float* dlog_decay, float* dbeta, float* dS_in,
                              void* workspace, size_t workspace_bytes, ttt_stream_t stream);

/*
 * Rotary positions over three axes, for the q and k of image and video tokens
 * (time or frame, height, width).  Of the d values of a head the first
 * rot[0] + rot[1] + rot[2] are rotated (the rest pass unchanged), as pairs:
 * the first rot[0]/2 pairs by the token's position on axis 0, the next
 * rot[1]/2 by axis 1, the next rot[2]/2 by axis 2.  Pair j (counted over all
 * axes, R = the sum of rot) is
 *   TTT_ROPE_HALF:  values j and j + R/2      TTT_ROPE_PAIRS: 2j and 2j + 1
 * and turns by position * base^(-e), with
 *   TTT_ROPE_FREQ_AXIS: e = i / (rot[a]/2), i counted within axis a
 *   TTT_ROPE_FREQ_HEAD: e = j / (R/2), over the whole head
 *   (x, y) -> (x cos - y sin, y cos + x sin); inverse != 0 turns back, which
 * is also the gradient: it maps dQ_out, dK_out to dQ, dK.
 * Angles are reduced to whole turns in fixed point, off by 2^-32 + |position|
 * 2^-62 of a turn at most; the rotation is fp32, rounded once.
 *  - d = 64, 128 or 256; rot[] even, >= 0, sum 2..d; base[] finite, >= 1.  With
 *    FREQ_HEAD every pair still uses its own axis' base.
 *  - positions: float [n][3] (whole numbers are exact to 2^24); fractions and
 *    negative positions are fine.  A position of infinity or NaN gives NaN.
 *    4-byte aligned.  n up to 2^30, up to 4,096 heads of q and of k.
 *  - Q: rows of q_heads*d values ldq apart, Q_out likewise ldq_out; K, K_out
 *    too, or k_heads = 0 with K = K_out = NULL.  Rows a multiple of 16 bytes
 *    apart.  Q_out may be Q and K_out K (in place, same row distance).
 */
enum { TTT_ROPE_HALF = 0, TTT_ROPE_PAIRS = 1 };
enum { TTT_ROPE_FREQ_AXIS = 0, TTT_ROPE_FREQ_HEAD = 1 };
typedef struct {
  int32_t d;
  int32_t rot[3];
  float base[3];
  int32_t layout;    /* TTT_ROPE_HALF or TTT_ROPE_PAIRS */
  int32_t freq;      /* TTT_ROPE_FREQ_* */
  int32_t precision; /* TTT_PREC_*: bf16 or float values */
} ttt_rope_config;
ttt_status ttt_rope(const ttt_rope_config* cfg, const void* Q, int64_t ldq, int32_t q_heads,
                    const void* K, int64_t ldk, int32_t k_heads, const float* positions,
                    int64_t n, void* Q_out, int64_t ldq_out, void* K_out, int64_t ldk_out,
                    int32_t inverse, ttt_stream_t stream);

/*
 * Layer norm (in front of the projections that make q, k, v and eta):
 *   y = (x - mean) * rstd * weight + bias,  rstd = 1/sqrt(var + eps),
 * over rows of `dim` values, var the mean square distance from the mean (taken
 * in a second pass over the row, which stays on chip).  X: rows ldx elements
 * apart; weight, bias: float [dim], each may be NULL (1 and 0); Y: [rows][dim]
 * dense; stats: float [rows][2] (mean, rstd) or NULL.  X and Y of the
 * precision's token type; Y may be X (then ldx = dim).
 * ttt_layer_norm_backward: from X, dY (rows lddy apart), weight and the stats
 *   of the forward call: dX ([rows][dim] dense, or NULL; it may be dY or X
 *   when that is dense), dweight and dbias (float [dim], each may be NULL).
 *   The sums over the rows are taken in fp32, in an order that depends on the
 *   sizes only.  dX is NULL or not, at least one output is wanted.  Rows = 0
 *   gives dweight = dbias = 0.  Workspace: ttt_norm_workspace_bytes(cfg, rows)
 *   (needed for dweight or dbias).
 *  - dim 1 .. 65536; eps >= 0, finite.  ldx, lddy >= dim, any value (rows that
 *    are multiples of 16 bytes, and so far apart, are faster).  Up to 2^30
 *    rows.  stats: 4-byte aligned.
 */
typedef struct {
  int64_t dim;
  float eps;
  int32_t precision; /* TTT_PREC_*: bf16 or float X, Y */
} ttt_norm_config;
size_t ttt_norm_workspace_bytes(const ttt_norm_config* cfg, int64_t rows);
ttt_status ttt_layer_norm(const ttt_norm_config* cfg, const void* X, int64_t ldx, int64_t rows,
                          const float* weight, const float* bias, void* Y, float* stats,
                          ttt_stream_t stream);
ttt_status ttt_layer_norm_backward(const ttt_norm_config* cfg, const void* X, int64_t ldx,
                                   const void* dY, int64_t lddy, int64_t rows,
                                   const float* weight, const float* stats, void* dX,
                                   float* dweight, float* dbias, void* workspace,
                                   size_t workspace_bytes, ttt_stream_t stream);

/*
 * Tracing.  With tracing on, every kernel launch of the library is bracketed
 * by two CUDA events on the caller's stream (host-side state: an event pool
 * and per-kernel totals, guarded by a mutex).  ttt_trace_read synchronises
 * the recorded events, adds their elapsed times to per-kernel totals and
 * copies up to `capacity` entries (name, launches, total milliseconds) into
 * `entries`; *count receives the number of kernel names seen.  reset != 0
 * clears the totals after reading.  Off by default.
 */
typedef struct {
  char name[32];
  int64_t launches;
  double total_ms;
} ttt_trace_entry;

ttt_status ttt_trace_enable(int32_t on);
ttt_status ttt_trace_read(ttt_trace_entry* entries, int32_t capacity, int32_t* count,
                          int32_t reset);

#ifdef __cplusplus
}
#endif

#endif /* RECON_CHUNK_TTT_H */
