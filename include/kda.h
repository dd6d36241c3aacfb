/*
 * libkda -- the Kimi Delta Attention (KDA) token mixer on AMD Instinct
 * MI355X (gfx950).  Plain C ABI: every tensor argument is a raw device
 * pointer plus sizes; no framework types cross this boundary.
 *
 * What is computed.  KDA is the gated delta-rule linear attention of the page
 * "Ling-3.0-flash: a 124B open MoE that runs like a 5B and reaches for 1M
 * tokens", section "KDA: constant-size memory over a very long context".  Per
 * sequence and head it keeps a fixed dk x dv state S (fp32 here).  For each
 * token t, with alpha_t the per-key-channel decay, beta_t the write strength:
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t,           y_t = o_t * sigmoid(z_t)  (when a gate is given)
 * (that section's own equation is missing from the page text; this is the
 * update its prose describes: decay as the erase, a delta-rule write, a read
 * with the query).  Before the recurrence q and k pass through a width-4
 * causal short conv and an L2 norm, v through a conv, alpha comes from a
 * softplus gate and beta from a sigmoid (same section; the conv width and the
 * 32 x 128 head shape are in the "Every architecture field" table of the page
 * "Ling 3.0 Flash", llm-architectures-explained).
 *
 * Conventions shared by every call.
 *  - Memory: every tensor pointer is a device pointer on the current HIP
 *    device, owned by the caller.  The library never allocates, frees or
 *    retains caller memory; scratch comes from a caller-provided workspace.
 *  - Layout: tensors are dense, row-major, fastest index last, 16-byte
 *    aligned.  [T, H, d] means token-major, then head, then channel.
 *  - Aliasing: only the recurrent state may alias (final_state may equal
 *    initial_state; the decode state is updated in place).  Any other overlap
 *    is rejected with KDA_ERR_INVALID_ARGUMENT.
 *  - Execution: calls enqueue work on `stream` (a hipStream_t; NULL is the
 *    null stream) and return without synchronising.  Host-side validation
 *    checks sizes, pointers, alignment and dtypes; the contents of cu_seqlens
 *    are trusted (non-decreasing, cu_seqlens[0] = 0, cu_seqlens[N] = T_tot).
 *  - Errors: calls return a status and never abort or throw.  After a non-OK
 *    return, outputs are undefined; kda_last_error_detail() gives a
 *    thread-local sentence naming the failing argument or HIP call.
 *  - Supported shapes: dk, dv in {16, 32, 64, 128}; H >= 1; N >= 1;
 *    T_tot >= 0 and below 2^31; sequences of length 0 are allowed.
 *  - Thread safety: no global mutable state; the error text and the optional
 *    kernel-timing records (kda_profile_enable) are per host thread.
 *  - Types: every call returns a kda_status_t value as a plain int, takes
 *    each dtype as an int32_t holding a kda_dtype_t value, and takes the
 *    stream as a void* holding a hipStream_t.  They are the same bits on the
 *    ABI; plain types keep this header free of the HIP headers, so a caller
 *    can bind it from any language (the Python binding uses ctypes).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1,   /* bad size, NULL or misaligned pointer, overlap */
    KDA_ERR_UNSUPPORTED = 2,        /* valid request this build does not implement */
    KDA_ERR_WORKSPACE_TOO_SMALL = 3,
    KDA_ERR_HIP = 4                 /* a HIP runtime call or kernel launch failed */
} kda_status_t;

typedef enum kda_dtype {
    KDA_F32 = 0,
    KDA_BF16 = 1
} kda_dtype_t;

/* Static text for a status code; never NULL. */
const char* kda_status_string(int status);

/* Thread-local detail of the last non-OK return on this thread ("" if none). */
const char* kda_last_error_detail(void);

/* ABI version of this header (major * 100 + minor). */
int kda_abi_version(void);

/*
 * kda_preprocess -- fused short conv, L2 norm and gates for a packed batch.
 * These are the steps the section "KDA: constant-size memory over a very
 * long context" of the page "Ling-3.0-flash: a 124B open MoE ..." applies
 * before the recurrence: q and k through a short causal conv and an L2 norm,
 * v through a conv, the decay from a softplus gate and the write strength
 * from a sigmoid (the conv width of 4 is in the "Every architecture field"
 * table of the page "Ling 3.0 Flash").
 *
 * For every sequence n (tokens cu_seqlens[n] .. cu_seqlens[n+1]-1), head h
 * and channel c:
 *   conv:  x~_t[c] = sum_{j=0..3} w[c][j] * x_{t-3+j}[c]   (tap 3 = current
 *          token; no bias, no activation).  Positions before the sequence
 *          start read conv_state[n] (oldest first) if given, else zero.
 *   norm:  q^ = q~ / sqrt(|q~|^2 + 1e-6) over the head's dk channels; same
 *          for k; v^ = v~.
 *   gates: log_alpha = -softplus(g) per key channel; beta = sigmoid(b) per head.
 * Arguments:
 *   T_tot, H, dk, dv     sizes; cu_seqlens: device int32 [N+1], or NULL for a
 *                        single sequence (then N must be 1);
 *   x_dtype              dtype of q_in, k_in, v_in, w_*, g_alpha, b_beta and
 *                        of q_out, k_out, v_out;
 *   q_in, k_in  [T_tot, H*dk];  v_in [T_tot, H*dv]   projected inputs;
 *   w_q, w_k    [H*dk, 4];      w_v  [H*dv, 4]       conv taps;
 *   g_alpha     [T_tot, H*dk]   decay logits;  b_beta [T_tot, H] write logits;
 *   conv_state  NULL, or fp32 [N, 3, H*(2*dk+dv)] (q channels, then k, then v):
 *               read as the history of each sequence, then overwritten with
 *               the last three raw tokens of that sequence (reaching back into
 *               the old history for sequences shorter than three);
 *   q_out, k_out [T_tot, H, dk]; v_out [T_tot, H, dv] (x_dtype);
 *   log_alpha_out fp32 [T_tot, H, dk]; beta_out fp32 [T_tot, H].
 */
int kda_preprocess(int64_t T_tot, int32_t H, int32_t dk, int32_t dv,
                   const int32_t* cu_seqlens, int32_t N, int32_t x_dtype,
                   const void* q_in, const void* k_in, const void* v_in,
                   const void* w_q, const void* w_k, const void* w_v,
                   const void* g_alpha, const void* b_beta,
                   float* conv_state,
                   void* q_out, void* k_out, void* v_out,
                   float* log_alpha_out, float* beta_out,
                   void* stream);

/*
 * Bytes of workspace kda_prefill_chunked needs for these sizes.  The bound
 * does not depend on the sequence lengths: it counts ceil(T_tot/64) + N
 * chunk slots (each sequence's chunks start at its own first token).
 * Returns 0 for unsupported or invalid sizes.
 */
size_t kda_prefill_workspace_bytes(int64_t T_tot, int32_t N, int32_t H, int32_t dk,
                                   int32_t dv, int32_t x_dtype);

/*
 * kda_prefill_chunked -- the recurrence over a packed batch of preprocessed
 * tokens, in chunks of 64 tokens.  The recurrence is the constant-size state
 * update and query read of the section "KDA: constant-size memory over a very
 * long context" of the page "Ling-3.0-flash: a 124B open MoE ...", with the
 * sigmoid output gate of the same section.  The result is that of the
 * token-by-token recurrence above (chunking changes only rounding): within a chunk the
 * writes are collected into a WY-style form (a unit-lower-triangular solve
 * over the chunk's keys) and the fp32 state is carried across chunks in
 * order, per sequence and head.
 * Arguments:
 *   cu_seqlens  device int32 [N+1], or NULL for a single sequence (N = 1);
 *   x_dtype     dtype of q, k, v, out_gate and out;
 *   gate_dtype  dtype of log_alpha and beta;
 *   q, k        [T_tot, H, dk] (L2-normalised keys keep every write a
 *               contraction);  v [T_tot, H, dv];
 *   log_alpha   [T_tot, H, dk], entries <= 0;  beta [T_tot, H];
 *   out_gate    NULL, or [T_tot, H, dv] logits z: out = o * sigmoid(z);
 *   initial_state NULL (zeros) or fp32 [N, H, dk, dv];
 *   final_state NULL (not wanted) or fp32 [N, H, dk, dv]; may equal
 *               initial_state (then updated in place);
 *   out         [T_tot, H, dv] (x_dtype);
 *   workspace   device scratch of at least kda_prefill_workspace_bytes()
 *               bytes, 256-byte aligned; contents on entry are ignored.
 * Sizes: H x (T_tot/64 + 1 + N) must stay below 2^32 (KDA_ERR_UNSUPPORTED
 * otherwise).
 */
int kda_prefill_chunked(int64_t T_tot, int32_t H, int32_t dk, int32_t dv,
                        const int32_t* cu_seqlens, int32_t N,
                        int32_t x_dtype, int32_t gate_dtype,
                        const void* q, const void* k, const void* v,
                        const void* log_alpha, const void* beta,
                        const void* out_gate,
                        const float* initial_state, float* final_state,
                        void* out,
                        void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * kda_prefill_layer -- kda_preprocess followed by kda_prefill_chunked in one
 * call, for bf16 inputs with dk = dv = 128 (the Ling-shaped heads): the
 * short conv, the L2 norm and the gates run inside the chunk kernel, so the
 * preprocessed q, k, v, log-decay and beta never go through device memory.
 * The result equals the two-call path up to rounding order.
 * Arguments: those of kda_preprocess for the raw inputs (q_in .. b_beta,
 * conv_state: read as the history, then replaced by the last three raw
 * tokens of each sequence) and of kda_prefill_chunked for the rest
 * (out_gate, initial_state, final_state, out, workspace sized by
 * kda_prefill_workspace_bytes with the same sizes).  Other head sizes or
 * dtypes return KDA_ERR_UNSUPPORTED: use the two calls.
 */
int kda_prefill_layer(int64_t T_tot, int32_t H, int32_t dk, int32_t dv,
                      const int32_t* cu_seqlens, int32_t N, int32_t x_dtype,
                      const void* q_in, const void* k_in, const void* v_in,
                      const void* w_q, const void* w_k, const void* w_v,
                      const void* g_alpha, const void* b_beta,
                      float* conv_state,
                      const void* out_gate,
                      const float* initial_state, float* final_state,
                      void* out,
                      void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * kda_prefill_layer_noalloc -- kda_prefill_layer for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops
 * and harnesses that forbid allocation.  Same computation, arguments and
 * errors as kda_prefill_layer, without the workspace: the call uses a fixed
 * scratch array of KDA_NOALLOC_SCRATCH_BYTES inside the library instead, and
 * allocates nothing (no hipMalloc, hipFree or allocating routine).
 *  - Each GPU the library runs on holds its own copy of the array, from the
 *    library's load until the process ends.  The first call on a device
 *    looks the copy up (no allocation); a caller that captures graphs can
 *    make that first call before capturing (T_tot = 0 is enough).
 *  - Sizes whose kda_prefill_workspace_bytes() exceeds
 *    KDA_NOALLOC_SCRATCH_BYTES are rejected with KDA_ERR_WORKSPACE_TOO_SMALL
 *    before any device work (at H = 32, d = 128, one sequence fits up to
 *    1,536 tokens).
 *  - Every call on one GPU shares that GPU's array, which keeps the last
 *    call's contents (nothing in it needs to start at zero).  Calls that
 *    overlap on one GPU (two host threads, or two streams) race on it and
 *    give undefined results: serialise them.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (64u << 20)
int kda_prefill_layer_noalloc(int64_t T_tot, int32_t H, int32_t dk, int32_t dv,
                              const int32_t* cu_seqlens, int32_t N, int32_t x_dtype,
                              const void* q_in, const void* k_in, const void* v_in,
                              const void* w_q, const void* w_k, const void* w_v,
                              const void* g_alpha, const void* b_beta,
                              float* conv_state,
                              const void* out_gate,
                              const float* initial_state, float* final_state,
                              void* out,
                              void* stream);

/*
 * State snapshots for prefix reuse: kda_prefill_chunked_snap and
 * kda_prefill_layer_snap are kda_prefill_chunked and kda_prefill_layer that
 * also write the state of each sequence after every snap_interval tokens
 * (counted from the sequence's start), so a prefix cache can resume a later
 * request from the longest cached prefix (the prefix caching of the page
 * "Ling-3.0-flash: a 124B open MoE ..."; for KDA the whole per-sequence
 * memory at a prefix is this fixed-size state plus the last three raw
 * tokens, which the caller has).  Snapshot m (m = 1 .. floor(len_n /
 * snap_interval)) of sequence n is the state after its first m *
 * snap_interval tokens (starting from initial_state[n] if given).
 * Extra arguments:
 *   snap_interval  tokens between snapshots, a positive multiple of 64;
 *   snapshots      fp32 [snap_capacity, H, dk, dv]; snapshot m of sequence n
 *                  is row snap_offsets[n] + m - 1;
 *   snap_capacity  rows available, at least T_tot / snap_interval (which
 *                  bounds the total); else KDA_ERR_INVALID_ARGUMENT;
 *   snap_offsets   device int32 [N + 1], written: the exclusive prefix sums
 *                  of floor(len_n / snap_interval); snap_offsets[N] = total.
 * The computation and every other output are those of the plain call.
 */
int kda_prefill_chunked_snap(int64_t T_tot, int32_t H, int32_t dk, int32_t dv,
                             const int32_t* cu_seqlens, int32_t N,
                             int32_t x_dtype, int32_t gate_dtype,
                             const void* q, const void* k, const void* v,
                             const void* log_alpha, const void* beta,
                             const void* out_gate,
                             const float* initial_state, float* final_state,
                             void* out,
                             void* workspace, size_t workspace_bytes,
                             int32_t snap_interval, float* snapshots,
                             int64_t snap_capacity, int32_t* snap_offsets,
                             void* stream);
int kda_prefill_layer_snap(int64_t T_tot, int32_t H, int32_t dk, int32_t dv,
                           const int32_t* cu_seqlens, int32_t N, int32_t x_dtype,
                           const void* q_in, const void* k_in, const void* v_in,
                           const void* w_q, const void* w_k, const void* w_v,
                           const void* g_alpha, const void* b_beta,
                           float* conv_state,
                           const void* out_gate,
                           const float* initial_state, float* final_state,
                           void* out,
                           void* workspace, size_t workspace_bytes,
                           int32_t snap_interval, float* snapshots,
                           int64_t snap_capacity, int32_t* snap_offsets,
                           void* stream);

/*
 * Gradients of kda_prefill_chunked (training).  For a loss whose gradients
 * with respect to the outputs y and the final states are dy and dS_final,
 * returns the gradients with respect to every input of the recurrence: q, k,
 * v, log_alpha, beta, the output-gate logits and the initial states.  They
 * are the adjoint of the chunked form (the recurrence of the section "KDA:
 * constant-size memory over a very long context" of the page "Ling-3.0-flash:
 * a 124B open MoE ..."; the pages train KDA from the first step), computed in
 * three passes: the forward again with the state kept at every chunk start,
 * the state gradient carried backwards over each sequence's chunks, and every
 * other gradient per chunk in parallel.  The gradient of the decay logits g
 * follows as dlog_alpha * -sigmoid(g), since log_alpha = -softplus(g).
 * Arguments: those of kda_prefill_chunked (any supported head size, both
 * dtypes; the output and final state are not recomputed), plus
 *   dy            [T_tot, H, dv] (x_dtype);
 *   dS_final      NULL (zero) or fp32 [N, H, dk, dv];
 *   grad_q, grad_k, grad_log_alpha [T_tot, H, dk], grad_v [T_tot, H, dv],
 *   grad_beta [T_tot, H]: fp32 outputs;
 *   grad_out_gate fp32 [T_tot, H, dv], required exactly when out_gate is given;
 *   grad_initial_state  NULL or fp32 [N, H, dk, dv].
 *   workspace     at least kda_backward_workspace_bytes(T_tot, N, H, dk, dv)
 *                 bytes, 256-byte aligned.
 */
size_t kda_backward_workspace_bytes(int64_t T_tot, int32_t N, int32_t H,
                                    int32_t dk, int32_t dv);
int kda_prefill_backward(int64_t T_tot, int32_t H, int32_t dk, int32_t dv,
                         const int32_t* cu_seqlens, int32_t N,
                         int32_t x_dtype, int32_t gate_dtype,
                         const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta,
                         const void* out_gate,
                         const float* initial_state,
                         const void* dy, const float* dS_final,
                         float* grad_q, float* grad_k, float* grad_v,
                         float* grad_log_alpha, float* grad_beta,
                         float* grad_out_gate, float* grad_initial_state,
                         void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * kda_decode_step -- one token per sequence, state updated in place: the
 * decode-time form of the recurrence of the section "KDA: constant-size
 * memory over a very long context" of the page "Ling-3.0-flash: a 124B open
 * MoE ..." (each new token costs the same fixed state read and write,
 * whatever the context length).
 * For each (b, h):  S' = Diag(alpha) S;  u = S'^T k;  S <- S' + beta k (v - u)^T;
 *                   o = S^T q;  out = o * sigmoid(z) (or o without a gate).
 * The state is read once and written once.
 * Arguments:
 *   q, k [B, H, dk], v [B, H, dv] (x_dtype), preprocessed;
 *   log_alpha [B, H, dk], beta [B, H] (gate_dtype);
 *   out_gate NULL or [B, H, dv] logits (x_dtype);
 *   state fp32 [B, H, dk, dv], in place;  out [B, H, dv] (x_dtype).
 */
int kda_decode_step(int32_t B, int32_t H, int32_t dk, int32_t dv,
                    int32_t x_dtype, int32_t gate_dtype,
                    const void* q, const void* k, const void* v,
                    const void* log_alpha, const void* beta,
                    const void* out_gate,
                    float* state, void* out,
                    void* stream);

/*
 * kda_decode_layer -- one token per sequence through the whole token mixer:
 * kda_preprocess for that token (conv against the caller's conv history, L2
 * norm, gates) fused with kda_decode_step, so a serving loop makes one call
 * per layer and token.  The preprocessed q, k, v are rounded to x_dtype
 * before the step (as kda_preprocess stores them); the gates stay fp32.
 * The result equals kda_preprocess (T_tot = B, N = B, cu_seqlens = 0..B)
 * followed by kda_decode_step with gate_dtype KDA_F32, up to rounding order.
 * States live in a pool: sequence b uses row state_indices[b] of state and
 * of conv_state (row b when state_indices is NULL, then state_slots must be
 * B).  This is the decode-time form of the recurrence and the conv in the
 * section "KDA: constant-size memory over a very long context" of the page
 * "Ling-3.0-flash: a 124B open MoE ...".
 * Arguments:
 *   q_in, k_in [B, H, dk], v_in [B, H, dv], g_alpha [B, H, dk], b_beta [B, H]
 *                 raw projections and gate logits of the new token (x_dtype);
 *   w_q, w_k [H*dk, 4], w_v [H*dv, 4]   conv taps (x_dtype), as kda_preprocess;
 *   conv_state    fp32 [state_slots, 3, H*(2*dk + dv)]: per slot the last
 *                 three raw tokens (oldest first; q, then k, then v columns),
 *                 the layout kda_preprocess reads and writes; rolled forward
 *                 by one token in place;
 *   out_gate      NULL or [B, H, dv] logits (x_dtype);
 *   state         fp32 [state_slots, H, dk, dv], updated in place;
 *   state_slots   rows in the two pools (>= 0);
 *   state_indices NULL or device int32 [B].  An entry outside
 *                 [0, state_slots) marks a padding row: its out row is set to
 *                 zero and no state is read or written.  Valid entries must be
 *                 distinct (two rows on one slot race); with the environment
 *                 variable KDA_DEBUG_CHECK=1 the call copies the indices to the
 *                 host, synchronising the stream, and rejects duplicates;
 *   out           [B, H, dv] (x_dtype).
 * Pool rows that no valid entry names are neither read nor written.
 */
int kda_decode_layer(int32_t B, int32_t H, int32_t dk, int32_t dv,
                     int32_t x_dtype,
                     const void* q_in, const void* k_in, const void* v_in,
                     const void* w_q, const void* w_k, const void* w_v,
                     const void* g_alpha, const void* b_beta,
                     float* conv_state,
                     const void* out_gate,
                     float* state, int32_t state_slots,
                     const int32_t* state_indices,
                     void* out,
                     void* stream);

/*
 * Speculative decoding: verify 1 + n draft tokens per sequence, commit later.
 *
 * The decoding on the page "Ling-3.0-flash: a 124B open MoE ..." proposes
 * three draft tokens per step (multi-token prediction) and verifies them in
 * one pass; how many are accepted is known only after that pass.  Each call
 * of kda_spec_verify, per sequence b and its pool row s = state_indices[b]:
 *   1. commits: the first accepted[b] tokens of the previous call on slot s
 *      (kept raw in the draft buffer) go through the conv (against the
 *      slot's conv history), the L2 norm, the gates and the recurrence, as
 *      kda_decode_layer would run them one by one; the slot's state and conv
 *      history are written back, holding those tokens;
 *   2. verifies: the T new raw tokens run from that state in order (token t's
 *      output reads the state after tokens 0..t), and their outputs are
 *      written; the state and conv history are NOT advanced by them.  Their
 *      raw values replace the slot's draft buffer, for the next call to commit.
 * So each call reads and writes the state once.  A call with T = 0 only
 * commits (use it to bring a slot up to date, e.g. when a sequence leaves
 * speculative mode).  The recurrence is that of kda_decode_step (section
 * "KDA: constant-size memory over a very long context" of the same page).
 * Arguments:
 *   B, T          sequences and new tokens per sequence (0 <= T <= 8);
 *   q_in, k_in [B, T, H, dk], v_in [B, T, H, dv], g_alpha [B, T, H, dk],
 *   b_beta [B, T, H]   raw projections and gate logits (x_dtype);
 *   w_q, w_k, w_v, conv_state, state, state_slots, state_indices
 *                 as for kda_decode_layer (pools of state_slots rows);
 *   out_gate      NULL or [B, T, H, dv] (x_dtype);
 *   accepted      NULL (commit nothing) or device int32 [B]: how many of the
 *                 previous call's tokens on that slot to commit, in
 *                 [0, that call's T]; values are clamped to [0, 8], and a
 *                 count above the previous T commits stale buffer contents;
 *   drafts        per slot kda_spec_draft_bytes(H, dk, dv, x_dtype) bytes
 *                 of device memory, owned by the caller, opaque (raw tokens
 *                 of the last call, in x_dtype: every call on one buffer
 *                 must use the same x_dtype, a commit-only call included);
 *                 contents matter only where accepted > 0;
 *   out           [B, T, H, dv] (x_dtype).
 * Padding rows (index outside the pool) get zero outputs and touch nothing.
 * A row with accepted = 0 and T = 0 is a no-op.
 */
size_t kda_spec_draft_bytes(int32_t H, int32_t dk, int32_t dv, int32_t x_dtype);
int kda_spec_verify(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                    int32_t x_dtype,
                    const void* q_in, const void* k_in, const void* v_in,
                    const void* w_q, const void* w_k, const void* w_v,
                    const void* g_alpha, const void* b_beta,
                    float* conv_state,
                    const void* out_gate,
                    float* state, int32_t state_slots,
                    const int32_t* state_indices,
                    const int32_t* accepted,
                    void* drafts,
                    void* out,
                    void* stream);

/*
 * Full attention: the layers that stand between the KDA layers of the hybrid
 * model (one in six there; the "Every architecture field" table of the page
 * "Ling 3.0 Flash" gives heads of 192, 128 and 64 rotary, over values of 128).
 *
 * Shared by the calls below.
 *  - Heads: H query heads over Hkv key and value heads (Hkv divides H); query
 *    head h reads key head h / (H / Hkv).  dk = dv = 16, 32, 64 or 128, or
 *    dk = 192 with dv = 128 (else KDA_ERR_UNSUPPORTED).
 *  - Types: x_dtype (fp32 or bf16) for every tensor without another type.
 *    Scores, softmax statistics and sums are fp32; with bf16 the weights are
 *    rounded to bf16 for their product with the values, and in the gradients
 *    also the scores' gradients (for their products with q and k) and the gated
 *    output gradient dy * sigmoid(z).  With fp32 nothing is rounded to less.
 *  - scale multiplies q . k; positive and finite.
 *  - out_gate: NULL, or logits z of out's shape: out = o * sigmoid(z).
 *  - A row that attends nothing gets 0, and -infinity as its lse.  A row that
 *    attends a score that is NaN or +infinity, or scores of -infinity alone, is
 *    NaN, and so is its lse.
 *  - Non-finite values reach the rows that attend them.  Other sequences'
 *    rows, memory behind a sequence's end, stale page contents and drafts that
 *    a row does not attend never reach it.  Within one sequence of
 *    kda_attn_prefill and its gradients, a non-finite row may also reach
 *    rows up to 127 tokens from it (0 x infinity in a shared tile).
 *  - Rows of T_tot behind the last sequence are neither read nor written:
 *    cu_seqlens[N] may be below T_tot.
 *  - Calls, or replays of captured graphs, that overlap in time need a
 *    workspace each; in turn on one stream they can share one.
 *
 * kda_attn_prefill -- causal attention over a packed batch of whole prompts:
 * token i of a sequence attends its tokens 0 .. i,
 *     s_ij = scale q_i . k_j,   o_i = sum_j softmax_j(s_ij) v_j,
 *     lse_i = log sum_j e^(s_ij).
 * Arguments:
 *   q [T_tot, H, dk]; k [T_tot, Hkv, dk]; v [T_tot, Hkv, dv];
 *   out [T_tot, H, dv];  lse NULL or fp32 [T_tot, H] (the gradients need it).
 * The call needs no workspace.  H x (T_tot/128 + min(N, T_tot)) must stay
 * below 2^24 (KDA_ERR_UNSUPPORTED otherwise).
 */
int kda_attn_prefill(int64_t T_tot, int32_t H, int32_t Hkv, int32_t dk, int32_t dv,
                     const int32_t* cu_seqlens, int32_t N, int32_t x_dtype, float scale,
                     const void* q, const void* k, const void* v,
                     const void* out_gate,
                     void* out, float* lse,
                     void* stream);

/*
 * kda_attn_prefill_backward -- gradients of kda_attn_prefill for output
 * gradients dy.  The scores are formed again from q, k and lse; key and value
 * gradients are summed over the query heads that share a head.  Every sum has
 * one owner and a fixed order: the same inputs give the same bits.  A row's
 * weights e^(s - lse) are as right as its fp32 lse, to about |lse| 2^-23 of
 * themselves (10^-3 at scores of 10^4; past 10^8 the gradients mean nothing).
 * Arguments: those of kda_attn_prefill, with out and lse as it wrote them, and
 *   dy            [T_tot, H, dv];
 *   grad_q [T_tot, H, dk], grad_k [T_tot, Hkv, dk], grad_v [T_tot, Hkv, dv]:
 *                 in x_dtype (they feed x_dtype products; the sums are fp32);
 *   grad_out_gate [T_tot, H, dv], required exactly when out_gate is given;
 *   workspace     at least kda_attn_backward_workspace_bytes() bytes (of the
 *                 same sizes; with_gate: whether out_gate is given), 256-byte
 *                 aligned; contents on entry are ignored.  Fewer tokens can
 *                 need more (their work is cut into more parts): a workspace
 *                 of kda_attn_backward_max_workspace_bytes() bytes holds every
 *                 call of up to max_T_tot tokens in any number of sequences.
 * H x (T_tot/128 + min(N, T_tot)) must stay below 2^23 and T_tot x H below
 * 2^28 (KDA_ERR_UNSUPPORTED otherwise).
 */
size_t kda_attn_backward_workspace_bytes(int64_t T_tot, int32_t N, int32_t H, int32_t Hkv,
                                         int32_t dk, int32_t dv, int32_t x_dtype, int32_t with_gate);
size_t kda_attn_backward_max_workspace_bytes(int64_t max_T_tot, int32_t H, int32_t Hkv,
                                             int32_t dk, int32_t dv, int32_t x_dtype, int32_t with_gate);
int kda_attn_prefill_backward(int64_t T_tot, int32_t H, int32_t Hkv, int32_t dk, int32_t dv,
                              const int32_t* cu_seqlens, int32_t N, int32_t x_dtype, float scale,
                              const void* q, const void* k, const void* v,
                              const void* out_gate, const void* out, const float* lse,
                              const void* dy,
                              void* grad_q, void* grad_k, void* grad_v, void* grad_out_gate,
                              void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * kda_attn_window_prefill, kda_attn_window_prefill_backward -- the same two
 * calls for layers that see a bounded part of what is behind them: token i of
 * a sequence attends its tokens j <= i with
 *     i - j < window   or   j < sinks,
 * the last `window` tokens, its own among them, and the sequence's first ones,
 * which stay visible.  A window of the sequence's length or more is causal
 * attention.  Work and time go by the pairs that are attended.
 * Arguments: those of kda_attn_prefill and kda_attn_prefill_backward, and
 *   window        >= 1;   sinks >= 0;
 *   workspace     (gradients) sized by kda_attn_window_backward_workspace_bytes()
 *                 with the call's sizes, window and sinks, or for every call of
 *                 up to max_T_tot tokens in any number of sequences, with that
 *                 window and those sinks, by
 *                 kda_attn_window_backward_max_workspace_bytes().
 * T_tot must be below 2^29, for the gradients H x (T_tot/128 + min(N, T_tot))
 * below 2^22, and the limits of the calls above hold (KDA_ERR_UNSUPPORTED
 * otherwise).  A row that is not finite may also reach
 * rows up to 190 tokens from those that attend it, and gradients of tokens as
 * far from those that such rows attend.
 */
int kda_attn_window_prefill(int64_t T_tot, int32_t H, int32_t Hkv, int32_t dk, int32_t dv,
                            const int32_t* cu_seqlens, int32_t N, int32_t x_dtype, float scale,
                            int32_t window, int32_t sinks,
                            const void* q, const void* k, const void* v,
                            const void* out_gate,
                            void* out, float* lse,
                            void* stream);
size_t kda_attn_window_backward_workspace_bytes(int64_t T_tot, int32_t N, int32_t H, int32_t Hkv,
                                                int32_t dk, int32_t dv, int32_t x_dtype, int32_t with_gate,
                                                int32_t window, int32_t sinks);
size_t kda_attn_window_backward_max_workspace_bytes(int64_t max_T_tot, int32_t H, int32_t Hkv,
                                                    int32_t dk, int32_t dv, int32_t x_dtype, int32_t with_gate,
                                                    int32_t window, int32_t sinks);
int kda_attn_window_prefill_backward(int64_t T_tot, int32_t H, int32_t Hkv, int32_t dk, int32_t dv,
                                     const int32_t* cu_seqlens, int32_t N, int32_t x_dtype, float scale,
                                     int32_t window, int32_t sinks,
                                     const void* q, const void* k, const void* v,
                                     const void* out_gate, const void* out, const float* lse,
                                     const void* dy,
                                     void* grad_q, void* grad_k, void* grad_v, void* grad_out_gate,
                                     void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * A paged cache of keys and values.
 *   k_cache [num_pages, Hkv, page_size, dk], v_cache [num_pages, Hkv,
 *   page_size, dv]: the pools (x_dtype; page_size a power of two, 16 .. 1024);
 *   page_table  int32 [slots, max_pages]: token p of a slot is row
 *               p % page_size of page page_table[slot][p / page_size]; an
 *               entry outside [0, num_pages) names no page (1 <= max_pages <
 *               2^23, max_pages * page_size < 2^31);
 *   lens        int32 [slots]: committed tokens of each slot;
 *   refs        int32 [num_pages]: table entries that name the page; a page
 *               whose count is not positive is free.
 * A slot's pages stand at the front of its table row; a slot without pages
 * has length 0 and -1 in its entries (page_table filled with -1, lens and
 * refs with 0 is an empty cache).  Calls on one cache are ordered by the
 * stream; two that overlap in time race.
 *
 * kda_attn_tree -- attention of a tree of drafted tokens over the cache: the
 * full-attention side of a kda_spec_verify call, and with T = 1 plain decode.
 * Token t of sequence b attends all lens[slot] tokens of its slot and the
 * drafted tokens j whose bit j is set in its mask word (its own bit
 * included: a word of 0 attends the cache alone).  The drafts' keys and
 * values are given dense and are not written to the cache; commit the
 * accepted ones with kda_cache_append.
 * Arguments:
 *   B, T          sequences and drafted tokens per sequence (0 <= T <= 64);
 *   q [B, T, H, dk], k_new [B, T, Hkv, dk], v_new [B, T, Hkv, dv];
 *   tree_mask     NULL (a chain: token t attends drafts 0 .. t) or int64 [B, T];
 *   slot_indices  NULL (sequence b uses slot b; then slots must be B) or
 *                 device int32 [B]; several sequences may name one slot.  An
 *                 index outside [0, slots) marks a padding row: its outputs
 *                 are 0 (lse -infinity) and nothing of it is read;
 *   out [B, T, H, dv]; lse NULL or fp32 [B, T, H];
 *   workspace     at least kda_attn_tree_workspace_bytes() bytes for
 *                 max_context = max_pages * page_size, 256-byte aligned.
 *                 Fewer sequences can need more (their keys are cut into more
 *                 parts): kda_attn_tree_max_workspace_bytes() bytes hold every
 *                 call of up to max_B sequences of up to max_T tokens over
 *                 tables of up to max_context (a query for setting up: it
 *                 takes up to milliseconds).
 * Tokens whose table entry names no page are not attended.  Lengths are
 * clamped to what a table row holds.  B x T x H must be below 2^30, and
 * B x Hkv x ceil(T x H/Hkv / 32) below 2^24 (B x Hkv rounded up to 8;
 * KDA_ERR_UNSUPPORTED otherwise).
 */
size_t kda_attn_tree_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t dk,
                                     int32_t dv, int32_t x_dtype, int64_t max_context);
size_t kda_attn_tree_max_workspace_bytes(int32_t max_B, int32_t max_T, int32_t H, int32_t Hkv, int32_t dk,
                                         int32_t dv, int32_t x_dtype, int64_t max_context);
int kda_attn_tree(int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t dk, int32_t dv,
                  int32_t x_dtype, float scale,
                  const void* q, const void* k_new, const void* v_new,
                  const int64_t* tree_mask, const void* out_gate,
                  const void* k_cache, const void* v_cache, int32_t num_pages, int32_t page_size,
                  const int32_t* page_table, int32_t slots, int32_t max_pages,
                  const int32_t* lens, const int32_t* slot_indices,
                  void* out, float* lse,
                  void* workspace, size_t workspace_bytes,
                  void* stream);

/*
 * kda_attn_window_tree -- kda_attn_tree for such layers, over the same cache.
 * The tokens of a row in order are the slot's lens[slot] tokens and then, by
 * their number, the drafts of the row's mask word, n in all; the row attends
 * those at places below `sinks` and from n - window on.  For a draft's own path
 * from the context (its own bit included) that is the view of
 * kda_attn_window_prefill.  A cached token whose entry names no page keeps its
 * place and is not attended, so pages that no row will see again can go.
 * Arguments: those of kda_attn_tree, and window >= 1, sinks >= 0; workspace by
 * the two functions below.  max_pages x page_size must be below 2^29
 * (KDA_ERR_UNSUPPORTED otherwise).
 */
size_t kda_attn_window_tree_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t dk,
                                            int32_t dv, int32_t x_dtype, int64_t max_context,
                                            int32_t window, int32_t sinks);
size_t kda_attn_window_tree_max_workspace_bytes(int32_t max_B, int32_t max_T, int32_t H, int32_t Hkv,
                                                int32_t dk, int32_t dv, int32_t x_dtype, int64_t max_context,
                                                int32_t window, int32_t sinks);
int kda_attn_window_tree(int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t dk, int32_t dv,
                         int32_t x_dtype, float scale, int32_t window, int32_t sinks,
                         const void* q, const void* k_new, const void* v_new,
                         const int64_t* tree_mask, const void* out_gate,
                         const void* k_cache, const void* v_cache, int32_t num_pages, int32_t page_size,
                         const int32_t* page_table, int32_t slots, int32_t max_pages,
                         const int32_t* lens, const int32_t* slot_indices,
                         void* out, float* lse,
                         void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * kda_cache_append -- writes the keys and values of new tokens into pages.
 * Sequence n's tokens are t = cu_seqlens[n] .. cu_seqlens[n+1] - 1; token t
 * comes from row rows[t] of k_new and v_new (row t when rows is NULL) and goes
 * to position lens[slot] + t - cu_seqlens[n] of its slot.  So one call takes a
 * packed batch of prompts (rows NULL) or the accepted path of each draft tree
 * (rows: b * T + the path's tokens, in order).  lens is read, not advanced:
 * the caller adds the counts when the tokens are committed.
 * Arguments:
 *   cu_seqlens int32 [N+1] or NULL (one sequence of T_tot tokens);
 *   k_new [src_rows, Hkv, dk], v_new [src_rows, Hkv, dv]; rows int32 [T_tot];
 *   slot_indices NULL (sequence n uses slot n) or int32 [N], distinct where
 *                the sequences are not empty.
 * Dropped: tokens at or behind cu_seqlens[N], of slots outside [0, slots),
 * from rows outside [0, src_rows), and at positions whose table entry names no
 * page (kda_cache_reserve gives a slot its pages first).  T_tot must be below
 * 2^27 (KDA_ERR_UNSUPPORTED otherwise).
 */
int kda_cache_append(int64_t T_tot, int32_t N, const int32_t* cu_seqlens,
                     int64_t src_rows, const int32_t* rows,
                     int32_t Hkv, int32_t dk, int32_t dv, int32_t x_dtype,
                     const void* k_new, const void* v_new,
                     void* k_cache, void* v_cache, int32_t num_pages, int32_t page_size,
                     const int32_t* page_table, int32_t slots, int32_t max_pages,
                     const int32_t* lens, const int32_t* slot_indices,
                     void* stream);

/*
 * The pages of a cache.  status (NULL or int32 [n], written): 0 done, 1 the
 * pool has too few free pages, 2 refused (a slot outside [0, slots), or as
 * said below); an entry that is not done changes nothing.  Free pages go out
 * lowest number first, in the order of the entries, so the results do not
 * depend on timing; the first entry that does not fit and every later one
 * that needs pages get status 1.  Workspace: at least
 * kda_cache_workspace_bytes(num_pages, slots, n) bytes (n = 0 for
 * kda_cache_compact), 256-byte aligned; contents on entry are ignored.  Lists
 * of slots must be shorter than 2^24 (KDA_ERR_UNSUPPORTED otherwise).
 *
 * kda_cache_free -- empties the listed slots: their entries become -1, their
 * lengths 0, and the counts of their pages drop by one each.  Slots outside
 * [0, slots) are skipped; naming a slot twice is naming it once.
 *
 * kda_cache_fork -- slot dst[i] becomes a copy of slot src[i]: the full pages
 * are shared (their counts rise), the rows in use of a partly filled last
 * page are copied to a new page, so both slots can be appended to.  Refused:
 * src[i] = dst[i], a dst that holds tokens or pages, and a dst that an earlier
 * entry of the call names.  A slot may be forked many times in one call.
 *
 * kda_cache_reserve -- gives slot slot_list[i] the pages that it lacks for
 * new_lens[i] tokens: every table entry behind those that hold its length, up
 * to the new length, that names no page gets one.  lens is not changed.  An
 * entry that holds a part of the length and names no page stays so, the last,
 * partly filled one too: its tokens are gone, a page there would put stale
 * contents in their place, and kda_cache_append drops what falls into it
 * (free such a slot and write its tokens again).
 * Refused: lengths that a table row does not hold, and a slot that an earlier
 * entry of the call names.
 *
 * kda_cache_compact -- moves the pages in use to the front of the pool (live
 * of them, written to live[0]): the k-th page in use at or behind `live` moves
 * to the k-th free page before it, counts and table entries follow.  The rest
 * stay where they are; pages from live[0] on are free after the call.
 *
 * kda_cache_copy -- row src[i] of a pool [rows, row_bytes] is copied to row
 * dst[i]: pages of a cache, or rows of the KDA state and conv-history pools
 * when a sequence is forked.  row_bytes is a multiple of 16.  Entries with a
 * row outside [0, rows), or with src[i] = dst[i], are skipped.  No row may be
 * written twice, or read and written, by one call (its contents would depend
 * on timing); with KDA_DEBUG_CHECK=1 the call checks that, synchronising the
 * stream.
 */
size_t kda_cache_workspace_bytes(int32_t num_pages, int32_t slots, int32_t n);
int kda_cache_free(int32_t n, const int32_t* slot_list, int32_t num_pages,
                   int32_t* page_table, int32_t slots, int32_t max_pages,
                   int32_t* lens, int32_t* refs, void* stream);
int kda_cache_fork(int32_t n, const int32_t* src, const int32_t* dst,
                   int32_t Hkv, int32_t dk, int32_t dv, int32_t x_dtype,
                   void* k_cache, void* v_cache, int32_t num_pages, int32_t page_size,
                   int32_t* page_table, int32_t slots, int32_t max_pages,
                   int32_t* lens, int32_t* refs,
                   int32_t* status,
                   void* workspace, size_t workspace_bytes, void* stream);
int kda_cache_reserve(int32_t n, const int32_t* slot_list, const int32_t* new_lens,
                      int32_t num_pages, int32_t page_size,
                      int32_t* page_table, int32_t slots, int32_t max_pages,
                      const int32_t* lens, int32_t* refs,
                      int32_t* status,
                      void* workspace, size_t workspace_bytes, void* stream);
int kda_cache_compact(int32_t Hkv, int32_t dk, int32_t dv, int32_t x_dtype,
                      void* k_cache, void* v_cache, int32_t num_pages, int32_t page_size,
                      int32_t* page_table, int32_t slots, int32_t max_pages,
                      int32_t* refs, int32_t* live,
                      void* workspace, size_t workspace_bytes, void* stream);
int kda_cache_copy(void* pool, int64_t row_bytes, int32_t rows,
                   const int32_t* src, const int32_t* dst, int32_t n, void* stream);

/*
 * kda_cache_weigh -- how much attention each cached token gets: for a
 * sequence's last tokens, whose queries are at hand, adds their attention
 * weights to what the tokens of its slot have gathered,
 *     weights[slot][j] += sum_i sum_h e^(scale q_ih . k_j - lse_ih),
 * over the queries i that attend token j and all heads h.  Sequence n's
 * queries t = cu_seqlens[n] .. cu_seqlens[n+1] - 1, c of them, are the last c
 * tokens of its slot (they have been appended and lens counts them): the i-th
 * stands at place p = lens[slot] - c + i and attends the places j <= p, with
 * window > 0 those with p - j < window or j < sinks.  So one call serves a
 * decode step, the accepted path of each draft tree (rows: b * T + the path's
 * tokens, in order), the last tokens of a prompt or all of it.  A call takes one
 * of two forms by the average, T_tot (H / Hkv) / N rows of a key head up to 32 or
 * above.  Either is right for any batch, but a prompt beside decode steps belongs
 * in a call of its own: 300 steps and 2,000 tokens of a prompt take 10 ms in one
 * call and 0.3 ms in two.
 * Arguments:
 *   q [src_rows, H, dk], lse fp32 [src_rows, H]: the queries and what the
 *                 attention call gave for them; rows int32 [T_tot] or NULL
 *                 (query t is row t);
 *   window        0 (every token up to the query's own) or as the attention
 *                 call's, with its sinks;
 *   weights       fp32 [slots, max_pages * page_size], added to; a slot's start
 *                 at 0 with it.  kda_cache_copy forks rows of it;
 *   slot_indices  NULL (sequence n uses slot n) or int32 [N], distinct where
 *                 the sequences are not empty;
 *   workspace     at least kda_cache_weigh_workspace_bytes() bytes, 256-byte
 *                 aligned; contents on entry are ignored ((1,024 + N) KiB hold
 *                 every call of up to N sequences).
 * Products, exponentials and sums are fp32, in a fixed order: the same inputs
 * give the same bits.  A weight is as right as its lse (see the gradients).
 * Skipped: slots outside [0, slots), rows outside [0, src_rows), queries
 * before the slot's first token, rows whose lse is not finite; a head's key that
 * is not finite gathers nothing from that head's queries.  Tokens that no query
 * attends and those whose entry names no page keep what they have.
 * T_tot and max_pages x page_size must be below 2^29, N below 2^23
 * (KDA_ERR_UNSUPPORTED otherwise).
 */
size_t kda_cache_weigh_workspace_bytes(int64_t T_tot, int32_t N, int32_t H, int32_t Hkv);
int kda_cache_weigh(int64_t T_tot, int32_t N, const int32_t* cu_seqlens,
                    int64_t src_rows, const int32_t* rows,
                    int32_t H, int32_t Hkv, int32_t dk, int32_t x_dtype, float scale,
                    int32_t window, int32_t sinks,
                    const void* q, const float* lse,
                    const void* k_cache, int32_t num_pages, int32_t page_size,
                    const int32_t* page_table, int32_t slots, int32_t max_pages,
                    const int32_t* lens, const int32_t* slot_indices,
                    float* weights,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * kda_cache_evict -- cuts slots down to `keep` tokens.  Of a slot that holds
 * more, the first `first` and the last `recent` tokens stay, and of those
 * between them the keep - first - recent that have gathered the largest
 * weights, the earlier of two that are equal (NaN is below every number).  They
 * move to the front of the slot's pages in their order, rows of k_cache and
 * v_cache and their weights; the weights behind them up to the old length
 * become 0, the table's entries behind them -1 and their pages' counts drop by
 * one each; lens becomes keep.  A slot of keep tokens or fewer is left alone.
 * Arguments:
 *   slot_list     int32 [n], n below 2^16 (KDA_ERR_UNSUPPORTED otherwise);
 *   keep          >= 1;   first, recent >= 0, together at most keep;
 *   weights       fp32 [slots, max_pages * page_size], as kda_cache_weigh;
 *   kept          NULL or int32 [n, keep], written: the old places of the tokens
 *                 that the slot holds now, rising, -1 behind them (a refused
 *                 entry: all -1);
 *   status        NULL or int32 [n], written: 0 done, 2 refused;
 *   workspace     at least kda_cache_evict_workspace_bytes(n, keep) bytes,
 *                 256-byte aligned; contents on entry are ignored.
 * Refused, changing nothing: a slot outside [0, slots) or that an earlier entry
 * names; a slot to be cut of which an entry within its length names no page;
 * one where a page that would be written, or a last page that stays partly
 * filled, has another entry that names it (refs above 1): pages of a shared
 * prefix of at most `first` tokens stay shared.  max_pages x page_size must be below
 * 2^29 and Hkv below 2^15 (KDA_ERR_UNSUPPORTED otherwise).
 */
size_t kda_cache_evict_workspace_bytes(int32_t n, int32_t keep);
int kda_cache_evict(int32_t n, const int32_t* slot_list, int32_t keep, int32_t first, int32_t recent,
                    int32_t Hkv, int32_t dk, int32_t dv, int32_t x_dtype,
                    void* k_cache, void* v_cache, int32_t num_pages, int32_t page_size,
                    int32_t* page_table, int32_t slots, int32_t max_pages,
                    int32_t* lens, int32_t* refs,
                    float* weights,
                    int32_t* kept, int32_t* status,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Kernel timing for profiling tools (not needed for normal use).
 * kda_profile_enable(1) makes every later call on the calling host thread
 * bracket each kernel it launches with a pair of HIP events recorded on the
 * call's stream; kda_profile_enable(0) stops it.  kda_profile_collect()
 * waits for the recorded events, sums them per kernel name since the last
 * collect, writes at most max_entries records to `out` and returns the number
 * of distinct kernels (or -KDA_ERR_HIP if an event failed).  Event objects
 * are pooled per thread; no device memory is allocated.
 */
typedef struct kda_kernel_time {
    char name[48];
    int64_t launches;
    double total_ms;
} kda_kernel_time_t;

int kda_profile_enable(int on);
int kda_profile_collect(kda_kernel_time_t* out, int max_entries);

/*
 * Peak-rate probes for measurement tools (not part of the token mixer): what
 * this device sustains, to report beside the published peaks.  Launches
 * `blocks` workgroups of 256 threads on `stream`:
 *   kind 0  each wave issues iters x 4 bf16 matrix-core products of
 *           16 x 16 x 32 (16,384 flops each): blocks * 4 * iters * 4 * 16384
 *           flops in all;
 *   kind 1  the same with fp32 products of 16 x 16 x 4 (2,048 flops each);
 *   kind 2  reads src_bytes (a multiple of 16, 16-byte aligned device memory
 *           at src) once, grid-stride.
 * out: device fp32 [blocks * 256], written (a checksum per thread).  Returns
 * KDA_ERR_INVALID_ARGUMENT for bad arguments.  The launch is timed by
 * kda_profile_enable like any kernel of the library ("probe_mfma_bf16",
 * "probe_mfma_f32", "probe_read").
 */
int kda_probe_peak(int32_t kind, int32_t blocks, int32_t iters, const void* src, int64_t src_bytes,
                   float* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
