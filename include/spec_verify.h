/*
 * spec_verify.h -- C ABI of the target-verification round of speculative
 * decoding on one GB300 (sm_103a).
 *
 * The round (sources, by page title and section):
 *  - "Model-neutral Speculative Decoding", section "The exactness
 *    transaction": evaluate the anchor and the proposal block in one target
 *    pass; sample target rows only through the first mismatch; commit the
 *    accepted prefix; emit exactly one correction or bonus token; for greedy
 *    decoding the speculative and autoregressive token ids match exactly; for
 *    stochastic decoding the target sampler advances once per emitted sample
 *    and never for a rejected suffix.
 *  - "Speculative Decoding (D5-R) -- Plan", section 3 "Mechanism -- one
 *    round": one nt = d+1 forward whose rows are the next token plus the d
 *    drafted candidates at contiguous positions; greedy argmax per verify row,
 *    accept while equal to the drafted token, always emit at least one token;
 *    the target writes d+1 KV rows in place and rejected slots are simply
 *    overwritten next round ("positions are data"); and the status notes on
 *    the weights-once batched verify and bitwise position-invariant verify
 *    attention.
 *  - "DFlash and DSpark Speculative Decoding", "How DSpark Works" and
 *    "Notes": lossless output under the strict rejection sampler (accept with
 *    min(1, p/q), else resample from norm(max(0, p - q))).
 *
 * Conventions for every function below:
 *  - Return value: SPEC_OK (0) or a negative SPEC_E_* code; the message of
 *    the last failure on the calling thread is in spec_last_error().
 *  - Pointers are DEVICE pointers owned by the caller unless a parameter says
 *    "host".  fp16 data is passed as uint16_t (IEEE binary16 bits).  Device
 *    arrays must be 16-byte aligned.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *    enqueued on it asynchronously, except for create/destroy/state calls,
 *    which synchronise.
 *  - On an error return nothing has been enqueued and no state has changed.
 *    Errors that can only be seen on the device (a token id out of range, a
 *    position past max_ctx, a non-finite logit) set the model's device error
 *    word: the round then commits nothing, writes -1 to its n_acc and emitted
 *    outputs, and spec_error_check() reports SPEC_E_INVALID.
 *  - A model or packed matrix is used from one stream at a time.
 *  - The library allocates device memory only in *_create, and, for the
 *    standalone entry points that need scratch, on first use per device
 *    (a cached, growing workspace).
 *  - Two environment variables, read once (at matrix / model creation for
 *    the first, at the first launch for the second), change how kernels are
 *    launched but never what they compute beyond the summation order of
 *    one GEMM's K split:
 *      SPEC_VERIFY_LINEAR_SPLIT  "KW:S" (every matrix) or "N:K:KW:S" entries,
 *        comma-separated: the K split of the verify GEMM (KW warps of a CTA
 *        and S CTAs share a tile's K range) instead of the library's choice.
 *        The split is fixed per matrix, so rows stay bitwise equal across nt
 *        under any setting; results under two settings may differ in the
 *        last bits.  Meant for tests and tuning.
 *      SPEC_VERIFY_PDL=0  launch every kernel as a plain stream-ordered
 *        launch (no programmatic dependent launch).  Results are unchanged.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_OK 0
#define SPEC_E_INVALID (-1)     /* bad argument, token id, non-finite value */
#define SPEC_E_SHAPE (-2)       /* size or alignment precondition violated */
#define SPEC_E_CUDA (-3)        /* a CUDA runtime call failed */
#define SPEC_E_OOM (-4)         /* device allocation failed */
#define SPEC_E_UNSUPPORTED (-5) /* mode not supported: fails closed */
#define SPEC_E_TIMEOUT (-6)     /* a bounded device wait ran out */

#define SPEC_Q4 4 /* 4-bit signed ints in [-8, 7], blocks of 32, fp16 scale */
#define SPEC_Q6 6 /* 6-bit signed ints in [-32, 31], blocks of 32, fp16 scale */
#define SPEC_Q8 8 /* 8-bit signed ints in [-128, 127], blocks of 32, fp16 scale */

#define SPEC_MAX_NT 16 /* rows per sequence in one round: anchor + up to 15 drafts */

/* Copies the last error message of the calling thread into buf. */
void spec_last_error(char* buf, size_t len);

/* ------------------------------------------------------------------------
 * Block-quantised matrix W[N][K] in canonical planes (device, caller-owned):
 *   qs     Q4 / Q6: [N][K/32][16] bytes.  Byte j of block b holds element
 *          32b+j in its low nibble and element 32b+j+16 in its high nibble.
 *          Q4 stores u = q + 8 (the q4_0 element order); Q6 stores the low 4
 *          bits of u = q + 32.
 *          Q8: [N][K/32][32] bytes, byte j of block b = element 32b+j as a
 *          two's-complement int8 (the q8_0 element order).
 *   qh     [N][K/32][8] bytes, Q6 only (NULL for Q4 and Q8): the high 2 bits
 *          of u, element j of the block at bits 2*(j%4) of byte j/4.
 *   scales [N][K/32] fp16.  W[n][k] = scale[n][k/32] * q[n][k].
 * The q4_0 / q8_0 weights of the pages' targets ("Speculative Decoding
 * (D5-R) -- Plan", status notes: the verify machinery extended to q8_0/q4_0)
 * are these planes with each block's scale split out of its bytes.
 * Preconditions: K % 32 == 0, N % 16 == 0.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t qtype; /* SPEC_Q4, SPEC_Q6 or SPEC_Q8 */
  int32_t N, K;
  const void* qs;
  const void* qh;
  const void* scales;
} spec_qweight;

/* A matrix repacked into the streaming layout of the verify GEMM. */
typedef struct spec_qmat spec_qmat;

/* Repacks `w` into a new device-resident matrix (the caller may free the
 * canonical planes after return).  max_rows bounds the nt of later
 * spec_linear_q calls (1..16*1024).  Synchronises `stream`. */
int spec_qmat_create(const spec_qweight* w, int max_rows, void* stream,
                     spec_qmat** out);
int spec_qmat_destroy(spec_qmat* m);

/* Weights-once multi-row dequant GEMM ("Speculative Decoding (D5-R) --
 * Plan", section 1: the batched verify is a weights-once round, not a
 * per-row restream):
 *   y[r][n] = sum_k W[n][k] * x[r][k],  r < nt,
 * x fp16 [nt][K] row-major, y fp32 [nt][N] row-major.  Every row is computed
 * by the same instruction sequence whatever nt is, so row r is bitwise equal
 * to the nt = 1 result for the same x row.  1 <= nt <= max_rows. */
int spec_linear_q(const spec_qmat* w, const uint16_t* x, int nt, float* y,
                  void* stream);

/* The same product on the tensor cores, as multi-sequence rounds run it
 * (tcgen05.mma with tensor-memory accumulators; rows are the N dimension):
 * each weight q * scale enters as an exact pair of fp16 numbers, hi =
 * fp16(q * scale) and lo = q * scale - hi (two MMAs per 16-k step), so every
 * product is exact and only the fp32 accumulation over K rounds.  Every row
 * is computed by the same instructions whatever R is, so a row's result does
 * not depend on the other rows; it differs from spec_linear_q's in the last
 * bits (that kernel accumulates each 32-block's integer sum and applies the
 * scale in fp32).  The matrix's (tile, 64-k chunk) work is cut once, at
 * creation, from N, K and the SM count (never from R): one CTA per tile, a
 * K split, or one run per SM that may cross a tile boundary; a tile cut
 * across CTAs is summed in k order, its CTAs launched cooperatively (all
 * resident).  1 <= R <= max_rows (launched in blocks of 192 rows). */
int spec_linear_q_tc(const spec_qmat* w, const uint16_t* x, int R, float* y,
                     void* stream);

/* ------------------------------------------------------------------------
 * Decoder model: RMSNorm -> QKV + rotate-half RoPE -> causal GQA attention
 * over the KV cache -> O + residual -> RMSNorm -> gate/up + SwiGLU -> down +
 * residual, n_layers times; final RMSNorm; LM head over the full vocabulary.
 * Every linear is a block-quantised matrix of any of the formats above
 * (SPEC_Q4, SPEC_Q6, SPEC_Q8).  Residual stream fp32, activations fp16, KV
 * cache fp16.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t n_layers; /* 0 allowed: LM head only (spec_lm_head) */
  int32_t hidden, n_q_heads, n_kv_heads, head_dim, ffn, vocab;
  int32_t max_ctx;  /* KV positions per sequence (at most 786432) */
  int32_t max_nt;   /* rows per sequence per round, <= SPEC_MAX_NT */
  int32_t max_seqs; /* sequence slots */
  float rms_eps;    /* e.g. 1e-6 */
  float rope_theta; /* e.g. 10000 */
  int32_t use_rope; /* 1: rotate q and new k at their absolute positions */
} spec_model_desc;

typedef struct {
  const uint16_t* embed;      /* fp16 [vocab][hidden] (NULL if n_layers == 0) */
  const float* norm_w;        /* fp32 [2*n_layers+1][hidden]: attn_l, ffn_l ..., final */
  const spec_qweight* wqkv;   /* HOST array [n_layers]; rows [q heads | k heads | v heads] */
  const spec_qweight* wo;     /* HOST array [n_layers]; [hidden][n_q_heads*head_dim] */
  const spec_qweight* wgu;    /* HOST array [n_layers]; rows [gate (ffn) ; up (ffn)] */
  const spec_qweight* wd;     /* HOST array [n_layers]; [hidden][ffn] */
  spec_qweight lm_head;       /* [vocab][hidden] */
} spec_model_weights;

typedef struct spec_model spec_model;

/* Creates a model: repacks all weights, allocates the fp16 KV cache
 * [n_layers][max_seqs][n_kv_heads][max_ctx][head_dim] (zeroed), activation
 * buffers for max_seqs*max_nt rows and the per-sequence state
 * (n_past = 0, emit_idx = 0, anchor = 0).  Synchronises `stream`. */
int spec_model_create(const spec_model_desc* desc, const spec_model_weights* w,
                      void* stream, spec_model** out);
int spec_model_destroy(spec_model* m);

/* Device pointers of layer `layer`'s K and V caches, each
 * [max_seqs][n_kv_heads][max_ctx][head_dim] fp16, for filling a context. */
int spec_model_kv_cache(spec_model* m, int layer, uint16_t** k, uint16_t** v);

/* Copies a context into the cache of slot `seq`, layer `layer`, positions
 * [pos0, pos0 + n_pos): k and v are fp16 [n_kv_heads][n_pos][head_dim]
 * (device or host memory).  Asynchronous on `stream`. */
int spec_kv_fill(spec_model* m, int layer, int seq, int pos0, int n_pos,
                 const uint16_t* k, const uint16_t* v, void* stream);

/* The reverse of spec_kv_fill: copies positions [pos0, pos0 + n_pos) of slot
 * `seq`, layer `layer` out to k and v, fp16 [n_kv_heads][n_pos][head_dim]
 * (device or host memory).  Asynchronous on `stream`. */
int spec_kv_read(spec_model* m, int layer, int seq, int pos0, int n_pos, uint16_t* k,
                 uint16_t* v, void* stream);

/* Diagnostics: copies up to `bytes` of an internal activation buffer of the
 * last target pass to dst (device or host).  which: 0 residual h fp32
 * [R][hidden], 1 normed input fp16 [R][hidden] (after the final norm: the LM
 * head input), 2 SwiGLU output fp16 [R][ffn], 3 attention output fp16
 * [R][n_q_heads*head_dim], 4 rotated q fp16 [R][n_q_heads][head_dim] (the
 * last layer's), 5 logits fp32 [R][vocab].  Asynchronous on `stream`. */
int spec_model_debug_read(spec_model* m, int which, void* dst, size_t bytes, void* stream);

/* Per-sequence transaction state, HOST arrays of n entries for the slots
 * seq_ids[0..n): n_past (committed positions), emit_idx (sampler slot of the
 * next emitted token), anchor (last committed token, row 0 of the next
 * round).  NULL arrays are skipped.  Synchronous. */
int spec_state_set(spec_model* m, int n, const int32_t* seq_ids,
                   const int32_t* n_past, const uint64_t* emit_idx,
                   const int32_t* anchor);
int spec_state_get(spec_model* m, int n, const int32_t* seq_ids, int32_t* n_past,
                   uint64_t* emit_idx, int32_t* anchor);

/* Synchronises `stream`, reads and clears a device error word: the model's
 * (m != NULL), else the one word this device's standalone entry points share
 * (spec_linear_q, spec_accept_*): bit 0x10 there is a weight or activation
 * copy that did not arrive within about a second.
 * Returns SPEC_OK or SPEC_E_INVALID (the bits are stored in *bits if not NULL). */
int spec_error_check(spec_model* m, void* stream, uint32_t* bits);

/* 1 (default): spec_verify_round replays one captured CUDA graph per
 * (n_seq, d, mode) shape -- for a greedy round the whole round, target pass,
 * accept and commit; the caller's arrays are kernel arguments of the graph,
 * updated in place when they change from one call to the next.  0: launches
 * kernels one by one. */
int spec_model_set_graphs(spec_model* m, int enable);

/* Which GEMM a round's linear layers (and LM head) run on is chosen by the
 * round's number of sequences, never by d: rounds of at least `min_seqs`
 * sequences use the tensor-core GEMM of spec_linear_q_tc, the others the
 * GEMM of spec_linear_q.  So a sequence's rows are bitwise the same at every
 * depth d for a given batch size, and greedy speculative decoding of a batch
 * is byte-identical to plain decoding of the same batch.  Default 2; 0 turns
 * the tensor-core GEMM off.  Synchronises the device and drops captured
 * graphs. */
int spec_model_set_tc_min_seqs(spec_model* m, int min_seqs);

/* In-round kernel timing.  enable = 1: the model's later rounds launch their
 * kernels one by one (no graph), with a CUDA event recorded before and after
 * each verify-GEMM launch and each attention launch (chunk + merge kernels);
 * the events see each kernel inside a real round (its inputs written by the
 * kernel before it, the caches as the round leaves them), at the price of
 * the serialisation an event imposes between neighbouring kernels.  Calling
 * it (enable 0 or 1) synchronises the device and clears the totals. */
int spec_model_profile(spec_model* m, int enable);

/* Kernel classes of spec_model_profile_read. */
#define SPEC_PROF_QKV 0       /* QKV GEMM + RoPE + KV write */
#define SPEC_PROF_O 1         /* O GEMM + residual */
#define SPEC_PROF_GATE_UP 2   /* gate/up GEMM + SwiGLU */
#define SPEC_PROF_DOWN 3      /* down GEMM + residual */
#define SPEC_PROF_LM_HEAD 4   /* LM head (+ logits) + argmax */
#define SPEC_PROF_ALL_GEMMS 5 /* classes 0-4 together */
#define SPEC_PROF_ATTN 6      /* verify attention (chunk + merge kernels) */

/* Totals since the last spec_model_profile call for one kernel class (HOST
 * outputs, each may be NULL): summed event-to-event seconds, launches, and
 * the algorithmic bytes (packed weights once, activations in, outputs out;
 * 0 for attention, whose bytes depend on positions held on the device) and
 * flops (2 * rows * N * K) of those launches.  Synchronises the device. */
int spec_model_profile_read(spec_model* m, int kind, double* seconds, int64_t* launches,
                            double* bytes, double* flops);

/* Test hook for the fail-closed path of the verify GEMM's bounded waits.
 * Every wait of a GEMM CTA on its copies (weights and activations, TMA bulk
 * copies completing on an mbarrier) gives up after about a second (131072
 * suspended tries of about 10 us), sets ERR_TIMEOUT (0x10) in the model's
 * error word, waits with the full budget for the copies it issued and
 * finishes without using them, so the round commits nothing and writes -1
 * outputs.  This call sets the try budget of the FIRST wait of each GEMM CTA
 * on its copies (the activation slice of the spec_linear_q kernel, the first
 * weight records of the tensor-core kernel) for the model's later rounds; 0
 * makes that wait give up at once.  Drains always keep the full budget.
 * 0 <= tries <= 131072; synchronises the device and drops captured graphs. */
int spec_model_set_wait_budget(spec_model* m, int tries);

/* Causal GQA attention of nt query rows per sequence over the KV cache of
 * `layer`, bitwise position-invariant: row i of sequence s (absolute
 * position n_past[s] + i) is computed exactly as it would be at nt = 1
 * ("Speculative Decoding (D5-R) -- Plan", status notes: batched verify
 * attention made bitwise position-invariant).  First writes k_new/v_new
 * [n_seq*nt][n_kv_heads][head_dim] at positions n_past..n_past+nt-1 of each
 * sequence; n_past itself is not changed.
 *   seq_ids  device int32 [n_seq] slots;  q fp16 [n_seq*nt][n_q_heads][head_dim]
 *   out      fp16 [n_seq*nt][n_q_heads*head_dim] */
int spec_verify_attn(spec_model* m, int layer, int n_seq, const int32_t* seq_ids,
                     int nt, const uint16_t* q, const uint16_t* k_new,
                     const uint16_t* v_new, uint16_t* out, void* stream);

/* Full-vocabulary LM head: logits[r][v] = sum_k W_lm[v][k] x[r][k] (fp32),
 * with a fused per-row argmax (ties to the lowest id).  x fp16 [R][hidden],
 * R <= max_seqs*max_nt; logits [R][vocab] or NULL; argmax int32 [R] or NULL.
 * A NaN logit sets the device error word. */
int spec_lm_head(spec_model* m, const uint16_t* x, int R, float* logits,
                 int32_t* argmax, void* stream);

/* Greedy accept ("Speculative Decoding (D5-R) -- Plan", section 3):
 *   a = number of leading i < d with argmax[s][i] == draft[s][i];
 *   emitted[s] = draft[s][0..a-1], argmax[s][a], then -1 padding;
 *   n_acc[s] = a.
 * argmax [n_seq][d+1], draft [n_seq][d], emitted [n_seq][d+1]. */
int spec_accept_greedy(const int32_t* argmax, const int32_t* draft, int n_seq,
                       int d, int32_t* n_acc, int32_t* emitted, void* stream);

/* Strict rejection sampling ("DFlash and DSpark Speculative Decoding",
 * "Notes"; sampler-advance rule of "Model-neutral Speculative Decoding", "The
 * exactness transaction").  For each sequence s, slot i < d, draft x:
 *   z = logits / temperature (fp32, round to nearest);
 *   W_v = floor(exp(z_v - max z) * 2^32) (own fp32 exp, identical on every
 *   platform), S = sum W_v; Wq, Sq likewise from q_logits;
 *   U = Philox4x32-10(key = seed, counter = (j lo, j hi, seq_ids[s], 0)) for
 *   the emitted slot j = emit_idx[s] + i;
 *   accept iff U[0] * Wq_x * S < 2^32 * W_x * Sq  (u < p_x / q_x, exact);
 *   on the first rejection resample from R_v = max(0, W_v*Sq - Wq_v*S) with
 *   threshold floor(U[1] * sum R / 2^32) and stop; after d accepts sample the
 *   bonus from row d with floor(U[1] * S / 2^32).
 * emit_idx[s] += n_acc[s] + 1: one sampler slot per emitted token, none for
 * the rejected suffix.
 *   p_logits fp32 [n_seq][d+1][V]; q_logits fp32 [n_seq][d][V] (may be NULL
 *   when d == 0); draft int32 [n_seq][d]; seq_ids int32 [n_seq];
 *   emit_idx uint64 [n_seq] (in/out); n_acc [n_seq]; emitted [n_seq][d+1].
 * Decisions are bit-identical to any correct implementation of the same
 * integer rules on the same fp32 logits. */
int spec_accept_stochastic(const float* p_logits, const float* q_logits,
                           const int32_t* draft, int n_seq, int d, int V,
                           float temperature, uint64_t seed,
                           const int32_t* seq_ids, uint64_t* emit_idx,
                           int32_t* n_acc, int32_t* emitted, void* stream);

/* Same computation, arguments and results as spec_accept_stochastic, but
 * this entry point allocates no memory at all.  It is for callers that cannot
 * call cudaMalloc: code whose device memory is owned by a custom allocator
 * or a fixed arena that forbids outside allocations, and latency-critical
 * loops that must not risk the implicit device synchronisation an
 * allocation can cause.  (The pages have no counterpart for this entry
 * point; it is an addition of this library.)
 *  - Scratch is one fixed array in the library's device globals (about 64 KB
 *    per GPU that loads the library, held until the process exits), so the
 *    batch is limited: n_seq <= 1024 and n_seq * (2d + 1) <= 4096; larger
 *    batches return SPEC_E_SHAPE with a message.  V is limited as for
 *    spec_accept_stochastic.
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress) with that device current; make that first call
 *    before any stream capture.
 *  - All calls share the one array: calls whose work overlaps on the GPU
 *    (different streams, or different host threads) race and must be ordered
 *    by the caller.  Each call clears the array's error word itself.
 *  - Errors seen on the device (non-finite logit, bad draft id) make the
 *    affected outputs -1 and leave emit_idx unchanged, as in
 *    spec_accept_stochastic; spec_error_check does not report them. */
int spec_accept_stochastic_noalloc(const float* p_logits, const float* q_logits,
                                   const int32_t* draft, int n_seq, int d, int V,
                                   float temperature, uint64_t seed,
                                   const int32_t* seq_ids, uint64_t* emit_idx,
                                   int32_t* n_acc, int32_t* emitted, void* stream);

typedef struct {
  int32_t greedy;      /* 1: greedy argmax accept; 0: strict rejection sampling */
  float temperature;   /* stochastic only, > 0 */
  uint64_t seed;       /* stochastic only: Philox key */
} spec_sampling;

/* One verify round ("Model-neutral Speculative Decoding", "The exactness
 * transaction", steps 3-6): rows [anchor, draft[s][0..d-1]] of each sequence
 * at positions n_past..n_past+d in one weights-once target pass (all layers
 * and the LM head), then the accept step, then the commit:
 *   n_past += n_acc + 1, emit_idx += n_acc + 1, anchor = last emitted token.
 * The new KV rows are written in place; rejected rows are overwritten later.
 *   seq_ids int32 [n_seq] (distinct slots < max_seqs: a slot named twice, or
 *   out of range, sets the device error word and the round commits nothing);
 *   draft int32 [n_seq][d];
 *   q_logits fp32 [n_seq][d][vocab] (draft distributions; NULL iff greedy);
 *   sampling: HOST pointer;  n_acc int32 [n_seq]; emitted int32 [n_seq][d+1];
 *   logits_out fp32 [n_seq*(d+1)][vocab] or NULL.
 * 1 <= n_seq <= max_seqs, 0 <= d < max_nt.  All arrays are device memory,
 * read and written in place on `stream`; n_acc and emitted must overlap
 * neither each other nor seq_ids / draft (SPEC_E_INVALID otherwise). */
int spec_verify_round(spec_model* m, int n_seq, const int32_t* seq_ids,
                      const int32_t* draft, int d, const float* q_logits,
                      const spec_sampling* sampling, int32_t* n_acc,
                      int32_t* emitted, float* logits_out, void* stream);

/* The same verify round with seq_ids, draft, n_acc and emitted in HOST
 * memory (any host memory; shapes as for spec_verify_round).  q_logits may
 * be device memory or host memory; host q_logits (pinned for full copy
 * bandwidth) are copied into a buffer the model allocated at creation, on a
 * stream of the model's own, while the round's target pass (which does not
 * read them) runs; the accept waits for the copy.
 * The small inputs are copied into the model's mapped pinned staging, which
 * the kernels read and write in place (no copy engine steps; a greedy round
 * with graphs on is one graph launch); the
 * call synchronises `stream` before it copies the outputs out, so they are
 * valid on return.  Calls on one model must not overlap (the staging is the
 * model's).  Errors: as spec_verify_round, plus SPEC_E_CUDA from the
 * synchronisation. */
int spec_verify_round_host(spec_model* m, int n_seq, const int32_t* seq_ids,
                           const int32_t* draft, int d, const float* q_logits,
                           const spec_sampling* sampling, int32_t* n_acc,
                           int32_t* emitted, void* stream);

/* ---------------------------------------------------------------------------
 * Adaptive draft depth: a host controller that picks the depth d of the next
 * verify round ("Speculative Decoding (D5-R) -- Plan", status notes, which
 * list the ingredients: smoothed acceptance estimates, a window of measured
 * round costs, hysteresis, trying unmeasured depths first, a cap on d; the
 * rules below are this library's reading).  Host only: no GPU work, no
 * stream, no model.
 *  - Position i = 1..d_max keeps decayed Beta counts (a_i, b_i).  A round at
 *    depth d in which a sequence accepted n drafts adds 1 to a_i for
 *    i <= min(n, d) and, if n < d, 1 to b_{n+1}; a negative n (a failed
 *    sequence) adds nothing.  All counts are first multiplied by `decay`.
 *  - p_i = (a_i + prior_accept) / (a_i + b_i + prior_accept + prior_reject)
 *    (prior_reject = 0: a position never observed has p_i = 1).
 *  - E(d) = sum_{k=0..d} prod_{i<=k} p_i tokens per round; c(d) = the
 *    minimum of the depth's last `cost_window` round times; r(d) = E / c.
 *  - While some depth in [d_min, d_max] has no round time, the deepest such
 *    depth is next (its r counts as +infinity).  Otherwise the smallest
 *    depth of maximal r replaces the current depth when its r exceeds the
 *    current r by the factor (1 + hysteresis).  The first depth is d_max.
 * Every double is rounded operation by operation, as written above. */
typedef struct {
  int32_t d_min, d_max;       /* 0 <= d_min <= d_max <= SPEC_MAX_NT - 1 */
  double prior_accept;        /* >= 0 */
  double prior_reject;        /* >= 0; prior_accept + prior_reject > 0 */
  double decay;               /* (0, 1] */
  double hysteresis;          /* >= 0 */
  int32_t cost_window;        /* 1..64 round times per depth */
} spec_depth_params;
typedef struct spec_depth_ctl spec_depth_ctl;

/* Defaults: d in [1, 7], prior (1, 0), decay 0.95, hysteresis 0.10, window 4. */
void spec_depth_params_default(spec_depth_params* p);
/* params NULL = the defaults.  SPEC_E_INVALID on a parameter out of range. */
int spec_depth_ctl_create(const spec_depth_params* params, spec_depth_ctl** out);
int spec_depth_ctl_destroy(spec_depth_ctl* c);
/* The depth of the next round. */
int spec_depth_ctl_next(const spec_depth_ctl* c, int32_t* d);
/* A finished round: its depth d (in [d_min, d_max]), the n_seq accepted
 * counts (HOST int32, e.g. spec_verify_round's n_acc copied back) and its
 * time in seconds (finite, > 0).  *next_d (may be NULL) gets the next depth.
 * SPEC_E_SHAPE / SPEC_E_INVALID leave the controller unchanged. */
int spec_depth_ctl_observe(spec_depth_ctl* c, int32_t d, int32_t n_seq, const int32_t* n_acc,
                           double round_seconds, int32_t* next_d);
/* Diagnostics: p[0..d_max] (p[0] = 1) and r[0..d_max] (0 below d_min,
 * +infinity for depths without a round time); either may be NULL. */
int spec_depth_ctl_estimates(const spec_depth_ctl* c, double* p, double* r);

/* ===========================================================================
 * Drafted trees: instead of one chain of drafts per sequence, the target
 * evaluates a tree of candidates (several tokens per position) in one pass,
 * and the accepted root-to-node path is committed.  The operators below are
 * the steps of such a round outside the linear layers: sampling candidates
 * (spec_sample), attention of the tree's nodes over the cache
 * (spec_tree_attn), acceptance along the tree (spec_accept_tree) and the
 * cache's pages (spec_pages_*).
 *
 * They allocate nothing and keep nothing between calls: scratch is the
 * caller's, errors seen on the device go to the caller's `status` array, and
 * calls may run at the same time on several streams, or be captured into
 * graphs, as long as the arrays that they write are not shared.
 * ======================================================================== */

/* A KV cache in pages (HOST struct of DEVICE pointers, all caller-owned; the
 * struct is read during the call only).  Position p of slot s lives in row
 * p % page_size of page table[s][p / page_size], in every layer.  A page is
 * free when its reference count is zero; a page that several slots hold
 * (after spec_pages_fork) is never written. */
typedef struct {
  uint16_t* k; /* fp16 [n_layers][n_pages][n_kv_heads][page_size][head_dim] */
  uint16_t* v; /* the same layout; both 16-byte aligned */
  int64_t layer_stride; /* elements from one layer to the next (>= a layer's, a multiple of 8) */
  int32_t n_layers, n_pages, n_kv_heads, page_size;
  int32_t head_dim;     /* a multiple of 8 (spec_tree_attn: 64 or 128) */
  int32_t n_slots, max_pages;
  int32_t* table; /* [n_slots][max_pages] page ids, -1 from the first entry without a page on */
  int32_t* refs;  /* [n_pages] slots that hold the page; NULL: pages fixed to their slots */
  int32_t* len;   /* [n_slots] committed positions */
} spec_pages;

/* Bits of a `status` entry (0: done).  An entry of a call whose status is not
 * 0 has changed nothing; the call's other entries are done all the same,
 * unless the function says otherwise. */
#define SPEC_ST_SLOT 1   /* slot or page id out of range, or named where it must not be */
#define SPEC_ST_PAGE 2   /* the table has no valid page where one is needed */
#define SPEC_ST_SHARED 4 /* the page is held by another slot */
#define SPEC_ST_FULL 8   /* not enough free pages, or more positions than max_pages hold */
#define SPEC_ST_TREE 16  /* bad parents, node count or path */
#define SPEC_ST_TIMEOUT 32 /* a bounded device wait ran out */
#define SPEC_ST_BLOCK 64   /* a block that the sequence does not have */

#define SPEC_MAX_TREE 64 /* nodes of a tree */

/* The model's own cache as pages: one page of max_ctx positions per slot
 * (page id = slot), table, and len = the model's n_past; refs is NULL, so
 * fork, extend and free refuse it (SPEC_E_UNSUPPORTED), and its pages are
 * copied from slot to slot by spec_pages_copy.  What spec_pages_commit
 * writes is what the model's later rounds read; of the slot's state it advances
 * n_past alone, so that a program that goes on with spec_verify_round there
 * sets anchor (the last emitted token, whose key and value are not in the cache
 * yet) and emit_idx with spec_state_set first. */
int spec_model_pages(spec_model* m, spec_pages* out);

/* Copies page src[i] to page dst[i] in every layer, i < n (device int32 [n]):
 * the first n_pos[i] positions of it (device int32 [n], 0 <= n_pos <=
 * page_size), or all of them if n_pos is NULL.  A dst that is named twice or
 * is also a src is refused (SPEC_ST_SLOT), each entry that names it.
 * Reference counts and tables are not looked at. */
int spec_pages_copy(const spec_pages* kv, int n, const int32_t* src, const int32_t* dst,
                    const int32_t* n_pos, int32_t* status, void* stream);

/* Slot dst[i] becomes a branch of slot src[i] (device int32 [n]): it gets the
 * src's length and shares the pages of its committed positions.  dst must
 * hold no pages, and appear neither twice nor as a src (SPEC_ST_SLOT); src
 * may be named any number of times. */
int spec_pages_fork(const spec_pages* kv, int n, const int32_t* src, const int32_t* dst,
                    int32_t* status, void* stream);

/* Makes positions [len, len + n_new[i]) of slot slots[i] writable (device
 * int32 [n], slots distinct, n <= 1024): the missing pages are taken, and a
 * partly filled last page that other slots hold too is replaced by a page of
 * its own with the filled positions copied -- the last of its holders, when
 * all of them are extended in one call, keeps it.  The pages taken are the
 * lowest free ones, in the order of the entries, an entry's copy before its
 * further pages: the result is a function of the arrays alone.  When the
 * free pages do not suffice for every entry that is in order, none gets any
 * (SPEC_ST_FULL).  copies int32 [n][2]: (page, its copy) of each entry, or
 * (-1, -1).  A shared page behind the last committed position (possible only
 * if len was lowered) is refused (SPEC_ST_SHARED). */
int spec_pages_extend(const spec_pages* kv, int n, const int32_t* slots, const int32_t* n_new,
                      int32_t* copies, int32_t* status, void* stream);

/* Commits rows of new keys and values behind a slot's committed positions, in
 * every layer: position len + j of slot slots[i] gets row path[i][j] of entry
 * i, j < n_path[i] (device; slots distinct; path int32 [n][nt], or NULL for
 * rows 0, 1, ...; 0 <= n_path <= nt).  With the path of spec_accept_tree this
 * compacts the accepted nodes of a tree into the cache; with path NULL it
 * appends a prompt.
 *   k_new, v_new  fp16 [n_layers][n][nt][n_kv_heads][head_dim], 16-byte
 *                 aligned; new_layer_stride elements from one layer to the
 *                 next (0: contiguous; a multiple of 8)
 *   new_len       int32 [n_slots]: new_len[slot] = len[slot] + n_path for the
 *                 call's slots; NULL: len itself, advanced in place
 * The pages must be there (spec_pages_extend) and held by this slot alone. */
int spec_pages_commit(const spec_pages* kv, int n, const int32_t* slots, int nt,
                      const uint16_t* k_new, const uint16_t* v_new, int64_t new_layer_stride,
                      const int32_t* path, const int32_t* n_path, int32_t* new_len,
                      int32_t* status, void* stream);

/* Gives back every page of the slots (device int32 [n], distinct) and sets
 * their length to 0.  Ids out of range in a slot's row of the table are
 * dropped (SPEC_ST_PAGE, the slot is empty all the same). */
int spec_pages_free(const spec_pages* kv, int n, const int32_t* slots, int32_t* status,
                    void* stream);

/* The trees of one round: n_seq sequences of up to nt nodes. */
typedef struct {
  int32_t n_seq, nt;       /* 1 <= nt <= SPEC_MAX_TREE */
  int32_t n_q_heads;       /* a positive multiple of the cache's n_kv_heads */
  int32_t window;          /* 0: every earlier position is visible; w > 0: the last w are */
  int32_t sinks;           /* with a window: the first `sinks` positions stay visible too */
  float scale;             /* of the scores; 0: 1 / sqrt(head_dim) */
  const int32_t* slots;    /* device [n_seq]; a slot may be named more than once */
  const int32_t* parents;  /* device [n_seq][nt]: an earlier node, or -1 (child of the
                              committed context); NULL: a chain, parent i - 1 */
  const int32_t* n_nodes;  /* device [n_seq], 0 <= n_nodes <= nt; NULL: nt each */
} spec_tree;

/* Attention of the trees' nodes over the committed cache of `layer` and over
 * themselves.  Node i of a sequence sits at position P_i = len + depth_i (a
 * child of the context has depth 0) and sees the committed positions p < len
 * and, of the nodes, itself and its ancestors; with a window w, of all these
 * only positions p < sinks or p > P_i - w.  q, k_new are already rotated to
 * P_i.  The cache is not written (spec_pages_commit does that for the
 * accepted path).
 *   q      fp16 [n_seq][nt][n_q_heads][head_dim], q_stride elements from one
 *          node's row to the next (0: contiguous)
 *   k_new, v_new  fp16 [n_seq][nt][n_kv_heads][head_dim], kv_stride elements
 *          from one node's row to the next (0: contiguous); strides are
 *          multiples of 8, so the rows may be parts of a fused QKV buffer
 *   out    fp16 [n_seq][nt][n_q_heads * head_dim]; rows of nodes >= n_nodes
 *          are left as they were; rows of a sequence whose status is not 0
 *          are NaN (for its first n_nodes rows, all nt if that is bad too)
 *   workspace  spec_tree_attn_workspace bytes, 16-byte aligned; its contents
 *          do not matter before and after the call
 *   status int32 [n_seq]: SPEC_ST_SLOT, SPEC_ST_PAGE, SPEC_ST_TREE,
 *          SPEC_ST_TIMEOUT
 * out and workspace overlap none of the inputs, nor each other.
 * The scores' statistics and sums are fp32, and the weights are multiplied as
 * pairs of fp16 numbers (2^-20 of a weight, 2^-36 of the row's largest), for any
 * number of rows.  The same call gives the same bits; which bits may depend on the other sequences of the call (the work
 * is cut evenly over the SMs), unlike spec_verify_attn, whose rows do not
 * depend on the batch. */
int spec_tree_attn(const spec_pages* kv, int layer, const spec_tree* t, const uint16_t* q,
                   int64_t q_stride, const uint16_t* k_new, const uint16_t* v_new,
                   int64_t kv_stride, uint16_t* out, void* workspace, size_t workspace_bytes,
                   int32_t* status, void* stream);

/* Bytes of workspace for spec_tree_attn on the current device (any slots,
 * lengths and trees of up to n_seq sequences of up to nt nodes). */
int spec_tree_attn_workspace(const spec_pages* kv, int n_seq, int nt, int n_q_heads,
                             size_t* bytes);

/* Test hook for the fail-closed path of spec_tree_attn's bounded waits (of the
 * kernel for more than 32 query rows a kv head).  A wait that gives up (131072
 * suspended tries of about 10 us) ends its CTA's loads and products; the CTA
 * lets those in flight end, and the sequences that it works on get
 * SPEC_ST_TIMEOUT and NaN.  This call sets the budget of the first wait of
 * each CTA's softmax for the calling thread's later calls (a captured call
 * keeps the one it was captured with); 0 makes that wait give up at once.
 * 0 <= tries <= 131072. */
int spec_tree_set_wait_budget(int tries);

/* Greedy acceptance along the trees: from node 0 (the anchor, parent -1), the
 * target's argmax at the current node selects the child that carries that
 * token (the lowest numbered of several), until none does.
 *   argmax, tokens, parents  int32 [n_seq][nt] (tokens[s][0], the anchor, is
 *          not looked at); n_nodes int32 [n_seq] or NULL; nt <= SPEC_MAX_TREE
 *   path   int32 [n_seq][nt]: node 0, then the accepted nodes, -1 behind
 *   n_path int32 [n_seq]: nodes in the path (1 + accepted drafts); 0 for a
 *          sequence without nodes, -1 for a tree that is not one (a parent
 *          not below its node, a count outside [0, nt], parent of node 0
 *          not -1): path and emitted are -1 then
 *   emitted int32 [n_seq][nt]: the accepted tokens, then the target's token
 *          at the last accepted node (n_path in all), -1 behind */
int spec_accept_tree(const int32_t* argmax, const int32_t* tokens, const int32_t* parents,
                     const int32_t* n_nodes, int n_seq, int nt, int32_t* path, int32_t* n_path,
                     int32_t* emitted, void* stream);

/* The value of a filtered-out logit: finite, with weight 0 at any temperature. */
#define SPEC_FILTERED (-3.402823466e+38f)

/* Samples one token per row from given random words, after temperature,
 * top-k, top-p and min-p, on the rejection sampler's integer weights
 * (spec_accept_stochastic): z = l / T, W_v = floor(exp(z_v - max z) * 2^32).
 * Tokens are ordered by logit, the largest first, equal logits by id.
 *   1. a logit of -infinity is never kept;
 *   2. top_k > 0: the first top_k tokens stay (T == 0: the first one);
 *   3. top_p < 1: of these, token j stays iff the weights before it sum to
 *      less than floor(top_p * 2^32) / 2^32 of their total, or it is the
 *      first;
 *   4. of these, tokens with W < floor(min_p * 2^32) go;
 *   5. the token drawn is the first kept id, in the order of ids, at which
 *      the running sum of the kept weights exceeds floor(u * total / 2^32).
 * All of it is integer arithmetic: results are bit-identical to any correct
 * implementation of these rules.
 *   logits  fp32 [R][V], V <= 1048512, ld elements from row to row (0: V)
 *   u       32-bit random words [R]
 *   temperature, top_k, top_p, min_p  per row, fp32 / int32 [R]; each may be
 *           NULL (1, 0 = off, 1 = off, 0 = off).  T >= 0 finite, top_k >= 0,
 *           0 <= top_p <= 1, 0 <= min_p <= 1
 *   token   int32 [R]
 *   n_kept  int32 [R] or NULL: the tokens that stayed
 *   filtered  fp32 [R][V] or NULL, ld_filtered elements from row to row (0:
 *           V): the logits that stayed, SPEC_FILTERED elsewhere; may be
 *           `logits` itself (with the same ld).  Given to
 *           spec_accept_stochastic as p_logits / q_logits, filtered rows
 *           make its rejection sampling lossless for the filtered
 *           distributions
 *   workspace  spec_sample_workspace bytes, 16-byte aligned (NULL if that is
 *           0: few or short rows); its contents do not matter before and
 *           after the call
 * A row with a NaN or +infinity, without any finite logit, whose largest
 * l / T overflows, or with a setting out of range gets token -1, n_kept 0 and
 * a filtered row of NaN (which spec_accept_stochastic refuses). */
int spec_sample(const float* logits, int R, int V, int64_t ld, const uint32_t* u,
                const float* temperature, const int32_t* top_k, const float* top_p,
                const float* min_p, int32_t* token, int32_t* n_kept, float* filtered,
                int64_t ld_filtered, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace for spec_sample of R rows of V logits (0: none needed;
 * many long rows are sampled in passes over all of them, few in one kernel:
 * the same results). */
int spec_sample_workspace(int R, int V, size_t* bytes);

/* ===========================================================================
 * Long contexts: a cache held in 4 bits, and attention over the blocks of a
 * cache that a cheap score selects for each query.  As the operators above,
 * these allocate nothing and keep nothing between calls, report errors seen on
 * the device in the caller's `status`, and may run at the same time on several
 * streams, or be captured, as long as the arrays that they write are not shared.
 * ======================================================================== */

/* A KV cache in pages whose rows are held in 4 bits: each 32 neighbouring
 * elements of a row are 16 bytes of codes and one fp16 scale, laid out as in
 * SPEC_Q4 (byte j: element j in the low nibble, element j + 16 in the high one;
 * u = q + 8), and an element's value is scale * q, q in [-8, 7].
 * spec_pages_q4_commit makes scales of at most eight significant bits, with
 * which every value is exact in fp16; other scales are taken, too, their
 * values then being rounded to fp16 where rows are attended to or read (above
 * 8188 to infinities where the product passes fp16's range).  An infinite or NaN
 * scale makes its elements infinite or NaN.  Rows that do not see a position know
 * nothing of its scale. */
typedef struct {
  uint8_t* k_qs; /* [n_layers][n_pages][n_kv_heads][page_size][head_dim / 32][16] */
  uint8_t* v_qs;
  uint16_t* k_scales; /* fp16 [n_layers][n_pages][n_kv_heads][page_size][head_dim / 32] */
  uint16_t* v_scales; /* all four 16-byte aligned */
  int64_t layer_stride; /* rows (of head_dim / 32 blocks) from one layer to the next (>= a layer's) */
  int32_t n_layers, n_pages, n_kv_heads, page_size;
  int32_t head_dim;     /* a multiple of 32 (attention: 64 or 128) */
  int32_t n_slots, max_pages;
  int32_t* table; /* these as in spec_pages */
  int32_t* refs;
  int32_t* len;
} spec_pages_q4;

/* spec_pages_copy, _fork, _extend and _free for a cache in 4 bits: the same
 * arguments, rules and status bits.  (A page's digests, below, are not copied with
 * it.) */
int spec_pages_q4_copy(const spec_pages_q4* kv, int n, const int32_t* src, const int32_t* dst,
                       const int32_t* n_pos, int32_t* status, void* stream);
int spec_pages_q4_fork(const spec_pages_q4* kv, int n, const int32_t* src, const int32_t* dst,
                       int32_t* status, void* stream);
int spec_pages_q4_extend(const spec_pages_q4* kv, int n, const int32_t* slots, const int32_t* n_new,
                         int32_t* copies, int32_t* status, void* stream);
int spec_pages_q4_free(const spec_pages_q4* kv, int n, const int32_t* slots, int32_t* status,
                       void* stream);

/* spec_pages_commit into a cache in 4 bits: the same arguments, rules and status
 * bits; the fp16 rows are quantised on their way.  Of 32 elements x, m is the
 * one of the largest magnitude (the first of several):
 *   scale = -m / 8, rounded to eight significant bits (to even) and then to fp16,
 *           its magnitude at most 8160; +0 where that is 0;
 *   q     = x / scale (fp32), rounded to a whole number (to even), kept in [-8, 7];
 *           0 where the scale is 0.
 * Elements that are not all finite get a NaN for their scale (and q = 0): whoever
 * sees them gets a NaN. */
int spec_pages_q4_commit(const spec_pages_q4* kv, int n, const int32_t* slots, int nt,
                         const uint16_t* k_new, const uint16_t* v_new, int64_t new_layer_stride,
                         const int32_t* path, const int32_t* n_path, int32_t* new_len,
                         int32_t* status, void* stream);

/* The reverse: position pos0[i] + j of slot slots[i], j < n_pos[i], as fp16 into
 * row j of entry i, every layer (device int32 [n]; 0 <= n_pos <= nt; a slot may
 * be named more than once).
 *   k, v  fp16 [n_layers][n][nt][n_kv_heads][head_dim], 16-byte aligned;
 *         rows j >= n_pos, and those of an entry whose status is not 0, are left
 *         as they were.  layer_stride elements from one layer to the next (0:
 *         contiguous; a multiple of 8)
 * The pages have to be there (SPEC_ST_PAGE); len is not looked at.  SPEC_ST_SLOT:
 * a slot out of range; SPEC_ST_TREE: n_pos outside [0, nt]; SPEC_ST_FULL: positions
 * below 0 or past what max_pages hold. */
int spec_pages_q4_read(const spec_pages_q4* kv, int n, const int32_t* slots, int nt,
                       const int32_t* pos0, const int32_t* n_pos, uint16_t* k, uint16_t* v,
                       int64_t layer_stride, int32_t* status, void* stream);

/* spec_tree_attn over a cache in 4 bits: the same arguments and rules.  The
 * trees' own keys and values, q and out are fp16.  With up to 32 query rows a kv
 * head (nodes x query heads of it) keys are multiplied as they are, code by code,
 * with the scale in fp32, and values as fp16; with more, both as fp16 (and
 * spec_tree_set_wait_budget holds). */
int spec_tree_attn_q4(const spec_pages_q4* kv, int layer, const spec_tree* t, const uint16_t* q,
                      int64_t q_stride, const uint16_t* k_new, const uint16_t* v_new,
                      int64_t kv_stride, uint16_t* out, void* workspace, size_t workspace_bytes,
                      int32_t* status, void* stream);

/* Bytes of workspace for spec_tree_attn_q4 on the current device. */
int spec_tree_attn_q4_workspace(const spec_pages_q4* kv, int n_seq, int nt, int n_q_heads,
                                size_t* bytes);

/* The digests of a cache's blocks: `block` neighbouring positions of a page (16,
 * 32, 64 or 128, a divisor of page_size) have the least and the largest value of
 * every channel of their keys, in every layer and kv head.  Beside the cache, and
 * addressed by its table: a page that several slots share has one digest. */
typedef struct {
  uint16_t* data; /* fp16 [n_layers][n_pages][n_kv_heads][page_size / block][2][head_dim], 16-byte
                     aligned: the least values, then the largest */
  int64_t layer_stride; /* elements from one layer to the next (>= a layer's, a multiple of 8) */
  int32_t n_layers, n_pages, n_kv_heads, page_size; /* the cache's */
  int32_t head_dim;     /* 64 or 128 */
  int32_t block;
  int32_t n_slots, max_pages;
  const int32_t* table; /* the cache's */
  const int32_t* len;
} spec_digest;

/* Digests of the blocks that hold positions [pos0[i], len) of slot slots[i], in
 * every layer, from all committed positions of these blocks (device int32 [n];
 * pos0 NULL: from 0 on; the last block may be filled partly).  After a commit pos0 is the length in
 * front of it; after an extension with a copy of a page it is the start of that
 * page.  A NaN among a channel's keys makes both of its values NaN.  `kv` has the
 * digest's sizes and a layer stride of whole rows (its table and len are not looked at).  Slots may be named more than once.
 * status: SPEC_ST_SLOT (slot out of range), SPEC_ST_FULL (pos0 below 0, or a length that the table cannot
 * have), SPEC_ST_PAGE (no valid page for some block; the others are done). */
int spec_block_digest(const spec_digest* dg, const spec_pages* kv, int n, const int32_t* slots,
                      const int32_t* pos0, int32_t* status, void* stream);
int spec_block_digest_q4(const spec_digest* dg, const spec_pages_q4* kv, int n, const int32_t* slots,
                         const int32_t* pos0, int32_t* status, void* stream);

/* Scores of every block of `layer` for each node's query: the largest logit that
 * any key between the block's least and largest values could have with any of the
 * kv head's query heads,
 *   scores[s][i][h][j] = max over the heads g of h: sum_d max(q_gd lo_jd, q_gd hi_jd)
 * (without the softmax's scale; fp32 sums), for the blocks j that hold positions
 * [0, len).  An infinite or NaN digest or query makes the scores that it has a part in
 * infinite or NaN.  For a negative softmax scale, pass -q.
 *   slots, n_nodes  as in spec_tree; at most 64 query heads a kv head
 *   q       fp16 as in spec_tree_attn
 *   scores  fp32 [n_seq][nt][n_kv_heads][ld]; what no block stands for, and rows of nodes >=
 *           n_nodes, is left as it was
 *   status  int32 [n_seq]: SPEC_ST_SLOT, SPEC_ST_TREE (node count), SPEC_ST_FULL (a length that
 *           the table cannot have, or more blocks than ld): no scores are written;
 *           SPEC_ST_PAGE (no valid page for some block, whose scores are -infinity) */
int spec_block_scores(const spec_digest* dg, int layer, int n_seq, const int32_t* slots, int nt,
                      const int32_t* n_nodes, int n_q_heads, const uint16_t* q, int64_t q_stride,
                      float* scores, int64_t ld, int32_t* status, void* stream);

/* The blocks that each row of scores selects: the first n_first and the last n_last
 * of the blocks that hold positions [0, len), and of the others those with the
 * largest scores, n_keep in all (all blocks if there are no more).  Equal scores:
 * the lowest block; a NaN counts as +infinity, -0 as 0.
 *   len     int32 [n_slots], slots and n_nodes as above, scores fp32 [n_seq][nt][n_kv_heads][ld]
 *   blocks  int32 [n_seq][nt][n_kv_heads][n_keep]: ascending, -1 behind; rows of nodes >=
 *           n_nodes are left as they were
 *   status  int32 [n_seq]: SPEC_ST_SLOT, SPEC_ST_TREE (node count), SPEC_ST_FULL (a length
 *           below 0, or more blocks than ld): the rows are -1 then
 * 1 <= n_keep <= 4096, n_first + n_last <= n_keep.  A row is read by as many threads as
 * ld asks for: an ld not far above the most blocks of a sequence is the fastest. */
int spec_block_select(const int32_t* len, int n_slots, int block, int n_seq, const int32_t* slots,
                      int nt, const int32_t* n_nodes, int n_kv_heads, const float* scores, int64_t ld,
                      int n_keep, int n_first, int n_last, int32_t* blocks, int32_t* status,
                      void* stream);

/* Attention of the trees' nodes over the committed positions of selected blocks, a
 * list for each node and kv head, and over themselves (a node sees itself and its
 * ancestors), otherwise as spec_tree_attn.
 *   t       window has to be 0 (SPEC_E_UNSUPPORTED: the lists take its place)
 *   blocks  int32 [n_seq][nt][n_kv_heads][n_keep], n_keep <= 4096: blocks of `block` positions
 *           (16, 32, 64 or 128, a divisor of page_size), -1: none.  A block that is named twice
 *           counts twice
 *   status  int32 [n_seq][nt][n_kv_heads]: SPEC_ST_SLOT, SPEC_ST_PAGE, SPEC_ST_TREE, and
 *           SPEC_ST_BLOCK for a block outside [0, len); the query heads of such a row are NaN.
 *           Rows of nodes >= n_nodes of status and out are left as they were (bad counts: all
 *           nt rows are NaN with SPEC_ST_TREE)
 * An infinite or NaN value in a row that a node sees makes its result infinite or NaN in that
 * channel; rows past len, and those of blocks on no list, may hold anything.
 * out overlaps none of the inputs.  A row's bits do not depend on the call's other rows, but
 * they may on how many there are. */
int spec_block_attn(const spec_pages* kv, int layer, const spec_tree* t, int block, int n_keep,
                    const int32_t* blocks, const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                    const uint16_t* v_new, int64_t kv_stride, uint16_t* out, int32_t* status,
                    void* stream);
int spec_block_attn_q4(const spec_pages_q4* kv, int layer, const spec_tree* t, int block, int n_keep,
                       const int32_t* blocks, const uint16_t* q, int64_t q_stride,
                       const uint16_t* k_new, const uint16_t* v_new, int64_t kv_stride,
                       uint16_t* out, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_VERIFY_H */
