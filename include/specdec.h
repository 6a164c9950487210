/*
 * specdec -- the draft-sample-and-verify step of block-parallel speculative
 * decoding on NVIDIA B200 (sm_100a), as a C-ABI library (libspecdec.so).
 *
 * The step (pages: aigest.pl "DeepSeek prezentuje DSpark"; telemetr.me DFlash
 * post; mkdocs.reaper.mx DeepSeek-V4.1-Flash "06-extensions", DSpark table):
 *   a parallel drafter gives base logits for K block positions in one pass;
 *   a sequential Markov head adds bias_i = U[prev] . W (rank r) before each
 *   draft token is sampled, prev being the last committed token for i = 0 and
 *   the previous draft token after that ("Innowacje w tworzeniu tokenów");
 *   the target's K+1 logit rows then verify the block by rejection sampling:
 *   the longest accepted prefix plus one extra token, with the target
 *   distribution preserved exactly ("Jak działa spekulatywne dekodowanie").
 *   Accept d_i iff u < min(1, p_i(d_i)/q_i(d_i)); at the first rejection emit
 *   a draw from max(p_i - q_i, 0) normalised (p_i if that is all zero); if all
 *   K pass, emit a bonus draw from target row K.  Greedy mode drafts arg-max
 *   tokens and accepts while arg-max(target_i) equals d_i.  tau = accepted + 1
 *   is the quantity in L = (T_draft + T_verify) / tau.
 *   p = softmax(target / T), q = softmax((base + bias) / T).
 *
 * Random numbers: Philox4x32-10 (Salmon et al., SC'11), key = seed,
 * counter = (position, row_offset + batch row, lo32(cycle), tag | bits 32..47 of cycle << 16),
 * word 0 mapped to [0,1) as (x >> 8) * 2^-24; tag 0 = draft draw, 1 = accept
 * test, 2 = residual or bonus draw.  Sampling is by inverse CDF in ascending
 * token order: the first token whose inclusive prefix mass exceeds u * total.
 * Ties in arg-max go to the lowest index.
 *
 * Layouts (row-major, V contiguous, caller-owned device memory):
 *   base        [B, K, V]    dtype        draft base logits
 *   target      [B, K+1, V]  dtype        target logits, row K = bonus row
 *   U           [V, r]       dtype        Markov factor, row = previous token
 *   W           [r, V]       dtype        Markov factor
 *   last_token  [B]          int32        last committed token
 *   draft       [B, K]       int32        draft tokens d_i
 *   out         [B, K+1]     int32        emitted tokens; entries >= tau are -1
 *   tau         [B]          int32        1 .. K+1
 *   p_draft     [B, K]       float        p_i(d_i) where the accept test ran, NaN after
 *   q_draft     [B, K]       float        q_i(d_i)
 *   biased_out  [B, K, V]    float        z = base + bias (optional)
 * dtype is SPEC_BF16 (bf16 logits and factors; bias products on tcgen05
 * tensor cores, fp32 accumulate) or SPEC_F32 (fp32 throughout).  All
 * arithmetic after loading is fp32.  In greedy mode p_draft / q_draft are
 * filled with NaN.
 *
 * Calls are asynchronous on `stream`.  Errors found on the host (bad sizes,
 * NULL pointers, a workspace too small) are returned before anything is
 * launched.  Errors found on the device (a token id out of range, a wait that
 * ran past spin_limit polls) are recorded in the workspace and returned by
 * spec_sync_status().  Every device-side wait is bounded; a kernel that gives
 * up records SPEC_ERR_TIMEOUT and returns, leaving the outputs undefined.
 * One workspace serves one stream at a time; calls that share a workspace
 * must be ordered on one stream.
 */
#ifndef SPECDEC_H
#define SPECDEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st *spec_stream_t; /* same type as cudaStream_t */

typedef enum {
  SPEC_OK = 0,
  SPEC_ERR_INVALID_ARG = -1,   /* NULL pointer, size out of range, bad temperature */
  SPEC_ERR_UNSUPPORTED = -2,   /* shape the kernels do not handle (message says which) */
  SPEC_ERR_CUDA = -3,          /* a CUDA runtime call failed */
  SPEC_ERR_TIMEOUT = -4,       /* a device-side wait exceeded spin_limit polls */
  SPEC_ERR_WORKSPACE = -5,     /* workspace NULL, too small or misaligned */
  SPEC_ERR_TOKEN_RANGE = -6    /* a token id (last_token / draft) outside [0, V) */
} spec_status;

typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1 } spec_dtype;

/* Flags */
#define SPEC_FLAG_FMA_BIAS 1u  /* compute the Markov bias with fp32 FMAs instead of tensor cores */
#define SPEC_FLAG_TRACE 2u     /* spec_cycle / spec_markov_bias_sample: record a device timeline.
                                  CTA 0 writes %globaltimer (ns) into the workspace at byte offset
                                  256 as uint64 [K+2][32]: row i < K = draft step i (slots: 0 start,
                                  1 rows gathered, 2 epilogue done, 3 partials published, 4 target
                                  rows streamed, 5 barrier passed, 6 partials combined, 7 owner
                                  draws done, 8 tokens known; 9..31 finer diagnostics: tensor-core
                                  issue, wait totals, per-chunk times), row K = final step, row
                                  K+1 = prologue.  Only the first batch group is recorded. */

typedef struct {
  int32_t B;             /* batch rows, >= 1 */
  int32_t K;             /* draft block length, 1 .. 1024 */
  int32_t V;             /* vocabulary, >= 1; bf16 needs V % 8 == 0, f32 V % 4 == 0 */
  int32_t r;             /* Markov rank: 0 (no head) or 1..256; bf16 tensor-core path needs r % 64 == 0 */
  int32_t dtype;         /* spec_dtype of base, target, U, W */
  int32_t draft_dtype;   /* spec_verify_block: spec_dtype of draft_logits */
  float temperature;     /* > 0 unless greedy */
  int32_t greedy;        /* 0 = stochastic, 1 = greedy */
  uint64_t seed;         /* Philox key */
  uint64_t cycle;        /* Philox counter words 2..3 (advance it every cycle) */
  uint64_t spin_limit;   /* polls before a device wait gives up; 0 = default (about 2 s) */
  uint32_t flags;        /* SPEC_FLAG_* */
  uint32_t row_offset;   /* global index of batch row 0: row b draws from Philox counter word
                            row_offset + b, so a batch split into shards (calls or GPUs) with
                            their starting rows draws exactly what one call over it draws;
                            row_offset + B must not exceed 2^31 */
} spec_params;

/* Bytes of device workspace the calls need for these parameters on the
 * current device (0 if the parameters are invalid).  Alignment: 256 bytes. */
size_t spec_workspace_size(const spec_params *p);

/* Zero a workspace (asynchronously on `stream`).  Required once before first
 * use, and again after any call whose spec_sync_status was not SPEC_OK. */
spec_status spec_workspace_init(void *workspace, size_t bytes, spec_stream_t stream);

/* Markov-head bias for one draft step (section "Innowacje w tworzeniu
 * tokenów"): bias[b, v] = sum_k U[prev[b], k] * W[k, v], fp32 accumulate.
 * prev [B] int32 (device), bias [B, V] float (device). */
spec_status spec_markov_bias(const spec_params *p, const void *U, const void *W,
                             const int32_t *prev, float *bias, void *workspace,
                             spec_stream_t stream);

/* Sequential drafting: for i = 0..K-1, z = base_i + U[prev] . W, d_i drawn
 * from softmax(z / T) (arg-max in greedy mode), prev = d_i.  One persistent
 * launch carries all K steps.  q_draft and biased_out may be NULL. */
spec_status spec_markov_bias_sample(const spec_params *p, const void *base, const void *U,
                                    const void *W, const int32_t *last_token, int32_t *draft,
                                    float *q_draft, float *biased_out, void *workspace,
                                    spec_stream_t stream);

/* Verification of given drafts against the target rows (section "Jak działa
 * spekulatywne dekodowanie"): draft_logits [B, K, V] are the final (biased)
 * draft logits in draft_dtype, draft [B, K] the tokens drawn from them.
 * One persistent launch with early exit (B <= 4096 and V up to 2048 tokens
 * per SM): positions are decided a few at a time, and the draft and target
 * rows of a position past a row's first rejection are never read.  So
 * q_draft[b, i] is written for the positions whose accept test ran (NaN
 * after), like p_draft.  Larger shapes take a multi-launch path that reads
 * every row and writes q_draft for all K positions.  p_draft and q_draft may
 * be NULL. */
spec_status spec_verify_block(const spec_params *p, const void *target, const void *draft_logits,
                              const int32_t *draft, int32_t *out, int32_t *tau, float *p_draft,
                              float *q_draft, void *workspace, spec_stream_t stream);

/* spec_verify_block with a verify length per request (the scheduler's K_b,
 * section "Optymalizacja weryfikacji i wydajności"): verify_len [B] int32
 * (device), K_b in 1..K.  Row b verifies positions 0..K_b-1 and draws its
 * bonus from target row K_b, so tau_b <= K_b + 1; rows past K_b are never
 * read.  A K_b outside 1..K is clamped and reported as SPEC_ERR_INVALID_ARG by
 * spec_sync_status.  Shapes the one-launch path does not take return
 * SPEC_ERR_UNSUPPORTED. */
spec_status spec_verify_block_kb(const spec_params *p, const void *target,
                                 const void *draft_logits, const int32_t *draft,
                                 const int32_t *verify_len, int32_t *out, int32_t *tau,
                                 float *p_draft, float *q_draft, void *workspace,
                                 spec_stream_t stream);

/* One whole cycle: drafting and verification fused in one persistent launch
 * (target rows are read only up to each row's first rejection).  draft,
 * p_draft and q_draft may be NULL. */
spec_status spec_cycle(const spec_params *p, const void *base, const void *target, const void *U,
                       const void *W, const int32_t *last_token, int32_t *draft, int32_t *out,
                       int32_t *tau, float *p_draft, float *q_draft, void *workspace,
                       spec_stream_t stream);

/* One cycle with a verify length per request (aigest.pl "DeepSeek prezentuje
 * DSpark", section "Optymalizacja weryfikacji i wydajności": a scheduler fixes
 * how many draft tokens of each request are verified, and its early stop keeps
 * the method lossless).  verify_len [B] int32 (device): K_b in 1..K.  Row b
 * drafts and verifies positions 0..K_b-1 and draws its bonus from target row
 * K_b, so tau_b <= K_b + 1 and the draws are the full block's first K_b draws
 * (the same random counters); draft[b, i] = -1 and q_draft[b, i] = NaN for
 * i >= K_b, and target rows past K_b are never read.  A K_b outside 1..K is
 * clamped and reported as SPEC_ERR_INVALID_ARG by spec_sync_status.  Tensor-core
 * path only (bf16, rank a multiple of 64 up to 256); other shapes return
 * SPEC_ERR_UNSUPPORTED.  spec_cycle is this call with every K_b = K. */
spec_status spec_cycle_kb(const spec_params *p, const void *base, const void *target,
                          const void *U, const void *W, const int32_t *last_token,
                          const int32_t *verify_len, int32_t *draft, int32_t *out, int32_t *tau,
                          float *p_draft, float *q_draft, void *workspace, spec_stream_t stream);

/* A decode loop: n_cycles cycles in one persistent launch (aigest.pl "DeepSeek
 * prezentuje DSpark", section "Jak działa spekulatywne dekodowanie DSpark?":
 * decoding repeats draft-and-verify cycles, each costing T_draft + T_verify
 * for its tau tokens).  The token a row emits last in cycle c (its correction
 * or its bonus token) is the committed token cycle c + 1 starts from, and
 * cycle c draws with Philox cycle counter p->cycle + c; cycle c is otherwise
 * spec_cycle_kb on slice c of the inputs.  Its verify lengths come from
 * verify_len, or from confidence scores (section "Optymalizacja weryfikacji i
 * wydajności": a score per draft position estimating the chance that its
 * token survives verification given accepted predecessors): K_b is the number
 * of leading positions whose prefix survival, the fp32 product of the scores
 * of positions 0..i taken in position order, is >= conf_threshold, and at
 * least 1 (a NaN score ends the prefix); or K with neither.
 *   base        [C, B, K, V]    dtype   (C = n_cycles; slice c feeds cycle c)
 *   target      [C, B, K+1, V]  dtype
 *   conf        [C, B, K]       float   or NULL
 *   verify_len  [C, B]          int32   or NULL (not both with conf)
 *   U, W, last_token            as for spec_cycle (last_token: cycle 0's)
 *   draft, p_draft, q_draft [C, B, K]; out [C, B, K+1]; tau [C, B]
 *   next_token  [B]             int32   the last token each row emitted in the
 *               last cycle (the next call's last_token); required when
 *               n_cycles > 1 (it carries the tokens between cycles), and it
 *               may be the same buffer as last_token.
 * n_cycles is 1..65536.  Tensor-core path only (bf16, rank a multiple of 64 up
 * to 256); other shapes return SPEC_ERR_UNSUPPORTED.  Device-side errors are
 * reported as for spec_cycle_kb. */
spec_status spec_decode_loop(const spec_params *p, int32_t n_cycles, const void *base,
                             const void *target, const float *conf, float conf_threshold,
                             const int32_t *verify_len, const void *U, const void *W,
                             const int32_t *last_token, int32_t *draft, int32_t *out, int32_t *tau,
                             float *p_draft, float *q_draft, int32_t *next_token, void *workspace,
                             spec_stream_t stream);

/* One cycle with the RNN sequential head in place of the Markov head
 * (aigest.pl "DeepSeek prezentuje DSpark", section "Innowacje w tworzeniu
 * tokenów": an optional RNN head tracks the whole block prefix).  The pages
 * give no formula; the reading implemented is an Elman recurrence in the
 * Markov head's factors:
 *   s_{-1} = 0,  s_i = bf16(clamp(U[prev_i] + Wh s_{i-1}, -1, 1)),  bias_i = s_i . W,
 * prev_i as for the Markov head.  (Wh s_{i-1})[j] is the fp32 fmaf chain over
 * k = 0..r-1 of s_{i-1}[k] * Wh[j, k] starting from 0, U[prev_i, j] is added
 * after it, and the result is clamped and rounded to bf16 (nearest, ties to
 * even), so the state is the same bit for bit on any implementation that
 * follows these steps.  Wh [r, r] bf16 (device), row j holding the weights of
 * output j.  The recurrence of step i + 1 is computed during step i across
 * the CTAs, so only its state update stays on the sequential path.  Otherwise
 * as spec_cycle.  Tensor-core path only (bf16, rank a multiple of 64 up to
 * 256); other shapes return SPEC_ERR_UNSUPPORTED. */
spec_status spec_cycle_rnn(const spec_params *p, const void *base, const void *target,
                           const void *U, const void *W, const void *Wh,
                           const int32_t *last_token, int32_t *draft, int32_t *out, int32_t *tau,
                           float *p_draft, float *q_draft, void *workspace, spec_stream_t stream);

/* spec_cycle without a workspace argument, for callers that cannot allocate
 * device memory when they run a cycle (code whose allocations all belong to a
 * framework pool, a host thread that must not call cudaMalloc because it
 * synchronises the device, a plugin that only receives input and output
 * buffers).  The pages have no counterpart: this is a deployment convenience.
 * Scratch lives in a fixed 8 MiB device array inside the library, present on
 * every GPU that loads it until the process exits; nothing is allocated per
 * call.  Shapes whose spec_workspace_size exceeds 8 MiB are rejected with
 * SPEC_ERR_WORKSPACE (and a message on stderr).  The first call on a device
 * looks up the array's device address (again after the device's context was
 * replaced, e.g. by cudaDeviceReset); make that first call before any stream
 * capture.  All calls share the array: calls that overlap on the GPU race, so
 * order them on one stream.  status_out (device int32, may be NULL) receives
 * the device-side status of the call, stream-ordered after it. */
spec_status spec_cycle_noalloc(const spec_params *p, const void *base, const void *target,
                               const void *U, const void *W, const int32_t *last_token,
                               int32_t *draft, int32_t *out, int32_t *tau, float *p_draft,
                               float *q_draft, int32_t *status_out, spec_stream_t stream);

/* Verify-length scheduler (host logic; no device work, no stream, callable
 * without a GPU).  mkdocs.reaper.mx DeepSeek-V4.1-Flash "06-extensions", DSpark
 * table: the scheduler chooses each request's verify length from the prefix
 * survival probabilities of the confidence head and the engine's throughput
 * curve measured beforehand, to maximise expected throughput under the current
 * load; aigest.pl "DeepSeek prezentuje DSpark", "Optymalizacja weryfikacji i
 * wydajności": that curve is SPS(B), profiled once at start-up.  Reading: with
 * S_{b,i} = prod_{j<=i} clamp(conf[b][j], 0, 1) (a NaN score counts as 0),
 * choose k_b in 1..K maximising
 *   E * SPS(M),  E = sum_b (1 + sum_{i<k_b} S_{b,i}),  M = sum_b (k_b + 1)
 * (expected tokens per step times steps per second for a target pass over M
 * rows); among equal maxima the smallest total length, among allocations of
 * that total the one taking the larger S first, ties to the lower row b.
 *   conf        [B, K] float, host    confidence scores per draft position
 *   sps         [n_sps] double, host  steps per second of a target pass over m
 *                                     rows, m = 0 .. n_sps-1; 0 past the table
 *   verify_len  [B] int32, host       output k_b, ready for spec_cycle_kb
 *   expected    [2] double, host      output (E, E * SPS(M)); may be NULL
 * Errors: SPEC_ERR_INVALID_ARG for a NULL pointer, B or K < 1, B*K > 2^26,
 * n_sps < 1, or an SPS entry that is negative, NaN or infinite (nothing is
 * written then).  Cost O(BK log BK) on the calling thread. */
spec_status spec_schedule_verify_len(const float *conf, int32_t B, int32_t K,
                                     const double *sps, int32_t n_sps, int32_t *verify_len,
                                     double *expected);

/* Keep [ptr, ptr + bytes) resident in L2 for kernels later launched on
 * `stream` (a persisting access-policy window on the stream; the persisting
 * L2 carve-out of the calling process's context is raised to fit, up to the
 * device maximum).  Meant for the Markov factor W, which every draft step
 * re-reads.  bytes = 0 removes the window and releases persisting lines.  The
 * carve-out belongs to this process's context and ends with it. */
spec_status spec_l2_persist(const void *ptr, size_t bytes, spec_stream_t stream);

/* ---------------------------------------------------------------------------
 * Operators around the sequential head.  The calls above fuse a head's lookup,
 * recurrence, vocabulary product and verification into one cycle; these offer
 * the same steps one by one, in the forms a program needs beside the cycle: a
 * head that is trained, that runs over long sequences, whose vocabulary factor
 * is held in 4 bits, or whose draws are made outside the library.  Chained, they
 * are: tokens -> rows of U (spec_embed) -> gated recurrence (spec_gated_scan)
 * -> vocabulary product and base logits (spec_bias_w4) -> probabilities ->
 * spec_verify_probs.  The pages give no counterpart of these forms.
 *
 * Rules shared by all of them.  Tensors are row-major device memory of the
 * current device, rows contiguous, any element alignment (16-byte aligned
 * pointers and row strides run faster); strides are in elements, 0 = dense.
 * Outputs may not overlap inputs unless a comment says so.  `workspace` holds
 * at least SPEC_WORKSPACE_MIN bytes (spec_embed_grad, the recurrence and
 * spec_bias_w4: what spec_embed_workspace_size, spec_scan_workspace_size and
 * spec_w4_workspace_size return), zeroed once by spec_workspace_init; errors
 * found on the device go there and are read by spec_sync_status.  Those three
 * also keep scratch in it, which calls of one stream may share among
 * themselves, but not with the calls above; spec_embed and spec_verify_probs
 * touch only the status and may share any workspace.
 * All calls can be captured into a CUDA graph.  Sums are taken in a fixed
 * order, and equal inputs give equal bits.
 * ------------------------------------------------------------------------- */
#define SPEC_WORKSPACE_MIN 256

typedef struct {
  int32_t n;             /* tokens, 0 .. 2^30 */
  int32_t V;             /* rows of the table, >= 1 */
  int32_t D;             /* row width, 1 .. 65536 */
  int32_t dtype;         /* spec_dtype of the table (lookup) or of its gradient */
  int32_t row_dtype;     /* spec_dtype of the rows: the lookup's output, the gradient's input */
  int32_t accumulate;    /* gradient: 0 = write the whole table gradient, 1 = add to it */
  float scale;           /* finite */
  int32_t reserved;      /* 0 */
  int64_t table_stride;  /* between table rows; 0 = D */
  int64_t row_stride;    /* between rows; 0 = D */
} spec_embed_params;

/* Bytes of workspace spec_embed_grad needs (0 if the parameters are invalid);
 * enough for spec_embed too. */
size_t spec_embed_workspace_size(const spec_embed_params *p);

/* Scaled lookup, the head's U[prev] by itself: rows[i] = scale * table[ids[i]],
 * multiplied in fp32 and rounded once.  ids [n] int32; -1 ("no token", as in
 * the outputs of the cycle) gives a row of zeros, any other id outside [0, V)
 * too, and is reported as SPEC_ERR_TOKEN_RANGE. */
spec_status spec_embed(const spec_embed_params *p, const void *table, const int32_t *ids,
                       void *rows, void *workspace, spec_stream_t stream);

/* Its gradient: dtable[v] (+)= scale * sum of drows[i] over the i with
 * ids[i] = v.  Each table row is written once, by fp32 sums in a fixed order
 * (ascending i, in pieces joined in order), rounded once.  With
 * accumulate = 0 every table row is written (rows no token names become 0);
 * with 1 only the rows named by a token are touched.  Ids outside [0, V) add
 * nothing; all but -1 are reported as SPEC_ERR_TOKEN_RANGE. */
spec_status spec_embed_grad(const spec_embed_params *p, const int32_t *ids, const void *drows,
                            void *dtable, void *workspace, spec_stream_t stream);

#define SPEC_SCAN_CHUNK 16 /* steps between two states kept for the gradient */

typedef struct {
  int32_t B;            /* sequences, >= 1 */
  int32_t T;            /* steps, >= 0 */
  int32_t D;            /* channels, >= 1 */
  int32_t dtype;        /* spec_dtype of gate, x, h and their gradients; states are float */
  int64_t gate_stride;  /* between the steps of gate and dgate; 0 = D; sequences are T steps apart */
  int64_t x_stride;     /* the same of x and dx */
  int64_t h_stride;     /* the same of h and dh */
} spec_scan_params;

/* Bytes of workspace the two calls below need on the current device (0 if the
 * parameters are invalid, or without a GPU). */
size_t spec_scan_workspace_size(const spec_scan_params *p);

/* Gated linear recurrence over sequences, a sequential head that trains by a
 * scan (beside spec_cycle_rnn's, which is sequential by its form):
 *   f_t = sigmoid(gate_t),  h_t = f_t h_{t-1} + (1 - f_t) x_t,  h_{-1} = h0.
 *   gate, x  [B, T, D] dtype
 *   h0       [B, D] float, or NULL (zeros)
 *   len      [B] int32, or NULL (all T): steps t >= len[b] do not belong to
 *            sequence b; h is left as it was there.  A length outside 0..T is
 *            clamped and reported as SPEC_ERR_INVALID_ARG.
 *   h        [B, T, D] dtype, or NULL
 *   h_last   [B, D] float, or NULL: the state after the last step (h0 where
 *            len is 0); may be the buffer of h0, as in step-by-step decoding
 *   states   [B, ceil(T / SPEC_SCAN_CHUNK), D] float, or NULL: the state before
 *            every SPEC_SCAN_CHUNK-th step, which the gradient needs (past the
 *            end of a sequence: its last state)
 * States are carried in fp32.  Gates beyond -87 and 87, and products of gates
 * below 2^-126, count as these: an infinite state or input stays infinite, as
 * in the formula. */
spec_status spec_gated_scan(const spec_scan_params *p, const void *gate, const void *x,
                            const float *h0, const int32_t *len, void *h, float *h_last,
                            float *states, void *workspace, spec_stream_t stream);

/* Its gradient, given dh [B, T, D] (dtype) of h and dh_last [B, D] (float, or
 * NULL) of h_last:
 *   delta_t = dh_t + f_{t+1} delta_{t+1}, dh_last added at the last step,
 *   dx_t = (1 - f_t) delta_t,  dgate_t = delta_t (h_{t-1} - x_t) f_t (1 - f_t),
 *   dh0 = f_0 delta_0 (dh_last where len is 0).
 * h_{t-1} is computed again in fp32 from `states`, as the forward call wrote
 * them for the same inputs.  dgate and dx are written over all T steps, with
 * zeros where t >= len[b]; dh is not read there.  dh0 may be NULL. */
spec_status spec_gated_scan_grad(const spec_scan_params *p, const void *gate, const void *x,
                                 const float *h0, const int32_t *len, const float *states,
                                 const void *dh, const float *dh_last, void *dgate, void *dx,
                                 float *dh0, void *workspace, spec_stream_t stream);

typedef struct {
  int32_t B;            /* rows, 1 .. 65536; taken 16 at a time */
  int32_t r;            /* features, a multiple of group, up to 65536 */
  int32_t V;            /* vocabulary, 1 .. 2^30 */
  int32_t group;        /* features that share a scale: 32, 64 or 128 */
  int32_t dtype;        /* spec_dtype of x */
  int32_t scale_dtype;  /* spec_dtype of wscale */
  int32_t base_dtype;   /* spec_dtype of base */
  int32_t out_dtype;    /* spec_dtype of out */
  int32_t x_rows;       /* rows of x when prev is given */
  int32_t reserved;     /* 0 */
  int64_t x_stride;     /* between rows of x; 0 = r */
  int64_t base_stride;  /* between rows of base; 0 = V */
  int64_t out_stride;   /* between rows of out; 0 = V */
} spec_w4_params;

/* Bytes of workspace spec_bias_w4 needs (0 if the parameters are invalid). */
size_t spec_w4_workspace_size(const spec_w4_params *p);

/* Vocabulary product with the factor W in 4 bits:
 *   out[b, v] = base[b, v] + sum_k X[b, k] * (code[v, k] - 8) * wscale[v, k / group],
 * X[b] = x[prev[b]] (the Markov bias of spec_markov_bias) or, with prev NULL,
 * x[b].  Products and the sum inside a group are exact or fp32, groups are
 * added in fp32 in a fixed order; out is rounded once.
 *   x       [B, r], or [x_rows, r] with prev; dtype
 *   prev    [B] int32, or NULL; an id outside [0, x_rows) is clamped and
 *           reported as SPEC_ERR_TOKEN_RANGE
 *   wq      [V, R/2] bytes, R = r rounded up to a multiple of 128; 16-byte
 *           aligned.  Two codes (0..15) a byte, the lower feature in the lower
 *           half; in each run of 128 features (64 bytes) the sixteen 4-byte
 *           words w = 0..15 stand in the order 4 (w mod 4) + floor(w / 4), so
 *           that 16 consecutive bytes hold one word of each 32 features;
 *           features past r hold code 8
 *   wscale  [V, r / group], scale_dtype
 *   base    [B, V] base_dtype, or NULL
 *   out     [B, V] out_dtype; may be base where type and stride are the same */
spec_status spec_bias_w4(const spec_w4_params *p, const void *x, const int32_t *prev,
                         const void *wq, const void *wscale, const void *base, void *out,
                         void *workspace, spec_stream_t stream);

/* Lay a factor W [r, V] (dtype w_dtype, as for spec_markov_bias) out for
 * spec_bias_w4: per token and group, scale = max |W| / 7 rounded to
 * scale_dtype, code = 8 + W / scale rounded to nearest even and clamped to
 * 0..15 (8 where the scale is 0).  A NaN counts as 0, an infinity as the largest
 * finite float of its sign.  Uses r, V, group and scale_dtype of p.  wq and wscale are outputs of the sizes above. */
spec_status spec_w4_quantize(const spec_w4_params *p, const void *W, int32_t w_dtype, void *wq,
                             void *wscale, spec_stream_t stream);

typedef struct {
  int32_t B;              /* batch rows, >= 1 */
  int32_t K;              /* block length, 1 .. 1024 */
  int32_t V;              /* vocabulary, 1 .. 2^30 */
  int32_t dtype;          /* spec_dtype of target */
  int32_t draft_dtype;    /* spec_dtype of draft_probs */
  int32_t reserved;       /* 0 */
  int64_t target_stride;  /* between vocabulary rows of target; 0 = V */
  int64_t draft_stride;   /* between vocabulary rows of draft_probs; 0 = V */
} spec_probs_params;

/* Verification of drafted tokens against the target's probabilities from given
 * random numbers: the rule of spec_verify_block for programs that hold
 * probabilities (after penalties or truncation, not softmax of logits) and
 * draw their own uniforms.
 *   target      [B, K+1, V]  dtype        p, row K = bonus row
 *   draft_probs [B, K, V]    draft_dtype  q
 *   draft       [B, K]       int32
 *   u_accept    [B, K]       float        uniforms in [0, 1)
 *   u_draw      [B]          float
 *   verify_len  [B]          int32, or NULL (all K): K_b in 0..K; 0 draws from
 *               row 0 (plain decoding); a negative length marks a row to skip,
 *               of which nothing is read or written; one above K is clamped
 *               and reported as SPEC_ERR_INVALID_ARG
 *   out [B, K+1], tau [B] int32; p_draft, q_draft [B, K] float or NULL, as
 *   for spec_verify_block (NaN past the positions whose test ran)
 * Position i is accepted iff u_accept * q_i(d_i) < p_i(d_i), compared exactly.
 * The draw takes the first token whose inclusive mass exceeds u_draw * total
 * (else the last one with mass), in ascending token order, from max(p_j - q_j, 0)
 * at the first rejection j (p_j where that has no mass), or from p_{K_b}.
 * Masses are summed in 64 bits: the order of the sums can decide only where
 * u_draw * total lies within (V + 2) 2^-52 of the total of a token's border.
 * A p that is NaN, infinite or negative has no mass; a q that is NaN or
 * negative counts as 0.  A row without any mass emits -1 there, has tau = the
 * number of accepted drafts, and is reported as SPEC_ERR_INVALID_ARG.  A draft outside [0, V) is rejected
 * and reported as SPEC_ERR_TOKEN_RANGE.  Only the rows of the first rejection
 * (or the bonus row) are read whole. */
spec_status spec_verify_probs(const spec_probs_params *p, const void *target,
                              const void *draft_probs, const int32_t *draft,
                              const float *u_accept, const float *u_draw,
                              const int32_t *verify_len, int32_t *out, int32_t *tau,
                              float *p_draft, float *q_draft, void *workspace,
                              spec_stream_t stream);

/* Synchronise `stream` and return the device-side status recorded in the
 * workspace by the calls issued on it (SPEC_OK if none failed). */
spec_status spec_sync_status(const void *workspace, spec_stream_t stream);

/* Human-readable name of a status code. */
const char *spec_status_string(spec_status s);

/* Number of kernel launches the last call on this thread issued. */
int32_t spec_last_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif
