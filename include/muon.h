/*
 * muon.h -- C ABI of the MI355X (gfx950) Muon optimizer step, and of the
 * transformer block's operators that train with it (last section).
 *
 * The operation (per hidden weight matrix W with gradient G and momentum
 * buffer M), as the pages describe it:
 *   - Guide page "NanoGPT Speedrun: The Ultimate Guide to Pushing LLM Training
 *     Efficiency to Its Limits", section "Optimizer and Training Strategy
 *     Tuning": Muon is applied to hidden-layer matrix weights only; the update
 *     is orthogonalised after a Nesterov momentum step.
 *   - Overview page "The NanoGPT speedrun", paragraph "Six records account for
 *     most of the speedup" (record #3): the momentum update is orthogonalised
 *     (approximately its polar factor U V^T) by five Newton-Schulz steps.
 *
 * What muon_step computes, per matrix (rows x cols, row-major):
 *   M <- fl32(mu*M + G)                       momentum, fp32 buffer, in place
 *   U  = G + mu*M   (nesterov != 0)  or  U = M
 *   X  = U, or U^T when rows > cols           short side first (m <= n)
 *   X <- X / (||X||_F + 1e-7)
 *   T times:  A = X X^T;  B = b*A + c*A*A;  X <- a*X + B*X
 *   W <- W - lr * s * O,  O = X (or X^T back in W's orientation)
 * s is the descriptor's `scale` (<= 0 means 1).  The polynomial, the
 * normalisation and s are readings of the pages, which name the iteration but
 * not its coefficients; a, b, c and T are arguments.
 *
 * Precision.  MUON_PATH_BF16: the three products take bf16 operands (rounded
 * to nearest even) and accumulate in fp32; A and B are stored bf16; the a*X
 * term reads X for the first `x_master_iters` iterations (default 3) as a
 * (hi, lo) pair, hi = bf16(X) (the operand copy) and lo one signed byte: the
 * distance from hi to X in the integer order of fp32 bit patterns, in units
 * of 256, rounded (about 16 significant bits, relative error <= 2^-15), and as
 * the bf16 copy alone afterwards.  Matrices whose short side is
 * below 128 take the fp32 arithmetic even on this path: their A*A and B*X
 * contractions are too short for bf16 rounding errors to average out.
 * MUON_PATH_F32: everything fp32.
 *
 * Ownership.  The caller owns every device buffer: weights, gradients,
 * momentum buffers and the workspace.  The library never allocates device
 * memory.  A plan (host object) holds the layout and its device tables, which
 * live inside the caller's workspace; the workspace must stay untouched and
 * alive for the plan's lifetime.  A plan is not re-entrant: calls on one plan
 * must be ordered (one stream, or synchronised streams).  Different plans
 * with different workspaces may run concurrently.
 *
 * Streams.  `hip_stream` is a hipStream_t passed as void* (NULL = the null
 * stream).  muon_step only enqueues work (it never waits for the device
 * unless a pointer change finds all 8 device copies of the matrix table
 * still in flight); inputs must stay alive until the stream has passed the
 * step.
 *
 * Graph capture.  A step may be enqueued into a capturing stream (HIP stream
 * capture); the graph then reads the plan's device copy of the matrix table
 * as it stood at capture time, so from then on the plan's pointers are fixed:
 * a step whose descriptors carry other pointers, during capture or after it,
 * fails with MUON_E_INVAL (make a new plan for new buffers).  Profiling must
 * be off while capturing (MUON_E_INVAL otherwise).  Replays and eager steps
 * of the same plan must be ordered like any two steps of one plan.
 *
 * Errors.  Every int-returning function returns MUON_OK (0) or a negative
 * MUON_E_* code and then sets a thread-local message readable with
 * muon_last_error().  No C++ exception crosses this ABI.  Gradient values are
 * not inspected: NaN/Inf in G propagate into M, X and W.
 */
#ifndef MUON_MI355X_H
#define MUON_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_OK 0
#define MUON_E_INVAL (-1)       /* bad argument: null pointer, size, T, non-finite scalar ... */
#define MUON_E_UNSUPPORTED (-2) /* dtype or leading dimension not supported */
#define MUON_E_MISMATCH (-3)    /* step descriptors do not match the plan */
#define MUON_E_WORKSPACE (-4)   /* workspace too small or not 256-byte aligned */
#define MUON_E_HIP (-5)         /* a HIP runtime call failed (message has its text) */

#define MUON_DTYPE_F32 0
#define MUON_DTYPE_BF16 1

#define MUON_PATH_BF16 0
#define MUON_PATH_F32 1

/* One hidden matrix.  All pointers are device pointers.  Row-major storage;
 * ld_w and ld_g are leading dimensions in elements and must equal cols (0 is
 * read as cols).  grad: MUON_DTYPE_BF16 or MUON_DTYPE_F32.  weight:
 * MUON_DTYPE_F32 or MUON_DTYPE_BF16.  momentum: always fp32, rows x cols.
 * weight must not alias grad or momentum. */
typedef struct muon_matrix_desc {
  void* weight;
  const void* grad;
  float* momentum;
  int64_t rows;
  int64_t cols;
  int64_t ld_w;
  int64_t ld_g;
  int32_t w_dtype;
  int32_t g_dtype;
  float scale;      /* per-matrix factor s of the weight step; <= 0 means 1 */
  int32_t reserved; /* must be 0 */
} muon_matrix_desc;

/* Plan options.  NULL means: MUON_PATH_BF16, x_master_iters 3, no zeroing,
 * max_T 64, 2 groups. */
typedef struct muon_options {
  int32_t path;           /* MUON_PATH_BF16 or MUON_PATH_F32 */
  int32_t x_master_iters; /* bf16 path: iterations 1..k read X in a*X as its
                             (bf16, low byte) pair; < 0 selects the default 3;
                             ignored on f32 */
  int32_t zero_momentum;  /* != 0: muon_init zeroes every momentum buffer */
  int32_t max_T;          /* largest T muon_step accepts; <= 0 selects 64 */
  int32_t groups;         /* 1: every launch on the caller's stream; 2 (or <= 0,
                             the default) to 4: that many matrix groups, each on a
                             stream of its own (see muon_plan_info.n_groups).  Two
                             measure fastest on MI355X: with 4 hardware queues per
                             process, more streams start to share queues. */
  int32_t fused;          /* != 0: a fused plan.  Every bf16 product of a step
                             (all T iterations of Gram, polynomial and update)
                             runs in one persistent launch, on the caller's stream
                             (groups is then ignored): the planner places each
                             matrix on one XCD, and the launch's blocks take the
                             tiles of their XCD in order, each waiting until the
                             tiles it reads are finished (muon_check reports a
                             wait that gave up).  Steps with T > 16 run the three
                             launches per iteration instead. */
} muon_options;

typedef struct muon_plan muon_plan;

/* Library version string, e.g. "muon-mi355x 1.0.0 (gfx950)".  Never NULL. */
const char* muon_version(void);

/* Bytes of device workspace muon_init needs for these matrices and options;
 * 0 on invalid arguments (see muon_last_error).  Host-only: no HIP call. */
size_t muon_workspace_size(const muon_matrix_desc* descs, int n, const muon_options* opts);

/* Validate the n descriptors, plan the launches and lay out the workspace
 * (device memory of ws_bytes >= muon_workspace_size(...), 256-byte aligned).
 * Uploads the plan's tables (and zeroes the momentum buffers when requested)
 * on hip_stream and waits for that stream before returning.  On success
 * *out_plan owns the host state. */
int muon_init(const muon_matrix_desc* descs, int n, const muon_options* opts,
              void* workspace, size_t ws_bytes, void* hip_stream, muon_plan** out_plan);

/* Enqueue one Muon step over every matrix of the plan on hip_stream.  Per
 * matrix group (muon_plan_info.n_groups; the first group on hip_stream itself,
 * each other one on a stream of its own, forked from and joined back into
 * hip_stream, so later work on hip_stream sees the whole step): 1 momentum launch and 1 norm launch, then 3 launches
 * per Newton-Schulz iteration (all matrices of one precision grouped in each
 * launch: 6 per iteration when the group mixes bf16 and fp32 matrices); T == 0
 * enqueues one weight-step launch instead of norm and iterations
 * (W <- W - lr*s*X0).  descs == NULL reuses the pointers the plan holds;
 * otherwise n must equal the plan's count and shapes, dtypes and scales must
 * match (pointers may differ).  Requirements: 0 <= T <= max_T,
 * 0 <= momentum <= 1, a, b, c, lr finite. */
int muon_step(muon_plan* plan, const muon_matrix_desc* descs, int n, float a, float b, float c,
              int T, float momentum, int nesterov, float lr, void* hip_stream);

/* muon_step with a polynomial of its own for every iteration: iteration t
 * (1-based) uses a = coeffs[3(t-1)], b = coeffs[3(t-1)+1], c = coeffs[3(t-1)+2].
 * The speedrun overview page ("The NanoGPT speedrun", paragraph "Reading
 * guide") names later records that tune the iteration's polynomials (Polar
 * Express); it gives no values, so the schedule is the caller's.  coeffs is a
 * host array of 3*T finite floats, read during the call (the caller may reuse
 * it on return); NULL is allowed only with T == 0. */
int muon_step_schedule(muon_plan* plan, const muon_matrix_desc* descs, int n, const float* coeffs, int T,
                       float momentum, int nesterov, float lr, void* hip_stream);

/* For callers that cannot allocate device memory (tight serving loops,
 * harnesses that forbid hipMalloc): one muon_step over
 * the n descriptors without a plan or a workspace.  The working memory (X
 * copies, A, B, partial sums, tables) is a static device array of 64 MiB
 * (MUON_SCRATCH_BYTES) that the library holds on every GPU it runs on until
 * the process ends; the call allocates nothing.  It plans on the host each
 * time, copies the tables into that array from pageable host memory on
 * hip_stream (a later call first waits for that copy to have run) and
 * enqueues the step there (groups and fused are ignored: one stream, three
 * launches per iteration).
 * That copy is not meant for stream capture: capture the planned muon_step
 * instead.
 * Arguments are those of muon_init (opts: path, x_master_iters and max_T;
 * zero_momentum must be 0) and muon_step; the stream must belong to the
 * current device.  A set whose working memory exceeds the array fails with
 * MUON_E_WORKSPACE (muon_workspace_size with fused 0 gives the need, within a
 * few KiB).
 * All calls on one GPU share its array and every call rewrites what it reads
 * before reading it, so only overlap matters: calls that can run at the same
 * time on one GPU (other streams, other host threads) race and must be
 * ordered by the caller. */
#define MUON_SCRATCH_BYTES (64u << 20)
int muon_step_scratch(const muon_matrix_desc* descs, int n, const muon_options* opts, float a, float b, float c,
                      int T, float momentum, int nesterov, float lr, void* hip_stream);

/* Free the plan's host state.  The workspace stays the caller's. */
int muon_destroy(muon_plan* plan);

/* Message of the last failed call on this thread ("" if none). */
const char* muon_last_error(void);

/* ---- introspection and measurement ---------------------------------------- */

/* Launch kinds, in the order they run within a step. */
#define MUON_KIND_MOMENTUM 0 /* momentum + Nesterov + Frobenius partial sums, writes X0 */
#define MUON_KIND_GRAM 1     /* A = X X^T (upper tiles, mirrored) */
#define MUON_KIND_POLY 2     /* B = b A + c A A (upper tiles, mirrored) */
#define MUON_KIND_UPDATE 3   /* X <- a X + B X; on the last iteration W <- W - lr s O */
#define MUON_KIND_APPLY 4    /* T == 0 only: W <- W - lr s X0 */
#define MUON_KIND_NORM 5     /* T > 0: 1 / (||U||_F + eps) per matrix from the momentum partials */
#define MUON_KIND_FUSED 6    /* fused plans: every bf16 product of the step in one launch */
#define MUON_KIND_COUNT 7

/* Host-only description of the plan these descriptors would get.  Returns
 * MUON_OK and fills the fields, or an error code.  `tiles` (optional) gets
 * the launch-ordered tile list of one kind as (matrix, tile_row, tile_col)
 * int32 triples, at most tile_cap triples; *n_tiles gets the full count. */
typedef struct muon_plan_info {
  int64_t workspace_bytes;
  int32_t n_matrices;
  int32_t tile;              /* tile edge of the fp32 Newton-Schulz products (128) */
  int32_t blocks[MUON_KIND_COUNT]; /* tile-table length of each launch kind: the grid of
                                      the momentum, norm and apply launches; the product
                                      kernels are persistent (2 blocks per CU) and
                                      stride through their table (all groups' tables,
                                      each padded to a multiple of 8) */
  int32_t x_master_iters;
  int32_t path;
  int32_t n_f32_matrices;    /* matrices whose products run in fp32 (see below) */
  int32_t n_groups;          /* matrix groups (contiguous, of equal cost) whose
                                steps run on streams of their own, forked from
                                and joined back into the caller's stream (1 to
                                4): momentum and norm have n_groups launches per
                                step, a product kind T * n_groups (times the
                                precisions present) */
  int32_t bf16_tile_rows;    /* bf16 polynomial and update products: output tile rows
                                (256); the short side of such a matrix is padded to a
                                multiple of it */
  int32_t bf16_tile_cols;    /* bf16 products: output tile columns (128); the Gram
                                product takes square tiles of this edge */
  int32_t fused;             /* 1: a fused plan (muon_options.fused); blocks[MUON_KIND_FUSED]
                                is then its queue length per iteration (all XCDs),
                                and kind MUON_KIND_FUSED lists the queue as
                                (xcd, product 1-3, matrix, tile_row, tile_col)
                                int32 quintuples, XCD by XCD, each XCD's entries
                                in the order its blocks take them */
} muon_plan_info;

int muon_describe(const muon_matrix_desc* descs, int n, const muon_options* opts,
                  muon_plan_info* info, int kind, int32_t* tiles, int tile_cap, int32_t* n_tiles);

/* Per-launch timing with HIP events (enable != 0 turns it on).  Each timed
 * launch of muon_step is issued with hipExtLaunchKernel and an event pair
 * that takes the dispatch's own start and end times, so timing adds no
 * event records to the stream; it does add host work per launch, and a step
 * with timing on must not be captured in a graph.  muon_profile_select
 * restricts the timed launches to the kinds whose bit (1 << MUON_KIND_*) is
 * set in kind_mask (default: all kinds).  muon_profile_read waits for the
 * events, adds their durations per kind into ms[MUON_KIND_COUNT] and
 * launches[MUON_KIND_COUNT] (totals since the last read), and resets the
 * totals. */
int muon_profile_enable(muon_plan* plan, int enable);
int muon_profile_select(muon_plan* plan, uint32_t kind_mask);
int muon_profile_read(muon_plan* plan, double* ms, int64_t* launches);

/* Fused plans: waits for hip_stream, then reports whether a fused launch of
 * this plan gave up a dependency wait since the last check (MUON_E_HIP with
 * the reason; that step's results are incomplete) and clears the report.
 * MUON_OK otherwise, and always for plans that are not fused.  A wait gives
 * up after the plan's poll limit (about 4 s by default), which a launch whose
 * blocks all run never reaches. */
int muon_check(muon_plan* plan, void* hip_stream);

/* Fused plans, for tests of the give-up path: polls of one dependency wait
 * before it gives up (> 0; default 1 << 24, 0.25 us apart) and a count added
 * to every wait's target (>= 0; default 0: with any larger value no wait is
 * ever met, so every block of the next fused launch gives up and returns).
 * MUON_E_INVAL for other values or a plan that is not fused. */
int muon_fused_limits(muon_plan* plan, int32_t spin_limit, int32_t dep_bias);

/* ---- operators of the block whose matrices the step trains ------------------
 *
 * A GPT-2-style block needs, besides products with its hidden matrices, a norm
 * and an attention whose gradients end in those matrices: layer norm, and
 * causal attention over packed sequences (the overview page "The NanoGPT
 * speedrun", record #12, trains on documents packed into one long sequence
 * with document masking).  What that attention reads are queries and keys that
 * are normalised for each head and rotated by position (the same page, records
 * #2 and #5), and what the first block reads are rows of an embedding table:
 * the embedding lookup, and the query/key norm with rotation.  Each has a
 * forward and a backward call.
 *
 * They follow the conventions of the step: the caller owns every buffer, the
 * library allocates nothing and never waits for the device; every pointer is a
 * device pointer of the current device, which hip_stream belongs to; calls
 * may be captured in a graph; errors are codes with a message in
 * muon_last_error().  A call keeps nothing: calls on different streams or
 * threads are independent as long as their buffers and workspaces are.  A call
 * whose output or workspace shares memory with another of its operands is
 * refused (MUON_E_INVAL).  Operands may lie between each other's rows in one
 * buffer if they step through it alike.
 * Results are bitwise reproducible (no floating-point atomics).  NaN and infinities are not
 * inspected; they propagate as in the formulas. */

/* Layer norm of `rows` rows of `cols` elements (cols <= 2^20).  Leading
 * dimensions are in elements (0 is read as cols).  x, y, dy and dx have
 * x_dtype; weight and bias have p_dtype, and a NULL one counts as ones or
 * zeros.  Arithmetic is fp32.  No alignment beyond an element's is needed.
 * rows times a leading dimension is at most 2^56. */
typedef struct muon_layernorm_desc {
  int64_t rows;
  int64_t cols;
  int64_t ld_x, ld_y, ld_dy, ld_dx;
  int32_t x_dtype;
  int32_t p_dtype;
  float eps;        /* >= 0 */
  int32_t reserved; /* must be 0 */
} muon_layernorm_desc;

/* y = (x - mean) * rstd * weight + bias, rstd = 1 / sqrt(var + eps), with the
 * row's mean and biased variance; mean[rows] and rstd[rows] (fp32) are written
 * for the backward call.  rows == 0 does nothing. */
int muon_layernorm_forward(const muon_layernorm_desc* desc, const void* x, const void* weight, const void* bias,
                           void* y, float* mean, float* rstd, void* hip_stream);

/* Bytes of device workspace muon_layernorm_backward needs for its parameter
 * gradients; 0 on invalid arguments.  Host-only. */
size_t muon_layernorm_workspace_size(const muon_layernorm_desc* desc);

/* Gradients of the forward call: dx (x_dtype), dweight[cols] and dbias[cols]
 * (fp32, overwritten; zero when rows == 0).  Any of the three may be NULL, but
 * not all if there are rows.  workspace (256-byte aligned) may be NULL when dweight and dbias are. */
int muon_layernorm_backward(const muon_layernorm_desc* desc, const void* dy, const void* x, const void* weight,
                            const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                            void* workspace, size_t ws_bytes, void* hip_stream);

/* Causal attention over `tokens` packed tokens.  cu_seqlens (device, seqs + 1
 * int32, cu_seqlens[0] = 0, not decreasing, last one <= tokens) holds the
 * sequences' offsets; a sequence may be empty.  Token i of a sequence attends
 * to its tokens 0 .. i.  Query head h reads key/value head
 * h / (q_heads / kv_heads).  head_dim: a multiple of 8, at most 128.  dtype:
 * MUON_DTYPE_BF16 or MUON_DTYPE_F32, of every operand.  scale, from 2^-60 to
 * 2^60, multiplies the scores.  (tokens / 128 + seqs + 1) * q_heads must stay
 * below 2^24 (fp32 with head_dim up to 64: (tokens / 64 + seqs + 1) * q_heads
 * below 2^23), or the call is refused (MUON_E_UNSUPPORTED).
 *
 * cu_seqlens is not checked (it is read on the device); offsets outside
 * [0, tokens] are clamped and decreasing ones make empty sequences, so no
 * access leaves the operands, but rows that two sequences claim are undefined.
 *
 * Rows behind the last sequence, cu_seqlens[seqs] .. tokens - 1, are never
 * read; in each output they are left as they were, or set to zero when the
 * output's flag is given.
 *
 * bf16: products take bf16 operands (probabilities and score gradients are
 * rounded to bf16 for theirs) and accumulate in fp32, where softmax
 * statistics are held.  fp32: fp32 throughout.  Scores and lse are fp32 numbers:
 * a weight is off by about 2^-22 of itself times its score's magnitude, and from
 * magnitudes of 2^30 on a row may be NaN.  A score of -inf has weight 0; a
 * row of nothing else is NaN.  What the mask hides does not count, whatever it
 * holds: a NaN or infinity in a token's k or v reaches the outputs of that
 * token and of later ones in its sequence, one in its q or dout the dk and dv
 * of that token and of earlier ones, as in the formulas.  (Blocks of
 * rows that meet one are computed twice: a call full of NaN takes three times
 * as long.) */
typedef struct muon_attention_desc {
  int64_t tokens;
  int32_t seqs;
  int32_t q_heads;
  int32_t kv_heads; /* divides q_heads */
  int32_t head_dim;
  int32_t dtype;
  float scale;
  int32_t reserved; /* must be 0 */
} muon_attention_desc;

/* One (tokens, heads, head_dim) operand: strides in elements, head_dim
 * contiguous.  data and both strides must be multiples of 16 bytes, and
 * token_stride at most 2^24 elements, head_stride 2^31.  Inputs may overlap or
 * repeat (slices of one projection, stride 0); the rows of an output must not
 * overlap. */
typedef struct muon_heads {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} muon_heads;

#define MUON_ATTENTION_ZERO_OUT 1 /* forward: zero out's rows behind the last sequence */
#define MUON_ATTENTION_ZERO_LSE 2 /* forward: and lse's */
#define MUON_ATTENTION_ZERO_DQ 1  /* backward: dq's, dk's, dv's */
#define MUON_ATTENTION_ZERO_DK 2
#define MUON_ATTENTION_ZERO_DV 4

/* out = softmax(scale q k^T) v, and lse[h * tokens + t] (fp32), the natural
 * logarithm of the sum of the exponentials, for the backward call. */
int muon_attention_forward(const muon_attention_desc* desc, const int32_t* cu_seqlens, const muon_heads* q,
                           const muon_heads* k, const muon_heads* v, const muon_heads* out, float* lse,
                           uint32_t flags, void* hip_stream);

/* Bytes of device workspace muon_attention_backward needs; 0 on invalid
 * arguments.  Host-only. */
size_t muon_attention_workspace_size(const muon_attention_desc* desc);

/* Gradients of the forward call, from its inputs, its out and lse, and dout.
 * dq, dk and dv are overwritten (they may be slices of one buffer); dk and dv
 * sum over the query heads of their group. */
int muon_attention_backward(const muon_attention_desc* desc, const int32_t* cu_seqlens, const muon_heads* dout,
                            const muon_heads* q, const muon_heads* k, const muon_heads* v, const muon_heads* out,
                            const float* lse, const muon_heads* dq, const muon_heads* dk, const muon_heads* dv,
                            uint32_t flags, void* workspace, size_t ws_bytes, void* hip_stream);

#define MUON_INDEX_I32 0
#define MUON_INDEX_I64 1

/* Norm of queries and keys for each head, with the position rotation in the
 * same pass: per token and head, with x the head's head_dim elements,
 *   z = x * weight / sqrt(mean(x^2) + eps),
 * and then, in the first `dim` elements of the rotation, each pair (a, b) is
 * turned by its angle, position * frequency:
 *   (a, b) <- (a cos - b sin, b cos + a sin).
 * q and k have heads and weights of their own (weights: p_dtype, head_dim
 * elements, the same for every head; NULL counts as ones).  head_dim: a
 * multiple of 8, at most 128.  dtype: of q, k and every operand in their shape.
 *
 * Positions: `positions` (device, one per token, position_dtype; any value),
 * or NULL: the offset within the token's sequence, with cu_seqlens (device,
 * seqs + 1 int32, as in attention), and the token's number without it.  Rows
 * behind the last sequence of cu_seqlens, if it is given, are never read; in
 * each output they are left as they were, or set to zero when the output's
 * flag is given.  cu_seqlens is not checked: with offsets that are not in
 * order, positions are undefined, but no access leaves the operands.
 *
 * Arithmetic is fp32, results are rounded once.  A position's angle is exact to
 * 2^-31 turns at magnitudes up to 2^32, and off by up to 2^-63 turns times a
 * farther position; its cosine and sine are taken in fp32 and off by up to
 * 2^-23 besides.  Squares are fp32 numbers, too: mean(x^2) + eps has
 * to lie between 2^-120 and 2^120. */
typedef struct muon_qk_norm_desc {
  int64_t tokens;
  int32_t seqs; /* of cu_seqlens */
  int32_t q_heads;
  int32_t k_heads;
  int32_t head_dim;
  int32_t dtype;
  int32_t p_dtype;
  int32_t position_dtype; /* MUON_INDEX_* */
  float eps;              /* >= 0 */
  int32_t reserved;       /* must be 0 */
} muon_qk_norm_desc;

#define MUON_PAIRS_HALVES 0     /* elements i and i + dim / 2 */
#define MUON_PAIRS_NEIGHBOURS 1 /* elements 2 i and 2 i + 1 */

/* frequencies: host array of dim / 2 angles in radians per position, each
 * within [-64, 64], read during the call.  dim: a multiple of 8, at most
 * head_dim; 0, or a NULL rotation, turns nothing. */
typedef struct muon_rotation {
  const double* frequencies;
  int32_t dim;
  int32_t pairs;
} muon_rotation;

#define MUON_QK_ZERO_Q 1 /* zero the rows of q_out (backward: dq) behind the last sequence */
#define MUON_QK_ZERO_K 2 /* and of k_out, dk */

int muon_qk_norm_forward(const muon_qk_norm_desc* desc, const muon_rotation* rotation, const int32_t* cu_seqlens,
                         const void* positions, const muon_heads* q, const muon_heads* k, const void* q_weight,
                         const void* k_weight, const muon_heads* q_out, const muon_heads* k_out, uint32_t flags,
                         void* hip_stream);

/* Bytes of device workspace muon_qk_norm_backward needs for its weight
 * gradients; 0 on invalid arguments.  Host-only. */
size_t muon_qk_norm_workspace_size(const muon_qk_norm_desc* desc);

/* Gradients of the forward call, from its inputs and the gradients dq_out and
 * dk_out of its outputs: dq, dk, and dq_weight and dk_weight (fp32, head_dim
 * elements, overwritten; zero without tokens), of which either may be NULL.
 * workspace (256-byte aligned) may be NULL when both are. */
int muon_qk_norm_backward(const muon_qk_norm_desc* desc, const muon_rotation* rotation, const int32_t* cu_seqlens,
                          const void* positions, const muon_heads* dq_out, const muon_heads* dk_out,
                          const muon_heads* q, const muon_heads* k, const void* q_weight, const void* k_weight,
                          const muon_heads* dq, const muon_heads* dk, float* dq_weight, float* dk_weight,
                          uint32_t flags, void* workspace, size_t ws_bytes, void* hip_stream);

/* Embedding: a table of `vocab` rows (below 2^30) of `cols` elements (at most
 * 2^20), and `tokens` ids (at most 2^30; id_dtype).  Leading dimensions are in
 * elements (0 is read as cols); no alignment beyond an element's is needed.
 * An id outside [0, vocab), such as the padding of a batch, has a row of zeros
 * and passes no gradient on. */
typedef struct muon_embedding_desc {
  int64_t tokens;
  int64_t vocab;
  int64_t cols;
  int64_t ld_table; /* of table and dtable */
  int64_t ld_out;   /* of out and dout */
  int32_t table_dtype;
  int32_t out_dtype;
  int32_t id_dtype; /* MUON_INDEX_* */
  float scale;      /* finite */
  int32_t reserved; /* must be 0 */
} muon_embedding_desc;

/* out[t] = scale * table[ids[t]], in fp32, rounded once.  tokens == 0 does nothing. */
int muon_embedding_forward(const muon_embedding_desc* desc, const void* ids, const void* table, void* out,
                           void* hip_stream);

/* Bytes of device workspace muon_embedding_backward needs; 0 on invalid
 * arguments.  Host-only. */
size_t muon_embedding_workspace_size(const muon_embedding_desc* desc);

#define MUON_EMBEDDING_ACCUMULATE 1 /* add to dtable instead of overwriting it */

/* Gradient of the forward call: dtable[v] = scale * sum of dout[t] over the
 * tokens with ids[t] == v, summed in fp32 and rounded once (dtable:
 * table_dtype, dout: out_dtype).  Rows of no token are set to zero, or with
 * MUON_EMBEDDING_ACCUMULATE neither read nor written. */
int muon_embedding_backward(const muon_embedding_desc* desc, const void* ids, const void* dout, void* dtable,
                            uint32_t flags, void* workspace, size_t ws_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_H */
