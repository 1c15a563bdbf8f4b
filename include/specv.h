/*
 * specv.h -- C ABI of the GB300 speculative-decoding verification library
 * (libspecv.so).
 *
 * Two operations, both defined on the pages this library restates (and the
 * paged key-value cache that the verified target reads, further below):
 *
 *   spec_verify    batched lossless draft verification.  For each request b
 *                  and draft position j < ell_b it forms the temperature
 *                  softmax p of target row j and q of draft row j over the full
 *                  vocabulary, accepts draft token x_j when u_j * q(x_j) <
 *                  p(x_j) (i.e. with probability min(1, p/q)), stops at the
 *                  first rejection n, and emits one more token: a draw from the
 *                  normalised residual max(p_n - q_n, 0) after a rejection, or a
 *                  bonus draw from p of target row ell_b when every tested
 *                  draft was accepted.
 *                  Sources: "UraionSpec: A Faithful Implementation of
 *                  Confidence-Scheduled Speculative Decoding" §2.1, eq.
 *                  (acceptance); "breaking down dspark and its lineage", section
 *                  "Preserving the target distribution during verification";
 *                  "AngelSpec" §1 and §4.1 (verified prefix plus one
 *                  target-generated bonus token).
 *
 *   spec_schedule  confidence-scheduled verify lengths.  Prefix survival
 *                  s_{b,k} = prod_{t<=k} c_{b,t} (s_{b,0} = 1), estimated progress
 *                  A_b(n) = sum_{k<=n} s_{b,k}, candidates taken in order of
 *                  survival (ties: shallower position, then lower request), and
 *                  the budget N = sum_b (ell_b + 1) chosen to maximise
 *                  tau(N) / C(N) against a piecewise-linear round-cost table.
 *                  Sources: "AngelSpec" §4.2, eqs. (19)-(24); "UraionSpec" §3.5,
 *                  Algorithm 1 (hardware-aware prefix scheduler).
 *
 * Conventions for every call:
 *   - All array pointers are DEVICE pointers unless marked host.  The caller
 *     owns every buffer; the library never allocates or frees device memory.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL
 *     is the legacy default stream).  No call synchronises the stream except
 *     spec_read_status.
 *   - A negative return value is an error detected on the host: nothing was
 *     launched and no output was written.  Errors found in device data (a bad
 *     token id, a NaN row, ...) mark the affected request (out_accept_len = -1,
 *     its tokens -1) and set a status word in the workspace, read with
 *     spec_read_status.  For spec_verify the word holds the status of the most
 *     recent call on that workspace (each call resets it); for the schedulers
 *     it is sticky until read.
 *   - Every device wait in the kernels is bounded; on expiry the call reports
 *     SPEC_ERR_TIMEOUT in the status word and the kernel returns.
 */
#ifndef SPECV_H
#define SPECV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* spec_stream_t; /* a cudaStream_t */

/* SPEC_F32 and SPEC_BF16: logits.  The cache calls also take SPEC_F16, and
 * SPEC_E4M3 (8 bits: 4 of exponent, 3 of mantissa) for the cache itself. */
typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1, SPEC_F16 = 2, SPEC_E4M3 = 3 } spec_dtype;

enum {
    SPEC_OK = 0,
    SPEC_ERR_NULL = -1,        /* a required pointer is NULL */
    SPEC_ERR_SHAPE = -2,       /* B, gamma, V or min_len out of range */
    SPEC_ERR_ALIGN = -3,       /* a pointer is not aligned to its element size / 16 B */
    SPEC_ERR_TEMPERATURE = -4, /* temperature not 0 and not in [1e-4, 1e4], or NaN */
    SPEC_ERR_VERIFY_LEN = -5,  /* device: verify_len[b] outside [0, gamma] */
    SPEC_ERR_TOKEN = -6,       /* device: draft token outside [0, V) at a tested position */
    SPEC_ERR_WORKSPACE = -7,   /* workspace smaller than the *_workspace_bytes value */
    SPEC_ERR_COST_TABLE = -8,  /* cost table: n outside [1, 32], knots not increasing, cost <= 0 */
    SPEC_ERR_NONFINITE = -9,   /* device: a needed logit row has a NaN, +inf, no finite value, or (T > 0)
                                  a largest |z| * log2(e) / T beyond the fp32 range */
    SPEC_ERR_TIMEOUT = -10,    /* device: a bounded wait expired (results of the call invalid) */
    SPEC_ERR_CUDA = -11,       /* a CUDA runtime call failed (launch, attribute query) */
    SPEC_ERR_UNIFORM = -12,    /* device: a used uniform outside [0, 1) */
    SPEC_ERR_CONFIDENCE = -13, /* device: a confidence outside [0, 1] or NaN */
    SPEC_ERR_ROW_INDEX = -14,  /* device: packed rows of a request outside the packed arrays */
    SPEC_ERR_POOL = -15,       /* device: no free pages left for a request */
    SPEC_ERR_CACHE_LEN = -16,  /* device: a cache length outside the request's page table or pages */
    SPEC_ERR_PAGE = -17,       /* device: a needed page table entry outside [0, pages), or a page with no reference */
    SPEC_ERR_REQUEST = -18,    /* device: a request id outside [0, B), or one that a call may not name twice */
    SPEC_ERR_PLAN = -19        /* device: a plan that spec_share_plan did not make, or made for other sizes */
};

/* Limits of this build. */
#define SPEC_MAX_BATCH 4096
#define SPEC_MAX_GAMMA 32
#define SPEC_MAX_SCHED_CANDIDATES 16384 /* B * (gamma - min_len) for spec_schedule */
#define SPEC_MAX_HEAD_DIM 256           /* of a cache; a multiple of 8, of 16 for SPEC_E4M3 */

/* ------------------------------------------------------------- verification */

/* Bytes of device workspace spec_verify needs for these sizes (0 if the sizes
 * are out of range).  Depends only on (B, gamma, V, dt). */
size_t spec_verify_workspace_bytes(int B, int gamma, int V, spec_dtype dt);

/*
 * Batched verification of B requests with up to gamma draft tokens each.
 *
 *   target_logits  [B, gamma+1, V] row-major, dt; row j of request b holds the
 *                  target logits for draft position j (row gamma: the position
 *                  after the last draft).  Aligned to the element size.
 *   draft_logits   [B, gamma, V] row-major, dt; may be NULL when temperature == 0
 *                  or gamma == 0 (never read then).
 *   draft_tokens   [B, gamma] int32; only positions j < ell_b are read.
 *   verify_len     [B] int32, ell_b in [0, gamma]; NULL means gamma for all.
 *                  Rows j > ell_b (target) and j >= ell_b (draft) are not read.
 *   temperature    0 = greedy (accept while x_j == argmax of target row j,
 *                  lowest index on ties; emit the argmax of row n); otherwise
 *                  p = softmax(z / T) with T in [1e-4, 1e4].
 *   uniforms       [B, gamma+2] fp32 in [0,1): slot j < gamma is the accept test
 *                  of position j, slot gamma the residual draw, slot gamma+1 the
 *                  bonus draw.  Not read (may be NULL) when temperature == 0.
 *   out_tokens     [B, gamma+1] int32: x_0..x_{n-1}, then the drawn token at
 *                  position n, then -1.
 *   out_accept_len [B] int32: n, the number of accepted drafts (-1 if the
 *                  request's inputs were invalid).
 *   workspace      device scratch of at least spec_verify_workspace_bytes(),
 *                  16-byte aligned; holds the status word of the most recent
 *                  call (reset by each call, read and cleared by
 *                  spec_read_status).  Its contents need no initialisation.
 *                  Two calls sharing one workspace must be ordered on the same
 *                  stream.
 * Draws use the inverse CDF: the token is the smallest v whose running sum of
 * weights exceeds u * (sum of weights).  Returns SPEC_OK or a host-detected
 * error (nothing launched).  B == 0 returns SPEC_OK without launching.
 * Stream order: the call's kernels are programmatic dependent launches, each
 * waiting (griddepcontrol.wait) for the work before it on `stream` before
 * touching global memory, and each letting the next kernel be scheduled early.
 * A caller's own kernel launched right after with programmatic stream
 * serialization must likewise wait before reading the outputs; ordinary
 * launches, copies and events see them complete.
 */
int spec_verify(const void* target_logits, const void* draft_logits, spec_dtype dt, int B,
                int gamma, int V, const int32_t* draft_tokens, const int32_t* verify_len,
                float temperature, const float* uniforms, int32_t* out_tokens,
                int32_t* out_accept_len, void* workspace, size_t workspace_bytes,
                spec_stream_t stream);

/*
 * Verification on packed logits ("AngelSpec" §4.2, "Packing and correctness":
 * after the budget is chosen, the unequal request prefixes are packed into one
 * dense verification batch and only those positions reach the target model).
 * Same method, outputs, workspace and errors as spec_verify; only where the
 * logit rows live differs:
 *   target_logits  [K_target, V], dt: request b's target rows 0..ell_b are rows
 *                  target_row[b] .. target_row[b] + ell_b.
 *   draft_logits   [K_draft, V], dt: request b's draft rows 0..ell_b-1 are rows
 *                  draft_row[b] .. draft_row[b] + ell_b - 1 (not read when
 *                  temperature == 0; may then be NULL, as may draft_row).
 *   target_row, draft_row  [B] int32 device arrays (the row index).  Any
 *                  placement is allowed (dense request-major packing is what
 *                  spec_pack_rows writes); a request whose rows fall outside
 *                  [0, K) is marked invalid with SPEC_ERR_ROW_INDEX and none of
 *                  its rows are read.
 *   verify_len     [B] int32 as for spec_verify (NULL: gamma for all).
 * Fixed launch shapes for given (B, gamma, V, dt, temperature), no host
 * synchronisation: capturable in a CUDA graph, one per batch shape.
 */
int spec_verify_packed(const void* target_logits, int K_target, const void* draft_logits, int K_draft,
                       const int32_t* target_row, const int32_t* draft_row, spec_dtype dt, int B,
                       int gamma, int V, const int32_t* draft_tokens, const int32_t* verify_len,
                       float temperature, const float* uniforms, int32_t* out_tokens,
                       int32_t* out_accept_len, void* workspace, size_t workspace_bytes,
                       spec_stream_t stream);

/*
 * Dense request-major packing of ragged prefixes (the layout of the packed
 * batch in "AngelSpec" §4.2): from verify_len [B] (device), writes
 *   target_row[b] = sum_{b' < b} (ell_b' + 1),   draft_row[b] = sum_{b' < b} ell_b',
 *   totals[0] = K_target = sum_b (ell_b + 1),    totals[1] = K_draft = sum_b ell_b
 * (all device int32; a verify length outside [0, gamma] counts as no rows).
 * One launch, no host synchronisation.  Requires B <= 4096.
 */
int spec_pack_rows(const int32_t* verify_len, int B, int gamma, int32_t* target_row, int32_t* draft_row,
                   int32_t* totals, spec_stream_t stream);

/*
 * Diagnostics of the last spec_verify that used `workspace` (same B, gamma, V,
 * dt; stream-ordered after it).  Each output is a device pointer or NULL:
 *   px, qx      [B, gamma] fp64: p(x_j), q(x_j) for j < ell_b, NaN elsewhere
 *               (and at temperature 0).
 *   resid_mass  [B] fp64: the total weight of the final draw, sum_v max(p - q, 0)
 *               after a rejection, sum_v p_v (= 1 up to rounding) for a bonus
 *               draw; NaN at temperature 0 or for an invalid request.
 *   status      [B] int32: per-request status (SPEC_OK or a device error code).
 */
int spec_verify_stats(const void* workspace, size_t workspace_bytes, int B, int gamma, int V,
                      spec_dtype dt, double* px, double* qx, double* resid_mass, int32_t* status,
                      spec_stream_t stream);

/* --------------------------------------------------------------- scheduling */

/* Piecewise-linear round cost C(N): knots (tokens[i], cost_ms[i]), i < n, with
 * strictly increasing tokens and positive costs; linear between knots, flat
 * beyond both ends.  Evaluated in fp64 as
 *   cost_ms[i] + ((N - tokens[i]) * (cost_ms[i+1] - cost_ms[i])) / (tokens[i+1] - tokens[i])
 * for tokens[i] <= N < tokens[i+1]. */
typedef struct {
    int n;
    double tokens[32];
    double cost_ms[32];
} spec_cost_table;

typedef enum {
    SPEC_SCHED_EXACT = 0,      /* first budget N that maximises tau(N)/C(N) over every N */
    SPEC_SCHED_ALGORITHM1 = 1, /* Algorithm 1: add candidates while tau/C strictly improves */
    SPEC_SCHED_DCUT = 2        /* D-cut: the table's "tokens" are budget ratios rho_i in (0, 1]
                                  (strictly increasing) and its costs C(B, rho_i); the budget is
                                  K_i = max(B(min_len+1), ceil(rho_i * B(gamma+1))) and the first
                                  maximum of tau(K_i) / C_i is taken ("AngelSpec" §4.2,
                                  eqs. (22)-(24)) */
} spec_sched_mode;

/* Bytes of device workspace spec_schedule needs (its status word). */
size_t spec_schedule_workspace_bytes(int B, int gamma);

/*
 * Per-request verify lengths for B requests with gamma draft positions.
 *   confidence      [B, gamma] fp32 in [0, 1]; confidence[b][k-1] is c_{b,k}.
 *   cost            HOST pointer, copied by value into the launch.
 *   min_len         every request keeps at least min_len drafts (0 <= min_len <= gamma).
 *   sts_temperature HOST [gamma] fp32 > 0 or NULL: Sequential Temperature
 *                   Scaling ("UraionSpec" §2.4): the scheduler uses the calibrated
 *                   confidence c_{b,k}^(1/T_k) (fp64 pow) in place of c_{b,k}.
 *   out_verify_len  [B] int32 in [min_len, gamma] (all -1 if a confidence is invalid).
 * Numbers: survival products are fp64, left to right; each survival is then
 * rounded to a multiple of 2^-46 (nearest, ties to even).  Candidates are
 * ordered by that value (ties: shallower position, then lower request) and
 * progress values are exact integer sums of it, so tau(N) does not depend on
 * the order of summation; objectives tau / C are fp64 with explicit rounding.
 * Results are reproducible bit for bit.  The status word in `workspace` is
 * sticky: set on an error, cleared by spec_read_status (zero the workspace
 * once before first use).  Requires B <= 4096, gamma <= 32,
 * B * (gamma - min_len) <= 16384.  One thread-block cluster per call.
 */
int spec_schedule(const float* confidence, int B, int gamma, const spec_cost_table* cost,
                  int min_len, spec_sched_mode mode, const float* sts_temperature,
                  int32_t* out_verify_len, void* workspace, size_t workspace_bytes,
                  spec_stream_t stream);

/*
 * Static verify lengths ("breaking down dspark and its lineage", section
 * "Verify smarter, not longer": a static confidence threshold, zero recovering
 * fixed-length verification; "UraionSpec" §3.5, the fixed-length and
 * static-threshold StaticScheduler).  Request b keeps its leading positions k
 * whose (optionally STS-calibrated) confidence is at least `threshold`, at most
 * max_len and at least min_len of them: threshold <= 0 gives fixed length
 * max_len, and then confidence may be NULL.  0 <= min_len <= max_len <= gamma.
 * Requests are independent: one with a confidence outside [0, 1] (or NaN) gets
 * verify length -1 and the status word SPEC_ERR_CONFIDENCE; the others are
 * scheduled as usual.  Other arguments as for spec_schedule; any B <= 4096.
 */
int spec_schedule_static(const float* confidence, int B, int gamma, float threshold, int max_len,
                         int min_len, const float* sts_temperature, int32_t* out_verify_len,
                         void* workspace, size_t workspace_bytes, spec_stream_t stream);

/*
 * Host-side STS fit ("UraionSpec" §2.4 and §3.6): for positions k = 1..gamma
 * in order, the temperature T_k on the grid (i+1)/10, i = 0..99 (the 100
 * points of 0.1..10) minimising the 15-bin expected calibration error of the
 * cumulative survival prod_{j<k} c_j^(1/T_j) * c_k^(1/T) against the labels
 * [accept_len >= k]; earlier positions keep their chosen T; ties go to the
 * smaller T.  All HOST pointers: confidence [n, gamma] fp32, accept_len [n]
 * int32 (observed with verify_len = gamma), out_temperature [gamma] fp32,
 * out_ece [gamma] fp64 or NULL.  Runs on the CPU, fp64.
 */
int spec_sts_fit(const float* confidence, const int32_t* accept_len, int n, int gamma,
                 float* out_temperature, double* out_ece);

/* ------------------------------------------- the target's key-value cache */

/*
 * A verification round needs the target's keys and values of every position so
 * far.  They live in pages of page_size tokens, and request b's position t is
 * token t % page_size of page page_table[b][t / page_size].  One round is
 *   spec_reserve_pages   pages for the tested tokens (positions cache_len[b] ..
 *                        cache_len[b] + ell_b: the last emitted token and the
 *                        ell_b drafts);
 *   spec_append_kv       rotary positions, and their keys and values into the
 *                        pages (per layer);
 *   spec_attend          their attention over the cache (per layer);
 *   spec_verify          on the logits that follow;
 *   spec_commit_pages    cache_len[b] += accept_len[b] + 1, and the pages that
 *                        held rejected drafts only are given back.
 * A single decoded token is the same with gamma = 0.  Query rows are laid out
 * as the target logits are: padded [B, gamma+1, ...], or packed with the row
 * index that spec_pack_rows writes (target_row).  No call synchronises; all
 * can be captured into one CUDA graph.
 *
 * State, all int32 on the device, owned by the caller:
 *   page_table [B, max_pages]  page ids; -1 where a request has no page
 *   num_pages  [B]             slots of the table that a request holds (a slot
 *                              behind a sliding window may be -1 all the same)
 *   ref_count  [pages]         table entries that name a page; 0 is free
 *   cache_len  [B]             positions whose keys and values are valid
 * Every call names the lowest free pages first, in request order, so results
 * do not depend on timing.
 *
 * Errors in device data set the workspace's status word (sticky until
 * spec_read_status; zero the workspace once before first use).
 */
typedef struct {
    void* k;            /* device: keys of layer 0, page 0, token 0, head 0; 16-byte aligned */
    void* v;            /* device: values, same strides */
    spec_dtype dt;      /* SPEC_F32, SPEC_BF16, SPEC_F16 or SPEC_E4M3 */
    int layers;         /* fork and compact move a page's tokens in every layer; others use layer 0 */
    int pages, page_size, kv_heads, head_dim; /* head_dim: a multiple of 8 (SPEC_E4M3: 16), at most 256 */
    /* strides in elements (16-byte multiples; the head_dim values are adjacent) */
    long long layer_stride, page_stride, token_stride, head_stride;
    const float* k_scale; /* device [kv_heads], SPEC_E4M3 only: the entry stands for entry * scale; */
    const float* v_scale; /* NULL: 1 */
} spec_cache;

/* Bytes of device workspace of spec_append_kv, spec_append_rows, spec_map_rows, spec_reserve_pages,
 * spec_commit_pages, spec_free_pages, spec_fork_pages (pages may be 0 for
 * these) and spec_compact_pages; 0 if out of range. */
size_t spec_cache_workspace_bytes(int B, int pages);

/* Bytes of device workspace of spec_attend for these sizes (0 if out of range). */
size_t spec_attend_workspace_bytes(int B, int gamma, int q_heads, int kv_heads, int head_dim);

/*
 * Attention of the tested tokens over the cache.  For query row j of request
 * b, at position p = cache_len[b] + j (0 <= j <= ell_b), and head h:
 *   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale * q . k_t),
 * over the visible positions t <= p with window == 0, p - t < window or t <
 * sinks; k_t and v_t of KV head h / (q_heads / kv_heads).
 *   q            device, dt (SPEC_F32, SPEC_BF16 or SPEC_F16), row r and head h
 *                at q + r * q_row_stride + h * q_head_stride elements (16-byte
 *                multiples); head_dim adjacent values.
 *   q_row        NULL: request b's rows are b*(gamma+1) + j (padded).  Else
 *                [B] int32: rows q_row[b] + j of `rows` rows (packed); a request
 *                whose rows fall outside is skipped with SPEC_ERR_ROW_INDEX.
 *   verify_len   [B] int32, ell_b in [0, gamma]; NULL means gamma for all.  A
 *                request with another value has no rows (SPEC_ERR_VERIFY_LEN).
 *   cache        dt equal to q's, or SPEC_E4M3 under SPEC_BF16 / SPEC_F16 rows.
 *                Positions cache_len[b] .. cache_len[b] + ell_b must have been
 *                appended.  Entries that no row sees have no influence, whatever
 *                they hold; pages that no row sees any position of may be missing.
 *   scale        finite; normally 1 / sqrt(head_dim).
 *   window       0: all earlier positions; else the last `window` positions,
 *                the token's own included.  sinks: first positions that stay
 *                visible under a window.
 *   out          [rows, q_heads, head_dim] dt, contiguous, 16-byte aligned.
 *                Rows that no request has are left as they were.
 *   out_lse      [rows, q_heads] fp32 or NULL: log sum_t w_t.
 * A request whose positions do not fit its page table (SPEC_ERR_CACHE_LEN), or
 * with a needed entry that is not a page (SPEC_ERR_PAGE), gets NaN rows.  A
 * value that is not finite reaches only the rows that see it.  Two launches.
 * Numbers: scores, running maximum and sum, and the output are fp32; with
 * 16-bit rows the weights are rounded to that type (to fp16 under a SPEC_E4M3
 * cache) for the product with v.  fp16 weights are scaled to its upper end: what
 * is below 2^-25 of the largest is held to 2^-36 of that.  Bit-reproducible for given arguments; how a
 * long cache is split depends on the whole batch's lengths, so a request's
 * last bits may change with its company.  Two calls that share a workspace
 * must be ordered on one stream.
 */
int spec_attend(const void* q, long long q_row_stride, long long q_head_stride, spec_dtype dt, int q_heads,
                const spec_cache* cache, const int32_t* page_table, int max_pages, const int32_t* cache_len,
                const int32_t* verify_len, const int32_t* q_row, int rows, int B, int gamma, float scale,
                int window, int sinks, void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                spec_stream_t stream);

/*
 * Attention of a batch whose requests share prefixes (branches of spec_fork_pages,
 * or any requests whose page tables begin with the same pages): the plan, made once
 * for a round and used by all its layers.
 *
 * Requests whose first max(1, ceil(least / page_size)) pages are the same, and full, are
 * a class, the lowest of them its head.  depth_b is the number of leading entries that
 * request b's row of the page table has like the head's, among pages that both have
 * filled (cache_len / page_size).  Of the depths d with d * page_size >= least, the one
 * with the largest d * (members of depth >= d but the head), on ties the smallest, makes
 * those members and the head a group that shares d pages.  The head leaves the class in
 * any case, and the rest is taken again until none is left.
 *   page_table .. B, gamma   as for spec_attend; verify_len and q_row may be NULL.
 *   least          shorter prefixes (in positions) are not shared; about 256.
 *   out_leader     [B] int32: the group's head; b itself if alone.
 *   out_shared     [B] int32: the pages that the group shares; 0 if alone.
 *   plan           device, spec_share_plan_bytes(), 16-byte aligned; needs no
 *                  initialisation.  Its first word is the status of the latest call
 *                  (spec_read_status): SPEC_ERR_VERIFY_LEN, SPEC_ERR_ROW_INDEX or
 *                  SPEC_ERR_CACHE_LEN of a request, which is then alone, with the rows
 *                  that it has in spec_attend.
 * The plan holds the lengths and rows of this call, and no page ids: it is to be
 * made again when they change or when a shared entry does.  Rows of two requests may
 * not overlap.  One launch.
 *
 * A plan pays where groups save much: (members - 1) * shared positions from about
 * 16,000 on for requests of one to five rows, from about 100,000 on for 17 (32/8 heads
 * of 128, bf16, a layer on the device: 64 requests of one token behind 2048 positions
 * spec_attend 89 us, spec_attend_shared 34; 4 behind 1024 12 and 14; 64 of 17 rows behind
 * 2048 80 and 81, behind 8192 245 and 170).  Below, spec_attend is the faster call.
 */
size_t spec_share_plan_bytes(int B, int gamma, int rows);
int spec_share_plan(const int32_t* page_table, int max_pages, int page_size, const int32_t* cache_len,
                    const int32_t* verify_len, const int32_t* q_row, int rows, int B, int gamma, int least,
                    int32_t* out_leader, int32_t* out_shared, void* plan, size_t plan_bytes, spec_stream_t stream);

/* Bytes of device workspace of spec_attend_shared; 0 if out of range (rows * q_heads
 * and B * (gamma+1) * q_heads / kv_heads are below 2^31 - 256).  `rows` is that of the
 * plan: B * (gamma+1), or the packed rows. */
size_t spec_attend_shared_workspace_bytes(int B, int gamma, int rows, int q_heads, int kv_heads, int head_dim);

/*
 * spec_attend (without a window) by a plan: the positions that a group shares are
 * read once for the rows of all its members.  rows, B, gamma, max_pages and the
 * cache's page_size are those that the plan was made with (else SPEC_ERR_PLAN, and
 * nothing is written); lengths and rows are the plan's.  Other arguments, errors of
 * requests and numbers as for spec_attend; rows of shared prefixes are sums of two
 * parts, joined in fp32.  A page of a shared prefix is taken from the row of the
 * page table of the group's head.  The workspace holds nothing between calls but
 * its status word; two calls that share one must be ordered on one stream.  After a
 * wait that ran out (SPEC_ERR_TIMEOUT) all rows of requests are NaN.  Two launches.
 */
int spec_attend_shared(const void* q, long long q_row_stride, long long q_head_stride, spec_dtype dt, int q_heads,
                       const spec_cache* cache, const int32_t* page_table, int max_pages, const void* plan,
                       size_t plan_bytes, int rows, int B, int gamma, float scale, void* out, float* out_lse,
                       void* workspace, size_t workspace_bytes, spec_stream_t stream);

/*
 * Rotary positions and the append of the tested tokens' keys and values.  Row
 * j of request b is at position p = cache_len[b] + j.  Pair i of the first
 * `rotary_dim` values of every q and k head is turned by the angle p * f_i:
 *   (x, y) -> mscale * (x cos - y sin, x sin + y cos),
 * pair i = values (i, i + rotary_dim/2), or (2i, 2i+1) if `interleaved`; the
 * other values pass unchanged.  The turned k and v go to the request's pages
 * (times the reciprocal of their scales, clamped to +-448 and rounded to nearest
 * even for SPEC_E4M3), the turned q to out_q.
 *   q, k, v      device, dt, row r and head h at r * row_stride + h * head_stride
 *                elements (16-byte multiples).
 *   row, rows    as q_row and rows of spec_attend.
 *   turns        device [rotary_dim / 2] uint64, or NULL with rotary_dim 0:
 *                f_i / (2 pi) as a fraction of 2^64 (the angle of any position
 *                is then an exact wrapping product).
 *   out_q        [rows, q_heads, head_dim] dt, contiguous; may be q itself if q
 *                is contiguous.  Rows that no request has are left as they were.
 * A position outside the page table (SPEC_ERR_CACHE_LEN) or without a page
 * (SPEC_ERR_PAGE) is not stored; its q row is turned all the same.
 * cache->dt must be dt, or SPEC_E4M3 under SPEC_BF16 / SPEC_F16.
 */
int spec_append_kv(const void* q, long long q_row_stride, long long q_head_stride, const void* k, const void* v,
                   long long k_row_stride, long long k_head_stride, long long v_row_stride,
                   long long v_head_stride, spec_dtype dt, int q_heads, const spec_cache* cache,
                   const int32_t* page_table, int max_pages, const int32_t* cache_len, const int32_t* verify_len,
                   const int32_t* row, int rows, int B, int gamma, const uint64_t* turns, int rotary_dim,
                   int interleaved, float mscale, void* out_q, void* workspace, size_t workspace_bytes,
                   spec_stream_t stream);

/*
 * Rotary positions and the append of rows by their slots: any number of rows, of
 * any requests (a step's prompts and single tokens as spec_map_rows lists them; a
 * drafter's context, which has no queries).  Row r, at position[r], is turned as by
 * spec_append_kv, and its k and v go to token slot[r] % page_size of page slot[r] /
 * page_size.
 *   position     [rows] int32; below 0: no row (its out_q is left as it was).
 *   slot         [rows] int64; below 0: the row is turned but not stored, and so is
 *                one behind the cache's last slot (SPEC_ERR_PAGE).  Two rows of one
 *                call may not name the same slot.
 *   q_heads      0 where there are no queries (q and out_q are not used then).
 * Other arguments as for spec_append_kv.  One launch.
 */
int spec_append_rows(const void* q, long long q_row_stride, long long q_head_stride, const void* k, const void* v,
                     long long k_row_stride, long long k_head_stride, long long v_row_stride,
                     long long v_head_stride, spec_dtype dt, int q_heads, const spec_cache* cache,
                     const int32_t* position, const int64_t* slot, int rows, const uint64_t* turns, int rotary_dim,
                     int interleaved, float mscale, void* out_q, void* workspace, size_t workspace_bytes,
                     spec_stream_t stream);

/*
 * Page tables and a slot map from the requests' lengths: new_len[b] positions, of any
 * number, behind cache_len[b] (a prompt's, a part of one, a single token, none).
 * Request b's slots are grown to hold them, with the lowest free pages in request
 * order as by spec_reserve_pages, and their rows are listed one request behind the
 * other: rows out_first[b] .. out_first[b] + new_len[b] - 1.
 *   out_first     [B+1] int32: sums of new_len; out_first[B] is the number of rows.  Sums
 *                 stop at 2^30 - 1.
 *   out_request   [rows] int32: b.
 *   out_position  [rows] int32: cache_len[b] + row - out_first[b].
 *   out_slot      [rows] int64: page * page_size + position % page_size, for
 *                 spec_append_rows.
 *   rows          what the arrays hold, below 2^30 - 1; rows behind the last one get -1 in all three.
 *   out_status    [B] int32: SPEC_OK, SPEC_ERR_POOL, SPEC_ERR_CACHE_LEN (a negative
 *                 length, more than max_pages slots) or SPEC_ERR_ROW_INDEX (rows that
 *                 end behind the arrays).  Such a request is left as it was, and its
 *                 rows have slot -1 (with a negative new_len it has none, with a
 *                 negative cache_len they have position -1).
 * A position whose entry is not a page gets slot -1 (SPEC_ERR_PAGE).  Once the rows
 * are appended, cache_len + new_len is the new length; spec_commit_pages with accept_len
 * = new_len - 1 sets it, and with -1 gives the new pages back.  Two launches.  With
 * B = 0 only out_first[0] = 0 and the -1 of all rows are written (out_first NULL: nothing).
 */
int spec_map_rows(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int pages, const int32_t* cache_len,
                  const int32_t* new_len, int B, int max_pages, int page_size, int rows, int32_t* out_first,
                  int32_t* out_request, int32_t* out_position, int64_t* out_slot, int32_t* out_status, void* workspace,
                  size_t workspace_bytes, spec_stream_t stream);

/*
 * Pages for the tested tokens: request b's slots are grown to hold cache_len[b]
 * + ell_b + 1 positions (verify_len NULL: gamma for all), with the lowest free
 * pages in request order.  Where the pool runs out, the first request that does
 * not fit and every growing request after it get none.
 *   out_status [B] int32: SPEC_OK, SPEC_ERR_POOL, SPEC_ERR_VERIFY_LEN or
 *   SPEC_ERR_CACHE_LEN (more than max_pages slots, or a negative length); a
 *   request with an error is left as it was.
 */
int spec_reserve_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int pages,
                       const int32_t* cache_len, const int32_t* verify_len, int B, int gamma, int max_pages,
                       int page_size, int32_t* out_status, void* workspace, size_t workspace_bytes,
                       spec_stream_t stream);

/*
 * After verification: out_cache_len[b] = cache_len[b] + accept_len[b] + 1 (b's
 * last emitted token and its accepted drafts), slots behind it are given back.
 * accept_len[b] = -1 (an invalid request) keeps cache_len[b].  With window > 0,
 * pages that hold neither a position below `sinks` nor one that the next token
 * (at out_cache_len[b]) sees are given back too, and their entries become -1.
 *   out_cache_len [B]: may be cache_len.
 * An accept length below -1, or a new length beyond the slots held, leaves the
 * request as it was (SPEC_ERR_CACHE_LEN).
 */
int spec_commit_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int pages,
                      const int32_t* cache_len, const int32_t* accept_len, int B, int max_pages, int page_size,
                      int window, int sinks, int32_t* out_cache_len, void* workspace, size_t workspace_bytes,
                      spec_stream_t stream);

/* Ends requests: gives back all pages of the n requests in `requests` [n]
 * (device), and sets their num_pages and cache_len to 0.  Naming one twice is
 * allowed; an id outside [0, B) is skipped (SPEC_ERR_REQUEST).  To the other
 * calls the place is then a request of length 0, with its tested tokens: at
 * verify_len 0 spec_reserve_pages takes one page for it in each round, and
 * spec_commit_pages with an accept length of -1 gives that back. */
int spec_free_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int pages, int32_t* cache_len,
                    const int32_t* requests, int n, int B, int max_pages, void* workspace, size_t workspace_bytes,
                    spec_stream_t stream);

/*
 * Branches: request dst[i] becomes a copy of request src[i] (i < n): what dst
 * held is given back, its slots name src's full pages (one more reference
 * each), and the partial last page is copied into a fresh one, in every layer
 * of `cache`, its first cache_len % page_size tokens.  num_pages[dst] and
 * cache_len[dst] follow.  One src may have many dst.
 *   out_status [n] int32: SPEC_OK; SPEC_ERR_REQUEST for an id outside [0, B), a
 *   dst named twice, or a dst that is also a src of this call (left as it was);
 *   SPEC_ERR_CACHE_LEN where src's length exceeds its slots, SPEC_ERR_PAGE where
 *   its last page is missing (left as it was); SPEC_ERR_POOL where no free page
 *   was left for the copy, in the order of i (dst is then empty).
 */
int spec_fork_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int32_t* cache_len,
                    const int32_t* src, const int32_t* dst, int n, int B, int max_pages, const spec_cache* cache,
                    int32_t* out_status, void* workspace, size_t workspace_bytes, spec_stream_t stream);

/*
 * Compaction: the N referenced pages move to the ids 0..N-1.  Pages below N
 * stay; the k-th lowest referenced page from N on goes to the k-th lowest free
 * one, with its tokens of all layers, and the tables and counts are renamed.
 * Table entries behind num_pages[b] become -1.  Whoever else keeps a page's id has
 * to keep it in a table too: a referenced page moves whether an entry names it or not.
 *   out_page_table [B, max_pages], out_ref_count [pages]: may be page_table and
 *   ref_count.  out_total [1] int32: N.
 */
int spec_compact_pages(const int32_t* page_table, const int32_t* num_pages, const int32_t* ref_count, int B,
                       int max_pages, const spec_cache* cache, int32_t* out_page_table, int32_t* out_ref_count,
                       int32_t* out_total, void* workspace, size_t workspace_bytes, spec_stream_t stream);

/* ------------------------------------------------- verification, no workspace */

/* Size of the device scratch array that spec_verify_static uses (8 MiB on each
 * device that loads the library, held until the process exits). */
#define SPEC_STATIC_WORKSPACE_BYTES (8u << 20)

/*
 * spec_verify without a workspace argument, for callers that cannot allocate
 * device memory where they verify (an allocator that must not grow inside a
 * capture or a latency-critical loop, a plugin handed only input and output
 * buffers, a runtime with a memory budget fixed at start-up).  It has no
 * counterpart on the pages: it is the same verification as spec_verify, with
 * the scratch taken from a statically sized array in device memory instead
 * of from the caller.
 *
 * Arguments, outputs and results are those of spec_verify.  It allocates
 * nothing (no cudaMalloc, no cudaFree).
 *   - Returns SPEC_ERR_WORKSPACE, launching nothing, when
 *     spec_verify_workspace_bytes(B, gamma, V, dt) exceeds
 *     SPEC_STATIC_WORKSPACE_BYTES (e.g. B=64, gamma=16, V=131072 bf16 needs
 *     about 1.1 MiB; B=256, gamma=16, V=131072 about 4.3 MiB).
 *   - Every call looks up the array's device address on the current device
 *     (so an address never outlives a cudaDeviceReset).  The first lookup on a
 *     device may load the library's device code; make that first call before
 *     any stream capture.
 *   - Every call on a device uses the same array and leaves its contents
 *     behind.  Nothing in it needs to start at zero.  Calls that can overlap
 *     on the GPU (different streams without ordering, or several host threads)
 *     race on it: order them on one stream.
 *   - The device status word lives in that array and cannot be read through
 *     this call; invalid requests are still reported per request
 *     (out_accept_len = -1).
 */
int spec_verify_static(const void* target_logits, const void* draft_logits, spec_dtype dt, int B, int gamma,
                       int V, const int32_t* draft_tokens, const int32_t* verify_len, float temperature,
                       const float* uniforms, int32_t* out_tokens, int32_t* out_accept_len,
                       spec_stream_t stream);

/*
 * Self-test of the bounded waits.  The streaming kernel waits on mbarriers for
 * its own bulk copies; every such wait gives up after 2 s of the GPU's global
 * timer and the call then reports SPEC_ERR_TIMEOUT instead of hanging.  This
 * call runs the same wait routine with a limit of limit_ns (1e3 .. 2e9):
 *   status[0], elapsed_ns[0]: a wait on a barrier nothing completes; expect
 *                             SPEC_ERR_TIMEOUT after about limit_ns;
 *   status[1], elapsed_ns[1]: a wait on a completed phase; expect SPEC_OK at once.
 * status [2] int32 and elapsed_ns [2] uint64 are device pointers.  One launch
 * of one warp.
 */
int spec_selftest_wait(long long limit_ns, int32_t* status, unsigned long long* elapsed_ns,
                       spec_stream_t stream);

/*
 * Test hook of the timeout paths (off by default).  The streaming kernel: while
 * `on` is nonzero, later spec_verify calls (made from any thread) treat the
 * first copy wait of every warp of the streaming kernel as expired, without
 * waiting for it.  The warps then let their copies in flight land (each wait
 * bounded as usual) and stop; the call marks every request invalid
 * (out_accept_len = -1) and its status word reads SPEC_ERR_TIMEOUT.  No copy
 * is lost and nothing hangs; it exercises the path that a bulk copy which
 * never completes would take.  The tensor-core attention kernel (spec_attend,
 * more than 16 rows a KV head): the first wait for query rows counts as run out,
 * with copies in flight.  All roles then run to their ends without waiting, the
 * copies land, and the status word reads SPEC_ERR_TIMEOUT; the rows hold
 * anything (those of spec_attend_shared, whose tensor-core kernel is the same: NaN).
 * Returns SPEC_OK.
 */
int spec_selftest_expire_first_wait(int on);

/* ------------------------------------------------------------------ status */

/* Synchronises `stream`, reads the device status word of `workspace` into
 * *status and clears it: for a verification workspace the status of the most
 * recent call on it, for a scheduler workspace the first error since the last
 * read.  Returns SPEC_OK or SPEC_ERR_CUDA. */
int spec_read_status(void* workspace, spec_stream_t stream, int* status);

/* A static English description of a status code. */
const char* spec_status_string(int status);

/* ---------------------------------------------------------------- profiling */

/* Registers two cudaEvent_t handles (as void*) that later spec_verify calls
 * record on their stream immediately before and after the row-statistics
 * kernel (the HBM-streaming pass), so a caller can time that kernel alone.
 * Pass NULL, NULL to stop.  Process-wide setting: calls racing with it on
 * other threads may record the old or the new pair. */
int spec_profile_events(void* before_row_stats, void* after_row_stats);

/* Number of kernels one spec_verify call launches for these arguments
 * (depends on temperature == 0 and B == 0 only). */
int spec_verify_kernel_count(int B, float temperature);

#ifdef __cplusplus
}
#endif

#endif /* SPECV_H */
