/*
 * dflash2.h -- C ABI of the MI355X (gfx950) DFlash 2 path selector.
 *
 * The selector is described on the page "DFlash 2: Keep Drafting Parallel",
 * section "A Lightweight Path Selector": keep the top 16 candidates of the
 * block drafter at every draft position, score every adjacent candidate pair
 * with the selector equation
 *
 *     S_t(a, b) = U_t(b) + < A(a) (.) H(h_t), B(b) >
 *
 * (U_t is the drafter's own logit, A and B are 256-dimensional token
 * embeddings, H(h_t) a gate computed from the drafter hidden state), and make
 * one walk over the precomputed scores, starting from the last verified
 * token.  This library reads H as a bias-free linear map d -> r,
 * H_t = W_H h_t, and the walk as a max-sum (Viterbi) pass with backtrack;
 * the section's literal greedy walk is available as a second walk mode, and
 * its sampling walk through dflash2_select_sample / dflash2_sample_walk,
 * whose uniforms dflash2_philox_uniforms can draw on the device.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer argument is a DEVICE pointer on the current HIP device,
 *    owned by the caller.  The library reads inputs, writes outputs, keeps no
 *    pointer after the call returns and never frees caller memory.
 *  - Every tensor is dense row-major (C order), last dimension contiguous.
 *  - Work is enqueued on `stream` and the call returns without waiting.
 *  - Scratch memory (top-K partials, gate partials, pair scores, arrival
 *    counters) comes from a cache owned by the library, one buffer per
 *    (device, stream); it grows with hipMalloc outside the launch and is
 *    zero-initialised when allocated.  Calls on the same stream are ordered; calls on different
 *    streams use different scratch.  Warm the cache with one call before
 *    capturing a stream into a HIP graph.
 *  - Argument errors are found on the host, before any launch: the call
 *    returns DF2_EINVAL or DF2_EUNSUPPORTED, enqueues nothing, and
 *    dflash2_last_error() describes the problem.  A failed launch returns
 *    DF2_EHIP.  Out-of-range token ids read on the device (prev_tok, or a
 *    caller's cand_idx, outside [0, V)) are replaced by token 0 and raise a
 *    device flag that dflash2_device_error() reports.
 *  - Non-finite logits (NaN) are outside the contract; +-inf are ordered.
 *  - Top-K order: value descending; equal values (IEEE, -0 == +0) go to the
 *    lower vocabulary index.  Walk ties go to the smaller predecessor rank,
 *    the final pick to the smaller rank.
 *  - The launch plan is chosen from the shapes and the device.  It can be
 *    overridden for measurement only through dflash2_plan_override(); the
 *    library never reads the environment.  The top-K plan never changes a
 *    result; the gate and convolution slice counts change the fp32 summation
 *    order of H and of the corrections (within the documented tolerances;
 *    dflash2_project keeps matching dflash2_select bit for bit).
 */
#ifndef DFLASH2_H
#define DFLASH2_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of logits, hidden, A_tab, B_tab and W_H (all the same). */
typedef enum { DF2_F32 = 0, DF2_BF16 = 1 } df2_dtype;

/*
 * The walk over the pair scores.
 *   DF2_WALK_VITERBI  max-sum pass plus backtrack: the path with the largest
 *                     total score (ties: smaller predecessor rank, then
 *                     smaller final rank).
 *   DF2_WALK_GREEDY   the greedy walk of the same section: from the last
 *                     verified token, each position takes the best successor
 *                     of the token chosen one step earlier,
 *                     j_0 = argmax_j S_0(prev, j), j_t = argmax_j S_t(j_{t-1}, j)
 *                     (ties: smaller rank); the score is the sum of the chosen
 *                     S_t, added in order of t.
 */
typedef enum { DF2_WALK_VITERBI = 0, DF2_WALK_GREEDY = 1 } df2_walk;

/* Plan knobs that dflash2_plan_override() can pin (0 = automatic). */
typedef enum {
    DF2_PLAN_SEGMENT_WGS = 0,   /* target count of top-K segment workgroups */
    DF2_PLAN_CHUNK_VECTORS = 1, /* 16-byte vectors per lane per chunk: 1, 2 or 4 */
    DF2_PLAN_MERGE_WORDS = 2,   /* most candidate words one row merge takes (<= 1024;
                                   automatic: 768 in dflash2_select, 1024 in dflash2_topk) */
    DF2_PLAN_GATE_SLICES = 3,   /* slices of d of the gate projection (<= 16) */
    DF2_PLAN_CONV_SLICES = 4,   /* k slices of the convolution's correction GEMM */
    DF2_PLAN_LAUNCHES = 5,      /* dflash2_select: 1 = one fused launch, 2 = scan, then
                                   merges, pairs and walk, 3 = scan with the row merges,
                                   then pairs and walk, 4 = as 3 with the walks in a third
                                   launch; automatic: 3, or 4 when the rows exceed one
                                   resident wave of workgroups */
    DF2_PLAN_LM_RANGES = 6,     /* dflash2_lmhead_topk: vocabulary ranges (<= 256) */
    DF2_PLAN_GATE_GIVEUP = 7    /* failure-handling tests only: 1 = in dflash2_select
                                   under launches 1 or 2 (the plans whose row merges
                                   wait for the gate) the row merges wait for one gate
                                   arrival more than will come, give up after 64
                                   sleeps and raise flag bit 2; that call's outputs
                                   are not valid */
} df2_plan_knob;

typedef enum {
    DF2_OK = 0,
    DF2_EINVAL = 1,        /* bad pointer, size or combination of sizes */
    DF2_EUNSUPPORTED = 2,  /* valid request outside what the library handles */
    DF2_EHIP = 3,          /* HIP runtime or launch failure */
    DF2_ENOMEM = 4         /* scratch allocation failed */
} df2_status;

/*
 * Problem sizes.
 *   B  sequences (B >= 0; B == 0 enqueues nothing)
 *   P  draft positions per sequence, the block size minus the verified
 *      token (1 <= P <= 64)
 *   V  vocabulary size (K <= V < 2^31)
 *   d  drafter hidden size (multiple of 32)
 *   r  embedding rank of A, B and H (multiple of 64, <= 512); the pages use 256
 */
typedef struct df2_dims {
    int32_t B, P, V, d, r;
    df2_dtype dtype;
} df2_dims;

/*
 * The whole selector ("A Lightweight Path Selector": top-K, pair scores, one
 * walk from the last verified token), enqueued as two kernel launches: the
 * vocabulary scan with the gate and the row merges, then the pair scores and
 * walks.  The plan knob DF2_PLAN_LAUNCHES can move the row merges into the
 * second launch or fuse everything into one; the results are the same bits
 * in every plan.
 *   logits   [B, P, V]   drafter logits U_t
 *   hidden   [B, P, d]   drafter hidden states h_t
 *   A_tab    [V, r]      predecessor embeddings A(.)
 *   B_tab    [V, r]      candidate embeddings B(.)
 *   W_H      [r, d]      gate map, H_t = W_H h_t
 *   prev_tok [B] int32   last verified token of each sequence
 *   K        candidates per position, 1 <= K <= min(V, 64) (the pages use 16)
 *   out_path  [B, P] int32   selected token at each draft position
 *   out_score [B] float      score of the selected path, sum_t S_t (fp32)
 * Arithmetic: inputs are read exactly; H and S accumulate in fp32.  With
 * bf16 tables the products G = A(a) (.) H_t enter the matrix cores as a bf16
 * high part plus a bf16 low part (about 16 significant bits, a relative
 * error near 2^-16 per product); B(b) is exact.  fp32 tables use the fp32
 * matrix instruction throughout.
 */
df2_status dflash2_select(const df2_dims* dims, const void* logits,
                          const void* hidden, const void* A_tab,
                          const void* B_tab, const void* W_H,
                          const int32_t* prev_tok, int32_t K,
                          int32_t* out_path, float* out_score,
                          hipStream_t stream);

/*
 * dflash2_select with a choice of walk (same section; see df2_walk).
 * Arguments as for dflash2_select; `walk` outside df2_walk is DF2_EINVAL.
 * dflash2_select is this call with DF2_WALK_VITERBI.
 */
df2_status dflash2_select_walk(const df2_dims* dims, const void* logits,
                               const void* hidden, const void* A_tab,
                               const void* B_tab, const void* W_H,
                               const int32_t* prev_tok, int32_t K,
                               df2_walk walk, int32_t* out_path,
                               float* out_score, hipStream_t stream);

/*
 * dflash2_select with the sampling walk (same section: sampling draws from
 * the same scores).  From the last verified token, position t draws its
 * candidate from the softmax of the pair scores of the token chosen at
 * t - 1 (row 0 at t = 0), at the given temperature:
 *     q_t(j) = exp((S_t(i, j) - max_k S_t(i, k)) / temperature) / (sum over k)
 *     j_t    = the first j whose running sum q_t(0) + ... + q_t(j) exceeds
 *              u[b][t] (running sums in rank order; the last j with
 *              q_t(j) > 0 if rounding leaves none).
 *   temperature  > 0 and finite, 1 / temperature finite in fp32 (else DF2_EINVAL)
 *   u         [B, P] float  caller's uniforms in [0, 1) (values outside are
 *                           clamped into it, NaN to 0); the library draws
 *                           no random numbers itself
 *   out_path  [B, P] int32  drawn token at each position
 *   out_q     [B, P] float  q_t(j_t): the draft probability of each drawn
 *                           token, for rejection sampling against the target
 *   out_score [B] float     sum_t S_t(j_{t-1}, j_t), added in order of t
 * Other arguments as for dflash2_select; u and out_q 4-byte aligned.
 * Arithmetic: fp32 (expf); scores must be finite.
 */
df2_status dflash2_select_sample(const df2_dims* dims, const void* logits,
                                 const void* hidden, const void* A_tab,
                                 const void* B_tab, const void* W_H,
                                 const int32_t* prev_tok, int32_t K,
                                 float temperature, const float* u,
                                 int32_t* out_path, float* out_q,
                                 float* out_score, hipStream_t stream);

/*
 * dflash2_select_sample that also returns what each token was drawn from, as
 * dflash2_verify takes it (one small launch more):
 *   out_cand [B, P, K] int32  candidates of each position, best first
 *   out_rows [B, P, K] float  q_t over them; the entry of the drawn token is
 *                             out_q bit for bit
 * Other arguments as for dflash2_select_sample.
 */
df2_status dflash2_select_sample_rows(const df2_dims* dims, const void* logits,
                                      const void* hidden, const void* A_tab,
                                      const void* B_tab, const void* W_H,
                                      const int32_t* prev_tok, int32_t K,
                                      float temperature, const float* u,
                                      int32_t* out_path, float* out_q,
                                      float* out_score, int32_t* out_cand,
                                      float* out_rows, hipStream_t stream);

/*
 * dflash2_select that allocates nothing, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid it).  Same arguments, arithmetic and results as
 * dflash2_select (the same kernels), but its scratch is a static device
 * array of 48 MiB (50331648 bytes) that each GPU holds from module load
 * until the process ends; the first call on a device looks up its address.
 * Every call on one GPU shares that array: calls that overlap in time on a
 * GPU (different streams, or threads) race and must be serialised by the
 * caller.  Each call clears the array's arrival counters with a small
 * kernel before its own launches (no memset, no allocation).  A problem
 * whose scratch exceeds 48 MiB returns DF2_EUNSUPPORTED before anything is
 * enqueued (the stress shape B = 256, P = 15, V = 262144, K = 32 needs about
 * 40 MB).  Its device flags are reported by dflash2_device_error().
 */
df2_status dflash2_select_noalloc(const df2_dims* dims, const void* logits,
                                  const void* hidden, const void* A_tab,
                                  const void* B_tab, const void* W_H,
                                  const int32_t* prev_tok, int32_t K,
                                  int32_t* out_path, float* out_score,
                                  hipStream_t stream);

/*
 * Top-K of each row ("keep the top 16 candidates at each position").
 *   logits  [rows, V] (dtype)
 *   out_idx [rows, K] int32  candidate token ids, best first
 *   out_val [rows, K] float  their logits widened to fp32 (a -0 logit is
 *                            returned as +0)
 * 1 <= K <= min(V, 64).  rows == 0 enqueues nothing.
 */
df2_status dflash2_topk(const void* logits, int64_t rows, int32_t V,
                        df2_dtype dtype, int32_t K, int32_t* out_idx,
                        float* out_val, hipStream_t stream);

/*
 * The drafter's LM head fused with top-K ("DFlash 2: Keep Drafting
 * Parallel", section "A Lightweight Path Selector": the selector works on
 * the drafter's own logits and needs no extra LM-head pass).  For each row m
 *     U(m, v) = sum_k W_lm[v][k] * hidden[m][k]      (v = 0 .. V-1)
 * is computed on the matrix cores (bf16 products, exact in fp32, summed in
 * fp32) and only its top K leave the chip: the [M, V] logits are never
 * written to memory.  The outputs are those of dflash2_topk applied to the
 * fp32 logits, and feed dflash2_pair_scores like its outputs do.
 *   hidden  [M, d] bf16   final hidden state of each draft position
 *   W_lm    [V, d] bf16   LM-head weight, one row per token
 *   out_idx [M, K] int32  candidate token ids, best first
 *   out_val [M, K] float  their fp32 logits (a -0 logit is returned as +0)
 * dtype must be DF2_BF16 (DF2_F32 returns DF2_EUNSUPPORTED).  1 <= K <=
 * min(V, 64); V <= 2^29; d a multiple of 64 in [64, 32768]; M <= 2^24
 * (M == 0 enqueues nothing); hidden and W_lm 16-byte aligned, outputs
 * 4-byte aligned.
 * Top-K order as everywhere (value descending, equal values to the lower
 * index); the fp32 sums differ from exact ones by at most a few units in
 * the last place of sum_k |W_lm[v][k] hidden[m][k]|, so near-equal logits at
 * the K-th place may order differently than in exact arithmetic.
 * Non-finite hidden states or weights are outside the contract.  The
 * per-range candidate lists go through the library's scratch.
 */
df2_status dflash2_lmhead_topk(const void* hidden, const void* W_lm, int64_t M, int32_t V,
                               int32_t d, df2_dtype dtype, int32_t K, int32_t* out_idx,
                               float* out_val, hipStream_t stream);

/*
 * Gate projection H = W_H h for M rows ("DFlash 2: Keep Drafting Parallel",
 * section "A Lightweight Path Selector": the context gate H(h_t) of the
 * drafter state, whose formula the page cuts off; read as a bias-free
 * linear map d -> r).
 *   hidden [M, d] (dtype), W_H [r, d] (dtype), out_H [M, r] float
 * d multiple of 32, r multiple of 64 and <= 1024; hidden, W_H and out_H
 * 16-byte aligned.  H is rounded exactly as inside dflash2_select (the same
 * slices of d, summed in the same order).
 */
df2_status dflash2_project(const void* hidden, const void* W_H, int64_t M,
                           int32_t d, int32_t r, df2_dtype dtype, float* out_H,
                           hipStream_t stream);

/*
 * Pair scores of the selector equation for every adjacent candidate pair
 * (same section: S_t(a, b) = U_t(b) + < A(a) (.) H(h_t), B(b) >, every
 * adjacent pair scored at once).
 *   cand_idx [B, P, K] int32, cand_val [B, P, K] float (from dflash2_topk)
 *   H        [B, P, r] float (from dflash2_project)
 *   A_tab, B_tab [V, r] (dims->dtype), prev_tok [B] int32
 *   out_S    [B, P, K, K] float, out_S[b][t][i][j] = S_t(pred_i, cand_j)
 * The predecessor of rank i at t >= 1 is cand_idx[b][t-1][i]; at t == 0
 * every row uses prev_tok[b], so all K rows of t == 0 are equal.
 * dims->d is ignored.
 */
df2_status dflash2_pair_scores(const df2_dims* dims, const int32_t* cand_idx,
                               const float* cand_val, const float* H,
                               const void* A_tab, const void* B_tab,
                               const int32_t* prev_tok, int32_t K,
                               float* out_S, hipStream_t stream);

/*
 * The walk alone (same section: the one sequential step is a walk over the
 * precomputed scores from the last verified token), read as a max-sum pass
 * over S plus backtrack.
 *   S        [B, P, K, K] float (row 0 of t == 0 is used)
 *   cand_idx [B, P, K] int32
 *   out_path [B, P] int32, out_score [B] float
 */
df2_status dflash2_viterbi(const float* S, const int32_t* cand_idx, int32_t B,
                           int32_t P, int32_t K, int32_t* out_path,
                           float* out_score, hipStream_t stream);

/*
 * The walk alone, either mode (see df2_walk; same section: the walk over
 * the precomputed scores, max-sum or greedy).  Arguments as for
 * dflash2_viterbi, which is this call with DF2_WALK_VITERBI; 1 <= P <= 64,
 * 1 <= K <= 64; S, cand_idx, out_path and out_score 4-byte aligned.
 */
df2_status dflash2_walk(const float* S, const int32_t* cand_idx, int32_t B,
                        int32_t P, int32_t K, df2_walk walk, int32_t* out_path,
                        float* out_score, hipStream_t stream);

/*
 * The sampling walk alone (see dflash2_select_sample; same section:
 * sampling draws from the same scores) over given scores.
 *   S [B, P, K, K] float, cand_idx [B, P, K] int32, as for dflash2_walk;
 *   u [B, P] float uniforms, temperature, out_path [B, P] int32,
 *   out_q [B, P] float, out_score [B] float.
 */
df2_status dflash2_sample_walk(const float* S, const int32_t* cand_idx,
                               const float* u, int32_t B, int32_t P, int32_t K,
                               float temperature, int32_t* out_path,
                               float* out_q, float* out_score,
                               hipStream_t stream);

/*
 * The distributions that a path's tokens were drawn from, over given scores
 * (see dflash2_select_sample_rows): out_rows[b][t] is the softmax over
 * temperature of S[b][t][i], i the rank of path[b][t - 1] in cand_idx[b][t - 1]
 * (row 0 at t == 0, and for a token that is no candidate).
 *   S [B, P, K, K] float, cand_idx [B, P, K] int32, path [B, P] int32,
 *   out_rows [B, P, K] float;  B P < 2^26
 */
df2_status dflash2_draft_rows(const float* S, const int32_t* cand_idx, const int32_t* path,
                              int32_t B, int32_t P, int32_t K, float temperature,
                              float* out_rows, hipStream_t stream);

/*
 * Uniforms for the sampling walk, drawn on the device from a counter-based
 * generator (same section: sampling draws from the same scores, one uniform
 * per draft position), so a serving loop need not bring them from the host.
 * The generator is Philox4x64-10 (Salmon, Moraes, Dror and Shaw, "Parallel
 * Random Numbers: As Easy as 1, 2, 3", SC 2011):
 *     out[i] = (x >> 40) * 2^-24,  x = word (i mod 4) of
 *              Philox4x64-10(counter = (i / 4, offset, 0, 0), key = (seed, 0))
 * exact in fp32 and in [0, 1); the values depend on (seed, offset, i) only.
 * Advance `offset` once per draft-verify cycle and pass the [B, P] result
 * as dflash2_select_sample's u (same stream).  seed and offset are kernel
 * arguments: a call captured into a HIP graph replays the same uniforms
 * every time (dflash2_philox_uniforms_next keeps the offset on the device
 * for that case).
 *   n    number of uniforms, 0 <= n <= 2^31 (n == 0 enqueues nothing;
 *        n < 0 is DF2_EINVAL, n > 2^31 DF2_EUNSUPPORTED)
 *   out  [n] float, device memory owned by the caller, 4-byte aligned
 *        (16-byte alignment lets whole blocks go out in one store)
 */
df2_status dflash2_philox_uniforms(uint64_t seed, uint64_t offset, int64_t n,
                                   float* out, hipStream_t stream);

/*
 * dflash2_philox_uniforms with the offset kept in device memory, for a
 * serving loop that replays a captured HIP graph: the uniforms use the
 * value *offset holds when the launch runs, then a second launch on the same
 * stream adds one to it, so every replay draws the next cycle's uniforms.
 * Nothing is allocated and no memset is enqueued.
 *   offset  [1] uint64, device memory owned by the caller, 8-byte aligned;
 *           calls that share it must be ordered (same stream)
 * Other arguments as for dflash2_philox_uniforms; n == 0 enqueues nothing
 * and leaves *offset as it is.
 */
df2_status dflash2_philox_uniforms_next(uint64_t seed, uint64_t* offset,
                                        int64_t n, float* out,
                                        hipStream_t stream);

/*
 * Two-tap dynamic depthwise convolution of the block drafter ("DFlash 2:
 * Keep Drafting Parallel", section "A Lightweight Local Convolution"),
 * applied around each attention and feed-forward sublayer:
 *     y_t[c] = k_{t,0}[c] x_t[c] + k_{t,1}[c] x_{t-1}[c],   x_{-1} = x_prev,
 *     k_{t,tap}[c] = base[tap][c] + corr_t[tap][c / 16],
 *     corr_t[tap][g] = sum_m W_c[tap][g][m] x_t[m].
 * The pages give a learned base plus a correction from the current hidden
 * state shared by 16 channels; the correction's form is this library's
 * reading (a bias-free linear map of x_t).
 *   x      [B, P, d]     (dtype) sublayer input at the draft positions
 *   x_prev [B, d]        (dtype) the same for the last verified token
 *   base   [2, d]        (dtype) base kernel, tap 0 (current) then tap 1 (previous)
 *   W_c    [2, d/16, d]  (dtype) correction map
 *   out    [B, P, d]     (dtype) y; fp32 arithmetic, bf16 output rounded to
 *                        nearest even; must not overlap x or x_prev
 * B >= 0 (B == 0 enqueues nothing), P >= 1, d a multiple of 512 in
 * [512, 8192]; every pointer 16-byte aligned.  The corrections go through
 * the library's scratch (as dflash2_project's partials do).
 */
df2_status dflash2_conv2(const void* x, const void* x_prev, const void* base,
                         const void* W_c, int32_t B, int32_t P, int32_t d,
                         df2_dtype dtype, void* out, hipStream_t stream);

/*
 * The target's side of a draft-verify cycle.  The target runs the last
 * verified token and the drafted ones as one block: their keys and values are
 * appended to a paged cache, they attend over it, and its output rows decide
 * which drafts stand.
 *
 * A paged cache of one layer and the new tokens of a batch:
 *   k_cache, v_cache  pages of [Hkv, page_size, D] elements each, page p at
 *                     element p * page_stride; 16-byte aligned
 *   block_table  [B, table_width] int32, rows table_stride apart: the pages of
 *                each sequence in order of position
 *   ctx_len      [B] int32    tokens the cache holds before the new ones
 *   tok_start    [B + 1] int32, ascending: sequence b's new tokens are rows
 *                tok_start[b] .. tok_start[b + 1] - 1 of the N token rows (any
 *                count, zero too); new token j has position ctx_len[b] + j.
 *                Attention does nothing and raises flag bit 4 if it descends
 *                before a sequence with tokens
 *   B, N         sequences, token rows (0: nothing is enqueued).  Rows that no
 *                sequence owns have no effect; outputs leave theirs as they are
 *   Hq, Hkv, D   query heads, key/value heads (Hq a multiple of Hkv; query
 *                head i reads key/value head i / (Hq / Hkv)), head size 64, 128 or 256
 *   page_size    a power of two up to 65536
 *   num_pages    pages in the cache; a page id outside [0, num_pages) raises
 *                device flag bit 3: nothing is written there, and reads take
 *                page 0 instead
 *   table_width  pages a sequence may have (table_width * page_size <= 2^30);
 *                with ctx_len + new tokens beyond them, flag bit 4 is raised: the
 *                append writes no token whose place they do not have, attention
 *                takes ctx_len as if the last new token had the last place
 * Token rows of queries, keys, values and outputs hold their heads one after
 * the other ([heads, D]); their stride from token to token is given in
 * elements, a multiple of 16 bytes, so that they may be parts of one row.
 * These entry points keep no scratch: workspace belongs to the caller, its
 * contents need not survive between calls, and calls that share one must be
 * ordered.  They allocate nothing, enqueue kernels only and can be captured.
 */
typedef struct df2_paged_kv {
    void* k_cache;
    void* v_cache;
    const int32_t* block_table;
    const int32_t* ctx_len;
    const int32_t* tok_start;
    int64_t page_stride, table_stride;
    int32_t B, N, Hq, Hkv, D, page_size, num_pages, table_width;
    df2_dtype dtype;
} df2_paged_kv;

/*
 * Appends the new tokens' keys and values to the cache, normed and rotated,
 * and norms and rotates their queries:
 *     y = x * rsqrt(mean(x^2) + eps) * w            (norm of each head)
 *     (a, b) -> (a cos - b sin, b cos + a sin)      angle = position * rope_freq[i]
 *   q       token rows of Hq heads, or NULL with out_q (keys and values only)
 *   k, v    token rows of Hkv heads; v is copied as it is
 *   q_norm, k_norm [D] (dtype) weights, or NULL: no norm; 16-byte aligned
 *   rope_freq [rot / 2] double  radians a position; rot: leading elements of a
 *           head that are rotated, a multiple of 16 (0: none, rope_freq unused)
 *   interleaved  pair i is elements (i, i + rot / 2) if 0, else (2i, 2i + 1)
 *   out_q   token rows of Hq heads; may be q itself with q's stride, else it must
 *           not overlap q, k or v (DF2_EINVAL)
 * fp32 arithmetic (angles reduced in fp64), one rounding at the store.  A
 * token with a negative position, or one behind the page table, is not written to
 * the cache; its query is turned by that position all the same.  N <= 2^26 - 4.
 */
df2_status dflash2_kv_append(const df2_paged_kv* kv, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const void* q_norm, const void* k_norm, float eps,
                             const double* rope_freq, int32_t rot, int32_t interleaved,
                             void* out_q, int64_t out_q_stride, hipStream_t stream);

/*
 * Attention of the new tokens over their sequences' cached positions
 * 0 .. ctx_len + n - 1 (n new tokens, whose keys and values are in the cache):
 *     out = softmax(scale * q k^T) v
 *   causal  new token t sees positions up to its own; 0: all of them (the
 *           drafter's block)
 *   window  0, or how many positions back from its own a token sees (its own
 *           counts); a token whose position is negative sees none and gets 0
 *   scale   positive and finite
 *   max_len an upper estimate of ctx_len + n over the batch for the launch
 *           plan, 0: table_width * page_size.  Speed and roundings (the order in
 *           which partial sums are added, the size of the blocks) depend on it,
 *           nothing else, so it need not be true; a near one is faster where there
 *           are few tokens.
 *   q, out  token rows of Hq heads (dtype); out must not overlap q (DF2_EINVAL)
 *   workspace  dflash2_paged_attention_workspace(kv, max_len) bytes (0: may be
 *           NULL), 16-byte aligned
 * Scores, softmax statistics and sums are fp32.  The probabilities of bf16 calls
 * enter the second product with 16 bits (a bf16 high part and a low one) in blocks
 * of up to 64 rows (tokens of a sequence times Hq / Hkv, on average: N * Hq / Hkv
 * over the smaller of B and N, rows and sequences that are idle among them), and rounded
 * to bf16 in larger ones, as of prompt chunks.  Keys and values that a token of
 * the batch sees must be finite; whatever else stands in the pages is not
 * used.  Queries must be finite or NaN: a head of a token whose query holds a NaN gives
 * NaN, and no other output does.  The work is counted in tiles of 32 to 128 keys: (N * Hq / Hkv / 32 + B)
 * * Hkv times the tiles of a whole page table must stay below 2^31
 * (DF2_EUNSUPPORTED).
 */
size_t dflash2_paged_attention_workspace(const df2_paged_kv* kv, int32_t max_len);
df2_status dflash2_paged_attention(const df2_paged_kv* kv, const void* q, int64_t q_stride,
                                   float scale, int32_t causal, int32_t window,
                                   int32_t max_len, void* out, int64_t out_stride,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * A paged cache of 4-bit values (a quarter of the bytes that attention reads of a
 * bf16 one, and a thirteenth more for the scales).  Its descriptor is df2_paged_kv with
 *   k_cache, v_cache  pages of Hkv heads; a head of a page holds its tokens' codes,
 *                page_size rows of D / 2 bytes (the first of two elements in the low
 *                half), then their scales, page_size rows of D / 32 bytes
 *   page_stride  in bytes, a multiple of 16
 *   page_size    16 at least
 *   dtype        of the token rows (queries, keys, values, outputs)
 * Each block of 32 neighbouring elements of a head has one scale, a power of two held
 * as its exponent plus 127, and codes of a sign and one of the magnitudes 0, 1/2, 1,
 * 3/2, 2, 3, 4, 6 (4-bit floats of the microscaling formats).  The append chooses the
 * smallest power, from 2^-120 to 2^120, of which the block's largest magnitude is at
 * most 7, and the nearest codes, ties to the even one; a block with an infinity or NaN
 * gets scale 255, which makes all of it NaN.  Scales 0 to 254 are read as 2^(byte - 127).
 */

/*
 * dflash2_kv_append into a 4-bit cache: same arguments, and queries by the same formula in
 * fp32 (their turns are made in fp64, so last bits may differ).  Keys are normed and
 * rotated in fp64 and rounded once, to their codes, so that a cache depends on nothing
 * but its tokens.
 */
df2_status dflash2_kv_append_fp4(const df2_paged_kv* kv, const void* q, int64_t q_stride,
                                 const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                 const void* q_norm, const void* k_norm, float eps,
                                 const double* rope_freq, int32_t rot, int32_t interleaved,
                                 void* out_q, int64_t out_q_stride, hipStream_t stream);

/*
 * dflash2_paged_attention over a 4-bit cache: same arguments, and the softmax over the
 * values that the codes stand for.  bf16 calls multiply them as bf16, which they are
 * exactly, and give probabilities 16 bits in blocks of up to 32 rows (counted as there;
 * above, rounded to bf16); scores, statistics and sums as there.  Scales of positions that a token of the
 * batch sees must be 7 to 247, as the append makes them for finite numbers; a sequence's
 * values, added up with weights of up to 2^8 before they are divided by the sum, must stay
 * finite in fp32 (any scale up to 2^87 will do: 6 * 2^(87 + 8 + 30) is below 2^128).  A block of keys with scale 255 makes the
 * outputs of the tokens that see it NaN (of the heads that read that key head), a block of values
 * leaves those of its sequence's tokens undefined; other sequences' are not touched.
 */
size_t dflash2_paged_attention_fp4_workspace(const df2_paged_kv* kv, int32_t max_len);
df2_status dflash2_paged_attention_fp4(const df2_paged_kv* kv, const void* q, int64_t q_stride,
                                       float scale, int32_t causal, int32_t window,
                                       int32_t max_len, void* out, int64_t out_stride,
                                       void* workspace, size_t workspace_bytes,
                                       hipStream_t stream);

/*
 * What all pages of a 4-bit cache hold, as numbers (dtype; exact, but infinities
 * beyond its range: under the scales 253 and 254): out_k, out_v [num_pages, Hkv, page_size, D], 16-byte aligned, a
 * cache as the operators over one of that type take it.  They must not overlap the cache
 * or each other.  block_table, ctx_len and tok_start may be NULL, B and N 0.  Up to 2^34
 * values in each.
 */
df2_status dflash2_kv_unpack_fp4(const df2_paged_kv* kv, void* out_k, void* out_v,
                                 hipStream_t stream);

/* What the rows given to dflash2_verify hold. */
typedef enum { DF2_TARGET_LOGITS = 0, DF2_TARGET_PROBS = 1 } df2_target_kind;

/*
 * Sizes of a verification: B sequences (0 enqueues nothing), P drafted
 * positions (1 .. 64), vocabulary V (<= 2^29), K candidates a position
 * (1 .. min(V, 64)); dtype and kind of the target rows.  B (P + 1) < 2^24.
 */
typedef struct df2_verify_dims {
    int32_t B, P, V, K;
    df2_dtype dtype;
    df2_target_kind kind;
} df2_verify_dims;

/*
 * Verification of drafted tokens against the target (same section: rejection
 * sampling restores the exact target distribution), from given uniforms.
 * With p_t the target's distribution after t drafted tokens (softmax of row t
 * over temperature, or row t over its sum) and q_t the draft's, which is
 * cand_prob on the candidates and 0 elsewhere:
 *     draft t is accepted while u[b][t] * q_t(path_t) < p_t(path_t);
 *     at the first t where it is not, the next token is drawn from
 *     max(p_t - q_t, 0); with all accepted, from the row behind the last;
 *     a draw takes the first v whose running sum exceeds u[b][P] * (whole sum).
 *   target    [B, P + 1, V] (dtype)
 *   path      [B, P] int32    drafted tokens (an id outside [0, V) is refused
 *                             and raises flag bit 5)
 *   cand_idx  [B, P, K] int32, distinct in a row, cand_prob [B, P, K] float:
 *             as dflash2_select_sample_rows returns them, or for a path chosen
 *             without sampling K = 1, the path itself with probability 1.  Where
 *             a draft is refused, an id outside [0, V) is left out and raises bit 1
 *   n_draft   [B] int32  drafts in use of each sequence (clamped to [0, P]),
 *             or NULL: P
 *   temperature  >= 0, at most 1e30, 1 / temperature finite in fp32; 0: a draft
 *             is accepted while it is the largest of its row (ties: lower id),
 *             and the next token is the largest; then cand_idx, cand_prob and u
 *             may be NULL.  With DF2_TARGET_PROBS only its being 0 matters.
 *   u         [B, P + 1] float, clamped into [0, 1)
 *   out_tok   [B, P + 1] int32  accepted drafts, the next token, then -1
 *   out_len   [B] int32         tokens that count: accepted drafts + 1
 *   out_prob  [B, P + 1] float  p of each such token (1 at temperature 0), then 0
 *   workspace dflash2_verify_workspace(dims) bytes, 16-byte aligned
 * Row sums are fp32 of fp32 weights (with up to 2^24 elements in all rows, fp64);
 * the row that a token is drawn from is summed in fp64, so that the token does
 * not depend on how sums are rounded, and the temperature is a double for the
 * same reason.
 * -inf logits have weight 0; other non-finite values are outside the
 * contract.  Where no token is left to draw (a row without weight, or
 * candidates' probabilities that add to more than 1), flag bit 6 is raised and
 * the token is 0 with probability 0.  At temperature 0 nothing is drawn: a row
 * without weight has its lowest id as the largest.
 */
size_t dflash2_verify_workspace(const df2_verify_dims* dims);
df2_status dflash2_verify(const df2_verify_dims* dims, const void* target, const int32_t* path,
                          const int32_t* cand_idx, const float* cand_prob,
                          const int32_t* n_draft, double temperature, const float* u,
                          int32_t* out_tok, int32_t* out_len, float* out_prob,
                          void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Pages of a paged cache for the next step, made on the device from the lengths of
 * the requests, so that a draft-verify cycle never waits for the host: what
 * dflash2_verify counts goes in as `advance`, and the block table and token starts
 * come out as the paged operators take them.
 *   block_table [B, table_width] int32, rows table_stride apart: pages of each
 *               request in order of position, its first held[b] entries
 *   held        [B] int32   pages that each request holds
 *   free_list   [num_pages] int32, free_count [1] int32: the ids of the free pages.
 *               A page is in the list's first free_count entries or held once
 *   B           requests (0: nothing is enqueued), at most 2^20
 *   N           token rows of the step, at most 2^30
 *   page_size, num_pages, table_width as in df2_paged_kv; num_pages at most 2^30
 * These four arrays are updated in place; calls that share them must be ordered.
 */
typedef struct df2_page_pool {
    int32_t* block_table;
    int32_t* held;
    int32_t* free_list;
    int32_t* free_count;
    int64_t table_stride;
    int32_t B, N, page_size, num_pages, table_width;
} df2_page_pool;

/*
 *   ctx_len     [B] int32   tokens that each request had in the cache before the last
 *               step, or what is left of them
 *   advance     [B] int32   tokens that have joined them since (none of a request that was not
 *               served), or NULL: none; a sum below 0 counts as 0
 *   n_new       [B] int32   new tokens it brings; negative: the request has ended
 * A request wants ceil((ctx_len + advance + n_new) / page_size) pages, one that has
 * ended none.  First pages beyond that (after refused drafts, say) go to the end of the free
 * list, in the order of the requests and positions, and their table entries become
 * -1.  Then missing pages are taken, in the same order, each from the list's end. (Pages
 * beyond what the list holds, where one was held twice, are dropped and raise bit 3.)
 * A request is served while all pages and rows that it and those before it ask for
 * are there; one that is not, or whose table is too narrow, keeps what it has and
 * gets no new tokens, and device flag bit 7 (bit 4: the table) is raised.
 *   ctx_out     [B] int32   ctx_len + advance (0: ended); may be ctx_len itself
 *   tok_start   [B + 1] int32  first row of each request's new tokens
 *   slots       [N] int64   page id * page_size + place in the page of each row, or NULL
 *   positions   [N] int32   its position, or NULL; both are -1 in rows of no request
 * Outputs must not overlap one another or the inputs, but for ctx_out in ctx_len's place
 * (DF2_EINVAL).  The result is the same whenever the inputs are.
 */
df2_status dflash2_plan_pages(const df2_page_pool* pool, const int32_t* ctx_len, const int32_t* advance,
                              const int32_t* n_new, int32_t* ctx_out, int32_t* tok_start,
                              int64_t* slots, int32_t* positions, hipStream_t stream);

/*
 * Penalties for repeated tokens, biases and grammar masks on rows of logits: the
 * target's rows before dflash2_verify, or the drafter's before the selection.  Of
 * token v's value x in row t of sequence b:
 *     y = x;  if v was seen before the row:  y = x > 0 ? x / repetition : x * repetition
 *     y -= frequency * c + presence * [c > 0]    (one after the other)
 *     y += bias of v;  v not allowed: y = -inf
 * Seen: v stands in the first history_len tokens of the history, or among the drafts
 * path[b][0 .. t - 1]; c: how often it stands in the history from prompt_len on, and
 * among those drafts.  fp32 arithmetic, one rounding at the store; values that nothing
 * happens to keep their bits.
 *   logits, out  rows of V values (dtype), row t of sequence b at b * seq_stride +
 *                t * row_stride elements; out may be logits itself with the same
 *                strides (then only what changes is touched), else must not overlap it
 *                (DF2_EINVAL); nor may a row of out overlap the lists, penalties or masks
 *   history      [B, L] int32, rows history_stride apart, or NULL; history_len [B]
 *                int32, clamped to [0, L]; prompt_len [B] int32, or NULL: 0
 *   path         [B, R - 1] int32, or NULL: no drafts
 *   repetition, frequency, presence  [B] float each, or NULL: 1, 0, 0
 *   bias_token   [B, M] int32, bias [B, M] float; of a token given twice the last counts
 *   mask         ceil(V / 32) words a row, bit v % 32 of word v / 32 set where token v
 *                is allowed; mask_seq_stride and mask_row_stride in words, 0: one row
 *                for all; or NULL
 * Ids outside [0, V) in the lists are left out (-1 fills them up).  B or R 0: nothing
 * is enqueued.  V <= 2^29, L (with path, L + R - 1) < 2^29.
 */
typedef struct df2_adjust {
    int32_t B, R, V, L, M;
    df2_dtype dtype;
    int64_t seq_stride, row_stride, out_seq_stride, out_row_stride;
    const int32_t* history;
    int64_t history_stride;
    const int32_t* history_len;
    const int32_t* prompt_len;
    const int32_t* path;
    const float* repetition;
    const float* frequency;
    const float* presence;
    const int32_t* bias_token;
    const float* bias;
    const int32_t* mask;
    int64_t mask_seq_stride, mask_row_stride;
} df2_adjust;
df2_status dflash2_adjust_logits(const df2_adjust* adjust, const void* logits, void* out, hipStream_t stream);

/*
 * Waits for `stream`, then reports and clears the device-side flags of its
 * scratch buffer and of the current device's no-allocation scratch: *flags
 * receives a bit mask (bit 0: a prev_tok outside
 * [0, V) was replaced by 0; bit 1: a cand_idx entry outside [0, V) was
 * replaced by 0; bit 2: a row merge of dflash2_select gave up waiting for
 * its gate rows (launches 1 or 2 only), which only a fault elsewhere can
 * cause, and its scores are then unreliable; bits 3 to 7: the paged operators,
 * dflash2_plan_pages and dflash2_verify, see there; theirs, and those of dflash2_select_noalloc,
 * are kept once a device and reported on any of its streams: work that still
 * runs on another stream may raise some that a later call reports).  A raised
 * flag can leave a late gate arrival counted in the stream's scratch, so after
 * reporting one the next call on that stream clears all its arrival counters
 * before it launches.  Returns DF2_OK, or DF2_EHIP.
 */
df2_status dflash2_device_error(hipStream_t stream, uint32_t* flags);

/*
 * Pins one plan knob for every later call of this process (value 0 restores
 * the automatic choice), for measurement and plan-invariance tests.  Values
 * out of a knob's range are clamped to what the shapes allow.  Returns
 * DF2_EINVAL for an unknown knob or a negative value.  Not for use while
 * another thread is enqueueing selector work.
 */
df2_status dflash2_plan_override(df2_plan_knob knob, int32_t value);

/* Frees every scratch buffer the library holds (call with no work in flight). */
df2_status dflash2_release(void);

/* Static description of a status code. */
const char* dflash2_status_string(df2_status s);

/* Detail of the last failure on the calling thread ("" if none). */
const char* dflash2_last_error(void);

/* Library version, "major.minor.patch". */
const char* dflash2_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH2_H */
