/*
 * dflash.h: C ABI of the GB300 (sm_103a) DFlash2 low-rank candidate selector.
 *
 * The method comes from the page "vllm.models.beam.nvidia.dflash2" (DFlash2 draft model
 * for Beam targets). For request r and block position (step) p, the selector:
 *   1. takes the top-K vocabulary candidates of the drafter's logits and their logits
 *      ("unary" scores)                  DFlash2BeamForCausalLM.compute_candidates
 *   2. projects the drafter hidden state to the codebook rank,
 *      h_p = W_proj . hidden[r, p]       DFlash2BeamCandidateSelector.__init__ / forward
 *   3. scores every candidate c against every candidate q one position back,
 *      E[r,p,q,c] = unary[r,p,c] + <pred_cb[cand[r,p-1,q]] * h_p, succ_cb[cand[r,p,c]]>,
 *      where the predecessor at p = 0 is the request's anchor token.
 *                                        DFlash2BeamCandidateSelector (class docstring)
 * Before them, the norm and rotation of queries and keys (dflash_qk_norm_rope) and the paged
 * key-value cache of the draft step's attention: its block tables (dflash_block_tables), its store
 * (dflash_store_kv, or in one pass with the norm and rotation, dflash_qk_norm_rope_store) and the
 * attention over it (dflash_paged_attention). Behind them, drafts drawn from the edge scores
 * (dflash_sample_path) and their verification against the target model's logits
 * (dflash_verify_drafts).
 * Around these: step 1 straight from the LM head without logits in memory
 * (dflash_lmhead_topk, dflash_selector_lmhead), steps 2 and 3 on given candidates
 * (dflash_selector_forward), and the best path through E (dflash_best_path, a reading: the
 * page does not show what consumes E).
 *
 * Conventions for every entry point:
 *   - Pointers are caller-owned DEVICE memory on the current CUDA device, unless a
 *     comment says otherwise. Tensors are contiguous and row-major, in the shapes given.
 *     bf16 tensors are passed as uint16_t bit patterns.
 *   - Every pointer must be 16-byte aligned (vector loads and TMA), or the call returns
 *     DFLASH_INVALID_ARGUMENT. The exceptions are `logits` (the top-k finds the 16-byte
 *     boundaries itself), `anchors`, `cand_ids`, `unary`, `edges` and the best path's
 *     `path`, `tokens` and `score` (accessed one element at a time, or staged with copies
 *     as wide as their alignment allows): their natural
 *     4-byte alignment suffices, so a slice of requests out of larger arrays stays valid. The same
 *     holds for every int32, int64 or fp32 array (positions, slots, frequencies, numbers and temperatures,
 *     probabilities, counts) of the norm and rotation, the sampled path and the verification.
 *     `hidden`, `h_out`, the weights and the workspace stay 16-byte aligned.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream). They
 *     allocate no device memory and do not synchronise the device; dflash_device_status,
 *     dflash_trace_end and dflash_selftest_wait_timeout are the exceptions, and say so. A
 *     non-OK status means nothing was launched, except DFLASH_CUDA_ERROR, which reports a
 *     launch failure.
 *   - Supported sizes: R, S >= 1; 1 <= K <= 32 and K <= V; V < 2^31; H a multiple of 8;
 *     rank a multiple of 8 in [8, 256]. Out-of-range sizes give DFLASH_INVALID_ARGUMENT
 *     (bad values) or DFLASH_UNSUPPORTED (valid but not implemented, for example K > 32).
 *   - Token ids are int32. Anchor ids outside [0, V) are caller errors. The kernels
 *     check every gathered id: a bad id never reaches memory, its scores are NaN, and
 *     the device status word records DFLASH_DEVICE_BAD_ID (see dflash_device_status).
 *   - Calls that overlap on the GPU must not share an output or a workspace.
 */
#ifndef DFLASH_H
#define DFLASH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The same type as cudaStream_t. */
typedef struct CUstream_st* dflash_stream_t;

typedef enum {
    DFLASH_OK = 0,
    DFLASH_INVALID_ARGUMENT = 1,    /* null or misaligned pointer, size out of range      */
    DFLASH_UNSUPPORTED = 2,         /* valid request outside the implemented envelope     */
    DFLASH_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes below the *_workspace_bytes query  */
    DFLASH_CUDA_ERROR = 4,          /* a CUDA runtime call or a launch failed             */
    DFLASH_NO_DEVICE = 5            /* the current device is not a GB300 (sm_103a), or none */
} dflash_status;

/* Bits of the device status word (dflash_device_status). */
#define DFLASH_DEVICE_BAD_ID 0x1u       /* a gathered token id was outside [0, V)        */
#define DFLASH_DEVICE_TIMEOUT 0x2u      /* a bounded wait inside a kernel gave up        */
#define DFLASH_DEVICE_BAD_LENGTH 0x4u   /* a request's lengths contradict each other or  */
                                        /* do not fit its row of the block table         */
#define DFLASH_DEVICE_NO_PAGES 0x8u     /* the list of free pages was too short          */
#define DFLASH_DEVICE_BAD_LOGITS 0x10u  /* a row of logits has a NaN or +inf, or only -inf */

/* A static string naming a status code. Never NULL. */
const char* dflash_status_string(int status);

/* A detail message for the last non-OK status returned on this host thread ("" if none).
 * The pointer stays valid until the next library call on this thread. */
const char* dflash_last_error(void);

/* ------------------------------------------------------------------------------------
 * Step 1: top-K candidates.
 * Source: DFlash2BeamForCausalLM.compute_candidates ("the selector's top-k candidate
 * ids and their logits at each position").
 *
 * logits    [R, S, V] float32   the drafter's vocabulary logits, one row per (r, p)
 * softcap, scale                the logits processor's options (second page,
 *                               DFlash2BeamForCausalLM.__init__: LogitsProcessor(soft_cap,
 *                               scale=output_multiplier)). The reported unary value is
 *                               scale * softcap * tanh(x / softcap), the cap first; softcap = 0
 *                               means no cap. scale must be > 0, so the map is increasing,
 *                               and candidates are selected and ordered on the raw logits.
 *                               Pass 0 and 1 for raw logits.
 * cand_ids  [R, S, K] int32     out: the K best token ids of each row, in candidate order
 * unary     [R, S, K] float32   out: their (processed) logits
 * workspace                     caller-owned device scratch of at least
 *                               dflash_topk_workspace_bytes(R, S, V, K) bytes. Its
 *                               contents on entry do not matter. The call overwrites it.
 *
 * Candidate order: logit descending; equal logits go to the lower token id; -0 equals
 * +0. A NaN with the sign bit clear ranks above +inf, and one with the sign set below
 * -inf. The unary value of a -0 logit is returned as +0.
 * ---------------------------------------------------------------------------------- */
size_t dflash_topk_workspace_bytes(int R, int S, int V, int K);

dflash_status dflash_topk_candidates(const float* logits, int R, int S, int V, int K,
                                     float softcap, float scale, int32_t* cand_ids,
                                     float* unary, void* workspace, size_t workspace_bytes,
                                     dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Top-K candidates without a workspace argument. The pages have no counterpart to this
 * call; it exists for callers that must not allocate device memory. Examples are a
 * plugin running inside an inference engine that has already claimed all device memory
 * for its own pool, and code that may not call cudaMalloc because the allocation would
 * synchronise the device or is forbidden at that point.
 *
 * Same inputs, outputs and results as dflash_topk_candidates with softcap = 0 and
 * scale = 1 (raw logits). The scratch is a fixed
 * 4 MiB array in device memory that the library holds on every GPU that loads it, until
 * the process exits. A call whose scratch need (about R*S*4 bytes of counters plus
 * 512 bytes per streaming warp) exceeds 4 MiB returns DFLASH_UNSUPPORTED and launches
 * nothing; use dflash_topk_candidates with a workspace then.
 * - The call allocates nothing: no cudaMalloc, no cudaFree, no allocating library routine.
 * - The first call on a device looks up the array's device address. Make that first call
 *   before any stream capture on the device. A lookup that fails is not remembered: the
 *   call returns DFLASH_CUDA_ERROR and the next call tries again.
 * - Every call on a device shares the one array. Each call clears the counters it needs
 *   (a memset on `stream`) before its kernel runs. Calls that overlap on the GPU (on
 *   different streams, or from several threads) race on the array: serialise them.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_topk_candidates_noalloc(const float* logits, int R, int S, int V, int K,
                                             int32_t* cand_ids, float* unary,
                                             dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Step 1 from the LM head: the candidate head without materialised logits.
 * Source: DFlash2BeamForCausalLM.compute_candidates, which calls
 * LogitsProcessor.get_top_k_tokens(lm_head, hidden_states, top_k).
 *
 * hidden    [R, S, H] bf16   drafter hidden states
 * lm_head   [V, H]    bf16   the LM head weight (vocabulary rows)
 * cand_ids  [R, S, K] int32  out: the K best token ids of each row, in candidate order
 * unary     [R, S, K] float  out: their (processed) logits
 * workspace                  at least dflash_lmhead_topk_workspace_bytes(R, S, V, K) bytes;
 *                            its contents on entry do not matter.
 *
 * logits[r,p,v] = sum_i hidden[r,p,i] * lm_head[v,i] are fp32 sums taken by the tensor
 * cores (tcgen05, operands staged by TMA). They never leave the chip. The candidate order,
 * softcap and scale are those of dflash_topk_candidates. Where two logits differ by less
 * than their fp32 accumulation error, their order may differ from an exact computation.
 * Requires H a multiple of 8.
 * ---------------------------------------------------------------------------------- */
size_t dflash_lmhead_topk_workspace_bytes(int R, int S, int V, int K);

dflash_status dflash_lmhead_topk(const uint16_t* hidden, const uint16_t* lm_head, int R, int S,
                                 int H, int V, int K, float softcap, float scale,
                                 int32_t* cand_ids, float* unary, void* workspace,
                                 size_t workspace_bytes, dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Step 2: hidden projection, h = hidden . W_proj^T with no bias.
 * Source: DFlash2BeamCandidateSelector.__init__ (hidden_projection: a bias-free linear
 * map hidden_size -> rank, in params_dtype) and forward (hidden must be bf16).
 *
 * hidden  [R, S, H]    bf16   drafter hidden states
 * w_proj  [rank, H]    bf16   projection weight, in the Linear [out, in] convention
 * h_out   [R, S, rank] bf16   out: fp32 accumulation, rounded to bf16 (nearest-even)
 * Runs on the tensor cores (tcgen05, operands staged by TMA). Like every compute call of
 * this library it needs a GB300 (compute capability 10.3): the library is built for
 * sm_103a only, and other devices get DFLASH_NO_DEVICE.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_hidden_projection(const uint16_t* hidden, const uint16_t* w_proj,
                                       int R, int S, int H, int rank, uint16_t* h_out,
                                       dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Step 3: edge scores.
 * Source: DFlash2BeamCandidateSelector (class docstring and forward): "[requests,
 * steps, top_k (predecessor), top_k]".
 *
 * pred_cb, succ_cb  [V, rank]     bf16    predecessor / successor codebooks
 * cand_ids          [R, S, K]     int32   candidates (step 1's output)
 * unary             [R, S, K]     float32 their logits
 * h                 [R, S, rank]  bf16    projected hidden states (step 2's output)
 * anchors           [R]           int32   anchor (bonus) token of each request
 * edges             [R, S, K, K]  float32 out: E[r, p, q, c], with q the predecessor
 *                                         index and c the candidate index
 *
 * E[r,p,q,c] = unary[r,p,c] + sum_j pred_cb[pid, j] * h[r,p,j] * succ_cb[cand[r,p,c], j],
 * with pid = cand[r,p-1,q] for p > 0 and pid = anchors[r] (every q) for p = 0. The
 * products and sums are taken in fp32.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_candidate_edges(const uint16_t* pred_cb, const uint16_t* succ_cb,
                                     const int32_t* cand_ids, const float* unary,
                                     const uint16_t* h, const int32_t* anchors, int R, int S,
                                     int K, int V, int rank, float* edges,
                                     dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * The whole selector in one call, with no host round trip. All three steps run on `stream`,
 * each kernel launched as the programmatic dependent of the one before it: a large projection
 * (step 2, more than 8 GFLOP) is launched first and the top-k (step 1) runs beside it; a
 * smaller projection is launched after the top-k and runs on the SMs the top-k's first
 * finished CTAs leave. The edges (step 3) take the SMs the top-k leaves as it finishes,
 * scoring each (r, p) tile as soon as the top-k has written the rows it needs and the
 * projection is done. The results do not depend on the order.
 * The call returns once everything is enqueued; later work on `stream` sees all outputs. It is
 * safe to capture in a CUDA graph; make one call on the device before capturing. The
 * workspace holds the top-k's and the edge tiles' bookkeeping (its size query includes
 * both; its contents on entry do not matter). The outputs, softcap and scale are as in the
 * three calls above; the edge scores use the processed unary values.
 * Source: the draft step captures the candidate head and the selector together
 * (module docstring of the page).
 * ---------------------------------------------------------------------------------- */
size_t dflash_selector_workspace_bytes(int R, int S, int V, int K);

dflash_status dflash_selector(const float* logits, const uint16_t* hidden,
                              const uint16_t* w_proj, const uint16_t* pred_cb,
                              const uint16_t* succ_cb, const int32_t* anchors, int R, int S,
                              int K, int V, int H, int rank, float softcap, float scale,
                              int32_t* cand_ids, float* unary, uint16_t* h_out, float* edges,
                              void* workspace, size_t workspace_bytes, dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * The selector's forward pass: steps 2 and 3 on candidates the caller already has.
 * Source: DFlash2BeamCandidateSelector.forward(candidate_ids, unary_logits, hidden_states,
 * anchor_token_ids), which scores the candidates with candidate_edges on the projected
 * hidden states and returns the edge scores [requests, steps, top_k (predecessor), top_k].
 *
 * cand_ids, unary, anchors, pred_cb, succ_cb, K, V, rank, edges  as in dflash_candidate_edges
 * hidden, w_proj, H, h_out                                      as in dflash_hidden_projection
 *
 * The projection writes h_out, then the edges read it; both run on `stream` and the call
 * returns once they are enqueued. No workspace. The ranges are those of the two calls. It
 * is not traced by dflash_trace_begin, which traces the calls that include step 1. It can be
 * captured in a CUDA graph; make one call on the device before capturing.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_selector_forward(const int32_t* cand_ids, const float* unary,
                                      const uint16_t* hidden, const int32_t* anchors,
                                      const uint16_t* w_proj, const uint16_t* pred_cb,
                                      const uint16_t* succ_cb, int R, int S, int K, int V, int H,
                                      int rank, uint16_t* h_out, float* edges,
                                      dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * The draft step from the LM head: steps 1 to 3 in one call, with step 1 taken straight
 * from the LM head as in dflash_lmhead_topk, so no logits are ever written.
 * Source: DFlash2BeamForCausalLM.compute_candidates takes the candidates from
 * get_top_k_tokens(lm_head, hidden, top_k), and the selector's forward scores them with the
 * same hidden states (DFlash2BeamCandidateSelector.forward).
 *
 * hidden, lm_head, H, softcap, scale, cand_ids, unary   as in dflash_lmhead_topk
 * w_proj, pred_cb, succ_cb, anchors, rank, h_out, edges as in dflash_selector
 * workspace  at least dflash_selector_lmhead_workspace_bytes(R, S, V, K) bytes; its contents
 *            on entry do not matter.
 *
 * The kernels run one after another on `stream`: projection, LM-head top-k, edges. The
 * LM-head top-k holds one CTA on every SM, so nothing runs beside it. The call returns once
 * everything is enqueued. The candidates may differ from an exact computation only where two
 * logits differ by less than their fp32 accumulation error (see dflash_lmhead_topk); the edge
 * scores are those of the candidates returned. Requires the ranges of dflash_selector and
 * H a multiple of 8. A traced call (dflash_trace_begin) records the same four events. It can
 * be captured in a CUDA graph; make one call on the device before capturing (the first call
 * sets the kernels' shared-memory limits).
 * ---------------------------------------------------------------------------------- */
size_t dflash_selector_lmhead_workspace_bytes(int R, int S, int V, int K);

dflash_status dflash_selector_lmhead(const uint16_t* hidden, const uint16_t* lm_head,
                                     const uint16_t* w_proj, const uint16_t* pred_cb,
                                     const uint16_t* succ_cb, const int32_t* anchors, int R,
                                     int S, int K, int V, int H, int rank, float softcap,
                                     float scale, int32_t* cand_ids, float* unary,
                                     uint16_t* h_out, float* edges, void* workspace,
                                     size_t workspace_bytes, dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Best path through the edge scores: one candidate per step for every request.
 * Reading: the pages say the selector rescores each position's top-k tokens against the
 * token before it (page "vllm.models.beam.nvidia.dflash2", module docstring) but show no
 * consumer of the scores. This call takes the plainest one: the path that maximises the sum
 * over p of E[r,p,c_{p-1},c_p], the predecessor row at p = 0 being q = 0 (every q row there
 * is the anchor's).
 *
 * edges     [R, S, K, K] float  edge scores as dflash_candidate_edges writes them
 * cand_ids  [R, S, K]    int32  the candidates
 * path      [R, S]       int32  out: the chosen candidate index c_p at each step
 * tokens    [R, S]       int32  out: cand_ids[r, p, c_p], the drafted tokens
 * score     [R]          float  out: the path's score
 *
 * Max-sum dynamic programming in fp32, in a fixed order: V_0[c] = E[r,0,0,c]; V_p[c] is the
 * running maximum over q = 0..K-1 of V_{p-1}[q] + E[r,p,q,c], replaced only by a strictly
 * larger sum (ties keep the lower q; IEEE compares, so a NaN never replaces and is never
 * replaced); the last candidate is the running maximum of V_{S-1}, same rule, and the path
 * follows the kept predecessors back. The result is therefore exactly reproducible.
 * Requires 1 <= K <= 32 and S <= 256 (DFLASH_UNSUPPORTED beyond). No workspace.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_best_path(const float* edges, const int32_t* cand_ids, int R, int S, int K,
                               int32_t* path, int32_t* tokens, float* score,
                               dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * A path through the edge scores drawn at random: the drafter's own distribution of each token,
 * given the one before it, is the softmax of that token's row of edge scores.
 * Reading: as for dflash_best_path, the pages do not show what consumes the scores; sampled drafts
 * need a distribution, which the verification of drafts then takes away.
 *
 * edges, cand_ids  as in dflash_best_path
 * uniforms     [R, S]    float  numbers drawn evenly from [0, 1), one for each choice
 * temperatures [R]       float  each request's T; or NULL, and `temperature` is T for all
 * path         [R, S]    int32  out: the chosen candidate index c_p at each step
 * tokens       [R, S]    int32  out: cand_ids[r, p, c_p]
 * probs        [R, S, K] float  out: the distribution that c_p was drawn from
 *
 * With the row E[r, p, c_{p-1}, :] (at p = 0: q = 0), probs[c] = w_c / sum_j w_j, w_c =
 * exp((E_c - max E) / T), and c_p is the smallest c with sum_{j<=c} w_j > u sum_j w_j. The choice is
 * made as with exact sums (it may differ where a sum is within 2^-45 of the border, and then too is of a
 * candidate with some weight); probs are fp32.
 * T below 2^-100 counts as 2^-100.
 * T = 0 takes the largest score (so do T < 0 and NaN), the first of equals, with probability 1; a row
 * whose largest score is +inf, or which has none but -inf and NaN, is taken the same way. In other rows
 * NaN scores have no weight. A uniform outside [0, 1) counts as the nearer end, NaN as 0. Weights
 * below 2^-126 of the largest may count as 0. Requires 1 <= K <= 32 and S <= 256
 * (DFLASH_UNSUPPORTED beyond). No workspace.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_sample_path(const float* edges, const int32_t* cand_ids, const float* uniforms,
                                 const float* temperatures, float temperature, int R, int S, int K,
                                 int32_t* path, int32_t* tokens, float* probs,
                                 dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Verification of drafted tokens against the target model's logits.
 * Source: DFlashSpeculator.propose hands its draft tokens to the target model; how that one takes or
 * leaves them is not on the pages. This is the standard rule, which keeps the target's distribution
 * whatever the drafter's is.
 *
 * logits       [T, V] of type dtype (DFLASH_BF16, DFLASH_FP16 or DFLASH_FP32), rows at row_stride
 *              elements: the target's logits of a step's new tokens. Natural alignment suffices.
 * query_start  [R + 1] int32, as dflash_block_tables writes it: request r has the rows from
 *              query_start[r] to query_start[r + 1] - 1, one for its last token and one for each of its
 *              drafts, n_r rows for n_r - 1 <= S drafts. No rows: nothing is done for the request.
 * draft_tokens [R, S] int32: draft i was made for row i's place, token i + 1 of the request's step
 * cand_ids     [R, S, K] int32 and draft_probs [R, S, K] float: the distribution q that each draft was
 *              drawn from, as dflash_sample_path gives it (an id that occurs twice has the sum); both
 *              NULL: each draft was certain
 * accept_uniforms [R, S], sample_uniforms [R] float  numbers drawn evenly from [0, 1)
 * temperatures [R] float  each request's T; or NULL, and `temperature` is T for all
 * tokens       [R, S + 1] int32  out: the drafts that were taken, one token behind them, then -1
 * counts       [R] int32         out: how many tokens that is, 0 for a request without rows
 * logprobs     [R, S + 1] float  out: log p of each token under the target (0 behind them), or NULL
 * workspace    at least dflash_verify_drafts_workspace_bytes(R, T, V) bytes; its contents on entry do
 *              not matter
 *
 * With p = softmax(logits / T) of row i, draft x is taken iff u q(x) < p(x). In the row of the first that
 * is not, a token is drawn from max(p - q, 0), normalised (from p, should less than 2^-36 be left); if all
 * are taken, from p of the last row. Drawn: the smallest v with sum_{j<=v} weight_j > u sum_j weight_j.
 * Tokens are those of exact arithmetic; only where a border is within about 2^-38 of a row's sum may
 * they differ, and then too the token drawn has some weight. T = 0 (so T < 0 and NaN): p is 1 at the
 * first of the row's largest logits; T counts as at least 2^-99 and at most 2^100. Masked logits may be
 * -inf or the type's lowest value; weights below 2^-125 of the largest may count as 0.
 * A sample uniform outside [0, 1) counts as the nearer end, NaN as 0.
 * A row that is reached and has a NaN, +inf or nothing but -inf ends its request without a token
 * (DFLASH_DEVICE_BAD_LOGITS). A draft that is reached and is outside [0, V) is not taken, a candidate
 * that is outside is left out of q, and DFLASH_DEVICE_BAD_ID is set. A request whose rows are out of
 * order, past T or more than S + 1 is refused: count 0, tokens -1 (DFLASH_DEVICE_BAD_LENGTH); if it makes
 * two other requests' rows overlap, their tokens are undefined. Rows behind a request's first rejected
 * draft have no effect. Rows at and behind query_start[R] are not read.
 * 0 <= S <= 255, K <= 32, V <= 2^20 (DFLASH_UNSUPPORTED beyond). Equal calls give equal bits. It can be
 * captured in a CUDA graph; make one call on the device before capturing.
 * ---------------------------------------------------------------------------------- */
size_t dflash_verify_drafts_workspace_bytes(int R, int T, int V);

dflash_status dflash_verify_drafts(const void* logits, int dtype, int T, int V, long long row_stride,
                                   const int32_t* query_start, const int32_t* draft_tokens, int R,
                                   int S, const int32_t* cand_ids, const float* draft_probs, int K,
                                   const float* accept_uniforms, const float* sample_uniforms,
                                   const float* temperatures, float temperature, int32_t* tokens,
                                   int32_t* counts, float* logprobs, void* workspace,
                                   size_t workspace_bytes, dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * The paged key-value cache that the drafter and the target model attend to. A cache is a
 * pool of pages of page_size token rows; a request owns the pages that its row of the block
 * table lists, and token j of it lives in row j % page_size of its page j / page_size. A slot
 * numbers a token row of the whole pool: page * page_size + row.
 * Source: the drafter's context keys and values already sit in a paged cache
 * (DFlash2BeamAttention), prepare_dflash_inputs builds positions and slots on the GPU, and
 * store_context_kv scatters keys and values by slot, optionally to fp8. The pages show only
 * the calls; the arithmetic is the standard one, spelled out below.
 *
 * Element types of tensors that are not bf16 alone. */
typedef enum {
    DFLASH_BF16 = 0,
    DFLASH_FP16 = 1,
    DFLASH_E4M3 = 2,   /* 8-bit floating point, 4 exponent bits, no infinities (cache only) */
    DFLASH_FP32 = 3    /* norm weights and logits only */
} dflash_dtype;

/* One layer's cache: key and value hold [num_pages, page_size, kv_heads, head_dim] elements
 * of type dtype, at the same strides (in elements; the innermost is 1), so both orders of
 * page rows and heads, and caches with keys and values interleaved, can be passed. (Here and in
 * the calls below a dimension of one element may have any stride.) Row addresses must be 16-byte
 * aligned. With DFLASH_E4M3 an element stands for itself times
 * k_scale or v_scale; with the other types both scales must be 1. A host struct; the calls read
 * it before they return. */
typedef struct {
    void* key;
    void* value;
    long long page_stride;
    long long token_stride;
    long long head_stride;
    int num_pages;
    int page_size;
    int kv_heads;
    int head_dim;
    int dtype;       /* dflash_dtype */
    float k_scale;
    float v_scale;
} dflash_kv_cache;

/* ------------------------------------------------------------------------------------
 * Block tables and slots of one step, from the requests' lengths.
 * Source: prepare_dflash_inputs (third page, DFlashSpeculator.propose), which builds
 * positions and slot mappings per request on the GPU.
 *
 * context_lens [R] int32   tokens each request has in the cache
 * new_lens     [R] int32   tokens this step adds to it
 * held_pages   [R] int32   pages its table row lists already (at least enough for its
 *                          context; more after a step whose tokens were rejected)
 * free_pages   [n_free]    page ids to take from, in order (int32)
 * block_table  [R, max_pages] int32  in/out: new pages are written behind the held ones;
 *                          nothing else of it is written
 * query_start  [R + 1] int32  out: first token of each request, and their number
 * kv_lens      [R] int32      out: context_lens + new_lens
 * held_out     [R] int32      out: pages listed after the call
 * positions    [T] int32      out: each new token's position in its request
 * slots        [T] int64      out: its slot
 * pages_needed [1] int32      out: pages taken from free_pages
 *
 * need_r = max(0, ceil((context_lens[r] + new_lens[r]) / page_size) - held_pages[r]); request r
 * takes the need_r pages of free_pages behind those of the requests before it. T is the room
 * for tokens: rows at and behind query_start[R] get position 0 and slot -1, which the store
 * skips. A request whose lengths are negative, whose context is longer than its held pages or
 * which needs more than max_pages is refused (DFLASH_DEVICE_BAD_LENGTH): it takes no pages. So
 * is one that free_pages has too few pages for (DFLASH_DEVICE_NO_PAGES; pages_needed is then
 * more than n_free). A refused request keeps its place in query_start, its slots are -1, its
 * kv_lens entry is 0 and its table row stays as it was. If the new tokens are more than T,
 * those past T are not written (DFLASH_DEVICE_BAD_LENGTH); query_start and pages_needed stop at
 * 2^31 - 1. Outputs must not overlap inputs (nor
 * kv_lens be context_lens: a step's lengths are the next one's context). 0 <= T; R <= 16384
 * (DFLASH_UNSUPPORTED beyond). One launch; no workspace; natural alignment suffices.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_block_tables(const int32_t* context_lens, const int32_t* new_lens,
                                  const int32_t* held_pages, const int32_t* free_pages, int R,
                                  int n_free, int page_size, int max_pages, int T,
                                  int32_t* block_table, int32_t* query_start, int32_t* kv_lens,
                                  int32_t* held_out, int32_t* positions, int64_t* slots,
                                  int32_t* pages_needed, dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Store new keys and values in the cache.
 * Source: store_context_kv (DFlash2BeamModel.precompute_and_store_context_kv): scatter by
 * slot, optionally to e4m3 with a scale for the layer.
 *
 * key, value  [T, kv_heads, head_dim] of type dtype (DFLASH_BF16 or DFLASH_FP16), each at its
 *             own token and head strides (in elements, multiples of 8), so slices of a fused
 *             projection's output can be passed
 * slots       [T] int64. A negative slot stores nothing. A slot outside the cache stores
 *             nothing and sets DFLASH_DEVICE_BAD_ID. Two tokens must not share a slot.
 *
 * The cache has the type dtype, and rows are copied; or DFLASH_E4M3, and an element x is stored
 * as x / scale rounded to the nearest e4m3 value, ties to even, |x / scale| clamped to 448
 * (NaN stays NaN). head_dim is a multiple of 8 up to 256 (16 for e4m3). T = 0 does nothing.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_store_kv(const void* key, const void* value, int dtype, const int64_t* slots,
                              int T, long long key_token_stride, long long key_head_stride,
                              long long value_token_stride, long long value_head_stride,
                              const dflash_kv_cache* cache, dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Rotation frequencies, as the calls below take them: the turns that pair j of a head makes from
 * one position to the next, f_j / (2 pi) modulo 1, as a whole number of 2^-64. Angles are exact modulo one
 * turn at every position of 32 bits for the frequency that is kept, which is off by a few 2^-53 of itself and
 * half of 2^-64.
 *
 * inv_freq     host, [rotary_dim / 2] radians per position; or NULL, and then
 *              f_j = base^(-2 j / rotary_dim), for long contexts divided by factor: every pair if
 *              original_len is 0; else a pair that makes at most turns_slow turns over original_len
 *              positions is, one that makes turns_fast or more is not, and in between f_j goes over
 *              linearly in the number of turns from the one to the other. (Rules that go over in the
 *              pair's index j, as model configurations labelled yarn usually mean, are not this one: give
 *              their inv_freq.)
 * frequencies  host, [rotary_dim / 2] out: copy them to device memory
 * A frequency that is not finite is refused.
 * A host function: no device is needed, and nothing is launched.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_rope_frequencies(int rotary_dim, double base, double factor,
                                      double original_len, double turns_slow, double turns_fast,
                                      const double* inv_freq, int64_t* frequencies);

/* What is done to queries and keys. A host struct; the calls read it before they return. */
typedef struct {
    const void* q_weight;       /* [head_dim], or NULL: queries are not normed              */
    const void* k_weight;       /* [head_dim], or NULL: keys are not normed                 */
    int weight_dtype;           /* the type of queries and keys, or DFLASH_FP32             */
    float eps;                  /* >= 0                                                     */
    const int64_t* frequencies; /* device, [rotary_dim / 2]; not read if rotary_dim is 0    */
    int rotary_dim;             /* even, 0 (no rotation) to head_dim                        */
    int interleaved;            /* pairs (2j, 2j + 1); 0: pairs (j, j + rotary_dim / 2)     */
    float rope_scale;           /* factor of the rotated values (1: a plain rotation)       */
} dflash_norm_rope;

/* ------------------------------------------------------------------------------------
 * Norm of each query and key head, then its rotation by position, in one pass.
 * Source: beam_qk_norm_rope (DFlash2BeamAttention): RMS norm of queries and keys for each head, then
 * their rotation. The pages show the call; the arithmetic is the standard one:
 *   y = x w / sqrt(mean(x^2) + eps) over a head's head_dim values (no norm where the weight is NULL),
 *   (a, b) -> rope_scale (a cos t - b sin t, b cos t + a sin t), t = positions[token] f_j,
 * for the pairs j of the first rotary_dim values; the others stay as they are, normed (without a norm: bit for
 * bit, but that a NaN may become another NaN).
 *
 * query, key  [T, q_heads, head_dim], [T, kv_heads, head_dim] of type dtype (DFLASH_BF16 or
 *             DFLASH_FP16) at the given strides (elements, multiples of 8, below 2^31). Either may have no
 *             heads.
 * positions   [T] int32, of any sign; not read if rotary_dim is 0
 * query_out, key_out  out, of the same shapes and type at their own strides. Each may be its own input
 *             (the same address and strides); else outputs must not overlap inputs.
 * Sums and products are fp32, rounded once at the end. (A head of zeros with eps 0 gives NaN, as the
 * formula does.) head_dim is a multiple of 8 up to 256. A head whose sum of squares passes fp32's range is
 * taken 2^-72 as large, one whose mean square and eps come to less than 2^-100 2^72 as large, and eps with it.
 * T = 0 does nothing. One launch, no workspace.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_qk_norm_rope(const void* query, const void* key, int dtype,
                                  const int32_t* positions, int T, int q_heads, int kv_heads,
                                  int head_dim, long long q_token_stride, long long q_head_stride,
                                  long long k_token_stride, long long k_head_stride,
                                  const dflash_norm_rope* how, void* query_out, void* key_out,
                                  long long q_out_token_stride, long long q_out_head_stride,
                                  long long k_out_token_stride, long long k_out_head_stride,
                                  dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * The same, with keys and values stored in the paged cache in the same pass.
 * Source: beam_qk_norm_rope with a slot mapping; and precompute_and_store_context_kv, which norms,
 * rotates and stores the context's keys without queries (q_heads = 0).
 *
 * value, slots, cache  as in dflash_store_kv. Keys go to the cache rounded once: what a call of
 *                      dflash_qk_norm_rope and one of dflash_store_kv give, but into an e4m3 cache
 *                      without a rounding to dtype before that to e4m3.
 * query, positions, how, query_out  as in dflash_qk_norm_rope
 * Queries of tokens whose slot is negative or outside the cache are written as any others.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_qk_norm_rope_store(
    const void* query, const void* key, const void* value, int dtype, const int32_t* positions,
    const int64_t* slots, int T, int q_heads, long long q_token_stride, long long q_head_stride,
    long long k_token_stride, long long k_head_stride, long long v_token_stride,
    long long v_head_stride, const dflash_norm_rope* how, const dflash_kv_cache* cache,
    void* query_out, long long q_out_token_stride, long long q_out_head_stride,
    dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Attention of new tokens over the paged cache, which holds their own keys and values too.
 * Source: DFlash2BeamAttention: a non-causal sliding-window attention of the 1 + N query block
 * over cached context (window_left, window_right); with window_right = 0 it is the causal
 * attention of the target model's prompts, verified blocks and single tokens.
 *
 * query        [T, q_heads, head_dim] of type dtype (DFLASH_BF16 or DFLASH_FP16) at the
 *              given strides (elements, multiples of 8); q_heads a multiple of kv_heads, query
 *              head h reading key head h / (q_heads / kv_heads)
 * cache        of the same type, or DFLASH_E4M3
 * block_table  [R, max_pages] int32; query_start [R + 1], kv_lens [R] int32, as
 *              dflash_block_tables writes them
 * out          [T, q_heads, head_dim] of type dtype, contiguous
 * lse          [T, q_heads] float, contiguous, or NULL
 * workspace    at least dflash_paged_attention_workspace_bytes(...) bytes (a token amount where
 *              head_dim, q_heads / kv_heads or R rule the tensor cores out); its contents on entry
 *              do not matter
 *
 * Token i of request r, of its n = query_start[r+1] - query_start[r], has position
 * p = kv_lens[r] - n + i and sees the keys j with max(0, p - window_left) <= j <=
 * min(kv_lens[r] - 1, p + window_right); -1 is no bound. Over them
 *   s_j = scale * <q, k_j>, then softcap * tanh(s_j / softcap) if softcap > 0,
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = log sum_j exp(s_j)  (natural).
 * A token that sees no key gets zeros and lse = -inf. What the cache holds at keys that a
 * token does not see has no effect on it, infinities and NaN included. Scores, maxima and sums
 * are fp32. The cap adds at most 2^-19 of a score, or 2^-21 softcap where softcap <= 64, to a score's
 * rounding; a softcap outside [2^-64, 2^64] counts as the nearer end. The products exp(s_j) v_j
 * take exp(s_j) relative to a running maximum, rounded to the query's type (to fp16 over an e4m3
 * cache), and are summed in fp32. Over an e4m3 cache bf16 queries are taken as fp16 times a power
 * of two for each row: what that loses is less than 2^-39 of the row's largest value (of one of
 * 2^-86 or more; smaller queries may be taken as 0).
 * Page ids outside the pool are never followed: tokens that see a key of such a page get NaN, the
 * others what they would get without it, and the status word records DFLASH_DEVICE_BAD_ID. Pages of
 * which no token sees a key (a window may have left them) can have any id. A request whose kv_lens does not fit max_pages, or
 * whose query_start is out of order or past T, is refused with DFLASH_DEVICE_BAD_LENGTH: its
 * rows are NaN or not written. Rows of out at and behind query_start[R] are not written.
 * head_dim is a multiple of 8 up to 256 (16 for e4m3). A result does not depend on what else
 * is in the batch beyond the rounding of its sums and of their order, and equal calls give equal
 * bits. head_dim 64 and 128 with pages of a power of two from 8 tokens on, q_heads / kv_heads up
 * to 128 and R up to 16384 run on the tensor cores, all others on the CUDA cores.
 * ---------------------------------------------------------------------------------- */
size_t dflash_paged_attention_workspace_bytes(int R, int T, int q_heads, int kv_heads,
                                              int head_dim);

dflash_status dflash_paged_attention(const void* query, int dtype, int T, int q_heads,
                                     long long q_token_stride, long long q_head_stride,
                                     const dflash_kv_cache* cache, const int32_t* block_table,
                                     int R, int max_pages, const int32_t* query_start,
                                     const int32_t* kv_lens, float scale, int window_left,
                                     int window_right, float softcap, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes,
                                     dflash_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Device status word. Reads the DFLASH_DEVICE_* bits that kernels on the current device
 * have set since the last clear. Clears them if `clear` is non-zero. Synchronises the
 * device. `flags` is a host pointer.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_device_status(uint32_t* flags, int clear);

/* ------------------------------------------------------------------------------------
 * Self-check of the wait limit. There is no counterpart on the pages; this is a test aid for
 * the failure path. It launches one thread that waits on an mbarrier nothing ever arrives
 * on, through the same bounded wait the pipelined kernels use (projection, LM-head top-k),
 * then one edge CTA that waits in the fused selector's ready queue for a tile nothing ever
 * pushes. Each wait gives up after about one second, sets DFLASH_DEVICE_TIMEOUT in the status
 * word, and the kernel returns: nothing traps or faults, nothing is written, and the context
 * stays usable. Synchronises the device; read and clear the bit with dflash_device_status.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_selftest_wait_timeout(void);

/* ------------------------------------------------------------------------------------
 * Stage tracing for dflash_selector and dflash_selector_lmhead. There is no counterpart on
 * the pages; this is a profiling aid.
 * dflash_trace_begin(n) creates 4 timing events for each of the next n selector calls
 * made from this process on the current device. Each traced call records them: at its
 * start, when the projection is done, when the top-k is done and when the edges are done,
 * and its kernels then run one after another (untraced, dflash_selector overlaps them), so
 * that each can be timed. dflash_trace_end waits for the events. It writes up to max_calls
 * rows of 3 stage times (ms) into `stage_ms` (a host array of 3 * max_calls floats): the
 * projection, the top-k and the edges, each the time between two events. It stores the row
 * count in *n_calls, then releases the events.
 * ---------------------------------------------------------------------------------- */
dflash_status dflash_trace_begin(int n_calls);
dflash_status dflash_trace_end(float* stage_ms, int max_calls, int* n_calls);

/* Library version, "major.minor.patch". */
const char* dflash_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_H */
