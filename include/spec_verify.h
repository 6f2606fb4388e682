/*
 * spec_verify.h -- C ABI of the GB300 (sm_103a) batched speculative-sampling
 * verify step.
 *
 * The operation (one call, B independent requests):
 *   For request b with gamma_b draft tokens x_0..x_{gamma_b-1}:
 *   1. p_i = softmax(t[b][i] / T_b) for the gamma_b + 1 target rows and
 *      q_i = softmax(d[b][i] / T_b) for the gamma_b draft rows.
 *      ("Fast Inference from Transformers via Speculative Decoding" explainer,
 *      PyTorch sketch Steps 1-2; toolsku "LLM speculative decoding
 *      optimisation", verify sketch.)
 *   2. Draft i is accepted iff u[b][i] < p_i(x_i) / q_i(x_i), the
 *      min(1, p/q) acceptance test; k is the first rejected position, or
 *      gamma_b when none is rejected.
 *      (disassemble-channel "Speculative Decoding theory", Step 3.)
 *   3. If k < gamma_b, one token is drawn at k from the residual
 *      max(0, p_k - q_k) / sum max(0, p_k - q_k) (from p_k if that sum is 0);
 *      otherwise a bonus token is drawn from p_{gamma_b}.  The draw is the
 *      inverse CDF over ascending token id driven by u[b][G]: the smallest j
 *      whose prefix sum exceeds u[b][G] times the total.
 *      (disassemble-channel, "modified distribution" and Step 3 bonus token.)
 *   Greedy mode replaces 1-3 by argmax matching: g_i = argmax t[b][i]
 *   (lowest id on ties), k = first i with x_i != g_i, and g_k is emitted.
 *   In spec_verify_sample a request with temperature exactly 0 takes these
 *   greedy steps (temperature -> 0 makes the acceptance an argmax match).
 *   (explainer, "Implementation points", greedy paragraph; zvxbase "draft
 *   length by load", K = 3 worked example.)
 *
 * Layouts (all row-major, rows contiguous with pitch V elements):
 *   target_logits  [B][G+1][V]  float32 or bf16
 *   draft_logits   [B][G][V]    same dtype as target_logits
 *   draft_tokens   [B][G]       int32, entries past gamma_b are ignored
 *   gamma          [B]          int32, 0 <= gamma_b <= G
 *   uniforms       [B][G+1]     float32 in [0,1): column i < gamma_b is the
 *                               acceptance draw of position i, column G the
 *                               resample/bonus draw
 *   temperature    [B]          float32, >= 0; 0 verifies that request by the
 *                               greedy steps below (no draft logits read)
 *   out_tokens     [B][G+1]     int32: x_0..x_{k-1}, the drawn token, then -1
 *   num_accepted   [B]          int32: accepted drafts k (emitted = k + 1)
 *
 * Ownership and concurrency: every pointer is caller-owned DEVICE memory, except
 * where a comment says host.  The library allocates and frees nothing and never
 * synchronises the stream (spec_verify_status excepted).  The workspace must be
 * zero-filled once when allocated; every call leaves it zeroed again, so one
 * workspace serves any number of calls issued in order on one stream.  Two
 * calls that may run concurrently need two workspaces.
 *
 * Errors: each entry point returns SV_OK (0) or a negative SV_ERR_* code, and
 * on error launches nothing.  Values inside device arrays cannot be checked on
 * the host: a gamma_b outside [0, G], a draft token outside [0, V), a uniform
 * outside [0, 1), a negative or non-finite temperature, or a row with no
 * finite logit (among the rows a call reads: spec_verify_set_lazy) sets a
 * bit in the workspace's status word (read it with
 * spec_verify_status) and is clamped to a legal value, so no call reads or
 * writes outside the arrays described above.  NaN logits are not supported.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream (cudaStream_t); NULL means the legacy default stream. */
typedef struct CUstream_st *sv_stream_t;

typedef enum { SV_F32 = 0, SV_BF16 = 1, SV_F16 = 2 } sv_dtype; /* SV_F16: paged caches only */

enum {
  SV_OK = 0,
  SV_ERR_SCALAR = -1,    /* B < 0, G outside [0, SV_MAX_GAMMA], V outside [1, SV_MAX_VOCAB], bad dtype */
  SV_ERR_NULL = -2,      /* a required pointer is NULL */
  SV_ERR_ALIGN = -3,     /* a pointer is not aligned to its element (workspace: 256 bytes) */
  SV_ERR_WORKSPACE = -4, /* ws_bytes < spec_verify_workspace_size(B, G, V) */
  SV_ERR_CUDA = -5,      /* the kernel launch failed (cudaGetLastError) */
  SV_ERR_STATIC_LIMIT = -6 /* spec_verify_sample_noalloc: the sizes need more scratch than
                              SV_NOALLOC_SCRATCH_BYTES */
};

/* Status-word bits set on the device for invalid values inside arrays. */
enum {
  SV_STATUS_BAD_GAMMA = 1u,       /* gamma_b outside [0, G]: clamped */
  SV_STATUS_BAD_TOKEN = 2u,       /* draft token outside [0, V): clamped */
  SV_STATUS_BAD_UNIFORM = 4u,     /* uniform outside [0, 1) or NaN: replaced by 0 */
  SV_STATUS_BAD_TEMPERATURE = 8u, /* temperature < 0, inf or NaN: replaced by 1 */
  SV_STATUS_NONFINITE_ROW = 16u,  /* a row whose maximum is not finite (among the rows the
                                     call reads: see spec_verify_set_lazy) */
  SV_STATUS_INTERNAL = 32u,       /* an inverse-CDF draw found no token (never expected) */
  SV_STATUS_TIMEOUT = 64u,        /* a bounded wait for a request's decision ran out; the
                                     request's outputs are incomplete and the workspace must
                                     be zero-filled again before reuse */
  SV_STATUS_BAD_PROB = 128u,      /* a probability outside [0, 1] or NaN: counted as 0 (above 1:
                                     as 1); or a row that sums to 0, or to 65536 or more */
  SV_STATUS_BAD_PAGE = 256u,      /* a page number outside the pool: not written, read as zeros */
  SV_STATUS_BAD_LENGTH = 512u     /* kv_len negative, or a step past the request's page table:
                                     that row or request is left out */
};

#define SV_MAX_GAMMA 31
#define SV_MAX_VOCAB (1 << 24)
#define SV_MAX_HEAD_DIM 128
/* Size of the scratch array built into the library for spec_verify_sample_noalloc. */
#define SV_NOALLOC_SCRATCH_BYTES (4u << 20)

/*
 * Bytes of device workspace that spec_verify_sample / spec_verify_greedy need
 * for these sizes (a multiple of 256); 0 if the sizes are invalid.
 */
size_t spec_verify_workspace_size(int B, int G, int V);

/*
 * Sampling verify step (steps 1-3 above) for B requests on `stream`.
 *   target_logits, draft_logits: device, dtype `dtype`, layouts above;
 *     draft_logits may be NULL when G == 0.
 *   draft_tokens: device int32 [B][G] (may be NULL when G == 0).
 *   gamma, uniforms, temperature: device, layouts above.
 *   out_tokens, num_accepted: device outputs, layouts above.
 *   p_tok, q_tok: optional device float64 [B][G] outputs (NULL to skip):
 *     p_i(x_i) and q_i(x_i) for evaluated positions i <= k (i < gamma_b), NaN
 *     elsewhere.
 *   workspace: device, 256-byte aligned, ws_bytes >= spec_verify_workspace_size,
 *     zero-filled before its first use.
 * B == 0 is a no-op.  Returns SV_OK or an SV_ERR_* code.
 */
int spec_verify_sample(const void *target_logits, const void *draft_logits, sv_dtype dtype,
                       int B, int G, int V, const int32_t *draft_tokens,
                       const int32_t *gamma, const float *uniforms,
                       const float *temperature, int32_t *out_tokens,
                       int32_t *num_accepted, double *p_tok, double *q_tok,
                       void *workspace, size_t ws_bytes, sv_stream_t stream);

/*
 * Greedy (argmax-match) verify step on the target rows only; no draft logits,
 * uniforms or temperature.  Arguments as for spec_verify_sample.
 */
int spec_verify_greedy(const void *target_logits, sv_dtype dtype, int B, int G, int V,
                       const int32_t *draft_tokens, const int32_t *gamma,
                       int32_t *out_tokens, int32_t *num_accepted, void *workspace,
                       size_t ws_bytes, sv_stream_t stream);

/*
 * Packed (varlen) layout: the same steps for requests whose rows are stored
 * back to back without padding, as serving engines lay out ragged verify
 * batches ("speculative decoding: draft length by load", per-request draft
 * lengths K; the padded layout above wastes (G - gamma_b) rows per request).
 *   cu_draft      device int32 [B+1]: cu_draft[0] = 0, cu_draft[b+1] - cu_draft[b]
 *                 = gamma_b in [0, G]; total_drafts (host) = cu_draft[B].
 *   target_logits [total_drafts + B][V]: request b's gamma_b + 1 target rows start
 *                 at row cu_draft[b] + b.
 *   draft_logits  [total_drafts][V]: request b's rows start at cu_draft[b]
 *                 (may be NULL when total_drafts == 0).
 *   draft_tokens  [total_drafts] int32, aligned with the draft rows.
 *   uniforms      [total_drafts + B] float32, one per target row: request b's
 *                 entry cu_draft[b] + b + i is the acceptance draw of draft i
 *                 (i < gamma_b), entry cu_draft[b] + b + gamma_b its final draw.
 *   p_tok, q_tok  optional float64 [total_drafts], aligned with the draft tokens.
 *   temperature [B], out_tokens [B][G+1], num_accepted [B]: as in the padded calls
 *   (G is the largest draft length; it sizes out_tokens and the workspace,
 *   spec_verify_workspace_size(B, G, V)).
 * A request whose cu_draft entries are inconsistent (negative, decreasing, past
 * total_drafts, or a length above G) sets SV_STATUS_BAD_GAMMA and is verified with
 * no drafts at an offset clamped into the arrays: no access leaves them.
 * Returns SV_OK, or SV_ERR_* as the padded calls (SV_ERR_SCALAR also for
 * total_drafts < 0).
 */
int spec_verify_sample_packed(const void *target_logits, const void *draft_logits,
                              sv_dtype dtype, int B, int G, int V, const int32_t *cu_draft,
                              int total_drafts, const int32_t *draft_tokens,
                              const float *uniforms, const float *temperature,
                              int32_t *out_tokens, int32_t *num_accepted, double *p_tok,
                              double *q_tok, void *workspace, size_t ws_bytes,
                              sv_stream_t stream);

/* Greedy verify step on the packed layout (target rows and draft tokens as in
 * spec_verify_sample_packed; no draft logits, uniforms or temperature). */
int spec_verify_greedy_packed(const void *target_logits, sv_dtype dtype, int B, int G, int V,
                              const int32_t *cu_draft, int total_drafts,
                              const int32_t *draft_tokens, int32_t *out_tokens,
                              int32_t *num_accepted, void *workspace, size_t ws_bytes,
                              sv_stream_t stream);

/*
 * Draft-token sampler: for each of B rows, one token from softmax(logits[b] /
 * temperature[b]) by the inverse CDF over ascending token id driven by
 * uniforms[b] (the smallest j whose prefix sum exceeds uniforms[b] times the
 * total); temperature[b] == 0 returns the row's argmax (lowest id on ties).
 * This is the draw a draft model makes at each of its steps ("Speculative
 * Decoding theory", step 1, draft generation x ~ q), and the same computation
 * as spec_verify_sample's bonus draw with G == 0.
 *   logits: device [B][V] float32 or bf16; uniforms, temperature: device [B]
 *   float32; tokens: device int32 [B] output.
 *   workspace: as for spec_verify_sample, sized spec_verify_workspace_size(B, 0, V).
 * Returns SV_OK or an SV_ERR_* code; invalid device values set status bits as
 * described above.
 */
int spec_verify_draw(const void *logits, sv_dtype dtype, int B, int V, const float *uniforms,
                     const float *temperature, int32_t *tokens, void *workspace,
                     size_t ws_bytes, sv_stream_t stream);

/*
 * Verification against probabilities: the steps at the top of this file from step
 * 2 on, where the caller holds p and q instead of logits.  A sampler that filters
 * (top-k, top-p, penalties, a grammar) ends in probabilities, and drafts that
 * were looked up rather than sampled have no q row at all.
 *   target_probs  [B][G+1][V] (packed: [total_drafts + B][V]), float32 or bf16
 *   draft_probs   [B][G][V] (packed: [total_drafts][V]), the same type; NULL:
 *                 each draft was certain, q_i is 1 at x_i and 0 elsewhere (the
 *                 test is u < p_i(x_i), the residual is p_k without x_k)
 * Draft i is accepted iff q_i(x_i) = 0 or u q_i(x_i) < p_i(x_i); k and the final
 * draw as in steps 2 and 3.  Rows need not sum to 1: a draw uses its weights'
 * own total.  Of a request, the calls read p and q at the drafts, row k of
 * target_probs and, after a rejection, row k of draft_probs.  The tests are
 * exact; the draw's weights are rounded by less than 2^-46 (p or p - q to a multiple
 * of 2^-46, so that one below 2^-47 counts as 0; the rounding error of p - q to one
 * of 2^-47), summed exactly, and compared with u times the total exactly:
 * a row should not sum to much less than 1 (where n entries sum to 2^-20, the
 * roundings move a boundary by about 2^-28 sqrt(n) of the total).  A residual
 * whose weights are all 0 draws from p_k; a row of zeros draws V - 1 and sets
 * SV_STATUS_BAD_PROB.  An entry that is no probability (negative, NaN, above 1)
 * sets that bit where it is read and counts as 0 (above 1: as 1).
 * The other arguments, the layouts, the workspace (status word only), errors and
 * ownership: as spec_verify_sample and spec_verify_sample_packed.
 */
int spec_verify_sample_probs(const void *target_probs, const void *draft_probs, sv_dtype dtype,
                             int B, int G, int V, const int32_t *draft_tokens,
                             const int32_t *gamma, const float *uniforms, int32_t *out_tokens,
                             int32_t *num_accepted, void *workspace, size_t ws_bytes,
                             sv_stream_t stream);
int spec_verify_sample_probs_packed(const void *target_probs, const void *draft_probs,
                                    sv_dtype dtype, int B, int G, int V, const int32_t *cu_draft,
                                    int total_drafts, const int32_t *draft_tokens,
                                    const float *uniforms, int32_t *out_tokens,
                                    int32_t *num_accepted, void *workspace, size_t ws_bytes,
                                    sv_stream_t stream);

/*
 * The target's KV cache across verify steps.  The target scores a request's last
 * token and its gamma_b drafts in one pass ("Speculative Decoding theory", Step
 * 2): gamma_b + 1 rows, at the packed row offsets cu_draft[b] + b.  Their keys and
 * values are appended behind the request's kv_len[b] tokens, the rows attend to
 * the cache, and after the verification the cache is rolled back by its length
 * alone (explainer, "Implementation points", KV rollback): the next step's
 * kv_len[b] is kv_len[b] + num_accepted[b] + 1, and what lies behind is
 * overwritten by the next append.
 *
 * A cache is a pool of pages of page_size tokens.  Element (page, token, head,
 * value) of the keys lies at k_pages + page * k_strides[0] + token * k_strides[1]
 * + head * k_strides[2] + value (elements), likewise for values, so pools stored
 * [page][token][head][value] and [page][head][token][value] both fit.  Token t of
 * request b lies in page page_table[b * max_pages + t / page_size], at t %
 * page_size.  Pages that two requests share are only read; a page that is
 * appended to belongs to one request.
 *   dtype      SV_BF16 or SV_F16
 *   page_size  a power of two from 16 to 4096
 *   head_dim   a multiple of 8, at most SV_MAX_HEAD_DIM
 *   strides    positive multiples of 8; pools 16-byte aligned
 * The struct itself is HOST memory, read during the call; its pointers are device
 * memory.
 */
typedef struct {
  void *k_pages, *v_pages;
  sv_dtype dtype;
  int num_pages, page_size, kv_heads, head_dim;
  int64_t k_strides[3], v_strides[3]; /* page, token, head */
  const int32_t *page_table;          /* [batch][max_pages]; entries past a request's
                                         tokens are not read */
  int max_pages, batch;
  const int32_t *kv_len;              /* [batch]: the request's own tokens before this step
                                         (a shared prefix is not counted) */
} sv_kv_cache;

/*
 * Appends a step's keys and values, and rotates its queries: row cu_draft[b] + b +
 * i (i <= gamma_b) of request b goes to token kv_len[b] + i.
 *   q            [total_drafts + batch][q_heads][head_dim], q_strides (HOST, row and
 *                head, elements); q_out likewise.  q_heads 0: no queries, q and q_out
 *                may be NULL.  q_out may not overlap itself (SV_ERR_SCALAR), nor k, v
 *                or, unless it is q with its strides, q (SV_ERR_ALIGN): their reaches
 *                are apart, or they are slices of one tensor with one row stride (or
 *                head stride), apart within it
 *   k, v         [total_drafts + batch][kv_heads][head_dim] with k_strides, v_strides;
 *                not within the slots that the call writes
 *   max_drafts   the largest gamma_b; any length (a prompt of n tokens is gamma_b =
 *                n - 1)
 *   freq         device int64 [rot_dim / 2]: pair j turns by freq[j] 2^-64 turns a
 *                position (a far position loses nothing); NULL with rot_dim 0
 *   rot_dim      even, at most head_dim: the first rot_dim values of a head turn, the
 *                others are copied.  Pairs are (j, j + rot_dim / 2), with interleaved
 *                (2j, 2j + 1): (a, c) -> rope_scale (a cos - c sin, c cos + a sin)
 *   positions    optional device int32 [total_drafts + batch]: a row's position (the
 *                depth of a tree draft's node); NULL: position_offset + kv_len[b] + i
 *                (position_offset: the length of a shared prefix)
 *   workspace    for the status word only: any of this library's, at least 4 bytes
 * The rotation is computed in 32 bits and rounded once.  A request whose cu_draft
 * entries are inconsistent (as in the packed calls, or a length above max_drafts)
 * is skipped (SV_STATUS_BAD_GAMMA).  total_drafts may exceed cu_draft[batch], here and in
 * spec_verify_attention: the rows behind the last request's are neither stored nor
 * rotated (a captured step of fixed size).  A row past the page table
 * (SV_STATUS_BAD_LENGTH) or on a page outside the pool (SV_STATUS_BAD_PAGE) is not
 * stored, its query is still rotated.  No other element of the pools is written.
 */
int spec_verify_kv_append(const void *q, const int64_t *q_strides, int q_heads, const void *k,
                          const int64_t *k_strides, const void *v, const int64_t *v_strides,
                          void *q_out, const int64_t *q_out_strides, const sv_kv_cache *cache,
                          const int32_t *cu_draft, int total_drafts, int max_drafts,
                          const int64_t *freq, int rot_dim, int interleaved, float rope_scale,
                          const int32_t *positions, int position_offset, void *workspace,
                          size_t ws_bytes, sv_stream_t stream);

/*
 * Bytes of workspace that spec_verify_attention needs for total_rows =
 * total_drafts + batch rows (more rows need more); 0 if the sizes are invalid.
 */
size_t spec_verify_attention_workspace_size(int total_rows, int q_heads, int head_dim);

/*
 * Attention of a step's rows over the cache, after their append.  Row i of request
 * b sees the shared prefix and the request's own tokens 0 .. kv_len[b] + i:
 *   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j)
 *   q, q_strides     as above (16-byte aligned, strides multiples of 8), the type of
 *                    the cache; q_heads a multiple of kv_heads, at most 128 a key
 *                    head; query head h reads key head h / (q_heads / kv_heads)
 *   prefix_table     device int32, ceil(prefix_len / page_size) pages that every
 *                    request reads before its own, with prefix_len (HOST) tokens;
 *                    read once for the whole batch.  A prefix, and a request's own
 *                    tokens with the step's, hold at most 2^31 - 4097 tokens
 *   draft_mask       optional device uint32 [total_drafts + batch], max_drafts <=
 *                    SV_MAX_GAMMA: bit j of a row's word says whether it sees row j of
 *                    its request's step (tree drafts), in place of j <= i; bits from
 *                    gamma_b + 1 on are ignored.  Tokens before the step are always
 *                    seen.
 *   scale            positive; a score scale q . k stays below 2^27 in magnitude (or is
 *                    infinite)
 *   out              [total_drafts + batch][q_heads][head_dim], dense, 16-byte aligned;
 *                    not within q's reach (SV_ERR_ALIGN)
 *   lse              optional float32 [total_drafts + batch][q_heads]: the natural log
 *                    of the sum of weights
 *   workspace        zero its first 4 bytes before the first use; the rest is
 *                    scratch.  One call at a time, in order on one stream: two calls
 *                    that may overlap, two captured graphs' among them, need two.
 * A row that sees nothing (an empty mask word, no tokens before, no prefix), or
 * whose scores are all -inf, gets zeros and lse -inf.  What the pool holds behind a
 * request's last token is never used, whatever it is; a NaN or an infinity among
 * the values of tokens that some row of a request sees reaches that request's
 * other rows of the step too.  Requests with inconsistent cu_draft entries
 * (SV_STATUS_BAD_GAMMA) or lengths (SV_STATUS_BAD_LENGTH: kv_len[b] + gamma_b + 1
 * tokens past the page table) are skipped, their rows of out and lse left as they
 * were; entries that name the same rows so often that the step's list of keys passes
 * 2^30 tiles leave out every request (SV_STATUS_BAD_GAMMA).  Scores, sums and parts are 32 bits; weights are rounded to the cache's
 * type for the product with the values (half a step of each weight; in fp16, of a
 * weight below 2^-21 of the largest, 2^-32 of the largest).  Results repeat bit for bit.
 */
int spec_verify_attention(const void *q, const int64_t *q_strides, int q_heads,
                          const sv_kv_cache *cache, const int32_t *prefix_table, int prefix_len,
                          const int32_t *cu_draft, int total_drafts, int max_drafts, float scale,
                          const uint32_t *draft_mask, void *out, float *lse, void *workspace,
                          size_t ws_bytes, sv_stream_t stream);

/*
 * spec_verify_sample_noalloc: spec_verify_sample with no caller workspace.
 * The pages on speculative decoding describe no such call: this is a
 * convenience of this library's interface, not a step of the method.
 *
 * Who needs it: callers that may not obtain device memory when they verify.
 * A serving loop that handed all free device memory to weights and the KV
 * cache when it started, and must not grow its footprint later, is one; C
 * code that drives this library without any device allocator of its own is
 * another.  This call allocates and frees nothing.
 *
 * Scratch: an array of SV_NOALLOC_SCRATCH_BYTES (4 MiB) that lives in the
 * library's device image.  If spec_verify_workspace_size(B, G, V) is larger,
 * the call returns SV_ERR_STATIC_LIMIT and runs nothing (4 MiB holds, for
 * example, B = 512 requests with G = 3 and V = 128256).
 *
 * First call on a device: it looks up the array's device address with
 * cudaGetSymbolAddress while that device is current and keeps it for later
 * calls on the same device (SV_ERR_CUDA if the look-up fails).  Make that
 * first call before any stream capture begins.  The kept address belongs to
 * the device's primary context: after cudaDeviceReset on that device it is
 * stale, and a later call would launch on a freed address.  A process that
 * resets a device must not call spec_verify_sample_noalloc on it again.
 *
 * Sharing: every call in the process uses the same array.  Each call first
 * zeroes the array's counters and flags (an asynchronous memset on `stream`),
 * then launches the same kernel as spec_verify_sample; the per-chunk partial
 * results stay in the array as the last call left them.  Calls that can
 * overlap on the GPU (other streams without ordering between them, other host
 * threads) race on the array and produce wrong results: issue them in order
 * on one stream.  Because of the memset, the status bits of spec_verify_status
 * are not available from this call; invalid device values are still clamped
 * as described at the top of this file.
 *
 * Arguments, layouts and the other return codes: as spec_verify_sample,
 * without workspace and ws_bytes.
 */
int spec_verify_sample_noalloc(const void *target_logits, const void *draft_logits,
                               sv_dtype dtype, int B, int G, int V,
                               const int32_t *draft_tokens, const int32_t *gamma,
                               const float *uniforms, const float *temperature,
                               int32_t *out_tokens, int32_t *num_accepted, double *p_tok,
                               double *q_tok, sv_stream_t stream);

/*
 * Copies the workspace's status word (SV_STATUS_* bits accumulated since the
 * last read) to *status_host (a HOST pointer), then clears it.  Synchronises
 * `stream`.  Returns SV_OK, SV_ERR_NULL or SV_ERR_CUDA.
 */
int spec_verify_status(void *workspace, sv_stream_t stream, uint32_t *status_host);

/* Static English text for an SV_OK / SV_ERR_* code. */
const char *spec_verify_strerror(int code);

/*
 * Schedules.  Three kernels compute every value with the same arithmetic, so
 * outputs do not depend on the schedule:
 *   - the resident cluster path: a batch small enough that one thread-block
 *     cluster per request fits on the GPU at once, with each warp holding one
 *     chunk of a draft position's target and draft rows in shared memory.  The
 *     partials, the decision and the residual block sums move through the
 *     cluster's shared memory, and the final draw walks resident data;
 *   - the streaming cluster path: one cluster per request as well, for batches
 *     of up to one cluster per SM (clusters of up to 16 CTAs, at least one),
 *     the warps streaming the request's chunks two at a time and re-reading
 *     the rejected row's chunks for the residual.  For larger batches the same
 *     kernel runs as one CTA per SM (sampling) or two (greedy), each taking
 *     whole requests in turn from a claim counter, longest request first
 *     (SV_ROUTE_CLAIMS).  The claim order takes 5 bytes of shared memory per
 *     request.  A sampling call of at least two requests per SM whose
 *     positions are read lazily (spec_verify_set_lazy) runs instead on a
 *     pipeline kernel (SV_ROUTE_PIPELINE): one CTA per SM keeps two requests
 *     in flight, its warps moving from one request's items to the other's
 *     without a barrier, and the warp that completes a stage, a residual pass
 *     or a draw runs what follows it;
 *   - the persistent grid, for batches whose claim order does not fit (tens
 *     of thousands of requests): chunks claimed from global counters,
 *     decisions published through global records.
 * The cluster paths replace the persistent grid's chain of global-memory
 * synchronisations (arrival counters, decision records, queue) with cluster
 * barriers.  These calls are not steps of the method: they exist for testing
 * and measurement.
 *
 * spec_verify_set_schedule: the policy for the calls that follow in this
 * process: SV_SCHEDULE_AUTO (the default: the first of the resident cluster
 * path, the streaming cluster path and the persistent grid that applies, as
 * above), SV_SCHEDULE_PERSISTENT (every call on the persistent grid) or
 * SV_SCHEDULE_STREAM (as AUTO without the resident path).  Returns the
 * previous policy, or SV_ERR_SCALAR for an unknown value.  SV_SCHEDULE_STREAM
 * also leaves out the pipeline kernel (its claims run on the streaming
 * kernel).
 *
 * spec_verify_route: the kernel (SV_ROUTE_*) that the next sampling
 * (greedy == 0) or greedy call of this shape, in the padded layout, on the
 * current device would use under the current policy, or SV_ERR_SCALAR for
 * invalid sizes.  If cluster_size is not NULL (a HOST pointer), it receives
 * the cluster size (CTAs per request) of a cluster path (1 for claims and the
 * pipeline), or 0.
 *
 * spec_verify_cluster_size: that cluster size alone (0 for the persistent
 * grid), or SV_ERR_SCALAR.
 */
#define SV_SCHEDULE_AUTO 0
#define SV_SCHEDULE_PERSISTENT 1
#define SV_SCHEDULE_STREAM 2
#define SV_ROUTE_PERSISTENT 0
#define SV_ROUTE_CLUSTER 1
#define SV_ROUTE_STREAM 2
#define SV_ROUTE_CLAIMS 3
#define SV_ROUTE_PIPELINE 4
int spec_verify_set_schedule(int schedule);
int spec_verify_route(sv_dtype dtype, int B, int G, int V, int greedy, int *cluster_size);

/*
 * spec_verify_set_wait_limit: the limit, in nanoseconds of the GPU's global
 * timer, of every bounded wait in the calls that follow in this process (a
 * bulk copy's completion, a decision record, a queue slot); 0 restores the
 * default of 2 s.  A wait that runs out sets SV_STATUS_TIMEOUT and its warp
 * stops taking work, so the call returns with incomplete outputs and the
 * workspace must be zero-filled again (as documented for that bit).  Not a
 * step of the method: it exists so that tests can make a wait run out
 * quickly.  Returns the previous limit.
 */
unsigned long long spec_verify_set_wait_limit(unsigned long long ns);

/*
 * spec_verify_set_lazy: how the request-claims schedules (SV_ROUTE_CLAIMS,
 * SV_ROUTE_PIPELINE) read a request's rows in the calls that follow in this
 * process.
 * 1 (the default): position by position.  In a greedy call (or a request
 * with temperature 0) target row i is reduced to its argmax and compared
 * with draft i before row i + 1 is read; the call stops at the first draft
 * that differs.  For a sampled request the target and draft rows of
 * position i are reduced and draft i is tested before the rows of position
 * i + 1 matter, and the bonus row gamma_b only after every draft was
 * accepted, as in the verification loop of disassemble-channel
 * "Speculative Decoding theory", Step 3, which stops at the first rejected
 * draft.  On the streaming kernel's claims, for a request with at least four
 * drafts, the CTA streams the next position while one is tested (what it read
 * of a position after the first rejection is not used); the pipeline kernel
 * instead streams its other request's position meanwhile.  Lazy stages lengthen a request while they shorten
 * the batch, so sampled requests are read this way only where the batch
 * holds at least two requests per CTA, and not when a request's rows alone
 * reach 80 % of a CTA's share of the batch's rows.  0: every row of every
 * request is reduced before any
 * test.  The outputs are identical either way: a position's arithmetic does
 * not depend on the order.  The other schedules always read every row.
 * Returns the previous setting, or SV_ERR_SCALAR for a value other than 0
 * or 1.
 */
int spec_verify_set_lazy(int on);
int spec_verify_cluster_size(sv_dtype dtype, int B, int G, int V, int greedy);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
