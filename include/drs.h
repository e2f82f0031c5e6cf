/*
 * drs.h -- C ABI of libdrs, the GB300 (sm_103a) implementation of the
 * DiffusionGemma per-row sampler statistics.
 *
 * The operations follow the page "vllm.model_executor.models.
 * diffusion_gemma_sampler": the module docstring (argmax, Gumbel-max sample,
 * softmax entropy and the softmax in the model dtype, the noise drawn inline),
 * sample_row_stats and its PyTorch definition sample_row_stats_reference,
 * and stash_converged_logprobs / _lp_topk_kernel (top-k logprobs of the rows
 * of converged slots, keys ordered by value then by lower index).
 *
 * Conventions for every entry point:
 *   - Array arguments are DEVICE pointers owned by the caller, unless stated
 *     otherwise. The library allocates no device memory in any call.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t passed as
 *     void*; NULL is the legacy default stream). Results are ready when the
 *     stream is.
 *   - Host-side argument checks return DRS_ERR_INVALID_ARG without
 *     launching anything. Launch failures return DRS_ERR_CUDA. A device-side
 *     wait that runs out of time makes the kernel skip its remaining writes
 *     and raise a device flag, read with drs_get_device_error().
 *   - The library cannot check the length of device arrays; the caller
 *     guarantees the sizes stated below.
 *   - Not thread-safe for concurrent calls that share one workspace.
 */
#ifndef DRS_H_
#define DRS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum drs_status {
    DRS_OK = 0,
    DRS_ERR_INVALID_ARG = -1,
    DRS_ERR_UNSUPPORTED = -2,
    DRS_ERR_CUDA = -3,
    DRS_ERR_DEVICE_TIMEOUT = -4
} drs_status;

typedef enum drs_probs_dtype {
    DRS_PROBS_NONE = 0,
    DRS_PROBS_BF16 = 1,
    DRS_PROBS_FP16 = 2
} drs_probs_dtype;

/* Element types of the token operators (drs_verify_drafts and below). BF16
 * and FP16 have the values of drs_probs_dtype. */
typedef enum drs_dtype {
    DRS_DTYPE_FP32 = 0,
    DRS_DTYPE_BF16 = 1,
    DRS_DTYPE_FP16 = 2
} drs_dtype;

/* Largest vocabulary (row length) the kernels accept (2^21). */
#define DRS_MAX_VOCAB 2097152

/* Largest sizes of the token operators: requests of drs_map_slots, tokens of
 * drs_embed_tokens_grad, columns of an embedding row. */
#define DRS_MAX_REQUESTS 1048576
#define DRS_MAX_TOKENS 268435456
#define DRS_MAX_WIDTH 1048576

/* Largest sizes of drs_token_logprobs: alternatives and rows. */
#define DRS_MAX_ALTERNATIVES 64
#define DRS_MAX_SCORE_ROWS 134217727

/*
 * Bytes of device workspace drs_row_stats needs (at least 256-byte aligned,
 * contents arbitrary: each call clears the counters it uses with an
 * asynchronous memset on its stream before its kernels run). The workspace
 * carries the row lists and the per-tile and per-row records through which
 * the kernels of one call pass their partial results: about 4.6 KiB per row
 * of 262144 columns, growing with rows and vocab. One workspace must not be
 * used by two calls that can run at the same time.
 */
size_t drs_row_stats_workspace_bytes(int64_t rows, int64_t vocab);

/*
 * Per-row statistics of temperature-scaled logits (sample_row_stats and
 * sample_row_stats_reference on the page above).
 *
 *   logits      fp32 [rows, vocab], row i at logits + i * row_stride, unit
 *               column stride. row_stride >= vocab; the columns between
 *               vocab and row_stride are never read.
 *   row0        global index of the first row (>= 0). Row i of this call
 *               is global row row0 + i: it keys the noise and picks the
 *               temperature, so a batch split over several calls or GPUs
 *               gives the results of one call. 0 for a whole batch.
 *   temps       fp32 [ceil((row0 + rows) / canvas_len)], one per slot of the
 *               whole batch; global row r uses T = temps[r / canvas_len].
 *               The scaled logit is the IEEE fp32
 *               quotient x / max(T, 1e-10f). T > 0 draws Gumbel noise; T <= 0
 *               is greedy (sample = argmax). NaN temperatures, NaN or +inf
 *               logits are not supported; -inf logits are.
 *   seed        noise key. The noise of (global row, col) is Philox4x32-10
 *               with key
 *               (lo32(seed), hi32(seed)) and counter (lo32(col/4),
 *               hi32(col/4), lo32(row), hi32(row)), word col % 4, mapped to
 *               u = max((word >> 8) * 2^-24, 1e-20f); g = -log(-log u). The
 *               same function is exposed by drs_philox_gumbel.
 *   argmax      int64 [rows]: lowest column of the largest scaled logit.
 *   sample      int64 [rows]: lowest column of the largest scaled logit + g.
 *   entropy     fp32 [rows]: entropy of softmax(scaled); -inf columns drop
 *               out; a row that is -inf everywhere has entropy 0.
 *   probs       probs_dtype NONE: must be NULL. BF16/FP16: 16-bit
 *               [rows, vocab] with row stride probs_row_stride >= vocab
 *               (elements), softmax(scaled) rounded to nearest even.
 *   workspace   device scratch of drs_row_stats_workspace_bytes(rows, vocab)
 *               bytes; may be NULL only when that function returns 0.
 *
 * rows == 0 returns DRS_OK without launching. vocab must be in
 * [1, DRS_MAX_VOCAB]; canvas_len >= 1.
 */
drs_status drs_row_stats(const float *logits, int64_t rows, int64_t vocab,
                         int64_t row_stride, const float *temps,
                         int64_t canvas_len, uint64_t seed, int64_t row0,
                         int64_t *argmax,
                         int64_t *sample, float *entropy,
                         drs_probs_dtype probs_dtype, void *probs,
                         int64_t probs_row_stride, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * drs_row_stats without a caller workspace. The page has no counterpart:
 * this entry point exists for callers that cannot allocate device memory
 * for the library -- plugin interfaces that hand over only input and
 * output buffers at enqueue time, or code that must not call cudaMalloc
 * (it can synchronise the device, or the memory budget is fixed at
 * start-up). Arguments, results and errors are those of drs_row_stats.
 *
 * The kernels' records live in a fixed device array inside the library
 * (640 KiB; every GPU that loads the library holds it until the process
 * exits). A call whose rows need a larger workspace runs in batches of rows
 * that fit, one after the other on the stream (at most 137 rows of 262144
 * columns per batch). The call allocates nothing. Its
 * first call on a device looks up the array's device address (with that
 * device current) and caches it; make that first call before any stream
 * capture. All calls on a device share the array: two calls that can run
 * at the same time on the GPU (different streams, overlapping) race and
 * corrupt each other's results. Each call resets the list counters at the
 * start of the array (an asynchronous memset on its stream) before its
 * kernels run; every other record in the array is written before it is read
 * within the same call, so what an earlier call left there is never used.
 * The cached address belongs to the device's CUDA context: after
 * cudaDeviceReset (or anything else that destroys the primary context) the
 * library must be unloaded and loaded again before this entry point is
 * called on that device.
 */
drs_status drs_row_stats_noalloc(const float *logits, int64_t rows, int64_t vocab,
                                 int64_t row_stride, const float *temps,
                                 int64_t canvas_len, uint64_t seed, int64_t row0,
                                 int64_t *argmax, int64_t *sample, float *entropy,
                                 drs_probs_dtype probs_dtype, void *probs,
                                 int64_t probs_row_stride, void *stream);

/*
 * Bytes of device workspace drs_row_stats_seeds needs for n_seeds seeds
 * (1 <= n_seeds <= 8; 0 otherwise). Same alignment and sharing rules as the
 * row-stats workspace.
 */
size_t drs_row_stats_seeds_workspace_bytes(int64_t rows, int64_t vocab, int32_t n_seeds);

/*
 * drs_row_stats for several noise seeds in one call: the argmax, entropy and
 * probabilities once, and a Gumbel-max sample per seed, from the same two
 * passes over the logits (the race of each seed runs on the tile already in
 * shared memory). Every argument of drs_row_stats has its meaning there;
 * in addition:
 *
 *   seeds       HOST uint64 [n_seeds], 1 <= n_seeds <= 8: the noise keys.
 *   samples     int64 [n_seeds, rows]: samples + s * rows is the sample of
 *               every row under seeds[s] (what drs_row_stats gives with that
 *               seed).
 *   workspace   drs_row_stats_seeds_workspace_bytes(rows, vocab, n_seeds).
 *
 * Returns DRS_ERR_INVALID_ARG for a null seeds array or n_seeds outside
 * [1, 8], otherwise as drs_row_stats.
 */
drs_status drs_row_stats_seeds(const float *logits, int64_t rows, int64_t vocab,
                               int64_t row_stride, const float *temps,
                               int64_t canvas_len, const uint64_t *seeds,
                               int32_t n_seeds, int64_t row0, int64_t *argmax,
                               int64_t *samples, float *entropy,
                               drs_probs_dtype probs_dtype, void *probs,
                               int64_t probs_row_stride, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace drs_row_stats_topk needs for k > 0 (256-byte
 * aligned, contents arbitrary: each call clears what it uses with
 * asynchronous memsets on its stream). 0 for k <= 0, where the call needs
 * drs_row_stats_workspace_bytes() instead. Same sharing rule as the
 * row-stats workspace.
 */
size_t drs_row_stats_topk_workspace_bytes(int64_t rows, int64_t vocab, int32_t k);

/*
 * drs_row_stats and the top-k logprobs of the rows of converged slots from
 * the same read of the logits (stash_converged_logprobs /
 * _lp_topk_kernel on the page above, whose stash reads the kept rows again
 * in a kernel of its own). Every argument of drs_row_stats has its meaning
 * there; in addition:
 *
 *   keep        uint8 [ceil((row0 + rows) / canvas_len)], one per slot of
 *               the whole batch like temps: global row r is converged when
 *               keep[r / canvas_len] != 0.
 *   k           0 <= k <= min(vocab, 1024); k == 0 is drs_row_stats (with
 *               its workspace size).
 *   out_ids     int32 [rows, k]: for a converged row, the columns of the k
 *               largest scaled logits, ordered by value and then by lower
 *               column (-0.0 equals +0.0). Rows of other slots are not
 *               written.
 *   out_logprobs fp32 [rows, k]: scaled - max - log(sum exp(scaled - max))
 *               of those columns (NaN for a row that is -inf everywhere).
 *   workspace   drs_row_stats_topk_workspace_bytes(rows, vocab, k) bytes.
 *
 * For k <= 64 the top-k candidates come out of the row statistics' own read
 * of the logits: in the cluster kernel the threshold from the CTAs' parts
 * (distributed shared memory) and the candidates from the row held in shared
 * memory; in the two passes the threshold from the first and the candidates
 * in the second. Rows whose candidates overflow the fixed lists (many equal
 * values) or that have no threshold are finished by the exact top-k kernel
 * on the same stream, which reads only those rows. For k > 64 the row
 * statistics and the exact top-k kernel run one after the other.
 */
drs_status drs_row_stats_topk(const float *logits, int64_t rows, int64_t vocab,
                              int64_t row_stride, const float *temps,
                              int64_t canvas_len, uint64_t seed, int64_t row0,
                              int64_t *argmax, int64_t *sample, float *entropy,
                              drs_probs_dtype probs_dtype, void *probs,
                              int64_t probs_row_stride, const uint8_t *keep,
                              int32_t k, int32_t *out_ids, float *out_logprobs,
                              void *workspace, size_t workspace_bytes,
                              void *stream);

/*
 * Bytes of device workspace drs_topk_logprobs needs (256-byte aligned,
 * contents arbitrary). Same sharing rule as the row-stats workspace.
 */
size_t drs_topk_workspace_bytes(int64_t rows, int64_t vocab, int32_t k);

/*
 * Top-k logprobs of the rows of converged slots (stash_converged_logprobs
 * and _lp_topk_kernel on the page above).
 *
 *   logits, rows, vocab, row_stride, temps, canvas_len: as drs_row_stats;
 *               rows must be a multiple of canvas_len.
 *   keep        uint8 [rows / canvas_len]: slot n is converged when
 *               keep[n] != 0. Rows of other slots are skipped and their
 *               outputs are not written.
 *   k           0 <= k <= min(vocab, 1024); k == 0 does nothing.
 *   out_ids     int32 [rows, k]: for a kept row, the columns of the k
 *               largest scaled logits, ordered by value and then by lower
 *               column (-0.0 equals +0.0).
 *   out_logprobs fp32 [rows, k]: scaled - max - log(sum exp(scaled - max))
 *               of those columns (NaN for a row that is -inf everywhere).
 *
 * For k <= 64 this runs the kernels of drs_row_stats_topk with the row
 * statistics off (rows of unconverged slots are not read); larger k, and
 * rows with many equal values, use the exact top-k kernel.
 */
drs_status drs_topk_logprobs(const float *logits, int64_t rows, int64_t vocab,
                             int64_t row_stride, const float *temps,
                             int64_t canvas_len, const uint8_t *keep,
                             int32_t k, int32_t *out_ids, float *out_logprobs,
                             void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * The sampler's noise, materialised (the generator of drs_row_stats).
 * Page "vllm.model_executor.models.diffusion_gemma_sampler",
 * sample_row_stats_reference: the Gumbel noise -log(-log u) of a uniform u
 * drawn like rand_like(...) and clamped below at 1e-20; the page's kernel
 * takes a seed, and the uniform is drawn here by Philox4x32-10 (Salmon,
 * Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
 * SC'11) keyed and laid out as the `seed` argument of drs_row_stats states.
 * For r in [0, rows), c in [0, vocab): out_bits[r * vocab + c] is the
 * Philox word of (row0 + r, c) and out_gumbel[r * vocab + c] the fp32
 * -log(-log u) of it, u = max((word >> 8) * 2^-24, 1e-20f). Either output
 * may be NULL; rows == 0 is a no-op. Outputs are caller-owned device
 * memory; invalid sizes return DRS_ERR_INVALID_ARG before any launch.
 */
drs_status drs_philox_gumbel(uint64_t seed, int64_t row0, int64_t rows,
                             int64_t vocab, uint32_t *out_bits,
                             float *out_gumbel, void *stream);

/*
 * The temperature-scaled logits of sample_row_stats_reference (page above):
 * out[i] = logits[i] / max(temp, 1e-10f) for i < n, the IEEE fp32 quotient
 * rounded to nearest even, computed by the same routine the row kernels use
 * (+-inf map to themselves). logits and out: device fp32 [n], 4-byte
 * aligned; they may be the same array. n == 0 is a no-op.
 */
drs_status drs_scaled_logits(const float *logits, int64_t n, float temp,
                             float *out, void *stream);

/*
 * Test hook for the failure path (not for production use). code != 0: in
 * the next row-statistics call of this process, CTA 0 of the first pass
 * never fills its first shared-memory stage. Its warps' bounded waits on the
 * stage run out (about 1 s), the CTA stops and raises the device flag that
 * drs_get_device_error reports; the call's results are not valid, the CUDA
 * context stays usable. The hook resets itself after one call; code 0
 * clears it.
 */
void drs_test_inject_fault(int code);

/*
 * Test hook (not for production use). on != 0: from now on every
 * row-statistics call of this process takes the two streaming passes over
 * the logits (list of rows, pass 1, merge, pass 2, finish) even where the
 * one-read cluster kernel would take it (rows that start 16-byte aligned,
 * vocab a multiple of 4 and at most 262144, one seed, k <= 64). Results are
 * the same within the tolerances of the method; the hook exists so that
 * both implementations can be tested and timed on the same inputs. on == 0
 * restores the automatic choice.
 */
void drs_test_two_pass(int on);

/*
 * Introspection (not part of the sampler): how a row-statistics call of
 * these sizes shares its rows on the current device. Calls whose rows start
 * 16-byte aligned, with vocab a multiple of 4 and at most 262144, one seed
 * and k <= 64 read each row once, split over the CTAs of a thread-block
 * cluster (*cluster_size CTAs per row, *clusters clusters resident at once,
 * one CTA per SM); such clusters fit only some of the GPU's SM groups, and on
 * large calls the *free_sms SMs they leave run the two streaming passes over
 * the tail of the call's row list at the same time. *cluster_rows is the
 * head of a list of `rows` entries; a call whose list is shorter (a top-k
 * call lists the rows of kept slots only) divides it in the same proportion
 * on the device. Other calls take the two passes alone: *cluster_rows, *cluster_size,
 * *clusters and *free_sms are then 0. probs_dtype: a drs_probs_dtype value;
 * stats: nonzero for the calls that compute the row statistics
 * (drs_row_stats, drs_row_stats_topk), 0 for the top-k calls
 * (drs_topk_logprobs, the stash). Top-k calls take no cluster kernel: they
 * read each row once in the first streaming pass and then only the columns
 * of the row's warps whose max reaches its top-k threshold (all outputs 0).
 * All outputs are HOST pointers. Returns DRS_OK, or DRS_ERR_INVALID_ARG for a
 * null pointer or sizes out of range.
 */
drs_status drs_row_split_plan(int64_t rows, int64_t vocab, int32_t k, int32_t n_seeds,
                              int probs_dtype, int32_t stats, int64_t *cluster_rows,
                              int32_t *cluster_size, int32_t *clusters, int32_t *free_sms);

/*
 * Measurement hook (not part of the sampler). enable != 0: from now on every
 * row-statistics call on the current device (drs_row_stats, its no-alloc and
 * top-k variants, drs_topk_logprobs for k <= 64) records a CUDA event on
 * its stream before each of six kernel slots (list of rows, pass 1, merge,
 * pass 2, cluster, finish) and after the last; the slots a call does not
 * launch (the two passes or the cluster kernel) measure about 0, and a
 * top-k call's finish slot times its gather (split_gather). The count
 * of recorded calls restarts at 0. enable == 0 stops recording. The events
 * of the last 64 calls are kept. Returns DRS_OK or DRS_ERR_CUDA (event
 * creation failed).
 */
drs_status drs_kernel_timing(int enable);

/*
 * Average device time in ms of each kernel slot of the recorded calls (see
 * drs_kernel_timing), in the order above, into the HOST array avg_ms[n]
 * (entries past the sixth are 0); *calls (HOST) receives the number of
 * calls averaged (at most 64). Waits for the recorded events. Returns
 * DRS_OK, DRS_ERR_INVALID_ARG (null pointer, n < 0) or DRS_ERR_CUDA.
 */
drs_status drs_kernel_times(float *avg_ms, int32_t n, int32_t *calls);

/*
 * Bytes of device workspace drs_stash_converged_logprobs needs (256-byte
 * aligned, contents arbitrary); 0 for arguments outside its ranges
 * (num_topk in [0, 1024]).
 */
size_t drs_stash_workspace_bytes(int64_t requests, int64_t canvas_len, int64_t vocab,
                                 int32_t num_topk);

/*
 * The stash of converged requests' logprobs (stash_converged_logprobs on
 * the page above, its docstring). Request j < requests owns logits rows
 * src[j] * canvas_len + p for p < valid[j], scaled by
 * max(temps[j], 1e-10). Where keep[j] != 0, stash row
 * slots[j] * canvas_len + p of the outputs receives `width` columns of
 * (id, value):
 *   column 0        the argmax of the scaled row (lowest column of the max);
 *   then            token_ids[j * ids_stride + c] for c < n_j =
 *                   min(num_token_ids[j], ids_stride) when token_ids is
 *                   given and n_j > 0 (a request's list holds ids_stride
 *                   ids; a larger count reads no further), else
 *                   the num_topk largest (value descending, lower column
 *                   first);
 *   then            id 0 with value -inf, up to `width`.
 * value: the logprob s - max - log(sum over the row of e^(s - max)) (NaN
 * when the row is -inf everywhere), or the scaled logit s itself when
 * logits_mode != 0; NaN for a token id outside [0, vocab).
 * out_ranks[stash row]: 1 + the number of columns whose scaled logit
 * exceeds column 0's (column 0 is the argmax, so 1).
 *
 *   logits          fp32, row r at logits + r * row_stride, r < logits_rows.
 *   src, slots, valid, num_token_ids   int32 [requests] (num_token_ids may
 *                   be null without token_ids).
 *   keep            uint8 [requests]; temps fp32 [requests].
 *   token_ids       null, or int32 [requests, ids_stride].
 *   out_ids         int32 [out_slots * canvas_len, width]; out_logprobs
 *                   fp32 and out_ranks int32 [out_slots * canvas_len] alike.
 *                   Rows of requests not kept, positions p >= valid[j], and
 *                   rows whose logits row or stash row falls outside
 *                   logits_rows or out_slots are not touched.
 *   workspace       drs_stash_workspace_bytes(requests, canvas_len, vocab,
 *                   num_topk) bytes.
 * The slots of kept requests must be distinct: two requests writing one
 * stash row race (which one lands is not defined).
 * All pointers are device memory owned by the caller; asynchronous on
 * `stream`. Returns DRS_ERR_INVALID_ARG for a null required pointer,
 * negative sizes, row_stride < vocab, num_topk outside [0, min(vocab,
 * 1024)], width < num_topk + 1, token_ids without num_token_ids or with
 * ids_stride < 1, or a small or unaligned workspace;
 * DRS_ERR_UNSUPPORTED for vocab > DRS_MAX_VOCAB or more than 2^31 - 1
 * stash rows; requests == 0 is a no-op.
 */
drs_status drs_stash_converged_logprobs(const float *logits, int64_t logits_rows, int64_t vocab,
                                        int64_t row_stride, int64_t canvas_len, int64_t requests,
                                        const int32_t *src, const int32_t *slots,
                                        const uint8_t *keep, const int32_t *valid,
                                        const float *temps, int32_t num_topk,
                                        const int32_t *num_token_ids, const int32_t *token_ids,
                                        int64_t ids_stride, int64_t out_slots, int32_t width,
                                        int32_t *out_ids, float *out_logprobs,
                                        int32_t *out_ranks, int logits_mode, void *workspace,
                                        size_t workspace_bytes, void *stream);

/*
 * Verification of drafted tokens against the target model's probabilities
 * (speculative sampling), with the random numbers given. The probabilities
 * are rows as drs_row_stats writes them, or fp32 ones. Request b has
 *   k_b = cu_drafts[b + 1] - cu_drafts[b]
 * drafted tokens (at most max_drafts; more are not looked at), its draft j
 * being entry r = cu_drafts[b] + j of draft_tokens, accept_u and the rows of
 * draft. The target has one row more per request: row cu_drafts[b] + b + j
 * is the distribution that draft j is held against, j == k_b the one after
 * the last draft.
 *   - Draft j is accepted when accept_u[r] * q < p, with p and q the target's
 *     and the draft's probability of draft_tokens[r] (the product is exact;
 *     q is 1 without draft probabilities). A token outside [0, vocab) is
 *     refused. Drafts count up to the first refused one.
 *   - Then one more token is drawn. After a refused draft: from the weights
 *     max(p - q, 0) of its position (the fp32 difference), or, without
 *     draft probabilities, from p without the refused token; where these
 *     weights are all 0, from p. After the last draft: from p of the next
 *     position. NaN and negative weights are 0; infinite ones are not supported.
 *     The token is the lowest column whose running sum of weights exceeds
 *     sample_u[b] times their total (the sums are good to about 1e-13);
 *     -1 where there is no weight at all.
 *
 *   target      target_dtype [target_rows, vocab], row stride target_stride.
 *   draft       draft_dtype [draft_rows, vocab], row stride draft_stride, or
 *               NULL (drafts without probabilities, such as looked-up ones).
 *   draft_rows  the number of drafted tokens; draft_tokens int64 and
 *               accept_u fp32 [draft_rows], uniform in [0, 1). Both may be
 *               NULL when it is 0.
 *   cu_drafts   int32 [requests + 1].
 *   sample_u    fp32 [requests], uniform in [0, 1).
 *   out_tokens  int64 [requests, max_drafts + 1]: the accepted drafts, the
 *               drawn token, then -1.
 *   out_accepted int32 [requests]: the number of accepted drafts. A
 *               request whose rows fall outside draft_rows or target_rows
 *               gets -1 here and in all its tokens.
 *
 * A row is read at most once (two with draft probabilities): the one that
 * the token is drawn from. No workspace. Rows that start 16-byte aligned are
 * read faster. requests == 0 is a no-op. Returns DRS_ERR_INVALID_ARG for
 * negative sizes, an unknown type, a stride below vocab, a null or unaligned
 * pointer; DRS_ERR_UNSUPPORTED for vocab > DRS_MAX_VOCAB or more than
 * 2^27 - 1 requests; DRS_ERR_CUDA on a device (a partition, say) that grants
 * no clusters of 16 CTAs, like drs_map_slots and drs_embed_tokens_grad.
 */
drs_status drs_verify_drafts(const void *target, drs_dtype target_dtype, int64_t target_rows,
                             int64_t target_stride, const void *draft, drs_dtype draft_dtype,
                             int64_t draft_rows, int64_t draft_stride, int64_t vocab,
                             const int64_t *draft_tokens, const int32_t *cu_drafts,
                             int64_t requests, int32_t max_drafts, const float *accept_u,
                             const float *sample_u, int64_t *out_tokens, int32_t *out_accepted,
                             void *stream);

/*
 * Block tables and slot maps of a paged cache, from the requests' lengths on
 * the GPU. Request b has lens[b] tokens in the cache and adds new_lens[b]
 * (negative lengths are 0). Its row of the block table holds the
 * ids of the blocks of block_size tokens that it has: columns [0, held[b]).
 * The call makes that ceil((lens + new) / block_size) blocks: missing ones
 * come from a ring of free block ids, blocks beyond go back to it (all of a
 * request whose lengths are 0), both in request order. Then every new token
 * gets its request, its position and its place in the cache.
 *
 *   block_table int32 [requests, max_blocks], row stride table_stride,
 *               updated in place: columns [held[b], out_held[b]) are written,
 *               no other.
 *   free_ring   int32 [ring_size], updated in place. ring_state[0] (head)
 *               and ring_state[1] (tail) count the ids ever taken and given:
 *               the free ids are free_ring[i % ring_size] for head <= i <
 *               tail. ring_size is at least the number of blocks of
 *               the cache. Ids given back in a call are free from the next.
 *   out_held    int32 [requests]: blocks now held (may be held itself).
 *   out_ring_state int64 [2]: the counters after the call (may be ring_state
 *               itself).
 *   out_lacking int32 [1]: blocks that lengths asked for and did not get: the
 *               ring ran out (a request is served when its blocks and those of
 *               the requests before it are there, and keeps what it holds
 *               otherwise) or the table's row has no more columns. 0 in
 *               ordinary operation.
 *   capacity    entries of the token arrays (a captured graph's size, say);
 *               tokens beyond it are left out.
 *   out_cu      int32 [requests + 1]: the first token of each request, and
 *               the number of tokens.
 *   out_request, out_position int32 [capacity], out_slot int64 [capacity]:
 *               token t = out_cu[b] + j has request b, position lens[b] + j
 *               and slot block_table[b][position / block_size] * block_size
 *               + position % block_size, -1 where the request has no block
 *               for it. Entries past the last token: -1, 0, -1.
 *
 * Arrays do not overlap except as said. One launch, two above 8192 entries;
 * no workspace; the arrays' contents cannot lead outside them. Positions are at most 2^31 - 1.
 * Returns DRS_ERR_INVALID_ARG for sizes out of range or a null or
 * unaligned pointer; DRS_ERR_UNSUPPORTED for more than DRS_MAX_REQUESTS
 * requests or 2^31 - 1 tokens.
 */
drs_status drs_map_slots(const int32_t *lens, const int32_t *new_lens, const int32_t *held,
                         int64_t requests, int32_t block_size, int32_t *block_table,
                         int64_t table_stride, int32_t max_blocks, int32_t *free_ring,
                         int64_t ring_size, const int64_t *ring_state, int64_t capacity,
                         int32_t *out_cu, int32_t *out_request, int32_t *out_position,
                         int64_t *out_slot, int32_t *out_held, int64_t *out_ring_state,
                         int32_t *out_lacking, void *stream);

/*
 * The embedding lookup with scaling: out[t] = scale * table[ids[t]], the
 * product taken in fp32 and rounded once. Rows of ids outside [0, vocab)
 * (padding) are 0.
 *
 *   table       dtype [vocab, width], row stride table_stride.
 *   ids         int32 or int64 [tokens] (id_bits 32 or 64).
 *   out         dtype [tokens, width], row stride out_stride.
 *
 * tokens == 0 is a no-op. Any alignment and stride; tables whose rows
 * start 16-byte aligned are read faster. Returns DRS_ERR_INVALID_ARG for
 * sizes out of range, an unknown type, a stride below width or a null or
 * unaligned pointer; DRS_ERR_UNSUPPORTED for vocab > DRS_MAX_VOCAB, width
 * > DRS_MAX_WIDTH or too many tokens for one launch (2^31 - 1 blocks).
 */
drs_status drs_embed_tokens(const void *table, drs_dtype dtype, int64_t vocab, int64_t width,
                            int64_t table_stride, const void *ids, int32_t id_bits,
                            int64_t tokens, float scale, void *out, int64_t out_stride,
                            void *stream);

/*
 * Bytes of device workspace drs_embed_tokens_grad needs (256-byte aligned,
 * contents arbitrary); 0 for no tokens or sizes out of range. Same sharing
 * rule as the row-stats workspace.
 */
size_t drs_embed_tokens_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width);

/*
 * The gradient of drs_embed_tokens with respect to its table:
 *   grad_table[v] = (accumulate ? grad_table[v] : 0)
 *                   + scale * sum of grad_out[t] over the tokens t with
 *                     ids[t] == v.
 * The sums are fp32 and are added in an order that depends on the ids alone
 * (equal calls give equal bits); the result is rounded once.
 * Ids outside [0, vocab) have no part in it. With accumulate only the rows of
 * ids that occur are read and written, else every row is written.
 *
 *   grad_out    grad_dtype [tokens, width], row stride grad_stride.
 *   ids, id_bits as drs_embed_tokens.
 *   grad_table  table_dtype [vocab, width], row stride table_stride.
 *   workspace   drs_embed_tokens_grad_workspace_bytes(tokens, vocab, width).
 *
 * Returns DRS_ERR_INVALID_ARG for sizes out of range, an unknown type, a
 * stride below width, a null or unaligned pointer or a small workspace;
 * DRS_ERR_UNSUPPORTED for sizes above DRS_MAX_TOKENS, DRS_MAX_VOCAB or
 * DRS_MAX_WIDTH, or too many tokens and columns for one launch (2^31 - 1
 * blocks).
 */
drs_status drs_embed_tokens_grad(const void *grad_out, drs_dtype grad_dtype, int64_t tokens,
                                 int64_t width, int64_t grad_stride, const void *ids,
                                 int32_t id_bits, float scale, int accumulate,
                                 void *grad_table, drs_dtype table_dtype, int64_t vocab,
                                 int64_t table_stride, void *workspace, size_t workspace_bytes,
                                 void *stream);

/*
 * Log probabilities of given tokens under softmax(logits / T), with the
 * distribution's entropy, the token's rank and the k largest alternatives,
 * from one read of the logits (scoring of prompts and samples, the forward
 * pass of a loss). With te = max(T, 1e-10), m = the row's largest logit,
 * S = the sum over the row of e^((x - m) / te):
 *   out_logprob  fp32 [rows]: (x_id - m) / te - ln S, the log probability of
 *                the row's token.
 *   out_entropy  fp32 [rows]: ln S - (1 / S) * the sum of
 *                e^((x - m) / te) (x - m) / te; -inf columns drop out.
 *   out_rank     int32 [rows]: 1 + the number of columns whose logit exceeds
 *                the token's.
 *   out_norm     fp32 [rows, 2]: (m, ln S), which drs_token_logprobs_grad
 *                takes in place of a second look for them.
 *   out_ids, out_logprobs  int32 and fp32 [rows, k]: the columns of the k
 *                largest logits (equal ones in column order, -0 equal to 0)
 *                and their log probabilities.
 * out_entropy, out_rank and out_norm may be NULL; so may out_ids and
 * out_logprobs when k is 0.
 * ln S and the entropy are at least 0 and log probabilities at most 0. All is
 * computed in fp32, quotients by te as products with 1 / te: where one logit
 * holds nearly all of the sum, ln S and its token's log probability are right
 * to a few steps of fp32 at 1, not of themselves.
 *
 *   logits      dtype [rows, vocab], row stride row_stride.
 *   ids         int32 or int64 [rows] (id_bits 32 or 64). A row whose id is
 *               outside [0, vocab) (padding) is passed over: its outputs are 0,
 *               0, 0, (0, 0), and -1 and -inf for the alternatives.
 *   temps       fp32 [ceil(rows / canvas_len)]: row r has
 *               T = temps[r / canvas_len] (finite or NaN, which is taken as
 *               1e-10). NULL: 1 for every row.
 *
 * A row that is -inf everywhere has no distribution: its log probabilities
 * are NaN, its entropy 0, its norm (-inf, -inf), its alternatives the first
 * columns. A row with NaN or +inf has NaN for what depends on its sum; NaN
 * columns rank below all others, with -inf ones in column order.
 *
 * One launch, no workspace. rows == 0 is a no-op. Any stride and alignment
 * that the type allows. Masks are best made of -inf: rows that begin with long
 * stretches of the type's lowest finite value are read twice.
 * Returns DRS_ERR_INVALID_ARG for sizes out of range
 * (k > vocab among them), an unknown type, a stride below vocab, a null or
 * unaligned pointer; DRS_ERR_UNSUPPORTED for vocab > DRS_MAX_VOCAB,
 * k > DRS_MAX_ALTERNATIVES or rows > DRS_MAX_SCORE_ROWS; DRS_ERR_CUDA for few
 * long rows on a device that grants no clusters of 16 CTAs.
 */
drs_status drs_token_logprobs(const void *logits, drs_dtype dtype, int64_t rows, int64_t vocab,
                              int64_t row_stride, const void *ids, int32_t id_bits,
                              const float *temps, int64_t canvas_len, int32_t k,
                              float *out_logprob, float *out_entropy, int32_t *out_rank,
                              float *out_norm, int32_t *out_ids, float *out_logprobs,
                              void *stream);

/*
 * The gradient of drs_token_logprobs' out_logprob and out_entropy with
 * respect to the logits:
 *   grad[r, j] = (1 / te) (g ([j == id] - p_j) - h p_j (ln p_j + H))
 * with p_j = e^((x_j - m) / te - ln S) from the forward call's norm, H its
 * entropy, g = grad_logprob[r] and h = grad_entropy[r]; computed in fp32 and
 * rounded once. Rows passed over in the forward call and rows that are -inf
 * everywhere (whose ln S is -inf) get zeros, rows with NaN or +inf get NaN; every
 * row is written, and nothing behind vocab.
 *
 *   logits, ids, id_bits, temps, canvas_len   as drs_token_logprobs.
 *   norm         fp32 [rows, 2], out_norm of the forward call.
 *   entropy      fp32 [rows], out_entropy of the forward call; needed with
 *                grad_entropy only.
 *   grad_logprob, grad_entropy  fp32 [rows]; NULL counts as zeros, one of
 *                them is given.
 *   grad         grad_dtype [rows, vocab], row stride grad_stride. It may be
 *                logits itself (of the same type and stride), and does not
 *                overlap it otherwise.
 *
 * One launch, no workspace; equal calls give equal bits. Errors as
 * drs_token_logprobs.
 */
drs_status drs_token_logprobs_grad(const void *logits, drs_dtype dtype, int64_t rows,
                                   int64_t vocab, int64_t row_stride, const void *ids,
                                   int32_t id_bits, const float *temps, int64_t canvas_len,
                                   const float *norm, const float *entropy,
                                   const float *grad_logprob, const float *grad_entropy,
                                   void *grad, drs_dtype grad_dtype, int64_t grad_stride,
                                   void *stream);

/*
 * Dropout from the counter-based generator, its mask never stored:
 *   out[r, j] = residual[r, j] + (kept ? x[r, j] / (1 - q) : 0)
 * in fp32, rounded once; without a residual the second term alone. The share
 * q dropped is p rounded to a multiple of 2^-16 (ties up), and 1 - q that
 * of the kept ones, so the expectation is exact; q = 1 drops all. What x
 * holds in a dropped place has no part in the result (NaN, infinities).
 * The mask is a function of (seed, global row row0 + r, column): element j is
 * dropped when the 16-bit number u < q 2^16, with u the lower (j even) or
 * upper (j odd) half of word (j % 8) / 2 of Philox4x32-10 with the key of
 * drs_row_stats and counter (j / 8, 0x64726F70, lo32(row), hi32(row)). The
 * counter's second word keeps it apart from the sampler's noise of the same
 * seed. A batch split over several calls draws what one call draws.
 *
 *   x           dtype [rows, width], row stride x_stride.
 *   residual    NULL, or out_dtype [rows, width], row stride residual_stride.
 *   seed        the key; device_seed, when not NULL, is read in its place on
 *               the GPU (one uint64): a captured graph then draws anew at
 *               each replay from what stands there.
 *   out         out_dtype [rows, width], row stride out_stride. It may be x
 *               (of the same type and stride) or residual (of the same
 *               stride) itself, and does not overlap them otherwise.
 *
 * One launch (q = 1 without a residual: a fill), no workspace. rows == 0 is
 * a no-op. Returns DRS_ERR_INVALID_ARG for sizes out of range, p outside [0, 1], an unknown
 * type, a stride below width, a null or unaligned pointer;
 * DRS_ERR_UNSUPPORTED for width > DRS_MAX_WIDTH or too many rows for one
 * launch (2^31 - 1 blocks).
 */
drs_status drs_dropout(const void *x, drs_dtype dtype, int64_t rows, int64_t width,
                       int64_t x_stride, const void *residual, int64_t residual_stride, float p,
                       uint64_t seed, const uint64_t *device_seed, int64_t row0, void *out,
                       drs_dtype out_dtype, int64_t out_stride, void *stream);

/*
 * The gradient of drs_dropout with respect to x, from the same p, seed and
 * row0: grad_x[r, j] = kept ? grad_out[r, j] / (1 - q) : 0 (that with
 * respect to the residual is grad_out itself). grad_x may be grad_out (of
 * the same type and stride). Errors as drs_dropout.
 */
drs_status drs_dropout_grad(const void *grad_out, drs_dtype grad_dtype, int64_t rows,
                            int64_t width, int64_t grad_stride, float p, uint64_t seed,
                            const uint64_t *device_seed, int64_t row0, void *grad_x,
                            drs_dtype x_dtype, int64_t x_stride, void *stream);

/* Static, human-readable name of a status code. */
const char *drs_status_string(drs_status s);

/*
 * Synchronise `stream`, then read and clear the device flag raised by a
 * kernel whose bounded wait ran out of time on the current device.
 * Returns DRS_OK, DRS_ERR_DEVICE_TIMEOUT or DRS_ERR_CUDA.
 */
drs_status drs_get_device_error(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DRS_H_ */
