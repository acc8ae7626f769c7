/*
 * kpool.h -- C ABI of the GB300 (sm_103a) KPool DSA indexer selection library.
 *
 * The operation (per packed batch of causal sequences):
 *   1. Mean-pool every kpool consecutive index keys of a sequence into one pooled
 *      key ("spark_model/layers/glm5next_dsa/tp.rs", module docs, "Why the
 *      indexer is REPLICATED": n_pools = seq / kpool). The pages do not name the
 *      pooling operator; this library reads it as the mean: an fp32 sum in key
 *      order, an IEEE fp32 division by kpool, round-to-nearest-even to the input
 *      dtype.
 *   2. Score every causally eligible (query row t, pool p) pair,
 *         s[t,p] = sum_h w[t,h] * relu(scale * q[t,h,:] . kpool[p,:]),
 *      a plain sum over heads taken before any top-k (same page and section).
 *      A row t (sequence-local) may use the pools p < floor((t+1)/kpool), i.e.
 *      the complete pools whose last key is at or before t.
 *   3. Keep the top budget = index_topk / kpool pools of each row, ordered by
 *      higher score first and then smaller pool index (tp.rs module docs: the
 *      deterministic tiebreak pinned because torch.topk's tie order is
 *      undefined). Rows with fewer eligible pools are padded with -1.
 *   4. Expand the chosen pools to token ids, append the row's own incomplete
 *      trailing pool and apply the causal / varlen mask ("NVIDIA/Megatron-LM
 *      pull request #8299", section "Change": pool expansion, tail append and
 *      mask filtering run on the [batch, sq, budget] pool ids).
 *
 * Sequences arrive packed (THD) with cumulative lengths cu_seqlens, as in the
 * pages' packed-THD tests (Megatron-LM #8299, section "Test plan"); a dense
 * batch [B, sq] is cu_seqlens = {0, sq, 2sq, ...}. Every index the library
 * returns is sequence-local.
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller; the library
 *     allocates no device memory. Scratch state lives in a caller-provided
 *     workspace of kpool_workspace_bytes() bytes (256-byte aligned).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream). The returned status covers host-side validation and launch
 *     errors; errors found on the device (malformed cu_seqlens, a bounded wait
 *     that ran out) are recorded in the workspace and read back with
 *     kpool_last_device_error().
 *   - Validation happens before anything touches the GPU: a call that returns
 *     KPOOL_ERR_INVALID_ARG / _UNSUPPORTED / _WORKSPACE launched nothing.
 *   - Calls that share a workspace must not overlap on the GPU.
 *
 * Layouts (row-major, contiguous):
 *   q          [T, H, d]            dtype   (16-byte aligned)
 *   k          [T, d]               dtype   (16-byte aligned)
 *   w          [T, H]               fp32
 *   cu_seqlens [S + 1]              int32   cu[0] = 0, nondecreasing, cu[S] = T
 *   pool ids   [T, budget]          int32   rank order, -1 padded
 *   token ids  [T, index_topk+kpool] int32  slot j*kpool + r = pool_ids[j]*kpool + r;
 *                                           slots index_topk + r = the row's tail;
 *                                           -1 where empty or masked
 *   pool scores[T, budget]          fp32    score of each chosen pool, -INFINITY on -1 slots
 */
#ifndef KPOOL_H_
#define KPOOL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KPOOL_OK = 0,
  KPOOL_ERR_INVALID_ARG = 1,    /* null/misaligned pointer, bad size, kpool < 1,
                                   index_topk % kpool != 0, malformed cu_seqlens */
  KPOOL_ERR_UNSUPPORTED = 2,    /* shape outside what the kernels implement */
  KPOOL_ERR_WORKSPACE = 3,      /* workspace null, misaligned or too small */
  KPOOL_ERR_CUDA = 4,           /* a CUDA runtime/driver call or launch failed */
  KPOOL_ERR_DEVICE_TIMEOUT = 5, /* a bounded device-side wait ran out */
  KPOOL_ERR_INTERNAL = 6        /* a device-side bounds guard fired (a library bug; the
                                   offending write was skipped) */
} kpool_status;

typedef enum { KPOOL_BF16 = 0, KPOOL_F32 = 1 } kpool_dtype;

/* Which score+select kernel kpool_select_ex runs. */
typedef enum {
  KPOOL_SCORE_AUTO = 0,   /* tensor-core kernel when the shape allows, else SIMT */
  KPOOL_SCORE_TC = 1,     /* tcgen05/TMEM kernel: bf16, H = 32, d = 128, budget <= 512 */
  KPOOL_SCORE_SIMT = 2    /* CUDA-core kernel: any H <= 64, d <= 256, budget <= 4096 */
} kpool_score_kernel;

typedef struct {
  int32_t score_kernel;       /* a kpool_score_kernel value */
  int32_t max_ctas;           /* 0: one persistent CTA per SM; > 0: cap (tests vary it) */
  void* const* stage_events;  /* NULL, or 5 cudaEvent_t (created by the caller) that are
                                 recorded on `stream` before the planning kernel and after
                                 the plan, pool, score+select and expand kernels, so a
                                 caller can time each kernel without a profiler; inside a
                                 stream capture they become event-record nodes of the
                                 graph, recorded again on every replay */
  int32_t row_begin;          /* with KPOOL_OPT_ROW_RANGE in flags: the call selects for the */
  int32_t row_end;            /* global rows [row_begin, row_end) only (else both zero)    */
  int32_t flags;              /* 0 or KPOOL_OPT_ROW_RANGE                                   */
  int32_t reserved;           /* must be zero */
} kpool_options;

/*
 * Query-row sharding ("NVIDIA/Megatron-LM pull request #8299", section "Change";
 * "NovaSky-AI/SkyRL pull request #2422", Summary): rows are independent, so a
 * group of G processes can each select a contiguous range of query rows and
 * all-gather the int32 pool ids; expansion then runs on the gathered
 * [T, budget] tensor (kpool_expand). With KPOOL_OPT_ROW_RANGE, kpool_select_ex
 * and kpool_select_pooled take the whole batch's q, k (or pooled keys), w and
 * cu_seqlens but score, select and expand only the global rows
 * [row_begin, row_end), 0 <= row_begin <= row_end <= T. Their outputs then hold
 * R = row_end - row_begin rows: out_pool_ids [R, budget], out_token_ids
 * [R, index_topk + kpool], row i being global row row_begin + i, each exactly
 * as the whole-batch call would write that row. An empty range is a no-op.
 * As on the pages, the sharded path returns no index scores: out_pool_scores
 * must be NULL (else KPOOL_ERR_INVALID_ARG). The workspace size is the
 * whole batch's. kpool_balanced_row_split() gives ranges of equal work.
 */
#define KPOOL_OPT_ROW_RANGE 1

/*
 * Workspace size, in bytes, for a call with these sizes. Pure host arithmetic;
 * never touches the GPU. Returns 0 for arguments kpool_select would reject.
 */
size_t kpool_workspace_bytes(int64_t total_tokens, int32_t num_seqs, int32_t heads, int32_t head_dim,
                             kpool_dtype dtype, int32_t kpool, int32_t index_topk);

/*
 * The whole selection (steps 1-4 above) for one packed batch.
 *   q, k, w, cu_seqlens  inputs as laid out above (device).
 *   scale                the fp32 factor inside the relu (any finite value).
 *   out_pool_ids         [T, budget] int32 (device), written for every row.
 *   out_token_ids        [T, index_topk + kpool] int32 (device), written for every row.
 *   out_pool_scores      [T, budget] fp32 (device) or NULL.
 *   workspace            device scratch of >= kpool_workspace_bytes(...) bytes.
 * T = 0 is a valid no-op. Requires d % 8 == 0 (16-byte rows) and heads >= 1.
 */
kpool_status kpool_select(const void* q, const void* k, const float* w, const int32_t* cu_seqlens,
                          int32_t num_seqs, int64_t total_tokens, int32_t heads, int32_t head_dim,
                          kpool_dtype dtype, int32_t kpool, int32_t index_topk, float scale,
                          int32_t* out_pool_ids, int32_t* out_token_ids, float* out_pool_scores,
                          void* workspace, size_t workspace_bytes, void* stream);

/* kpool_select with explicit options (NULL = defaults). */
kpool_status kpool_select_ex(const void* q, const void* k, const float* w, const int32_t* cu_seqlens,
                             int32_t num_seqs, int64_t total_tokens, int32_t heads, int32_t head_dim,
                             kpool_dtype dtype, int32_t kpool, int32_t index_topk, float scale,
                             int32_t* out_pool_ids, int32_t* out_token_ids, float* out_pool_scores,
                             void* workspace, size_t workspace_bytes, void* stream,
                             const kpool_options* options);

/*
 * Splits the rows of a packed batch into `parts` contiguous ranges of near-equal
 * work for query-row sharding. cu_seqlens is a HOST array [num_seqs + 1] (as the
 * device one); out_bounds, a HOST array of parts + 1 int32, receives
 * 0 = b[0] <= b[1] <= ... <= b[parts] = T, range g being rows [b[g], b[g+1]).
 * A row's work is its causal pair count floor((t+1)/kpool) (t sequence-local)
 * plus row_weight (the per-row cost of ranking, in pair units; 0 balances pairs
 * alone). The split minimises nothing globally: boundary g is the first row at
 * which the running work reaches g/parts of the total, so every range's work is
 * within one row's work of an equal share. The pages split rows evenly
 * (rank r takes rows [r*ceil(sq/G), ...)); under the causal mask that gives the
 * last rank about 2G-1 times the first rank's pairs, which this split avoids.
 * Pure host code; returns KPOOL_ERR_INVALID_ARG for malformed cu_seqlens,
 * kpool < 1, parts < 1 or row_weight < 0.
 */
kpool_status kpool_balanced_row_split(const int32_t* cu_seqlens, int32_t num_seqs, int32_t kpool,
                                      int64_t row_weight, int32_t parts, int32_t* out_bounds);

/*
 * Step 1 alone: writes the pooled keys [P, d] (dtype, P = sum_b floor(L_b/kpool),
 * sequences back to back) to out_pooled_keys, which must hold
 * floor(T/kpool) * d elements. Uses the workspace for the per-sequence offsets.
 */
kpool_status kpool_pool_keys(const void* k, const int32_t* cu_seqlens, int32_t num_seqs,
                             int64_t total_tokens, int32_t head_dim, kpool_dtype dtype, int32_t kpool,
                             void* out_pooled_keys, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Step 1 with gated pooling instead of the mean. The pages name a per-token,
 * per-channel compress gate (index_kpool_compress_gate, [head_dim, hidden]) and a
 * per-position embedding (index_kpool_compress_ape, [kpool, head_dim]) in the
 * GLM-5.3 DSA shard plan ("spark_model/layers/glm5next_dsa/tp.rs") and pass
 * "gate scores" to the fused top-k ("NVIDIA/Megatron-LM pull request #8299",
 * section "Mechanism"), but give no formula; this library reads them as gated
 * compression:
 *     kp[p,c] = sum_j softmax_j(gate[t_j,c]) * (k[t_j,c] + ape[j,c]),
 * t_j the pool's j-th token, computed in fp32 and rounded to the key dtype. A
 * zero gate and embedding reproduce the mean pooling bit for bit.
 *   gate  [T, d] fp32, 16-byte aligned (the gate scores, already projected from
 *         the hidden state)
 *   ape   [kpool, d] fp32, 16-byte aligned
 * Output and workspace as for kpool_pool_keys. Feed the result to
 * kpool_select_pooled.
 */
kpool_status kpool_pool_keys_gated(const void* k, const float* gate, const float* ape, const int32_t* cu_seqlens,
                                   int32_t num_seqs, int64_t total_tokens, int32_t head_dim, kpool_dtype dtype,
                                   int32_t kpool, void* out_pooled_keys, void* workspace, size_t workspace_bytes,
                                   void* stream);
/*
 * kpool_select_ex for pooled keys the caller already has (from kpool_pool_keys,
 * kpool_pool_keys_gated or a cache): steps 2-4 only. pooled_keys holds
 * floor(T/kpool) * d elements of dtype (the size kpool_pool_keys writes into),
 * the first P rows being the pools of cu_seqlens back to back; it is 16-byte
 * aligned and non-NULL even when no sequence holds a complete pool. Same workspace and
 * options as kpool_select_ex; the stage event after the pooling step is recorded
 * right after the planning one.
 */
kpool_status kpool_select_pooled(const void* q, const void* pooled_keys, const float* w, const int32_t* cu_seqlens,
                                 int32_t num_seqs, int64_t total_tokens, int32_t heads, int32_t head_dim,
                                 kpool_dtype dtype, int32_t kpool, int32_t index_topk, float scale,
                                 int32_t* out_pool_ids, int32_t* out_token_ids, float* out_pool_scores,
                                 void* workspace, size_t workspace_bytes, void* stream,
                                 const kpool_options* options);
/*
 * Full index scores, the pages' return_index_scores output ("NVIDIA/Megatron-LM
 * pull request #8299", section "Change": the op can return the index scores,
 * which it computes in row chunks of at most 2 GiB). Writes step 2's score of
 * every (row, pool) pair of a range of query rows instead of selecting:
 *   out_scores  [R, ld] fp32 (device, 4-byte aligned), R = row_end - row_begin:
 *               element (i, p), row i being global row row_begin + i (position t
 *               of its sequence), is s[t,p] for the sequence's pool p when
 *               p < floor((t+1)/kpool), and -INFINITY for every other p < ld.
 *   ld          row stride in elements, >= 1. Every row of the range needs
 *               ld >= floor((t+1)/kpool) (ld = floor(T/kpool) always suffices);
 *               a row that is wider keeps its first ld scores and the call records
 *               KPOOL_ERR_INVALID_ARG on the device (kpool_last_device_error).
 *   options     as for kpool_select_ex: KPOOL_OPT_ROW_RANGE picks the rows (the
 *               whole batch without it), so a caller bounds memory by calling once
 *               per chunk of rows; score_kernel picks the family, and the scores
 *               are bit-identical to the out_pool_scores a kpool_select_ex call with
 *               the same score kernel returns for the pools it selects.
 * q, k, w, cu_seqlens, the shape arguments, scale and the workspace are those of
 * kpool_select (workspace: kpool_workspace_bytes(T, S, H, d, dtype, kpool, 0)).
 * Supported shapes: the tensor-core kernel for bf16, H = 32, d = 128; the SIMT
 * kernel for H <= 64, d <= 256. The 4th and 5th stage events are both recorded
 * after the score kernel. An empty range or T = 0 is a no-op.
 */
kpool_status kpool_index_scores(const void* q, const void* k, const float* w, const int32_t* cu_seqlens,
                                int32_t num_seqs, int64_t total_tokens, int32_t heads, int32_t head_dim,
                                kpool_dtype dtype, int32_t kpool, float scale, float* out_scores, int64_t ld,
                                void* workspace, size_t workspace_bytes, void* stream,
                                const kpool_options* options);

/* kpool_index_scores for pooled keys the caller already has (as kpool_select_pooled). */
kpool_status kpool_index_scores_pooled(const void* q, const void* pooled_keys, const float* w,
                                       const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                       int32_t heads, int32_t head_dim, kpool_dtype dtype, int32_t kpool, float scale,
                                       float* out_scores, int64_t ld, void* workspace, size_t workspace_bytes,
                                       void* stream, const kpool_options* options);

/*
 * Step 4 alone: expands pool ids [T, budget] (as kpool_select writes them) into
 * token ids [T, index_topk + kpool], appending each row's tail and applying the
 * causal/varlen mask. Ids outside [0, floor((t+1)/kpool)) are treated as -1.
 */
kpool_status kpool_expand(const int32_t* pool_ids, const int32_t* cu_seqlens, int32_t num_seqs,
                          int64_t total_tokens, int32_t kpool, int32_t index_topk,
                          int32_t* out_token_ids, void* stream);

/*
 * Selection for an explicit set of query rows against pooled keys that already
 * exist: the decode / short-query case, where a few new query tokens score a
 * long pooled-key cache ("spark_model/layers/glm5next_dsa/tp.rs", module docs,
 * "Why the indexer is REPLICATED": at a 262,144-token context one decode token
 * scores n_pools = 65,536 pools). Row r sits at sequence-local position
 * row_pos[r] of sequence row_seq[r] of the key batch described by cu_seqlens,
 * and gets exactly what row row_pos[r] of kpool_select would get for a query
 * q[r] with weights w[r]: the top budget of the pools p < floor((t+1)/kpool) of
 * its sequence (higher score, then smaller pool index), -1 padded, rank order,
 * expanded to token ids with its incomplete trailing pool appended.
 *   q               [R, H, d] dtype (16-byte aligned); row r is that row's query.
 *   w               [R, H] fp32.
 *   row_seq, row_pos [R] int32 (device): 0 <= row_seq < S, 0 <= row_pos < L_b.
 *   pooled_keys     [P, d] dtype, as kpool_pool_keys writes them for cu_seqlens
 *                   (16-byte aligned; may be NULL only when T / kpool == 0).
 *   cu_seqlens      [S + 1] int32 of the key sequences, as for kpool_pool_keys.
 *   out_pool_ids    [R, budget] int32; out_token_ids [R, index_topk + kpool] int32;
 *   out_pool_scores [R, budget] fp32 or NULL.
 *   workspace       >= kpool_rows_workspace_bytes(R, T, S, kpool, index_topk) bytes.
 * Supported: bf16, H = 32, d = 128, budget <= 512 (else KPOOL_ERR_UNSUPPORTED).
 * R = 0 is a valid no-op. A row whose row_seq or row_pos is out of range gets
 * all -1 outputs and the call records KPOOL_ERR_INVALID_ARG on the device
 * (kpool_last_device_error); malformed cu_seqlens records the same and every
 * row gets -1 outputs. The call allocates and synchronises nothing, so a decode
 * loop can capture it into a CUDA graph; its second to fourth kernels are
 * launched with programmatic stream serialization (each waits on the device for
 * the one before it).
 */
size_t kpool_rows_workspace_bytes(int32_t num_rows, int64_t total_tokens, int32_t num_seqs, int32_t kpool,
                                  int32_t index_topk);
kpool_status kpool_select_rows(const void* q, const float* w, const int32_t* row_seq, const int32_t* row_pos,
                               int32_t num_rows, const void* pooled_keys, const int32_t* cu_seqlens,
                               int32_t num_seqs, int64_t total_tokens, int32_t heads, int32_t head_dim,
                               kpool_dtype dtype, int32_t kpool, int32_t index_topk, float scale,
                               int32_t* out_pool_ids, int32_t* out_token_ids, float* out_pool_scores,
                               void* workspace, size_t workspace_bytes, void* stream);
/*
 * kpool_select_rows with options (NULL = defaults). score_kernel must be
 * KPOOL_SCORE_AUTO; max_ctas > 0 caps the score kernel's grid (CTAs); stage_events, when
 * not NULL, holds 4 cudaEvent_t recorded on `stream` before the planning kernel
 * and after the planning, score and select kernels (event-record nodes when the
 * stream is being captured into a graph).
 */
kpool_status kpool_select_rows_ex(const void* q, const float* w, const int32_t* row_seq, const int32_t* row_pos,
                                  int32_t num_rows, const void* pooled_keys, const int32_t* cu_seqlens,
                                  int32_t num_seqs, int64_t total_tokens, int32_t heads, int32_t head_dim,
                                  kpool_dtype dtype, int32_t kpool, int32_t index_topk, float scale,
                                  int32_t* out_pool_ids, int32_t* out_token_ids, float* out_pool_scores,
                                  void* workspace, size_t workspace_bytes, void* stream,
                                  const kpool_options* options);

/*
 * Attention around the selection. Three operators share one formula over
 * different sets of visible keys. For a query row with visible keys J, query
 * head h and its key head h / (q_heads / kv_heads):
 *     s[j] = scale * q[h] . k[j]
 *     out[h] = sum_J exp(s[j]) v[j] / sum_J exp(s[j]),   lse[h] = log sum_J exp(s[j])
 * A row that sees no key, or whose every visible score is -INFINITY, gets
 * out = 0 and lse = -INFINITY. What a key that a row does not see holds
 * (infinities and NaN included) does not reach that row. Scores, weights' sums
 * and outputs are kept in fp32; with bf16 inputs the weights are rounded to bf16
 * for the product with v, and out is rounded once.
 *
 * Heads: q_heads is a multiple of kv_heads, the quotient at most 128.
 * head_dim <= 256 and a multiple of 16 bytes. scale is finite and > 0.
 *
 * Workspace (256-byte aligned, kpool_attention_workspace_bytes bytes) for every
 * one of them; what the device finds wrong with cu_seqlens, prefix or row_seq
 * is recorded there as KPOOL_ERR_INVALID_ARG (kpool_last_device_error): a
 * sequence or row with an out-of-range prefix or sequence id gets out = 0 and
 * lse = -INFINITY; with malformed cumulative lengths the outputs' values are
 * unspecified, and nothing outside the given arrays is read or written.
 * The calls allocate and synchronise nothing and can be captured into a graph; the
 * same inputs give the same bits. out and out_lse overlap no input.
 */

/* A [tokens, heads, head_dim] tensor on the device: element (t, h, c) is at
 * data + t * token_stride + h * head_stride + c (strides in elements, positive).
 * data and both strides are multiples of 16 bytes, so a cache may keep its heads
 * apart ([heads, tokens, head_dim]) or lie beside another tensor in one row. */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} kpool_heads;

typedef struct {
  int32_t q_heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t dtype;    /* a kpool_dtype: q, k, v and out */
  float scale;
  int32_t reserved; /* must be zero */
} kpool_attention_shape;

/* Workspace size for up to q_rows query rows of up to num_seqs sequences, for any of the three
 * calls; 0 for shapes or sizes that they refuse as KPOOL_ERR_INVALID_ARG. bf16 at head_dim 64 or
 * 128: partial results of up to 41 MB, and the bits of a prompt's selection (q_rows^2 / 8 bytes, at
 * most 128 MiB; longer prompts do without them). */
size_t kpool_attention_workspace_bytes(int64_t q_rows, int32_t num_seqs, const kpool_attention_shape* shape);

/*
 * Causal attention of a packed batch: sequence b's query rows
 * [cu_q[b], cu_q[b+1]) are the last ones of its key tokens [cu_k[b], cu_k[b+1]):
 * row i of nq sees the keys j <= i + (nk - nq). Equal lengths are a whole prompt; more
 * keys than rows a later chunk of one (or, with one row, a decode step); with
 * fewer keys than rows the first rows see nothing.
 *   q, out      [q_rows, q_heads, head_dim];  k, v  [k_tokens, kv_heads, head_dim]
 *   cu_q, cu_k  [num_seqs + 1] int32 (device), from 0 to q_rows / k_tokens
 *   out_lse     [q_rows, q_heads] fp32 or NULL
 *   options     NULL, or a score_kernel (KPOOL_SCORE_TC: bf16, head_dim 64 or 128) with
 *               every other field zero. (With no key token at all the CUDA-core kernel
 *               writes the empty rows, whatever is asked for.)
 */
kpool_status kpool_attention_prompt(const kpool_heads* q, const kpool_heads* k, const kpool_heads* v,
                                    const int32_t* cu_q, const int32_t* cu_k, int32_t num_seqs, int64_t q_rows,
                                    int64_t k_tokens, const kpool_attention_shape* shape, const kpool_heads* out,
                                    float* out_lse, void* workspace, size_t workspace_bytes, void* stream,
                                    const kpool_options* options);

/*
 * Attention of drafted tokens over a cache. Sequence b owns the cache tokens
 * [cu_k[b], cu_k[b+1]), holds prefix[b] committed keys and, right after them, the
 * keys of its n = cu_q[b+1] - cu_q[b] drafted nodes (prefix[b] + n must fit). Node i
 * (query row cu_q[b] + i) sees every committed key and the nodes its mask names:
 *   mask   [q_rows, mask_words] int32 (device): bit j % 32 of word j / 32 of a
 *          row is set when that row sees node j of its sequence (its ancestors and
 *          itself); bits at n and beyond are ignored, nodes past 32 * mask_words
 *          are seen by no row.
 *          NULL (mask_words = 0): a chain, node i sees the nodes j <= i; with one
 *          node per sequence that is an ordinary decode step.
 * The cache beyond prefix[b] + n is not read into any result. Other arguments as above.
 */
kpool_status kpool_attention_tree(const kpool_heads* q, const kpool_heads* k, const kpool_heads* v,
                                  const int32_t* cu_q, const int32_t* cu_k, const int32_t* prefix,
                                  const int32_t* mask, int32_t mask_words, int32_t num_seqs, int64_t q_rows,
                                  int64_t k_tokens, const kpool_attention_shape* shape, const kpool_heads* out,
                                  float* out_lse, void* workspace, size_t workspace_bytes, void* stream,
                                  const kpool_options* options);

/*
 * Attention over selected tokens: row r sees the keys token_ids[r, 0..width) of its
 * sequence, as kpool_select / kpool_select_rows leave them (width = index_topk +
 * kpool, sequence-local ids, -1 where empty). An id outside [0, L_b) is not seen; an id
 * that appears twice counts twice. The order of the ids does not matter but for
 * rounding.
 *   token_ids  [q_rows, width] int32 (device)
 *   row_seq    [q_rows] int32 (device): the row's sequence, as for kpool_select_rows; or
 *              NULL when the query rows are the key tokens' own (q_rows = k_tokens,
 *              as for kpool_select): row r is then of the sequence that holds token r.
 *   options    NULL picks a kernel by the sizes (short lists a warp each, a prompt's rows
 *              together, else gathered); KPOOL_SCORE_TC keeps to the tcgen05 kernels, which take
 *              token strides of k and v below 2^31 elements (else KPOOL_ERR_UNSUPPORTED)
 */
kpool_status kpool_attention_selected(const kpool_heads* q, const kpool_heads* k, const kpool_heads* v,
                                      const int32_t* token_ids, int32_t width, const int32_t* row_seq,
                                      const int32_t* cu_k, int32_t num_seqs, int64_t q_rows, int64_t k_tokens,
                                      const kpool_attention_shape* shape, const kpool_heads* out, float* out_lse,
                                      void* workspace, size_t workspace_bytes, void* stream,
                                      const kpool_options* options);

/*
 * Attention over a key/value cache in pages. A pool of num_pages pages of page_size tokens each holds the caches
 * of all sequences: key j of sequence b is token j % page_size of page
 * page_table[b * max_pages + j / page_size]. Sequence b holds lengths[b] keys, and its query rows
 * [cu_q[b], cu_q[b+1]) are the last ones of them: row i of n sees the keys j <= i + lengths[b] - n, as for
 * kpool_attention_prompt. cu_q NULL: one row per sequence (q_rows = num_seqs), a decode step.
 *   k, v        [num_pages, page_size, kv_heads, head_dim], with any page, token and head strides
 *   page_table  [num_seqs, max_pages] int32 (device); entries behind a sequence's last key are not read
 *   lengths     [num_seqs] int32 (device), 0 to max_pages * page_size (which is below 2^30)
 * A page may serve several sequences. What a page holds behind a sequence's last key does not reach its rows. A
 * length out of range gives the sequence's rows 0 and -INFINITY, a page outside the pool leaves the sequence's rows
 * unspecified (nothing outside the given arrays is read); both record KPOOL_ERR_INVALID_ARG. The workspace is that of
 * the other attention calls, kpool_attention_workspace_bytes. options: as for kpool_attention_prompt.
 */
typedef struct {
  void* data;
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
} kpool_pages;

kpool_status kpool_attention_paged(const kpool_heads* q, const kpool_pages* k, const kpool_pages* v,
                                   const int32_t* page_table, int32_t max_pages, int32_t num_pages, int32_t page_size,
                                   const int32_t* lengths, const int32_t* cu_q, int32_t num_seqs, int64_t q_rows,
                                   const kpool_attention_shape* shape, const kpool_heads* out, float* out_lse,
                                   void* workspace, size_t workspace_bytes, void* stream,
                                   const kpool_options* options);

/*
 * Latent attention: keys and values of all heads come from one latent vector a token, beside a rotated part that
 * all heads share. Two forms of it, for prompts and for caches.
 */
typedef struct {
  int32_t heads;
  int32_t key_dim;     /* channels of a key without its rotated part; absorbed: of the latent vector */
  int32_t rotary_dim;  /* channels of the rotated part */
  int32_t value_dim;   /* channels of a value; absorbed: key_dim */
  int32_t dtype;       /* a kpool_dtype: of every tensor */
  float scale;
} kpool_latent_shape;

/*
 * The expanded form, for prompts: every head has keys and values of its own, projected from the latent vectors by
 * the caller, and the keys of all heads end with the same rotated channels. With [a, b] for a beside b,
 *     s[j] = scale * q[h] . [k[j, h], k_rotary[j]],  out[h] = sum_J exp(s[j]) v[j, h] / sum_J exp(s[j])
 * over the keys that kpool_attention_prompt's rows see.
 *   q          [q_rows, heads, key_dim + rotary_dim]
 *   k          [k_tokens, heads, key_dim];  v, out  [., heads, value_dim]
 *   k_rotary   [k_tokens, rotary_dim]: its head_stride is not used, but valid
 * Each part is a multiple of 16 bytes; key_dim + rotary_dim and value_dim are at most 256. options: as for
 * kpool_attention_prompt (KPOOL_SCORE_TC: bf16, 128 + 64 channels, values of 128).
 */
size_t kpool_latent_prompt_workspace_bytes(int64_t q_rows, int32_t num_seqs, const kpool_latent_shape* shape);
kpool_status kpool_attention_latent_prompt(const kpool_heads* q, const kpool_heads* k, const kpool_heads* k_rotary,
                                           const kpool_heads* v, const int32_t* cu_q, const int32_t* cu_k,
                                           int32_t num_seqs, int64_t q_rows, int64_t k_tokens,
                                           const kpool_latent_shape* shape, const kpool_heads* out, float* out_lse,
                                           void* workspace, size_t workspace_bytes, void* stream,
                                           const kpool_options* options);

/*
 * The absorbed form, for caches: the caller has multiplied the queries into the latent space, so that the cached
 * vector c of a token, latent channels first, is its key as a whole and its value in the latent channels:
 *     s[j] = scale * q[h] . c[j],  out[h] = sum_J exp(s[j]) c[j][0:key_dim] / sum_J exp(s[j])
 * (the caller projects out to the heads' values). The cache is in pages, as for kpool_attention_paged.
 *   q          [q_rows, heads, key_dim + rotary_dim];  out  [q_rows, heads, key_dim]
 *   cache      [num_pages, page_size, key_dim + rotary_dim]; head_stride is not used
 *   token_ids  NULL with width = KPOOL_WHOLE_CACHE: a row sees all lengths[b] tokens of its sequence; or
 *              [q_rows, width] int32 (device), as kpool_select / kpool_select_rows leave them: a row sees the tokens
 *              that are named (ids outside [0, lengths[b]) are not seen, an id that appears twice counts twice)
 *   row_seq    [q_rows] int32 (device): the row's sequence; NULL: row r is of sequence r (q_rows = num_seqs)
 * A row whose sequence does not exist gets 0 and -INFINITY (and KPOOL_ERR_INVALID_ARG is recorded). Each part is a
 * multiple of 16 bytes, key_dim + rotary_dim at most 1,024. options: KPOOL_SCORE_TC takes bf16, 512 + 64 channels (its
 * workspace holds partial results of up to 40 MB). out and out_lse overlap no input, here and in the calls above.
 */
#define KPOOL_WHOLE_CACHE (-1)
size_t kpool_latent_workspace_bytes(int64_t q_rows, int32_t num_seqs, const kpool_latent_shape* shape);
kpool_status kpool_attention_latent(const kpool_heads* q, const kpool_pages* cache, const int32_t* page_table,
                                    int32_t max_pages, int32_t num_pages, int32_t page_size, const int32_t* lengths,
                                    const int32_t* token_ids, int32_t width, const int32_t* row_seq, int32_t num_seqs,
                                    int64_t q_rows, const kpool_latent_shape* shape, const kpool_heads* out,
                                    float* out_lse, void* workspace, size_t workspace_bytes, void* stream,
                                    const kpool_options* options);

/*
 * Rotary positions. Channel pair (a, b) number i of a head of the token at position t becomes
 *     (a cos x - b sin x, b cos x + a sin x) * magnitude,   x = t f[i]
 * with KPOOL_ROTARY_INVERSE x = -t f[i] (which, with the same magnitude, is the gradient's way back, too). The
 * rotated channels are [offset, offset + rotary_dim) of each head; pair i is channels i and i + rotary_dim / 2 of
 * them, or with KPOOL_ROTARY_INTERLEAVED channels 2 i and 2 i + 1. The other channels are copied. Products
 * and sums are in fp32, rounded once; angles are exact to 2^-24 of a half turn at any position (by a table of
 * kpool_rotary_table, whose entries are right to a few units).
 *   in, out    [tokens, heads, head_dim], any token and head strides (multiples of the element; faster where those of
 *              q and k, their bases, head_dim and offset are all multiples of 16 bytes); out is in itself (same
 *              strides), or overlaps no input
 *   positions  [tokens] int32 (device), any value
 *   table      [rotary_dim / 2] int64 (device): f[i] in turns a token, a fraction in units of 2^-64
 * q and k (NULL: none) are two tensors of the same tokens, each with sizes of its own.
 */
#define KPOOL_ROTARY_INTERLEAVED 1
#define KPOOL_ROTARY_INVERSE 2

typedef struct {
  kpool_heads in;
  kpool_heads out;
  int32_t heads;
  int32_t head_dim;  /* at most 4,096, as heads */
  int32_t offset;
  int32_t reserved;  /* must be zero */
} kpool_rotary_part;

typedef struct {
  int32_t rotary_dim; /* even */
  int32_t dtype;      /* a kpool_dtype */
  int32_t flags;
  float magnitude;    /* finite */
} kpool_rotary_shape;

kpool_status kpool_rotary(const kpool_rotary_part* q, const kpool_rotary_part* k, const int32_t* positions,
                          const int64_t* table, int64_t tokens, const kpool_rotary_shape* shape, void* stream);

/*
 * A table for kpool_rotary, written to host memory (out: [rotary_dim / 2]): f[i] = base^(-2 i / rotary_dim) radians a
 * token, stretched for contexts longer than the model was trained on:
 *     f[i] * (keep + (1 - keep) / factor),  keep = clamp((turns - low) / (high - low), 0, 1),
 *     turns = original_length * f[i] / 2 pi
 * (pairs that turn often within the original context stay as they are, slow ones are stretched by factor);
 * original_length 0 stretches all pairs alike, factor 1 none.
 */
kpool_status kpool_rotary_table(int32_t rotary_dim, double base, double factor, double original_length, double low,
                                double high, int64_t* out);

/*
 * Synchronises `stream`, then reads the device error word the last call on this
 * workspace recorded: KPOOL_OK, KPOOL_ERR_INVALID_ARG (malformed cu_seqlens),
 * KPOOL_ERR_DEVICE_TIMEOUT (a bounded wait ran out), KPOOL_ERR_INTERNAL (a
 * bounds guard fired), or KPOOL_ERR_CUDA if the synchronisation or copy failed.
 */
kpool_status kpool_last_device_error(const void* workspace, void* stream);

/*
 * Exercises the bounded device-side wait used by the pipelined kernel: one CTA
 * waits on a barrier that nothing ever completes, gives up after
 * `spin_limit` polls, records KPOOL_ERR_DEVICE_TIMEOUT in the workspace error
 * word and returns. No fault, trap or hang is involved. Asynchronous; read the
 * result with kpool_last_device_error().
 */
kpool_status kpool_wait_timeout_selftest(void* workspace, size_t workspace_bytes, int64_t spin_limit,
                                         void* stream);

/*
 * Capacity of the library's built-in scratch array used by
 * kpool_select_static_scratch: 48 MiB, enough for one batch of about 750,000
 * tokens at kpool 4, d 128, bf16 (kpool_workspace_bytes() <= this value).
 */
#define KPOOL_STATIC_SCRATCH_BYTES ((size_t)48 << 20)

/*
 * kpool_select for callers that cannot allocate device memory. The pages have
 * no counterpart to this entry point; it exists for callers such as a plugin or
 * custom operator inside a framework that owns all device memory, or a
 * real-time path that must never pay cudaMalloc's implicit synchronisation,
 * which have no workspace to pass. It runs the same kernels as kpool_select with
 * the scratch taken from a file-scope __device__ array of
 * KPOOL_STATIC_SCRATCH_BYTES that every GPU loading the library holds until the
 * process exits. Inputs and outputs are still the caller's device buffers.
 *   - The arguments are checked as kpool_select checks them, so a shape the
 *     kernels do not implement returns KPOOL_ERR_UNSUPPORTED at any size. Only a
 *     call that passes those checks and whose kpool_workspace_bytes(...) exceeds
 *     KPOOL_STATIC_SCRATCH_BYTES returns KPOOL_ERR_WORKSPACE (split the batch),
 *     before any GPU work.
 *   - The first call on each device looks up the array's device address (with
 *     that device current) and caches it: make that first call before any
 *     stream capture.
 *   - All calls on a device share the one array, which keeps the last call's
 *     contents: calls that overlap on the GPU race and must be serialised.
 *   - It allocates nothing (no cudaMalloc/cudaFree or allocating library call).
 *   - Errors found on the device (malformed cu_seqlens, which leaves the outputs
 *     unwritten as with kpool_select; a bounded wait that ran out) land in the
 *     shared array's header: read them with
 *     kpool_static_scratch_last_device_error().
 */
kpool_status kpool_select_static_scratch(const void* q, const void* k, const float* w,
                                         const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                         int32_t heads, int32_t head_dim, kpool_dtype dtype, int32_t kpool,
                                         int32_t index_topk, float scale, int32_t* out_pool_ids,
                                         int32_t* out_token_ids, float* out_pool_scores, void* stream);

/*
 * kpool_last_device_error for kpool_select_static_scratch: synchronises `stream`,
 * then returns the device error word the last call on this device's built-in
 * scratch array recorded (KPOOL_OK, KPOOL_ERR_INVALID_ARG for malformed
 * cu_seqlens, KPOOL_ERR_DEVICE_TIMEOUT, KPOOL_ERR_INTERNAL), or KPOOL_ERR_CUDA if
 * the look-up, synchronisation or copy failed. Allocates nothing.
 */
kpool_status kpool_static_scratch_last_device_error(void* stream);

/* Static, human-readable name of a status code. */
const char* kpool_status_string(kpool_status status);

/*
 * Name of the CUDA error behind the most recent KPOOL_ERR_CUDA returned to the
 * calling host thread ("cudaSuccess" if none). Static string; never touches the GPU.
 */
const char* kpool_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* KPOOL_H_ */
