// kpool_attn_api.cu -- the C ABI of the attention operators declared in include/kpool.h:
// argument checks, workspace size and the choice of kernel family. Nothing here
// allocates device memory or synchronises.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kpool_attn.cuh"

namespace kpool {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool shape_ok(const kpool_attention_shape* s) {
  if (s == nullptr || s->reserved != 0) return false;
  if (s->dtype != KPOOL_BF16 && s->dtype != KPOOL_F32) return false;
  if (s->q_heads < 1 || s->kv_heads < 1 || s->q_heads % s->kv_heads != 0 || s->head_dim < 1) return false;
  if ((int64_t(s->head_dim) * (s->dtype == KPOOL_BF16 ? 2 : 4)) % 16 != 0) return false;
  return isfinite(s->scale) && s->scale > 0.0f;
}

bool sizes_ok(int64_t rows, int64_t tokens, int32_t seqs) {
  return rows >= 0 && rows <= INT32_MAX / 2 && tokens >= 0 && tokens <= INT32_MAX / 2 && seqs >= 0 &&
         seqs <= INT32_MAX / 2 && (rows == 0 || seqs >= 1);
}

// Base and strides in multiples of 16 bytes, no stride shorter than a head, and byte
// strides below 2^40, the limit of a tensor map.
bool heads_ok(const kpool_heads* t, const kpool_attention_shape& s) {
  const int64_t e = s.dtype == KPOOL_BF16 ? 2 : 4;
  if (t == nullptr || t->data == nullptr || !aligned(t->data, 16)) return false;
  for (const int64_t st : {t->token_stride, t->head_stride})
    if (st < s.head_dim || st >= (int64_t(1) << 38) || (st * e) % 16 != 0) return false;
  return true;
}

kpool_status attention(AttnParams& p, const kpool_heads* q, const kpool_heads* k, const kpool_heads* v,
                       const kpool_heads* out, float* out_lse, int32_t num_seqs, int64_t q_rows, int64_t k_tokens,
                       const kpool_attention_shape* shape, void* workspace, size_t workspace_bytes, void* stream_ptr,
                       const kpool_options* options) {
  if (!shape_ok(shape) || !sizes_ok(q_rows, k_tokens, num_seqs)) return KPOOL_ERR_INVALID_ARG;
  kpool_options opt{};
  if (options) opt = *options;
  if (opt.score_kernel < KPOOL_SCORE_AUTO || opt.score_kernel > KPOOL_SCORE_SIMT || opt.max_ctas != 0 ||
      opt.stage_events != nullptr || opt.row_begin != 0 || opt.row_end != 0 || opt.flags != 0 || opt.reserved != 0)
    return KPOOL_ERR_INVALID_ARG;
  const int32_t group = shape->q_heads / shape->kv_heads;
  if (shape->head_dim > 256 || group > 128 || shape->q_heads > 4096) return KPOOL_ERR_UNSUPPORTED;
  const kpool_dtype dtype = kpool_dtype(shape->dtype);
  const bool tc_ok = attn_tc_supported(dtype, shape->head_dim);
  if (opt.score_kernel == KPOOL_SCORE_TC && !tc_ok) return KPOOL_ERR_UNSUPPORTED;
  if (q_rows == 0) return KPOOL_OK;
  if (!heads_ok(q, *shape) || !heads_ok(out, *shape)) return KPOOL_ERR_INVALID_ARG;
  // with no key token there is nothing to point at
  if (k_tokens > 0 && (!heads_ok(k, *shape) || !heads_ok(v, *shape))) return KPOOL_ERR_INVALID_ARG;
  const bool gathers = p.mode == kAttnSelected && k_tokens > 0;
  if (gathers && opt.score_kernel == KPOOL_SCORE_TC && !attn_gather_supported(k->token_stride, v->token_stride))
    return KPOOL_ERR_UNSUPPORTED;
  if (!p.cu_k || !aligned(p.cu_k, 4) || !aligned(out_lse, 4)) return KPOOL_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < kpool_attention_workspace_bytes(q_rows, num_seqs, shape))
    return KPOOL_ERR_WORKSPACE;

  p.q = q->data;
  p.q_ts = q->token_stride;
  p.q_hs = q->head_stride;
  if (k_tokens > 0) {
    p.k = k->data;
    p.k_ts = k->token_stride;
    p.k_hs = k->head_stride;
    p.v = v->data;
    p.v_ts = v->token_stride;
    p.v_hs = v->head_stride;
  }
  p.out = out->data;
  p.o_ts = out->token_stride;
  p.o_hs = out->head_stride;
  p.lse = out_lse;
  p.S = num_seqs;
  p.R = int32_t(q_rows);
  p.T = k_tokens;
  p.Hq = shape->q_heads;
  p.Hkv = shape->kv_heads;
  p.G = group;
  p.D = shape->head_dim;
  p.scale = shape->scale;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (tc_ok && k_tokens > 0 && p.mode == kAttnSelected && opt.score_kernel == KPOOL_SCORE_AUTO) {
    int sms = 0;
    if (!note_cuda_error(device_sm_count(&sms))) return KPOOL_ERR_CUDA;
    if (attn_warp_wanted(p, sms)) return note_cuda_error(launch_attn_warp(p, sms, ws, stream)) ? KPOOL_OK : KPOOL_ERR_CUDA;
  }
  const bool tc = tc_ok && k_tokens > 0 && opt.score_kernel != KPOOL_SCORE_SIMT &&
                  (!gathers || attn_gather_supported(p.k_ts, p.v_ts));
  const cudaError_t e = tc ? launch_attn_tc(p, ws, stream) : launch_attn_simt(p, dtype, ws, stream);
  return note_cuda_error(e) ? KPOOL_OK : KPOOL_ERR_CUDA;
}

}  // namespace
}  // namespace kpool

using namespace kpool;

extern "C" {

size_t kpool_attention_workspace_bytes(int64_t q_rows, int32_t num_seqs, const kpool_attention_shape* shape) {
  if (!shape_ok(shape) || !sizes_ok(q_rows, 0, num_seqs)) return 0;
  size_t bytes = sizeof(WorkspaceHeader);
  if (attn_tc_supported(kpool_dtype(shape->dtype), shape->head_dim))
    bytes += ((attn_partial_bytes(q_rows, shape->q_heads / shape->kv_heads, shape->head_dim) + 255) & ~size_t(255)) +
             attn_list_bytes(q_rows) + attn_mask_bytes(q_rows);
  return bytes;
}

kpool_status kpool_attention_prompt(const kpool_heads* q, const kpool_heads* k, const kpool_heads* v,
                                    const int32_t* cu_q, const int32_t* cu_k, int32_t num_seqs, int64_t q_rows,
                                    int64_t k_tokens, const kpool_attention_shape* shape, const kpool_heads* out,
                                    float* out_lse, void* workspace, size_t workspace_bytes, void* stream,
                                    const kpool_options* options) {
  if (q_rows > 0 && (!cu_q || !aligned(cu_q, 4))) return KPOOL_ERR_INVALID_ARG;
  AttnParams p{};
  p.mode = kAttnPrompt;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  return attention(p, q, k, v, out, out_lse, num_seqs, q_rows, k_tokens, shape, workspace, workspace_bytes, stream,
                   options);
}

kpool_status kpool_attention_tree(const kpool_heads* q, const kpool_heads* k, const kpool_heads* v,
                                  const int32_t* cu_q, const int32_t* cu_k, const int32_t* prefix,
                                  const int32_t* mask, int32_t mask_words, int32_t num_seqs, int64_t q_rows,
                                  int64_t k_tokens, const kpool_attention_shape* shape, const kpool_heads* out,
                                  float* out_lse, void* workspace, size_t workspace_bytes, void* stream,
                                  const kpool_options* options) {
  if (q_rows > 0 && (!cu_q || !aligned(cu_q, 4) || !prefix || !aligned(prefix, 4))) return KPOOL_ERR_INVALID_ARG;
  if (mask_words < 0 || mask_words > (1 << 20) || (mask != nullptr) != (mask_words > 0) || !aligned(mask, 4))
    return KPOOL_ERR_INVALID_ARG;
  AttnParams p{};
  p.mode = kAttnTree;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.prefix = prefix;
  p.mask = mask;
  p.mask_words = mask_words;
  return attention(p, q, k, v, out, out_lse, num_seqs, q_rows, k_tokens, shape, workspace, workspace_bytes, stream,
                   options);
}

kpool_status kpool_attention_selected(const kpool_heads* q, const kpool_heads* k, const kpool_heads* v,
                                      const int32_t* token_ids, int32_t width, const int32_t* row_seq,
                                      const int32_t* cu_k, int32_t num_seqs, int64_t q_rows, int64_t k_tokens,
                                      const kpool_attention_shape* shape, const kpool_heads* out, float* out_lse,
                                      void* workspace, size_t workspace_bytes, void* stream,
                                      const kpool_options* options) {
  if (width < 0 || width > INT32_MAX / 2) return KPOOL_ERR_INVALID_ARG;
  if (q_rows > 0 && width > 0 && (!token_ids || !aligned(token_ids, 4))) return KPOOL_ERR_INVALID_ARG;
  if (!aligned(row_seq, 4) || (row_seq == nullptr && q_rows != k_tokens)) return KPOOL_ERR_INVALID_ARG;
  AttnParams p{};
  p.mode = kAttnSelected;
  p.ids = token_ids;
  p.width = width;
  p.row_seq = row_seq;
  p.cu_k = cu_k;
  return attention(p, q, k, v, out, out_lse, num_seqs, q_rows, k_tokens, shape, workspace, workspace_bytes, stream,
                   options);
}

}  // extern "C"
