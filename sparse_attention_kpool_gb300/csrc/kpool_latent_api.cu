// kpool_latent_api.cu -- the C ABI of kpool_attention_latent declared in include/kpool.h: argument checks,
// workspace size and the choice of kernel. Nothing here allocates device memory or synchronises.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kpool_latent.cuh"

namespace kpool {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool shape_ok(const kpool_latent_shape* s) {
  if (s == nullptr || (s->dtype != KPOOL_BF16 && s->dtype != KPOOL_F32)) return false;
  const int64_t e = s->dtype == KPOOL_BF16 ? 2 : 4;
  for (const int32_t d : {s->key_dim, s->rotary_dim})
    if (d < 1 || (d * e) % 16 != 0) return false;
  return s->heads >= 1 && s->value_dim == s->key_dim && isfinite(s->scale) && s->scale > 0.0f;
}

bool sizes_ok(int64_t rows, int32_t seqs) {
  return rows >= 0 && rows <= INT32_MAX / 2 && seqs >= 0 && seqs <= INT32_MAX / 2 && (rows == 0 || seqs >= 1);
}

// A base and strides in multiples of 16 bytes, no stride shorter than the `dim` channels that lie there.
bool tensor_ok(const void* data, int64_t outer, int64_t inner, int64_t dim, int64_t e) {
  if (data == nullptr || !aligned(data, 16)) return false;
  for (const int64_t st : {outer, inner})
    if (st < dim || st >= (int64_t(1) << 38) || (st * e) % 16 != 0) return false;
  return true;
}

}  // namespace
}  // namespace kpool

using namespace kpool;

extern "C" {

size_t kpool_latent_workspace_bytes(int64_t q_rows, int32_t num_seqs, const kpool_latent_shape* shape) {
  if (!shape_ok(shape) || !sizes_ok(q_rows, num_seqs)) return 0;
  size_t bytes = sizeof(WorkspaceHeader);
  if (latent_tc_supported(kpool_dtype(shape->dtype), shape->key_dim, shape->rotary_dim) && shape->heads <= 4096)
    bytes += latent_tc_bytes(shape->heads);
  return bytes;
}

kpool_status kpool_attention_latent(const kpool_heads* q, const kpool_pages* cache, const int32_t* page_table,
                                    int32_t max_pages, int32_t num_pages, int32_t page_size, const int32_t* lengths,
                                    const int32_t* token_ids, int32_t width, const int32_t* row_seq, int32_t num_seqs,
                                    int64_t q_rows, const kpool_latent_shape* shape, const kpool_heads* out,
                                    float* out_lse, void* workspace, size_t workspace_bytes, void* stream_ptr,
                                    const kpool_options* options) {
  if (!shape_ok(shape) || !sizes_ok(q_rows, num_seqs)) return KPOOL_ERR_INVALID_ARG;
  if (max_pages < 0 || num_pages < 0 || page_size < 1 || int64_t(max_pages) * page_size > INT32_MAX / 2 ||
      num_pages > INT32_MAX / 2 || width < -1 || width > INT32_MAX / 2)
    return KPOOL_ERR_INVALID_ARG;
  kpool_options opt{};
  if (options) opt = *options;
  if (opt.score_kernel < KPOOL_SCORE_AUTO || opt.score_kernel > KPOOL_SCORE_SIMT || opt.max_ctas != 0 ||
      opt.stage_events != nullptr || opt.row_begin != 0 || opt.row_end != 0 || opt.flags != 0 || opt.reserved != 0)
    return KPOOL_ERR_INVALID_ARG;
  if (row_seq == nullptr && q_rows != num_seqs) return KPOOL_ERR_INVALID_ARG;
  if (token_ids == nullptr ? width > 0 : width < 0) return KPOOL_ERR_INVALID_ARG;
  const kpool_dtype dtype = kpool_dtype(shape->dtype);
  const int64_t dim = int64_t(shape->key_dim) + shape->rotary_dim, e = dtype == KPOOL_BF16 ? 2 : 4;
  if (dim > 1024 || shape->heads > 4096) return KPOOL_ERR_UNSUPPORTED;
  const bool tc_ok = latent_tc_supported(dtype, shape->key_dim, shape->rotary_dim);
  if (opt.score_kernel == KPOOL_SCORE_TC && !tc_ok) return KPOOL_ERR_UNSUPPORTED;
  if (q_rows == 0) return KPOOL_OK;
  if (q == nullptr || !tensor_ok(q->data, q->token_stride, q->head_stride, dim, e)) return KPOOL_ERR_INVALID_ARG;
  if (out == nullptr || !tensor_ok(out->data, out->token_stride, out->head_stride, shape->value_dim, e))
    return KPOOL_ERR_INVALID_ARG;
  const bool some = max_pages > 0 && num_pages > 0;  // (else there is nothing to point at)
  if (some && (cache == nullptr || !tensor_ok(cache->data, cache->page_stride, cache->token_stride, dim, e)))
    return KPOOL_ERR_INVALID_ARG;
  if (max_pages > 0 && (!page_table || !aligned(page_table, 4))) return KPOOL_ERR_INVALID_ARG;
  if (!lengths || !aligned(lengths, 4) || !aligned(token_ids, 4) || !aligned(row_seq, 4) || !aligned(out_lse, 4))
    return KPOOL_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < kpool_latent_workspace_bytes(q_rows, num_seqs, shape))
    return KPOOL_ERR_WORKSPACE;

  LatentParams p{};
  p.q = q->data;
  p.q_ts = q->token_stride;
  p.q_hs = q->head_stride;
  if (some) {
    p.cache = cache->data;
    p.c_ps = cache->page_stride;
    p.c_ts = cache->token_stride;
  }
  p.out = out->data;
  p.o_ts = out->token_stride;
  p.o_hs = out->head_stride;
  p.lse = out_lse;
  p.table = page_table;
  p.lengths = lengths;
  p.ids = token_ids;
  p.row_seq = row_seq;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.width = width;
  p.S = num_seqs;
  p.R = int32_t(q_rows);
  p.H = shape->heads;
  p.L = shape->key_dim;
  p.P = shape->rotary_dim;
  p.scale = shape->scale;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const bool tc = tc_ok && some && opt.score_kernel != KPOOL_SCORE_SIMT;
  const cudaError_t err = tc ? launch_latent_tc(p, ws, stream) : launch_latent_simt(p, dtype, ws, stream);
  return note_cuda_error(err) ? KPOOL_OK : KPOOL_ERR_CUDA;
}

}  // extern "C"
