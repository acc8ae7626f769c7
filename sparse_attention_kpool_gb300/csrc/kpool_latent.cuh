// kpool_latent.cuh -- shared pieces of attention over latent vectors (kpool_attention_latent): the call's
// parameters, the tokens that a row sees and where they lie, and the launch wrappers of the kernels.
//
// A token is one vector of L + P channels for all heads: key as a whole, value in its first L channels.
//   s[j] = scale * q . c[j],  out = sum_J exp(s[j]) c[j][0:L] / sum_J exp(s[j]),  lse = log sum_J exp(s[j]).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kpool_internal.cuh"

namespace kpool {

struct LatentParams {
  const void* q;         // [R, H, L + P]
  const void* cache;     // [num_pages, page_size, L + P]
  void* out;             // [R, H, L]
  float* lse;            // [R, H] or null
  int64_t q_ts, q_hs, o_ts, o_hs, c_ps, c_ts;  // strides, elements
  const int32_t* table;    // [S, max_pages]
  const int32_t* lengths;  // [S]
  const int32_t* ids;      // [R, width]
  const int32_t* row_seq;  // [R], or null: row r is of sequence r
  int32_t max_pages, page_size, num_pages;
  int32_t width;           // -1: no ids, rows see the whole cache
  int32_t S, R, H, L, P;
  float scale;
};

// Sequence of row r and the keys that it holds; 0 keys where the call's arrays are malformed.
__device__ __forceinline__ int latent_seq(const LatentParams& p, int r, int* b) {
  *b = p.row_seq ? __ldg(p.row_seq + r) : r;
  if (*b < 0 || *b >= p.S) return 0;
  const int n = __ldg(p.lengths + *b);
  return n >= 0 && n <= int64_t(p.max_pages) * p.page_size ? n : 0;
}

__host__ __device__ __forceinline__ bool latent_listed(const LatentParams& p) { return p.width >= 0; }

// Places that a row walks: its whole cache, or its list of ids.
__device__ __forceinline__ int latent_places(const LatentParams& p, int keys) {
  return keys == 0 ? 0 : latent_listed(p) ? p.width : keys;
}

// Element offset of the token at place j of row r (sequence b of n keys); -1 where nothing is seen. *bad: the table
// names a page that the pool does not have.
__device__ __forceinline__ int64_t latent_token(const LatentParams& p, int r, int b, int n, int j, bool* bad) {
  int id = j;
  if (latent_listed(p)) id = j < p.width ? __ldg(p.ids + int64_t(r) * p.width + j) : -1;
  if (id < 0 || id >= n) return -1;
  const int in_table = id / p.page_size;
  const int page = __ldg(p.table + int64_t(b) * p.max_pages + in_table);
  if (page < 0 || page >= p.num_pages) {
    *bad = true;
    return -1;
  }
  return int64_t(page) * p.c_ps + int64_t(id - in_table * p.page_size) * p.c_ts;
}

// One warp checks the call's device arrays (beside the work, which relies on none of it).
__device__ __forceinline__ void latent_check(const LatentParams& p, WorkspaceHeader* hdr) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll 4
  for (int b = lane; b < p.S; b += 32) {
    const int n = __ldg(p.lengths + b);
    bad |= n < 0 || n > int64_t(p.max_pages) * p.page_size;
  }
  if (p.row_seq) {
#pragma unroll 8
    for (int r = lane; r < p.R; r += 32) {
      const int b = __ldg(p.row_seq + r);
      bad |= b < 0 || b >= p.S;
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0 && bad) record_error(hdr, KPOOL_ERR_INVALID_ARG);
}

// Tensor-core kernel: bf16, 512 + 64 channels.
bool latent_tc_supported(kpool_dtype dtype, int32_t latent, int32_t rotary);
size_t latent_tc_bytes(int32_t heads);  // of workspace, behind the header
cudaError_t launch_latent_tc(const LatentParams& p, char* ws, cudaStream_t stream);

// CUDA-core kernel: fp32 or bf16, up to 1,024 channels in all.
cudaError_t launch_latent_simt(const LatentParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream);

}  // namespace kpool
