// kpool_tmap.cu -- tensor maps (TMA descriptors) for the bf16 operands of the
// tensor-core kernels: a [rows, 128] row-major bf16 matrix read in boxes of 64
// columns x box_rows rows with 128-byte swizzle, the shared-memory layout the MMA
// operand descriptors (kpool_ptx.cuh, smem_desc_kmajor_sw128) describe.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kpool_internal.cuh"

namespace kpool {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once through the runtime (no link against libcuda).
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// The encoder wants the device's context on the calling thread, which a thread that has made no runtime call of its own
// that needs one does not have yet: a failed call is made once more behind cudaSetDevice, which puts it there.
template <typename... Args>
bool encode(EncodeTiledFn fn, Args... args) {
  if (fn(args...) == CUDA_SUCCESS) return true;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
  return fn(args...) == CUDA_SUCCESS;
}

}  // namespace

bool make_tmap_bf16_k128(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {cuuint64_t(128), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(128) * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(fn, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

bool make_tmap_bf16_heads(CUtensorMap* map, const void* base, uint64_t tokens, uint64_t heads, uint64_t dim,
                          int64_t token_stride, int64_t head_stride, uint32_t box_tokens, uint32_t box_heads) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {dim, heads, tokens};
  const cuuint64_t strides[2] = {cuuint64_t(head_stride) * 2, cuuint64_t(token_stride) * 2};
  const cuuint32_t box[3] = {64, box_heads, box_tokens};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(fn, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

bool make_tmap_bf16_pages(CUtensorMap* map, const void* base, uint64_t pages, uint64_t page_size, uint64_t heads,
                          uint64_t dim, int64_t page_stride, int64_t token_stride, int64_t head_stride,
                          uint32_t box_tokens) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {dim, heads, page_size, pages};
  const cuuint64_t strides[3] = {cuuint64_t(head_stride) * 2, cuuint64_t(token_stride) * 2, cuuint64_t(page_stride) * 2};
  const cuuint32_t box[4] = {64, 1, box_tokens, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(fn, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace kpool
