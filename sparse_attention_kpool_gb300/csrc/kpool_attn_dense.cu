// kpool_attn_dense.cu -- selected-token attention of a whole prompt as masked dense attention.
//
// Gathering costs every row its own copy of its keys out of L2. Rows of a prompt share most
// of theirs: a tile of 64 rows reads each key once for all of them when it goes over all keys of its
// sequence and masks what a row did not select. That does (keys / selected) times the
// products and still wins while a sequence is not too long (attn_selected_times). The ids
// become bits, 32 keys a word, and the prompt kernel runs with them as its mask.
//
// A bit cannot say that a row names a key twice: such rows are listed and the gathering kernel
// recomputes them afterwards. The kernels of the call find the row stride of the mask (from the
// longest sequence), whether it fits, and whether no row selected a key after its own on the device:
//   init (1 CTA)          stride, enabled, causal = finite = 1, no listed rows
//   mask (a CTA per row)  bits in shared memory, then out; a listed row, a later key or an infinity or NaN
//                         among the token's values is noted (with none the dense kernel cleans no V tile)
#include <cuda_runtime.h>
#include <math.h>

#include "kpool_attn.cuh"

namespace kpool {
namespace {

__global__ void __launch_bounds__(256) dense_init_kernel(const __grid_constant__ AttnParams p, AttnDense* ctl,
                                                         int64_t capacity) {
  __shared__ int s_max;
  if (threadIdx.x == 0) s_max = 0;
  __syncthreads();
  int longest = 0;
  for (int b = threadIdx.x; b < p.S; b += blockDim.x) {
    const int lo = __ldg(p.cu_k + b), hi = __ldg(p.cu_k + b + 1);
    if (lo >= 0 && hi >= lo && hi <= p.T) longest = max(longest, hi - lo);
  }
  atomicMax(&s_max, longest);
  __syncthreads();
  if (threadIdx.x == 0) {
    const int words = (s_max + 127) / 128 * 4;
    ctl->words = words;
    ctl->enabled = int64_t(p.R) * words * 4 <= capacity;
    ctl->causal = 1;
    ctl->listed = 0;
    ctl->finite = 1;
  }
}

__global__ void __launch_bounds__(256) dense_mask_kernel(const __grid_constant__ AttnParams p, AttnDense* ctl,
                                                         uint32_t* mask, int32_t* list) {
  extern __shared__ uint32_t bits[];
  if (!ctl->enabled) return;
  const int r = blockIdx.x, words = ctl->words;
  int k0, nk;
  attn_selected_seq(p, r, &k0, &nk);
  const int own = (nk + 127) / 128 * 4, pos = r - k0;
  for (int w = threadIdx.x; w < own; w += 256) bits[w] = 0;
  __syncthreads();
  const int32_t* ids = p.ids + int64_t(r) * p.width;
  bool twice = false, later = false;
  auto put = [&](int word, uint32_t b) { twice |= (atomicOr(bits + word, b) & b) != 0; };
  // pools put neighbouring ids side by side: four ids of one word cost one atomic
  const bool wide = (reinterpret_cast<uintptr_t>(ids) & 15) == 0;
  const int quads = wide ? p.width / 4 : 0;
  for (int x = threadIdx.x; x < quads; x += 256) {
    const int4 v = __ldg(reinterpret_cast<const int4*>(ids) + x);
    const int id[4] = {v.x, v.y, v.z, v.w};
    int word = -1;
    uint32_t acc = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (id[i] < 0 || id[i] >= nk) continue;
      later |= id[i] > pos;
      const uint32_t b = 1u << (id[i] & 31);
      if ((id[i] >> 5) != word) {
        if (word >= 0) put(word, acc);
        word = id[i] >> 5;
        acc = 0;
      }
      twice |= (acc & b) != 0;
      acc |= b;
    }
    if (word >= 0) put(word, acc);
  }
  for (int x = 4 * quads + threadIdx.x; x < p.width; x += 256) {
    const int id = __ldg(ids + x);
    if (id < 0 || id >= nk) continue;
    later |= id > pos;
    put(id >> 5, 1u << (id & 31));
  }
  // The row's own values, every token's once over the grid: a bf16 exponent of all ones carries into bit 15 or 31.
  const int pieces = p.D / 8;
  bool wild = false;
  for (int x = threadIdx.x; x < p.Hkv * pieces; x += 256) {
    const int h = x / pieces, c = x - h * pieces;
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + int64_t(r) * p.v_ts +
                                                         int64_t(h) * p.v_hs + 8 * c));
    constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u;
    wild |= ((((q.x & kExp) + kOne) | ((q.y & kExp) + kOne) | ((q.z & kExp) + kOne) | ((q.w & kExp) + kOne)) &
             0x80008000u) != 0;
  }
  if (wild) ctl->finite = 0;
  const int any = __syncthreads_or((twice ? 1 : 0) | (later ? 2 : 0));  // nonzero if any thread's is
  if (any) {
    const int dup = __syncthreads_or(twice), aft = __syncthreads_or(later);
    if (threadIdx.x == 0) {
      if (dup) list[atomicAdd(&ctl->listed, 1)] = r;
      if (aft) ctl->causal = 0;
    }
  }
  uint4* out = reinterpret_cast<uint4*>(mask + int64_t(r) * words);
  for (int w = threadIdx.x; w < own / 4; w += 256) out[w] = reinterpret_cast<const uint4*>(bits)[w];
}

}  // namespace

AttnSelectedTimes attn_selected_times(const AttnParams& p, int sms) {
  // From the measured parts of either way: a gathered (row, key head) takes 3 and 1.25 for each
  // tile of 128 ids (few of them are cut into runs); a dense item (256 / G rows) 6 and 2 for each tile of its
  // keys, the kernels around it 25.
  // Measured dense / gathered: 32 / 8 heads of 128, 3,000 rows x 24 ids 114 / 684, 1,500 x 516 56 / 742,
  // 16,000 x 512 1,676 / 6,407, 100 x 32 17 / 31; 64 / 1 heads, 600 x 1,004 25 / 63, 2,000 x 128 110 / 63,
  // 3,000 x 68 182 / 89.
  const double items = double(p.R) * p.Hkv / sms, tiles = double((p.width + 127) / 128);
  const double all = items * (3.0 + 1.25 * tiles), cut = 1.2 * tiles < 8.0 ? 1.2 * tiles : 8.0;
  AttnSelectedTimes t{6.0 + (all > cut ? all : cut), INFINITY};
  if (p.row_seq != nullptr || p.width == 0 || p.S > kAttnMaxRunSeqs) return t;
  const int64_t keys = p.T / p.S;  // of a sequence, on average: a row goes over half of them
  if (int64_t(p.R) * ((keys + 127) / 128) * 16 > int64_t(attn_mask_bytes(p.R))) return t;
  t.dense = 25.0 + items * p.G / 256.0 * (6.0 + 2.0 * double(keys) / 256.0);
  return t;
}

cudaError_t launch_attn_dense_mask(const AttnParams& p, AttnDense* ctl, uint32_t* mask, int32_t* list,
                                   cudaStream_t stream) {
  const int64_t capacity = int64_t(attn_mask_bytes(p.R));
  dense_init_kernel<<<1, 256, 0, stream>>>(p, ctl, capacity);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // A mask that fits has at most capacity / R bytes a row; its rows are the T = R key tokens' own, so that is
  // at most 4 KB (2^27 bytes at 32,768 rows), which needs no higher limit.
  const int64_t row_bytes = capacity / p.R < (p.T + 127) / 128 * 16 ? capacity / p.R : (p.T + 127) / 128 * 16;
  const int smem = int(row_bytes & ~int64_t(15));
  dense_mask_kernel<<<uint32_t(p.R), 256, smem, stream>>>(p, ctl, mask, list);
  return cudaGetLastError();
}

}  // namespace kpool
