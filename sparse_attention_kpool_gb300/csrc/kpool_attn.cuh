// kpool_attn.cuh -- shared pieces of the attention entry points: the call's
// parameters, which keys a row sees, the row tiles of a packed batch, and the
// launch wrappers of the kernel families.
//
// All three operators are one formula over different sets of visible keys:
//   s[j] = scale * q . k[j],  out = sum_J exp(s[j]) v[j] / sum_J exp(s[j]),
//   lse = log sum_J exp(s[j]);  no visible key: out = 0, lse = -inf.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kpool_internal.cuh"

namespace kpool {

enum AttnMode { kAttnPrompt = 0, kAttnTree = 1, kAttnSelected = 2 };

// A prompt's selection as masked dense attention (kpool_attn_dense.cu): written on the device by
// the call's first kernels.
struct AttnDense {
  int32_t words;     // 32-bit words of a row of the mask, a multiple of 4
  int32_t enabled;   // the mask fits: the dense kernel works, the gathering one only on the listed rows
  int32_t causal;    // no row selected a key after its own
  int32_t listed;    // rows that name a key twice
  int32_t finite;    // v holds no infinity or NaN
};

struct AttnParams {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;                                // [R, Hq] or null
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;  // token / head strides, elements
  const int32_t* cu_q;                       // [S + 1] query rows (prompt, tree)
  const int32_t* cu_k;                       // [S + 1] key tokens
  const int32_t* prefix;                     // [S] committed keys (tree)
  const int32_t* mask;                       // [R, mask_words] or null (tree)
  const int32_t* ids;                        // [R, width] (selected)
  const int32_t* row_seq;                    // [R] or null (selected)
  int32_t mask_words, width;
  const AttnDense* dense;                    // null, or what the dense form of a selection goes by
  const int32_t* list;                       // with dense, gathering: the listed rows
  int32_t S, R;
  int64_t T;
  int32_t Hq, Hkv, G, D;
  float scale;
  AttnMode mode;
};

// Keys in pages (prompt): key j of sequence b is token j % page_size of page table[b * max_pages + j / page_size]; k and
// v are the pages, with these strides between them. cu_q may be null: a row per sequence.
struct AttnPagedParams : AttnParams {
  const int32_t* table;                      // [S, max_pages]
  const int32_t* lengths;                    // [S] keys of a sequence
  int32_t max_pages, page_size, num_pages;
  int64_t k_ps, v_ps;
};

// Keys whose last channels are shared by all heads (prompt): D = Dn + those of kr, and values of Dv channels.
struct AttnSharedParams : AttnParams {
  const void* kr;                            // [T, D - Dn]
  int64_t kr_ts;
  int32_t Dn, Dv;
};

template <class P>
constexpr bool kPagedKeys = std::is_same<P, AttnPagedParams>::value;
template <class P>
constexpr bool kSharedKeys = std::is_same<P, AttnSharedParams>::value;

// Query rows, keys and committed prefix of one sequence, clipped so that nothing
// read through them leaves the call's arrays whatever the arrays hold. `ok` is
// false when the sequence's entries are malformed: its rows then get zeros.
struct AttnSeq {
  int32_t q0, nq;     // first query row and their number
  int32_t k0, nk;     // first key token (pages: the sequence itself) and the keys that exist for some row
  int32_t prefix;     // row i sees keys < prefix (+ i + 1 when causal); may be negative (prompt)
  bool ok;
};

// First query row of sequence b (b <= S).
template <class P>
__host__ __device__ __forceinline__ int attn_q0(const P& p, int b) {
  if constexpr (kPagedKeys<P>)
    if (p.cu_q == nullptr) return b;
#ifdef __CUDA_ARCH__
  return __ldg(p.cu_q + b);
#else
  return p.cu_q[b];
#endif
}

// Keys that a sequence's pages can hold.
__host__ __device__ __forceinline__ int64_t attn_page_keys(const AttnPagedParams& p) {
  return int64_t(p.max_pages) * p.page_size;
}

template <class P>
__device__ __forceinline__ AttnSeq attn_seq(const P& p, int b) {
  AttnSeq s;
  s.q0 = attn_q0(p, b);
  const int64_t q1 = attn_q0(p, b + 1);
  int64_t k1;
  if constexpr (kPagedKeys<P>) {
    s.k0 = b;
    const int n = __ldg(p.lengths + b);
    k1 = int64_t(b) + n;
    s.ok = n >= 0 && n <= attn_page_keys(p);
  } else {
    s.k0 = __ldg(p.cu_k + b);
    k1 = __ldg(p.cu_k + b + 1);
    s.ok = s.k0 >= 0 && k1 >= s.k0 && k1 <= p.T;
  }
  s.ok = s.ok && s.q0 >= 0 && q1 >= s.q0 && q1 <= p.R;
  if (!s.ok) {
    // rows inside the call's range still get their zeros
    s.q0 = max(0, min(s.q0, p.R));
    s.nq = int32_t(max(int64_t(0), min(q1, int64_t(p.R)) - s.q0));
    s.k0 = s.nk = s.prefix = 0;
    return s;
  }
  s.nq = int32_t(q1 - s.q0);
  const int64_t extent = k1 - s.k0;
  if (p.mode == kAttnTree) {
    const int64_t pre = p.prefix ? __ldg(p.prefix + b) : 0;
    if (pre < 0 || pre + s.nq > extent) {
      s.ok = false;
      s.nk = s.prefix = 0;
      return s;
    }
    s.prefix = int32_t(pre);
    s.nk = s.prefix + s.nq;
  } else {
    s.prefix = int32_t(extent - s.nq);
    s.nk = int32_t(extent);
  }
  return s;
}

__device__ __forceinline__ int attn_mask_words(const AttnParams& p) {
  return p.dense ? __ldg(&p.dense->words) : p.mask_words;
}

// No row sees keys after prefix + its own index (without a mask, or by what the mask was made from).
__device__ __forceinline__ bool attn_causal(const AttnParams& p) {
  return p.mask == nullptr || (p.dense && __ldg(&p.dense->causal));
}

// Does row i of the sequence (global query row q0 + i) see key j? (prompt, tree; j < nk)
__device__ __forceinline__ bool attn_sees(const AttnParams& p, const AttnSeq& s, int i, int j) {
  const int slot = j - s.prefix;
  if (p.mask == nullptr) return slot <= i;
  if (slot < 0) return true;
  const int words = attn_mask_words(p);
  if (slot >= 32 * words || slot >= s.nq) return false;
  return (uint32_t(__ldg(p.mask + int64_t(s.q0 + i) * words + (slot >> 5))) >> (slot & 31)) & 1u;
}

// Keys [0, end) hold every key that some row before i1 sees.
__device__ __forceinline__ int attn_keys_end(const AttnParams& p, const AttnSeq& s, int i1) {
  if (!s.ok || s.nk == 0) return 0;
  if (!attn_causal(p)) return s.nk;
  return int(max(int64_t(0), min(int64_t(s.nk), int64_t(s.prefix) + i1)));
}

// A packed batch is cut into tiles of `tt` query rows that do not cross sequences.
// Sequence b's tiles are numbered from cu_q[b] / tt + b: a sequence of n rows has
// ceil(n / tt) of them, at most floor(cu[b+1]/tt) - floor(cu[b]/tt) + 1, so the ranges
// do not overlap, R / tt + S numbers cover all, and a binary search finds a number's
// sequence without any scan or planning kernel; numbers without a tile are skipped.
// A form that takes one row of every sequence (kRows) numbers its tiles by the sequences themselves, R = S of them.
// (Not every tile of one token is such a form's: groups of 65 to 128 heads leave row tiles of one token in any call.)
template <bool kRows>
inline int64_t attn_tiles(int64_t R, int64_t S, int64_t tt) { return kRows ? R : R / tt + S; }

template <class P>
__host__ __device__ __forceinline__ int attn_seq_of_tile(const P& p, int tile, int tt) {
  int lo = 0, hi = p.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (attn_q0(p, mid) / tt + mid <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Sequence of tile number `tile` < attn_tiles, and its first token there; the number has no tile where that is negative or
// not one of the sequence's.
template <bool kRows, class P>
__host__ __device__ __forceinline__ int attn_tile_seq(const P& p, int tile, int tt) {
  return kRows ? tile : attn_seq_of_tile(p, tile, tt);
}
template <bool kRows, class P>
__host__ __device__ __forceinline__ int attn_tile_token(const P& p, int b, int tile, int tt) {
  return kRows ? 0 : (tile - (attn_q0(p, b) / tt + b)) * tt;
}

// The header's error word, first and last: one thread clears it at the start of the call, and one warp
// checks the device arrays of the whole call (beside the work, which relies on none of it).
__device__ __forceinline__ void attn_clear_error(WorkspaceHeader* hdr) { hdr->error = KPOOL_OK; }

template <class P>
__device__ __forceinline__ void attn_check(const P& p, WorkspaceHeader* hdr) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int b = lane; b <= p.S; b += 32) {
    int k = 0;
    if constexpr (kPagedKeys<P>) {
      if (b < p.S) {
        const int n = __ldg(p.lengths + b);
        if (n < 0 || n > attn_page_keys(p)) bad = true;
      }
      if (!p.cu_q) continue;
    } else {
      k = __ldg(p.cu_k + b);
      if (b == 0 ? k != 0 : k < __ldg(p.cu_k + b - 1)) bad = true;
      if (b == p.S && k != p.T) bad = true;
    }
    if (p.mode == kAttnSelected) continue;
    const int q = __ldg(p.cu_q + b);
    if (b == 0 ? q != 0 : q < __ldg(p.cu_q + b - 1)) bad = true;
    if (b == p.S && q != p.R) bad = true;
    if (p.mode == kAttnTree && b < p.S && p.prefix) {
      const int64_t pre = __ldg(p.prefix + b);
      const int64_t rows = int64_t(__ldg(p.cu_q + b + 1)) - q, extent = int64_t(__ldg(p.cu_k + b + 1)) - k;
      if (pre < 0 || pre + rows > extent) bad = true;
    }
  }
  if (p.mode == kAttnSelected && p.row_seq != nullptr) {
#pragma unroll 8
    for (int r = lane; r < p.R; r += 32) {
      const int b = __ldg(p.row_seq + r);
      bad |= b < 0 || b >= p.S;
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0 && bad) record_error(hdr, KPOOL_ERR_INVALID_ARG);
}

// The page that key j of sequence b lies in; -1 (and *bad) where the table names none of the pool's.
__device__ __forceinline__ int attn_page(const AttnPagedParams& p, int b, int j, bool* bad) {
  const int page = __ldg(p.table + int64_t(b) * p.max_pages + j / p.page_size);
  if (page >= 0 && page < p.num_pages) return page;
  *bad = true;
  return -1;
}

// Key tokens of selected row r: first token and number (0 when the row has no valid sequence).
__device__ __forceinline__ void attn_selected_seq(const AttnParams& p, int r, int* k0, int* nk) {
  int b = p.row_seq ? __ldg(p.row_seq + r) : seq_of_row(p.cu_k, p.S, r);
  *k0 = *nk = 0;
  if (b < 0 || b >= p.S) return;
  const int lo = __ldg(p.cu_k + b), hi = __ldg(p.cu_k + b + 1);
  if (lo < 0 || hi < lo || hi > p.T) return;
  *k0 = lo;
  *nk = hi - lo;
}

// The persistent tensor-core form: its runs (CTAs) and the sequences it takes. Beside it, whole row tiles per CTA
// (kpool_attn_tc.cu, launch): up to kAttnWholeKeys keys; kAttnLikeKeys keys a sequence at one or two row tiles
// per SM; from kAttnDirectItems row tiles per SM and kAttnDirectKeys keys a sequence on. (Over pages the host knows no
// lengths: the first by what a table can hold, the last by the device.)
constexpr int kAttnMaxRuns = 152;
constexpr int kAttnMaxRunSeqs = 8192;
constexpr int kAttnWholeKeys = 1024;
constexpr int kAttnLikeKeys = 2600;
constexpr int kAttnDirectItems = 6;
constexpr int kAttnDirectKeys = 8192;
constexpr int kAttnJoinBytes = 64;   // per run: what the join of the rows before it needs
constexpr int kAttnTileRows = 128;   // MMA rows: row tile t's tokens fill the first 128 / G * G rows from 128 t on
// Rows of one partial result of a call of R query rows: up to the last row that the form's row tiles (one or two) give
// a token, so with two of them the gap that a G which does not divide 128 leaves before row 128 is counted.
inline int attn_slot_rows(int64_t R, int32_t G, int row_tiles) {
  const int64_t tt = kAttnTileRows / G;
  int64_t rows = (R < tt ? R : tt) * G;
  if (row_tiles == 2 && R > tt) rows = kAttnTileRows + (R < 2 * tt ? R - tt : tt) * G;
  return int((rows + 3) & ~int64_t(3));  // keeps every partial result 16-byte aligned
}
// AttnDense, the runs' join items and the partial results of the persistent form: two per run,
// [rows][D] fp32 and (m, l) per row.
inline size_t attn_partial_bytes(int64_t R, int32_t G, int32_t D) {
  return 256 + size_t(kAttnMaxRuns) * kAttnJoinBytes +
         size_t(2 * kAttnMaxRuns) * size_t(attn_slot_rows(R, G, 2)) * size_t(D + 2) * sizeof(float);
}

// The dense form of a selection: whether the host tries it, the bytes of its mask for R rows, and the
// kernels that fill the mask. (Longer prompts than the mask holds are gathered.)
inline size_t attn_mask_bytes(int64_t R) {
  const int64_t all = R * ((R + 127) / 128) * 16;
  return size_t(all < (int64_t(128) << 20) ? all : (int64_t(128) << 20));
}
inline size_t attn_list_bytes(int64_t R) { return (size_t(R) * 4 + 255) & ~size_t(255); }
struct AttnSelectedTimes {  // microseconds, estimated; dense is infinite where it cannot be had
  double gathered, dense;
};
AttnSelectedTimes attn_selected_times(const AttnParams& p, int sms);
cudaError_t launch_attn_dense_mask(const AttnParams& p, AttnDense* ctl, uint32_t* mask, int32_t* list,
                                   cudaStream_t stream);

// Tensor-core kernel: bf16, head_dim 64 or 128, at least one key token; over selected tokens
// also token strides of k and v that attn_gather_supported takes.
bool attn_tc_supported(kpool_dtype dtype, int32_t head_dim);
// The same for keys with a shared part: 128 + 64 channels, values of 128.
bool attn_tc_shared_supported(kpool_dtype dtype, int32_t own, int32_t shared, int32_t value);
bool attn_gather_supported(int64_t k_ts, int64_t v_ts);
cudaError_t launch_attn_tc(const AttnParams& p, char* ws, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnPagedParams& p, char* ws, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnSharedParams& p, char* ws, cudaStream_t stream);

// Selected tokens by one warp an item, in registers: what attn_tc_supported takes, any strides. Wanted where it
// beats the other two ways.
bool attn_warp_wanted(const AttnParams& p, int sms);
cudaError_t launch_attn_warp(const AttnParams& p, int sms, char* ws, cudaStream_t stream);

// CUDA-core kernel: fp32 or bf16, any head_dim <= 256 (of keys and of values).
cudaError_t launch_attn_simt(const AttnParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream);
cudaError_t launch_attn_simt(const AttnPagedParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream);
cudaError_t launch_attn_simt(const AttnSharedParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream);

}  // namespace kpool
