// kpool_attn_simt.cu -- the attention operators on the CUDA cores: fp32 inputs at fp32
// precision, and the head sizes the tensor-core kernels do not take.
//
// One CTA holds 16 (query row, head) pairs that share a key head and walks the keys in
// blocks of 32 with the running maximum and sum of a softmax (one pass over K and V, nothing
// written but the result). Groups of 4 warps (four groups, two for heads above 128) take every
// fourth (second) block and add up at the end: the calls that come here are small, and one
// group alone waits out the latency of each block in turn (60 against 31 us for 345 rows of 8
// heads of 64). A lane scores one key for its warp's four rows, so a 16-byte read of K from
// shared memory feeds 16 multiply-adds; for the second product a lane owns 4 (or 8) channels and
// reads V the same way. K rows are padded by 16 bytes, which spreads the lanes' 16-byte reads
// over all banks.
#include <cuda_bf16.h>
#include <math.h>

#include "kpool_attn.cuh"

namespace kpool {
namespace {

constexpr int kVRows = 16;        // (row, head) pairs per CTA
constexpr int kPerWarp = 4;
constexpr int kGroupThreads = 128;
constexpr int kKeys = 32;         // keys per block: one per lane
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.sync %0, %1;" ::"r"(group + 1), "n"(kGroupThreads) : "memory");
}

// Shared memory, in floats: Q, then each group's K and V block; the groups' results overlay the blocks.
inline __host__ __device__ int group_floats(int D, int Dv) { return kKeys * (D + Dv + 4 + 4 * kPerWarp); }

// Channels of v and the result.
template <class P>
__host__ __device__ __forceinline__ int value_channels(const P& p) {
  if constexpr (kSharedKeys<P>) return p.Dv;
  else return p.D;
}

template <typename E, int kGroups, class P>
__global__ void __launch_bounds__(kGroupThreads* kGroups, kGroups == 4 ? 2 : 1)
    attn_simt_kernel(const __grid_constant__ P p, int gt, int tt, WorkspaceHeader* hdr) {
  constexpr int kH = kGroups == 4 ? 1 : 2;  // 128-channel parts of a head
  extern __shared__ __align__(16) float smem[];
  const int D = p.D, Dv = value_channels(p), ldk = D + 4;
  const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x % kGroupThreads;
  float* s_q = smem;                                        // [kVRows][D]
  float* s_k = s_q + kVRows * D + group * group_floats(D, Dv);  // [kKeys][D + 4]
  float* s_v = s_k + kKeys * ldk;                               // [kKeys][Dv]
  float* s_p = s_v + kKeys * Dv;                                // [4 warps][kKeys][kPerWarp]
  const int lane = tid & 31, warp = tid >> 5;
  const bool checks = blockIdx.x == 0 && blockIdx.y == 0;
  if (checks && threadIdx.x == 0) attn_clear_error(hdr);

  // the CTA's rows: tokens [i0, i1) of a sequence x heads [g0, g0 + gt) of key head hk
  const int gb_n = (p.G + gt - 1) / gt;
  const int hk = blockIdx.y / gb_n, g0 = (blockIdx.y % gb_n) * gt;
  AttnSeq sq{};
  int i0, i1, end;
  const bool selected = p.mode == kAttnSelected;
  const int32_t* ids = nullptr;
  if (selected) {
    const int r = blockIdx.x;
    attn_selected_seq(p, r, &sq.k0, &sq.nk);
    sq.q0 = 0;
    i0 = r;
    i1 = r + 1;
    ids = p.ids + int64_t(r) * p.width;
    end = sq.nk > 0 ? p.width : 0;
  } else {
    const int b = attn_tile_seq<false>(p, blockIdx.x, tt);
    sq = attn_seq(p, b);
    i0 = attn_tile_token<false>(p, b, blockIdx.x, tt);
    if (i0 < 0 || i0 >= sq.nq) {
      __syncwarp();
      if (checks && threadIdx.x < 32) attn_check(p, hdr);
      return;
    }
    i1 = min(i0 + tt, sq.nq);
    end = attn_keys_end(p, sq, i1);
  }

  const E* q = static_cast<const E*>(p.q);
  const E* kk = static_cast<const E*>(p.k) + int64_t(hk) * p.k_hs;
  const E* vv = static_cast<const E*>(p.v) + int64_t(hk) * p.v_hs;
  const int chunks = D / 4, pieces = max(D, Dv) / 4;
  bool bad_page = false;
  for (int x = threadIdx.x; x < kVRows * chunks; x += kGroupThreads * kGroups) {
    const int r = x / chunks, c = x % chunks, i = i0 + r / gt, g = g0 + r % gt;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r / gt < tt && i < i1 && g < p.G)
      f = load4(q + int64_t(sq.q0 + i) * p.q_ts + int64_t(hk * p.G + g) * p.q_hs + 4 * c);
    store4(s_q + r * D + 4 * c, f);
  }

  const float c2 = p.scale * kLog2e;
  float m[kPerWarp], l[kPerWarp];
  float4 o[kPerWarp][kH];
  int tok[kPerWarp];  // the warp's rows: token index, or -1 where the slot holds no row
#pragma unroll
  for (int r = 0; r < kPerWarp; ++r) {
    const int vr = warp * kPerWarp + r;
    const int i = i0 + vr / gt;
    tok[r] = (vr / gt < tt && i < i1 && g0 + vr % gt < p.G) ? i : -1;
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int h = 0; h < kH; ++h) o[r][h] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  __syncthreads();
  for (int j0 = group * kKeys; j0 < end; j0 += kGroups * kKeys) {
    group_sync(group);
    // two pieces of K and V in flight per thread; piece x is channels 4 (x % pieces).. of key x / pieces
    for (int x0 = tid; x0 < kKeys * pieces; x0 += 2 * kGroupThreads) {
      float4 a[2], b[2];
      int at[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int x = x0 + y * kGroupThreads, jj = x / pieces, c = 4 * (x - jj * pieces);
        at[y] = x < kKeys * pieces ? jj * 1024 + c : -1;
        a[y] = b[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (at[y] < 0 || j0 + jj >= end) continue;
        const int id = selected ? __ldg(ids + j0 + jj) : j0 + jj;
        if (id < 0 || id >= sq.nk) continue;
        if constexpr (kPagedKeys<P>) {  // a page that the pool does not have reads as zeros
          const int page = attn_page(p, sq.k0, id, &bad_page), in = id % p.page_size;
          if (page < 0) continue;
          a[y] = load4(kk + int64_t(page) * p.k_ps + in * p.k_ts + c);
          b[y] = load4(vv + int64_t(page) * p.v_ps + in * p.v_ts + c);
        } else if constexpr (kSharedKeys<P>) {
          const int64_t t = int64_t(sq.k0) + id;
          if (c < p.Dn) a[y] = load4(kk + t * p.k_ts + c);
          else if (c < D) a[y] = load4(static_cast<const E*>(p.kr) + t * p.kr_ts + (c - p.Dn));
          if (c < Dv) b[y] = load4(vv + t * p.v_ts + c);
        } else {
          const int64_t t = int64_t(sq.k0) + id;
          a[y] = load4(kk + t * p.k_ts + c);
          b[y] = load4(vv + t * p.v_ts + c);
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (at[y] < 0) continue;
        const int jj = at[y] >> 10, c = at[y] & 1023;
        if (!kSharedKeys<P> || c < D) store4(s_k + jj * ldk + c, a[y]);
        if (!kSharedKeys<P> || c < Dv) store4(s_v + jj * Dv + c, b[y]);
      }
    }
    group_sync(group);

    float s[kPerWarp] = {0.f, 0.f, 0.f, 0.f};
    const float* kr = s_k + lane * ldk;
    const float* qr = s_q + warp * kPerWarp * D;
    for (int c = 0; c < D; c += 4) {
      const float4 a = load4(kr + c);
#pragma unroll
      for (int r = 0; r < kPerWarp; ++r) {
        const float4 b = load4(qr + r * D + c);
        s[r] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s[r]))));
      }
    }
    const int j = j0 + lane;
    bool in = j < end;
    if (selected && in) {
      const int id = __ldg(ids + j);
      in = id >= 0 && id < sq.nk;
    }
    unsigned seen[kPerWarp];
    float pr[kPerWarp];
#pragma unroll
    for (int r = 0; r < kPerWarp; ++r) {
      const bool see = tok[r] >= 0 && in && (selected || attn_sees(p, sq, tok[r], j));
      seen[r] = __ballot_sync(0xffffffffu, see);
      const float x = see ? s[r] * c2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      mx = fmaxf(mx, m[r]);
      const float base = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: every weight below is exp2(-inf) = 0
      const float f = exp2f(m[r] - base);
      pr[r] = exp2f(x - base);
      float sum = pr[r];
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      l[r] = fmaf(l[r], f, sum);
      m[r] = mx;
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        o[r][h].x *= f;
        o[r][h].y *= f;
        o[r][h].z *= f;
        o[r][h].w *= f;
      }
    }
    // the rows' weights key by key: one 16-byte read gives a key's four
    float4* pw = reinterpret_cast<float4*>(s_p) + warp * kKeys;
    __syncwarp();
    pw[lane] = make_float4(pr[0], pr[1], pr[2], pr[3]);
    __syncwarp();
    const int n = min(kKeys, end - j0);
    const bool all = (seen[0] & seen[1] & seen[2] & seen[3]) == 0xffffffffu;
    auto add = [&](int jj, bool masked) {
      const float4 w = pw[jj];
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const int c = h * 128 + lane * 4;
        if (c >= Dv) break;
        const float4 b = load4(s_v + jj * Dv + c);
#pragma unroll
        for (int r = 0; r < kPerWarp; ++r) {
          const float x = r == 0 ? w.x : r == 1 ? w.y : r == 2 ? w.z : w.w;
          // a key the row does not see adds nothing, whatever its value holds
          if (masked && !((seen[r] >> jj) & 1u)) continue;
          o[r][h].x = fmaf(x, b.x, o[r][h].x);
          o[r][h].y = fmaf(x, b.y, o[r][h].y);
          o[r][h].z = fmaf(x, b.z, o[r][h].z);
          o[r][h].w = fmaf(x, b.w, o[r][h].w);
        }
      }
    };
    if (all) {
#pragma unroll 4
      for (int jj = 0; jj < kKeys; ++jj) add(jj, false);
    } else {
#pragma unroll 2
      for (int jj = 0; jj < n; ++jj) add(jj, true);
    }
  }

  // the groups' results: [group][kVRows][Dv] sums, then [group][kVRows] (m, l); group g finishes row g of each warp
  __syncthreads();
  float* s_o = smem + kVRows * D;
  float2* s_ml = reinterpret_cast<float2*>(s_o + kGroups * kVRows * Dv);
#pragma unroll
  for (int r = 0; r < kPerWarp; ++r) {
    const int vr = group * kVRows + warp * kPerWarp + r;
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const int c = h * 128 + lane * 4;
      if (c < Dv) store4(s_o + vr * Dv + c, o[r][h]);
    }
    if (lane == 0) s_ml[vr] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  E* out = static_cast<E*>(p.out);
#pragma unroll
  for (int r = 0; r < kPerWarp; ++r) {
    if (tok[r] < 0 || r % kGroups != group) continue;
    const int vr = warp * kPerWarp + r;
    m[r] = -INFINITY;
    for (int g = 0; g < kGroups; ++g) m[r] = fmaxf(m[r], s_ml[g * kVRows + vr].x);
    const float base = m[r] == -INFINITY ? 0.f : m[r];
    l[r] = 0.f;
#pragma unroll
    for (int h = 0; h < kH; ++h) o[r][h] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < kGroups; ++g) {
      const float2 ml = s_ml[g * kVRows + vr];
      // a group without any weight adds nothing; with a NaN among its scores its sum passes on
      const float w = ml.x == -INFINITY ? 1.f : exp2f(ml.x - base);
      l[r] = fmaf(ml.y, w, l[r]);
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const int c = h * 128 + lane * 4;
        if (c >= Dv) break;
        const float4 f = load4(s_o + (g * kVRows + vr) * Dv + c);
        o[r][h].x = fmaf(f.x, w, o[r][h].x);
        o[r][h].y = fmaf(f.y, w, o[r][h].y);
        o[r][h].z = fmaf(f.z, w, o[r][h].z);
        o[r][h].w = fmaf(f.w, w, o[r][h].w);
      }
    }
    const int64_t row = sq.q0 + tok[r];
    const int head = hk * p.G + g0 + (warp * kPerWarp + r) % gt;
    const bool none = m[r] == -INFINITY && l[r] == 0.f;  // (a NaN score leaves l NaN: not empty)
    const float inv = none ? 0.f : 1.f / l[r];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const int c = h * 128 + lane * 4;
      if (c >= Dv) break;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!none) f = make_float4(o[r][h].x * inv, o[r][h].y * inv, o[r][h].z * inv, o[r][h].w * inv);
      store4(out + row * p.o_ts + int64_t(head) * p.o_hs + c, f);
    }
    if (lane == 0 && p.lse) p.lse[row * p.Hq + head] = none ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
  }
  if (bad_page) record_error(hdr, KPOOL_ERR_INVALID_ARG);
  __syncwarp();
  if (checks && threadIdx.x < 32) attn_check(p, hdr);
}

template <typename E, int kGroups, class P>
cudaError_t launch(const P& p, const dim3& grid, int gt, int tt, WorkspaceHeader* hdr, cudaStream_t stream) {
  auto bytes = [](int D, int Dv) {
    return sizeof(float) * (size_t(kVRows) * D + size_t(kGroups) * group_floats(D, Dv));
  };
  auto kernel = attn_simt_kernel<E, kGroups, P>;
  static std::atomic<uint64_t> ready{0};
  const size_t most = bytes(kSharedKeys<P> || kGroups == 2 ? 256 : 128, kGroups == 4 ? 128 : 256);
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kernel), most, &ready);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kGroupThreads * kGroups, bytes(p.D, value_channels(p)), stream>>>(p, gt, tt, hdr);
  return cudaGetLastError();
}

template <class P>
cudaError_t launch_family(const P& p, kpool_dtype dtype, char* ws, cudaStream_t stream) {
  // heads of a group share the CTA's key blocks; what is left of the 16 slots takes more tokens
  const int gt = p.G < kVRows ? p.G : kVRows;
  const int tt = p.mode == kAttnSelected ? 1 : kVRows / gt;
  const int64_t tiles = p.mode == kAttnSelected ? p.R : attn_tiles<false>(p.R, p.S, tt);
  const dim3 grid(uint32_t(tiles), uint32_t(p.Hkv * ((p.G + gt - 1) / gt)));
  WorkspaceHeader* hdr = reinterpret_cast<WorkspaceHeader*>(ws);
  const bool narrow = value_channels(p) <= 128;
  if (dtype == KPOOL_BF16)
    return narrow ? launch<__nv_bfloat16, 4>(p, grid, gt, tt, hdr, stream)
                  : launch<__nv_bfloat16, 2>(p, grid, gt, tt, hdr, stream);
  return narrow ? launch<float, 4>(p, grid, gt, tt, hdr, stream) : launch<float, 2>(p, grid, gt, tt, hdr, stream);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream) {
  return launch_family(p, dtype, ws, stream);
}
cudaError_t launch_attn_simt(const AttnPagedParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream) {
  return launch_family(p, dtype, ws, stream);
}
cudaError_t launch_attn_simt(const AttnSharedParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream) {
  return launch_family(p, dtype, ws, stream);
}

}  // namespace kpool
