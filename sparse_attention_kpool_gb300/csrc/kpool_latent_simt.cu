// kpool_latent_simt.cu -- attention over latent vectors on the CUDA cores: fp32 at fp32 precision, and the
// sizes that the tensor-core kernel does not take.
//
// A CTA has up to eight heads of a row and walks the row's tokens in blocks of 32, each read once into
// shared memory for all of them (one vector is key and value), with the running maximum and sum of a
// softmax. A warp has two heads: for the scores a lane has a token, for the second product it owns every 32nd
// group of four channels. A token's row in shared memory is padded by 16 bytes, which spreads the lanes' 16-byte
// reads over all banks.
#include <cuda_bf16.h>
#include <math.h>

#include "kpool_latent.cuh"

namespace kpool {
namespace {

constexpr int kWarps = 4;
constexpr int kPerWarp = 2;              // heads of a warp
constexpr int kHeads = kWarps * kPerWarp;
constexpr int kKeys = 32;
constexpr int kMaxChannels = 1024;
constexpr int kParts = kMaxChannels / 128;  // 128-channel parts of a value
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

// Shared memory, in floats: Q, the block of tokens, the weights.
inline int smem_floats(int E) { return kHeads * E + kKeys * (E + 4) + kWarps * kKeys * kPerWarp; }

template <typename E>
__global__ void __launch_bounds__(32 * kWarps)
    latent_simt_kernel(const __grid_constant__ LatentParams p, WorkspaceHeader* hdr) {
  extern __shared__ __align__(16) float smem[];
  const int C = p.L + p.P, ld = C + 4, chunks = C / 4;
  float* s_q = smem;                    // [kHeads][C]
  float* s_c = s_q + kHeads * C;        // [kKeys][C + 4]
  float* s_p = s_c + kKeys * ld;        // [kWarps][kKeys][kPerWarp]
  __shared__ int64_t s_at[kKeys];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool checks = blockIdx.x == 0 && blockIdx.y == 0;
  if (checks && threadIdx.x == 0) hdr->error = KPOOL_OK;
  const int r = blockIdx.x, h0 = blockIdx.y * kHeads;
  int b;
  const int n = latent_seq(p, r, &b), end = latent_places(p, n);
  bool bad = false;

  const E* q = static_cast<const E*>(p.q) + int64_t(r) * p.q_ts;
  const E* cache = static_cast<const E*>(p.cache);
  for (int x = threadIdx.x; x < kHeads * chunks; x += 32 * kWarps) {
    const int h = x / chunks, c = 4 * (x - h * chunks);
    store4(s_q + h * C + c, h0 + h < p.H ? load4(q + (h0 + h) * p.q_hs + c) : make_float4(0.f, 0.f, 0.f, 0.f));
  }
  const float c2 = p.scale * kLog2e;
  float m[kPerWarp], l[kPerWarp];
  float4 o[kPerWarp][kParts];
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int x = 0; x < kParts; ++x) o[i][x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  for (int j0 = 0; j0 < end; j0 += kKeys) {
    __syncthreads();
    if (warp == 0) s_at[lane] = latent_token(p, r, b, n, j0 + lane, &bad);
    __syncthreads();
    for (int x = threadIdx.x; x < kKeys * chunks; x += 32 * kWarps) {
      const int jj = x / chunks, c = 4 * (x - jj * chunks);
      const int64_t at = s_at[jj];
      store4(s_c + jj * ld + c, at >= 0 ? load4(cache + at + c) : make_float4(0.f, 0.f, 0.f, 0.f));
    }
    __syncthreads();

    float s[kPerWarp] = {0.f, 0.f};
    const float* kr = s_c + lane * ld;
    const float* qr = s_q + warp * kPerWarp * C;
    for (int c = 0; c < C; c += 4) {
      const float4 a = load4(kr + c);
#pragma unroll
      for (int i = 0; i < kPerWarp; ++i) {
        const float4 f = load4(qr + i * C + c);
        s[i] = fmaf(a.x, f.x, fmaf(a.y, f.y, fmaf(a.z, f.z, fmaf(a.w, f.w, s[i]))));
      }
    }
    const bool see = s_at[lane] >= 0;
    const uint32_t seen = __ballot_sync(0xffffffffu, see);
    float w[kPerWarp];
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
      const float x = see ? s[i] * c2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      mx = fmaxf(mx, m[i]);
      const float base = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: every weight is exp2(-inf) = 0
      const float f = exp2f(m[i] - base);
      w[i] = exp2f(x - base);
      float sum = w[i];
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      l[i] = fmaf(l[i], f, sum);
      m[i] = mx;
#pragma unroll
      for (int x = 0; x < kParts; ++x) {
        if (x * 128 >= p.L) break;
        o[i][x].x *= f;
        o[i][x].y *= f;
        o[i][x].z *= f;
        o[i][x].w *= f;
      }
    }
    float2* pw = reinterpret_cast<float2*>(s_p) + warp * kKeys;
    __syncwarp();
    pw[lane] = make_float2(w[0], w[1]);
    __syncwarp();
#pragma unroll 1
    for (int jj = 0; jj < kKeys; ++jj) {
      if (!((seen >> jj) & 1u)) continue;  // a token that the row does not see adds nothing
      const float2 f = pw[jj];
#pragma unroll
      for (int x = 0; x < kParts; ++x) {
        const int c = x * 128 + lane * 4;
        if (x * 128 >= p.L) break;
        if (c >= p.L) continue;
        const float4 v = load4(s_c + jj * ld + c);
        o[0][x].x = fmaf(f.x, v.x, o[0][x].x);
        o[0][x].y = fmaf(f.x, v.y, o[0][x].y);
        o[0][x].z = fmaf(f.x, v.z, o[0][x].z);
        o[0][x].w = fmaf(f.x, v.w, o[0][x].w);
        o[1][x].x = fmaf(f.y, v.x, o[1][x].x);
        o[1][x].y = fmaf(f.y, v.y, o[1][x].y);
        o[1][x].z = fmaf(f.y, v.z, o[1][x].z);
        o[1][x].w = fmaf(f.y, v.w, o[1][x].w);
      }
    }
  }

  E* out = static_cast<E*>(p.out) + int64_t(r) * p.o_ts;
#pragma unroll
  for (int i = 0; i < kPerWarp; ++i) {
    const int h = h0 + warp * kPerWarp + i;
    if (h >= p.H) continue;
    const bool none = m[i] == -INFINITY && l[i] == 0.f;  // (a NaN score leaves l NaN: not empty)
    const float inv = none ? 0.f : 1.f / l[i];
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
      const int c = x * 128 + lane * 4;
      if (x * 128 >= p.L) break;
      if (c >= p.L) continue;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!none) f = make_float4(o[i][x].x * inv, o[i][x].y * inv, o[i][x].z * inv, o[i][x].w * inv);
      store4(out + h * p.o_hs + c, f);
    }
    if (lane == 0 && p.lse) p.lse[int64_t(r) * p.H + h] = none ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
  }
  if (bad) record_error(hdr, KPOOL_ERR_INVALID_ARG);
  __syncwarp();
  if (checks && threadIdx.x < 32) latent_check(p, hdr);
}

template <typename E>
cudaError_t launch(const LatentParams& p, WorkspaceHeader* hdr, cudaStream_t stream) {
  auto kernel = latent_simt_kernel<E>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kernel),
                                           sizeof(float) * size_t(smem_floats(kMaxChannels)), &ready);
  if (e != cudaSuccess) return e;
  const dim3 grid(uint32_t(p.R), uint32_t((p.H + kHeads - 1) / kHeads));
  kernel<<<grid, 32 * kWarps, sizeof(float) * size_t(smem_floats(p.L + p.P)), stream>>>(p, hdr);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_simt(const LatentParams& p, kpool_dtype dtype, char* ws, cudaStream_t stream) {
  WorkspaceHeader* hdr = reinterpret_cast<WorkspaceHeader*>(ws);
  return dtype == KPOOL_BF16 ? launch<__nv_bfloat16>(p, hdr, stream) : launch<float>(p, hdr, stream);
}

}  // namespace kpool
