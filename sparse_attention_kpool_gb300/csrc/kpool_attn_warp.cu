// kpool_attn_warp.cu -- attention over short lists of selected tokens: bf16, head size 64 or 128.
//
// A gathered item of the tcgen05 kernel is a token's heads of one key head, 128 MMA rows for
// at most 128 heads and a tile of 128 ids: with 8 heads and 24 ids nearly all of it is padding, and
// an item costs 3 us however little it holds (30 us for 64 rows x 68 ids of 32 / 8 heads, 9 here). Here a warp has up to 16 heads of one (token, key
// head) and 16 ids a step, all in registers (mma.sync m16n8k16): nothing is staged in shared
// memory, so many items are in flight per SM and hide each other's latency.
//
// Layout. A product does not depend on the order of the axis that it sums over, nor on
// how its columns are named, as long as both operands agree: lane 4g + t reads 16 bytes of
// key g (channels 8t of every 32) for Q K^T and takes them as two k-steps' operands, with the same
// channels of Q; for P V it reads 16 bytes (channels 8g of every 64) of the keys 2t, 2t + 1, 2t + 8 and
// 2t + 9, pairs the keys' bytes, and column g of product y is channel 8g + y. The scores of a step
// leave the first product as the second one takes its weights, and a lane ends with 8 neighbouring
// channels of the result: every access to memory is 16 bytes of a fully used sector.
#include <cuda_bf16.h>
#include <math.h>

#include "kpool_attn.cuh"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;  // ids per step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// c += A B: A 16 x 16 (rows g, g + 8), B 16 x 8, bf16 with fp32 sums.
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, bool in) {
  return in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ uint32_t word(const uint4& u, int i) {
  return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}

// kRows: the 8-row halves of the product that hold heads (1: at most 8 heads). kSplit: a CTA's four warps
// share an item, each taking every fourth step, and the first adds up; else each has its own.
template <int D, int kRows, bool kSplit>
__global__ void __launch_bounds__(32 * kWarps, kRows == 2 ? 2 : D == 128 ? 3 : 4)
    attn_warp_kernel(const __grid_constant__ AttnParams p, int head_tiles, int64_t items, WorkspaceHeader* hdr) {
  constexpr int kC = D / 32, kH = D / 64;
  constexpr int kVals = kH * 8 * 2 * kRows;
  __shared__ float s_o[kSplit ? (kWarps - 1) * (kVals + 2 * kRows) * 32 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  if (blockIdx.x == 0 && threadIdx.x == 0) attn_clear_error(hdr);
  const int64_t item = kSplit ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * kWarps + warp;

  if (item < items) {
    const int tile = int(item % head_tiles);
    const int64_t rest = item / head_tiles;
    const int hk = int(rest % p.Hkv), r = int(rest / p.Hkv);
    int k0, nk;
    attn_selected_seq(p, r, &k0, &nk);
    const int32_t* ids = p.ids + int64_t(r) * p.width;
    const int end = nk > 0 ? p.width : 0;
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(p.k) + int64_t(hk) * p.k_hs + 8 * t;
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(p.v) + int64_t(hk) * p.v_hs + 8 * g;

    const int j_first = kSplit ? warp * kStep : 0, j_step = kSplit ? kWarps * kStep : kStep;
    auto read_id = [&](int j) {
      const int id = lane < kStep && j + lane < end ? __ldg(ids + j + lane) : -1;
      return id < nk ? id : -1;
    };
    int id = read_id(j_first);

    // Q: rows g (and g + 8), the channels 8t of every 32
    uint4 q[kRows][kC];
#pragma unroll
    for (int h = 0; h < kRows; ++h) {
      const int head = tile * 16 + 8 * h + g;
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + int64_t(r) * p.q_ts +
                                (int64_t(hk) * p.G + head) * p.q_hs + 8 * t;
#pragma unroll
      for (int c = 0; c < kC; ++c) q[h][c] = load8(qr + 32 * c, head < p.G);
    }

    const float c2 = p.scale * kLog2e;
    float m[kRows], l[kRows], o[kRows][kH][8][2];
#pragma unroll
    for (int h = 0; h < kRows; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int x = 0; x < kH; ++x)
#pragma unroll
        for (int y = 0; y < 8; ++y) o[h][x][y][0] = o[h][x][y][1] = 0.f;
    }

    for (int j = j_first; j < end; j += j_step) {
      const uint32_t valid = __ballot_sync(0xffffffffu, id >= 0);
      uint4 kf[2][kC], vf[4][kH];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int i = __shfl_sync(0xffffffffu, id, 8 * n + g);
        const __nv_bfloat16* at = kb + (int64_t(k0) + i) * p.k_ts;
#pragma unroll
        for (int c = 0; c < kC; ++c) kf[n][c] = load8(at + 32 * c, i >= 0);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int i = __shfl_sync(0xffffffffu, id, 8 * (n >> 1) + 2 * t + (n & 1));
        const __nv_bfloat16* at = vb + (int64_t(k0) + i) * p.v_ts;
#pragma unroll
        for (int x = 0; x < kH; ++x) vf[n][x] = load8(at + 64 * x, i >= 0);
      }
      id = read_id(j + j_step);
      if (valid == 0) continue;

      float s[2][4] = {};
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            mma16816(s[n], word(q[0][c], 2 * half), kRows == 2 ? word(q[kRows - 1][c], 2 * half) : 0u,
                     word(q[0][c], 2 * half + 1), kRows == 2 ? word(q[kRows - 1][c], 2 * half + 1) : 0u,
                     word(kf[n][c], 2 * half), word(kf[n][c], 2 * half + 1));

      uint32_t a[2][2] = {};  // [keys 0-7, 8-15][row half]: the weights, as the second product takes them
#pragma unroll
      for (int h = 0; h < kRows; ++h) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 8 * (e >> 1) + 2 * t + (e & 1);
          x[e] = (valid >> key) & 1u ? s[e >> 1][2 * h + (e & 1)] * c2 : -INFINITY;
        }
        float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = fmaxf(mx, m[h]);
        const float base = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: every weight below is exp2(-inf) = 0
        if (__any_sync(0xffffffffu, mx > m[h])) {
          const float f = ptx::exp2_approx(m[h] - base);
          l[h] *= f;
#pragma unroll
          for (int z = 0; z < kH; ++z)
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              o[h][z][y][0] *= f;
              o[h][z][y][1] *= f;
            }
          m[h] = mx;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = ptx::exp2_approx(x[e] - base);
        l[h] += (x[0] + x[1]) + (x[2] + x[3]);
        // bf16 weights, half a step (2^-8) off each, as in the other tensor-core kernels; the sum keeps fp32
        a[0][h] = pack2(x[0], x[1]);
        a[1][h] = pack2(x[2], x[3]);
      }
#pragma unroll
      for (int z = 0; z < kH; ++z)
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const uint32_t pick = y & 1 ? 0x7632 : 0x5410;
          const uint32_t b0 = __byte_perm(word(vf[0][z], y >> 1), word(vf[1][z], y >> 1), pick);
          const uint32_t b1 = __byte_perm(word(vf[2][z], y >> 1), word(vf[3][z], y >> 1), pick);
          float c[4] = {o[0][z][y][0], o[0][z][y][1], kRows == 2 ? o[kRows - 1][z][y][0] : 0.f,
                        kRows == 2 ? o[kRows - 1][z][y][1] : 0.f};
          mma16816(c, a[0][0], a[0][1], a[1][0], a[1][1], b0, b1);
          o[0][z][y][0] = c[0];
          o[0][z][y][1] = c[1];
          if (kRows == 2) {
            o[kRows - 1][z][y][0] = c[2];
            o[kRows - 1][z][y][1] = c[3];
          }
        }
    }

#pragma unroll
    for (int h = 0; h < kRows; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if (kSplit) {
      float* mine = s_o + (warp - 1) * (kVals + 2 * kRows) * 32 + lane;
      if (warp > 0) {
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
          mine[(2 * h) * 32] = m[h];
          mine[(2 * h + 1) * 32] = l[h];
#pragma unroll
          for (int z = 0; z < kH; ++z)
#pragma unroll
            for (int y = 0; y < 16; ++y)
              mine[(2 * kRows + (h * kH + z) * 16 + y) * 32] = o[h][z][y >> 1][y & 1];
        }
      }
      __syncthreads();  // (an item is a CTA's: all of its warps come here)
      if (warp == 0) {
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
          float mx = m[h];
          for (int w = 0; w < kWarps - 1; ++w) mx = fmaxf(mx, s_o[(w * (kVals + 2 * kRows) + 2 * h) * 32 + lane]);
          const float base = mx == -INFINITY ? 0.f : mx;
          // without any weight a part adds nothing; with a NaN among its scores its sum passes on
          const float f = m[h] == -INFINITY ? 1.f : ptx::exp2_approx(m[h] - base);
          l[h] *= f;
#pragma unroll
          for (int z = 0; z < kH; ++z)
#pragma unroll
            for (int y = 0; y < 16; ++y) o[h][z][y >> 1][y & 1] *= f;
          for (int w = 0; w < kWarps - 1; ++w) {
            const float* part = s_o + w * (kVals + 2 * kRows) * 32 + lane;
            const float pm = part[2 * h * 32], pf = pm == -INFINITY ? 1.f : ptx::exp2_approx(pm - base);
            l[h] = fmaf(part[(2 * h + 1) * 32], pf, l[h]);
#pragma unroll
            for (int z = 0; z < kH; ++z)
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                float& x = o[h][z][y >> 1][y & 1];
                x = fmaf(part[(2 * kRows + (h * kH + z) * 16 + y) * 32], pf, x);
              }
          }
          m[h] = mx;
        }
      }
    }
    if (!kSplit || warp == 0) {
#pragma unroll
      for (int h = 0; h < kRows; ++h) {
        const int head = tile * 16 + 8 * h + g;
        if (head >= p.G) continue;
        const bool none = m[h] == -INFINITY && l[h] == 0.f;  // (a NaN score leaves l NaN: not empty)
        const float inv = none ? 0.f : 1.f / l[h];
        const int64_t row_head = int64_t(hk) * p.G + head;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(r) * p.o_ts + row_head * p.o_hs + 16 * t;
#pragma unroll
        for (int z = 0; z < kH; ++z)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (!none)
              u = make_uint4(pack2(o[h][z][0][e] * inv, o[h][z][1][e] * inv), pack2(o[h][z][2][e] * inv, o[h][z][3][e] * inv),
                             pack2(o[h][z][4][e] * inv, o[h][z][5][e] * inv), pack2(o[h][z][6][e] * inv, o[h][z][7][e] * inv));
            *reinterpret_cast<uint4*>(out + 64 * z + 8 * e) = u;
          }
        if (t == 0 && p.lse) p.lse[int64_t(r) * p.Hq + row_head] = none ? -INFINITY : (m[h] + log2f(l[h])) * kLn2;
      }
    }
  }
  if (blockIdx.x == 0 && warp == 0) {
    __syncwarp();
    attn_check(p, hdr);
  }
}

template <int D>
cudaError_t launch(const AttnParams& p, char* ws, cudaStream_t stream, bool split) {
  const int rows = p.G <= 8 ? 1 : 2, head_tiles = (p.G + 15) / 16;
  const int64_t items = int64_t(p.R) * p.Hkv * head_tiles;
  const int64_t grid = split ? items : (items + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    kernel<<<uint32_t(grid), 32 * kWarps, 0, stream>>>(p, head_tiles, items, reinterpret_cast<WorkspaceHeader*>(ws));
    return cudaGetLastError();
  };
  if (rows == 1) return split ? go(attn_warp_kernel<D, 1, true>) : go(attn_warp_kernel<D, 1, false>);
  return split ? go(attn_warp_kernel<D, 2, true>) : go(attn_warp_kernel<D, 2, false>);
}

}  // namespace

// Few items: the CTA's warps share each, which pays from three steps on (one step takes a microsecond).
static bool warp_split(const AttnParams& p, int sms) {
  return int64_t(p.R) * p.Hkv * ((p.G + 15) / 16) <= 8 * int64_t(sms) && p.width > 2 * kStep;
}

bool attn_warp_wanted(const AttnParams& p, int sms) {
  // Microseconds, from the measured parts: an item (16 heads) takes 0.1 and, a step of 16 ids, 0.12 of an SM's time at
  // head size 128 (8 KB: 36 bytes a cycle out of L2), twice that out of HBM; a warp alone needs 0.9 a step.
  // Measured here / the better of gathered and dense: 32 / 8 heads of 128, 64 rows x 68 ids 8.8 / 30, x 1,028
  // 67 / 60; 1 row x 20 4.8 / 8.3, x 260 7.9 / 10.8, x 1,028 18.8 / 14.2; prompts of 500 x 20 14 / 23, x 68 26 / 23,
  // 3,000 x 20 61 / 110, x 68 122 / 115; 24 / 4 heads of 64, 3,000 x 68 31 / 86, x 260 82 / 86, x 1,028 267 / 87;
  // 64 / 1 heads of 128, 3,000 x 68 73 / 89, x 260 194 / 155.
  const int64_t keys = p.T / p.S;  // a prompt's rows have no more to name than their sequences hold
  const double ids = double(p.row_seq == nullptr && keys < p.width ? keys : p.width);
  const double steps = ceil(ids / kStep), part = p.D / 128.0;
  const double items = double(p.R) * p.Hkv * ((p.G + 15) / 16) / sms;
  const double far = double(p.T) * p.Hkv * p.D * 4.0 > 96e6 ? 2.0 : 1.0;  // K and V do not stay in L2
  const double alone = steps / (warp_split(p, sms) ? kWarps : 1) * (0.3 + 0.6 * part);
  const double all = items * (0.1 + steps * 0.12 * part * far);
  const AttnSelectedTimes other = attn_selected_times(p, sms);
  return 4.0 + (alone > all ? alone : all) < (other.dense < other.gathered ? other.dense : other.gathered);
}

cudaError_t launch_attn_warp(const AttnParams& p, int sms, char* ws, cudaStream_t stream) {
  const bool split = warp_split(p, sms);
  return p.D == 64 ? launch<64>(p, ws, stream, split) : launch<128>(p, ws, stream, split);
}

}  // namespace kpool
