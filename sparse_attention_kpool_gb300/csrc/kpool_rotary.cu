// kpool_rotary.cu -- rotary positions: the C ABI of kpool_rotary / kpool_rotary_table and its kernel.
//
// Channel pair (a, b) number i of a head at position t becomes
//   (a cos x - b sin x, b cos x + a sin x) * magnitude,  x = t f[i]  (the inverse: -t f[i]).
//
// Angles. Only x modulo a turn matters, and t is a whole number: the table holds f[i] / 2 pi as a
// 64-bit fraction of a turn, and the low 64 bits of t times that are the fraction of a turn at t,
// exact but for the table's own error, which kpool_rotary_table keeps to a few units of 2^-64 turns (t of them at t: 2^-30
// of a half turn at 2^31). In fp32 t f[i] at a million tokens would be off by 0.06, and in fp64 the reduction would cost
// what the rest does. The top 32 bits go to fp32 (half a step is 2^-25 of a half turn at most), then through sincospif.
//
// What bounds it. Every channel is read and written once and a pair takes six operations: HBM. A thread has
// eight bf16 (four fp32) pairs of a token, takes their cosines and sines once and applies them to several
// heads of q or k one after the other, 16 bytes at a time: neighbouring threads share whole 128-byte lines, and have
// neighbouring heads (105 against 113 us for heads in runs of eight). 32,768 tokens of 32 + 8 heads of 128: 104 us = 6.4
// TB/s, 95 % of the measured copy rate; 4,099 tokens of 64 heads of 192 with 64 rotated channels: 39 us, 5.2 TB/s; the same
// in fp32 197 us, 6.8 TB/s, and 71, 5.7. Where a row or a part of q or k does not lie on whole 16-byte words, both go by
// single elements: 156 us, 152 where it is k alone.
#include <cuda_bf16.h>
#include <math.h>

#include "kpool_internal.cuh"

namespace kpool {
namespace {

constexpr int kThreads = 128;

struct RotaryPart {
  const char* in;
  char* out;
  int64_t in_ts, in_hs, out_ts, out_hs;  // bytes
  int32_t heads, at;                     // at: first rotated channel
  int32_t dim;
  int32_t copies;                        // pieces of V channels that stay as they are
  int32_t per, groups;                   // heads of a thread, and threads for all heads
  uint32_t blocks;
};

struct RotaryParams {
  RotaryPart part[2];
  const int32_t* positions;
  const uint64_t* table;
  int64_t tokens;
  int32_t pairs;                         // of a head
  int32_t inverse;
  float magnitude;
};

template <typename E>
__device__ __forceinline__ float to_f32(E x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E>
__device__ __forceinline__ E from_f32(float x);
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

// V elements, read and written as one (16 bytes where V fills them).
template <typename E, int V>
struct alignas(V * sizeof(E)) Vec {
  E e[V];
};

// kPairs: neighbouring channels are a pair; else channel i and i + pairs.
template <typename E, int V, bool kPairs>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  const bool second = blockIdx.x >= p.part[0].blocks;
  const RotaryPart& w = p.part[second];
  const int64_t unit = int64_t(blockIdx.x - (second ? p.part[0].blocks : 0)) * kThreads + threadIdx.x;
  const int turns = p.pairs / V;       // threads of a head
  const int64_t row = unit / turns;    // token and group of heads
  const int slot = int(unit - row * turns);
  const int64_t t = row / w.groups;
  if (t >= p.tokens) return;
  // every groups-th head: neighbouring threads have neighbouring heads
  const int h0 = int(row - t * w.groups), h1 = w.heads, step = w.groups;
  const int64_t in_step = w.in_hs * step, out_step = w.out_hs * step;
  const char* in = w.in + t * w.in_ts + h0 * w.in_hs;
  char* out = w.out + t * w.out_ts + h0 * w.out_hs;
  using T = Vec<E, V>;

  // The thread's pieces a and b of V channels. Halves: b is a's other half. Neighbours: pieces number `slot` and
  // slot + turns, with V / 2 pairs each (one of V = 1 is a channel of the pair).
  constexpr int kIn = kPairs && V > 1 ? V / 2 : V;  // pairs that follow one another in the table
  float cs[V], sn[V];
  const int64_t pos = __ldg(p.positions + t);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint64_t x = uint64_t(pos) * __ldg(p.table + (slot + (i / kIn) * turns) * kIn + i % kIn);
    sincospif(float(int32_t(x >> 32)) * 0x1p-31f, &sn[i], &cs[i]);
    cs[i] *= p.magnitude;
    sn[i] *= p.inverse ? -p.magnitude : p.magnitude;
  }
  const bool wide = kPairs && V > 1;
  const int ca = (w.at + (kPairs && V == 1 ? 2 : 1) * slot * V) * int(sizeof(E));
  const int cb = ca + (wide ? turns * V : kPairs ? 1 : p.pairs) * int(sizeof(E));
  // Two heads at a time, their reads before their writes: in place every piece is read and written by one thread, which
  // the compiler does not know. (Four: 118 registers, 133 us for 32,768 tokens of 32 + 8 heads of 128; two 104, one 107.)
  constexpr int kBatch = 2;
  for (int h = h0; h < h1; h += kBatch * step) {
    T a[kBatch], b[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      if (h + y * step >= h1) break;
      a[y] = *reinterpret_cast<const T*>(in + y * in_step + ca);
      b[y] = *reinterpret_cast<const T*>(in + y * in_step + cb);
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      if (h + y * step >= h1) break;
      T u, v;
      if constexpr (kPairs && V > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int j = 2 * (i % kIn);
          const T& from = i < kIn ? a[y] : b[y];
          T& to = i < kIn ? u : v;
          const float c = to_f32(from.e[j]), d = to_f32(from.e[j + 1]);
          to.e[j] = from_f32<E>(c * cs[i] - d * sn[i]);
          to.e[j + 1] = from_f32<E>(d * cs[i] + c * sn[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float c = to_f32(a[y].e[i]), d = to_f32(b[y].e[i]);
          u.e[i] = from_f32<E>(c * cs[i] - d * sn[i]);
          v.e[i] = from_f32<E>(d * cs[i] + c * sn[i]);
        }
      }
      *reinterpret_cast<T*>(out + y * out_step + ca) = u;
      *reinterpret_cast<T*>(out + y * out_step + cb) = v;
    }
    // The thread's share of the channels that stay. (Threads of their own for them make the warps of both wait: 57 against
    // 39 us for 4,099 tokens of 64 heads of 192.)
    for (int x = slot; x < w.copies; x += turns) {
      const int c = (x * V + (x * V >= w.at ? 2 * p.pairs : 0)) * int(sizeof(E));
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
        if (h + y * step < h1) a[y] = *reinterpret_cast<const T*>(in + y * in_step + c);
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
        if (h + y * step < h1) *reinterpret_cast<T*>(out + y * out_step + c) = a[y];
    }
    in += kBatch * in_step;
    out += kBatch * out_step;
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool heads_ok(const kpool_heads& t, int32_t dim, int64_t e) {
  if (t.data == nullptr || !aligned(t.data, uintptr_t(e))) return false;
  for (const int64_t st : {t.token_stride, t.head_stride})
    if (st < dim || st >= (int64_t(1) << 38)) return false;
  return true;
}

// All of a tensor's rotated and copied pieces are whole 16-byte words.
bool wide(const kpool_rotary_part& p, int64_t e) {
  for (const kpool_heads* t : {&p.in, &p.out})
    if (!aligned(t->data, 16) || (t->token_stride * e) % 16 != 0 || (t->head_stride * e) % 16 != 0) return false;
  return (p.offset * e) % 16 == 0 && (p.head_dim * e) % 16 == 0;
}

template <typename E, int V>
cudaError_t launch(const RotaryParams& p, bool interleaved, uint32_t blocks, cudaStream_t stream) {
  if (interleaved)
    rotary_kernel<E, V, true><<<blocks, kThreads, 0, stream>>>(p);
  else
    rotary_kernel<E, V, false><<<blocks, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace kpool

using namespace kpool;

extern "C" {

kpool_status kpool_rotary_table(int32_t rotary_dim, double base, double factor, double original_length, double low,
                                double high, int64_t* out) {
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > 65536 || out == nullptr) return KPOOL_ERR_INVALID_ARG;
  if (!(isfinite(base) && base > 0.0 && isfinite(factor) && factor > 0.0)) return KPOOL_ERR_INVALID_ARG;
  if (!(isfinite(original_length) && original_length >= 0.0)) return KPOOL_ERR_INVALID_ARG;
  if (original_length > 0.0 && !(isfinite(low) && isfinite(high) && low >= 0.0 && high > low))
    return KPOOL_ERR_INVALID_ARG;
  // In long double, whose 64 bits or more are the table's: in double the fast pairs would be off by 2^-56 of a turn and
  // more, at a position of 2^31 by more than fp32 leaves. (2 pi as two doubles.)
  const long double turn = static_cast<long double>(6.283185307179586476925) + 2.449293598294706414e-16;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const long double f = powl(base, -2.0L * i / rotary_dim);
    long double keep = 0.0L;
    if (original_length > 0.0) {
      const long double at = (original_length * f / turn - low) / (static_cast<long double>(high) - low);
      keep = fminl(1.0L, fmaxl(0.0L, at));
    }
    const long double g = f * (keep + (1.0L - keep) / factor) / turn;
    if (!isfinite(static_cast<double>(g))) return KPOOL_ERR_INVALID_ARG;
    // a fraction of a turn, in units of 2^-64 (whole turns do not matter, one that it rounds up to included)
    const long double units = floorl(ldexpl(fmodl(g, 1.0L), 64) + 0.5L);
    out[i] = units < ldexpl(1.0L, 64) ? int64_t(uint64_t(units)) : 0;
  }
  return KPOOL_OK;
}

kpool_status kpool_rotary(const kpool_rotary_part* q, const kpool_rotary_part* k, const int32_t* positions,
                          const int64_t* table, int64_t tokens, const kpool_rotary_shape* shape, void* stream_ptr) {
  if (shape == nullptr || q == nullptr || tokens < 0 || tokens > INT32_MAX / 2) return KPOOL_ERR_INVALID_ARG;
  if (shape->dtype != KPOOL_BF16 && shape->dtype != KPOOL_F32) return KPOOL_ERR_INVALID_ARG;
  if (shape->rotary_dim < 2 || shape->rotary_dim % 2 != 0 || !isfinite(shape->magnitude)) return KPOOL_ERR_INVALID_ARG;
  if ((shape->flags & ~(KPOOL_ROTARY_INTERLEAVED | KPOOL_ROTARY_INVERSE)) != 0) return KPOOL_ERR_INVALID_ARG;
  const int64_t e = shape->dtype == KPOOL_BF16 ? 2 : 4;
  const kpool_rotary_part* parts[2] = {q, k};
  for (const kpool_rotary_part* w : parts) {
    if (w == nullptr) continue;
    if (w->heads < 1 || w->head_dim < 1 || w->reserved != 0 || w->offset < 0 ||
        int64_t(w->offset) + shape->rotary_dim > w->head_dim)
      return KPOOL_ERR_INVALID_ARG;
    if (w->heads > 4096 || w->head_dim > 4096) return KPOOL_ERR_UNSUPPORTED;
  }
  if (tokens == 0) return KPOOL_OK;
  for (const kpool_rotary_part* w : parts) {
    if (w == nullptr) continue;
    if (!heads_ok(w->in, w->head_dim, e) || !heads_ok(w->out, w->head_dim, e)) return KPOOL_ERR_INVALID_ARG;
    // in place means the same places
    if (w->in.data == w->out.data &&
        (w->in.token_stride != w->out.token_stride || w->in.head_stride != w->out.head_stride))
      return KPOOL_ERR_INVALID_ARG;
  }
  if (!positions || !aligned(positions, 4) || !table || !aligned(table, 8)) return KPOOL_ERR_INVALID_ARG;

  RotaryParams p{};
  p.positions = positions;
  p.table = reinterpret_cast<const uint64_t*>(table);
  p.tokens = tokens;
  p.pairs = shape->rotary_dim / 2;
  p.inverse = (shape->flags & KPOOL_ROTARY_INVERSE) != 0;
  p.magnitude = shape->magnitude;
  // 16-byte pieces where every row and part begins and ends on one, else single elements
  const int full = int(16 / e);
  const bool vec = p.pairs % full == 0 && wide(*q, e) && (k == nullptr || wide(*k, e));
  const int v = vec ? full : 1;
  int sms = 0;
  if (!note_cuda_error(device_sm_count(&sms))) return KPOOL_ERR_CUDA;
  int64_t blocks = 0;
  for (int i = 0; i < 2; ++i) {
    RotaryPart& r = p.part[i];
    const kpool_rotary_part* w = parts[i];
    r.groups = 1;
    if (w == nullptr) continue;
    r.in = static_cast<const char*>(w->in.data);
    r.out = static_cast<char*>(w->out.data);
    r.in_ts = w->in.token_stride * e;
    r.in_hs = w->in.head_stride * e;
    r.out_ts = w->out.token_stride * e;
    r.out_hs = w->out.head_stride * e;
    r.heads = w->heads;
    r.at = w->offset;
    r.dim = w->head_dim;
    const int rest = r.in == r.out ? 0 : w->head_dim - shape->rotary_dim;
    r.copies = rest / v;
    const int turns = p.pairs / v;
    // Heads of a thread: eight share a thread's cosines and sines; fewer while that leaves SMs without 1,024
    // threads each.
    r.per = 8;
    while (r.per > 1 && tokens * turns * ((r.heads + r.per - 1) / r.per) < int64_t(1024) * sms) r.per /= 2;
    r.groups = (r.heads + r.per - 1) / r.per;
    const int64_t n = (tokens * turns * r.groups + kThreads - 1) / kThreads;
    blocks += n;
    if (blocks > INT32_MAX) return KPOOL_ERR_UNSUPPORTED;
    r.blocks = uint32_t(n);
  }
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const bool il = (shape->flags & KPOOL_ROTARY_INTERLEAVED) != 0;
  const uint32_t b = uint32_t(blocks);
  cudaError_t err;
  if (shape->dtype == KPOOL_BF16)
    err = vec ? launch<__nv_bfloat16, 8>(p, il, b, stream) : launch<__nv_bfloat16, 1>(p, il, b, stream);
  else
    err = vec ? launch<float, 4>(p, il, b, stream) : launch<float, 1>(p, il, b, stream);
  return note_cuda_error(err) ? KPOOL_OK : KPOOL_ERR_CUDA;
}

}  // extern "C"
