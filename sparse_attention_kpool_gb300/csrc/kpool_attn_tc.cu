// kpool_attn_tc.cu -- attention on the 5th-generation tensor cores (bf16, head_dim 64 or
// 128): one pass over K and V with the running maximum and sum of a softmax.
//
// Rows. The G query heads that share a key head and TT = 128 / G tokens fill the 128 rows of
// an MMA (row = token * G + head of the group), so a K/V tile read once serves all of them,
// decode steps of one token included. Four forms (Form):
//   kTwo     two such row tiles per CTA, 2 * TT tokens that share every K/V tile;
//   kOne     one row tile, where sequences have fewer rows: its K/V tiles alternate between
//            the two softmax groups, each with its own accumulator and statistics, added up at
//            the end;
//   kGather  kOne for the heads of one token over the keys that its ids name: four warps
//            copy them, 16 bytes a lane (cp.async), into the layout that TMA writes. (TMA's
//            gather of four rows moved 6 bytes a cycle and SM, these copies 27; 2048 rows x
//            2052 ids of 64 / 1 heads: 1222 against 288 us.)
//   kDense   kTwo under a mask of bits for all keys (kpool_attn_dense.cu).
//   kPagedOne, kPagedTwo   kOne and kTwo over a cache in pages, a TMA box for what lies in one page;
//   kPagedTokens  kPagedTwo, the tokens of small pages by plain copies;
//   kPagedRows  decode steps over pages: as kGather, but for whole caches of any length.
//
// Roles (12 warps; kGather 16): warps 0-3 and 4-7 are the softmax groups 0 and 1, a thread
// per row; warp 8 loads by TMA; warps 9 and 10 issue the MMAs of group 0 and 1 (warp 9 owns
// TMEM); warp 11 cleans V tiles (below), warps 12-15 gather. Per 128-key tile of a group:
// S = Q K^T (128 x 128, fp32 in TMEM); its thread reads the row, takes the maximum, writes
// P = 2^(c s - c m) as bf16 over S in TMEM and adds its fp32 sum; O += P V with P read from
// TMEM. K and V share one ring of tiles in the order in which the MMAs consume them.
//
// What bounds it. Of an MMA's 64 cycles at full rate, Q K^T alone (both operands from shared
// memory) takes 93 and P V alone (one from TMEM) 75; alternating they run at 64, so the tensor
// core could do a pair of tiles in 2048 cycles. A tile's chain, softmax (1260 cycles: 128
// exponentials at 4 cycles a warp instruction are 512 of them), handing P over (390), P V and
// the next Q K^T (1200), handing S over (400), is 3250, and with two groups in flight that is
// the time of a pair. 32,768 tokens of 32 / 8 heads of 128: 5.95 ms = 1.48 PFLOP/s, 86 % of
// the measured sustained rate of a large product. Decode is bound by HBM: 792 MB of caches in
// 136 us = 5.8 TB/s, 86 % of the measured copy rate. Short sequences pay 4 to 6 us of start,
// masks and epilogue per row tile.
// Over pages, decode steps of the same sizes: 132 us, 6.0 TB/s in the kernel (kPagedRows).
// Keys with a shared part (192 channels, values of 128): a turn's products are 18 instructions in 1,470
// cycles (P V 75 each, Q K^T at N = 96 80: operands from shared memory), two groups 2,915 a pair of tiles of
// 96 keys; 16,384 tokens of 32 heads: 2.03 ms = 1.35 PFLOP/s (2.10 with new inputs in every call).
//
// Running maximum. O is rescaled only when a row's maximum has grown by more than 8 in the
// exponent: weights then reach at most 2^8, which costs neither bf16 nor fp32 any precision,
// and the rescale (a pass over O in TMEM) becomes rare. P is rounded to bf16 (half a step is
// 2^-8 of a weight) because the second product takes bf16; the row sum adds the weights before
// that rounding, in fp32. Exponentials are the hardware's (2 ulp).
//
// Masked places. A key that a row does not see gets s = -inf, so what K holds there does not
// matter. A weight of zero does not silence V, though (0 * NaN): in the tiles that some row
// does not see entirely, warp 11 first overwrites V rows past the last visible key with
// zeros, replaces every other infinity or NaN by zero and raises a flag; rows that do see such
// a value add it in the epilogue. (kGather writes zeros for ids outside the sequence.)
//
// Work. A pass over (sequence, key head, row tile, K/V tile): whole row tiles, one to a CTA,
// or a persistent CTA per SM with an equal run of all K/V tiles of the call, found by every CTA
// itself from the lengths on the device; unfinished rows go to the workspace as (m, l, O) and
// a second kernel joins them in the order of the runs, so results repeat bit for bit. launch()
// has the rule and both sides' times.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <utility>

#include "kpool_attn.cuh"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

// Keys of a tile. 96 with a shared part of the keys: two tiles of K (192 channels) and of V then fit beside Q of two row
// tiles; with 128 there is room for one V, whose next tile is waited for (5,200 cycles a pair of tiles, half of them).
template <class P>
constexpr int kTile = kSharedKeys<P> ? 96 : 128;
constexpr int kTileRows = kAttnTileRows;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;  // growth of the maximum (in powers of two) that O is not rescaled for
// 1 s. Legitimate waits are microseconds, and for the cleaning warp's first tile as long as the tiles before it in
// the segment take (1.7 us each: 14 ms after a million keys).
constexpr uint64_t kMaxWaitNs = 1000000000ull;
constexpr int kGatherWarps = 4;
// Gathered tiles whose validity bits are held: the producer is at most the ring of tiles (8 slots,
// four K and four V) plus the two K tiles of lead ahead of the softmax.
constexpr int kBitsRing = 8;
constexpr int kSegRing = 4;    // segments handed from the producer to the other roles

// The forms of the kernel: one or two row tiles of consecutive tokens, one token's heads over gathered keys, or
// two row tiles under a mask of bits for all keys (the dense form of a selection); one or two over pages, by TMA, or
// two by plain copies; a token's heads over pages, by plain copies.
enum Form { kOne, kTwo, kGather, kDense, kPagedOne, kPagedTwo, kPagedTokens, kPagedRows };

// Where a tile of the ring lies, and the parity of its use of that slot.
struct Place {
  uint32_t slot, par;
};

// DK: channels of Q and K, DV: of V and the result. With DK > DV the last DK - DV channels of K come from a tensor
// of their own without heads, and K and V have rings of their own.
template <int DK, int DV, Form F>
struct Cfg {
  static constexpr bool TOKENS = F == kPagedTokens;
  static constexpr bool TWO = F == kTwo || F == kDense || F == kPagedTwo || TOKENS;
  static constexpr bool PAGED = F == kPagedOne || F == kPagedTwo || F == kPagedRows || TOKENS;
  static constexpr bool SHARED = DK != DV;
  static constexpr bool GATHER = F == kGather || F == kPagedRows;  // keys come by plain copies
  using Params = std::conditional_t<PAGED, AttnPagedParams, std::conditional_t<SHARED, AttnSharedParams, AttnParams>>;
  // The ring holds K(0) .. K(kAhead - 1), then K(j), V(j - kAhead) in turn: the order in which the MMAs use
  // them, K one tile (one-tile form: one per group) ahead.
  static constexpr int kAhead = TWO ? 1 : 2;
  static constexpr int kThreads = GATHER ? 512 : 384;
  static constexpr int kTileKeys = kTile<Params>;
  static constexpr int kScoreCols = kTileKeys / 32;      // 32-column pieces of a row's scores
  static constexpr int kPCol = kTileKeys / 2;            // a tile's weights, bf16, replace the upper half of its scores
  static constexpr int kQBytes = kTileRows * DK * 2;     // one Q tile
  static constexpr int kQBlock = kTileRows * 128;        // a 64-column block of one
  static constexpr int kTileBytes = kTileKeys * DK * 2;  // one K tile
  static constexpr int kVBytes = kTileKeys * DV * 2;     // one V tile
  static constexpr int kHalf = kTileKeys * 128;          // a 64-column block of a tile
  static constexpr int kBlocks = DK / 64, kVBlocks = DV / 64;
  static constexpr int kQTiles = TWO ? 2 : 1;
  // rings apart: the first kKSlots slots hold K, the others V; as many as fit beside Q at 192 + 128 channels
  static constexpr int kKSlots = TWO ? 2 : 3, kVSlots = 2;
  static constexpr int kStages = SHARED ? kKSlots + kVSlots : DK == 64 ? 8 : (TWO ? 5 : 6);
  static constexpr int kOffRing = kQTiles * kQBytes;
  static constexpr int kOffBar = kOffRing + (SHARED ? kKSlots * kTileBytes + kVSlots * kVBytes : kStages * kTileBytes);
  // full[stages] empty[stages] clean[stages] dirty[stages] q_full q_empty s_full[2] p_ready[2] o_final o_free done
  // seg_full[ring] seg_empty[ring] turn[2]
  static constexpr int kNumBars = 4 * kStages + 11 + 2 * kSegRing;
  static constexpr int kOffMisc = (kOffBar + 8 * kNumBars + 15) & ~15;  // 16-byte words follow
  static constexpr int kOffSeg = kOffMisc + 80;
  static constexpr int kOffStat = kOffSeg + 64 * kSegRing;         // [2][128] float2 (m, l), one-tile form only
  static constexpr int kOffBits = kOffStat + (TWO ? 0 : 2 * kTileRows * 8);  // [kBitsRing] x 128 bits
  static_assert(kOffBits % 16 == 0 && kOffSeg % 16 == 0 && kOffStat % 16 == 0, "16-byte accesses");
  static constexpr int kSmem = kOffBits + (GATHER ? 16 * kBitsRing : 0);
  static_assert(kSmem <= 232448, "exceeds the 227 KB per-CTA shared memory limit");

  // Use number u of the ring (of the K or the V ring where they are apart), and a slot's bytes from the ring's start.
  __device__ static __forceinline__ Place k_slot(uint32_t u) {
    if (SHARED) return {u % kKSlots, (u / kKSlots) & 1};
    return {u % kStages, (u / kStages) & 1};
  }
  __device__ static __forceinline__ Place v_slot(uint32_t u) {
    if (SHARED) return {kKSlots + u % kVSlots, (u / kVSlots) & 1};
    return k_slot(u);
  }
  __device__ static __forceinline__ uint32_t slot_at(uint32_t slot) {
    if (SHARED && slot >= kKSlots) return kKSlots * kTileBytes + (slot - kKSlots) * kVBytes;
    return slot * kTileBytes;
  }
  // K and V of tile j of a segment of n tiles; `use`: ring uses before the segment, two a tile.
  __device__ static __forceinline__ Place k_place(uint32_t use, int j) {
    return k_slot(SHARED ? use / 2 + j : use + uint32_t(j + max(0, j - kAhead)));
  }
  __device__ static __forceinline__ Place v_place(uint32_t use, int j, int n) {
    return v_slot(SHARED ? use / 2 + j : use + uint32_t(min(n, j + kAhead + 1) + j));
  }
};

struct Misc {
  int64_t base;       // persistent form: first position of sequence b
  int64_t lo, hi;     // positions of this CTA
  int64_t total;
  int32_t runs;       // runs that have tiles
  int32_t b;
  int32_t whole;      // pages: row tiles of a head where the lengths want whole items, else 0
  uint32_t tmem;
  volatile int32_t abort;
  volatile int32_t bad_page;           // a page of the table that the pool does not have
  volatile int32_t bad_seg[kSegRing];  // 1 + the last segment of this slot with an infinity or NaN in a cleaned V tile
};
static_assert(sizeof(Misc) <= 80, "Misc fits its space");

// ------------------------------------------------------------------ work segments

struct Seg {
  AttnSeq sq;
  int hk, tok0;
  int kt0, n;      // first K/V tile of this CTA and their number (0: no row sees a key; -1: the work is done)
  int n0;          // tiles that the first row tile needs (two)
  int end;         // keys that some row sees
  int all;         // keys that every row sees
  int8_t whole;    // no other CTA has tiles of these rows
  int8_t slot;     // partial slot of the CTA: 0 when an earlier run began the item, else 1
};
static_assert(sizeof(Seg) <= 64, "Seg fits its space");

template <class P>
__device__ __forceinline__ int tile_cost(const P& p, const AttnSeq& s, int t, int ttb) {
  const int end = attn_keys_end(p, s, min((t + 1) * ttb, s.nq));
  return max(1, (end + kTile<P> - 1) / kTile<P>);
}

// Beginning and finishing an item (Q, first product, epilogue) takes about as long as this
// many tiles; it is counted when runs are cut, as positions before the item's first tile.
constexpr int kItemCost = 3;

// sum over i in [0, n) of floor((a i + b) / m), in steps of Euclid's algorithm on (m, a)
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t ans = 0;
  while (n > 0) {
    if (a >= m) {
      ans += int64_t(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      ans += int64_t(n) * (b / m);
      b %= m;
    }
    const uint64_t y = uint64_t(a) * n + b;
    if (y < m) break;
    if (y >> 32) {
      n = uint32_t(y / m);
      b = uint32_t(y % m);
    } else {
      n = uint32_t(y) / m;
      b = uint32_t(y) % m;
    }
    const uint32_t x = m;
    m = a;
    a = x;
  }
  return ans;
}

__device__ __forceinline__ int row_tiles(const AttnSeq& s, int ttb) { return (s.nq + ttb - 1) / ttb; }

// Positions of one head's row tiles [0, t), t <= row_tiles: tile u ends at key prefix + (u + 1) ttb
// (the last at prefix + nq) and counts at least one key tile.
template <class P>
__device__ __forceinline__ int64_t head_cost(const P& p, const AttnSeq& s, int t, int ttb) {
  if (t == 0) return 0;
  if (!s.ok || s.nk == 0) return int64_t(t) * (kItemCost + 1);
  if (!attn_causal(p)) return int64_t(t) * (kItemCost + (s.nk + kTile<P> - 1) / kTile<P>);
  const int nt = row_tiles(s, ttb), m = min(t, nt - 1);
  const int z = s.prefix < 0 ? min(m, -s.prefix / ttb) : 0;  // tiles without any key
  int64_t c = int64_t(t) * kItemCost + z;
  c += floor_sum(uint32_t(m - z), kTile<P>, uint32_t(ttb), uint32_t(s.prefix + (z + 1) * ttb + kTile<P> - 1));
  if (t == nt) c += max(1, (s.prefix + s.nq + kTile<P> - 1) / kTile<P>);
  return c;
}

template <class P>
__device__ __forceinline__ int64_t seq_cost(const P& p, const AttnSeq& s, int ttb) {
  return head_cost(p, s, row_tiles(s, ttb), ttb) * p.Hkv;
}

// The segments of a CTA. Positions number the K/V tiles of the call: by sequence, key
// head, row tile, then key tile (after kItemCost positions for the item itself); a row tile
// without any key counts as one. A border among an item's first positions lies before its first tile.
struct SegIter {
  int64_t pos, hi;
  int64_t item;            // first position of the present item
  int b, hk, t, nt, c;     // its sequence, key head and row tile; the head's row tiles, the item's key tiles
  AttnSeq sq;

  template <class P>
  __device__ __forceinline__ void start(const P& p, const Misc* m, int ttb) {
    pos = m->lo;
    hi = m->hi;
    b = m->b;
    if (pos >= hi) return;
    sq = attn_seq(p, b);
    nt = row_tiles(sq, ttb);
    const int64_t per_head = head_cost(p, sq, nt, ttb), off = pos - m->base;
    hk = int(off / per_head);
    const int64_t in_head = off - hk * per_head;
    t = 0;
    for (int top = nt - 1; t < top;) {  // the last tile that begins at or before the position
      const int mid = (t + top + 1) >> 1;
      if (head_cost(p, sq, mid, ttb) <= in_head) t = mid; else top = mid - 1;
    }
    item = pos - (in_head - head_cost(p, sq, t, ttb));
    c = tile_cost(p, sq, t, ttb);
  }
  __device__ __forceinline__ int64_t first_tile() const { return item + kItemCost; }
  template <class P>
  __device__ __forceinline__ bool next(const P& p, int ttb, Seg* s) {
    if (pos >= hi) return false;
    if (pos == first_tile() + c) {  // the item is done
      item = pos;
      if (++t == nt) {
        t = 0;
        if (++hk == p.Hkv) {
          hk = 0;
          do {
            sq = attn_seq(p, ++b);
          } while (sq.nq == 0);
          nt = row_tiles(sq, ttb);
        }
      }
      c = tile_cost(p, sq, t, ttb);
    }
    const int64_t tile0 = first_tile();
    if (hi <= tile0) return false;  // (only as the run's last item)
    s->sq = sq;
    s->hk = hk;
    s->tok0 = t * ttb;
    s->kt0 = int(max(pos - tile0, int64_t(0)));
    s->n = int(min(int64_t(c), hi - tile0)) - s->kt0;
    s->whole = s->n == c;
    s->slot = s->kt0 > 0 ? 0 : 1;
    pos = tile0 + s->kt0 + s->n;
    return true;
  }

  // The same for whole items, every grid-th to a CTA in the order of whole_seg, without gaps in their numbers (which would
  // leave some CTAs an item more than others). pos and item count a head's row tiles here.
  __device__ __forceinline__ void start_whole(int head_tiles) {
    hi = head_tiles;
    pos = hi + blockIdx.x;  // (the first head begins like the others)
    hk = -1;
  }
  template <class P>
  __device__ __forceinline__ bool next_whole(const P& p, int ttb, Seg* s) {
    while (pos >= hi) {
      pos -= hi;
      if (++hk == p.Hkv) return false;
      b = p.S;
      item = 0;
      nt = 0;
    }
    while (pos >= item + nt) {
      if (--b < 0) return false;
      item += nt;
      sq = attn_seq(p, b);
      nt = row_tiles(sq, ttb);
    }
    t = nt - 1 - int(pos - item);
    s->sq = sq;
    s->hk = hk;
    s->tok0 = t * ttb;
    s->kt0 = 0;
    s->n = tile_cost(p, sq, t, ttb);
    s->whole = 1;
    s->slot = 0;
    pos += gridDim.x;
    return true;
  }
};

// How the work is cut: into runs; into whole items, one to a CTA; or into runs or whole items as the lengths say, which
// over pages the device alone knows.
enum Cut { kRuns, kWhole, kByLengths };

// One CTA per row tile: head by head (a head's K and V stay in L2), the deepest row tiles of each first.
template <bool kRows, class P>
__device__ __forceinline__ bool whole_seg(const P& p, int ttb, int tiles, Seg* s) {
  s->hk = blockIdx.x / tiles;
  const int tile = tiles - 1 - int(blockIdx.x % tiles), b = attn_tile_seq<kRows>(p, tile, ttb);
  s->sq = attn_seq(p, b);
  s->tok0 = attn_tile_token<kRows>(p, b, tile, ttb);
  if (s->tok0 < 0 || s->tok0 >= s->sq.nq) return false;
  s->kt0 = 0;
  s->n = tile_cost(p, s->sq, s->tok0 / ttb, ttb);
  s->whole = 1;
  s->slot = 0;
  return true;
}

// Gathered form: every row and key head has the same number of tiles, and positions run over
// rows, then key heads (the heads of a token lie together in memory).
__device__ __forceinline__ int gather_tiles(const AttnParams& p) {
  return max(1, (p.width + kTile<AttnParams> - 1) / kTile<AttnParams>);
}

__device__ __forceinline__ int64_t gather_total(const AttnParams& p) {
  const int rows = p.list && p.dense->enabled ? p.dense->listed : p.R;
  return int64_t(rows) * p.Hkv * gather_tiles(p);
}

__device__ __forceinline__ bool gather_seg(const AttnParams& p, int64_t* pos, int64_t hi, Seg* s) {
  if (*pos >= hi) return false;
  const int nt = gather_tiles(p);
  const int64_t item = *pos / nt;
  int r = int(item / p.Hkv);
  s->hk = int(item - int64_t(r) * p.Hkv);
  if (p.list && p.dense->enabled) r = __ldg(p.list + r);
  s->kt0 = int(*pos - item * nt);
  s->n = int(min(int64_t(nt - s->kt0), hi - *pos));
  s->whole = s->n == nt;
  s->slot = s->kt0 > 0 ? 0 : 1;
  *pos += s->n;
  attn_selected_seq(p, r, &s->sq.k0, &s->sq.nk);
  s->sq.q0 = r;
  s->sq.nq = 1;
  s->sq.prefix = 0;
  s->sq.ok = true;
  s->tok0 = 0;
  s->end = s->sq.nk > 0 ? p.width : 0;
  if (s->end == 0) s->n = 0;
  s->n0 = s->n;
  s->all = 0;
  return true;
}

// The rest of a segment's fields; tt: tokens of a row tile, ttb: of all row tiles of the CTA.
template <class P>
__device__ __forceinline__ void finish_seg(const P& p, int tt, int ttb, Seg* s) {
  s->end = attn_keys_end(p, s->sq, min(s->tok0 + ttb, s->sq.nq));
  if (s->end == 0) s->n = 0;
  const int end0 = attn_keys_end(p, s->sq, min(s->tok0 + tt, s->sq.nq));
  s->n0 = max(0, min(s->n, (end0 + kTile<P> - 1) / kTile<P> - s->kt0));
  s->all = p.mask ? s->sq.prefix : s->sq.prefix + s->tok0 + 1;
}

// A run has at least this many positions: shorter ones would spend their time on their start, and a row
// on joining them.
constexpr int kMinRun = 3;
__host__ __device__ __forceinline__ int64_t run_count(int64_t total, int64_t ctas) {
  const int64_t n = total / kMinRun < ctas ? total / kMinRun : ctas;
  return n < 1 ? 1 : n;
}

// The positions of the runs: run r of n begins at floor(total r / n), without a 64-bit division per run.
struct Cuts {
  int64_t each;        // total / n
  uint32_t rest, n;    // total % n
  __device__ __forceinline__ Cuts(int64_t total, uint32_t runs)
      : each(total / runs), rest(uint32_t(total - each * runs)), n(runs) {}
  __device__ __forceinline__ int64_t lo(uint32_t r) const { return each * r + rest * r / n; }  // rest * r < n * n
};

// Every thread of the CTA: this CTA's run of positions [total * i / n, total * (i + 1) / n)
// and the sequence it starts in. `scratch` holds S 64-bit words of shared memory.
template <class P>
__device__ __forceinline__ void find_run(const P& p, int ttb, int64_t* scratch, int64_t i, int64_t ctas, int cut,
                                         Misc* m) {
  for (int b = threadIdx.x; b < p.S; b += blockDim.x) scratch[b] = seq_cost(p, attn_seq(p, b), ttb);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t sum = 0;
    for (int b = lane; b < p.S; b += 32) sum += scratch[b];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (kPagedKeys<P> && cut == kByLengths) {
      int64_t keys = 0;
      int tiles = 0, most = 0;
      for (int b = lane; b < p.S; b += 32) {
        const AttnSeq s = attn_seq(p, b);
        keys += s.nk;
        most = max(most, s.nk);
        tiles += row_tiles(s, ttb);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        keys += __shfl_xor_sync(0xffffffffu, keys, d);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        tiles += __shfl_xor_sync(0xffffffffu, tiles, d);
      }
      if (lane == 0)
        m->whole = keys >= int64_t(kAttnDirectKeys) * p.S && int64_t(most) * p.S <= 2 * keys ? tiles : 0;
    }
    const int64_t n = run_count(sum, ctas);
    const Cuts cuts(sum, uint32_t(n));
    const int64_t lo = i < n ? cuts.lo(uint32_t(i)) : sum, hi = i < n ? cuts.lo(uint32_t(i) + 1) : sum;
    int64_t run = 0;
    bool found = false;
    for (int b0 = 0; b0 < p.S && !found; b0 += 32) {
      const int64_t own = b0 + lane < p.S ? scratch[b0 + lane] : 0;
      int64_t inc = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      const bool mine = lo < run + inc && lo >= run + inc - own;
      if (mine) {
        m->b = b0 + lane;
        m->base = run + inc - own;
      }
      found = __any_sync(0xffffffffu, mine);
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      m->lo = lo;
      m->hi = found ? hi : lo;
      m->total = sum;
      m->runs = int(n);
    }
  }
  __syncthreads();
}

// What the join of the rows that the border before run r cuts needs; runs = 0: nothing to join here.
struct JoinItem {
  int64_t item;          // position of the first tile of the rows' item
  int64_t each;          // Cuts of the call
  uint32_t rest;
  int32_t tiles;         // K/V tiles of the item
  int32_t runs;
  int32_t q0, nq;        // query rows of the sequence
  int32_t tok0, hk;
  int32_t pad[5];
};
static_assert(sizeof(JoinItem) == kAttnJoinBytes, "join items are laid out in the workspace");

// Run r begins with the segment s of an item of c tiles, the first at position tile0. The join is
// left to the first non-empty run that begins inside an item.
__device__ __forceinline__ void write_join(JoinItem* out, const Seg& s, int64_t tile0, int c, int64_t total, int r,
                                           int n) {
  JoinItem j{};
  j.item = tile0;
  bool own = s.kt0 > 0;
  const Cuts cuts(total, n);
  const int64_t pos = cuts.lo(r);
  for (int b = r - 1; own && b > 0 && cuts.lo(b) > tile0; --b) own = cuts.lo(b) == pos;
  j.each = cuts.each;
  j.rest = cuts.rest;
  j.tiles = c;
  j.runs = own ? n : 0;
  j.q0 = s.sq.q0;
  j.nq = s.sq.nq;
  j.tok0 = s.tok0;
  j.hk = s.hk;
  *out = j;
}

// ------------------------------------------------------------------------- waits

// Keys that lie in one page wherever a multiple of them begins: the largest power of two up to a tile that divides
// the page size.
__host__ __device__ __forceinline__ int piece_rows(int page_size) {
  const int low = page_size & -page_size;
  return low < kTile<AttnPagedParams> ? low : kTile<AttnPagedParams>;
}

// Pages follow one another in memory, so that a token of the pool has a number.
bool pages_adjoin(const AttnPagedParams& p) {
  return p.k_ps == p.page_size * p.k_ts && p.v_ps == p.page_size * p.v_ts &&
         int64_t(p.num_pages) * p.page_size <= INT32_MAX && attn_gather_supported(p.k_ts, p.v_ts);
}

// Bounded wait; also gives up when another role did.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Misc* m) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (int i = 1;; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (m->abort) return false;
    if ((i & 63) == 0 && ptx::globaltimer_ns() - t0 > kMaxWaitNs) {
      m->abort = 1;
      return false;
    }
  }
}

// Barrier of the 8 softmax warps that also tells all of them whether one has given up.
__device__ __forceinline__ bool group_bar_or(bool flag) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.or.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(flag ? 1u : 0u)
      : "memory");
  return out != 0;
}

// Visibility of 32 keys from key j on to row i of the sequence, as bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

template <class P>
__device__ __forceinline__ uint32_t seen_bits(const P& p, const AttnSeq& s, int i, int j) {
  if (p.mask == nullptr) return low_bits(s.prefix + i + 1 - j);
  const int slot = j - s.prefix;  // first of the 32 keys as a node; negative: committed keys come first
  if (slot <= -32) return 0xffffffffu;
  const int words = attn_mask_words(p);
  const int32_t* row = p.mask + int64_t(s.q0 + i) * words;
  auto word = [&](int w) { return w < words ? uint32_t(__ldg(row + w)) : 0u; };
  uint32_t bits;
  if (slot < 0) {
    bits = (word(0) & low_bits(s.nq)) << -slot | low_bits(-slot);
  } else {
    const int w = slot >> 5, sh = slot & 31;
    bits = __funnelshift_r(word(w), word(w + 1), sh) & low_bits(s.nq - slot);
  }
  return bits;
}

// K/V tile kt holds keys that some row of the segment does not see.
__device__ __forceinline__ bool tile_masked(const Seg* s, int kt, int keys) { return (kt + 1) * keys > s->all; }

// Rows rsub + kRowsPer * I of a warp's 32, all present: the token a lane wants comes from the lane that
// holds its id; the destination differs by constants but for two address bits.
template <int kRowsPer, int... I>
__device__ __forceinline__ void fetch_rows(uint32_t dst, const char* base, int tok, uint32_t ts_bytes, int rsub,
                                           std::integer_sequence<int, I...>) {
  (ptx::cp_async_16_at<kRowsPer * I * 128>(
       dst ^ (((kRowsPer * I) & 7) << 4),
       base + uint64_t(uint32_t(__shfl_sync(0xffffffffu, tok, rsub + kRowsPer * I))) * ts_bytes),
   ...);
}

// The same, for rows of which some may be absent (token -1): zeros.
template <int kRowsPer>
__device__ __forceinline__ void copy_rows(uint32_t dst, const char* base, int tok, uint32_t ts_bytes, int rsub) {
  if (__all_sync(0xffffffffu, tok >= 0)) {
    fetch_rows<kRowsPer>(dst, base, tok, ts_bytes, rsub, std::make_integer_sequence<int, 32 / kRowsPer>{});
    return;
  }
#pragma unroll 4
  for (int i = 0; i < 32 / kRowsPer; ++i) {
    const int t = __shfl_sync(0xffffffffu, tok, rsub + kRowsPer * i);
    const char* from = base + uint64_t(uint32_t(max(t, 0))) * ts_bytes;
    ptx::cp_async_16((dst ^ (((kRowsPer * i) & 7) << 4)) + kRowsPer * i * 128, from, t >= 0 ? 16u : 0u);
  }
}

// 32 N columns of scores from TMEM column `col` on.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t col, uint32_t (&s)[N][32]) {
#pragma unroll
  for (int c = 0; c < N; ++c) ptx::tc_ld_32x32b_x32(col + 32 * c, s[c]);
  ptx::tc_wait_ld();
#pragma unroll
  for (int c = 0; c < N; ++c) ptx::tc_reg_fence(s[c]);
}

template <int N>
__device__ __forceinline__ float max_score(const uint32_t (&s)[N][32]) {
  constexpr int kChains = N == 3 ? 3 : 4;
  float mx[4];
#pragma unroll
  for (int c = 0; c < kChains; ++c) {
    const int first = c * N / kChains, from = N == 2 ? 16 * (c & 1) : 0, n = N * 32 / kChains;
    mx[c] = __uint_as_float(s[first][from]);
#pragma unroll
    for (int x = 1; x < n - 1; x += 2)
      mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(s[first][from + x])), __uint_as_float(s[first][from + x + 1]));
    mx[c] = fmaxf(mx[c], __uint_as_float(s[first][from + n - 1]));
  }
  if (kChains == 3) mx[3] = mx[2];
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// Transposes 4 x 4 pieces of 16 bytes within each quad of lanes: piece r of lane i becomes piece i of
// lane r. A thread holds a row of the result; after this four lanes hold 64 contiguous bytes of one row,
// and a store instruction of the warp touches 8 lines instead of 32.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4], int lane) {
  auto swap = [&](uint4& a, uint4& b, int d) {  // lanes without bit d give b and get b, the others a
    const bool up = lane & d;
    uint4 t = up ? a : b;
    t.x = __shfl_xor_sync(0xffffffffu, t.x, d);
    t.y = __shfl_xor_sync(0xffffffffu, t.y, d);
    t.z = __shfl_xor_sync(0xffffffffu, t.z, d);
    t.w = __shfl_xor_sync(0xffffffffu, t.w, d);
    if (up) a = t; else b = t;
  };
  swap(v[0], v[1], 1);
  swap(v[2], v[3], 1);
  swap(v[0], v[2], 2);
  swap(v[1], v[3], 2);
}

__device__ __forceinline__ bool bad_bf16(uint32_t x) { return (x & 0x7F80u) == 0x7F80u; }

// -------------------------------------------------------------------- the kernel

template <int DK, int DV, Form F>
__global__ void __launch_bounds__(Cfg<DK, DV, F>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_r,
                   const __grid_constant__ typename Cfg<DK, DV, F>::Params p, int tiles, int cut, float* part, int slot_rows,
                   JoinItem* joins, WorkspaceHeader* hdr) {
  using C = Cfg<DK, DV, F>;
  constexpr int kTileKeys = C::kTileKeys, kPCol = C::kPCol;
  constexpr bool TWO = C::TWO, GATHER = C::GATHER, DENSE = F == kDense, PAGED = C::PAGED, TOKENS = C::TOKENS,
                 LISTED = F == kGather, ROWS = F == kPagedRows;
  // runs, or by the lengths (which only kPagedTwo goes by)
  const bool in_runs = F == kPagedTwo ? cut != kWhole : cut == kRuns;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::kStages;
  uint64_t* clean = bars + 2 * C::kStages;
  uint64_t* dirty = bars + 3 * C::kStages;
  uint64_t* q_full = bars + 4 * C::kStages;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;   // [2]
  uint64_t* p_ready = q_full + 4;  // [2]
  uint64_t* o_final = q_full + 6;
  uint64_t* o_free = q_full + 7;
  uint64_t* done = q_full + 8;
  uint64_t* seg_full = q_full + 9;              // [kSegRing]
  uint64_t* seg_empty = seg_full + kSegRing;    // [kSegRing]: all that read segments
  uint64_t* turn = seg_empty + kSegRing;        // [2]: it is this issuer's turn
  Seg* ring = reinterpret_cast<Seg*>(smem + C::kOffSeg);
  Misc* misc = reinterpret_cast<Misc*>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tt = GATHER ? 1 : kTileRows / p.G, ttb = C::kQTiles * tt;  // tokens of a row tile, of the CTA's row tiles

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this kernel's end itself
  if (blockIdx.x == 0 && threadIdx.x == 0 && !p.list) attn_clear_error(hdr);
  // dense form: with nothing but finite values there is nothing to clean
  const bool no_cleaning = GATHER || (DENSE && p.dense->finite);
  if (DENSE && !p.dense->enabled) {  // the gathering kernel does all rows
    if (threadIdx.x == 0 && in_runs) joins[blockIdx.x].runs = 0;
    return;
  }
  if constexpr (LISTED) {
    // (listed rows, mostly none: whole items, so that there is nothing to join)
    const int64_t total = gather_total(p), unit = p.list ? gather_tiles(p) : 1;
    const Cuts cuts(total / unit, gridDim.x);
    const int64_t lo = cuts.lo(blockIdx.x) * unit, hi = cuts.lo(blockIdx.x + 1) * unit;
    if (p.list && lo == hi) return;
    if (threadIdx.x == 0) {
      misc->lo = lo;
      misc->hi = hi;
    }
  } else if (in_runs) {
    find_run(p, ttb, reinterpret_cast<int64_t*>(smem), blockIdx.x, gridDim.x, cut, misc);
    ptx::fence_proxy_async_smem();  // the scratch lies where TMA writes next
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(full + i, GATHER ? 33 * kGatherWarps : 1);
      ptx::mbar_init(empty + i, 2);
      ptx::mbar_init(clean + i, 1);
      ptx::mbar_init(dirty + i, 1);
    }
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 2);
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(turn + g, 1);
      ptx::mbar_init(s_full + g, 1);
      ptx::mbar_init(p_ready + g, 4);
    }
    ptx::mbar_init(o_final, 2);
    ptx::mbar_init(o_free, 8);
    ptx::mbar_init(done, 2);
    for (int i = 0; i < kSegRing; ++i) {
      ptx::mbar_init(seg_full + i, 1);
      ptx::mbar_init(seg_empty + i, 10 + (GATHER ? kGatherWarps : 1));
    }
    ptx::fence_mbar_init();
    misc->abort = 0;
    misc->bad_page = 0;
    for (int i = 0; i < kSegRing; ++i) misc->bad_seg[i] = 0;
  }
  if (warp == 9) {
    ptx::tmem_alloc(&misc->tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc->tmem;
  const int whole = F == kPagedTwo && cut == kByLengths ? misc->whole : 0;  // (row tiles of a head)

  // the segment with number i, once the producer has written it (null: give up)
  auto segment = [&](int i) -> const Seg* {
    return wait_bar(seg_full + i % kSegRing, (i / kSegRing) & 1, misc) ? ring + i % kSegRing : nullptr;
  };
  if (warp >= 8) {
    // (512 x 128 or 384 x 168 registers at launch cover 256 x 176 + 256 x 80 and 256 x 208 + 128 x 72)
    if (GATHER) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (GATHER && warp == 8) {
      if (lane == 0) {  // ---------------------------------------------- segments and Q tiles
        int64_t pos = LISTED ? misc->lo : 0;
        SegIter it;
        if (!LISTED && in_runs) it.start(p, misc, ttb);
        uint32_t q_loads = 0;
        Seg sg{};
        for (int i = 0;; ++i) {
          const int64_t at = pos;
          bool more;
          if constexpr (LISTED) more = gather_seg(p, &pos, misc->hi, &sg);
          else more = !in_runs ? i == 0 && whole_seg<ROWS>(p, ttb, tiles, &sg) : it.next(p, ttb, &sg);
          if (i == 0 && in_runs && !p.list) {  // (else whole items: nothing to join)
            if (!more) joins[blockIdx.x].runs = 0;
            else if constexpr (LISTED)
              write_join(joins + blockIdx.x, sg, at - sg.kt0, gather_tiles(p), gather_total(p), blockIdx.x, gridDim.x);
            else write_join(joins + blockIdx.x, sg, it.first_tile(), it.c, misc->total, blockIdx.x, misc->runs);
          }
          if (!LISTED && more) finish_seg(p, tt, ttb, &sg);
          if (!more) sg.n = -1;
          if (i >= kSegRing && !wait_bar(seg_empty + i % kSegRing, (i / kSegRing - 1) & 1, misc)) break;
          ring[i % kSegRing] = sg;
          ptx::mbar_arrive(seg_full + i % kSegRing);
          if (!more) break;
          if (sg.n == 0) continue;
          if (q_loads > 0 && !wait_bar(q_empty, (q_loads - 1) & 1, misc)) break;
          ptx::mbar_arrive_expect_tx(q_full, C::kBlocks * uint32_t(p.G) * 128);
          ++q_loads;
#pragma unroll
          for (int h = 0; h < C::kBlocks; ++h)
            ptx::tma_load_3d(smem + h * C::kQBlock, &tm_q, q_full, 64 * h, sg.hk * p.G, sg.sq.q0);
        }
        if (q_loads) ptx::mbar_wait_bounded(q_full, (q_loads - 1) & 1, int64_t(1) << 40, kMaxWaitNs);
      }
    } else if (GATHER && warp >= 12) {  // ------------------------------------ gathering warps
      // Warp w fetches keys [32 w, 32 w + 32) of every tile, 16 bytes a lane, into the swizzled
      // layout that TMA would write. An id outside the sequence reads nothing and leaves zeros,
      // so no weight of zero meets an infinity or NaN.
      constexpr int kChunks = DK / 8;              // 16-byte pieces of a row
      constexpr int kRowsPer = 32 / kChunks;       // rows per warp instruction
      const int w = warp - 12, c = lane % kChunks, rsub = lane / kChunks;
      // the lane's place in the warp's first rows; a row's pieces are permuted by its number's low bits
      const uint32_t dst0 = ptx::smem_addr(smem + C::kOffRing) + uint32_t(c >> 3) * C::kHalf +
                            uint32_t(w * 32 + rsub) * 128 + (((c & 7) ^ rsub) << 4);
      uint32_t fills = 0, tile = 0;
      bool ok = true;
      const Seg* sg;
      bool bad_page = false;
      // What the lane reads ahead for its key of a tile: its id, or the page that it lies in.
      auto load_id = [&](int kt) {
        const int j = kt * kTileKeys + w * 32 + lane;
        if constexpr (LISTED) return j < p.width ? __ldg(p.ids + int64_t(sg->sq.q0) * p.width + j) : -1;
        else if constexpr (PAGED) return j < sg->end ? ptx::ldg_ordered(p.table + int64_t(sg->sq.k0) * p.max_pages + j / p.page_size) : -1;
        else return -1;
      };
      // tok: the lane's key as a token of k and v, -1 where it is not seen
      auto load_kv = [&](const void* src, int64_t hs, uint32_t ts_bytes, int tok, bool is_k) {
        const int st = fills % C::kStages;
        if (fills >= C::kStages &&
            !__all_sync(0xffffffffu, wait_bar(empty + st, (fills / C::kStages - 1) & 1, misc)))
          return false;
        __syncwarp();
        ++fills;
        if (is_k) {
          const uint32_t bits = __ballot_sync(0xffffffffu, tok >= 0);
          if (lane == 0) reinterpret_cast<uint32_t*>(smem + C::kOffBits)[4 * (tile % kBitsRing) + w] = bits;
          ++tile;
        }
        const char* base = static_cast<const char*>(src) + (int64_t(sg->hk) * hs + c * 8) * 2;
        copy_rows<kRowsPer>(dst0 + st * C::kTileBytes, base, tok, ts_bytes, rsub);
        ptx::cp_async_arrive(full + st);                     // when this lane's pieces have landed
        if (lane == 0) ptx::mbar_arrive(full + st);          // and the warp's word of bits is written
        return true;
      };
      for (int i = 0;; ++i) {
        sg = segment(i);
        if (!__all_sync(0xffffffffu, sg != nullptr) || sg->n < 0) break;
        const int n = sg->n, kt0 = sg->kt0, nk = sg->sq.nk, k0 = sg->sq.k0;
        int next = n > 0 ? load_id(kt0) : 0, tok = -1, tok1 = -1, tok2 = -1;  // tokens of tiles j, j - 1, j - 2
        for (int j = 0; ok && n > 0 && j < n + 2; ++j) {
          tok2 = tok1;
          tok1 = tok;
          if (j < n) {
            if constexpr (LISTED) {
              tok = next >= 0 && next < nk ? next + k0 : -1;
            } else if constexpr (PAGED) {
              const int key = (kt0 + j) * kTileKeys + w * 32 + lane;
              const bool have = next >= 0 && next < p.num_pages;
              tok = have ? next * p.page_size + key % p.page_size : -1;
              bad_page |= !have && key < sg->end;
            }
            if (j + 1 < n) next = load_id(kt0 + j + 1);
            ok = load_kv(p.k, p.k_hs, uint32_t(p.k_ts * 2), tok, true);
          }
          if (ok && j >= 2) ok = load_kv(p.v, p.v_hs, uint32_t(p.v_ts * 2), tok2, false);
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(seg_empty + i % kSegRing);
      }
      if (bad_page) misc->bad_page = 1;
      ptx::cp_async_wait_all();                    // every copy has landed before the CTA exits
    } else if (warp == 8) {  // ------------------------------------------------- TMA producer
      // One lane, or over pages all of them, each with its own pieces of a tile.
      if (PAGED || lane == 0) {
        SegIter it;
        if (whole) it.start_whole(whole);
        else if (in_runs) it.start(p, misc, ttb);
        uint32_t fills[2] = {0, 0}, q_loads = 0;  // of the ring, or of K's and V's
        bool ok = true, bad_page = false;
        Seg sg{};
        // Pages of the lane's first piece: of the tile whose K is loaded next, of the tiles before, whose V is; the next one.
        [[maybe_unused]] int rows = 1, pages[C::kAhead + 1] = {}, next_page = -1;
        // Or, token by token: the lane's keys lane, lane + 32, ... of those tiles as tokens of the pool (-1: none).
        constexpr int kOwn = kTileKeys / 32, kChunks = DK / 8, kRowsPer = 32 / kChunks;
        [[maybe_unused]] int toks[C::kAhead + 1][kOwn] = {}, next_pages[kOwn] = {};
        if constexpr (PAGED) rows = piece_rows(p.page_size);
        auto read_page = [&](int kt) {
          if constexpr (TOKENS) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
              const int j = kt * kTileKeys + lane + 32 * i, before = j - kTileKeys;
              const bool have = kt > sg.kt0 && next_pages[i] >= 0 && next_pages[i] < p.num_pages;
#pragma unroll
              for (int x = C::kAhead; x > 0; --x) toks[x][i] = toks[x - 1][i];
              toks[0][i] = have ? next_pages[i] * p.page_size + before % p.page_size : -1;
              bad_page |= !have && kt > sg.kt0 && before < sg.end;
              next_pages[i] = -1;
              if (j < sg.end)
                next_pages[i] = ptx::ldg_ordered(p.table + int64_t(sg.sq.k0) * p.max_pages + j / p.page_size);
            }
          } else if constexpr (PAGED) {
#pragma unroll
            for (int x = C::kAhead; x > 0; --x) pages[x] = pages[x - 1];
            pages[0] = next_page;
            const int j = kt * kTileKeys + lane * rows;
            next_page = -1;
            if (lane * rows < kTileKeys && j < sg.end)
              next_page = ptx::ldg_ordered(p.table + int64_t(sg.sq.k0) * p.max_pages + j / p.page_size);
          }
        };
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          const bool r = wait_bar(bar, parity, misc);
          return PAGED ? bool(__all_sync(0xffffffffu, r)) : r;
        };
        auto load_kv = [&](bool is_k, int kt) {
          uint32_t& f = fills[C::SHARED && !is_k];
          const Place at = is_k ? C::k_slot(f) : C::v_slot(f);
          const uint32_t st = at.slot, depth = !C::SHARED ? C::kStages : is_k ? C::kKSlots : C::kVSlots;
          if (f >= depth && !wait(empty + st, at.par ^ 1)) return false;
          ++f;
          uint8_t* dst = smem + C::kOffRing + C::slot_at(st);
          const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
          if constexpr (TOKENS) {
            const char* base = static_cast<const char*>(is_k ? p.k : p.v) +
                               (int64_t(sg.hk) * (is_k ? p.k_hs : p.v_hs) + (lane % kChunks) * 8) * 2;
            const uint32_t ts_bytes = uint32_t((is_k ? p.k_ts : p.v_ts) * 2);
            const int rsub = lane / kChunks;
            // (as the gathering warps place their pieces)
            const uint32_t to = ptx::smem_addr(dst) + uint32_t(lane % kChunks >> 3) * C::kHalf + uint32_t(rsub) * 128 +
                                (((lane & 7) ^ rsub) << 4);
#pragma unroll
            for (int x = 0; x < kOwn; ++x) {
              const int tok = is_k ? toks[0][x] : toks[C::kAhead][x];
              if (!__any_sync(0xffffffffu, tok >= 0)) continue;  // keys past the last one that a row sees
              copy_rows<kRowsPer>(to + x * 32 * 128, base, tok, ts_bytes, rsub);
            }
            ptx::cp_async_arrive_inc(full + st);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full + st);
          } else if constexpr (PAGED) {
            // Pieces of `rows` keys lie in one page each; the keys past the last one that a row sees are not loaded.
            const int key0 = kt * kTileKeys, pieces = min(kTileKeys / rows, (sg.end - key0 + rows - 1) / rows);
            if (lane == 0) ptx::mbar_arrive_expect_tx(full + st, uint32_t(pieces * rows * 128 * C::kVBlocks));
            __syncwarp();
            for (int x = lane; x < pieces; x += 32) {
              const int j = key0 + x * rows;
              int page = is_k ? pages[0] : pages[C::kAhead];  // of the lane's first piece, read ahead
              if (x >= 32) page = __ldg(p.table + int64_t(sg.sq.k0) * p.max_pages + j / p.page_size);
              if (page < 0 || page >= p.num_pages) {
                bad_page = true;
                page = -1;  // (zeros)
              }
#pragma unroll
              for (int h = 0; h < C::kVBlocks; ++h)
                ptx::tma_load_4d(dst + h * C::kHalf + x * rows * 128, tm, full + st, 64 * h, sg.hk, j % p.page_size, page);
            }
          } else {
            ptx::mbar_arrive_expect_tx(full + st, is_k ? C::kTileBytes : C::kVBytes);
#pragma unroll
            for (int h = 0; h < C::kVBlocks; ++h)
              ptx::tma_load_3d(dst + h * C::kHalf, tm, full + st, 64 * h, sg.hk, sg.sq.k0 + kt * kTileKeys);
            if (C::SHARED && is_k) {
#pragma unroll
              for (int h = C::kVBlocks; h < C::kBlocks; ++h)
                ptx::tma_load_3d(dst + h * C::kHalf, &tm_r, full + st, 64 * (h - C::kVBlocks), 0,
                                 sg.sq.k0 + kt * kTileKeys);
            }
          }
          if (!is_k && !no_cleaning && tile_masked(&sg, kt, kTileKeys) && lane == 0) ptx::mbar_arrive(dirty + st);
          return true;
        };
        for (int i = 0;; ++i) {
          const bool more = !in_runs ? i == 0 && whole_seg<ROWS>(p, ttb, tiles, &sg)
                            : whole  ? it.next_whole(p, ttb, &sg)
                                     : it.next(p, ttb, &sg);
          if (i == 0 && in_runs && lane == 0) {
            if (more && !whole) write_join(joins + blockIdx.x, sg, it.first_tile(), it.c, misc->total, blockIdx.x, misc->runs);
            else joins[blockIdx.x].runs = 0;
          }
          if (more) finish_seg(p, tt, ttb, &sg); else sg.n = -1;
          if (i >= kSegRing && !wait(seg_empty + i % kSegRing, (i / kSegRing - 1) & 1)) break;
          if (lane == 0) {
            ring[i % kSegRing] = sg;
            ptx::mbar_arrive(seg_full + i % kSegRing);
          }
          if (!more) break;
          if (sg.n == 0) continue;
          if (q_loads > 0 && !wait(q_empty, (q_loads - 1) & 1)) break;
          ++q_loads;
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(q_full, C::kQTiles * C::kBlocks * uint32_t(tt * p.G) * 128);
            for (int g = 0; g < C::kQTiles; ++g)
#pragma unroll
              for (int h = 0; h < C::kBlocks; ++h)
                ptx::tma_load_3d(smem + g * C::kQBytes + h * C::kQBlock, &tm_q, q_full, 64 * h, sg.hk * p.G,
                                 sg.sq.q0 + sg.tok0 + g * tt);
          }
          read_page(sg.kt0);
          for (int j = 0; ok && j < sg.n + C::kAhead; ++j) {
            read_page(sg.kt0 + j + 1);
            if (j < sg.n) ok = load_kv(true, sg.kt0 + j);
            if (ok && j >= C::kAhead) ok = load_kv(false, sg.kt0 + j - C::kAhead);
          }
          if (!ok) break;
        }
        if (PAGED && bad_page) misc->bad_page = 1;
        if (TOKENS) ptx::cp_async_wait_all();
        // every copy armed above lands before the CTA exits
        auto land = [&](uint32_t first, uint32_t depth, uint32_t f) {
          for (uint32_t s2 = 0; s2 < depth && s2 < f; ++s2)
            ptx::mbar_wait_bounded(full + first + s2, ((f - 1 - s2) / depth) & 1, int64_t(1) << 40, kMaxWaitNs);
        };
        land(0, C::SHARED ? C::kKSlots : C::kStages, fills[0]);
        if (C::SHARED) land(C::kKSlots, C::kVSlots, fills[1]);
        if (q_loads) ptx::mbar_wait_bounded(q_full, (q_loads - 1) & 1, int64_t(1) << 40, kMaxWaitNs);
      }
    } else if (warp == 9 || warp == 10) {
      if (lane == 0) {  // ------------------------------------ MMA issuers, one per softmax group
        const int g = warp - 9;
        // Descriptors of the Q tile and of the first ring slot; the others differ in the address field
        // (bytes / 16) only, so a step is one addition.
        const uint64_t q_desc =
            ptx::smem_desc_kmajor_sw128(ptx::smem_addr(smem + (TWO ? g * C::kQBytes : 0)));
        const uint64_t k_desc = ptx::smem_desc_kmajor_sw128(ptx::smem_addr(smem + C::kOffRing));
        const uint64_t v_desc = ptx::smem_desc_mnmajor_sw128(ptx::smem_addr(smem + C::kOffRing), C::kHalf);
        constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(kTileRows, kTileKeys);
        constexpr uint32_t idesc_o = ptx::idesc_bf16_f32_bn(kTileRows, DV);
        const uint32_t s_acc = tmem + g * 128, o_acc = tmem + 256 + g * DV;
        uint32_t use = 0, q_uses = 0, p_uses = 0, turns = 0;  // ring uses before this segment, Q tiles, P tiles
        uint32_t clean_par = 0;                    // bit per ring slot
        bool ok = true;
        const Seg* sg;
        auto landed = [&](Place u) {
          const bool r = wait_bar(full + u.slot, u.par, misc);
          if (GATHER || TOKENS) ptx::fence_proxy_async_smem();  // the tile was written by ordinary copies
          return r;
        };
        // The issuers take turns, a tile's P V and the next tile's Q K^T at a time. Left to themselves
        // the groups fall into step: both do their softmax while the tensor core idles, then both wait
        // for it (7.8 against 6.1 ms for one 32,768-token prompt of 32 heads).
        if (g == 1) ptx::mbar_arrive(turn);
        auto my_turn = [&]() {
          const bool r = wait_bar(turn + g, turns & 1, misc);
          ++turns;
          return r;
        };
        auto qk = [&](Place u, bool pass) {
          const uint64_t b = k_desc + (C::slot_at(u.slot) >> 4);
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            // handed on a little early: the other's first product follows without a gap
            if (kk == DK / 32 && pass) ptx::mbar_arrive(turn + (g ^ 1));
            const uint32_t q_step = ((kk >> 2) * C::kQBlock + (kk & 3) * 32) >> 4;
            const uint32_t step = ((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4;
            ptx::tc_mma_f16(s_acc, q_desc + q_step, b + step, idesc_s, kk > 0 ? 1u : 0u);
          }
          ptx::tc_commit(s_full + g);
        };
        auto pv = [&](Place u, bool first) {
          const uint64_t b = v_desc + (C::slot_at(u.slot) >> 4);
#pragma unroll
          for (int kk = 0; kk < kTileKeys / 16; ++kk)
            ptx::tc_mma_f16_ts(o_acc, s_acc + kPCol + kk * 8, b + kk * (2048 >> 4), idesc_o,
                               (kk > 0 || !first) ? 1u : 0u);
        };
        for (int i = 0; ok && (sg = segment(i)) != nullptr && sg->n >= 0; ++i) {
          const int n = sg->n, kt0 = sg->kt0;
          if (n > 0) {
            // Every tile of the ring is waited for in order and released by both issuers, used or not:
            // a slot's barriers then never get two phases ahead of either.
            const int n0 = TWO && g == 0 ? sg->n0 : n;
            auto mine = [&](int j) { return TWO ? j < n0 : (j & 1) == g; };
            const int last = TWO ? n0 - 1 : n - 1 - ((n - 1 - g) & 1);  // the group's last tile (< 0: none)
            auto score = [&](int j, Place u, bool pass) {
              if (mine(j)) {
                qk(u, pass);
                if (j == last) ptx::tc_commit(q_empty);
                ptx::tc_commit(empty + u.slot);
              } else {
                ptx::mbar_arrive(empty + u.slot);
                if (pass) ptx::mbar_arrive(turn + (g ^ 1));
              }
            };
            if (!(ok = wait_bar(q_full, q_uses & 1, misc))) break;
            if (last < 0) ptx::mbar_arrive(q_empty);
            for (int j = 0; j < min(n, C::kAhead); ++j) {
              const Place u = C::k_place(use, j);
              if (!(ok = landed(u))) break;
              ptx::tc_fence_after();
              score(j, u, false);
            }
            if (!ok) break;
            if (q_uses > 0 && !(ok = wait_bar(o_free, (q_uses - 1) & 1, misc))) break;
            ++q_uses;
            for (int j = 0; j < n; ++j) {
              const int jk = j + C::kAhead;
              const Place uk = C::k_place(use, jk), uv = C::v_place(use, j, n);
              if (jk < n && !(ok = landed(uk))) break;
              if (!(ok = landed(uv))) break;
              const uint32_t slot = uv.slot;
              const bool masked = !no_cleaning && tile_masked(sg, kt0 + j, kTileKeys);
              if (mine(j)) {
                if (masked && !(ok = wait_bar(clean + slot, (clean_par >> slot) & 1, misc))) break;
                if (!(ok = wait_bar(p_ready + g, p_uses & 1, misc))) break;
                ++p_uses;
                if (!(ok = my_turn())) break;
                ptx::tc_fence_after();
                pv(uv, TWO ? j == 0 : j < 2);
                if (jk < n) score(jk, uk, true);
                else ptx::mbar_arrive(turn + (g ^ 1));
                ptx::tc_commit(empty + slot);
              } else {
                if (TWO) {  // (one: a turn belongs to a pair of tiles)
                  if (!(ok = my_turn())) break;
                  ptx::mbar_arrive(turn + (g ^ 1));
                }
                if (jk < n) score(jk, uk, false);
                ptx::mbar_arrive(empty + slot);
              }
              if (masked) clean_par ^= 1u << slot;
            }
            if (ok && !TWO && g == 1 && (n & 1)) {
              if ((ok = my_turn())) ptx::mbar_arrive(turn);
            }
            if (!ok) break;
            ptx::tc_commit(o_final);
            use += 2 * n;
          }
          ptx::mbar_arrive(seg_empty + i % kSegRing);
        }
        ptx::tc_commit(done);  // every MMA issued above completes before TMEM is freed
        ptx::mbar_wait_bounded(done, 0, int64_t(1) << 40, kMaxWaitNs);
      }
    } else if (GATHER) {  // (warp 11)
      if (blockIdx.x == 0) attn_check(p, hdr);
    } else {  // --------------------------------------------------------- V cleaning warp
      uint32_t use = 0, dirty_par = 0;
      bool ok = true;
      const Seg* sg;
      for (int i = 0; ok && (sg = segment(i)) != nullptr && sg->n >= 0; ++i) {
        const int n = sg->n, kt0 = sg->kt0;
        for (int j = no_cleaning ? n : max(0, sg->all / kTileKeys - kt0); j < n; ++j) {
          const Place u = C::v_place(use, j, n);
          const uint32_t slot = u.slot;
          // The producer says when it has begun to fill the slot with this tile: the slot's
          // full barrier is then in this tile's phase, not one of the same parity before.
          ok = __all_sync(0xffffffffu, wait_bar(dirty + slot, (dirty_par >> slot) & 1, misc) &&
                                           wait_bar(full + slot, u.par, misc));
          dirty_par ^= 1u << slot;
          if (!ok) break;
          uint8_t* v = smem + C::kOffRing + C::slot_at(slot);
          // Keys before `seen` are seen by every row and stay as they are; keys from `live` on by none.
          const int base = (kt0 + j) * kTileKeys, live = sg->end - base, seen = max(0, sg->all - base);
          bool bad = false;
          // 16 bytes per lane; block h holds columns [64 h, 64 h + 64) of all keys, 128 bytes a key
          for (int h = 0; h < C::kVBlocks; ++h) {
            uint4* block = reinterpret_cast<uint4*>(v + h * C::kHalf);
            const int first = seen * 8, checked = min(live, kTileKeys) * 8;
            // eight pieces at a time are read and tested together; they are all but always as they should be
            for (int x0 = first + lane; x0 < checked; x0 += 8 * 32) {
              uint4 q[8];
              uint32_t wild = 0;
#pragma unroll
              for (int y = 0; y < 8; ++y)
                q[y] = x0 + 32 * y < checked ? block[x0 + 32 * y] : make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                // an exponent of all ones carries into bit 15 or 31
                constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u;
                wild |= ((q[y].x & kExp) + kOne) | ((q[y].y & kExp) + kOne) | ((q[y].z & kExp) + kOne) |
                        ((q[y].w & kExp) + kOne);
              }
              if (wild & 0x80008000u) {
                bad = true;
#pragma unroll 1
                for (int x = x0; x < min(checked, x0 + 8 * 32); x += 32) {
                  uint4 f = block[x];
                  uint32_t* e = reinterpret_cast<uint32_t*>(&f);
#pragma unroll
                  for (int y = 0; y < 4; ++y) {
                    if (bad_bf16(e[y])) e[y] &= 0xFFFF0000u;
                    if (bad_bf16(e[y] >> 16)) e[y] &= 0x0000FFFFu;
                  }
                  block[x] = f;
                }
              }
            }
#pragma unroll 4
            for (int x = max(first, checked) + lane; x < kTileKeys * 8; x += 32) block[x] = make_uint4(0, 0, 0, 0);
          }
          if (bad) misc->bad_seg[i % kSegRing] = i + 1;
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(clean + slot);
        }
        use += 2 * n;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(seg_empty + i % kSegRing);
      }
      __syncwarp();
      if (blockIdx.x == 0) attn_check(p, hdr);
    }
  } else {  // -------------------------------------------------------------- softmax groups
    if (GATHER) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int g = warp >> 2;                 // group
    const int row = threadIdx.x & 127;       // row of the tile
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + g * 128;
    const uint32_t o_col = tmem + lane_base + 256 + g * DV;
    const int tok_in = row / p.G, head_in = row - tok_in * p.G;
    const float c2 = p.scale * kLog2e;
    uint32_t s_uses = 0, finals = 0, tile = 0;
    bool ok = true;
    for (int is = 0;; ++is) {
      const Seg* sg = segment(is);
      ok = __all_sync(0xffffffffu, sg != nullptr);
      if (TWO ? !ok : group_bar_or(!ok)) break;
      if (sg->n < 0) break;
      const int i = sg->tok0 + (TWO ? g * tt : 0) + tok_in;   // token of the sequence
      const bool valid = tok_in < tt && i < sg->sq.nq;
      // a warp without any row only keeps the barriers going (two row tiles: not worth a test)
      const bool live = TWO || __any_sync(0xffffffffu, valid);
      const int n_all = sg->n, n = TWO && g == 0 ? sg->n0 : n_all;
      const int first = TWO ? 0 : g, step = TWO ? 1 : 2;
      float m = -INFINITY;
      uint64_t l2[2] = {0, 0};
      for (int j = first; j < n; j += step) {
        const int kt = sg->kt0 + j;
        uint4 seen;
        if (DENSE && live) {  // the row's bits of the tile, 16-byte aligned words
          const int words = attn_mask_words(p), im = min(i, sg->sq.nq - 1);
          seen = __ldg(reinterpret_cast<const uint4*>(p.mask + int64_t(sg->sq.q0 + im) * words) + kt);
        }
        ok = __all_sync(0xffffffffu, wait_bar(s_full + g, s_uses & 1, misc));
        if (!ok) break;
        ++s_uses;
        if (!live) {
          if (lane == 0) ptx::mbar_arrive(p_ready + g);
          continue;
        }
        ptx::tc_fence_after();
        // Keys that some row does not see: -inf over their scores in TMEM, 32 columns at a time and only
        // where a row of the warp needs it. (As straight code on the 128 registers below it took three
        // times as long: it runs once or twice per row tile and is fetched anew each time.)
        const uint32_t* w = reinterpret_cast<const uint32_t*>(smem + C::kOffBits) + 4 * ((tile + j) % kBitsRing);
        if (GATHER ? (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu : !DENSE && tile_masked(sg, kt, kTileKeys)) {
          const int im = min(i, sg->sq.nq - 1);
#pragma unroll 1
          for (int c = 0; c < C::kScoreCols; ++c) {
            const uint32_t bits = GATHER ? w[c] : seen_bits(p, sg->sq, im, kt * kTileKeys + 32 * c);
            if (!__any_sync(0xffffffffu, bits != 0xffffffffu)) continue;
            uint32_t x32[32];
            ptx::tc_ld_32x32b_x32(s_col + 32 * c, x32);
            ptx::tc_wait_ld();
            ptx::tc_reg_fence(x32);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!((bits >> x) & 1u)) x32[x] = 0xFF800000u;  // -inf
            ptx::tc_st_32x32b_x32(s_col + 32 * c, x32);
          }
          ptx::tc_wait_st();
        }
        // Two row tiles: the row's 128 scores stay in registers. One row tile: 64 at a time, the upper ones last,
        // and the lower ones are read again for their weights; half the code and registers, which is what
        // counts beside the gathering warps (350 -> 319 us for 2048 rows x 2052 ids of 64 heads; with two
        // row tiles the second read costs 5 % at 32,768 tokens).
        constexpr int kHeld = TWO || C::kScoreCols == 3 ? C::kScoreCols : 2, kReads = C::kScoreCols / kHeld;
        uint32_t s[kHeld][32];
        float mt = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < kReads; ++h) {
          load_scores<kHeld>(s_col + 32 * kHeld * h, s);
          if (DENSE) {
#pragma unroll
            for (int c = 0; c < kHeld; ++c) {
              const uint32_t bits = c == 0 ? seen.x : c == 1 ? seen.y : c == 2 ? seen.z : seen.w;
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (!((bits >> x) & 1u)) s[c][x] = 0xFF800000u;
            }
          }
          mt = fmaxf(mt, max_score<kHeld>(s));
        }
        const bool grow = mt > m && (mt - m) * c2 > kLazy;
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? mt : m;
          const float f = grow ? ptx::exp2_approx((m - mn) * c2) : 1.0f;
          m = mn;
          if (j != first) {  // S of this tile was issued after the last P V of the group: O is at rest
            const uint64_t ff = ptx::pack_f32x2(f, f);
            l2[0] = ptx::fma_f32x2(l2[0], ff, 0);
            l2[1] = ptx::fma_f32x2(l2[1], ff, 0);
#pragma unroll
            for (int c = 0; c < DV / 16; ++c) {
              uint32_t o[16];
              ptx::tc_ld_32x32b_x16(o_col + 16 * c, o);
              ptx::tc_wait_ld();
              ptx::tc_reg_fence(o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              ptx::tc_st_32x32b_x16(o_col + 16 * c, o);
            }
          }
        }
        const float nb = m == -INFINITY ? 0.0f : -m * c2;
        const uint64_t c22 = ptx::pack_f32x2(c2, c2), nb2 = ptx::pack_f32x2(nb, nb);
#pragma unroll 1
        for (int h = kReads - 1; h >= 0; --h) {
          if (kReads > 1 && h == 0) load_scores<kHeld>(s_col, s);
#pragma unroll
          for (int c = 0; c < kHeld; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const uint64_t e = ptx::fma_f32x2(
                  ptx::pack_f32x2(__uint_as_float(s[c][2 * x]), __uint_as_float(s[c][2 * x + 1])), c22, nb2);
              float a, b;
              ptx::unpack_f32x2(e, a, b);
              a = ptx::exp2_approx(a);
              b = ptx::exp2_approx(b);
              l2[x & 1] = ptx::add_f32x2(l2[x & 1], ptx::pack_f32x2(a, b));
              pk[x] = ptx::pack_bf16(a, b);
            }
            ptx::tc_st_32x32b_x16(s_col + kPCol + 16 * (kHeld * h + c), pk);
          }
        }
        ptx::tc_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_ready + g);
      }
      if (TWO && !ok) break;
      float l;
      {
        float a, b, c, d;
        ptx::unpack_f32x2(l2[0], a, b);
        ptx::unpack_f32x2(l2[1], c, d);
        l = (a + b) + (c + d);
      }
      // ------------------------------------------------------------------------ epilogue
      float w0 = 1.0f, w1 = 0.0f;                       // factors of the groups' accumulators
      bool has0 = TWO ? n > 0 : n_all > 0, has1 = !TWO && n_all > 1;
      if (!TWO) {  // add up the two groups' statistics
        float2* st = reinterpret_cast<float2*>(smem + C::kOffStat);
        st[g * kTileRows + row] = make_float2(m, l);
        if (group_bar_or(!ok)) break;
        const float2 a = st[row], b = st[kTileRows + row];
        m = fmaxf(a.x, b.x);
        const float mb = m == -INFINITY ? 0.0f : m;
        w0 = ptx::exp2_approx((a.x - mb) * c2);
        w1 = ptx::exp2_approx((b.x - mb) * c2);
        if (m == -INFINITY) w0 = w1 = 1.0f;  // nothing, or a NaN that l carries on
        l = a.y * w0 + b.y * w1;
      }
      if (n_all > 0) ok = __all_sync(0xffffffffu, wait_bar(o_final, finals & 1, misc));
      if (TWO ? !ok : group_bar_or(!ok)) break;  // (one: the statistics have been read, too)
      ptx::tc_fence_after();
      const bool none = m == -INFINITY && l == 0.0f;
      const bool fix = !GATHER && n_all > 0 && misc->bad_seg[is % kSegRing] == is + 1;
      const int64_t grow_row = int64_t(sg->sq.q0) + i;
      const int head = sg->hk * p.G + head_in;
      const float inv = none ? 0.0f : 1.0f / l;
      // where this lane's pieces of the quad's rows go
      int64_t out_at[4];
      {
        const int64_t own = valid ? grow_row * p.o_ts + int64_t(head) * p.o_hs : -1;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          out_at[r] = __shfl_sync(0xffffffffu, own, (lane & 28) + r);
          if (out_at[r] >= 0) out_at[r] += (TWO ? 0 : g * (DV / 2)) + 8 * (lane & 3);
        }
      }
      const int prow = TWO ? g * kTileRows + row : row;
      float* pslot = part + (size_t(blockIdx.x) * 2 + sg->slot) * size_t(slot_rows) * (DV + 2);
      // columns of this thread: all (two), or the group's half (one)
      constexpr int kCols = TWO ? DV : DV / 2;
      const int col0 = TWO ? 0 : g * kCols;
      const uint32_t oa = tmem + lane_base + 256 + (TWO ? g * DV : 0) + col0, ob = tmem + lane_base + 256 + DV + col0;
#pragma unroll 1
      for (int c = 0; live && c < kCols / 32; ++c) {
        uint32_t o[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = 0;
        if (has0) {
          ptx::tc_ld_32x32b_x32(oa + 32 * c, o);
          ptx::tc_wait_ld();
          ptx::tc_reg_fence(o);
        }
        if (!TWO) {
          uint32_t o1[32];
          if (has1) {
            ptx::tc_ld_32x32b_x32(ob + 32 * c, o1);
            ptx::tc_wait_ld();
            ptx::tc_reg_fence(o1);
          }
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            float v = __uint_as_float(o[x]) * w0;
            if (has1) v = fmaf(__uint_as_float(o1[x]), w1, v);
            o[x] = __float_as_uint(v);
          }
        }
        if (fix && valid && !none) {
          // infinities and NaN that the cleaning took out of V: a row that sees them gets them back
          const int j0 = max(sg->kt0 * kTileKeys, sg->all);
          const int j1 = min((sg->kt0 + n_all) * kTileKeys, sg->end);
          const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + int64_t(sg->hk) * p.v_hs + col0 + 32 * c;
          for (int j = j0; j < j1; ++j) {
            if (!attn_sees(p, sg->sq, i, j)) continue;
            int64_t at = (int64_t(sg->sq.k0) + j) * p.v_ts;
            if constexpr (PAGED) {
              bool none_such = false;
              const int page = attn_page(p, sg->sq.k0, j, &none_such);
              if (none_such) continue;
              at = int64_t(page) * p.v_ps + (j % p.page_size) * p.v_ts;
            }
            const uint32_t* e = reinterpret_cast<const uint32_t*>(v + at);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const uint32_t u = __ldg(e + x);
              if (bad_bf16(u)) o[2 * x] = __float_as_uint(__uint_as_float(o[2 * x]) + __uint_as_float(u << 16));
              if (bad_bf16(u >> 16))
                o[2 * x + 1] = __float_as_uint(__uint_as_float(o[2 * x + 1]) + __uint_as_float(u & 0xFFFF0000u));
            }
          }
        }
        if (sg->whole) {
          uint4 u[4];
          uint32_t* e = reinterpret_cast<uint32_t*>(u);
#pragma unroll
          for (int x = 0; x < 16; ++x)
            e[x] = none ? 0u
                        : ptx::pack_bf16(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
          quad_transpose(u, lane);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (out_at[r] >= 0)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + out_at[r] + 32 * c) = u[r];
          }
        } else {
          float* dst = pslot + col0 + 32 * c + 4 * (lane & 3);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 u[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              u[x] = make_uint4(o[16 * h + 4 * x], o[16 * h + 4 * x + 1], o[16 * h + 4 * x + 2], o[16 * h + 4 * x + 3]);
            quad_transpose(u, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int to = (prow & ~3) + r;
              if (to < slot_rows) *reinterpret_cast<uint4*>(dst + size_t(to) * DV + 16 * h) = u[r];
            }
          }
        }
      }
      if (TWO || g == 0) {
        if (sg->whole) {
          if (valid && p.lse)
            p.lse[grow_row * p.Hq + head] = none ? -INFINITY : (m * c2 + log2f(l)) * kLn2;
        } else if (prow < slot_rows) {
          pslot[size_t(slot_rows) * DV + 2 * prow] = m;
          pslot[size_t(slot_rows) * DV + 2 * prow + 1] = l;
        }
      }
      if (n_all > 0) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(o_free);
        ++finals;
      }
      tile += n_all;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(seg_empty + is % kSegRing);
    }
    ptx::tc_fence_before();
  }
  // ------------------------------------------------------------------------------ teardown
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0 && misc->abort) record_error(hdr, KPOOL_ERR_DEVICE_TIMEOUT);
  if (PAGED && threadIdx.x == 0 && misc->bad_page) record_error(hdr, KPOOL_ERR_INVALID_ARG);
  if (warp == 9) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------- join
//
// CTA x adds up, in the order of the runs, the partial results of the rows that the border
// before run x + 1 cuts (if that run was the first to begin inside them: its producer left the
// item's data). A lane holds D / 32 channels of a row. kSplit: the 8 warps of a CTA share four
// rows and each takes every eighth run, four at a time (few items, each cut into many runs: reading
// one run after the other made 100 us of 154); else a warp has two rows, most of them cut into
// two or three runs, and reads two at a time. What is read is a few MB just written; the join adds
// 9 to 18 us to a call of 100 us and more. (Four rows a warp, one run at a time: 138 against 136 us
// for 16 decode tokens over caches of up to 32,767 keys, prompts alike.)

template <int D>
struct JoinRow {
  static constexpr int kPer = D / 32;
  float acc[kPer], m, l;
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int y = 0; y < kPer; ++y) acc[y] = 0.0f;
  }
  // adds the part (o, pm, pl); one without any weight adds nothing, with a NaN among its scores its sum passes on
  __device__ __forceinline__ void add(const float (&o)[kPer], float pm, float pl, float c2) {
    const float mn = fmaxf(m, pm), base = mn == -INFINITY ? 0.0f : mn;
    const float f = m == -INFINITY ? 1.0f : exp2f((m - base) * c2);
    const float w = pm == -INFINITY ? 1.0f : exp2f((pm - base) * c2);
    l = l * f + pl * w;
#pragma unroll
    for (int y = 0; y < kPer; ++y) acc[y] = acc[y] * f + o[y] * w;
    m = mn;
  }
};

template <int D, bool kSplit>
__global__ void __launch_bounds__(256)
    attn_join_kernel(const __grid_constant__ AttnParams p, int tt, const JoinItem* joins, const float* part,
                     int slot_rows) {
  constexpr int kPer = D / 32, kRows = kSplit ? 4 : 2, kJoinBatch = kSplit ? 4 : 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // in every CTA: the call ends after both kernels have
  const JoinItem it = joins[blockIdx.x + 1];
  if (it.runs == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the runs that hold tiles of the item: from `first` while they begin before its end
  auto run_lo = [&](int r) { return it.each * r + it.rest * uint32_t(r) / uint32_t(it.runs); };
  int first = blockIdx.x;
  while (first > 0 && run_lo(first) > it.item) --first;
  const float c2 = p.scale * kLog2e;
  const size_t stride = size_t(slot_rows) * (D + 2);
  int vr[kRows], tok[kRows];
  JoinRow<D> row[kRows];
  bool any = false;
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    vr[x] = (kSplit ? int(blockIdx.y) : int(blockIdx.y) * 8 + warp) * kRows + x;
    const int q_tile = vr[x] / kTileRows, in = (vr[x] - q_tile * kTileRows) / p.G;
    tok[x] = vr[x] < slot_rows && in < tt && it.tok0 + q_tile * tt + in < it.nq ? it.tok0 + q_tile * tt + in : -1;
    any |= tok[x] >= 0;
    row[x].clear();
  }
  if (!any) return;
  const int64_t end = it.item + it.tiles;
  for (int r0 = first + (kSplit ? warp : 0); r0 < it.runs && run_lo(r0) < end;
       r0 += kJoinBatch * (kSplit ? 8 : 1)) {
    float o[kJoinBatch][kRows][kPer];
    float2 ml[kJoinBatch][kRows];
    bool has[kJoinBatch];
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) {
      const int r = r0 + b * (kSplit ? 8 : 1);
      const int64_t lo = run_lo(r), hi = run_lo(r + 1);
      has[b] = r < it.runs && lo < end && hi > it.item && hi > lo;
      if (!has[b]) continue;
      const float* s = part + (size_t(r) * 2 + (lo > it.item ? 0 : 1)) * stride;
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        if (tok[x] < 0) continue;
        ml[b][x] = *reinterpret_cast<const float2*>(s + size_t(slot_rows) * D + 2 * vr[x]);
        const float* at = s + size_t(vr[x]) * D + kPer * lane;
        if (D == 128) {
          const float4 f = *reinterpret_cast<const float4*>(at);
          o[b][x][0] = f.x;
          o[b][x][1] = f.y;
          o[b][x][kPer - 2] = f.z;
          o[b][x][kPer - 1] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(at);
          o[b][x][0] = f.x;
          o[b][x][1] = f.y;
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b)
#pragma unroll
      for (int x = 0; x < kRows; ++x)
        if (has[b] && tok[x] >= 0) row[x].add(o[b][x], ml[b][x].x, ml[b][x].y, c2);
  }
  if (kSplit) {  // warp x < 4 finishes row x, adding the warps' parts in their order
    __shared__ float s_o[8][kRows][D];
    __shared__ float2 s_ml[8][kRows];
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
#pragma unroll
      for (int y = 0; y < kPer; ++y) s_o[warp][x][kPer * lane + y] = row[x].acc[y];
      if (lane == 0) s_ml[warp][x] = make_float2(row[x].m, row[x].l);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
      if (x != warp) {
        tok[x] = -1;
        continue;
      }
      row[x].clear();
      for (int w = 0; w < 8; ++w) {
        float o[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y) o[y] = s_o[w][x][kPer * lane + y];
        row[x].add(o, s_ml[w][x].x, s_ml[w][x].y, c2);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    if (tok[x] < 0) continue;
    const bool none = row[x].m == -INFINITY && row[x].l == 0.0f;
    const float inv = none ? 0.0f : 1.0f / row[x].l;
    const int head = it.hk * p.G + (vr[x] % kTileRows) % p.G;
    const int64_t at = int64_t(it.q0) + tok[x];
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + at * p.o_ts + int64_t(head) * p.o_hs + kPer * lane;
#pragma unroll
    for (int y = 0; y < kPer; y += 2)
      *reinterpret_cast<uint32_t*>(dst + y) =
          none ? 0u : ptx::pack_bf16(row[x].acc[y] * inv, row[x].acc[y + 1] * inv);
    if (lane == 0 && p.lse)
      p.lse[at * p.Hq + head] = none ? -INFINITY : (row[x].m * c2 + log2f(row[x].l)) * kLn2;
  }
}

template <int DK, int DV, Form F>
cudaError_t launch(const typename Cfg<DK, DV, F>::Params& p, char* ws, cudaStream_t stream) {
  using C = Cfg<DK, DV, F>;
  constexpr bool GATHER = C::GATHER, LISTED = F == kGather;
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int tt = GATHER ? 1 : kTileRows / p.G, ttb = C::kQTiles * tt;
  CUtensorMap tq, tk, tv, tr;
  if (!make_tmap_bf16_heads(&tq, p.q, uint64_t(p.R), uint64_t(p.Hq), DK, p.q_ts, p.q_hs, uint32_t(tt), uint32_t(p.G)))
    return cudaErrorInvalidValue;
  tk = tv = tr = tq;  // (gathered: not used, keys and values come by plain copies)
  if constexpr (C::PAGED && !GATHER && !C::TOKENS) {
    const uint32_t rows = uint32_t(piece_rows(p.page_size));
    if (!make_tmap_bf16_pages(&tk, p.k, uint64_t(p.num_pages), uint64_t(p.page_size), uint64_t(p.Hkv), DK, p.k_ps, p.k_ts,
                              p.k_hs, rows) ||
        !make_tmap_bf16_pages(&tv, p.v, uint64_t(p.num_pages), uint64_t(p.page_size), uint64_t(p.Hkv), DV, p.v_ps, p.v_ts,
                              p.v_hs, rows))
      return cudaErrorInvalidValue;
  } else if (!GATHER && !C::TOKENS) {
    if (!make_tmap_bf16_heads(&tk, p.k, uint64_t(p.T), uint64_t(p.Hkv), DV, p.k_ts, p.k_hs, C::kTileKeys, 1) ||
        !make_tmap_bf16_heads(&tv, p.v, uint64_t(p.T), uint64_t(p.Hkv), DV, p.v_ts, p.v_hs, C::kTileKeys, 1))
      return cudaErrorInvalidValue;
    if constexpr (C::SHARED)
      if (!make_tmap_bf16_heads(&tr, p.kr, uint64_t(p.T), 1, DK - DV, p.kr_ts, DK - DV, C::kTileKeys, 1))
        return cudaErrorInvalidValue;
  }
  const int64_t tiles = attn_tiles<GATHER>(p.R, p.S, ttb);  // (gathered: a row each)
  const int64_t items = tiles * p.Hkv;
  // Equal runs of all K/V tiles fill the SMs whatever the lengths are, and cost a join (about five tiles' time)
  // and the starts of the items they cut. Whole items, one to a CTA, are taken instead (us, 32 / 8 heads of 128
  // unless said otherwise):
  //  - where an item has few tiles at most: one prompt of 600 tokens 16 against 28, of 900 21 against 36, a
  //    decode step at 900 keys 14 against 22;
  //  - for one or two items per SM of like sequences, which end about together: 1,500 tokens 38 against 46,
  //    4 x 300 22 against 28, 1,400 of 64 / 1 heads 47 against 62 (32 x 256, ten per SM: 87 against 68);
  //  - for long sequences with many items (deepest first, a head's K and V in L2): 32,768 tokens 6.1 against
  //    6.5 ms;
  //  - for gathered items, all of the same tiles, where their rounding up to the SMs costs less than the join.
  // The second rule goes by the mean of the keys. Where they have a shared part it is kept to prompts as a whole: chunks
  // can be as unlike as the caches before them (16 heads: prompts 2 x 1,024 33 against 47, of 100, 2,000 and 700 62 / 61;
  // chunks of 4 x 512 over 2,000 keys each 51 / 65, but 8 x 256 over a cache of 5,000 and seven of 300 101 / 49).
  // Over pages only the device knows the lengths; what the table holds bounds a sequence's (whole items / runs):
  //  - few tiles at most, up to one item per SM: pages of 16, 16 decode steps of 900 keys 18.5 / 26.6, 4 of 100 10.3 /
  //    14.4 (two items per SM, of 1,000 keys and, the others, 50: 31 / 24.5);
  //  - perhaps long: kByLengths, pages of 64. 8 chunks of 1,024 rows over 30,000 keys 2,740 / 3,080 to 3,510, over 8,192
  //    749 / 782, 2 x 4,096 over 60,000 5,320 / 5,870; but prompts 64 x 256 184 / 136, 128 x 100 176 / 92, 16 x 2,048 686
  //    / 598, and lengths of 1,000 to 30,000 side by side (the longest more than twice their mean) 1,597 / 1,393;
  //  - token by token (kPagedTokens) never: 8 x 1,024 over 20,000 keys 5,750 / 5,600, 128 x 100 238 / 158.
  const int64_t nt = (p.width + C::kTileKeys - 1) / C::kTileKeys;
  const bool even = LISTED && (nt + 2) * ((items + sms - 1) / sms) <= items * nt / sms + 5;
  const int ctas = sms < kAttnMaxRuns ? sms : kAttnMaxRuns;
  const bool many = C::TWO && items >= int64_t(kAttnDirectItems) * sms;
  bool small, direct = p.S > kAttnMaxRunSeqs;
  int cut = kRuns;
  if constexpr (C::PAGED) {
    small = items <= sms && attn_page_keys(p) <= kAttnWholeKeys;
    if (F == kPagedTwo && many && attn_page_keys(p) >= kAttnDirectKeys) cut = kByLengths;
  } else {
    small = !p.list && (even || ((LISTED ? p.width : p.T) <= kAttnWholeKeys && items <= 4 * sms));
    const bool like = F == kTwo && (!C::SHARED || p.T == p.R) && items >= sms && 2 * items <= 5 * sms &&
                      p.T <= int64_t(kAttnLikeKeys) * p.S;
    direct = direct || like || (many && p.T >= int64_t(kAttnDirectKeys) * p.S);
  }
  direct = !LISTED && (direct || small);
  if (direct && items > INT32_MAX) return cudaErrorInvalidValue;
  if (direct || small) cut = kWhole;
  int grid = cut == kWhole ? int(items) : ctas;
  if (LISTED && !small && !p.list) grid = int(run_count(items * nt, grid));
  const int slot_rows = attn_slot_rows(GATHER ? 1 : p.R, p.G, C::kQTiles);
  JoinItem* joins = reinterpret_cast<JoinItem*>(ws + sizeof(WorkspaceHeader) + 256);
  float* part = reinterpret_cast<float*>(joins + kAttnMaxRuns);
  WorkspaceHeader* hdr = reinterpret_cast<WorkspaceHeader*>(ws);
  auto kernel = attn_tc_kernel<DK, DV, F>;
  static std::atomic<uint64_t> ready{0};
  e = allow_dynamic_smem(reinterpret_cast<const void*>(kernel), C::kSmem, &ready);
  if (e != cudaSuccess) return e;
  kernel<<<grid, C::kThreads, C::kSmem, stream>>>(tq, tk, tv, tr, p, int(tiles), cut, part, slot_rows, joins, hdr);
  e = cudaGetLastError();
  if (e != cudaSuccess || cut == kWhole || p.list || grid < 2) return e;
  cudaLaunchConfig_t cfg{};
  // many runs to an item: a CTA's warps share its rows; else each has its own
  const bool split = items * (slot_rows <= 64 ? 4 : 16) <= grid;
  const int join_rows = split ? 4 : 16;
  cfg.gridDim = dim3(uint32_t(grid - 1), uint32_t((slot_rows + join_rows - 1) / join_rows));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, split ? attn_join_kernel<DV, true> : attn_join_kernel<DV, false>, p, tt,
                         static_cast<const JoinItem*>(joins),
                         static_cast<const float*>(part), slot_rows);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool attn_tc_supported(kpool_dtype dtype, int32_t head_dim) {
  return dtype == KPOOL_BF16 && (head_dim == 64 || head_dim == 128);
}

bool attn_tc_shared_supported(kpool_dtype dtype, int32_t own, int32_t shared, int32_t value) {
  return dtype == KPOOL_BF16 && own == 128 && shared == 64 && value == 128;
}

bool attn_gather_supported(int64_t k_ts, int64_t v_ts) {
  return k_ts < (int64_t(1) << 31) && v_ts < (int64_t(1) << 31);  // byte strides in 32 bits
}

cudaError_t launch_attn_tc(const AttnParams& p, char* ws, cudaStream_t stream) {
  if (p.mode == kAttnSelected) {
    AttnParams g = p;
    int sms = 0;
    const cudaError_t q = device_sm_count(&sms);
    if (q != cudaSuccess) return q;
    const AttnSelectedTimes times = attn_selected_times(p, sms);
    if (times.dense < times.gathered) {
      AttnDense* ctl = reinterpret_cast<AttnDense*>(ws + sizeof(WorkspaceHeader));
      char* at = ws + sizeof(WorkspaceHeader) + ((attn_partial_bytes(p.R, p.G, p.D) + 255) & ~size_t(255));
      int32_t* list = reinterpret_cast<int32_t*>(at);
      uint32_t* mask = reinterpret_cast<uint32_t*>(at + attn_list_bytes(p.R));
      const cudaError_t e = launch_attn_dense_mask(p, ctl, mask, list, stream);
      if (e != cudaSuccess) return e;
      AttnParams d = p;
      d.mode = kAttnTree;
      d.cu_q = p.cu_k;
      d.mask = reinterpret_cast<const int32_t*>(mask);
      d.dense = ctl;
      const cudaError_t f = launch_attn_tc(d, ws, stream);
      if (f != cudaSuccess) return f;
      g.dense = ctl;
      g.list = list;
    }
    return p.D == 64 ? launch<64, 64, kGather>(g, ws, stream) : launch<128, 128, kGather>(g, ws, stream);
  }
  if (p.dense) return p.D == 64 ? launch<64, 64, kDense>(p, ws, stream) : launch<128, 128, kDense>(p, ws, stream);
  // Two row tiles per CTA read K and V half as often, but want sequences that fill them; the lengths are on the
  // device, so the call's mean decides (one / two row tiles, us, 32 / 8 heads of 128, 32 tokens a row tile):
  //  - like sequences: 8 x 30 over 8,000 keys 64 / 71, 8 x 33 85 / 72, 8 x 64 90 / 77, 4 x 200 over 6,000 91 / 100;
  //    prompts 32 x 256 83 / 69, 8 x 1,000 138 / 109, 1 x 2,048 62 / 56, 32,768 tokens 6,860 / 5,916;
  //    chunks over 30,000 keys, 128 rows 91 / 76, 512 rows 218 / 211; 16 decode tokens 136 / 151;
  //  - mixed ones lose by it whatever the mean is: 64 decode tokens over 4,000 keys and a chunk of 2,048 rows over
  //    8,192 316 / 404, of 512 rows 221 / 273; 16 over 8,000 and a prompt of 2,048 129 / 147; 8 trees of 1 to 64
  //    nodes 98 / 97.
  const bool two = int64_t(p.R) > int64_t(p.S) * (kTileRows / p.G);
  if (p.D == 64) return two ? launch<64, 64, kTwo>(p, ws, stream) : launch<64, 64, kOne>(p, ws, stream);
  return two ? launch<128, 128, kTwo>(p, ws, stream) : launch<128, 128, kOne>(p, ws, stream);
}

cudaError_t launch_attn_tc(const AttnPagedParams& p, char* ws, cudaStream_t stream) {
  // Decode steps by plain copies, where the pages follow one another in memory; chunks by TMA, a box for what lies in one
  // page (us, 32 / 8 heads of 128, plain copies / TMA): 16 decode tokens over pages of 8 132 / 268, of 16 132 / 187, of
  // 64 131 / 136. Chunks copy the tokens of pages whose boxes are one or two keys high, with one warp, as fast for any
  // pages: 300 rows over 12,000 keys 169 / 481 with pages of 1, 169 / 264 of 2 and 6, against 154 of 4, 107 of 8, 83 of 16, 70
  // of 64 by TMA; eight chunks of 20 over 700 43 / 86 and 43 / 53. (By both ways in one kernel the loading warp's registers
  // do not suffice: 5 to 10 % more with pages of 64.)
  const bool adjoin = pages_adjoin(p), rows = p.cu_q == nullptr && adjoin;
  const bool tokens = adjoin && piece_rows(p.page_size) <= 2;
  const bool two = int64_t(p.R) > int64_t(p.S) * (kTileRows / p.G);  // (as above)
  if (p.D == 64)
    return rows     ? launch<64, 64, kPagedRows>(p, ws, stream)
           : tokens ? launch<64, 64, kPagedTokens>(p, ws, stream)
           : two    ? launch<64, 64, kPagedTwo>(p, ws, stream)
                    : launch<64, 64, kPagedOne>(p, ws, stream);
  return rows     ? launch<128, 128, kPagedRows>(p, ws, stream)
         : tokens ? launch<128, 128, kPagedTokens>(p, ws, stream)
         : two    ? launch<128, 128, kPagedTwo>(p, ws, stream)
                  : launch<128, 128, kPagedOne>(p, ws, stream);
}

cudaError_t launch_attn_tc(const AttnSharedParams& p, char* ws, cudaStream_t stream) {
  const bool two = int64_t(p.R) > int64_t(p.S) * (kTileRows / p.G);  // (as above)
  return two ? launch<192, 128, kTwo>(p, ws, stream) : launch<192, 128, kOne>(p, ws, stream);
}

}  // namespace kpool
