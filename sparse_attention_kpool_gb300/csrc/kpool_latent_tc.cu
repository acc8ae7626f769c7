// kpool_latent_tc.cu -- attention over latent vectors on the 5th-generation tensor cores: bf16, 512 + 64
// channels (the latent, then its rotated part), over a cache in pages, whole or by token ids.
//
// Rows. The heads of one query row share every token, and a token is key and value at once: a tile
// of 64 tokens is copied once into shared memory and feeds both products. Up to 64 heads a CTA:
//   S [64 heads x 64 tokens] = Q C^T         36 steps of 16 channels, Q and C from shared memory;
//   O^T [512 channels x heads] += C^T P^T    four blocks of 128 channels, C as the A operand.
// The second product is transposed because 64 heads x 512 fp32 channels would fill tensor memory with rows
// to spare in its lanes only; as 4 x (128 lanes x heads columns) they take 256 of 512 columns, beside two
// buffers of scores. More than 64 heads are split evenly over CTAs side by side that walk
// the same tokens at the same time, so that the second reads what the first brought into L2.
//
// Roles (14 warps): warps 0-7 softmax, eight threads to a head's 64 scores (the layout in which a 16-row
// accumulator is read); warps 8-11 copy tokens, 16 bytes a lane (cp.async), rows of 1,152 bytes wherever the ids
// and the page table put them (TMA of whole pages: 108.1 against 106.5 us for the first case below); warp 12 issues the MMAs and owns
// tensor memory; warp 13 hands out segments and loads Q. The scores of tile j + 1 are issued while the softmax of
// tile j runs if that tile has landed by then, else behind the second product of tile j. A slot's parts (rotated block,
// four blocks of channels) are freed one by one, the first as soon as the tile is scored.
//
// What bounds it. Of a tile (74 KB; 3,100 cycles of an SM's share of the measured copy rate at 1.9 GHz) the products
// take 2,470 cycles at 64 heads: operands from shared memory come at about 90 bytes a cycle, 36 x 4 KB in 1,390 and 16 x
// 6 KB in 1,080. The softmax between them (860, of which exponentials and stores are 550) and the handing over (150 +
// 200) are hidden only where the next tile has landed in time: two tiles are what fits beside 64 heads of Q (whose space is
// that of 64 heads in every call; beside 32 a third tile would fit).
//   - 32 sequences of 64 heads, 389,566 tokens (449 MB): 101 us, of it 88 the tiles (5.1 TB/s, 3,900 cycles each: a tile
//     takes 2,800 from HBM, so its scores wait for it), the rest the join;
//   - 512 rows x 2,052 ids of 128 heads (2.3 GB out of L2): 390 us, 2,850 cycles a tile, the tensor core 87 % of them.
//
// Masked places: tokens that are not seen are written as zeros (no infinity meets a weight of zero) and
// score -inf. P is rounded to bf16 (half a step is 2^-8 of a weight) because the second product takes
// bf16; the row sum adds the weights before that rounding, in fp32. Exponentials are the hardware's (2 ulp). O is rescaled
// only when a maximum has grown by more than 8 in the exponent, as in kpool_attn_tc.cu.
//
// Work. A run per CTA (per group of CTAs, above 64 heads) of about equally many tiles, found by every CTA itself
// from the lengths on the device; unfinished rows go to the workspace as (m, l, O) and a second kernel joins
// them in the order of the runs, so results repeat bit for bit.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include "kpool_latent.cuh"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr int kLatent = 512, kRotary = 64, kDim = kLatent + kRotary;
constexpr int kKeys = 64;                    // tokens of a tile
constexpr int kHeads = 64;                   // MMA rows of the first product
constexpr int kBlock = kKeys * 128;          // bytes of 64 channels of a tile, of 64 heads of Q
constexpr int kBlocks = kDim / 64;
constexpr int kTileBytes = kBlocks * kBlock;
constexpr int kStages = 2;
// A tile's parts, in the order in which they are freed and copied: the rotated block, which nothing reads after the
// scores, then the 128-channel blocks of the second product. (Scored part by part as they land, a tile's first product
// takes 2,300 cycles instead of 1,250: 200 a wait and the start of its steps.)
constexpr int kParts = 1 + kLatent / 128;
__host__ __device__ constexpr int part_block(int c) { return c == 0 ? kLatent / 64 : 2 * (c - 1); }  // first 64-channel block
__host__ __device__ constexpr int part_blocks(int c) { return c == 0 ? 1 : 2; }
constexpr int kSoftWarps = 8, kCopyWarps = 4, kMmaWarp = kSoftWarps + kCopyWarps, kSegWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kSegWarp + 1);
constexpr int kCopyRows = kKeys / kCopyWarps;  // tokens of a tile that a warp copies
constexpr int kSegRing = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;                // growth of the maximum (in powers of two) that O is not rescaled for
constexpr uint64_t kMaxWaitNs = 1000000000ull;  // 1 s; legitimate waits are microseconds

// Shared memory: Q, the tiles, P, then
constexpr int kOffTiles = kTileBytes;
constexpr int kOffP = kOffTiles + kStages * kTileBytes;
constexpr int kOffMax = kOffP + kBlock;                  // [2][2][64] fp32: maxima of a tile's halves; sums at the end
constexpr int kOffSeg = kOffMax + 4 * kHeads * 4;
// [kBitsRing] x 64 bits, the tokens of a tile that are seen. A tile's are written when the scores of the tile kStages
// before are done, and read by its softmax; scores are at most one tile ahead of it.
constexpr int kBitsRing = 4;
constexpr int kOffBits = kOffSeg + 48 * kSegRing;
constexpr int kOffBar = kOffBits + 8 * kBitsRing;
// full[2] empty[2][5] q_full q_empty s_full[2] p_ready p_empty o_final o_free done seg_full[4] seg_empty[4]
constexpr int kNumBars = kStages * (1 + kParts) + 9 + 2 * kSegRing;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;
constexpr int kSmem = kOffMisc + 72;
static_assert(kSmem <= 232448, "exceeds the 227 KB per-CTA shared memory limit");
static_assert(kOffSeg % 16 == 0 && kOffBits % 8 == 0 && kOffBar % 8 == 0 && kOffMisc % 8 == 0, "aligned accesses");

struct Misc {
  int64_t base;      // first position of row r
  int64_t lo, hi;    // positions of this run
  int64_t total;
  int32_t runs;      // runs that have tiles
  int32_t row;
  uint32_t tmem;
  volatile int32_t abort;
  volatile int32_t bad_page;
  volatile int32_t dead[3];  // a softmax warp gave up at an even or odd tile, or between segments
};
static_assert(sizeof(Misc) <= 72, "Misc fits its space");

struct Seg {
  int32_t row, seq, keys;  // query row, its sequence and the keys that one holds
  int32_t end;             // places to walk
  int32_t kt0, n;          // first tile here and their number (0: the row sees nothing; -1: the work is done)
  int8_t whole;            // no other run has tiles of this row
  int8_t slot;             // partial slot of the CTA: 0 when an earlier run began the row, else 1
};
static_assert(sizeof(Seg) <= 48, "Seg fits its space");

// Beginning and finishing a row (Q, first product, epilogue) takes about as long as this many tiles; it is counted
// when runs are cut, as positions before the row's first tile.
constexpr int kRowCost = 2;
constexpr int kMaxRuns = 152;
constexpr int kMaxRunRows = 8192;   // rows whose lengths a CTA adds up itself (whole rows above)

__device__ __forceinline__ int row_tiles(const LatentParams& p, int r) {
  int b;
  return max(1, (latent_places(p, latent_seq(p, r, &b)) + kKeys - 1) / kKeys);
}
// Over ids every row has the tiles of the list, whatever its sequence holds.
__host__ __device__ __forceinline__ int id_tiles(const LatentParams& p) {
  return p.width <= kKeys ? 1 : (p.width + kKeys - 1) / kKeys;
}

// (Runs of three positions and more would spare joins: one row of 2,052 ids and 64 heads 22.6 us, of one 16.5.)
__host__ __device__ __forceinline__ int64_t run_count(int64_t total, int64_t runs) { return total < runs ? total : runs; }

// The positions of the runs: run r of n begins at floor(total r / n).
struct Cuts {
  int64_t each;
  uint32_t rest, n;
  __device__ __forceinline__ Cuts(int64_t total, uint32_t runs)
      : each(total / runs), rest(uint32_t(total - each * runs)), n(runs) {}
  __device__ __forceinline__ int64_t lo(uint32_t r) const { return each * r + rest * r / n; }  // rest * r < n * n
};

// Every thread of the CTA: the positions of run i of up to `runs`, and the row that it begins in. `scratch` holds R
// 64-bit words (without ids).
__device__ __forceinline__ void find_run(const LatentParams& p, int64_t* scratch, int i, int runs, Misc* m) {
  if (latent_listed(p)) {
    if (threadIdx.x == 0) {
      const int per = id_tiles(p) + kRowCost;
      m->total = int64_t(p.R) * per;
      m->runs = int(run_count(m->total, runs));
      const Cuts cuts(m->total, uint32_t(m->runs));
      m->lo = i < m->runs ? cuts.lo(i) : m->total;
      m->hi = i < m->runs ? cuts.lo(i + 1) : m->total;
      m->row = int(m->lo / per);
      m->base = int64_t(m->row) * per;
    }
    __syncthreads();
    return;
  }
  for (int r = threadIdx.x; r < p.R; r += kThreads) scratch[r] = row_tiles(p, r) + kRowCost;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t sum = 0;
    for (int r = lane; r < p.R; r += 32) sum += scratch[r];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const int64_t n = run_count(sum, runs);
    const Cuts cuts(sum, uint32_t(n));
    const int64_t lo = i < n ? cuts.lo(i) : sum, hi = i < n ? cuts.lo(i + 1) : sum;
    int64_t run = 0;
    bool found = false;
    for (int r0 = 0; r0 < p.R && !found; r0 += 32) {
      const int64_t own = r0 + lane < p.R ? scratch[r0 + lane] : 0;
      int64_t inc = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      const bool mine = lo < run + inc && lo >= run + inc - own;
      if (mine) {
        m->row = r0 + lane;
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

// Rows of a partial result of `per` heads: their 16-byte words stay aligned.
__host__ __device__ __forceinline__ int part_rows(int per) { return (per + 15) & ~15; }

// What the join of a row that several runs have parts of needs; runs = 0: nothing to join.
struct JoinItem {
  int64_t item;       // position of the row's first tile
  int64_t each;       // Cuts of the call
  uint32_t rest;
  int32_t tiles;
  int32_t runs;
  int32_t row;
  int32_t first;      // the run that has the row's first tile
  int32_t pad[3];
};
static_assert(sizeof(JoinItem) == 48, "join items are laid out in the workspace");

// The segments of a run of positions.
struct SegIter {
  int64_t pos, hi, item;   // item: first position of the present row
  int row, c;              // c: its tiles
  __device__ __forceinline__ void start(const LatentParams& p, const Misc* m) {
    pos = m->lo;
    hi = m->hi;
    row = m->row;
    item = m->base;
    c = pos < hi ? tiles(p) : 0;
  }
  __device__ __forceinline__ int tiles(const LatentParams& p) const { return latent_listed(p) ? id_tiles(p) : row_tiles(p, row); }
  __device__ __forceinline__ bool next(const LatentParams& p, Seg* s) {
    if (pos >= hi) return false;
    if (pos == item + kRowCost + c) {
      item = pos;
      ++row;
      c = tiles(p);
    }
    const int64_t tile0 = item + kRowCost;
    if (hi <= tile0) return false;  // (only as the run's last row)
    s->row = row;
    s->kt0 = int(max(pos - tile0, int64_t(0)));
    s->n = int(min(int64_t(c), hi - tile0)) - s->kt0;
    s->whole = s->n == c;
    s->slot = s->kt0 > 0 ? 0 : 1;
    pos = tile0 + s->kt0 + s->n;
    return true;
  }
};

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

__device__ __forceinline__ void soft_sync() {
  asm volatile("barrier.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
}

// per: heads of a CTA (a multiple of 16 when there are several); groups: CTAs that share a run's tokens.
__global__ void __launch_bounds__(kThreads, 1)
    latent_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ LatentParams p, int per,
                     int groups, int direct, float* part, JoinItem* joins, WorkspaceHeader* hdr) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages * kParts;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;   // [2]
  uint64_t* p_ready = q_full + 4;
  uint64_t* p_empty = q_full + 5;
  uint64_t* o_final = q_full + 6;
  uint64_t* o_free = q_full + 7;
  uint64_t* done = q_full + 8;
  uint64_t* seg_full = q_full + 9;             // [kSegRing]
  uint64_t* seg_empty = seg_full + kSegRing;   // [kSegRing]
  auto seg_at = [&](int i) { return reinterpret_cast<Seg*>(smem + kOffSeg + 48 * (i % kSegRing)); };
  float* maxima = reinterpret_cast<float*>(smem + kOffMax);
  Misc* misc = reinterpret_cast<Misc*>(smem + kOffMisc);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform)
  const int run = blockIdx.x / groups, group = blockIdx.x - run * groups, runs = gridDim.x / groups;
  const int head0 = group * per, heads = min(per, p.H - head0), cols = (heads + 15) & ~15;
  const int slots = part_rows(per);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this kernel's end itself
  if (blockIdx.x == 0 && threadIdx.x == 0) hdr->error = KPOOL_OK;
  if (!direct) {
    find_run(p, reinterpret_cast<int64_t*>(smem), run, runs, misc);
    ptx::fence_proxy_async_smem();  // the scratch lies where TMA writes next
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) ptx::mbar_init(full + i, kCopyWarps);
    for (int i = 0; i < kStages * kParts; ++i) ptx::mbar_init(empty + i, 1);
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    ptx::mbar_init(s_full, 1);
    ptx::mbar_init(s_full + 1, 1);
    ptx::mbar_init(p_empty, 1);
    ptx::mbar_init(p_ready, kSoftWarps);
    ptx::mbar_init(o_final, 1);
    ptx::mbar_init(o_free, kSoftWarps);
    ptx::mbar_init(done, 1);
    for (int i = 0; i < kSegRing; ++i) {
      ptx::mbar_init(seg_full + i, 1);
      ptx::mbar_init(seg_empty + i, kSoftWarps + kCopyWarps + 1);
    }
    ptx::fence_mbar_init();
    misc->abort = 0;
    misc->bad_page = 0;
    misc->dead[0] = misc->dead[1] = misc->dead[2] = 0;
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&misc->tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc->tmem;
  auto segment = [&](int i) -> const Seg* {
    return wait_bar(seg_full + i % kSegRing, (i / kSegRing) & 1, misc) ? seg_at(i) : nullptr;
  };

  if (warp == kSegWarp) {  // ---------------------------------------------------- segments and Q
    if (lane == 0) {
      SegIter it;
      if (!direct) it.start(p, misc);
      uint32_t q_loads = 0;
      Seg s{};
      for (int i = 0;; ++i) {
        bool more;
        if (direct) {
          s.row = run + i * runs;
          more = s.row < p.R;
          if (more) {
            s.kt0 = 0;
            s.n = latent_listed(p) ? id_tiles(p) : row_tiles(p, s.row);
            s.whole = 1;
            s.slot = 0;
          }
        } else {
          more = it.next(p, &s);
        }
        if (!direct && group == 0) {
          // The run that begins a row leaves its join: with fewer rows than runs in the row's place, else in the run's
          // own (only the last row that it begins can be cut).
          const bool by_row = p.R <= runs;
          if (more && s.kt0 == 0) {
            const Cuts cuts(misc->total, uint32_t(misc->runs));
            JoinItem j{};
            j.item = it.item + kRowCost;
            j.each = cuts.each;
            j.rest = cuts.rest;
            j.tiles = it.c;
            j.runs = s.whole ? 0 : misc->runs;
            j.row = s.row;
            j.first = run;
            joins[by_row ? s.row : run] = j;
          } else if (!by_row && i == 0) {
            joins[run].runs = 0;
          }
        }
        if (more) {
          s.keys = latent_seq(p, s.row, &s.seq);
          s.end = latent_places(p, s.keys);
          if (s.end == 0) s.n = 0;
        } else {
          s.n = -1;
        }
        if (i >= kSegRing && !wait_bar(seg_empty + i % kSegRing, (i / kSegRing - 1) & 1, misc)) break;
        *seg_at(i) = s;
        ptx::mbar_arrive(seg_full + i % kSegRing);
        if (!more) break;
        if (s.n == 0) continue;
        if (q_loads > 0 && !wait_bar(q_empty, (q_loads - 1) & 1, misc)) break;
        ptx::mbar_arrive_expect_tx(q_full, kTileBytes);
        ++q_loads;
#pragma unroll
        for (int h = 0; h < kBlocks; ++h)
          ptx::tma_load_3d(smem + h * kBlock, &tm_q, q_full, 64 * h, head0, s.row);
      }
      if (q_loads) ptx::mbar_wait_bounded(q_full, (q_loads - 1) & 1, int64_t(1) << 40, kMaxWaitNs);
    }
    __syncwarp();
    if (blockIdx.x == 0) latent_check(p, hdr);
  } else if (warp == kMmaWarp) {  // ----------------------------------------------- MMA issuer
    // The warp stays together, its values are the same in all lanes, and one lane issues: 33 cycles an instruction of
    // the first product, 48 for code that only lane 0 runs (its operands pass through registers of the lane).
    const uint64_t q_desc = ptx::smem_desc_kmajor_sw128(ptx::smem_addr(smem));
    const uint64_t c_desc = ptx::smem_desc_kmajor_sw128(ptx::smem_addr(smem + kOffTiles));
    const uint64_t v_desc = ptx::smem_desc_mnmajor_sw128(ptx::smem_addr(smem + kOffTiles), kBlock);
    const uint64_t p_desc = ptx::smem_desc_kmajor_sw128(ptx::smem_addr(smem + kOffP));
    constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(kHeads, kKeys);
    const uint32_t idesc_o = ptx::idesc_bf16_f32_am(128, cols);
    const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t u = 0, q_uses = 0;  // tiles, segments with tiles
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return bool(__all_sync(0xffffffffu, wait_bar(bar, parity, misc)));
    };
    for (int i = 0; ok; ++i) {
      const Seg* s = segment(i);
      if (!__all_sync(0xffffffffu, s != nullptr)) break;
      const int n = __shfl_sync(0xffffffffu, s->n, 0);
      if (n < 0) break;
      if (n > 0 && !(ok = wait(q_full, q_uses & 1))) break;
      int scored = 0;  // tiles of the segment whose scores are issued
      auto score = [&](uint32_t v) {
        ptx::fence_proxy_async_smem();  // the tile was written by ordinary copies
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t b = c_desc + v % kStages * (kTileBytes >> 4);
          const uint32_t to = acc + 256 + 64 * (v & 1);
#pragma unroll
          for (int kk = 0; kk < kDim / 16; ++kk) {
            const uint32_t step = ((kk >> 2) * kBlock + (kk & 3) * 32) >> 4;
            ptx::tc_mma_f16(to, q_desc + step, b + step, idesc_s, kk > 0 ? 1u : 0u);
          }
          ptx::tc_commit(s_full + (v & 1));
          ptx::tc_commit(empty + v % kStages * kParts);
          if (scored == n - 1) ptx::tc_commit(q_empty);
        }
        __syncwarp();
        ++scored;
      };
      for (int j = 0; j < n; ++j, ++u) {
        const uint32_t st = u % kStages;
        if (scored == j) {
          if (!(ok = wait(full + st, (u / kStages) & 1))) break;
          score(u);
        }
        // While the weights are made, the next scores if their tile is there by then: the second product frees the
        // slot of the tile after, so it does not wait for the next one to land.
        if (scored < n && scored == j + 1) {
          const uint64_t t0 = ptx::globaltimer_ns();
          for (int polls = 1; !__all_sync(0xffffffffu, ptx::mbar_test(p_ready, u & 1)); ++polls) {
            if (__all_sync(0xffffffffu, ptx::mbar_test(full + (u + 1) % kStages, ((u + 1) / kStages) & 1))) {
              score(u + 1);
              break;
            }
            if ((polls & 255) == 0 && __any_sync(0xffffffffu, misc->abort || ptx::globaltimer_ns() - t0 > kMaxWaitNs)) break;
          }
        }
        if (!(ok = wait(p_ready, u & 1))) break;
        if (j == 0 && q_uses > 0 && !(ok = wait(o_free, (q_uses - 1) & 1))) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t a = v_desc + st * (kTileBytes >> 4);
#pragma unroll
          for (int c = 0; c < kLatent / 128; ++c) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              ptx::tc_mma_f16(acc + 64 * c, a + ((2 * c * kBlock + kk * 2048) >> 4), p_desc + (kk * 32 >> 4), idesc_o,
                              (kk > 0 || j > 0) ? 1u : 0u);
            ptx::tc_commit(empty + st * kParts + c + 1);
          }
          ptx::tc_commit(p_empty);
          if (j == n - 1) ptx::tc_commit(o_final);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (n > 0) ++q_uses;
      if (lane == 0) ptx::mbar_arrive(seg_empty + i % kSegRing);
    }
    if (ptx::elect_one()) ptx::tc_commit(done);  // every MMA issued above completes before TMEM is freed
    ptx::mbar_wait_bounded(done, 0, int64_t(1) << 40, kMaxWaitNs);
  } else if (warp >= kSoftWarps) {  // --------------------------------------- copying warps
    // Warp w copies the tokens [16 w, 16 w + 16) of a tile, four at a time: eight lanes take 128 bytes of each. Where a
    // tile's tokens lie is looked up while the tile before is on its way: ids two tiles ahead, pages one.
    const int w = warp - kSoftWarps, c = lane & 7, sub = lane >> 3;
    const char* base = static_cast<const char*>(p.cache) + c * 16;
    const uint32_t dst0 = ptx::smem_addr(smem + kOffTiles) + uint32_t(w * kCopyRows + sub) * 128;
    uint32_t u = 0;
    bool ok = true, bad = false;
    const Seg* s;
    for (int i = 0;; ++i) {
      s = segment(i);
      if (!__all_sync(0xffffffffu, s != nullptr) || s->n < 0) break;
      const int n = s->n, keys = s->keys, end = s->end, kt0 = s->kt0;
      const int32_t* table = p.table + int64_t(s->seq) * p.max_pages;
      const int32_t* ids = p.ids + int64_t(s->row) * p.width;
      // The id at the lane's place of tile j, lanes 0-15 for the warp's tokens; -1: none.
      auto id_of = [&](int j) {
        const int place = (kt0 + j) * kKeys + w * kCopyRows + lane;
        if (j >= n || lane >= kCopyRows || place >= end) return -1;
        return latent_listed(p) ? ptx::ldg_ordered(ids + place) : place;
      };
      int id1 = id_of(0), page = -1, in_page = 0, id = -1;
      auto look_up = [&]() {  // the page of the id that was read before
        id = id1 >= 0 && id1 < keys ? id1 : -1;
        const int at = id / p.page_size;
        in_page = id - at * p.page_size;
        page = id >= 0 ? ptx::ldg_ordered(table + at) : -1;
      };
      if (n > 0) {
        look_up();
        id1 = id_of(1);
      }
      for (int j = 0; j < n; ++j, ++u) {
        const uint32_t st = u % kStages;
        if (id >= 0 && (page < 0 || page >= p.num_pages)) {
          bad = true;
          page = -1;
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, page >= 0);
        // everything but the copies themselves comes before the slot is free
        const char* from[kCopyRows / 4];
        uint32_t bytes[kCopyRows / 4];
        const int64_t at = page >= 0 ? int64_t(page) * p.c_ps + int64_t(in_page) * p.c_ts : -1;
#pragma unroll
        for (int q = 0; q < kCopyRows / 4; ++q) {
          const int64_t t = __shfl_sync(0xffffffffu, at, 4 * q + sub);
          from[q] = base + (t >= 0 ? t : 0) * 2;
          bytes[q] = t >= 0 ? 16u : 0u;
        }
        if (j + 1 < n) {
          look_up();
          id1 = id_of(j + 2);
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          if (u >= kStages)
            ok = __all_sync(0xffffffffu, wait_bar(empty + st * kParts + part, (u / kStages - 1) & 1, misc));
          if (!ok) break;
          __syncwarp();
          if (part == 0 && lane == 0)
            reinterpret_cast<uint16_t*>(smem + kOffBits)[4 * (u % kBitsRing) + w] = uint16_t(bits);
#pragma unroll
          for (int q = 0; q < kCopyRows / 4; ++q) {
            // the row's number modulo eight permutes its 16-byte pieces
            const uint32_t dst = dst0 + st * kTileBytes + q * 512 + ((c ^ ((q * 4 + sub) & 7)) << 4);
#pragma unroll
            for (int h = part_block(part); h < part_block(part) + part_blocks(part); ++h)
              ptx::cp_async_16(dst + h * kBlock, from[q] + h * 128, bytes[q]);
          }
        }
        if (!ok) break;
        ptx::cp_async_arrive_inc(full + st);  // the phase waits for this lane's pieces
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full + st);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(seg_empty + i % kSegRing);
    }
    if (bad) misc->bad_page = 1;
    ptx::cp_async_wait_all();  // every copy has landed before the CTA exits
  } else {  // ---------------------------------------------------------------- softmax
    // Warps w and w + 4 share the heads [16 w, 16 w + 16), a half of a tile's tokens each: lane 4 g + t has the heads
    // 16 w + g and 8 further, tokens 8 x + 2 t and the next of every eight. Every warp keeps the maxima of all 64 heads
    // (lane i: heads i and i + 32) and finds by itself, from the halves' maxima of the tile, which of them grow.
    const int half = warp >> 2, g = lane >> 2, t = lane & 3;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const float c2 = p.scale * kLog2e;
    const int row0 = (warp & 3) * 16 + g;
    const bool live = (warp & 3) * 16 < cols;  // (other heads' weights are not read)
    uint8_t* p_row = smem + kOffP + row0 * 128 + t * 4;
    uint32_t u = 0, finals = 0;
    bool ok = true;
    // value of heads i, i + 32 (in lane i) for the lane's own two heads
    auto own = [&](const float (&x)[2], int h) {
      const float lo = __shfl_sync(0xffffffffu, x[0], (row0 + 8 * h) & 31), hi = __shfl_sync(0xffffffffu, x[1], (row0 + 8 * h) & 31);
      return row0 + 8 * h < 32 ? lo : hi;
    };
    for (int is = 0;; ++is) {
      const Seg* sg = segment(is);
      // (all warps leave together: whoever gives up says so before a barrier, and all read it behind it)
      if (!__all_sync(0xffffffffu, sg != nullptr)) misc->dead[2] = 1;
      soft_sync();
      if (misc->dead[2]) break;
      const int n = sg->n;
      if (n < 0) break;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      float nb[2] = {0.f, 0.f};  // what the lane's own heads' exponents begin with: minus their maxima
      for (int j = 0; j < n; ++j, ++u) {
        if (!__all_sync(0xffffffffu, wait_bar(s_full + (u & 1), (u >> 1) & 1, misc))) misc->dead[u & 1] = 1;
        ptx::tc_fence_after();
        uint32_t s[16];
        ptx::tc_ld_16x256b_x4(tmem + 256 + 64 * (u & 1) + lanes + 32 * half, s);
        const uint32_t bits = *reinterpret_cast<const volatile uint32_t*>(smem + kOffBits + 8 * (u % kBitsRing) + 4 * half);
        ptx::tc_wait_ld();
        ptx::tc_reg_fence(s);
        if (bits != 0xffffffffu) {
          const uint32_t mine = bits >> (2 * t);
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (!((mine >> (8 * x + y)) & 1u)) s[4 * x + y] = s[4 * x + 2 + y] = 0xFF800000u;  // -inf
        }
        float* mx = maxima + (u & 1) * 2 * kHeads;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mt = __uint_as_float(s[2 * h]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mt = fmaxf(fmaxf(mt, __uint_as_float(s[4 * x + 2 * h])), __uint_as_float(s[4 * x + 2 * h + 1]));
          mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
          mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
          if (t == 0) mx[half * kHeads + row0 + 8 * h] = mt;
        }
        soft_sync();
        if (misc->dead[u & 1]) {
          ok = false;
          break;
        }
        bool grow[2];
        float top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(mx[lane + 32 * h], mx[kHeads + lane + 32 * h]);
          grow[h] = top[h] > m[h] && (top[h] - m[h]) * c2 > kLazy;
        }
        const bool rescale = __any_sync(0xffffffffu, grow[0] || grow[1]);  // (the same in every warp)
        float f[2];
        if (rescale) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[h] = grow[h] ? ptx::exp2_approx((m[h] - top[h]) * c2) : 1.0f;
            if (grow[h]) m[h] = top[h];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            l[h] *= own(f, h);
            const float mine = own(m, h);
            nb[h] = mine == -INFINITY ? 0.0f : -mine * c2;
          }
        }
        uint32_t weights[2][4];
        if (live) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float a = ptx::exp2_approx(fmaf(__uint_as_float(s[4 * x + 2 * h]), c2, nb[h]));
              const float b = ptx::exp2_approx(fmaf(__uint_as_float(s[4 * x + 2 * h + 1]), c2, nb[h]));
              l[h] += a + b;
              weights[h][x] = ptx::pack_bf16(a, b);
            }
        }
        // When the second product of the tile before is done, O is at rest and P may be written. (A warp whose wait runs
        // out says so at the next barrier; the others' waits then end, too.)
        if (u > 0 && !__all_sync(0xffffffffu, wait_bar(p_empty, (u - 1) & 1, misc))) misc->dead[(u + 1) & 1] = 1;
        if (rescale && j > 0) {
          ptx::tc_fence_after();
          const int per_block = cols / 16;
#pragma unroll 1
          for (int x = 0; x < 2 * per_block; ++x) {
            const int c = 2 * half + x / per_block, col = (x % per_block) * 16;
            const uint32_t at = tmem + lanes + 64 * c + col;
            uint32_t o[16];
            ptx::tc_ld_32x32b_x16(at, o);
            ptx::tc_wait_ld();
            ptx::tc_reg_fence(o);
#pragma unroll
            for (int y = 0; y < 16; ++y)
              o[y] = __float_as_uint(__uint_as_float(o[y]) *
                                     __shfl_sync(0xffffffffu, col < 32 ? f[0] : f[1], (col & 31) + y));
            ptx::tc_st_32x32b_x16(at, o);
          }
          ptx::tc_wait_st();
        }
        if (live) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              *reinterpret_cast<uint32_t*>(p_row + h * 1024 + (((4 * half + x) ^ g) << 4)) = weights[h][x];
          ptx::fence_proxy_async_smem();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_ready);
      }
      if (!ok) break;
      // ------------------------------------------------------------------------ epilogue
      // The sums of both halves, in shared memory like the maxima (whose last readers are behind a barrier).
      float* sums = maxima + (u & 1) * 2 * kHeads;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) sums[half * kHeads + row0 + 8 * h] = l[h];
      }
      if (n > 0 && !__all_sync(0xffffffffu, wait_bar(o_final, finals & 1, misc))) misc->dead[u & 1] = 1;
      soft_sync();
      if (misc->dead[u & 1]) break;
      ptx::tc_fence_after();
      float* pslot = part + (size_t(blockIdx.x) * 2 + sg->slot) * size_t(slots) * (kLatent + 2);
      float inv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int head = lane + 32 * h;
        const float sum = sums[head] + sums[kHeads + head];
        const bool none = m[h] == -INFINITY && sum == 0.0f;  // (a NaN score leaves the sum NaN: not empty)
        inv[h] = none ? 0.0f : 1.0f / sum;
        if (warp != 0 || head >= heads) continue;
        if (sg->whole) {
          if (p.lse)
            p.lse[int64_t(sg->row) * p.H + head0 + head] = none ? -INFINITY : (m[h] * c2 + log2f(sum)) * kLn2;
        } else {
          *reinterpret_cast<float2*>(pslot + size_t(slots) * kLatent + 2 * head) = make_float2(m[h], sum);
        }
      }
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(sg->row) * p.o_ts + int64_t(head0) * p.o_hs;
      const int per_block = cols / 16;
#pragma unroll 1
      for (int x = 0; x < 2 * per_block; ++x) {
        const int c = 2 * half + x / per_block, col = (x % per_block) * 16;
        uint32_t o[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] = 0;
        if (n > 0) {
          ptx::tc_ld_32x32b_x16(tmem + lanes + 64 * c + col, o);
          ptx::tc_wait_ld();
          ptx::tc_reg_fence(o);
        }
        const int ch = 128 * c + 32 * (warp & 3) + lane;
        if (sg->whole) {
          // neighbouring lanes exchange halves of two heads: each then writes two channels of one head
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            const float fa = __shfl_sync(0xffffffffu, col < 32 ? inv[0] : inv[1], (col & 31) + y);
            const float fb = __shfl_sync(0xffffffffu, col < 32 ? inv[0] : inv[1], (col & 31) + y + 1);
            // (no weight at all: zeros, whatever the products hold)
            const float a = fa == 0.0f ? 0.0f : __uint_as_float(o[y]) * fa;
            const float b = fb == 0.0f ? 0.0f : __uint_as_float(o[y + 1]) * fb;
            const bool odd = lane & 1;
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
            const int head = col + y + odd;
            if (head < heads)
              *reinterpret_cast<uint32_t*>(out + head * p.o_hs + (ch & ~1)) =
                  odd ? ptx::pack_bf16(got, b) : ptx::pack_bf16(a, got);
          }
        } else {
#pragma unroll
          for (int y = 0; y < 16; ++y)
            if (col + y < heads) pslot[size_t(col + y) * kLatent + ch] = __uint_as_float(o[y]);
        }
      }
      if (n > 0) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(o_free);
        ++finals;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(seg_empty + is % kSegRing);
    }
    ptx::tc_fence_before();
  }
  // ------------------------------------------------------------------------------ teardown
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0 && misc->abort) record_error(hdr, KPOOL_ERR_DEVICE_TIMEOUT);
  if (threadIdx.x == 0 && misc->bad_page) record_error(hdr, KPOOL_ERR_INVALID_ARG);
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------- join
//
// CTA x adds up, in the order of the runs, the partial results of the row that item x names, a head or a quarter of one
// to a warp (Join):
//   kFewParts   a head a warp, 16 channels a lane, two parts at a time: enough heads to fill the card, few parts of each;
//   kSomeParts  a quarter of a head a warp, four channels a lane, eight parts at a time;
//   kManyParts  the 8 warps of a CTA share a quarter, each taking every eighth part: few heads in all, each cut into very many.
// What is read was just written: 132 KB a part of 64 heads. A row cut by n borders has n + 1 parts, so 152 runs over 16 rows
// leave 167 of them at most, 22 MB.
enum Join { kFewParts, kSomeParts, kManyParts };
constexpr int kSomeBatch = 8;

// By the heads of all rows, which are the warps there are, and a row's parts (us of the whole call, whole caches of 300,000
// tokens in all, or 30,000 a row):
//   many / some   4 rows of 16 heads 41 / 51, of 32 45 / 52; 8 of 16 64 / 66, of 32 71 / 68, of 64 82 / 70; 4 of 128 74 / 64;
//                 more than nine rows, less than 16 parts each: 10 of 16 76 / 75, 20 of 16 81 / 73;
//   some / few    9 rows of 64 heads 77 / 82, 20 of 32 79 / 79, 32 of 16 73 / 75; 16 of 64 83 / 82, 48 of 32 80 / 77, 76 of 64 92
//                 / 79, 48 of 128 142 / 126; 200 of 16 78 / 73, of 4 70 / 71.
inline Join join_form(int64_t rows, int32_t heads, int runs) {
  if (rows * heads >= 768) return kFewParts;
  return rows * heads <= 192 && rows * 2 * kSomeBatch <= runs ? kManyParts : kSomeParts;
}

template <Join J>
__global__ void __launch_bounds__(256)
    latent_join_kernel(const __grid_constant__ LatentParams p, int per, int groups, int runs, const JoinItem* joins,
                       const float* part) {
  constexpr int kWords = J == kFewParts ? 4 : 1;               // float4 of a lane
  constexpr int kPieces = kLatent / (128 * kWords);            // warps' pieces of a head
  constexpr int kBatch = J == kFewParts ? 2 : kSomeBatch, kStep = J == kManyParts ? 8 : 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // in every CTA: the call ends after both kernels have
  const JoinItem it = joins[blockIdx.x];
  // (after a wait that ran out an item may never have been written)
  if (it.runs <= 0 || it.runs > runs || it.first < 0 || it.first >= runs || it.row < 0 || it.row >= p.R) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = J == kManyParts ? int(blockIdx.y) : int(blockIdx.y) * 8 + warp;
  const int head = unit / kPieces, ch = unit % kPieces * 128 * kWords + 4 * lane;
  const int group = head / per, h = head - group * per;
  const bool live = head < p.H;
  auto run_lo = [&](int r) { return it.each * r + it.rest * uint32_t(r) / uint32_t(it.runs); };
  const float c2 = p.scale * kLog2e;
  const int64_t end = it.item + it.tiles;
  float4 acc[kWords];
#pragma unroll
  for (int x = 0; x < kWords; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.0f;
  // adds a part (o, pm, pl); one without any weight adds nothing, with a NaN among its scores its sum passes on
  auto add = [&](const float4 (&o)[kWords], float pm, float pl) {
    const float mn = fmaxf(m, pm), base = mn == -INFINITY ? 0.0f : mn;
    const float f = m == -INFINITY ? 1.0f : exp2f((m - base) * c2);
    const float w = pm == -INFINITY ? 1.0f : exp2f((pm - base) * c2);
    l = l * f + pl * w;
#pragma unroll
    for (int x = 0; x < kWords; ++x) {
      acc[x].x = acc[x].x * f + o[x].x * w;
      acc[x].y = acc[x].y * f + o[x].y * w;
      acc[x].z = acc[x].z * f + o[x].z * w;
      acc[x].w = acc[x].w * f + o[x].w * w;
    }
    m = mn;
  };
  const int slots = part_rows(per);
  const size_t stride = size_t(slots) * (kLatent + 2);
  // the runs that have tiles of the row: they begin before its end, and end behind its first tile
  for (int r0 = it.first + (J == kManyParts ? warp : 0); live && r0 < it.runs && run_lo(r0) < end; r0 += kStep * kBatch) {
    float4 o[kBatch][kWords];
    float2 ml[kBatch];
    bool has[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = r0 + b * kStep;
      const int64_t lo = run_lo(r), hi = run_lo(r + 1);
      has[b] = r < it.runs && lo < end && hi > it.item && hi > lo;
      if (!has[b]) continue;
      const float* s = part + ((size_t(r) * groups + group) * 2 + (r == it.first ? 1 : 0)) * stride;
      ml[b] = __ldcg(reinterpret_cast<const float2*>(s + size_t(slots) * kLatent + 2 * h));
#pragma unroll
      for (int x = 0; x < kWords; ++x)
        o[b][x] = __ldcg(reinterpret_cast<const float4*>(s + size_t(h) * kLatent + ch + 128 * x));
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (has[b]) add(o[b], ml[b].x, ml[b].y);
  }
  if (J == kManyParts) {  // the first warp adds the others' parts in their order
    __shared__ float4 s_o[8][32];
    __shared__ float2 s_ml[8];
    s_o[warp][lane] = acc[0];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) return;
    for (int x = 1; x < 8; ++x) {
      float4 o[kWords];
      o[0] = s_o[x][lane];
      add(o, s_ml[x].x, s_ml[x].y);
    }
  }
  if (!live) return;
  const bool none = m == -INFINITY && l == 0.0f;
  const float inv = none ? 0.0f : 1.0f / l;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(it.row) * p.o_ts + head * p.o_hs + ch;
#pragma unroll
  for (int x = 0; x < kWords; ++x) {
    uint2 v = make_uint2(0, 0);
    if (!none)
      v = make_uint2(ptx::pack_bf16(acc[x].x * inv, acc[x].y * inv), ptx::pack_bf16(acc[x].z * inv, acc[x].w * inv));
    *reinterpret_cast<uint2*>(out + 128 * x) = v;
  }
  if (lane == 0 && ch == 0 && p.lse)
    p.lse[int64_t(it.row) * p.H + head] = none ? -INFINITY : (m * c2 + log2f(l)) * kLn2;
}

// Heads split evenly over CTAs of at most 64, whole sixteens where there are several.
int head_groups(int32_t heads) { return (heads + kHeads - 1) / kHeads; }
int heads_per(int32_t heads) {
  const int groups = head_groups(heads), each = (heads + groups - 1) / groups;
  return groups == 1 ? heads : (each + 15) & ~15;
}

}  // namespace

bool latent_tc_supported(kpool_dtype dtype, int32_t latent, int32_t rotary) {
  return dtype == KPOOL_BF16 && latent == kLatent && rotary == kRotary;
}

size_t latent_tc_bytes(int32_t heads) {
  const int groups = head_groups(heads);
  const size_t runs = groups > kMaxRuns ? 1 : kMaxRuns / groups;
  return align256(sizeof(JoinItem) * kMaxRuns) +
         runs * groups * 2 * size_t(part_rows(heads_per(heads))) * (kLatent + 2) * sizeof(float);
}

cudaError_t launch_latent_tc(const LatentParams& p, char* ws, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int per = heads_per(p.H), groups = head_groups(p.H);
  CUtensorMap tq;
  if (!make_tmap_bf16_heads(&tq, p.q, uint64_t(p.R), uint64_t(p.H), kDim, p.q_ts, p.q_hs, 1, kHeads))
    return cudaErrorInvalidValue;
  if (sms > kMaxRuns) sms = kMaxRuns;
  int runs = groups > sms ? 1 : sms / groups;
  // Equal runs of tiles fill the SMs and cost a join (whole rows where lists fill the SMs evenly: 160 rows x 2,052 ids 79.9
  // against 79.3 us); whole rows only where there are more lengths than a CTA adds up.
  const bool direct = !latent_listed(p) && p.R > kMaxRunRows;
  if (!direct && latent_listed(p)) runs = int(run_count(int64_t(p.R) * (id_tiles(p) + kRowCost), runs));
  JoinItem* joins = reinterpret_cast<JoinItem*>(ws + sizeof(WorkspaceHeader));
  float* part = reinterpret_cast<float*>(ws + sizeof(WorkspaceHeader) + align256(sizeof(JoinItem) * kMaxRuns));
  WorkspaceHeader* hdr = reinterpret_cast<WorkspaceHeader*>(ws);
  static std::atomic<uint64_t> ready{0};
  e = allow_dynamic_smem(reinterpret_cast<const void*>(latent_tc_kernel), kSmem, &ready);
  if (e != cudaSuccess) return e;
  latent_tc_kernel<<<runs * groups, kThreads, kSmem, stream>>>(tq, p, per, groups, direct ? 1 : 0, part, joins, hdr);
  e = cudaGetLastError();
  if (e != cudaSuccess || direct || runs < 2) return e;
  cudaLaunchConfig_t cfg{};
  const Join join = join_form(p.R, p.H, runs);
  const int units = join == kFewParts ? p.H : p.H * (kLatent / 128);
  cfg.gridDim = dim3(uint32_t(p.R <= runs ? p.R : runs), uint32_t(join == kManyParts ? units : (units + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = join == kFewParts    ? latent_join_kernel<kFewParts>
                : join == kSomeParts ? latent_join_kernel<kSomeParts>
                                     : latent_join_kernel<kManyParts>;
  e = cudaLaunchKernelEx(&cfg, kernel, p, per, groups, runs, static_cast<const JoinItem*>(joins),
                         static_cast<const float*>(part));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kpool
