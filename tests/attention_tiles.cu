// Prints where the tile numbers of a call lie, by the rule that the attention kernels use, on the host. A case is a line
//   paged rows tt S n cu_q[0..n)      (n = 0: without cu_q, a row per sequence)
// and its answer the numbers of tiles, then sequence and first token of each. cu_q may go on behind its S + 1 entries:
// reading them shows as a sequence that does not exist.
#include <cstdio>
#include <vector>

#include "kpool_attn.cuh"

using namespace kpool;

template <bool kRows, class P>
void print(const P& p, int tt) {
  const int tiles = int(attn_tiles<kRows>(p.R, p.S, tt));
  std::printf("%d", tiles);
  for (int t = 0; t < tiles; ++t) {
    const int b = attn_tile_seq<kRows>(p, t, tt);
    std::printf(" %d %d", b, attn_tile_token<kRows>(p, b, t, tt));
  }
  std::printf("\n");
}

int main() {
  int paged, rows, tt, S, n;
  while (std::scanf("%d %d %d %d %d", &paged, &rows, &tt, &S, &n) == 5) {
    std::vector<int32_t> cu(n);
    for (int32_t& x : cu)
      if (std::scanf("%d", &x) != 1) return 1;
    AttnPagedParams p{};
    p.cu_q = n ? cu.data() : nullptr;
    p.S = S;
    p.R = n ? cu[S] : S;
    if (!paged) print<false>(static_cast<const AttnParams&>(p), tt);
    else if (rows) print<true>(p, tt);
    else print<false>(p, tt);
  }
}
