// grpo_index.cuh -- index arithmetic of the head and the embedding that has to
// hold up to their largest sizes, where sums of 31-bit numbers pass 2^31.  Plain
// functions of whole numbers, for the kernels and the host alike.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GRPO_HD __host__ __device__ __forceinline__
#else
#define GRPO_HD inline
#endif

namespace grpo {

// ---------------------------------------------------------------- sort
static constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
static constexpr int kSortOne = 4096;  // tokens that one CTA sorts

// Tokens a CTA of the sort takes: one chunk of up to kSortOne, or up to 256
// chunks of at least 2,048, each of whole groups of threads.
GRPO_HD int64_t sort_chunk(int64_t N) {
  const int64_t least = N > kSortOne ? 2048 : N > 0 ? N : 1, even = (N + 255) / 256;
  return ((even > least ? even : least) + kSortThreads - 1) / kSortThreads * kSortThreads;
}

// The tokens [from, end) of N that a warp has of its CTA's chunk; a part that
// lies behind the last token ends before it begins.  (from + part is formed
// where it is at most N only: the last chunk may end at 2^31.)
struct SortPart {
  int from, end;
};
GRPO_HD SortPart sort_part(int chunk, int cta, int warp, int N) {
  const int part = chunk / kSortWarps, from = cta * chunk + warp * part;
  return SortPart{from, N - from < part ? N : from + part};
}

// ---------------------------------------------------------------- tiles
// Rows of tiles that are taken together, `row` bytes of operands each: 32 MB of
// them, so that they stay in L2 while the columns pass, and no more than the mt
// there are (their product with the columns' tiles is formed in 31 bits).  8,192 x
// 4,096 x 65,536 bf16 takes 2.52 ms, with 16 MB 2.57, with 64 or all 2.68; 16,384 x
// 2,048 x 65,536 2.36, 2.34 and 2.40; the gradient of 8,192 x 2,048 x 65,536 3.91,
// 3.81 and 4.06.
GRPO_HD int rows_together(int64_t row, int64_t mt) {
  const int64_t fit = (32ll << 20) / row, most = mt > 1 ? mt : 1;
  return (int)(fit < 1 ? 1 : fit < most ? fit : most);
}

// Tile u of mt x nt: blocks of mb rows of tiles, in which the rows come first.
struct TilePlace {
  int row, col;
};
GRPO_HD TilePlace tile_place(int u, int mt, int mb, int nt) {
  const int blk = u / (mb * nt), left = u - blk * mb * nt;
  const int across = mt - blk * mb < mb ? mt - blk * mb : mb;
  return TilePlace{blk * mb + left % across, left / across};
}

}  // namespace grpo
