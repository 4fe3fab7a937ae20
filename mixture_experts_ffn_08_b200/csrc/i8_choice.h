// Which kernel and which tile an int8 product takes: rules on sizes and the number of SMs alone, in plain
// C++, so that a test can ask them without a GPU.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kI8SmallRows = 32;  // an M-tile of at most this many rows loads this many of A
constexpr int kI8PairTile = 0;    // a tile of 256 x 256 over two SMs; else a tile is named by its width

enum I8Kernel {
  I8_DOT = 0,         // integer dot products, a warp per `channels` channels of all `rows` rows
  I8_SPLIT = 1,       // one round of 128 x bn tiles in ks parts of K, `rows` rows of A loaded
  I8_PERSISTENT = 2,  // bn wide tiles of one SM, or kI8PairTile
};

struct I8Choice {
  I8Kernel kernel;
  int rows, channels;  // I8_DOT; rows also I8_SPLIT
  int bn, ks;
};

inline long long i8_cdiv(long long a, long long b) { return (a + b - 1) / b; }

// out[M, N] of a reduction over K, M >= 1.
inline I8Choice i8_linear_choice(int M, int N, int K, int sms) {
  // One to four rows: dot products, which read each row of A once per channel, where that beats the
  // tensor cores (us, dot products and tensor cores: 2 x 4096 x 7168 7.4 and 8.6, 2 x 256 x 14336 8.5
  // and 7.2, 3 x 6144 x 4096 6.8 and 8.3, 3 x 576 x 7168 7.6 and 5.2, 4 x 512 x 4096 3.0 and 3.8,
  // 4 x 6144 x 4096 9.5 and 8.2).  Two channels per warp for two rows of three blocks per SM or
  // more: 2 x 7168 x 2048 3.9 against 4.6, 2 x 5120 x 2048 3.3 against 3.1.
  const bool few_macs = K <= 4096 && static_cast<long long>(N) * K * (M - 1) <= (48LL << 20);
  if (M == 1 || (M == 2 && K <= 8192) || ((M == 3 || M == 4) && few_macs))
    return {I8_DOT, M, M == 2 && N >= 48LL * sms ? 2 : 1, 0, 0};
  const long long mt = i8_cdiv(M, 128);
  // More 128 x 128 tiles than SMs: persistent, two-SM tiles for more than 128 rows (where those tiles
  // fit one round the other kernel is faster: 512 x 4736 x 4096 11.7 us against 16.2, 256 x 9472 x 1024
  // 6.6 against 9.7)
  if (mt * i8_cdiv(N, 128) > sms) {
    if (M > 128) return {I8_PERSISTENT, 0, 0, kI8PairTile, 1};
    const bool wide = i8_cdiv(i8_cdiv(N, 256), sms) * 2 <= i8_cdiv(i8_cdiv(N, 128), sms);
    return {I8_PERSISTENT, 0, 0, wide ? 256 : 128, 1};
  }
  // One round of tiles of 128 x bn over ks parts of K each: the shortest by this estimate in ns,
  // fitted to 170 shapes of 8 to 512 rows (0.6 % above the best choice, 8 % at most).  A K-block
  // takes its issue or its bytes, and the longer the more CTAs load; a tile its sums; parts an
  // exchange.  Clusters of four do not reach all SMs (144 CTAs of them took two rounds).
  const int KB = static_cast<int>(i8_cdiv(K, 128)), box = M <= 32 ? 32 : (M <= 64 ? 64 : 128);
  int best_bn = 128, best_ks = 1;
  float best = -1.f;
  for (int bn = 32; bn <= 128; bn *= 2)
    for (int ks = 1; ks <= 4 && ks * 2 <= KB + 1; ks *= 2) {
      const long long ctas = mt * i8_cdiv(N, bn) * ks;
      if (ctas > (ks == 4 ? sms - 20 : sms)) continue;
      const float rows = box + bn, sums = bn * box;
      const float issue = 140.f + rows * 0.2f, load = rows * 0.94f;
      const float cost = i8_cdiv(KB, ks) * ((issue > load ? issue : load) + ctas * rows * 0.001f) + sums / 15.f +
                         (ks > 1 ? 200.f + sums * 0.19f : 0.f);
      if (best < 0.f || cost < best) {
        best = cost;
        best_bn = bn;
        best_ks = ks;
      }
    }
  return {I8_SPLIT, box, 0, best_bn, best_ks};
}

// Width of a one-SM tile for m_tiles tiles of about tile_rows rows by `rows` weight rows (both of gate
// and up): the narrower ones where the wide ones leave SMs idle.  Rounds of tiles times the ns that a
// K-block of one takes (as above).  One token through two of eight experts of 4096 x 14336: 75 us, 94
// with tiles of 256 alone; 33 tokens through eight of 256 x 128: 10.5 us against 13.6.  A batch that
// fills the SMs many times keeps the widest tiles, which read the rows of A least often.
inline int i8_tile_width(long long m_tiles, int tile_rows, long long rows, int sms) {
  int best_bn = 256;
  float best = -1.f;
  for (int bn = 256; bn >= 64; bn /= 2) {
    const float r = (tile_rows <= kI8SmallRows ? kI8SmallRows : 128) + bn, issue = 140.f + r * 0.2f, load = r * 0.94f;
    const float cost = i8_cdiv(m_tiles * i8_cdiv(rows, bn), sms) * (issue > load ? issue : load);
    if (best < 0.f || cost < best) {
      best = cost;
      best_bn = bn;
    }
  }
  return best_bn;
}

struct I8ExpertTiles {
  int gate_up, down;  // kI8PairTile or a width
};

// Tiles of the experts' two products, for `pairs` rows over E experts of H x I.
// Two-SM tiles where the average expert has 160 rows or more and the tiles go round the SM pairs
// twice, else one-SM tiles.  Measured on B200, 32 experts of 4096 x 1536: 192 rows each 159 us
// against 177, 128 rows 149 against 138; eight experts of 1024 x 512, 512 rows each (16 x 4 pair
// tiles) 34 against 26.  (The kernels take the schedule from the counts, in both layouts.)
inline I8ExpertTiles i8_expert_tiles(long long pairs, int E, int H, int I, int sms) {
  const bool tall = pairs >= 160LL * E;
  const long long m_tiles = pairs / 128 + (pairs < E ? pairs : E);  // at most
  const int rows = static_cast<int>(pairs / E < 128 ? pairs / E : 128);
  const bool pair_gu = tall && pairs / 256 * (I / 128) >= sms;
  const bool pair_dn = tall && pairs / 256 * ((H + 255) / 256) >= sms;
  return {pair_gu ? kI8PairTile : i8_tile_width(m_tiles, rows, 2LL * I, sms),
          pair_dn ? kI8PairTile : i8_tile_width(m_tiles, rows, H, sms)};
}

}  // namespace moe
