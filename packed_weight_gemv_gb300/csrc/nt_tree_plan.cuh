// nt_tree_plan.cuh -- how the tree attention splits its work over CTAs: host arithmetic, and what the
// kernels share of it.
#pragma once

#include <limits.h>
#include <stdint.h>

#include <algorithm>

namespace nt {

constexpr int kTaKeys = 64;             // keys per tile
constexpr int kTaFill = 152;            // CTAs that fill the GPU once (one per SM)
constexpr int kTaPieces = 4;            // tiles of rows that a CTA's share may touch
constexpr int kTaPiece = 12;            // tiles that one more of them costs (with 6, 65 tiles of 64 row tiles took 48.4 us in shares, 46.4 in splits)
// Up to kTaFewRows query rows per key-value head; a split's results stand few_rows(R) rows apart.
constexpr int kTaFewRows = 32;
constexpr int few_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }

// Equal shares of `work` tiles: the first tile of CTA c, and the CTA whose share holds tile x.
__host__ __device__ inline int64_t share_from(int64_t work, int c, int ctas) { return work * c / ctas; }
__host__ __device__ inline int64_t share_with(int64_t work, int64_t x, int ctas) { return ((x + 1) * ctas - 1) / work; }

struct TaPlan {
  int dup, rows, mtiles, tiles, pre_tiles;
  int nsplit;     // 0: every CTA an equal share of all tiles
  int parts;      // splits of a row at most
  int64_t units;  // CTAs
};
inline TaPlan ta_plan(int B, int Hq, int Hkv, int prefix) {
  TaPlan p;
  const int R = B * (Hq / Hkv);
  p.dup = R <= 64 ? 2 : 1;
  p.rows = R <= kTaFewRows ? few_rows(R) : 128 / p.dup;
  p.mtiles = (R + p.rows - 1) / p.rows;
  p.pre_tiles = (int)(((int64_t)prefix + kTaKeys - 1) / kTaKeys);
  p.tiles = p.pre_tiles + (B + kTaKeys - 1) / kTaKeys;
  const int64_t groups = (int64_t)Hkv * p.mtiles;
  // Splits as the GPU holds them, but few enough that what the join spends on one more is worth the tiles it
  // takes off the others. In units of about a seventh of a tile's time (few rows: a quarter of a pair of tiles')
  // the join takes one for a split and its launch 20 (12). Measured: one key-value head of 20 rows over 12,000 keys, D 64:
  // 152 splits 17.7 us, 64 10.9, 32 9.9; one row group of 4 over 200 keys unsplit 5.3 us, in 5 parts 5.9; over 1,500
  // keys in 7 parts 6.3, in 13 6.7, in 2 8.9.
  const bool few = R <= kTaFewRows;
  const int most = (int)std::max<int64_t>(1, std::min<int64_t>(p.tiles, kTaFill / groups));
  const int at_once = few ? 2 : 1, step = few ? 4 : 7, launch = few ? 12 : 20;
  p.nsplit = most;
  for (int steps = ((p.tiles + most - 1) / most + at_once - 1) / at_once, best = INT_MAX; step * steps < best; ++steps) {
    const int n = std::min(most, (p.tiles + at_once * steps - 1) / (at_once * steps));
    const int cost = step * steps + n + (n > 1 ? launch : 0);
    if (cost < best) {
      best = cost;
      p.nsplit = n;
    }
    if (n == 1) break;
  }
  p.units = groups * p.nsplit;
  p.parts = p.nsplit;
  // Whole splits leave SMs idle where they do not fill the GPU (64 tiles of rows: 128 CTAs of two splits), or
  // fill it with little more than once (160: two rounds). Equal shares then begin and end within a tile of rows, at
  // the cost of a second start and end, about kTaPiece tiles.
  const int64_t work = groups * p.tiles, share = (work + kTaFill - 1) / kTaFill;
  const int64_t pieces = (share + p.tiles - 2) / p.tiles + 1;
  const int64_t rounds = (p.units + kTaFill - 1) / kTaFill * ((p.tiles + p.nsplit - 1) / p.nsplit) + (p.nsplit > 1 ? 3 : 0);
  if (!few && work >= kTaFill && pieces <= kTaPieces && share + 3 + kTaPiece * (pieces - 1) < rounds) {
    p.nsplit = 0;
    p.units = kTaFill;
    p.parts = (int)std::min<int64_t>(p.units, (p.tiles + share - 2) / share + 1);
  }
  return p;
}
inline bool ta_joins(const TaPlan& p) { return p.nsplit != 1; }
// Rows of results that the splits of any prefix take: kTaFill CTAs, and in shares one more for each tile of rows.
inline int64_t ta_split_rows(const TaPlan& p, int64_t groups) {
  if (groups > kTaPieces * kTaFill) return 0;  // never split
  return (kTaFill + groups) * p.rows;
}

}  // namespace nt
