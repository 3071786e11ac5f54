// nt_tree_plan.cuh -- how the tree attention splits its work over CTAs: host arithmetic, and what the
// kernels share of it.
#pragma once

#include <limits.h>
#include <stdint.h>

#include <algorithm>

namespace nt {

constexpr int kTaKeys = 64;             // keys per tile
constexpr int kTaFill = 152;            // CTAs that fill the GPU once (one per SM of a GB300; the workspace's size, which is asked for without a device, goes by it)
constexpr int kTaPieces = 4;            // tiles of rows that a CTA's share may touch
constexpr int kTaPiece = 12;            // tiles that one more of them costs (with 6, 65 tiles of 64 row tiles took 48.4 us in shares, 46.4 in splits)
// Up to kTaFewRows query rows per key-value head; a split's results stand few_rows(R) rows apart.
constexpr int kTaFewRows = 32;
constexpr int kTaFewNodes = 32;         // nodes whose mask is one word
constexpr int few_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }
constexpr int kTfCluster = 8;           // CTAs of a cluster
constexpr int kTfClusterTiles = 96;     // tiles of keys up to which a cluster takes a head

// Equal shares of `work` tiles: the first tile of CTA c, and the CTA whose share holds tile x.
__host__ __device__ inline int64_t share_from(int64_t work, int c, int ctas) { return work * c / ctas; }
__host__ __device__ inline int64_t share_with(int64_t work, int64_t x, int ctas) { return ((x + 1) * ctas - 1) / work; }

struct TaPlan {
  int few;        // the form for few rows
  int dup, rows, mtiles, tiles, pre_tiles;
  int nsplit;     // 0: every CTA an equal share of all tiles
  int cluster;    // few rows: a cluster holds the splits of a tile of rows and joins them
  int parts;      // splits of a row at most
  int64_t units;  // CTAs
};
// clusters: so many clusters of the form for few rows run at a time.
inline TaPlan ta_form(int B, int Hq, int Hkv, int prefix, bool few, int clusters = 0) {
  TaPlan p;
  const int R = B * (Hq / Hkv);
  p.few = few;
  p.dup = R <= 64 ? 2 : 1;
  p.rows = few ? few_rows(R) : 128 / p.dup;
  p.mtiles = (R + p.rows - 1) / p.rows;
  p.pre_tiles = (int)(((int64_t)prefix + kTaKeys - 1) / kTaKeys);
  p.tiles = p.pre_tiles + (B + kTaKeys - 1) / kTaKeys;
  p.cluster = 0;
  const int64_t groups = (int64_t)Hkv * p.mtiles;
  // A cluster joins its splits over distributed shared memory instead of in a second kernel. From its 8 CTAs' own number of
  // tiles up to 12 tiles each that is the faster way (one node, 8 heads of D 128, in a replayed graph: over 800 keys 5.7 us,
  // in splits 6.2; 4,000 7.3 and 7.8; 8 nodes over 6,000 12.0 and 12.5, over 8,191 14.4 and 13.7). With 8 heads 64 of the
  // SMs have work then.
  if (few && p.tiles >= kTfCluster && p.tiles <= kTfClusterTiles && groups <= clusters) {
    p.cluster = 1;
    p.nsplit = p.parts = kTfCluster;
    p.units = groups * kTfCluster;
    return p;
  }
  // Splits as the GPU holds them, but few enough that what the join spends on one more is worth the tiles it
  // takes off the others. In units of about a seventh of a tile's time (few rows: a quarter of a pair of tiles')
  // the join takes one for a split and its launch 20 (12). Measured: one key-value head of 20 rows over 12,000 keys, D 64:
  // 152 splits 17.7 us, 64 10.9, 32 9.9; one row group of 4 over 200 keys unsplit 5.3 us, in 5 parts 5.9; over 1,500
  // keys in 7 parts 6.3, in 13 6.7, in 2 8.9.
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
  // fill it with little more than once (160: two waves). Equal shares then begin and end within a tile of rows, at
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
// What a form of the plan takes, in hundredths of a microsecond as measured: a call's start and end, each step
// of a CTA (a pair of tiles with few rows, one tile with many), the join. At 32 / 8 heads of 128, fp32, the form for
// few rows (in splits) and the one for many: 16 nodes over 400 keys 9.0 and 10.7 us, 4,000 13.0 and 15.6, 32,000 36.1 and
// 37.6; 25 nodes 9.2 and 11.7, 16.3 and 16.5, 58.8 and 41.4; bf16, 25 nodes 8.5 and 9.7, 15.0 and 12.8. In a cluster, 12 to
// 32 nodes of 1 and 4 key-value heads over 450 to 6,000 keys, a join of 190 chose the slower form by 0.01 us on average and
// 0.33 at most (the splits' cost in its place: 0.05 and 0.94).
inline int64_t ta_cost(const TaPlan& p, bool f32, int D) {
  const int at_once = p.few ? 2 : 1;
  const int64_t steps = ((p.tiles + p.nsplit - 1) / p.nsplit + at_once - 1) / at_once * ((p.units + kTaFill - 1) / kTaFill);
  const int64_t join = p.cluster ? 190 : p.nsplit > 1 ? 200 + 8 * p.nsplit : 0;
  if (p.few) return (D == 128 ? 500 : 450) + 100 * steps + join;
  if (D == 128) return (f32 ? 750 : 600) + (p.dup == 2 ? 0 : f32 ? 80 : 100) + (f32 ? 105 : 60) * steps + join;
  return (f32 ? 560 : 460) + (p.dup == 2 ? 0 : f32 ? 40 : 100) + (f32 ? 60 : 50) * steps + join;
}
// Up to kTaFewRows rows the form for few rows; up to kTaFewNodes nodes also in several tiles of rows, where that costs
// less than the form for many: short sequences.
inline TaPlan ta_plan(int B, int Hq, int Hkv, int prefix, bool f32, int D, int clusters = 0) {
  const int R = B * (Hq / Hkv);
  if (R <= kTaFewRows) return ta_form(B, Hq, Hkv, prefix, true, clusters);
  const TaPlan many = ta_form(B, Hq, Hkv, prefix, false);
  if (B > kTaFewNodes || many.nsplit == 0) return many;
  const TaPlan few = ta_form(B, Hq, Hkv, prefix, true, clusters);
  return ta_cost(few, f32, D) < ta_cost(many, f32, D) ? few : many;
}
inline bool ta_joins(const TaPlan& p) { return p.nsplit != 1 && !p.cluster; }  // in a second kernel
// Rows of results that the splits of any prefix take: kTaFill CTAs, and in shares one more for each tile of rows
// (several tiles of few rows take less).
inline int64_t ta_split_rows(int B, int Hq, int Hkv) {
  const TaPlan p = ta_form(B, Hq, Hkv, 0, B * (Hq / Hkv) <= kTaFewRows);
  const int64_t groups = (int64_t)Hkv * p.mtiles;
  if (groups > kTaPieces * kTaFill) return (int64_t)kTaFill * kTaFewRows;  // split in the form for few rows at most
  return (kTaFill + groups) * p.rows;
}

}  // namespace nt
