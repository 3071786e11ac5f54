// Checks how the tree attention splits its work: every tile of keys of every tile of rows once, pieces and
// results within the kernel's barriers and the workspace, the join's view of a row tile's parts.
#include <cstdio>
#include <random>
#include <vector>

#include "nt_tree_plan.cuh"

using namespace nt;

static int fail(const char* what, int B, int Hq, int Hkv, int prefix) {
  std::printf("%s: B %d Hq %d Hkv %d prefix %d\n", what, B, Hq, Hkv, prefix);
  return 1;
}

static int check(int B, int Hq, int Hkv, int prefix, bool f32, int* shares, int* several) {
  const TaPlan p = ta_plan(B, Hq, Hkv, prefix, f32, prefix % 2 ? 64 : 128);
  const int R = B * (Hq / Hkv);
  const int64_t groups = (int64_t)Hkv * p.mtiles, work = groups * p.tiles;
  if (p.pre_tiles * (int64_t)kTaKeys < prefix || p.tiles - p.pre_tiles != (B + kTaKeys - 1) / kTaKeys)
    return fail("tiles", B, Hq, Hkv, prefix);
  if ((int64_t)p.mtiles * p.rows < R || (p.few && (p.rows > kTaFewRows || B > kTaFewNodes)) || (R <= kTaFewRows && !p.few)) return fail("rows", B, Hq, Hkv, prefix);
  const int64_t room = ta_split_rows(B, Hq, Hkv) / p.rows;
  *several += p.few && p.mtiles > 1;
  if (p.nsplit > 0) {
    if (p.nsplit > p.tiles || p.units != groups * p.nsplit) return fail("splits", B, Hq, Hkv, prefix);
    if (p.nsplit > 1 && (p.units > room || p.units > kTaFill)) return fail("workspace of splits", B, Hq, Hkv, prefix);
    return 0;
  }
  ++*shares;
  const int ctas = (int)p.units;
  if (p.few || ctas > work) return fail("shares", B, Hq, Hkv, prefix);
  std::vector<char> used(room, 0);
  int64_t next = 0;
  for (int c = 0; c < ctas; ++c) {
    int64_t from = share_from(work, c, ctas);
    const int64_t end = share_from(work, c + 1, ctas);
    if (from != next || end <= from) return fail("a share's ends", B, Hq, Hkv, prefix);
    const int64_t id0 = from / p.tiles;
    for (int piece = 0; from < end; ++piece) {
      const int64_t id = id0 + piece, t0 = from - id * p.tiles, n = std::min(end - id * p.tiles, (int64_t)p.tiles) - t0;
      if (piece >= kTaPieces || n < 1 || t0 < 0 || (piece > 0 && t0 != 0)) return fail("pieces", B, Hq, Hkv, prefix);
      if (share_with(work, from, ctas) != c || share_with(work, from + n - 1, ctas) != c) return fail("whose share", B, Hq, Hkv, prefix);
      if (n < p.tiles) {
        const int64_t slot = c + id;
        if (slot >= room || used[slot]) return fail("workspace of shares", B, Hq, Hkv, prefix);
        used[slot] = 1;
      }
      from += n;
    }
    next = end;
  }
  if (next != work) return fail("the last tile", B, Hq, Hkv, prefix);
  for (int64_t id = 0; id < groups; ++id) {  // the join reads the parts that were written
    const int64_t a = share_with(work, id * p.tiles, ctas), b = share_with(work, (id + 1) * p.tiles - 1, ctas);
    for (int64_t c = a; a != b && c <= b; ++c)
      if (!used[c + id]) return fail("the join's parts", B, Hq, Hkv, prefix);
  }
  return 0;
}

int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  int cases = 0, shares = 0, several = 0;
  for (; cases < 30000; ++cases) {
    const int Hkv = cases % 3 == 0 ? pick(1, 700) : pick(1, 40), Hq = Hkv * pick(1, cases % 5 == 0 ? 64 : 8);
    const int B = pick(1, 256), prefix = (int)((double)(1 << pick(0, 20)) * (rng() % 1000) / 1000.0);
    if (check(B, Hq, Hkv, prefix, cases & 1, &shares, &several)) return 1;
  }
  for (int prefix : {0, 1, 2147483391})
    for (int B : {1, 256})
      for (int Hkv : {1, 8, 152, 153, 608, 609, 4096}) {
        ++cases;
        if (prefix < 100 ? check(B, Hkv, Hkv, prefix, true, &shares, &several) : ta_plan(B, Hkv, Hkv, prefix, true, 128).nsplit < 0) return 1;
      }
  if (shares < 1000 || several < 100) return fail("too few shares, or row tiles of few rows", shares, several, 0, 0);
  std::printf("ok %d (%d in shares, %d in tiles of few rows)\n", cases, shares, several);
  return 0;
}
