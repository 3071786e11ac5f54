// Checks the tree attention's plans with clusters, as a GPU gives them: what runs is what the plan says and what its cost was
// formed from. A cluster holds all of a tile of rows' splits, none of them empty, and needs no second kernel.
#include <cstdio>
#include <random>

#include "nt_tree_plan.cuh"

using namespace nt;

int main() {
  std::mt19937 rng(5);
  int n = 0, clustered = 0, several = 0, other = 0;
  for (; n < 30000; ++n) {
    const int Hkv = 1 + rng() % (n % 3 ? 8 : 40), Hq = Hkv * (1 + rng() % 9), B = 1 + rng() % (n % 4 ? 32 : 256), D = n % 2 ? 64 : 128;
    const int prefix = rng() % (n % 5 ? 8000 : 40000), clusters = rng() % 24;
    const bool f32 = rng() % 2;
    const TaPlan p = ta_plan(B, Hq, Hkv, prefix, f32, D, clusters), q = ta_plan(B, Hq, Hkv, prefix, f32, D, 0);
    const int64_t groups = (int64_t)Hkv * p.mtiles;
    const bool fits = p.few && p.tiles >= kTfCluster && p.tiles <= kTfClusterTiles && groups <= clusters;
    const char* bad = nullptr;
    if (q.cluster) bad = "a cluster where none runs";
    else if (!!p.cluster != fits) bad = "a cluster where the rule has none, or none where it has one";
    else if (p.cluster && (p.nsplit != kTfCluster || p.parts != p.nsplit || p.units != groups * p.nsplit || ta_joins(p))) bad = "a cluster's splits";
    else if (p.cluster && p.tiles < p.nsplit) bad = "an empty split";
    else if (!p.cluster && ta_joins(p) != (p.nsplit != 1)) bad = "the join";
    else if (p.few && B * (Hq / Hkv) > kTaFewRows && ta_cost(p, f32, D) >= ta_cost(ta_form(B, Hq, Hkv, prefix, false), f32, D)) bad = "the dearer form";
    if (bad) {
      std::printf("%s: B %d Hq %d Hkv %d prefix %d D %d clusters %d\n", bad, B, Hq, Hkv, prefix, D, clusters);
      return 1;
    }
    clustered += p.cluster;
    several += p.cluster && p.mtiles > 1;
    other += p.few != q.few;
  }
  std::printf("ok %d plans, %d in clusters, %d of those with several tiles of rows, %d of another form than without clusters\n", n, clustered,
              several, other);
  return clustered < 500 || several < 100 || other < 20;
}
