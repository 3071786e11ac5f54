// Checks how the paged attention cuts its work into shares: walks every CTA's pieces as the kernels do and compares them with what the
// joins rely on.
#include <cstdio>
#include <random>
#include <vector>

#include "nt_paged.cuh"

using namespace nt;

template <int kStart>
static int check(const std::vector<int>& tiles, int grid, int near, long* split_jobs) {
  const int jobs = (int)tiles.size();
  std::vector<int64_t> off(jobs + 1, 0);
  for (int j = 0; j < jobs; ++j) off[j + 1] = off[j] + tiles[j] + kStart;
  PaCut<kStart> cut;
  cut.set(off[jobs], grid, near);
  auto job_of = [&](int64_t x) {
    int lo = 0, hi = jobs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (off[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  auto end_of = [&](int c) {  // a share's end
    const int64_t x = cut.from(c);
    if (x >= cut.work) return cut.work;
    const int j = job_of(x);
    return cut.snap(x, off[j], tiles[j] + kStart);
  };
  std::vector<int> done(jobs, 0);
  std::vector<std::vector<int>> who(jobs);
  if (cut.from(0) != 0 || cut.from(cut.ctas) != cut.work) return std::printf("ends\n"), 1;
  for (int c = 0; c < cut.ctas; ++c) {
    const int64_t from = end_of(c), end = end_of(c + 1);
    if (c == 0 && from != 0) return std::printf("the first share\n"), 1;
    if (end < from) return std::printf("shares fall\n"), 1;
    int j = job_of(cut.from(c));
    if (from >= off[j + 1]) ++j;
    bool place[2] = {false, false};
    for (; j < jobs && off[j] + kStart < end && from < end; ++j) {
      const int64_t tile = off[j] + kStart;
      const int t0 = (int)std::max<int64_t>(0, from - tile), n = (int)std::min<int64_t>(tiles[j], end - tile) - t0;
      if (n <= 0) return std::printf("an empty piece\n"), 1;
      if (t0 != done[j]) return std::printf("a gap\n"), 1;
      done[j] += n;
      if (n < tiles[j]) {
        if (place[t0 == 0]) return std::printf("two parts in one place\n"), 1;
        place[t0 == 0] = true;
        who[j].push_back(c);
      }
    }
  }
  for (int j = 0; j < jobs; ++j) {
    if (done[j] != tiles[j]) return std::printf("job %d: %d of %d tiles\n", j, done[j], tiles[j]), 1;
    if (who[j].empty()) continue;
    ++*split_jobs;
    const int c0 = cut.first_from(off[j] + kStart + cut.near) - 1, c1 = cut.first_from(off[j] + kStart + tiles[j] - cut.near + 1) - 1;
    if (who[j].front() != c0 || who[j].back() != c1 || (int)who[j].size() != c1 - c0 + 1) return std::printf("the join's view\n"), 1;
  }
  return 0;
}

int main() {
  std::mt19937 rng(1);
  auto up_to = [&](int n) { return (int)(rng() % (unsigned)n); };
  long split = 0;
  for (int k = 0; k < 40000; ++k) {
    const int jobs = 1 + up_to(k % 4 == 0 ? 3 : k % 4 == 1 ? 20 : k % 4 == 2 ? 200 : 1500), most = 1 + up_to(k % 3 == 0 ? 3 : k % 3 == 1 ? 60 : 2000);
    std::vector<int> tiles(jobs);
    for (int& t : tiles) t = 1 + up_to(most);
    const int grid = k % 7 == 0 ? 1 + up_to(320) : 152, near = 1 + up_to(8);
    int bad = 0;
    switch (up_to(4)) {
      case 0: bad = check<1>(tiles, grid, near, &split); break;
      case 1: bad = check<3>(tiles, grid, near, &split); break;
      case 2: bad = check<5>(tiles, grid, near, &split); break;
      default: bad = check<8>(tiles, grid, near, &split);
    }
    if (bad) return std::printf("case %d: %d jobs of up to %d tiles, grid %d, near %d\n", k, jobs, most, grid, near), 1;
  }
  // far beyond 32 bits
  long none = 0;
  if (check<5>(std::vector<int>(3000, 1 << 24), 152, 6, &none)) return 1;
  std::printf("ok, %ld units split\n", split);
  return split == 0;
}
