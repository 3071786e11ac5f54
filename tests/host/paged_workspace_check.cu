// Checks where a call of the paged attention keeps what in its workspace: what must be 0 between calls stands where no call of another
// shape writes anything else, and a workspace for the largest numbers of tokens and heads is large enough for fewer.
#include <cstdio>
#include <random>

#include "nt_paged.cuh"

using namespace nt;

int main() {
  std::mt19937 rng(1);
  auto pick = [&](std::initializer_list<int> x) { return x.begin()[rng() % x.size()]; };
  size_t counters = 0, lowest = SIZE_MAX;
  for (int k = 0; k < 20000; ++k) {
    const int Hkv = pick({1, 2, 3, 8, 40}), G = pick({1, 2, 4, 5, 8, 9, 64}), D = pick({64, 128}), T = 1 + (int)(rng() % (unsigned)pick({4, 300, 9000}));
    const PaLayout l = paged_layout(T, Hkv * G, Hkv, D);
    if (k == 0) counters = l.count;
    if (l.count != counters) return std::printf("the counters' place depends on the call\n"), 1;
    if (l.join < kWsHeaderBytes || l.join + kPaManyCtas * sizeof(PaJoin) > l.count) return std::printf("join\n"), 1;
    if (l.count + kPaFewCtas * sizeof(unsigned int) > l.part) return std::printf("the parts begin among the counters\n"), 1;
    if (l.part < lowest) lowest = l.part;
    if (l.part > l.scratch || l.scratch > l.ml || l.ml >= l.bytes) return std::printf("order\n"), 1;
    if (l.part % 256 || l.scratch % 256 || l.ml % 256) return std::printf("alignment\n"), 1;
    const int64_t rows = (int64_t)T * G, slots = rows <= kPaFewRows ? 0 : 2 * kPaManyCtas;
    if ((l.scratch - l.part) / (4 * D) < (size_t)(2 * kPaFewCtas * kPaFewRows)) return std::printf("parts of few rows\n"), 1;
    if ((l.scratch - l.part) / (4 * D) < (size_t)(slots * (rows <= 128 ? 128 : 256))) return std::printf("parts of many rows\n"), 1;
    if (slots && l.ml - l.scratch < (size_t)kPaManyCtas * 2 * 128 * D * 4) return std::printf("sums\n"), 1;
    const PaLayout fewer = paged_layout(1 + (int)(rng() % (unsigned)T), Hkv * G, Hkv, D);
    if (fewer.bytes > l.bytes) return std::printf("fewer tokens want more\n"), 1;
  }
  if (counters + kPaFewCtas * sizeof(unsigned int) > lowest) return std::printf("the parts of some call begin among the counters\n"), 1;
  std::printf("ok\n");
  return 0;
}
