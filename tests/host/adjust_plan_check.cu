// Checks how the logit adjustments split their rows: every row in one group, groups within the kernel's bounds.
// With arguments B V B V ... it prints the rows of a group of each on a GPU of 152 SMs.
#include <cstdio>
#include <cstdlib>
#include <random>

#include "nt_adjust_plan.cuh"

using namespace nt;

int main(int argc, char** argv) {
  if (argc > 1) {
    for (int i = 1; i + 1 < argc; i += 2) std::printf("%d ", adjust_group(std::atoi(argv[i]), std::atoi(argv[i + 1]), 152));
    return 0;
  }
  std::mt19937 rng(1);
  int several = 0, n = 0;
  for (; n < 20000; ++n) {
    const int B = 1 + rng() % (n % 3 ? 300 : 65535), V = 1 + rng() % (n % 5 ? 300000 : 2147418110), sms = n % 2 ? 152 : 1 + rng() % 300;
    const int group = adjust_group(B, V, sms), groups = (B + group - 1) / group;
    if (group < 1 || group > kAdjRows || (long long)group * groups < B || (long long)group * (groups - 1) >= B || groups > 65535) {
      std::printf("B %d V %d SMs %d: groups of %d\n", B, V, sms, group);
      return 1;
    }
    several += group > 1;
  }
  std::printf("ok %d shapes, %d with several rows to a group\n", n, several);
  return 0;
}
