// nt_adjust_plan.cuh -- how the logit adjustments split their rows over CTAs: host arithmetic.
#pragma once

#include <algorithm>

namespace nt {

constexpr int kAdjThreads = 256;
constexpr int kAdjPer = 8;                  // tokens per thread
constexpr int kAdjChunk = kAdjPer * kAdjThreads;
constexpr int kAdjPerSm = 4;                // CTAs that an SM holds (64 registers a thread; asking the compiler for 4 cost 2 us)
constexpr int kAdjRows = 16;                // rows of a group at most

// Rows of a group: as many groups as one wave of CTAs holds, alike, or whole waves of them where a group would have
// too many rows (64 rows of 151,936, 75 chunks, 608 CTAs at a time, in a graph: 7 groups 18.5 us, 8 16.1, 10 18.6).
inline int adjust_group(int B, int V, int sms) {
  const int chunks = (V + kAdjChunk - 1) / kAdjChunk;
  const int wave = std::max(1, kAdjPerSm * sms / chunks), least = (B + kAdjRows - 1) / kAdjRows;
  const int groups = std::min(B, (least + wave - 1) / wave * wave);
  return (B + groups - 1) / groups;
}

}  // namespace nt
