// nt_pages.cuh -- what the calls over a paged cache share: pages, and the arguments of the bookkeeping kernels.
#pragma once

#include <atomic>

#include "nt_kernels.cuh"

namespace nt {

constexpr int kPageMaxSeqs = 4096;          // sequences of a call
constexpr int kPagedMaxTokens = 1 << 20;    // new tokens of a call
constexpr int kCopyPairs = 1024;            // pairs that a CTA of the copy holds at a time
constexpr int kPageMaxPairs = 1 << 30;      // of a copy or a compaction: 2 n stays an int
constexpr int kBeamMaxRows = 65536;         // rows of logits of a beam selection
constexpr int kBeamMaxVocab = 1 << 24;
constexpr int kFaultPaged = 6;              // nt_set_test_fault: nt_paged_attention issues no copies

inline bool page_ok(int page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }
inline int page_shift(int page) {
  int s = 0;
  while (1 << s < page) ++s;
  return s;
}
inline bool overlap(const void* x, size_t nx, const void* y, size_t ny) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + ny && b < a + nx;
}
// Pages that `rows` rows take.
__host__ __device__ inline int pages_of(int rows, int shift) { return (int)(((int64_t)rows + (1 << shift) - 1) >> shift); }

struct ForkArgs {
  const int32_t *table, *length, *parent;
  int32_t *refs, *table_out, *length_out;
  uint32_t* n_bad;
  int S_in, S_out, width, page, page_shift, n_pages;
};
struct ExtendArgs {
  int32_t *table, *length;
  const int32_t* q_start;
  int32_t *refs, *rows, *pos, *pairs;
  uint32_t* n_bad;
  int S, width, T, page, page_shift, n_pages, wide;  // wide: refs stands on a 16-byte boundary
};
struct CopyArgs {
  uint16_t* kc[128];
  uint16_t* vc[128];
  const int32_t* pairs;
  int n, shares, jobs, Hkv, D, ts, page, n_pages;  // shares: CTAs of a job
};
struct CompactArgs {
  int32_t *refs, *table;
  const int32_t* length;
  int32_t *pairs, *n_used;
  uint32_t* n_bad;
  int32_t* map;  // where each page goes
  int n_pages, S, width, page_shift, cap;
};

// A kernel's dynamic shared memory beyond 48 KB, allowed once per device (done: the kernel's own flags).
template <typename K>
nt_status allow_smem(K* kern, int bytes, std::atomic<int> (&done)[64]) {
  int dev = 0;
  NT_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return set_error(NT_ERR_CUDA, "device index out of range");
  if (done[dev].load(std::memory_order_acquire)) return NT_OK;
  NT_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  done[dev].store(1, std::memory_order_release);
  return NT_OK;
}

}  // namespace nt
