// nt_pages.cu -- the bookkeeping of a paged key-value cache that several sequences share: tables that follow the beams of a
// step, pages for new tokens, copies of shared pages before they are written, and compaction.
//
// A page is free when its count (refs) is 0; there is no other list. Pages are given out lowest first and sequences are
// served in order, so the tables that come out do not depend on how the threads run. What is counted with atomics are sums
// of integers, whose order does not matter.
//
// All but the copies are a launch and a few dependent memory round trips: fork, extension and copies of 8 beams over 36 layers are
// 13 us in a replayed graph, of 32 groups of 8 over 4 layers 23. The copies are bound by memory: 1,440 pages of 2 layers (16 rows
// of 8 heads of 128, 378 MB read and written) move at 5.2 TB/s of the 6.7 that a plain copy reaches, a job (layer, tensor, head) to a CTA,
// eight of its pages at a time.
#include <algorithm>

#include "nt_pages.cuh"

namespace nt {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageLayers = 128;
constexpr int kPerThread = 8;  // counts that a thread looks at together

// Exclusive sum over the CTA's 1,024 threads; `total` gets the sum of all.
__device__ __forceinline__ int block_scan(int x, int* warps, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane == 31) warps[warp] = y;
  __syncthreads();
  int w = warps[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int z = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += z;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return y - x + (warp ? before : 0);
}

// CTA r < S_in: the pages of row r gain its children and lose the row itself. Further CTAs: row r - S_in of the new table.
__global__ void __launch_bounds__(128) page_fork_kernel(const ForkArgs a) {
  __shared__ int s_children;
  dependent_launch_wait();
  const int i = threadIdx.x;
  const int most = (int)min((int64_t)a.width * a.page, (int64_t)INT32_MAX);
  if (blockIdx.x < (unsigned)a.S_in) {
    const int r = blockIdx.x;
    const int held = pages_of(min(max(a.length[r], 0), most), a.page_shift);
    int n = 0;
    if (i == 0) s_children = 0;
    __syncthreads();
    for (int s = i; s < a.S_out; s += 128) n += a.parent[s] == r;
    if (n) atomicAdd(&s_children, n);
    __syncthreads();
    const int more = s_children - 1;
    int bad = 0;
    for (int p = i; p < held; p += 128) {
      const int id = a.table[(int64_t)r * a.width + p];
      if ((unsigned)id >= (unsigned)a.n_pages) ++bad;
      else if (more) atomicAdd(a.refs + id, more);
    }
    if (bad && a.n_bad) atomicAdd(a.n_bad, (uint32_t)bad);
    return;
  }
  const int r = blockIdx.x - a.S_in, up = a.parent[r];
  const bool there = (unsigned)up < (unsigned)a.S_in;
  const int len = there ? min(max(a.length[up], 0), most) : 0, held = pages_of(len, a.page_shift);
  if (i == 0) {
    a.length_out[r] = len;
    if (!there && up != -1 && a.n_bad) atomicAdd(a.n_bad, 1u);
  }
  for (int p = i; p < a.width; p += 128) a.table_out[(int64_t)r * a.width + p] = p < held ? a.table[(int64_t)up * a.width + p] : -1;
}

// One CTA. Demands of the sequences, their running sum, and free pages in order until the demand is met; then every free page
// finds the sequence and place that its number among the free ones falls to.
__global__ void __launch_bounds__(kPageThreads) page_extend_kernel(const ExtendArgs a) {
  extern __shared__ int smem[];
  int* upto = smem;              // [S] demands summed up to and with a sequence
  int* hold = upto + a.S;        // [S] the partly filled last page, or -1
  int* first = hold + a.S;       // [S + 1] first token
  int* old = first + a.S + 1;    // [S] length before, or -1: cannot be extended
  __shared__ int s_warps[32];
  __shared__ int s_bad;
  dependent_launch_wait();
  const int i = threadIdx.x;
  // free pages among eight
  auto look = [&](int p0, int (&c)[kPerThread]) {
    int n = 0;
    if (p0 + kPerThread <= a.n_pages && a.wide) {
#pragma unroll
      for (int k = 0; k < kPerThread; k += 4) {
        const int4 v = *reinterpret_cast<const int4*>(a.refs + p0 + k);
        c[k] = v.x; c[k + 1] = v.y; c[k + 2] = v.z; c[k + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kPerThread; ++k) c[k] = p0 + k < a.n_pages ? a.refs[p0 + k] : 1;
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) n += c[k] == 0;
    return n;
  };
  if (i == 0) s_bad = 0;
  int c[kPerThread];
  const int early = look(i * kPerThread, c);  // asked for before anything is known of the demand
  for (int s = i; s <= a.S; s += kPageThreads) first[s] = min(max(a.q_start[s], 0), a.T);
  __syncthreads();
  const int most = (int)min((int64_t)a.width * a.page, (int64_t)INT32_MAX);
  for (int s = i; s < a.S; s += kPageThreads) {
    const int len = a.length[s], n = max(first[s + 1] - first[s], 0);
    int page = -1;
    bool ok = len >= 0 && len <= most - n;
    if (ok && n > 0 && (len & (a.page - 1))) {
      page = a.table[(int64_t)s * a.width + (len >> a.page_shift)];
      ok = (unsigned)page < (unsigned)a.n_pages;
    }
    hold[s] = ok ? page : -1;
    old[s] = ok ? len : -1;
  }
  __syncthreads();
  // Who shares a last page gives it up, in order, until one is alone with it.
  int carry = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPageThreads) {
    const int s = s0 + i;
    int d = 0;
    if (s < a.S && old[s] >= 0) {
      const int n = max(first[s + 1] - first[s], 0), page = hold[s];
      d = pages_of(old[s] + n, a.page_shift) - pages_of(old[s], a.page_shift);
      if (page >= 0) {
        int left = a.refs[page];
        if (left > 1) {
#pragma unroll 8
          for (int t = 0; t < s; ++t) left -= hold[t] == page;
          if (left > 1) d |= 1 << 30;
        }
      }
    }
    const bool copies = d >> 30 & 1;
    d = (d & ~(1 << 30)) + copies;
    int total;
    const int before = block_scan(d, s_warps, &total);
    if (s < a.S) upto[s] = (carry + before + d) | (copies ? INT32_MIN : 0);  // the sign tells that the first page is a copy
    carry += total;
  }
  __syncthreads();
  const int demand = carry;
  auto sum = [&](int s) { return s < 0 ? 0 : upto[s] & INT32_MAX; };
  const int step = kPageThreads * kPerThread;
  int have = 0, before = 0;
  for (int p0 = 0; p0 < a.n_pages && have < demand; p0 += step) {
    int total;
    before = block_scan(p0 == 0 ? early : look(p0 + i * kPerThread, c), s_warps, &total);
    have += total;
  }
  // sequences whose demand, with those before, is not met are left as they were
  int served = 0;  // sequences from the start on
  for (int hi = a.S; served < hi;) {
    const int mid = (served + hi) / 2;
    if (sum(mid) <= have) served = mid + 1;
    else hi = mid;
  }
  const int give = sum(served - 1);
  int given = 0;
  for (int p0 = 0; p0 < a.n_pages && given < give; p0 += step) {
    int total = have;
    const int at = p0 + i * kPerThread;
    int f = before;  // as found above, where one round holds all
    if (a.n_pages > step) f = given + block_scan(look(at, c), s_warps, &total);
    for (int k = 0; k < kPerThread && f < give; ++k) {
      if (c[k] != 0) continue;
      int s = 0;  // the sequence whose share holds number f
      for (int hi = served - 1; s < hi;) {
        const int mid = (s + hi) / 2;
        if (sum(mid) > f) hi = mid;
        else s = mid + 1;
      }
      const int place = f - sum(s - 1) - (upto[s] < 0), pages = pages_of(old[s], a.page_shift);
      a.table[(int64_t)s * a.width + pages + place] = at + k;
      if (place < 0) a.pairs[2 * s + 1] = at + k;
      a.refs[at + k] = 1;
      ++f;
    }
    given += total;
  }
  __syncthreads();
  for (int s = i; s < a.S; s += kPageThreads) {
    const int n = max(first[s + 1] - first[s], 0);
    const bool ok = s < served && old[s] >= 0, copies = ok && upto[s] < 0;
    if (copies) atomicSub(a.refs + hold[s], 1);
    a.pairs[2 * s] = copies ? hold[s] : -1;
    if (!copies) a.pairs[2 * s + 1] = -1;
    if (ok) a.length[s] = old[s] + n;
    else if (n > 0 && a.n_bad) atomicAdd(&s_bad, 1);
  }
  // rows and positions
  for (int t = i; t < a.T; t += kPageThreads) {
    int s = 0;  // the last sequence that starts at t or before
    for (int hi = a.S; s < hi;) {
      const int mid = (s + hi) / 2;
      if (first[mid] <= t) s = mid + 1;
      else hi = mid;
    }
    --s;
    int row = -1, pos = 0;
    if (s >= 0 && t < first[s + 1] && old[s] >= 0) {
      pos = old[s] + t - first[s];
      if (s < served) row = a.table[(int64_t)s * a.width + (pos >> a.page_shift)] * a.page + (pos & (a.page - 1));
    }
    a.rows[t] = row;
    a.pos[t] = pos;
  }
  __syncthreads();
  if (i == 0 && s_bad) atomicAdd(a.n_bad, (uint32_t)s_bad);
}

// Copies of pages: the pairs that are there, then every CTA some of them for one job (layer, keys or values, head) after another, in
// rounds of 256 threads x 16 bytes, eight pages' loaded before any is stored: a page of one head stands in one piece of memory.
__global__ void __launch_bounds__(256) page_copy_kernel(const __grid_constant__ CopyArgs a) {
  __shared__ int2 s_pair[kCopyPairs];
  __shared__ int s_count[8];
  dependent_launch_wait();
  const int i = threadIdx.x;
  const int vecs = a.page * a.D / 8;  // 16-byte pieces of a page of one head
  for (int p0 = 0; p0 < a.n; p0 += kCopyPairs) {
    // in their order: every CTA has the same list
    int n = 0;
    const int end = min(a.n, p0 + kCopyPairs);
    for (int p1 = p0; p1 < end; p1 += 256) {
      const int p = p1 + i;
      const int from = p < end ? a.pairs[2 * p] : -1, to = p < end ? a.pairs[2 * p + 1] : -1;
      const bool there = (unsigned)from < (unsigned)a.n_pages && (unsigned)to < (unsigned)a.n_pages;
      const unsigned who = __ballot_sync(0xffffffffu, there);
      __syncthreads();  // the pairs and counts before have been read
      if ((i & 31) == 0) s_count[i >> 5] = __popc(who);
      __syncthreads();
      int at = n + __popc(who & ((1u << (i & 31)) - 1));
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < i >> 5) at += s_count[w];
        n += s_count[w];
      }
      if (there) s_pair[at] = make_int2(from, to);
    }
    __syncthreads();
    constexpr int kAtOnce = 8;
    for (int job = blockIdx.x % a.jobs; job < a.jobs; job += gridDim.x) {  // (one, unless there are more jobs than CTAs)
      const int lv = job / a.Hkv, h = job - lv * a.Hkv;
      uint4* base = reinterpret_cast<uint4*>(((lv & 1) ? a.vc[lv >> 1] : a.kc[lv >> 1]) + (int64_t)h * a.ts * a.D);
      for (int p = blockIdx.x / a.jobs; p < n; p += a.shares * kAtOnce) {
        for (int e = i; e < vecs; e += 256) {
          uint4 v[kAtOnce];
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k)
            if (p + k * a.shares < n) v[k] = base[(int64_t)s_pair[p + k * a.shares].x * vecs + e];
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k)
            if (p + k * a.shares < n) base[(int64_t)s_pair[p + k * a.shares].y * vecs + e] = v[k];
        }
      }
    }
  }
}

// One CTA: the pages in use (U of them), then the i-th one at U or behind goes to the i-th free one below U.
__global__ void __launch_bounds__(kPageThreads) page_compact_kernel(const CompactArgs a) {
  __shared__ int s_warps[32];
  dependent_launch_wait();
  const int i = threadIdx.x;
  int used = 0;
  for (int p = i; p < a.n_pages; p += kPageThreads) used += a.refs[p] != 0;
  int U;
  block_scan(used, s_warps, &U);
  int from = 0, to = 0;  // pages found so far
  for (int p0 = 0; p0 < a.n_pages; p0 += kPageThreads) {
    const int p = p0 + i;
    const int c = p < a.n_pages ? a.refs[p] : 0;
    const bool is_from = p < a.n_pages && c != 0 && p >= U, is_to = p < a.n_pages && c == 0 && p < U;
    int total;
    const int at = block_scan((is_from ? 1 : 0) | (is_to ? 1 << 16 : 0), s_warps, &total);
    if (is_from) a.pairs[2 * (from + (at & 0xffff))] = p;
    if (is_to) a.pairs[2 * (to + (at >> 16)) + 1] = p;
    if (p < a.n_pages) a.map[p] = p;
    from += total & 0xffff;
    to += total >> 16;
  }
  __syncthreads();  // from == to
  for (int m = i; m < a.cap; m += kPageThreads) {
    if (m >= from) {
      a.pairs[2 * m] = a.pairs[2 * m + 1] = -1;
      continue;
    }
    const int p = a.pairs[2 * m], q = a.pairs[2 * m + 1];
    a.map[p] = q;
    a.refs[q] = a.refs[p];
    a.refs[p] = 0;
  }
  if (i == 0) *a.n_used = U;
}

__global__ void __launch_bounds__(256) page_remap_kernel(const CompactArgs a) {
  dependent_launch_wait();
  const int64_t all = (int64_t)a.S * a.width;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < all; x += (int64_t)gridDim.x * 256) {
    const int s = (int)(x / a.width), p = (int)(x - (int64_t)s * a.width);
    if (p >= pages_of(max(a.length[s], 0), a.page_shift)) continue;
    const int id = a.table[x];
    if ((unsigned)id < (unsigned)a.n_pages) a.table[x] = a.map[id];
    else if (a.n_bad) atomicAdd(a.n_bad, 1u);
  }
}

// ---- host -----------------------------------------------------------------------------------
nt_status check_pages(int page, int n_pages, int width) {
  if (!page_ok(page)) return set_error(NT_ERR_INVALID_ARG, "page must be 16, 32, 64, 128 or 256 rows");
  if (n_pages < 1 || (int64_t)n_pages * page > INT32_MAX) return set_error(NT_ERR_INVALID_ARG, "need n_pages >= 1 and n_pages * page in the int range");
  if (width < 1) return set_error(NT_ERR_INVALID_ARG, "need width >= 1");
  return NT_OK;
}

}  // namespace
}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_page_fork(const int32_t* table, const int32_t* length, int S_in, int width, const int32_t* parent, int S_out, int page,
                       int32_t* refs, int n_pages, int32_t* table_out, int32_t* length_out, uint32_t* n_bad_opt, void* stream) {
  clear_error();
  if (!table || !length || !parent || !refs || !table_out || !length_out) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  NT_TRY(check_pages(page, n_pages, width));
  if (S_in < 1 || S_in > kPageMaxSeqs || S_out < 1 || S_out > kPageMaxSeqs)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= S_in, S_out <= 4096");
  if (!aligned(table, 4) || !aligned(length, 4) || !aligned(parent, 4) || !aligned(refs, 4) || !aligned(table_out, 4) ||
      !aligned(length_out, 4) || (n_bad_opt && !aligned(n_bad_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  const size_t in = (size_t)S_in * width * 4, out = (size_t)S_out * width * 4, li = (size_t)S_in * 4, lo = (size_t)S_out * 4;
  if (overlap(table, in, table_out, out) || overlap(length, li, length_out, lo) || overlap(parent, lo, table_out, out) ||
      overlap(parent, lo, length_out, lo))
    return set_error(NT_ERR_INVALID_ARG, "the new table and lengths must not overlap the old ones or parent");
  NT_TRY(check_device());
  const ForkArgs a{table, length, parent, refs, table_out, length_out, n_bad_opt, S_in, S_out, width, page, page_shift(page), n_pages};
  NT_CUDA_TRY(launch_kernel(page_fork_kernel, dim3((unsigned)(S_in + S_out)), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), true, a));
  return check_launch("page_fork_kernel");
}

nt_status nt_page_extend(int32_t* table, int32_t* length, int S, int width, const int32_t* q_start, int T, int page, int32_t* refs,
                         int n_pages, int32_t* rows, int32_t* pos, int32_t* pairs, uint32_t* n_bad_opt, void* stream) {
  clear_error();
  if (!table || !length || !q_start || !refs || !rows || !pos || !pairs) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  NT_TRY(check_pages(page, n_pages, width));
  if (S < 1 || S > kPageMaxSeqs || T < 1 || T > kPagedMaxTokens)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= S <= 4096 and 1 <= T <= 1048576");
  if (!aligned(table, 4) || !aligned(length, 4) || !aligned(q_start, 4) || !aligned(refs, 4) || !aligned(rows, 4) ||
      !aligned(pos, 4) || !aligned(pairs, 4) || (n_bad_opt && !aligned(n_bad_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  NT_TRY(check_device());
  const ExtendArgs a{table, length, q_start, refs, rows, pos, pairs, n_bad_opt, S, width, T, page, page_shift(page), n_pages, aligned(refs, 16)};
  const size_t smem = ((size_t)4 * S + 1) * sizeof(int);
  static std::atomic<int> allowed[64];
  if (smem > 48 * 1024) NT_TRY(allow_smem(page_extend_kernel, (4 * kPageMaxSeqs + 1) * (int)sizeof(int), allowed));
  NT_CUDA_TRY(launch_kernel(page_extend_kernel, dim3(1), dim3(kPageThreads), smem, reinterpret_cast<cudaStream_t>(stream), true, a));
  return check_launch("page_extend_kernel");
}

nt_status nt_page_copy(uint16_t* const* k_caches, uint16_t* const* v_caches, int n_layers, int Hkv, int D, int t_stride, int page,
                       const int32_t* pairs, int n, void* stream) {
  clear_error();
  if (!k_caches || !v_caches || !pairs) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (!page_ok(page)) return set_error(NT_ERR_INVALID_ARG, "page must be 16, 32, 64, 128 or 256 rows");
  if (n_layers < 1 || Hkv < 1 || Hkv > 65535 || t_stride < page || n < 1 || n > kPageMaxPairs)
    return set_error(NT_ERR_INVALID_ARG, "need n_layers >= 1, 1 <= Hkv <= 65535, t_stride >= page and 1 <= n <= 2^30");
  if (D < 8 || D > 256 || D % 8 != 0) return set_error(NT_ERR_UNSUPPORTED, "head dimension must be a multiple of 8 up to 256");
  if (!aligned(pairs, 4)) return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  for (int i = 0; i < n_layers; ++i) {
    if (!k_caches[i] || !v_caches[i]) return set_error(NT_ERR_INVALID_ARG, "NULL cache");
    if (!aligned(k_caches[i], 16) || !aligned(v_caches[i], 16)) return set_error(NT_ERR_ALIGNMENT, "caches must be 16-byte aligned");
  }
  NT_TRY(check_device());
  for (int l0 = 0; l0 < n_layers; l0 += kPageLayers) {
    const int L = std::min(kPageLayers, n_layers - l0);
    CopyArgs a{};
    std::copy(k_caches + l0, k_caches + l0 + L, a.kc);
    std::copy(v_caches + l0, v_caches + l0 + L, a.vc);
    a.pairs = pairs;
    a.n = n;
    a.jobs = L * 2 * Hkv;
    a.Hkv = Hkv;
    a.D = D;
    a.ts = t_stride;
    a.page = page;
    a.n_pages = t_stride / page;
    // CTAs that fill the GPU, but no more shares of the pairs than there are
    a.shares = std::max(1, std::min(n, (6 * device_sm_count() + a.jobs - 1) / a.jobs));
    const int64_t ctas = std::min<int64_t>((int64_t)a.jobs * a.shares, 1 << 20);
    NT_CUDA_TRY(launch_kernel(page_copy_kernel, dim3((unsigned)ctas), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), true, a));
  }
  return check_launch("page_copy_kernel");
}

nt_status nt_page_compact_workspace_size(int n_pages, size_t* bytes) {
  clear_error();
  if (!bytes || n_pages < 1) return set_error(NT_ERR_INVALID_ARG, "need n_pages >= 1 and a result pointer");
  *bytes = kWsHeaderBytes + (size_t)n_pages * 4;
  return NT_OK;
}

nt_status nt_page_compact(int32_t* refs, int n_pages, int32_t* table, const int32_t* length, int S, int width, int page, int32_t* pairs,
                          int n, int32_t* n_used, uint32_t* n_bad_opt, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (!refs || !table || !length || (!pairs && n != 0) || !n_used) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  NT_TRY(check_pages(page, n_pages, width));
  if (S < 1 || S > kPageMaxSeqs || n < n_pages / 2 || n > kPageMaxPairs)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= S <= 4096 and n_pages / 2 <= n <= 2^30");
  if (!aligned(refs, 4) || !aligned(table, 4) || !aligned(length, 4) || !aligned(pairs, 4) || !aligned(n_used, 4) ||
      (n_bad_opt && !aligned(n_bad_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  if (!ws || !aligned(ws, 16) || ws_bytes < kWsHeaderBytes + (size_t)n_pages * 4)
    return set_error(NT_ERR_WORKSPACE, "workspace NULL, misaligned or smaller than nt_page_compact_workspace_size");
  NT_TRY(check_device());
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const CompactArgs a{refs, table, length, pairs, n_used, n_bad_opt, reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kWsHeaderBytes),
                      n_pages, S, width, page_shift(page), n};
  NT_CUDA_TRY(launch_kernel(page_compact_kernel, dim3(1), dim3(kPageThreads), 0, st, true, a));
  NT_TRY(check_launch("page_compact_kernel"));
  const int64_t blocks = ((int64_t)S * width + 255) / 256;
  NT_CUDA_TRY(launch_kernel(page_remap_kernel, dim3((unsigned)std::min<int64_t>(blocks, 4 * device_sm_count())), dim3(256), 0, st, true, a));
  return check_launch("page_remap_kernel");
}

}  // extern "C"
