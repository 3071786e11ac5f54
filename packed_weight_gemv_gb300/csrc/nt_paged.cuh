// nt_paged.cuh -- what the kernels of the paged attention share: arguments, the work of a call and its division, and the join
// of parts.
//
// A unit is a tile of query rows (a row = one token and one of the G query heads of a key-value head) of one sequence; with every
// key-value head it stands for, it has to pass over the tiles of keys that any of its rows sees. Lengths are known on the device
// only, so every CTA works out the division itself: all (unit, head, tile) in a row, cut into equal shares, one per CTA. A share
// begins and ends anywhere, so a unit's keys may be split over CTAs; then each leaves its part (weighted sum, maximum, sum of weights)
// in the workspace and the one that comes last joins them, in the order of the keys.
#pragma once

#include "nt_pages.cuh"

namespace nt {

constexpr int kPaFewRows = 8;     // rows up to which a sequence's tokens take the kernel without tensor cores
constexpr int kPaFewCtas = 320, kPaManyCtas = 160;  // of a launch at most (the workspace's size, asked for without a device, goes by them)
constexpr int kPaMaxGroup = 64;
constexpr uint64_t kPaTimeoutNs = 2000000000ull;

enum : int { kPaAll = 0, kPaFew = 1, kPaMany = 2 };  // which sequences a launch takes: any; up to kPaFewRows rows; more

// A unit that several CTAs of the tensor-core kernel share, left by the one with its first tile: row r is token tok0 + (rest + r) / G.
struct PaJoin {
  int tok0, head0, rest, rows, last;  // last: the CTA with its last tile; rows 0: nothing to join
};
struct PaArgs {
  const void* q;            // [T][Hq][D], tokens q_stride elements apart
  void* out;                // [T][Hq][D]
  const uint16_t *k, *v;    // [Hkv][ts][D]
  const int32_t *table, *q_start, *length;
  const float* slopes;      // [Hq] or null
  uint32_t* n_bad;
  unsigned int* err;        // the workspace's status header [code, CTA]
  unsigned int* count;      // [units x heads] parts that have arrived, all 0 between calls
  float* part;              // [2 x CTAs][rows][D] weighted sums
  float2* ml;               // [2 x CTAs][rows] (maximum, sum of weights)
  PaJoin* join;             // [CTAs]
  float* scratch;           // [CTAs][2][D][128] sums taken off the tensor cores
  uint64_t timeout_ns;
  int64_t q_stride;
  int64_t jobs;             // places of `count`
  int fault, which;
  int T, S, Hq, Hkv, G, width, page, shift, n_pages, ts;
  int window;               // INT32_MAX: none
  float cap, scale;         // scale = 1 / sqrt(D)
};

#ifdef __CUDACC__
namespace {

// Sequence s as the call sees it.
struct PaSeq {
  int t0, n, len;  // first token, tokens, rows with them
};
__device__ __forceinline__ PaSeq pa_seq(const PaArgs& a, int s) {
  PaSeq q;
  q.t0 = min(max(a.q_start[s], 0), a.T);
  q.n = min(max(a.q_start[s + 1], q.t0), a.T) - q.t0;
  q.len = (int)min(min((int64_t)max(a.length[s], 0), (int64_t)a.width * a.page), (int64_t)INT32_MAX - 1024);
  return q;
}
__device__ __forceinline__ int pa_row_tiles(const PaArgs& a, int n, int rows) {
  const int64_t r = (int64_t)n * a.G;
  if (a.which != kPaAll && (r <= kPaFewRows) != (a.which == kPaFew)) return 0;
  return (int)((r + rows - 1) / rows);
}
struct PaUnit {
  int s, mt;          // sequence, tile of rows
  int t0, n, len;     // as in PaSeq
  int rows;           // live rows
  int p0, p1;         // positions of its first and last token
  int tile0, tiles;   // tiles of keys
};
template <int kKeys>
__device__ __forceinline__ PaUnit pa_unit(const PaArgs& a, const PaSeq& q, int s, int mt, int rows) {
  PaUnit u;
  u.s = s;
  u.mt = mt;
  u.t0 = q.t0;
  u.n = q.n;
  u.len = q.len;
  const int r0 = mt * rows, all = q.n * a.G;
  u.rows = min(rows, all - r0);
  u.p0 = q.len - q.n + r0 / a.G;
  u.p1 = q.len - q.n + (r0 + u.rows - 1) / a.G;
  const int lo = (int)max((int64_t)0, (int64_t)u.p0 - a.window + 1), hi = max(u.p1 + 1, 0);
  u.tile0 = lo / kKeys;
  u.tiles = max(1, (hi + kKeys - 1) / kKeys - u.tile0);  // one, all of it masked, where nothing is seen
  return u;
}

// Exclusive sum over a CTA of kThreads; `total` gets the sum of all. warps: 32 places of shared memory.
template <int kThreads>
__device__ __forceinline__ int64_t pa_scan(int64_t x, int64_t* warps, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t y = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = y;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t z = warps[w];
    if (w < warp) before += z;
    all += z;
  }
  *total = all;
  return before + y - x;
}

// A CTA's share: [from, end) of all work; the unit that `from` falls into, its number, and the work before it.
struct PaShare {
  int64_t work, from, end, off;
  int s, mt, unit;
  int ctas;  // with a share: no more than there are tiles
};
__device__ __forceinline__ int64_t pa_from(int64_t work, int c, int ctas) { return work * c / ctas; }
__device__ __forceinline__ int pa_with(int64_t work, int64_t x, int ctas) { return (int)(((x + 1) * ctas - 1) / work); }

// A unit's work for a head is its tiles and kStart, what beginning and ending a piece costs in tiles.
// starts: S places of shared memory (scratch); all threads of the CTA, every one gets the share.
template <int kThreads, int kKeys, int kStart>
__device__ PaShare pa_share(const PaArgs& a, int rows, int* starts) {
  __shared__ int64_t s_warps[32];
  __shared__ int s_first[3];
  __shared__ int64_t s_off;
  const int i = threadIdx.x;
  int64_t units = 0;
  for (int s0 = 0; s0 < a.S; s0 += kThreads) {
    const int s = s0 + i;
    int64_t total;
    const int64_t at = pa_scan<kThreads>(s < a.S ? pa_row_tiles(a, pa_seq(a, s).n, rows) : 0, s_warps, &total);
    if (s < a.S) starts[s] = (int)(units + at);
    units += total;
  }
  PaShare r{};
  if (units * a.Hkv > a.jobs) return r;  // starts that do not rise name more tokens than there are: no work
  __syncthreads();
  auto tiles = [&](int64_t u, int* s_out, int* mt_out) -> int64_t {
    if (u >= units) return 0;
    int s = 0;
    for (int hi = a.S - 1; s < hi;) {  // the last sequence that starts at u or before
      const int mid = (s + hi + 1) / 2;
      if (starts[mid] <= u) s = mid;
      else hi = mid - 1;
    }
    *s_out = s;
    *mt_out = (int)u - starts[s];
    return (int64_t)(pa_unit<kKeys>(a, pa_seq(a, s), s, *mt_out, rows).tiles + kStart) * a.Hkv;
  };
  int s = 0, mt = 0;
  int64_t mine = 0, at = 0;
  for (int64_t u0 = 0; u0 < units; u0 += kThreads) {
    int64_t total;
    mine = tiles(u0 + i, &s, &mt);
    at = r.work + pa_scan<kThreads>(mine, s_warps, &total);
    r.work += total;
  }
  r.ctas = (int)min((int64_t)gridDim.x, r.work);
  if ((int)blockIdx.x >= r.ctas) return r;  // nothing left for this CTA
  r.from = pa_from(r.work, blockIdx.x, r.ctas);
  r.end = pa_from(r.work, blockIdx.x + 1, r.ctas);
  if (units <= kThreads) {
    if (at <= r.from && r.from < at + mine) {
      s_first[0] = s;
      s_first[1] = mt;
      s_first[2] = i;
      s_off = at;
    }
  } else {
    int64_t sum = 0;
    for (int64_t u0 = 0; u0 < units && sum <= r.from; u0 += kThreads) {
      int64_t total;
      mine = tiles(u0 + i, &s, &mt);
      at = sum + pa_scan<kThreads>(mine, s_warps, &total);
      if (at <= r.from && r.from < at + mine) {
        s_first[0] = s;
        s_first[1] = mt;
        s_first[2] = (int)(u0 + i);
        s_off = at;
      }
      sum += total;
    }
  }
  __syncthreads();
  r.s = s_first[0];
  r.mt = s_first[1];
  r.unit = s_first[2];
  r.off = s_off;
  return r;
}

// A piece of a share: tiles [t0, t0 + n) of one unit and head. The kStart at the front of its work have no tile.
struct PaPiece {
  PaUnit u;
  int g, t0, n;
  int c0, c1;      // CTAs with the unit's first and last tile for this head
  int slot;        // where this CTA leaves its part
  int job;         // unit and head: the place of the counter
};
template <int kKeys, int kStart>
struct PaWalk {
  PaShare sh;
  int rows;
  int g = 0;
  PaSeq q;
  PaUnit u;
  __device__ __forceinline__ PaWalk(const PaArgs& a, const PaShare& share, int rows_) : sh(share), rows(rows_) {
    if (sh.from >= sh.end) return;
    q = pa_seq(a, sh.s);
    u = pa_unit<kKeys>(a, q, sh.s, sh.mt, rows);
    g = (int)((sh.from - sh.off) / (u.tiles + kStart));
    sh.off += (int64_t)g * (u.tiles + kStart);
  }
  // sh.off: the work before this unit and head. A share that ends among the first kStart has no tile of it.
  __device__ __forceinline__ bool more() const { return sh.off + kStart < sh.end; }
  __device__ __forceinline__ PaPiece piece(const PaArgs& a) const {
    PaPiece p;
    p.u = u;
    p.g = g;
    const int64_t tile = sh.off + kStart;  // the first one
    p.t0 = (int)max((int64_t)0, sh.from - tile);
    p.n = (int)min((int64_t)u.tiles, sh.end - tile) - p.t0;
    p.c0 = p.c1 = blockIdx.x;
    p.slot = slot(blockIdx.x);
    p.job = sh.unit * a.Hkv + g;
    return p;
  }
  __device__ __forceinline__ void parts(PaPiece& p) const {  // of a piece that is not all of its unit
    p.c0 = pa_with(sh.work, sh.off + kStart, sh.ctas);
    p.c1 = pa_with(sh.work, sh.off + kStart + u.tiles - 1, sh.ctas);
  }
  // Where CTA c leaves its part of this unit and head: in its first place if its share begins among the unit's tiles.
  __device__ __forceinline__ int slot(int c) const { return 2 * c + (pa_from(sh.work, c, sh.ctas) <= sh.off + kStart); }
  __device__ __forceinline__ void next(const PaArgs& a) {
    sh.off += u.tiles + kStart;
    if (!more()) return;
    if (++g < a.Hkv) return;
    g = 0;
    ++sh.unit;
    ++sh.mt;
    while (sh.mt >= pa_row_tiles(a, q.n, rows)) {  // there is one: work is left
      sh.mt = 0;
      q = pa_seq(a, ++sh.s);
    }
    u = pa_unit<kKeys>(a, q, sh.s, sh.mt, rows);
  }
};

}  // namespace
#endif  // __CUDACC__

// Up to 8 rows of a sequence to a CTA (max_rows: the most that a sequence is expected to have).
nt_status launch_paged_few(const PaArgs& a, int dtype, int D, int64_t max_rows, cudaStream_t st);
// Any number of rows, on the tensor cores.
nt_status launch_paged_many(const PaArgs& a, int dtype, int D, int64_t max_rows, cudaStream_t st);

}  // namespace nt
