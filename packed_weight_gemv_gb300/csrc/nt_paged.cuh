// nt_paged.cuh -- what the kernels of the paged attention share: arguments, the work of a call and its division, and the join
// of parts.
//
// A unit is a tile of query rows (a row = one token and one of the G query heads of a key-value head) of one sequence; with every
// key-value head it stands for, it has to pass over the tiles of keys that any of its rows sees. Lengths are known on the device
// only, so every CTA works out the division itself: all (unit, head, tile) in a row, cut into shares that are as good as equal, one per
// CTA. A unit's keys may so be split over CTAs; then each leaves its part (weighted sum, maximum, sum of weights) in the workspace,
// and they are joined in the order of the keys: those of few rows by the CTA that comes last, the others by a kernel behind.
#pragma once

#include <cuda.h>

#include "nt_pages.cuh"

namespace nt {

constexpr int kPaFewRows = 8;     // rows up to which a sequence's tokens take the kernel for few rows
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
  unsigned int* count;      // [kPaFewCtas] parts that have arrived of the unit that a CTA has the first tile of, all 0 between calls
  float* part;              // [2 x CTAs][rows][D] weighted sums
  float2* ml;               // [2 x CTAs][rows] (maximum, sum of weights)
  PaJoin* join;             // [CTAs]
  float* scratch;           // [CTAs][2][D][128] sums taken off the tensor cores
  uint64_t timeout_ns;
  int64_t q_stride;
  int64_t most;             // units x heads that a call can have
  int fault, which;
  int T, S, Hq, Hkv, G, width, page, shift, n_pages, ts;
  int window;               // INT32_MAX: none
  float cap, scale;         // scale = 1 / sqrt(D)
};

// The workspace of a call. What has to be 0 when a call begins stands at places that do not depend on its sizes: a server hands one
// workspace to steps of any sizes, and what one of them leaves behind must not be another's counters. A CTA has the first tile of one
// unit at most that goes on in other CTAs, so the CTA names the counter.
struct PaLayout {
  size_t join, count, part, scratch, ml, bytes;
};
inline PaLayout paged_layout(int T, int Hq, int Hkv, int D) {
  // Parts of a launch take a slot each, two per CTA; on the tensor cores each has up to 256 rows (fewer where the call has), and a
  // CTA's sums beside.
  const int64_t rows = (int64_t)T * (Hq / Hkv), few = 2 * kPaFewCtas * kPaFewRows;
  const int64_t many = rows <= kPaFewRows ? 0 : (int64_t)2 * kPaManyCtas * (rows <= 128 ? 128 : 256);
  const size_t parts = (size_t)(many > few ? many : few), sums = rows <= kPaFewRows ? 0 : (size_t)kPaManyCtas * 2 * 128 * D;
  PaLayout l;
  l.join = kWsHeaderBytes;
  l.count = l.join + (kPaManyCtas * sizeof(PaJoin) + 255) / 256 * 256;
  l.part = l.count + (kPaFewCtas * sizeof(unsigned int) + 255) / 256 * 256;
  l.scratch = l.part + parts * D * sizeof(float);
  l.ml = l.scratch + sums * sizeof(float);
  l.bytes = l.ml + parts * sizeof(float2);
  return l;
}

#ifdef __CUDACC__
namespace {

// cap tanh(y). By tanh(y) = 1 - 2 / (1 + e^2y), within 2^-21 of the cap (with a rounded quotient a tile of 128 keys took three times as
// long); and, for small y, by its series y - y^3/3 + 2 y^5/15 - 17 y^7/315 + 62 y^9/2835 - 1382 y^11/155925, the next term of which is
// 2^-32 of the cap at a quarter: up to there it is taken where the first form's loss of what is small next to 1 would show.
constexpr float kCapSmall = 0.25f;
__device__ __forceinline__ float cap_whole(float y, float cap) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * 2.885390081777927f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));  // within 2^-23 (1 / inf = 0)
  return fmaf(-2.0f * cap, r, cap);
}
__device__ __forceinline__ float cap_series(float y, float cap) {
  const float z = y * y;
  float p = fmaf(z, -0.0088632355f, 0.0218694885f);
  p = fmaf(z, p, -0.0539682540f);
  p = fmaf(z, p, 0.1333333333f);
  p = fmaf(z, p, -0.3333333333f);
  return cap * y * fmaf(z, p, 1.0f);
}

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
  int lo;             // the first key that any of them sees
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
  const int hi = max(u.p1 + 1, 0);
  u.lo = (int)max((int64_t)0, (int64_t)u.p0 - a.window + 1);
  u.tile0 = u.lo / kKeys;
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

__host__ __device__ inline int64_t pa_div(int64_t x, int64_t y) {  // x >= 0, y > 0
  return (x | y) >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// How the work of a call is cut. A unit's work for a head is its tiles and kStart, what beginning and ending a piece costs in tiles.
// Equal shares, whose ends move to that of a unit and head where that is nearer than `near` tiles: a CTA would otherwise begin
// and end a piece for next to nothing.
template <int kStart>
struct PaCut {
  int64_t work, base, near;
  int ctas, rem;
  __host__ __device__ inline void set(int64_t all, int grid, int most) {
    work = all;
    ctas = (int)(all < grid ? all : (int64_t)grid);
    base = ctas ? pa_div(all, ctas) : 0;
    rem = (int)(all - base * ctas);
    near = base / 2 < most ? base / 2 : most;
    if (near < 1) near = 1;
  }
  __host__ __device__ inline int64_t from(int c) const { return base * c + (c < rem ? c : rem); }
  // The first CTA whose share begins at y or behind.
  __host__ __device__ inline int first_from(int64_t y) const {
    const int64_t big = (base + 1) * rem;
    return (int)(y <= big ? pa_div(y + base, base + 1) : rem + pa_div(y - big + base - 1, base));
  }
  // The end x of a share among the work [off, off + w) of a unit and head.
  __host__ __device__ inline int64_t snap(int64_t x, int64_t off, int64_t w) const {
    const int64_t lo = off + kStart + near, hi = off + w - near;
    if (lo > hi) return x - off < off + w - x ? off : off + w;
    return x < lo ? off : x > hi ? off + w : x;
  }
};

// A CTA's share: [from, end) of all work; the unit and head that `from` falls into, and the work before it.
template <int kStart>
struct PaShare {
  PaCut<kStart> cut;
  int64_t from, end, off;
  int s, mt, g;
};

// starts: S places of shared memory (scratch); all threads of the CTA, every one gets the share. near: see PaCut.
template <int kThreads, int kKeys, int kStart>
__device__ PaShare<kStart> pa_share(const PaArgs& a, int rows, int near, int* starts) {
  const int lane = threadIdx.x & 31;
  PaShare<kStart> r{};
  // A few sequences and units: every warp works it out for itself.
  if (a.S <= 32) {
    PaSeq q{};
    int n = 0;
    if (lane < a.S) {
      q = pa_seq(a, lane);
      n = pa_row_tiles(a, q.n, rows);
    }
    int upto = n;
    bool many = n > 32;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int z = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += z;
      many |= upto > 32;  // (before it could overflow)
    }
    if (!__any_sync(0xffffffffu, many)) {
      const int units = __shfl_sync(0xffffffffu, upto, 31);
      if ((int64_t)units * a.Hkv > a.most) return r;  // starts that do not rise name more tokens than there are: no work
      int s = 0;  // of unit `lane`: the sequences that end at or before it
#pragma unroll
      for (int d = 16; d; d /= 2)
        if (__shfl_sync(0xffffffffu, upto, s + d - 1) <= lane) s += d;
      s = min(s, 31);
      const int mt = lane - (__shfl_sync(0xffffffffu, upto, s) - __shfl_sync(0xffffffffu, n, s));
      PaSeq mine;
      mine.t0 = __shfl_sync(0xffffffffu, q.t0, s);
      mine.n = __shfl_sync(0xffffffffu, q.n, s);
      mine.len = __shfl_sync(0xffffffffu, q.len, s);
      int64_t w = 0;
      if (lane < units) w = (int64_t)(pa_unit<kKeys>(a, mine, s, mt, rows).tiles + kStart);
      const int64_t w_all = w * a.Hkv;
      int64_t end = w_all;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int64_t z = __shfl_up_sync(0xffffffffu, end, d);
        if (lane >= d) end += z;
      }
      r.cut.set(__shfl_sync(0xffffffffu, end, 31), gridDim.x, near);
      if ((int)blockIdx.x >= r.cut.ctas) return r;
      const int64_t x0 = r.cut.from(blockIdx.x), x1 = r.cut.from(blockIdx.x + 1);
      const unsigned h0 = __ballot_sync(0xffffffffu, end - w_all <= x0 && x0 < end), h1 = __ballot_sync(0xffffffffu, end - w_all <= x1 && x1 < end);
      const int u0 = __ffs(h0) - 1, u1 = h1 ? __ffs(h1) - 1 : 0;
      const int64_t off0 = __shfl_sync(0xffffffffu, end - w_all, u0), off1 = __shfl_sync(0xffffffffu, end - w_all, u1);
      const int64_t w0 = __shfl_sync(0xffffffffu, w, u0), w1 = __shfl_sync(0xffffffffu, w, u1);
      r.s = __shfl_sync(0xffffffffu, s, u0);
      r.mt = __shfl_sync(0xffffffffu, mt, u0);
      r.g = (int)pa_div(x0 - off0, w0);
      r.off = off0 + r.g * w0;
      r.from = r.cut.snap(x0, r.off, w0);
      r.end = h1 ? r.cut.snap(x1, off1 + pa_div(x1 - off1, w1) * w1, w1) : r.cut.work;
      return r;
    }
  }
  __shared__ int64_t s_warps[32];
  __shared__ int s_first[2];
  __shared__ int64_t s_at[4];  // work before the units of both ends, and a head's
  const int i = threadIdx.x;
  int64_t units = 0;
  for (int s0 = 0; s0 < a.S; s0 += kThreads) {
    const int s = s0 + i;
    int64_t total;
    const int64_t at = pa_scan<kThreads>(s < a.S ? pa_row_tiles(a, pa_seq(a, s).n, rows) : 0, s_warps, &total);
    if (s < a.S) starts[s] = (int)(units + at);
    units += total;
  }
  if (units * a.Hkv > a.most) return r;  // as above
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
  int64_t mine = 0, at = 0, work = 0;
  for (int64_t u0 = 0; u0 < units; u0 += kThreads) {
    int64_t total;
    mine = tiles(u0 + i, &s, &mt);
    at = work + pa_scan<kThreads>(mine, s_warps, &total);
    work += total;
  }
  r.cut.set(work, gridDim.x, near);
  if ((int)blockIdx.x >= r.cut.ctas) return r;  // nothing left for this CTA
  const int64_t x0 = r.cut.from(blockIdx.x), x1 = r.cut.from(blockIdx.x + 1);
  auto found = [&] {
    if (at <= x0 && x0 < at + mine) {
      s_first[0] = s;
      s_first[1] = mt;
      s_at[0] = at;
      s_at[1] = mine / a.Hkv;
    }
    if (at <= x1 && x1 < at + mine) {
      s_at[2] = at;
      s_at[3] = mine / a.Hkv;
    }
  };
  if (units <= kThreads) {
    found();
  } else {
    int64_t sum = 0;
    for (int64_t u0 = 0; u0 < units && sum <= x1; u0 += kThreads) {
      int64_t total;
      mine = tiles(u0 + i, &s, &mt);
      at = sum + pa_scan<kThreads>(mine, s_warps, &total);
      found();
      sum += total;
    }
  }
  __syncthreads();
  r.s = s_first[0];
  r.mt = s_first[1];
  r.g = (int)pa_div(x0 - s_at[0], s_at[1]);
  r.off = s_at[0] + r.g * s_at[1];
  r.from = r.cut.snap(x0, r.off, s_at[1]);
  r.end = x1 < work ? r.cut.snap(x1, s_at[2] + pa_div(x1 - s_at[2], s_at[3]) * s_at[3], s_at[3]) : work;
  return r;
}

// A piece of a share: tiles [t0, t0 + n) of one unit and head. The kStart at the front of its work have no tile.
struct PaPiece {
  PaUnit u;
  int g, t0, n;
  int c0, c1;      // CTAs with the unit's first and last tile for this head (PaWalk::parts)
  int slot;        // where this CTA leaves its part
};
template <int kKeys, int kStart>
struct PaWalk {
  PaShare<kStart> sh;
  int rows;
  PaSeq q;
  PaUnit u;
  __device__ __forceinline__ PaWalk(const PaArgs& a, const PaShare<kStart>& share, int rows_) : sh(share), rows(rows_) {
    if (sh.from >= sh.end) return;
    q = pa_seq(a, sh.s);
    u = pa_unit<kKeys>(a, q, sh.s, sh.mt, rows);
    if (sh.from >= sh.off + u.tiles + kStart) next(a);  // the share begins where this unit and head end
  }
  // sh.off: the work before this unit and head. A share begins and ends with one, or among its tiles.
  __device__ __forceinline__ bool more() const { return sh.off + kStart < sh.end && sh.from < sh.end; }
  __device__ __forceinline__ PaPiece piece(const PaArgs& a) const {
    PaPiece p;
    p.u = u;
    p.g = sh.g;
    const int64_t tile = sh.off + kStart;  // the first one
    p.t0 = (int)max((int64_t)0, sh.from - tile);
    p.n = (int)min((int64_t)u.tiles, sh.end - tile) - p.t0;
    p.c0 = p.c1 = blockIdx.x;
    p.slot = 2 * blockIdx.x + (p.t0 == 0);
    return p;
  }
  // Of a piece that is not all of its unit and head. CTA c leaves its part in place 2 c, c0 in 2 c0 + 1 (its share may have begun with
  // a part of another).
  __device__ __forceinline__ void parts(PaPiece& p) const {
    p.c0 = sh.cut.first_from(sh.off + kStart + sh.cut.near) - 1;
    p.c1 = sh.cut.first_from(sh.off + kStart + u.tiles - sh.cut.near + 1) - 1;
  }
  __device__ __forceinline__ void next(const PaArgs& a) {
    sh.off += u.tiles + kStart;
    if (!more()) return;
    if (++sh.g < a.Hkv) return;
    sh.g = 0;
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

// Boxes of 64 dimensions x box_rows rows of the pool, 128-byte swizzle; rows behind it read as zeros.
nt_status paged_map(CUtensorMap* map, const uint16_t* base, int D, int box_rows, const PaArgs& a);
// Up to 8 rows of a sequence to a CTA (max_rows: the most that a sequence is expected to have).
nt_status launch_paged_few(const PaArgs& a, int dtype, int D, int64_t max_rows, cudaStream_t st);
// Any number of rows, on the tensor cores.
nt_status launch_paged_many(const PaArgs& a, int dtype, int D, int64_t max_rows, cudaStream_t st);

}  // namespace nt
