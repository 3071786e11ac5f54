// nt_paged_few.cu -- paged attention of sequences with up to 8 query rows per key-value head: single tokens, and two or more
// where few heads share one.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(x_j log2(e) - m)
//
// Such a call is bound by reading keys and values once. Its products are few, so they run on mma.sync (m16n8k16, bf16, fp32 sums): it
// takes 16 rows at least, which the terms of the values share: an fp32 query is three bf16 terms (nothing is lost) in rows of their own,
// its weights three as well, and the rows are summed behind; weights of bf16 queries are two rounded terms (2^-17). (On the fp32 units a block of 16
// keys took 770 instructions, on eight warps of an SM 141 us for 64 sequences of 158,000 rows together; now 122, 5.4 TB/s, with a warp's chain of
// dependent steps next to memory as the bound. A single token over 4,094 rows is latency: 12 us.)
//
// A warp takes a block of 16 keys (D 64: 32) at a time: the scores come out of the MMAs in the places where the weights go in. The
// reference m of a row is raised only when a score exceeds it by 2^8. Accumulators go to sums that round to nearest every kFlush
// blocks, as the tensor core cuts its sums off.
//
// Every warp has a ring of blocks of its own, filled by TMA (boxes of 16 rows, 128-byte swizzle) that runs ahead of the weighing over
// the ends of pieces; the warps of a CTA meet only through the counter that tells the last one of a piece to join their sums.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "nt_tree_attn.cuh"
#include "nt_paged.cuh"

namespace nt {
namespace {

constexpr int kFewKeys = 64;  // keys per tile of the division
constexpr int kFewStart = 5, kFewNear = 6;

__device__ __forceinline__ void load_matrices(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void load_matrices_turned(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = v;
  else *reinterpret_cast<uint2*>(p) = make_uint2(pack_rn(v.x, v.y), pack_rn(v.z, v.w));
}

struct FewMaps {
  CUtensorMap k, v;  // boxes of 64 dimensions x 16 rows
};

template <typename T, int D, int R>
struct FewShape {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kBlock = 2048 / D;          // keys of a warp at a time
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kHalf = kBlock * D * 2;      // a block's keys, or its values: 4 KB
  static constexpr int kPlaces = 6;                 // of a warp's ring: keys and values in turn
  static constexpr int kRing = kWarps * kPlaces * kHalf;
  static constexpr int kSmem = kRing + kWarps * R * D * 4 + 1024;
  // Rows of an MMA: up to four query rows' three terms in rows 0-3, 4-7 and 8-11 of one; eight rows' in 0-7 and 8-15 of one and 0-7 of
  // another.
  static constexpr int kTiles = kF32 && R > 4 ? 2 : 1;
  // Weights: rows 0-3, 8-11 and 4-7 hold the terms of up to four fp32 rows' weights without loss; of eight rows', rows 0-7 and 8-15 two
  // terms and a second MMA the third (1 % longer over memory).
  static constexpr int kTermsP = kF32 ? 3 : 2;
  // 2^-23 of a sum is cut at most for each k-step: 2^-17 over 64 steps.
  static constexpr int kFlush = 64 / (kBlock / 16);
};
// A unit and head that several CTAs share, for the join behind the pieces.
struct FewPart {
  int there, c0, c1, mt, t0, rows, g;
};

template <typename T, int D, int R, bool kExtra>
__global__ void __launch_bounds__(FewShape<T, D, R>::kThreads, 1)
    paged_few_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ PaArgs a) {
  using S = FewShape<T, D, R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // each warp's ring of blocks; the warps' sums of a piece
  constexpr int kFewWarps = S::kWarps, kFewThreads = S::kThreads;
  float(*s_o)[R][D] = reinterpret_cast<float(*)[R][D]>(smem + S::kRing);
  __shared__ float s_m[kFewWarps][R], s_l[kFewWarps][R];
  __shared__ __align__(8) uint64_t bars[kFewWarps * S::kPlaces + 1];
  __shared__ FewPart s_part[2];
  __shared__ int s_fail, s_arrived, s_last[2];
  volatile int* fail = &s_fail;
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
  const int g = lane >> 2, t2 = 2 * (lane & 3);  // an MMA's row (and g + 8) and first column of this lane
  const uint32_t free_bar = smem_u32(bars) + 8 * kFewWarps * S::kPlaces, full0 = smem_u32(bars) + 8 * warp * S::kPlaces;
  if (i < kFewWarps * S::kPlaces + 1) {
    bar_init(smem_u32(bars) + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (i == 0) s_fail = s_arrived = s_part[0].there = s_part[1].there = 0;
  dependent_launch_wait();
  const PaShare<kFewStart> share = pa_share<kFewThreads, kFewKeys, kFewStart>(a, R, kFewNear, reinterpret_cast<int*>(smem));
  __syncthreads();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before copies over the division's scratch
  PaWalk<kFewKeys, kFewStart> walk(a, share, R), ahead = walk;
  uint8_t* ring = smem + warp * S::kPlaces * S::kHalf;

  // What is to be copied runs ahead of what is weighed: the block `next` of the pieces that `ahead` walks over, its pages asked for.
  constexpr int kSubs = S::kBlock / 16;
  PaPiece ap{};
  int next = 0, next_hi = 0, issued = 0;
  // Bit h: no row sees the h-th 16 keys of the block, as the first tile of keys begins before the first one that is seen; their page
  // may be gone. kBad: an entry out of range has been met. (In one register: with another one 64 sequences took 126 us instead of 122.)
  constexpr int kBad = 1 << 8;
  int notes = 0;
  int id[kSubs];
  auto ask = [&] {
    const int32_t* ids = a.table + (int64_t)ap.u.s * a.width;
#pragma unroll
    for (int h = 0; h < kSubs; ++h) id[h] = next + 16 * h < next_hi && !(notes >> h & 1) ? ids[(next + 16 * h) >> a.shift] : -1;
  };
  auto enter = [&] {  // the next piece of which this warp has a block
    for (; ahead.more() && a.fault == 0; ahead.next(a)) {
      ap = ahead.piece(a);
      next = (ap.u.tile0 + ap.t0) * kFewKeys + warp * S::kBlock;
      next_hi = min(ap.u.p1 + 1, (ap.t0 + ap.u.tile0 + ap.n) * kFewKeys);
      if (next < next_hi) {
        notes &= kBad;
#pragma unroll
        for (int h = 0; h < kSubs; ++h) notes |= next + 16 * h + 15 < ap.u.lo ? 1 << h : 0;
        ask();
        return;
      }
    }
    next = next_hi = 0;
  };
  // Keys (an even place of the order) or values of the block at `next`; zeros where no row sees or nothing is there.
  auto copy = [&] {
    if (next >= next_hi) return;
    const int k = issued % S::kPlaces;
    const bool val = issued & 1;
    if (lane == 0) {
      const uint32_t bar = full0 + 8 * k, to = smem_u32(ring + k * S::kHalf);
      bar_expect_tx(bar, S::kHalf);
#pragma unroll
      for (int h = 0; h < kSubs; ++h) {
        const int key = next + 16 * h;
        int y = a.ts;
        if (key < next_hi) {
          if ((unsigned)id[h] < (unsigned)a.n_pages) y = (id[h] << a.shift) + (key & (a.page - 1));
          else if (!(notes >> h & 1)) notes |= kBad;
        }
#pragma unroll
        for (int x = 0; x < D; x += 64) tma_3d(to + h * 32 * D + x * 32, val ? &maps.v : &maps.k, x, y, ap.g, bar);
      }
    }
    ++issued;
    if (!val) return;
    next += kFewWarps * S::kBlock;
    if (next < next_hi) {
      notes &= kBad;  // (only the first block of a piece begins so early)
      ask();
    } else {
      ahead.next(a);
      enter();
    }
  };
  // Dimensions t2, t2 + 1 and t2 + 8, + 9 of every 16 of a row's query; asked for before the first copies wait for their pages.
  const int row = R > 4 ? g : g & 3;
  float2 qf[D / 16][2];
  auto queries = [&](const PaPiece& p) {
    const int ra = p.u.mt * R + min(row, p.u.rows - 1), tok = ra / a.G;
    const T* q = static_cast<const T*>(a.q) + (int64_t)(p.u.t0 + tok) * a.q_stride + (int64_t)(p.g * a.G + ra - tok * a.G) * D + t2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if constexpr (S::kF32) {
          qf[k][y] = *reinterpret_cast<const float2*>(q + k * 16 + y * 8);
        } else {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(q + k * 16 + y * 8);
          qf[k][y] = make_float2(__uint_as_float(w), 0.0f);
        }
      }
  };
  enter();
  if (walk.more()) queries(walk.piece(a));
#pragma unroll 1
  for (int k = 0; k < S::kPlaces; ++k) copy();

  // The warps' sums of a piece: a whole one is written, a part left for the join of the CTAs. Threads from, from + step, ..
  auto join = [&](PaPiece p, int from, int step) {
    const PaUnit& u = p.u;
    const bool split_up = p.n < u.tiles;
    for (int e = from; e < u.rows * (D / 4); e += step) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, s_m[w][r]);
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float f = s_m[w][r] == M ? 1.0f : ex2(s_m[w][r] - M);
        const float4 y = *reinterpret_cast<const float4*>(&s_o[w][r][c]);
        L = fmaf(s_l[w][r], f, L);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
      }
      if (split_up) {
        const int64_t to = (int64_t)p.slot * R + r;
        *reinterpret_cast<float4*>(a.part + to * D + c) = x;
        if (c == 0) a.ml[to] = make_float2(M, L);
      } else {
        const float f = L == 0.0f ? 0.0f : 1.0f / L;  // L = 0: the row sees nothing
        const int ra = u.mt * R + r, tok = ra / a.G;
        T* to = static_cast<T*>(a.out) + ((int64_t)(u.t0 + tok) * a.Hq + p.g * a.G + ra - tok * a.G) * D + c;
        store4(to, make_float4(x.x * f, x.y * f, x.z * f, x.w * f));
      }
    }
    if (split_up && from == 0) {
      walk.parts(p);
      s_part[p.t0 == 0] = FewPart{1, p.c0, p.c1, u.mt, u.t0, u.rows, p.g};
    }
  };
  auto later = [](PaWalk<kFewKeys, kFewStart> w) {  // whether a piece follows this one, which ends with its unit and head
    w.sh.off += w.u.tiles + kFewStart;
    return w.more();
  };
  bool ok = true, last_open = false;
  PaPiece last_piece{};
  int used = 0, pieces = 0;
  for (; walk.more(); walk.next(a), ++pieces) {
    PaPiece p = walk.piece(a);
    const PaUnit& u = p.u;
    auto token = [&](int r) { return (u.mt * R + min(r, u.rows - 1)) / a.G; };  // rows behind the last one repeat it
    auto head = [&](int r) { return p.g * a.G + (u.mt * R + min(r, u.rows - 1)) % a.G; };
    uint32_t q[S::kTiles][D / 16][4];
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t low = 0, high = 0, more = 0;  // rows g and g + 8, and row g of the second MMA
        if constexpr (S::kF32) {
          uint32_t w[3];
          split(qf[k][y].x, qf[k][y].y, w);
          w[1] ^= 0x80008000u;
          if constexpr (R > 4) {
            low = w[0];
            high = w[1];
            more = w[2];
          } else {
            low = g < 4 ? w[0] : w[1];
            high = g < 4 ? w[2] : 0u;
          }
        } else {
          low = R > 4 || g < 4 ? __float_as_uint(qf[k][y].x) : 0u;
        }
        q[0][k][2 * y] = low;
        q[0][k][2 * y + 1] = high;
        if constexpr (S::kTiles > 1) {
          q[S::kTiles - 1][k][2 * y] = more;
          q[S::kTiles - 1][k][2 * y + 1] = 0u;
        }
      }
    {  // the next piece's are asked for while this one is weighed
      PaWalk<kFewKeys, kFewStart> after = walk;
      after.next(a);
      if (after.more()) queries(after.piece(a));
    }
    const int pos = u.len - u.n + token(row);
    const float slope = kExtra && a.slopes ? a.slopes[head(row)] : 0.0f;
    const int hi = min(u.p1 + 1, (p.t0 + u.tile0 + p.n) * kFewKeys);            // no row sees this key or one behind it
    const int64_t sure_lo = max((int64_t)0, (int64_t)u.p1 - a.window + 1);      // every row sees from here
    const int sure_hi = u.p0;                                                   // to here
    constexpr int kCols = S::kBlock / 8;
    const float f = kExtra ? 1.4426950408889634f : a.scale * 1.4426950408889634f;
    const float to_cap = kExtra && a.cap > 0.0f ? a.scale / a.cap : 0.0f;
    const bool mine = R > 4 || g < 4;  // lanes whose row g is a query's
    float o[D / 8][4], sums[D / 8][2], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      sums[n][0] = sums[n][1] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    }
    auto flush = [&] {  // rows g and g + 8 hold the products of a weight's first two terms
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sums[n][e] += o[n][e] + o[n][e + 2];
          o[n][e] = o[n][e + 2] = 0.0f;
        }
    };
    int since = 0;  // blocks since the accumulators were empty

#pragma unroll 1
    for (int base = (u.tile0 + p.t0) * kFewKeys + warp * S::kBlock; base < hi; base += kFewWarps * S::kBlock) {
      auto arrived = [&] {
        ok = ok && bar_wait_warp(full0 + 8 * (used % S::kPlaces), (uint32_t)(used / S::kPlaces) & 1u, fail, a.timeout_ns);
        return smem_u32(ring + used % S::kPlaces * S::kHalf);
      };
      auto read = [&] {  // the place is free again
        __syncwarp();
        ++used;
        copy();
      };
      // 16 bytes (chunk c, 8 dimensions) of key r of a place
      auto chunk = [&](int r, int c) { return (uint32_t)((r >> 4) * 32 * D + (c >> 3) * 2048 + (r & 15) * 128 + (((c & 7) ^ (r & 7)) << 4)); };
      const uint32_t kp = arrived();
      if (!ok) break;
      const bool whole = base >= sure_lo && base + S::kBlock - 1 <= sure_hi;  // every row sees every key
      float s4[S::kTiles][kCols][4], other[S::kTiles][kCols][4];  // even and odd steps: two chains of MMAs, not one
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s4[t][n][e] = other[t][n][e] = 0.0f;
#pragma unroll
      for (int h = 0; h < kSubs; ++h)
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];  // keys 0-7 and 8-15 of the 16, dimensions 0-7 and 8-15 of the step
          load_matrices(kp + chunk(h * 16 + (lane >> 4) * 8 + (lane & 7), 2 * k + (lane >> 3 & 1)), b);
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t) {
            mma_16816(k & 1 ? other[t][2 * h] : s4[t][2 * h], q[t][k], b[0], b[1]);
            mma_16816(k & 1 ? other[t][2 * h + 1] : s4[t][2 * h + 1], q[t][k], b[2], b[3]);
          }
        }
      read();
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s4[t][n][e] += other[t][n][e];
      // The terms' rows together: keys base + 8 n + t2 + e of row g.
      float s[kCols][2];
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = s4[0][n][e];
          if constexpr (S::kF32) {
            if constexpr (R > 4) {
              x += s4[0][n][e + 2] + s4[S::kTiles - 1][n][e];
            } else {  // (rows 12-15 are zero: lanes g and g + 4 get the same sum)
              x += s4[0][n][e + 2];
              x += __shfl_xor_sync(0xffffffffu, x, 16);
            }
          }
          s[n][e] = x;
        }
      unsigned seen = ~0u;
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = base + 8 * n + t2 + e;
          if constexpr (kExtra) {
            float x = s[n][e] * (a.cap > 0.0f ? to_cap : a.scale);
            if (a.cap > 0.0f) x = fabsf(x) < kCapSmall ? cap_series(x, a.cap) : cap_whole(x, a.cap);
            if (a.slopes) x -= slope * (float)(pos - key);
            s[n][e] = x;
          }
          s[n][e] *= f;
          if (!whole && (key > pos || (int64_t)key + a.window <= pos)) {
            s[n][e] = -INFINITY;
            seen &= ~(1u << (2 * n + e));
          }
          mx = fmaxf(mx, s[n][e]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, mine && mx > m + kTaLazy)) {
        const float to = fmaxf(m, mx), corr = to == m ? 1.0f : ex2(m - to);
        l *= corr;
        m = to;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          sums[n][0] *= corr;
          sums[n][1] *= corr;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= corr;
        }
      }
      const float mu = m == -INFINITY ? 0.0f : m;
      uint32_t w[kSubs][4], third[kSubs][2];  // eight rows' third terms: an MMA of their own onto the rows of the first ones
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        const float x = ex2(s[n][0] - mu), y = ex2(s[n][1] - mu);
        l += x + y;
        uint32_t term[S::kTermsP];
        split(x, y, term);
        w[n >> 1][2 * (n & 1)] = mine ? term[0] : S::kTermsP > 2 ? term[S::kTermsP - 1] : 0u;
        third[n >> 1][n & 1] = term[S::kTermsP - 1];
        w[n >> 1][2 * (n & 1) + 1] = mine ? term[1] ^ 0x80008000u : 0u;
      }
      const uint32_t vp = arrived();
      if (!ok) break;
      if (!whole) {
        // A value that is not finite goes to the rows that see it by itself, and out of the products.
        uint4* at = reinterpret_cast<uint4*>(ring + used % S::kPlaces * S::kHalf);
        bool odd = false;
#pragma unroll
        for (int e = 0; e < S::kHalf / 512; ++e) {
          const uint4 v = at[e * 32 + lane];
          odd |= word_bad(v.x) || word_bad(v.y) || word_bad(v.z) || word_bad(v.w);
        }
        if (__any_sync(0xffffffffu, odd)) {
          for (int r = 0; r < S::kBlock; ++r) {
            // (which lane of the row's four has this key's bit)
            const unsigned bits = __shfl_sync(0xffffffffu, seen, (lane & 28) | ((r & 7) >> 1));
            if (!mine || !(bits >> (2 * (r >> 3) + (r & 1)) & 1u)) continue;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(ring + used % S::kPlaces * S::kHalf + chunk(r, n) + 2 * t2);
              if (!isfinite(low_f(v))) sums[n][0] += low_f(v);
              if (!isfinite(high_f(v))) sums[n][1] += high_f(v);
            }
          }
          __syncwarp();
          for (int e = lane; e < S::kHalf / 2; e += 32) {
            uint16_t* v = reinterpret_cast<uint16_t*>(at) + e;
            if ((*v & 0x7f80u) == 0x7f80u) *v = 0;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy over them
          __syncwarp();
        }
      }
#pragma unroll
      for (int h = 0; h < kSubs; ++h)
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t b[4];  // keys 0-7 and 8-15 of two chunks of dimensions
          load_matrices_turned(vp + chunk(h * 16 + (lane >> 3 & 1) * 8 + (lane & 7), 2 * n + (lane >> 4)), b);
          if constexpr (S::kF32 && R > 4) {
            const uint32_t low[4] = {third[h][0], 0u, third[h][1], 0u};
            mma_16816(o[2 * n], low, b[0], b[1]);
            mma_16816(o[2 * n + 1], low, b[2], b[3]);
          }
          mma_16816(o[2 * n], w[h], b[0], b[1]);
          mma_16816(o[2 * n + 1], w[h], b[2], b[3]);
        }
      read();
      if (++since == S::kFlush) {
        flush();
        since = 0;
      }
    }
    flush();
    if constexpr (S::kTermsP > 2 && R <= 4) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) sums[n][e] += __shfl_xor_sync(0xffffffffu, sums[n][e], 16);
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    // the piece before has been joined (the warps do not wait for one another otherwise)
    if (pieces > 0) ok = ok && bar_wait_warp(free_bar, (uint32_t)(pieces - 1) & 1u, fail, a.timeout_ns);
    if (mine) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) *reinterpret_cast<float2*>(&s_o[warp][g][8 * n + t2]) = make_float2(sums[n][0], sums[n][1]);
      if (t2 == 0) {
        s_m[warp][g] = m;
        s_l[warp][g] = l;
      }
    }
    if (!ok) break;
    if (p.t0 + p.n < u.tiles || !later(walk)) {  // the share's last piece: all warps join it, behind the loop
      last_piece = p;
      last_open = true;
      break;
    }
    __threadfence_block();
    __syncwarp();
    int arrived = 0;
    if (lane == 0) arrived = atomicAdd(&s_arrived, 1);
    if (__shfl_sync(0xffffffffu, arrived, 0) != kFewWarps - 1) continue;
    // the last warp to come joins them
    __threadfence_block();
    join(p, lane, 32);
    __syncwarp();
    if (lane == 0) {
      s_arrived = 0;
      __threadfence_block();
      bar_arrive(free_bar);
    }
  }
  if (!ok) {  // every copy must land before the CTA may exit
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
    for (int k = used; k < issued; ++k)
      while (!bar_try(full0 + 8 * (k % S::kPlaces), (uint32_t)(k / S::kPlaces) & 1u))
        if (globaltimer_ns() > deadline) break;
  }
  if (__any_sync(0xffffffffu, notes & kBad) && lane == 0 && a.n_bad) atomicAdd(a.n_bad, 1u);
  __syncthreads();
  if (last_open) join(last_piece, i, kFewThreads);  // (unless a wait ran out somewhere, all warps are here with the same piece)
  __syncthreads();
  if (*fail) {
    if (i == 0 && atomicCAS(a.err, 0u, kTaErrWait) == 0u) a.err[1] = blockIdx.x;
    return;
  }
  // The parts that this CTA has left: whoever comes last joins all of a unit and head.
  if (i < 2) {
    s_last[i] = 0;
    if (s_part[i].there) {
      __threadfence();  // (of this thread for all, which have met it)
      const unsigned before = atomicAdd(a.count + s_part[i].c0, 1u);
      s_last[i] = before == (unsigned)(s_part[i].c1 - s_part[i].c0);
      if (s_last[i]) a.count[s_part[i].c0] = 0;
      __threadfence();
    }
  }
  __syncthreads();
  // A warp takes every eighth part, three asked for at a time; then the warps' sums are joined as those of a piece are. (Unrolled over 16
  // parts this took 4 us: code that an SM has not run yet comes from L2.)
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!s_last[k]) continue;
    const FewPart part = s_part[k];
    constexpr int kItems = R * D / 128, kBatch = 3;  // four dimensions each of a lane's rows
    float4 x[kItems];
    float M[kItems], L[kItems];
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      M[e] = -INFINITY;
      L[e] = 0.0f;
    }
    auto row_of = [&](int e) { return D == 128 ? e : 2 * e + (lane >> 4); };
    const int col = lane * 4 % D;
#pragma unroll 1
    for (int b0 = part.c0 + warp; b0 <= part.c1; b0 += kBatch * kFewWarps) {
      float4 y[kBatch][kItems];
      float2 ml[kBatch][kItems];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int cta = b0 + b * kFewWarps;
        const int64_t from = (int64_t)(2 * min(cta, part.c1) + (cta == part.c0)) * R;
#pragma unroll
        for (int e = 0; e < kItems; ++e) {
          y[b][e] = __ldcg(reinterpret_cast<const float4*>(a.part + (from + row_of(e)) * D + col));
          ml[b][e] = __ldcg(a.ml + from + row_of(e));
          if (cta > part.c1) ml[b][e] = make_float2(-INFINITY, 0.0f);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (b0 + b * kFewWarps > part.c1) break;
#pragma unroll
        for (int e = 0; e < kItems; ++e) {
          const float to = fmaxf(M[e], ml[b][e].x);
          const float f0 = M[e] == to ? 1.0f : ex2(M[e] - to), f1 = ml[b][e].x == to ? 1.0f : ex2(ml[b][e].x - to);
          M[e] = to;
          L[e] = fmaf(L[e], f0, ml[b][e].y * f1);
          x[e] = make_float4(fmaf(x[e].x, f0, y[b][e].x * f1), fmaf(x[e].y, f0, y[b][e].y * f1), fmaf(x[e].z, f0, y[b][e].z * f1),
                             fmaf(x[e].w, f0, y[b][e].w * f1));
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      *reinterpret_cast<float4*>(&s_o[warp][row_of(e)][col]) = x[e];
      if (col == 0) {
        s_m[warp][row_of(e)] = M[e];
        s_l[warp][row_of(e)] = L[e];
      }
    }
    __syncthreads();
    PaPiece whole{};
    whole.u.mt = part.mt;
    whole.u.t0 = part.t0;
    whole.u.rows = part.rows;
    whole.u.tiles = whole.n = 1;
    whole.g = part.g;
    join(whole, i, kFewThreads);
    __syncthreads();
  }
}

template <typename T, int D, int R, bool kExtra>
nt_status launch_few(const FewMaps& maps, const PaArgs& a, cudaStream_t st) {
  using S = FewShape<T, D, R>;
  static std::atomic<int> allowed[64];
  static_assert(S::kRing >= kPageMaxSeqs * (int)sizeof(int), "the division's scratch");
  NT_TRY(allow_smem(paged_few_kernel<T, D, R, kExtra>, S::kSmem, allowed));
  const int ctas = std::min(device_sm_count(), kPaFewCtas);
  NT_CUDA_TRY(launch_kernel(paged_few_kernel<T, D, R, kExtra>, dim3((unsigned)ctas), dim3(S::kThreads), S::kSmem, st, true, maps, a));
  return check_launch("paged_few_kernel");
}
template <typename T, int D>
nt_status launch_few_rows(const FewMaps& maps, const PaArgs& a, int64_t max_rows, cudaStream_t st) {
  const bool extra = a.cap > 0.0f || a.slopes;
  if (max_rows <= 4) return extra ? launch_few<T, D, 4, true>(maps, a, st) : launch_few<T, D, 4, false>(maps, a, st);
  return extra ? launch_few<T, D, 8, true>(maps, a, st) : launch_few<T, D, 8, false>(maps, a, st);
}

}  // namespace

nt_status launch_paged_few(const PaArgs& a, int dtype, int D, int64_t max_rows, cudaStream_t st) {
  FewMaps maps;
  NT_TRY(paged_map(&maps.k, a.k, D, 16, a));
  NT_TRY(paged_map(&maps.v, a.v, D, 16, a));
  if (dtype == NT_F32) return D == 64 ? launch_few_rows<float, 64>(maps, a, max_rows, st) : launch_few_rows<float, 128>(maps, a, max_rows, st);
  return D == 64 ? launch_few_rows<uint16_t, 64>(maps, a, max_rows, st) : launch_few_rows<uint16_t, 128>(maps, a, max_rows, st);
}

}  // namespace nt
