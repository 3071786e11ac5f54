// nt_tree_attention.cu -- attention of a drafted token tree over a bf16 key-value cache: every
// node sees the sequence's cached rows and the tree rows its mask names.
//
//   out[b][h] = sum_t p_t v_t / sum_t p_t,   p_t = 2^(q . k_t log2(e) / sqrt(D) - m)
//
// The R = B * Hq / Hkv query rows that share a key-value head read the cache once: they are the
// M side of tcgen05.mma (128 rows to a tile), 64 keys at a time the N side of the scores, and the
// weights, written back to tensor memory, the A operand of the weighted values. (Up to 32 rows have a
// kernel with the sides turned, nt_tree_few.cu, which also takes more of them over shorter sequences.)
//
// Products are exact: queries enter as bf16 terms (three for fp32 queries, which hold every bit of
// a value; one for bf16 queries), keys and values are bf16, and the weights are three bf16 terms
// cut from the fp32 weight without loss (fp32 queries) or two rounded ones (bf16 queries: 2^-18 of
// a weight at most, either way, next to 2^-8 of the output; a third term made 64 nodes over 32K 10 % slower).
// Scores, weights, sums and the output accumulate in fp32.
//
// CTA (384 threads): one tile of rows, one key-value head, a range of 64-key tiles.
//   warps 0, 3     -- (one lane each) 64-row TMA boxes of keys, of values (128-byte swizzle) into a ring;
//   warps 1, 2     -- (one lane each) the scores' MMAs, the weighted values'. One issuer for both spent
//                     its time in waits of 100 to 300 cycles, one behind the other;
//   warps 4-7, 8-11 - two groups (thread = row = tensor-memory lane) that turn the scores of every
//                     other tile into weights, one in its arithmetic while the other waits for a
//                     tile. The reference maximum m of a row is raised only when a score exceeds it
//                     by 2^8, and the accumulator rescaled only then; both groups add to one
//                     accumulator, so they decide on m tile after tile, in turns.
// Up to 64 rows are spread over the lanes: each row stands in two lanes, each of which weighs half of
// every tile's keys with a maximum and sum of its own and leaves zeros elsewhere; their accumulators
// are joined at the end. So the instructions of the softmax, which would otherwise be two warps',
// are shared by four.
// The keys of one head are split over CTAs so that the GPU is filled once; the parts' results
// (weighted sum, m, sum) meet in the workspace and a second kernel joins them.
//
// fp32 queries at D 128 are bound by the tensor pipe and the softmax alike (six bf16 products: 1,690
// cycles per tile, 0.88 us; a tile takes 1.05): 25 nodes over 26,000 keys, 32 / 8 heads, in a replayed graph 35.7 us = 107
// MB at 3.0 TB/s, of which 9.4 us are a call of one tile and 2.5 the join. bf16 queries: 768 cycles per
// tile, 0.6 us taken, and 0.8 us more every 16 tiles: 64 nodes over 32,704 keys 45.4 us = 755 TFLOP/s of the one product that the formula
// asks for. At D 64 the softmax's instructions bound it: 255 nodes over 16,001 keys, 32 / 4 heads, 86 us.
//
// What a node does not see has no part in its result: the rows past the sequence and past the
// tree are beyond the extent of their tensor maps (zeros), masked scores are replaced, and a tree
// value that is not finite is taken out of shared memory before the product and added to the
// nodes that see it at the end.
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>
#include <type_traits>

#include "nt_tree_attn.cuh"

namespace nt {
namespace {

template <typename T, int D>
struct TaShape {
  static constexpr int kTermsQ = sizeof(T) == 4 ? 3 : 1;
  static constexpr int kTermsP = sizeof(T) == 4 ? 3 : 2;
  static constexpr int kSlot = kTaKeys * D * 2;            // bytes of a ring slot: one tile's keys or values
  // Tensor-memory columns: the accumulator, the query terms, a buffer of scores and one of weights for
  // each group. Where they do not fit (fp32 queries, D = 128) the smallest query term is a
  // shared-memory operand (51 cycles per MMA instead of 32), and the weights' terms, which the MMAs read
  // smallest first, take turns in four places of one term each: tile j + 1's go where tile j's have
  // been read, down to the largest. (One buffer of scores and two of weights took 38.4 us at 25
  // nodes over 26K, one of weights and two of scores 39.5.)
  static constexpr int kTermCols = kTaKeys / 2;
  static constexpr bool kTight = D + kTermsQ * D / 2 + 2 * kTaKeys + 2 * kTermsP * kTermCols > kTaTmemCols;
  static constexpr int kTermsQT = kTermsQ - (kTight ? 1 : 0);  // query terms in tensor memory
  static constexpr int kPlaces = kTight ? 4 : 2 * kTermsP;     // of weight terms
  static constexpr int kColO = 0, kColQ = D, kColS = D + kTermsQT * D / 2, kColP = kColS + 2 * kTaKeys;
  // The tensor core cuts its fp32 sums off instead of rounding them: 64 keys cost about 4.4e-7 of the final sum,
  // always toward zero (measured: values of one sign, 1,001 tiles in one accumulator, 4.4e-4). So the accumulator is
  // added to sums that round to nearest, and started afresh, every kFlush tiles: 8 with fp32 queries; 16
  // with bf16 queries, 7e-6, no more than their weights' own rounding.
  static constexpr int kFlush = sizeof(T) == 4 ? 8 : 16;
  // Of the D / 2 dimensions that a thread looks after kSumsT are summed in tensor memory, where it has room, and
  // the others in registers. Once for 16 tiles the softmax stops for it between two tiles (64 bf16 nodes over 32K
  // 46.1 us; inside the loop over tiles, whose code it makes slower, 48.6; without these sums 43.7); more often it is
  // better woven in (fp32, 64 nodes 70.8 us, between tiles 74.9).
  static constexpr bool kBetween = sizeof(T) == 2;
  static constexpr int kSumsT = kBetween ? 32 : 0;
  static constexpr int kColSums = kColP + kPlaces * kTermCols;
  static_assert(!kTight || kTermsP == 3, "the turns of the places");
  // Columns of term t (0 the largest) of tile j's weights.
  __device__ static __forceinline__ int weights(int j, int t) {
    return kColP + kTermCols * (kTight ? (3 * j + 2 - t) & 3 : (j & 1) * kTermsP + t);
  }
  static constexpr int kLowBytes = kTight ? 128 * D * 2 : 0;
  // Ring and query term take 192 KB for either D: a second CTA on an SM would only wait for the first
  // one's tensor memory (with 96 KB at D = 64 a call behind another took 368 us instead of 220).
  static constexpr int kStages = (192 * 1024 - kLowBytes) / kSlot;
  static_assert(kStages % 2 == 0, "keys keep to even slots, values to odd ones but for the ends");
  // The queries pass through the end of the ring on their way to tensor memory: per warp 32 rows of
  // half the dimensions, 16 bytes apart from a multiple of 128 so that a column of rows has no
  // bank conflicts.
  static constexpr int kQRow = D / 2 * (int)sizeof(T), kQPitch = kQRow + 16;
  static constexpr int kQSlot = kStages - (kTaSoftmax * kQPitch + kSlot - 1) / kSlot;  // first ring slot they use
  static constexpr int kPitch = D + 4;                     // floats: staged output rows
  static constexpr int kSmem = kStages * kSlot + kLowBytes + 1024;  // and alignment
  static_assert(kQSlot >= kTaFirst, "the queries' staging slots are filled after them");
  static_assert(kColSums + 2 * kSumsT <= kTaTmemCols, "tensor-memory columns");
  static_assert(128 * kPitch * 4 <= kStages * kSlot, "the output is staged in the ring");
};

// Ring order of a CTA's n tiles: keys of tiles 0 and 1, then keys j + 2 and values j in turn.
__device__ __forceinline__ int ring_key(int j) { return j < 2 ? j : 2 * j - 2; }
__device__ __forceinline__ int ring_val(int j, int n) { return min(2 * j + 3, n + j); }

// kShares: the CTA takes an equal share of all tiles, which may touch several tiles of rows; otherwise a
// split of one of them. (One code for both, with the loop over pieces, took 39.1 us instead of 36.0 at 25 nodes over 26K.)
template <typename T, int D, int DUP, bool kShares>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_attn_kernel(const __grid_constant__ TaMaps maps, const TaArgs a) {
  using S = TaShape<T, D>;
  constexpr int kRows = 128 / DUP;      // rows of a tile
  constexpr int kCols = kTaKeys / DUP;  // keys of a tile that one thread weighs
  constexpr int kDims = D / 2;          // dimensions of a row that one thread looks after outside the tiles
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kBars = 2 * S::kStages + 13;
  constexpr int kPieces = kShares ? kTaPieces : 1;
  __shared__ __align__(8) uint64_t bars[kPieces][kBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_fail, s_bad;
  __shared__ float s_m[128], s_l[2][128];
  volatile int* fail = &s_fail;
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
  int id = 0, g, mt, rows, t0, n;  // tile of rows among those of all heads; its head, place, rows, first tile of keys, tiles
  bool last = true;
  auto locate = [&](int piece) {
    if constexpr (kShares) {
      const int64_t work = (int64_t)a.groups * a.tiles;
      const int64_t from = share_from(work, blockIdx.x, gridDim.x), end = share_from(work, blockIdx.x + 1, gridDim.x);
      const int id0 = (int)(from / a.tiles);
      id = id0 + piece;
      g = id / a.mtiles;
      mt = id % a.mtiles;
      t0 = piece == 0 ? (int)(from - (int64_t)id0 * a.tiles) : 0;
      n = (int)min(end - (int64_t)id * a.tiles, (int64_t)a.tiles) - t0;
      last = (int64_t)(id + 1) * a.tiles >= end;
    } else {
      const int unit = blockIdx.x, sp = unit / a.mtiles % a.nsplit;
      g = unit / a.mtiles / a.nsplit;
      mt = unit % a.mtiles;
      t0 = (int)((int64_t)a.tiles * sp / a.nsplit);
      n = (int)((int64_t)a.tiles * (sp + 1) / a.nsplit) - t0;
    }
    rows = min(kRows, a.R - mt * kRows);
  };
  locate(0);
  // computed here, before the wait below (and with fewer registers spilled)
  asm volatile("" : "+r"(g), "+r"(mt), "+r"(rows), "+r"(t0), "+r"(n));
  for (int x = i; x < kPieces * kBars; x += kTaThreads) {
    const int b = x % kBars - 2 * S::kStages;  // the groups' four warps arrive at pfull and sfree, all eight at qfull and flushed
    bar_init(smem_u32(bars) + 8 * x, b == 2 || b == 3 || b == 6 || b == 7 ? 4 : b == 10 || b == 11 ? kTaSoftmax / 32 : b == 12 ? 2 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (i == 0) {
    s_fail = 0;
    s_bad = 0;
  }
  if (i < 128) s_m[i] = -INFINITY;
  if (warp == kTaScore) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(kTaTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = tmem_slot;
  // The set-up above overlaps the previous kernel; nothing below reads an input before its end.
  dependent_launch_wait();

  // Each piece of a share has barriers of its own.
  for (int piece = 0;; ++piece) {
    const uint32_t full0 = smem_u32(bars[piece]), empty0 = full0 + 8 * S::kStages, sfull0 = empty0 + 8 * S::kStages;
    const uint32_t pfull0 = sfull0 + 16, pvdone0 = pfull0 + 16, sfree0 = pvdone0 + 16;
    const uint32_t readmost0 = sfree0 + 16, qfull = readmost0 + 16, flushed = qfull + 8, drain = flushed + 8;
    auto full = [&](int k) { return full0 + 8 * (k % S::kStages); };
    auto empty = [&](int k) { return empty0 + 8 * (k % S::kStages); };
    auto turn = [&](int k) { return (uint32_t)(k / S::kStages) & 1u; };
    auto slot = [&](int k) { return smem_u32(ring + (k % S::kStages) * S::kSlot); };
    auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, fail, a.timeout_ns); };

    if (warp == kTaKeyLoad || warp == kTaValueLoad) {
      if (elect_one()) {
        const bool val = warp == kTaValueLoad;
        int j = 0;
        for (; j < n && !a.fault; ++j) {
          const int k = val ? ring_val(j, n) : ring_key(j);
          if (k >= S::kStages && !wait(empty(k), turn(k) ^ 1u)) break;
          // The first tiles' keys and values, then the queries (which pass through the ring's end), then
          // the rest: with the whole ring asked for at once the queries arrived 4 us later.
          if (k >= kTaFirst && !wait(qfull, 0)) break;
          const int t = t0 + j;
          const bool tree = t >= a.pre_tiles;
          const CUtensorMap* map = val ? (tree ? &maps.vt : &maps.vp) : (tree ? &maps.kt : &maps.kp);
          const int y = (tree ? t - a.pre_tiles : t) * kTaKeys;
          bar_expect_tx(full(k), S::kSlot);
#pragma unroll
          for (int x = 0; x < D; x += 64) tma_3d(slot(k) + x * kTaKeys * 2, map, x, y, g, full(k));
        }
        // every copy must land before the CTA may exit
        const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
        for (int d = max(0, j - S::kStages); d < j; ++d) {
          const int k = val ? ring_val(d, n) : ring_key(d);
          if (k + S::kStages < 2 * n && *fail == 0) continue;  // its slot has been filled again since
          while (!bar_try(full(k), turn(k)))
            if (globaltimer_ns() > deadline) break;
        }
      }
      __syncwarp();
    } else if (warp == kTaScore) {
      if (elect_one()) {
        bool ok = wait(qfull, 0);
        tm_fence_after();
        for (int j = 0; ok && j < n; ++j) {
          const int k = ring_key(j);
          ok = wait(full(k), turn(k));
          if (ok && j >= 2) ok = wait(sfree0 + 8 * (j & 1), ((j >> 1) - 1) & 1);  // the group's last scores have been taken
          if (!ok) break;
          tm_fence_after();
          const uint32_t d = tmem + S::kColS + (j & 1) * kTaKeys;
          const uint64_t bd = sdesc(slot(k), 16);
          // the smallest terms first: the tensor core cuts its sums off, so a sum loses least while it is small
#pragma unroll
          for (int t = S::kTermsQ - 1; t >= 0; --t)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t b = bd + ((kk >> 2) * (kTaKeys * 128) + (kk & 3) * 32) / 16;
              const uint32_t more = t < S::kTermsQ - 1 || kk > 0;
              if (t < S::kTermsQT)
                mma_tmem_a(d, tmem + S::kColQ + t * (D / 2) + 8 * kk, b, idesc_bf16(kTaKeys, false), more);
              else
                mma_smem_a(d, sdesc(smem_u32(ring + S::kStages * S::kSlot), 16) + ((kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16, b,
                           idesc_bf16(kTaKeys, false), more);
            }
          mma_commit(sfull0 + 8 * (j & 1));
          mma_commit(empty(k));
        }
        mma_commit(drain);
      }
      __syncwarp();
    } else if (warp == kTaValue) {
      if (elect_one()) {
        for (int j = 0; j < n; ++j) {
          const int k = ring_val(j, n);
          const bool fresh = j % S::kFlush == 0;
          bool ok = wait(full(k), turn(k));
          if (fresh && j > 0) ok = ok && wait(flushed, (j / S::kFlush - 1) & 1);  // the other group has taken its part
          if (!ok || !wait(pfull0 + 8 * (j & 1), (j >> 1) & 1)) break;
          tm_fence_after();
          const uint64_t bd = sdesc(slot(k), kTaKeys * 128);
#pragma unroll
          for (int t = S::kTermsP - 1; t >= 0; --t) {
            const uint32_t p = tmem + S::weights(j, t);
#pragma unroll
            for (int kk = 0; kk < kTaKeys / 16; ++kk)  // 16 keys: 2,048 bytes of each 64 dimensions
              mma_tmem_a(tmem + S::kColO, p + 8 * kk, bd + kk * 2048 / 16, idesc_bf16(D, true, t == 1),
                         t < S::kTermsP - 1 || kk > 0 || !fresh);
            if (S::kTight && t == 1) mma_commit(readmost0 + 8 * (j & 1));
          }
          mma_commit(pvdone0 + 8 * (j & 1));
          mma_commit(empty(k));
        }
        mma_commit(drain);
      }
      __syncwarp();
    } else {
      const int quarter = warp & 3, group = (warp - kTaFirstSoftmax) >> 2, ln = quarter * 32 + lane;  // tensor-memory lane
      const int r = ln % kRows, part = ln / kRows;  // row, and which keys of a tile its lane weighs (one for a warp)
      const int b = node_of(mt * kRows + r, a.inv_g);
      const bool live = r < rows;
      const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
      {  // the row's query terms into tensor memory, kDims dimensions each
        constexpr int kVecs = S::kQRow / 16, kAtOnce = 32 / kVecs;  // 16-byte pieces of a part of a row; parts per load
        uint8_t* stage = ring + S::kQSlot * S::kSlot + (warp - kTaFirstSoftmax) * 32 * S::kQPitch;
        uint4 v[kVecs];
#pragma unroll
        for (int e = 0; e < kVecs; ++e) {
          const int ri = (quarter * 32 + e * kAtOnce + lane / kVecs) % kRows, ra = mt * kRows + ri;
          const int rb = node_of(ra, a.inv_g);
          const T* q = static_cast<const T*>(a.q) + ((int64_t)rb * a.Hq + g * a.G + (ra - rb * a.G)) * D + group * kDims;
          v[e] = ri < rows ? reinterpret_cast<const uint4*>(q)[lane % kVecs] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int e = 0; e < kVecs; ++e)
          *reinterpret_cast<uint4*>(stage + (e * kAtOnce + lane / kVecs) * S::kQPitch + lane % kVecs * 16) = v[e];
        __syncwarp();
        const uint4* own = reinterpret_cast<const uint4*>(stage + lane * S::kQPitch);
#pragma unroll 2
        for (int c = 0; c < kDims; c += 16) {
          uint32_t w[S::kTermsQ][8];
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 u = own[c / 4 + e];
              uint32_t x[3], y[3];
              split(__uint_as_float(u.x), __uint_as_float(u.y), x);
              split(__uint_as_float(u.z), __uint_as_float(u.w), y);
#pragma unroll
              for (int t = 0; t < S::kTermsQ; ++t) {
                const uint32_t sign = t == 1 ? 0x80008000u : 0u;
                w[t][2 * e] = x[t] ^ sign;
                w[t][2 * e + 1] = y[t] ^ sign;
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 u = own[c / 8 + e];
              w[0][4 * e] = u.x; w[0][4 * e + 1] = u.y; w[0][4 * e + 2] = u.z; w[0][4 * e + 3] = u.w;
            }
          }
#pragma unroll
          for (int t = 0; t < S::kTermsQT; ++t) tm_st8(tl + S::kColQ + t * (D / 2) + (group * kDims + c) / 2, w[t]);
          if constexpr (S::kTight) {  // rows of 64 dimensions, 16-byte pieces in the order of the 128-byte swizzle
            uint8_t* low = ring + S::kStages * S::kSlot + group * (128 * 128) + ln * 128;
            const uint32_t* x = w[S::kTermsQ - 1];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(low + (((c / 8 + e) ^ (ln & 7)) * 16)) = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
        tm_st_wait();
        tm_fence_before();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before MMAs that read it, copies over the staging slots
        bar_arrive_warp(qfull, lane);
      }
      // warps of rows past the last one only keep the barriers going (their lanes' weights are
      // whatever the columns hold, and reach no row that is read)
      const bool idle = r - lane >= rows;
      const int c0 = part * kCols;  // this thread's first key of a tile
      const uint32_t ocol = tl + S::kColO + group * kDims;  // its half of the accumulator
      const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      float m = -INFINITY, l = 0.0f;  // the lane's reference maximum (log2 units) as this group knows it, its weight sum
      // What the accumulator has been added to, in units of a reference of its own.
      constexpr int kRegs = kDims - S::kSumsT;
      float acc[kRegs > 0 ? kRegs : 1], sums_m = -INFINITY;
      bool summed = false;
      if constexpr (kRegs > 0) {
#pragma unroll
        for (int e = 0; e < kRegs; ++e) acc[e] = 0.0f;
      }
      const uint32_t tsums = tl + S::kColSums + group * S::kSumsT;
      // After a wait that ran out a warp keeps walking the tiles, as the other group's turns need it,
      // and leaves the rest out.
      bool ok = true;
      // Tile j's products have been added. A parity tells a phase from the next one only, so a caller
      // knows of tile j - 2 before it asks for j: room(j) leaves tile j - 2's known.
      auto done = [&](int j) {
        ok = ok && bar_wait_warp(pvdone0 + 8 * (j & 1), (j >> 1) & 1, fail, a.timeout_ns);
        tm_fence_after();
      };
      auto rescale = [&](float to) {  // what this thread holds, to another reference
        const float corr = m == to ? 1.0f : ex2(m - to);
        l *= corr;
        m = to;
        return corr;
      };
      // o, dimensions c .. c + 15 in units of reference `unit`, plus what has been summed of them.
      auto with_sums = [&](int c, float (&o)[16], float scale) {
        if (c < S::kSumsT) {
          if (summed) {
            float old[16];
            tm_load(tsums + c, old);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(old[e], scale, o[e]);
          }
        } else if constexpr (kRegs > 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = fmaf(acc[c - S::kSumsT + e], scale, o[e]);
        }
      };
      // The accumulator before tile j, in units of reference `unit`, to the sums.
      auto flush = [&](int j, float unit) {
        done(j - 1);
        if (ok && !idle) {
          const float scale = sums_m == unit ? 1.0f : ex2(sums_m - unit);
#pragma unroll
          for (int c = 0; c < kDims; c += 16) {
            float o[16];
            tm_load(ocol + c, o);
            with_sums(c, o, scale);
            if (c < S::kSumsT) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e]);
              tm_store(tsums + c, w);
            } else if constexpr (kRegs > 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[c - S::kSumsT + e] = o[e];
            }
          }
          if constexpr (S::kSumsT > 0) tm_st_wait();
          sums_m = unit;
          summed = true;
        }
        tm_fence_before();
        if (ok) bar_arrive_warp(flushed, lane);
      };
      auto room = [&](int j) {  // for tile j's weights: what stood in their places has been read
        if (!S::kTight) {
          if (j >= 2) done(j - 2);
        } else if (j >= 1) {  // all but the largest term of the tile before, and so everything before that
          ok = ok && bar_wait_warp(readmost0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, fail, a.timeout_ns);
          tm_fence_after();
        }
      };
      auto commit = [&]() {
        tm_st_wait();
        tm_fence_before();
        if (ok) bar_arrive_warp(pfull0 + 8 * group, lane);
      };
      float unit = -INFINITY;  // the row's reference before this group's tile
      // The accumulator starts afresh at tiles j0 = kFlush, 2 kFlush, ...: group 1 adds it to the sums after its
      // tile j0 - 1, group 0 with its weights of tile j0 ready.
      for (int j = group, j0 = S::kFlush;; j += 2, j0 += S::kFlush) {
        const int stop = S::kBetween && j0 < n ? j0 - group : n;
        for (; j < n; j += 2) {
          const int t = t0 + j;
          const bool tree = t >= a.pre_tiles;
          ok = ok && bar_wait_warp(sfull0 + 8 * group, (j >> 1) & 1, fail, a.timeout_ns);
          tm_fence_after();
          float s[kCols];
          if (ok && !idle) {
            tm_load(tl + S::kColS + group * kTaKeys + c0, s);
          } else {
#pragma unroll
            for (int c = 0; c < kCols; ++c) s[c] = 0.0f;
          }
          tm_fence_before();
          if (ok) bar_arrive_warp(sfree0 + 8 * group, lane);
          if (tree) {  // take tree values that are not finite out of the product
            const int k = ring_val(j, n);
            ok = ok && bar_wait_warp(full(k), turn(k), fail, a.timeout_ns);
            bool bad = false;
            for (int e = ln; ok && e < S::kSlot / 16; e += 128) {
              uint4* p = reinterpret_cast<uint4*>(ring + (k % S::kStages) * S::kSlot) + e;
              const uint4 v = *p;
              if (word_bad(v.x) || word_bad(v.y) || word_bad(v.z) || word_bad(v.w)) {
                uint16_t* h = reinterpret_cast<uint16_t*>(p);
                for (int x = 0; x < 8; ++x)
                  if ((h[x] & 0x7f80u) == 0x7f80u) h[x] = 0;
                bad = true;
              }
            }
            if (bad) s_bad = 1;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          const int left = tree ? a.B - (t - a.pre_tiles) * kTaKeys : a.prefix - t * kTaKeys;  // keys of the tile
          if (tree || left < kTaKeys) {
            uint64_t seen = ~0ull;
            if (tree) {
              const uint32_t* w = a.mask + (int64_t)(live ? b : 0) * a.words + (t - a.pre_tiles) * 2;
              seen = w[0];
              if (left > 32) seen |= (uint64_t)w[1] << 32;
            }
            if (left < kTaKeys) seen &= (1ull << left) - 1;
            if (!live) seen = 0;
            seen >>= c0;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (!(seen >> c & 1)) s[c] = -INFINITY;
          }
          float mx2[2] = {s[0], s[1]};
#pragma unroll
          for (int c = 2; c + 1 < kCols; c += 2) mx2[c >> 1 & 1] = max3(mx2[c >> 1 & 1], s[c], s[c + 1]);
          const float mx = fmaxf(mx2[0], mx2[1]) * a.scale_log2;
          if (!S::kBetween && group == 1 && j > 1 && (j - 1) % S::kFlush == 0) flush(j - 1, m);
          // this tile's reference, after the one of the tile before it
          if (j > 0) turn_wait(quarter, group);
          if (!idle) {
            const float known = s_m[ln];
            unit = known;
            if (__any_sync(0xffffffffu, known != m || mx > m + kTaLazy)) {
              rescale(known);
              if (__any_sync(0xffffffffu, mx > m + kTaLazy)) {
                const float corr = rescale(fmaxf(m, mx));
                s_m[ln] = m;
                if (j % S::kFlush != 0) {  // the accumulator starts afresh otherwise
                  if (j > 1) done(j - 2);  // room(j - 2) told of j - 4
                  done(j - 1);
#pragma unroll 1
                  for (int c = 0; ok && c < D; c += 16) {
                    float o[16];
                    tm_load(tl + S::kColO + c, o);
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * corr);
                    tm_store(tl + S::kColO + c, w);
                  }
                }
              }
            }
          }
          if (j + 1 < n) turn_pass(quarter, group);
          if (!idle && ok) {
            const float mu = m == -INFINITY ? 0.0f : m;  // nothing seen so far: every weight is 2^-inf
            float2 ls = make_float2(0.0f, 0.0f);
            const float2 sc = make_float2(a.scale_log2, a.scale_log2), mm = make_float2(-mu, -mu);
#pragma unroll
            for (int ch = 0; ch < kCols; ch += 16) {  // 16 keys at a time, for the registers' sake
              uint32_t w[S::kTermsP][8];
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                const float2 x = fma2(make_float2(s[ch + c], s[ch + c + 1]), sc, mm);
                const float2 pp = make_float2(ex2(x.x), ex2(x.y));
                ls = add2(ls, pp);
                uint32_t term[S::kTermsP];
                split(pp.x, pp.y, term);
#pragma unroll
                for (int tt = 0; tt < S::kTermsP; ++tt) w[tt][c / 2] = term[tt];
              }
              if (ch == 0) room(j);
#pragma unroll
              for (int tt = 0; tt < S::kTermsP; ++tt) tm_store(tl + S::weights(j, tt) + (c0 + ch) / 2, w[tt]);
            }
            l += ls.x + ls.y;
            if constexpr (DUP > 1) {  // the keys that other lanes weigh
#pragma unroll
              for (int tt = 0; tt < S::kTermsP; ++tt)
#pragma unroll
                for (int c = 0; c < kTaKeys / 2; c += 8)
                  if (c / (kCols / 2) != part) tm_store(tl + S::weights(j, tt) + c, zero);
            }
          }
          // An idle warp also waits for its group's last products: its arrival below must not count for them.
          if (idle) room(j);
          if (j == stop) break;
          if (!S::kBetween && group == 0 && j > 0 && j % S::kFlush == 0) flush(j, unit);
          commit();
        }
        if (j >= n) break;
        if (group == 1) commit();
        flush(j0, group == 1 ? m : unit);
        if (group == 0) commit();
      }
      // the last tile is the other group's, and starts afresh
      if (!S::kBetween && group == 1 && n > 1 && (n - 1) % S::kFlush == 0) flush(n - 1, m);
      // the row's accumulator, staged in the ring (every copy and MMA has finished by then)
      ok = bar_wait_warp(drain, 0, fail, a.timeout_ns) && ok;
      tm_fence_after();
      asm volatile("bar.sync 9, 256;" ::: "memory");  // both groups' last word on the references
      if (ok) {
        rescale(s_m[ln]);
        const float scale = sums_m == m ? 1.0f : ex2(sums_m - m);
        float* st = reinterpret_cast<float*>(ring) + ln * S::kPitch + group * kDims;
#pragma unroll
        for (int c = 0; c < kDims; c += 16) {
          float o[16];
          tm_load(ocol + c, o);
          with_sums(c, o, scale);
#pragma unroll
          for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(st + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        s_l[group][ln] = l;
      }
    }
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    if (warp == kTaScore && (last || *fail))
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTaTmemCols) : "memory");
    if (*fail) {
      if (i == 0 && atomicCAS(a.err, 0u, kTaErrWait) == 0u) a.err[1] = blockIdx.x;
      return;
    }
    // join the lanes of each row; a split's sum goes to the workspace, a whole one to the output
    const float* st = reinterpret_cast<const float*>(ring);
#pragma unroll 4
    for (int e = i; e < rows * (D / 4); e += kTaThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int d = 0; d < DUP; ++d) M = fmaxf(M, s_m[r + d * kRows]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int d = 0; d < DUP; ++d) {
        const int ln = r + d * kRows;
        const float4 x = *reinterpret_cast<const float4*>(st + ln * S::kPitch + c);
        const float w = DUP == 1 || s_m[ln] == M ? 1.0f : ex2(s_m[ln] - M);
        L = fmaf(s_l[0][ln] + s_l[1][ln], w, L);
        o.x = fmaf(x.x, w, o.x);
        o.y = fmaf(x.y, w, o.y);
        o.z = fmaf(x.z, w, o.z);
        o.w = fmaf(x.w, w, o.w);
      }
      const int rr = mt * kRows + r, b = node_of(rr, a.inv_g);
      if (s_bad) {  // tree values that are not finite, for the nodes that see them
        for (int k = max(t0 - a.pre_tiles, 0) * kTaKeys; k < min(a.B, (t0 + n - a.pre_tiles) * kTaKeys); ++k) {
          if (!(a.mask[(int64_t)b * a.words + (k >> 5)] >> (k & 31) & 1u)) continue;
          const uint2 v = *reinterpret_cast<const uint2*>(a.vtree + (int64_t)g * a.head_stride + (int64_t)k * D + c);
          if (!isfinite(low_f(v.x))) o.x += low_f(v.x);
          if (!isfinite(high_f(v.x))) o.y += high_f(v.x);
          if (!isfinite(low_f(v.y))) o.z += low_f(v.y);
          if (!isfinite(high_f(v.y))) o.w += high_f(v.y);
        }
      }
      if (kShares ? n < a.tiles : a.nsplit > 1) {
        // a share's pieces each move on to another CTA or tile of rows
        const int64_t to = (kShares ? (int64_t)blockIdx.x + id : (int64_t)blockIdx.x) * kRows + r;
        *reinterpret_cast<float4*>(a.part + to * D + c) = o;
        if (c == 0) a.ml[to] = make_float2(M, L);
      } else {
        const float s = L == 0.0f ? 0.0f : 1.0f / L;  // L = 0: the node sees nothing
        const int64_t to = ((int64_t)b * a.Hq + g * a.G + (rr - b * a.G)) * D + c;
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = make_float4(o.x * s, o.y * s, o.z * s, o.w * s);
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) = make_uint2(pack_rn(o.x * s, o.y * s), pack_rn(o.z * s, o.w * s));
      }
    }
    if (last) break;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next piece's copies over the staged rows
    __syncthreads();
    if (i < 128) s_m[i] = -INFINITY;
    if (i == 0) s_bad = 0;
    __syncthreads();
    locate(piece + 1);
  }
}

// Joins the splits of a row: W warps of a CTA share a row (warp w takes splits w, w + W, ...), a
// lane D / 32 of its dimensions. A warp asks for kBatch splits together with their maxima, so up to
// kBatch * W splits take one round trip to L2. As a programmatic dependent launch this kernel adds
// 3 us to a call of 25 nodes over 26K; joining in the kernel above behind a barrier of the splits
// added 6, and its cooperative launch took away the overlap with the kernel before (2.5 us).
template <typename T, int D, int W, int kBatch>
__global__ void __launch_bounds__(128) tree_attn_join_kernel(const TaArgs a, int rows_per_tile) {
  constexpr int E = D / 32;
  __shared__ float s_m[4], s_l[4], s_o[W > 1 ? 4 : 1][D];
  dependent_launch_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % W;
  const int64_t row = min((int64_t)blockIdx.x * (4 / W) + warp / W, (int64_t)a.B * a.Hq - 1);  // b * Hq + h
  const int b = (int)(row / a.Hq), h = (int)(row % a.Hq), g = h / a.G;
  const int rr = b * a.G + h % a.G, mt = rr / rows_per_tile, r = rr % rows_per_tile;
  int64_t first = ((int64_t)g * a.nsplit * a.mtiles + mt) * rows_per_tile + r, step = (int64_t)a.mtiles * rows_per_tile;
  int splits = a.nsplit;
  if (splits == 0) {  // shares of all tiles: from the one with the first of this tile of rows to the one with the last
    const int64_t id = (int64_t)g * a.mtiles + mt;
    const int64_t work = (int64_t)a.groups * a.tiles;
    const int64_t from = share_with(work, id * a.tiles, a.ctas);
    splits = (int)(share_with(work, (id + 1) * a.tiles - 1, a.ctas) - from) + 1;
    if (splits == 1) return;  // written already
    first = (from + id) * rows_per_tile + r;
    step = rows_per_tile;
  }
  using V = typename std::conditional<E == 4, float4, float2>::type;
  float M = -INFINITY, L = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int s0 = w; s0 < splits; s0 += kBatch * W) {
    V x[kBatch];
    float2 ml[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int s = s0 + k * W;
      const int64_t at = first + min(s, splits - 1) * step;
      x[k] = __ldcg(reinterpret_cast<const V*>(a.part + at * D) + lane);
      ml[k] = __ldcg(a.ml + at);
      if (s >= splits) ml[k] = make_float2(-INFINITY, 0.0f);
    }
    float mn = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
    const float corr = M == mn ? 1.0f : ex2(M - mn);  // M = -inf: nothing seen so far, all sums 0
    L *= corr;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= corr;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (s0 + k * W >= splits) break;
      const float wt = ml[k].x == mn ? 1.0f : ex2(ml[k].x - mn);
      L = fmaf(ml[k].y, wt, L);
      const float* xe = reinterpret_cast<const float*>(&x[k]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(xe[e], wt, acc[e]);
    }
    M = mn;
  }
  if constexpr (W > 1) {
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = L;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (w != 0) return;
    float mn = -INFINITY;
#pragma unroll
    for (int k = 0; k < W; ++k) mn = fmaxf(mn, s_m[warp + k]);
    L = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float wt = s_m[warp + k] == mn ? 1.0f : ex2(s_m[warp + k] - mn);
      L = fmaf(s_l[warp + k], wt, L);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(s_o[warp + k][lane * E + e], wt, acc[e]);
    }
  }
  const float s = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= s;
  const int64_t at = row * D + lane * E;
  if constexpr (sizeof(T) == 4) {
    float* y = static_cast<float*>(a.out) + at;
    if constexpr (E == 4) *reinterpret_cast<float4*>(y) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    else *reinterpret_cast<float2*>(y) = make_float2(acc[0], acc[1]);
  } else {
    uint32_t* y = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at);
#pragma unroll
    for (int e = 0; e < E; e += 2) y[e / 2] = pack_rn(acc[e], acc[e + 1]);
  }
}

// ---- host -----------------------------------------------------------------------------------
size_t tree_attn_ws_bytes(int B, int Hq, int Hkv, int D) {
  return kWsHeaderBytes + (size_t)ta_split_rows(B, Hq, Hkv) * (D * 4 + sizeof(float2));
}

std::mutex g_ta_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_ta_encode = nullptr;

nt_status ta_setup() {
  std::lock_guard<std::mutex> lock(g_ta_mu);
  if (!g_ta_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    NT_CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q));
    if (q != cudaDriverEntryPointSuccess || !fn) return set_error(NT_ERR_CUDA, "cuTensorMapEncodeTiled not available");
    g_ta_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  return NT_OK;
}

// Rows [0, rows) of every head from `base` on, boxes of 64 dimensions x 64 rows; further rows read as 0.
nt_status ta_map(CUtensorMap* map, const uint16_t* base, int D, int rows, int Hkv, int ts) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ts * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)kTaKeys, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_ta_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box,
                                 estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(NT_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")");
  return NT_OK;
}

template <typename T, int D, int DUP, bool kShares>
nt_status launch_tree_attn(const TaMaps& maps, const TaArgs& a, const TaPlan& p, cudaStream_t st) {
  static std::atomic<int> attr_set[64];  // per device: the ring's dynamic shared memory allowed
  int dev = 0;
  NT_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return set_error(NT_ERR_CUDA, "device index out of range");
  constexpr int smem = TaShape<T, D>::kSmem;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    NT_CUDA_TRY(cudaFuncSetAttribute(tree_attn_kernel<T, D, DUP, kShares>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    attr_set[dev].store(1, std::memory_order_release);
  }
  NT_CUDA_TRY(launch_kernel(tree_attn_kernel<T, D, DUP, kShares>, dim3((unsigned)p.units), dim3(kTaThreads), smem, st, true, maps, a));
  return check_launch("tree_attn_kernel");
}
template <typename T, int D>
nt_status launch_tree_attn_all(const TaMaps& maps, const TaArgs& a, const TaPlan& p, int dtype, cudaStream_t st) {
  nt_status s;
  if (p.few) s = launch_tree_few(maps, a, dtype, D, st);
  else if (p.nsplit == 0) s = p.dup == 2 ? launch_tree_attn<T, D, 2, true>(maps, a, p, st) : launch_tree_attn<T, D, 1, true>(maps, a, p, st);
  else s = p.dup == 2 ? launch_tree_attn<T, D, 2, false>(maps, a, p, st) : launch_tree_attn<T, D, 1, false>(maps, a, p, st);
  NT_TRY(s);
  if (ta_joins(p)) {
    const int64_t rows = (int64_t)a.B * a.Hq;
    // Warps per row and splits at a time: one round trip for up to 32 splits, and no load twice for few.
    const int w = p.parts > 4 ? 4 : 1;
    auto join = p.parts > 16 ? tree_attn_join_kernel<T, D, 4, 8> : p.parts > 8 ? tree_attn_join_kernel<T, D, 4, 4>
                : p.parts > 4 ? tree_attn_join_kernel<T, D, 4, 2> : p.parts > 2 ? tree_attn_join_kernel<T, D, 1, 4>
                : tree_attn_join_kernel<T, D, 1, 2>;
    NT_CUDA_TRY(launch_kernel(join, dim3((unsigned)((rows * w + 3) / 4)), dim3(128), 0, st, true, a, p.rows));
    NT_TRY(check_launch("tree_attn_join_kernel"));
  }
  return NT_OK;
}
}  // namespace
}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_tree_attention_workspace_size(int B, int Hq, int Hkv, int D, int prefix, size_t* bytes) {
  clear_error();
  if (!bytes || B < 1 || B > kTreeMaxNodes || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || prefix < 0)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= B <= 256, Hq a multiple of Hkv >= 1, prefix >= 0 and a result pointer");
  if (D != 64 && D != 128) return set_error(NT_ERR_UNSUPPORTED, "head dimension must be 64 or 128");
  if ((int64_t)B * Hq > kTreeMaxRows) return set_error(NT_ERR_INVALID_ARG, "B * Hq leaves the supported range (1048576)");
  *bytes = tree_attn_ws_bytes(B, Hq, Hkv, D);
  return NT_OK;
}

nt_status nt_tree_attention(const void* q, int dtype, const uint16_t* k_cache, const uint16_t* v_cache, int B, int Hq,
                            int Hkv, int D, int prefix, int tree_row0, int t_stride, const uint32_t* mask,
                            int mask_words, void* out, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (!q || !k_cache || !v_cache || !mask || !out) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (dtype != NT_F32 && dtype != NT_BF16) return set_error(NT_ERR_INVALID_ARG, "dtype must be NT_F32 or NT_BF16");
  if (D != 64 && D != 128) return set_error(NT_ERR_UNSUPPORTED, "head dimension must be 64 or 128");
  if (B < 1 || B > kTreeMaxNodes || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || mask_words < (B + 31) / 32)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= B <= 256, Hq a multiple of Hkv >= 1 and mask_words >= ceil(B / 32)");
  if ((int64_t)B * Hq > kTreeMaxRows) return set_error(NT_ERR_INVALID_ARG, "B * Hq leaves the supported range (1048576)");
  if (prefix < 0 || tree_row0 < prefix || (int64_t)tree_row0 + B > t_stride)
    return set_error(NT_ERR_INVALID_ARG, "need 0 <= prefix <= tree_row0 and tree_row0 + B <= t_stride");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(mask, 4))
    return set_error(NT_ERR_ALIGNMENT, "q, out and the caches must be 16-byte, the mask 4-byte aligned");
  if (!ws || !aligned(ws, 16) || ws_bytes < tree_attn_ws_bytes(B, Hq, Hkv, D))
    return set_error(NT_ERR_WORKSPACE, "workspace NULL, misaligned or smaller than nt_tree_attention_workspace_size");
  NT_TRY(check_device());
  NT_TRY(ta_setup());
  int clusters = 0;
  if (B <= kTaFewNodes) NT_TRY(set_up_tree_few(B * (Hq / Hkv), dtype, D, &clusters));  // up to kTaFewRows rows are no more nodes
  const TaPlan p = ta_plan(B, Hq, Hkv, prefix, dtype == NT_F32, D, clusters);
  TaArgs a{};
  a.q = q;
  a.out = out;
  a.mask = mask;
  a.vtree = v_cache + (int64_t)tree_row0 * D;
  a.head_stride = (int64_t)t_stride * D;
  a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + kWsHeaderBytes);
  a.part = reinterpret_cast<float*>(a.ml + ta_split_rows(B, Hq, Hkv));
  a.err = static_cast<unsigned int*>(ws);
  a.timeout_ns = test_fault_timeout_ns(kTaTimeoutNs);
  a.fault = test_fault() == kFaultTree;
  a.B = B;
  a.Hq = Hq;
  a.G = Hq / Hkv;
  a.R = B * a.G;
  a.words = mask_words;
  a.prefix = prefix;
  a.pre_tiles = p.pre_tiles;
  a.tiles = p.tiles;
  a.nsplit = p.nsplit;
  a.cluster = p.cluster;
  a.mtiles = p.mtiles;
  a.groups = Hkv * p.mtiles;
  a.ctas = (int)p.units;
  a.inv_g = 1.0f / (float)a.G;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  TaMaps maps;
  // without a sequence its maps are not used; they still have to be valid
  NT_TRY(ta_map(&maps.kp, k_cache, D, std::max(prefix, 1), Hkv, t_stride));
  NT_TRY(ta_map(&maps.vp, v_cache, D, std::max(prefix, 1), Hkv, t_stride));
  NT_TRY(ta_map(&maps.kt, k_cache + (int64_t)tree_row0 * D, D, B, Hkv, t_stride));
  NT_TRY(ta_map(&maps.vt, a.vtree, D, B, Hkv, t_stride));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == NT_F32)
    return D == 64 ? launch_tree_attn_all<float, 64>(maps, a, p, dtype, st) : launch_tree_attn_all<float, 128>(maps, a, p, dtype, st);
  return D == 64 ? launch_tree_attn_all<uint16_t, 64>(maps, a, p, dtype, st) : launch_tree_attn_all<uint16_t, 128>(maps, a, p, dtype, st);
}

}  // extern "C"
