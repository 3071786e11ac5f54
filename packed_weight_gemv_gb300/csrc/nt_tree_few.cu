// nt_tree_few.cu -- attention of a drafted token tree with few query rows: single tokens and small
// trees, up to 32 rows B * Hq / Hkv per key-value head (the formula and the rules on what a node sees
// are the same as for more rows). Over shorter sequences also more rows, 32 to a CTA.
//
// With the query rows on the M side of tcgen05.mma, 128 of them to a tile, few rows cost the tensor
// pipe as much as 128 do: 0.88 us per 64 keys for fp32 queries, above the 0.7 us that a CTA's share of
// the memory rate takes. So the products are turned: keys are the M side of the scores, 128 to a
// tile, dimensions the M side of the weighted values, and the rows the N side -- all terms of all
// rows together, so the three terms of an fp32 query or weight are columns of one product, summed in
// registers, instead of three products.
//
//   S[key][term, row] = K q      O[dim][term, row] = V^T p      (A and B from shared memory)
//
// A thread is a key of the scores and a dimension of the sums. Its weights go to shared memory, 8
// rows of a term to a 16-byte store, and each tile's sums come back to registers, where they are
// rounded to nearest: the tensor core, which cuts its sums off, adds 128 keys at most.
//
// CTA (384 threads): a key-value head, a range of 64-key tiles taken in pairs.
//   warps 0, 3     -- TMA copies of keys and of values, a ring each;
//   warps 1, 2     -- the scores' MMAs, the sums';
//   warps 4-7, 8-11 - two groups, each with every other pair of tiles, a maximum, sum and accumulator of
//                     its own, so they meet only at the end. The maxima are raised when a score of any row
//                     exceeds its maximum by 2^8.
//
// Bound by the memory for long sequences and by latency for short ones. 32 / 8 heads of 128, fp32, join
// included, in a replayed graph: one node over 32,767 keys 26.1 us = 5.1 TB/s, 76 % of the measured copy rate (bf16 26.3;
// with rows on the M side 35.5); one node over 4,095 keys 7.9, over 800 5.7, over 50 (unsplit) 4.2. 8 nodes (32 rows)
// over 32,700 take 29.9: a group's steps for 32 rows, one behind the other, bound them (13 or 14 pairs of tiles to a
// CTA, 1.9 us each; 25 % of the issue slots, 19 % of the tensor pipe).
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "nt_tree_attn.cuh"

namespace nt {
namespace {

constexpr int kTfKeys = 2 * kTaKeys;    // keys of a pair of tiles
constexpr float kTfLowest = -3.0e38f;   // reference of a row that has seen nothing (its weights are 0)

constexpr int up16(int n) { return (n + 15) / 16 * 16; }

template <typename T, int D, int RP>
struct TfShape {
  static constexpr int kTermsQ = sizeof(T) == 4 ? 3 : 1;
  static constexpr int kTermsP = sizeof(T) == 4 ? 3 : 2;
  static constexpr int kNQ = up16(kTermsQ * RP), kNP = up16(kTermsP * RP);  // columns: term * RP + row
  static constexpr int kSlot = kTfKeys * D * 2;                   // a pair's keys or values
  static constexpr int kBlock = kTfKeys * 128;                    // bytes of 64 columns of weights, or 64 dimensions
  static constexpr int kP = (kNP + 63) / 64 * kBlock, kQ = kNQ * D * 2;
  static constexpr int kSlots = (222 * 1024 - 2 * kP - kQ) / kSlot;
  static constexpr int kKeySlots = (kSlots + 1) / 2, kValSlots = kSlots / 2;
  static constexpr int kAtV = kKeySlots * kSlot, kAtP = kSlots * kSlot, kAtQ = kAtP + 2 * kP;
  static constexpr int kSmem = kAtQ + kQ + 1024;                  // and alignment
  static constexpr int kColS = 0, kColO = 2 * kNQ;                // tensor-memory columns, one of each per group
  static_assert(kValSlots >= 2 && 2 * (kNQ + kNP) <= kTaTmemCols, "ring and tensor memory");
  static_assert(3 * RP * D * 4 <= kSlots * kSlot, "the sums are staged in the ring");
};

__host__ __device__ constexpr uint32_t idesc_few(int n, bool rows) {  // both operands K-major, or both with the reduction along rows
  return (1u << 4) | (1u << 7) | (1u << 10) | (rows ? 3u << 15 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// The terms' columns of 8 rows, summed from the smallest on; the second term's sign is turned. One wait for
// all the loads, in one statement with them: registers of a load on its way must not be moved or spilled.
template <int TERMS, int RP>
__device__ __forceinline__ void tm_terms8(uint32_t addr, float (&x)[8]) {
  if constexpr (TERMS == 1) {
    asm volatile(
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        " tcgen05.wait::ld.sync.aligned;"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
        : "r"(addr)
        : "memory");
  } else {
    float mid[8];
    if constexpr (TERMS == 3) {
      float low[8];
      asm volatile(
          " tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n"
          " tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n"
          " tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];\n"
          " tcgen05.wait::ld.sync.aligned;"
          : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
            "=f"(mid[0]), "=f"(mid[1]), "=f"(mid[2]), "=f"(mid[3]), "=f"(mid[4]), "=f"(mid[5]), "=f"(mid[6]), "=f"(mid[7]),
            "=f"(low[0]), "=f"(low[1]), "=f"(low[2]), "=f"(low[3]), "=f"(low[4]), "=f"(low[5]), "=f"(low[6]), "=f"(low[7])
          : "r"(addr), "r"(addr + RP), "r"(addr + 2 * RP)
          : "memory");
#pragma unroll
      for (int e = 0; e < 8; ++e) mid[e] -= low[e];
    } else {
      asm volatile(
          " tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n"
          " tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n"
          " tcgen05.wait::ld.sync.aligned;"
          : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
            "=f"(mid[0]), "=f"(mid[1]), "=f"(mid[2]), "=f"(mid[3]), "=f"(mid[4]), "=f"(mid[5]), "=f"(mid[6]), "=f"(mid[7])
          : "r"(addr), "r"(addr + RP)
          : "memory");
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] -= mid[e];
  }
}
// Sums of N values (8, 16 or 32 of them) over a warp: lane r gets value r's, and lanes N on repeat
// them. Half of the values go to the other half of the lanes at every step.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int e = 0; e < o; ++e) {
      const float send = up ? v[e] : v[e + o], keep = up ? v[e + o] : v[e];
      v[e] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}
__device__ __forceinline__ float warp_max(float x) {  // NaN left out
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Whether any thread of a group says so.
__device__ __forceinline__ bool group_any(int group, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(1 + group)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of the cluster's CTA `rank`, at the address that this CTA has it.
__device__ __forceinline__ float2 peer_ld2(uint32_t addr, int rank) {
  float2 v;
  asm volatile("{\n .reg .b32 p;\n mapa.shared::cluster.u32 p, %2, %3;\n ld.shared::cluster.v2.f32 {%0,%1}, [p];\n}\n"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_ld4(uint32_t addr, int rank) {
  float4 v;
  asm volatile("{\n .reg .b32 p;\n mapa.shared::cluster.u32 p, %4, %5;\n ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [p];\n}\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}

template <typename T, int D, int RP>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_few_kernel(const __grid_constant__ TaMaps maps, const TaArgs a) {
  using S = TfShape<T, D, RP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[2 * S::kSlots + 10];
  __shared__ uint32_t tmem_slot, s_mask[RP];
  __shared__ int s_fail, s_bad;
  __shared__ __align__(16) float s_nm[2][RP];  // minus a group's reference maxima (log2 units)
  __shared__ __align__(16) float s_corr[2][RP];  // what a raise of them scales sums by
  __shared__ float2 s_ml[RP];  // a row's (m, sum) for the other CTAs of a cluster
  __shared__ float s_w[2][4][RP];  // a warp's largest scores; at the end its sums
  const uint32_t keyfull = smem_u32(bars), keyempty = keyfull + 8 * S::kKeySlots;
  const uint32_t valfull = keyempty + 8 * S::kKeySlots, valempty = valfull + 8 * S::kValSlots;
  const uint32_t sfull0 = valempty + 8 * S::kValSlots, sfree0 = sfull0 + 16, pfull0 = sfree0 + 16, pvdone0 = pfull0 + 16;
  const uint32_t qfull = pvdone0 + 16, drain = qfull + 8;
  volatile int* fail = &s_fail;
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31;

  // A cluster's CTAs are neighbours; otherwise the tiles of rows that read the same keys are.
  const int unit = blockIdx.x, g = unit / (a.nsplit * a.mtiles), in_head = unit - g * (a.nsplit * a.mtiles);
  const int mt = a.cluster ? in_head / a.nsplit : in_head % a.mtiles, sp = a.cluster ? in_head % a.nsplit : in_head / a.mtiles;
  const int r0 = mt * RP, rows = min(RP, a.R - r0);
  const int t0 = (int)((int64_t)a.tiles * sp / a.nsplit), n = (int)((int64_t)a.tiles * (sp + 1) / a.nsplit) - t0;
  const int pairs = (n + 1) / 2;

  if (i == 0) {
    for (int s = 0; s < 2 * S::kSlots; ++s) bar_init(smem_u32(bars) + 8 * s, 1);
    for (int b = 0; b < 2; ++b) {
      bar_init(sfull0 + 8 * b, 1);
      bar_init(sfree0 + 8 * b, 4);  // the warps of the group
      bar_init(pfull0 + 8 * b, 4);
      bar_init(pvdone0 + 8 * b, 1);
    }
    bar_init(qfull, kTaSoftmax / 32);
    bar_init(drain, 2);
    s_fail = 0;
    s_bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (i < 2 * RP) s_nm[i / RP][i % RP] = -kTfLowest;
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

  auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, fail, a.timeout_ns); };

  if (warp == kTaKeyLoad || warp == kTaValueLoad) {
    if (elect_one()) {
      const bool val = warp == kTaValueLoad;
      const int slots = val ? S::kValSlots : S::kKeySlots;
      const uint32_t full = val ? valfull : keyfull, empty = val ? valempty : keyempty;
      const uint32_t at = smem_u32(ring) + (val ? S::kAtV : 0);
      int j = 0;
      for (; j < pairs && !a.fault; ++j) {
        const int k = j % slots;
        if (j >= slots && !wait(empty + 8 * k, (j / slots - 1) & 1)) break;
        bar_expect_tx(full + 8 * k, S::kSlot);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = t0 + 2 * j + u;
          const bool tree = t >= a.pre_tiles;
          const CUtensorMap* map = val ? (tree ? &maps.vt : &maps.vp) : (tree ? &maps.kt : &maps.kp);
          // past the CTA's last tile: rows beyond the tree's, which read as zeros
          const int y = 2 * j + u < n ? (tree ? t - a.pre_tiles : t) * kTaKeys : tree ? 4 * kTreeMaxNodes : a.prefix;
#pragma unroll
          for (int x = 0; x < D; x += 64) tma_3d(at + k * S::kSlot + x / 64 * S::kBlock + u * (kTaKeys * 128), map, x, y, g, full + 8 * k);
        }
      }
      // every copy must land before the CTA may exit
      const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
      for (int d = max(0, j - slots); d < j; ++d)
        while (!bar_try(full + 8 * (d % slots), (d / slots) & 1))
          if (globaltimer_ns() > deadline) break;
    }
    __syncwarp();
  } else if (warp == kTaScore) {
    if (elect_one()) {
      bool ok = wait(qfull, 0);
      tm_fence_after();
      for (int j = 0; ok && j < pairs; ++j) {
        const int k = j % S::kKeySlots;
        ok = wait(keyfull + 8 * k, (j / S::kKeySlots) & 1);
        if (ok && j >= 2) ok = wait(sfree0 + 8 * (j & 1), ((j >> 1) - 1) & 1);  // the group's last scores have been taken
        if (!ok) break;
        tm_fence_after();
        const uint64_t ad = sdesc(smem_u32(ring) + k * S::kSlot, 16), bd = sdesc(smem_u32(ring) + S::kAtQ, 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_smem_a(tmem + S::kColS + (j & 1) * S::kNQ, ad + ((kk >> 2) * S::kBlock + (kk & 3) * 32) / 16,
                     bd + ((kk >> 2) * (S::kNQ * 128) + (kk & 3) * 32) / 16, idesc_few(S::kNQ, false), kk > 0);
        mma_commit(sfull0 + 8 * (j & 1));
        mma_commit(keyempty + 8 * k);
      }
      mma_commit(drain);
    }
    __syncwarp();
  } else if (warp == kTaValue) {
    if (elect_one()) {
      for (int j = 0; j < pairs; ++j) {
        const int k = j % S::kValSlots;
        if (!wait(valfull + 8 * k, (j / S::kValSlots) & 1) || !wait(pfull0 + 8 * (j & 1), (j >> 1) & 1)) break;
        tm_fence_after();
        // with 64 dimensions the second half of the M side reads them again
        const uint64_t ad = sdesc(smem_u32(ring) + S::kAtV + k * S::kSlot, D == 128 ? S::kBlock : 0);
        const uint64_t bd = sdesc(smem_u32(ring) + S::kAtP + (j & 1) * S::kP, S::kBlock);
#pragma unroll
        for (int kk = 0; kk < kTfKeys / 16; ++kk)  // 16 keys: 2,048 bytes of each block
          mma_smem_a(tmem + S::kColO + (j & 1) * S::kNP, ad + kk * 2048 / 16, bd + kk * 2048 / 16, idesc_few(S::kNP, true), kk > 0);
        mma_commit(pvdone0 + 8 * (j & 1));
        mma_commit(valempty + 8 * k);
      }
      mma_commit(drain);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, group = (warp - kTaFirstSoftmax) >> 2, ln = quarter * 32 + lane;  // key, dimension
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    {  // the query terms: rows of 64 dimensions, 16-byte pieces in the order of the 128-byte swizzle
      const int idx = i - 32 * kTaFirstSoftmax;
      if (idx < RP) s_mask[idx] = idx < rows ? a.mask[(int64_t)node_of(r0 + idx, a.inv_g) * a.words] : 0u;
      uint8_t* qs = ring + S::kAtQ;
      constexpr int kAll = RP * (D / 8), kPer = (kAll + kTaSoftmax - 1) / kTaSoftmax;  // pieces of 8 dimensions
      uint4 v[kPer][sizeof(T) / 2];
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const int e = idx + p * kTaSoftmax, r = e / (D / 8), b = node_of(r0 + r, a.inv_g);
        const T* q = static_cast<const T*>(a.q) + ((int64_t)b * a.Hq + g * a.G + (r0 + r - b * a.G)) * D + e % (D / 8) * 8;
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h)
          v[p][h] = r < rows ? reinterpret_cast<const uint4*>(q)[h] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const int e = idx + p * kTaSoftmax, r = e / (D / 8), c = e % (D / 8);
        uint32_t w[S::kTermsQ][4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[3], y[3];
            split(__uint_as_float(v[p][h].x), __uint_as_float(v[p][h].y), x);
            split(__uint_as_float(v[p][h].z), __uint_as_float(v[p][h].w), y);
#pragma unroll
            for (int t = 0; t < 3; ++t) {
              w[t][2 * h] = x[t];
              w[t][2 * h + 1] = y[t];
            }
          }
        } else {
          w[0][0] = v[p][0].x; w[0][1] = v[p][0].y; w[0][2] = v[p][0].z; w[0][3] = v[p][0].w;
        }
        if (e < kAll) {
#pragma unroll
          for (int t = 0; t < S::kTermsQ; ++t) {
            const int nr = t * RP + r;
            *reinterpret_cast<uint4*>(qs + (c >> 3) * (S::kNQ * 128) + nr * 128 + (((c & 7) ^ (nr & 7)) * 16)) =
                make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      bar_arrive_warp(qfull, lane);
      asm volatile("bar.sync 3, 256;" ::: "memory");  // s_mask
    }
    float acc[RP];  // dimension ln of the rows' weighted sums
    float2 l[RP / 2];
#pragma unroll
    for (int r = 0; r < RP; ++r) acc[r] = 0.0f;
#pragma unroll
    for (int r = 0; r < RP / 2; ++r) l[r] = make_float2(0.0f, 0.0f);
    uint8_t* prow = ring + S::kAtP + group * S::kP + ln * 128;  // this key's weights
    const float2 sc = make_float2(a.scale_log2, a.scale_log2);
    // After a wait that ran out a warp keeps walking the tiles, as its group's barriers need it.
    bool ok = true;
    auto take = [&](int j) {  // pair j's sums to registers
      ok = ok && bar_wait_warp(pvdone0 + 8 * group, (j >> 1) & 1, fail, a.timeout_ns);
      tm_fence_after();
      if (ok) {
#pragma unroll
        for (int c = 0; c < RP; c += 8) {
          float o[8];
          tm_terms8<S::kTermsP, RP>(tl + S::kColO + group * S::kNP + c, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[c + e] += o[e];
        }
      }
    };
    for (int j = group; j < pairs; j += 2) {
      ok = ok && bar_wait_warp(sfull0 + 8 * group, (j >> 1) & 1, fail, a.timeout_ns);
      tm_fence_after();
      float s[RP];
#pragma unroll
      for (int c = 0; c < RP; c += 8) {
        float x[8] = {};
        if (ok) tm_terms8<S::kTermsQ, RP>(tl + S::kColS + group * S::kNQ + c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[c + e] = x[e];
      }
      tm_fence_before();
      if (ok) bar_arrive_warp(sfree0 + 8 * group, lane);
      {  // what the rows see of this key
        const int t = t0 + 2 * j + (ln >> 6), key = ln & 63;
        uint32_t seen = 0u;
        if (t - t0 < n) {
          if (t < a.pre_tiles) {
            if (key < a.prefix - t * kTaKeys) seen = ~0u;
          } else if (key < a.B) {  // all of the tree is one tile
#pragma unroll
            for (int r = 0; r < RP; ++r) seen |= (s_mask[r] >> key & 1u) << r;
          }
        }
        if (seen != ~0u) {
#pragma unroll
          for (int r = 0; r < RP; ++r)
            if (!(seen >> r & 1u)) s[r] = -INFINITY;
        }
      }
      const int tree = a.pre_tiles - t0 - 2 * j;  // which half is the tree's
      if (tree < 2 && tree >= 0 && a.pre_tiles < t0 + n) {  // take its values that are not finite out of the product
        const int k = j % S::kValSlots;
        // Pair j - 2's products tell that the values before pair j's have left the slot: a parity alone could answer for them.
        if (j >= 2) ok = ok && bar_wait_warp(pvdone0 + 8 * group, ((j >> 1) - 1) & 1, fail, a.timeout_ns);
        ok = ok && bar_wait_warp(valfull + 8 * k, (j / S::kValSlots) & 1, fail, a.timeout_ns);
        bool bad = false;
        for (int e = ln; ok && e < a.B * (D / 8); e += 128) {
          const int row = e / (D / 8), c = e % (D / 8);
          uint4* p = reinterpret_cast<uint4*>(ring + S::kAtV + k * S::kSlot + (c >> 3) * S::kBlock + (tree * kTaKeys + row) * 128 + (c & 7) * 16);
          const uint4 v = *p;
          if (word_bad(v.x) || word_bad(v.y) || word_bad(v.z) || word_bad(v.w)) {
            uint16_t* h = reinterpret_cast<uint16_t*>(p);
            for (int x = 0; x < 8; ++x)
              if ((h[x] & 0x7f80u) == 0x7f80u) h[x] = 0;
            bad = true;
          }
        }
        if (bad) s_bad = 1;
      }
      if (j >= 2) take(j - 2);
      float mx = -INFINITY;
#pragma unroll
      for (int r = 0; r < RP; r += 2) {
        const float2 x = fma2(make_float2(s[r], s[r + 1]), sc, *reinterpret_cast<const float2*>(&s_nm[group][r]));
        mx = max3(mx, x.x, x.y);
      }
      if (group_any(group, mx > kTaLazy)) {
        float mine = -INFINITY;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float w = warp_max(s[r]);
          if (lane == r) mine = w;
        }
        if (lane < RP) s_w[group][quarter][lane] = mine;
        group_sync(group);
        if (ln < RP) {
          const float top = fmaxf(fmaxf(s_w[group][0][ln], s_w[group][1][ln]), fmaxf(s_w[group][2][ln], s_w[group][3][ln]));
          const float old = -s_nm[group][ln], to = fmaxf(old, top * a.scale_log2);
          s_corr[group][ln] = old == to ? 1.0f : ex2(old - to);
          s_nm[group][ln] = -to;
        }
        group_sync(group);
#pragma unroll
        for (int r = 0; r < RP; r += 2) {
          const float2 corr = *reinterpret_cast<const float2*>(&s_corr[group][r]);
          acc[r] *= corr.x;
          acc[r + 1] *= corr.y;
          l[r / 2].x *= corr.x;
          l[r / 2].y *= corr.y;
        }
      }
#pragma unroll
      for (int c = 0; c < RP; c += 8) {
        uint32_t w[S::kTermsP][4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int r = c + e;
          const float2 x = fma2(make_float2(s[r], s[r + 1]), sc, *reinterpret_cast<const float2*>(&s_nm[group][r]));
          const float2 pp = make_float2(ex2(x.x), ex2(x.y));
          l[r / 2] = add2(l[r / 2], pp);
          uint32_t term[S::kTermsP];
          split(pp.x, pp.y, term);
#pragma unroll
          for (int t = 0; t < S::kTermsP; ++t) w[t][e / 2] = term[t];
        }
#pragma unroll
        for (int t = 0; t < S::kTermsP; ++t) {
          const int q = (t * RP + c) / 8;  // 8 columns: a 16-byte piece
          *reinterpret_cast<uint4*>(prow + (q >> 3) * S::kBlock + (((q & 7) ^ (ln & 7)) * 16)) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tm_fence_before();
      if (ok) bar_arrive_warp(pfull0 + 8 * group, lane);
    }
    if (pairs > group) take(group + (pairs - 1 - group) / 2 * 2);
    ok = bar_wait_warp(drain, 0, fail, a.timeout_ns) && ok;
    tm_fence_after();
    asm volatile("bar.sync 3, 256;" ::: "memory");
    // the sums, staged in the ring (every copy and MMA has finished by then)
    float* st = reinterpret_cast<float*>(ring) + group * RP * D;
    if (ok && ln < D) {
#pragma unroll
      for (int r = 0; r < RP; ++r) st[r * D + ln] = acc[r];
    }
    float sums[RP];
#pragma unroll
    for (int r = 0; r < RP; r += 2) {
      sums[r] = l[r / 2].x;
      sums[r + 1] = l[r / 2].y;
    }
    const float sum = warp_sums(sums, lane);
    if (lane < RP) s_w[group][quarter][lane] = sum;
  }
  tm_fence_before();
  __syncthreads();
  if (warp == kTaScore)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTaTmemCols) : "memory");
  if (*fail) {
    if (i == 0 && atomicCAS(a.err, 0u, kTaErrWait) == 0u) a.err[1] = blockIdx.x;
    if (!a.cluster) return;  // a cluster's other CTAs wait for this one below
  }
  auto emit = [&](int r, int c, float4 o, float L) {
    const int b = node_of(r0 + r, a.inv_g);
    const float s = L == 0.0f ? 0.0f : 1.0f / L;  // L = 0: the node sees nothing
    const int64_t at = ((int64_t)b * a.Hq + g * a.G + (r0 + r - b * a.G)) * D + c;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(o.x * s, o.y * s, o.z * s, o.w * s);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_rn(o.x * s, o.y * s), pack_rn(o.z * s, o.w * s));
  };
  // join the groups; a split's sum goes to the workspace or stays for its cluster, a whole one to the output
  const float* st = reinterpret_cast<const float*>(ring);
  float* sums = reinterpret_cast<float*>(ring) + 2 * RP * D;  // [RP][D], the groups' joined
  for (int e = i; e < rows * (D / 4); e += kTaThreads) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    const float M = -fminf(s_nm[0][r], s_nm[1][r]);
    float L = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const float m = -s_nm[d][r], w = m == M ? 1.0f : ex2(m - M);
      const float4 x = *reinterpret_cast<const float4*>(st + (d * RP + r) * D + c);
      L = fmaf((s_w[d][0][r] + s_w[d][1][r]) + (s_w[d][2][r] + s_w[d][3][r]), w, L);
      o.x = fmaf(x.x, w, o.x);
      o.y = fmaf(x.y, w, o.y);
      o.z = fmaf(x.z, w, o.z);
      o.w = fmaf(x.w, w, o.w);
    }
    if (s_bad) {  // tree values that are not finite, for the nodes that see them
      for (int k = 0; k < a.B; ++k) {
        if (!(s_mask[r] >> k & 1u)) continue;
        const uint2 v = *reinterpret_cast<const uint2*>(a.vtree + (int64_t)g * a.head_stride + (int64_t)k * D + c);
        if (!isfinite(low_f(v.x))) o.x += low_f(v.x);
        if (!isfinite(high_f(v.x))) o.y += high_f(v.x);
        if (!isfinite(low_f(v.y))) o.z += low_f(v.y);
        if (!isfinite(high_f(v.y))) o.w += high_f(v.y);
      }
    }
    if (a.cluster) {
      *reinterpret_cast<float4*>(sums + r * D + c) = o;
      if (c == 0) s_ml[r] = make_float2(M, L);
    } else if (a.nsplit > 1) {
      const int64_t at = (int64_t)unit * RP + r;
      *reinterpret_cast<float4*>(a.part + at * D + c) = o;
      if (c == 0) a.ml[at] = make_float2(M, L);
    } else {
      emit(r, c, o, L);
    }
  }
  if (!a.cluster) return;
  // Each CTA of the cluster joins its part of the rows' values over all of them.
  cluster_sync();
  const int items = rows * (D / 4), per = (items + a.nsplit - 1) / a.nsplit;
  for (int e = sp * per + i; e < min(items, (sp + 1) * per); e += kTaThreads) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    float2 ml[kTfCluster];
    float4 x[kTfCluster];
    float M = kTfLowest, L = 0.0f;
#pragma unroll
    for (int k = 0; k < kTfCluster; ++k) {
      ml[k] = make_float2(kTfLowest, 0.0f);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < a.nsplit) {
        ml[k] = peer_ld2(smem_u32(s_ml + r), k);
        x[k] = peer_ld4(smem_u32(sums + r * D + c), k);
      }
    }
#pragma unroll
    for (int k = 0; k < kTfCluster; ++k) M = fmaxf(M, ml[k].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kTfCluster; ++k) {
      const float w = ml[k].x == M ? 1.0f : ex2(ml[k].x - M);
      L = fmaf(ml[k].y, w, L);
      o.x = fmaf(x[k].x, w, o.x);
      o.y = fmaf(x[k].y, w, o.y);
      o.z = fmaf(x[k].z, w, o.z);
      o.w = fmaf(x[k].w, w, o.w);
    }
    emit(r, c, o, L);
  }
  cluster_sync();  // no CTA's shared memory goes while another may read it
}

// ---- host -----------------------------------------------------------------------------------
cudaLaunchConfig_t few_config(cudaLaunchAttribute (&attr)[2], unsigned units, int smem, int cluster, cudaStream_t st) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units);
  cfg.blockDim = dim3(kTaThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cfg;
}

// The kernel's dynamic shared memory allowed on this device; how many of its clusters run at a time.
template <typename T, int D, int RP>
nt_status set_up_few(int* clusters) {
  static std::atomic<int> set[64];     // per device
  static std::atomic<int> active[64];
  int dev = 0;
  NT_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return set_error(NT_ERR_CUDA, "device index out of range");
  if (!set[dev].load(std::memory_order_acquire)) {
    constexpr int smem = TfShape<T, D, RP>::kSmem;
    NT_CUDA_TRY(cudaFuncSetAttribute(tree_few_kernel<T, D, RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = few_config(attr, kTfCluster, smem, kTfCluster, nullptr);
    int n = 0;
    NT_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, tree_few_kernel<T, D, RP>, &cfg));
    active[dev].store(n, std::memory_order_relaxed);
    set[dev].store(1, std::memory_order_release);
  }
  *clusters = active[dev].load(std::memory_order_relaxed);
  return NT_OK;
}
template <typename T, int D>
nt_status set_up_few_rows(int R, int* clusters) {
  return few_rows(R) == 8 ? set_up_few<T, D, 8>(clusters) : few_rows(R) == 16 ? set_up_few<T, D, 16>(clusters) : set_up_few<T, D, 32>(clusters);
}

template <typename T, int D, int RP>
nt_status launch_few(const TaMaps& maps, const TaArgs& a, cudaStream_t st) {
  constexpr int smem = TfShape<T, D, RP>::kSmem;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = few_config(attr, (unsigned)(a.groups * a.nsplit), smem, a.cluster ? a.nsplit : 1, st);
  NT_CUDA_TRY(cudaLaunchKernelEx(&cfg, tree_few_kernel<T, D, RP>, maps, a));
  return check_launch("tree_few_kernel");
}
template <typename T, int D>
nt_status launch_few_rows(const TaMaps& maps, const TaArgs& a, cudaStream_t st) {
  return few_rows(a.R) == 8 ? launch_few<T, D, 8>(maps, a, st)
         : few_rows(a.R) == 16 ? launch_few<T, D, 16>(maps, a, st) : launch_few<T, D, 32>(maps, a, st);
}

}  // namespace

nt_status set_up_tree_few(int R, int dtype, int D, int* clusters) {
  if (dtype == NT_F32) return D == 64 ? set_up_few_rows<float, 64>(R, clusters) : set_up_few_rows<float, 128>(R, clusters);
  return D == 64 ? set_up_few_rows<uint16_t, 64>(R, clusters) : set_up_few_rows<uint16_t, 128>(R, clusters);
}

nt_status launch_tree_few(const TaMaps& maps, const TaArgs& a, int dtype, int D, cudaStream_t st) {
  if (dtype == NT_F32) return D == 64 ? launch_few_rows<float, 64>(maps, a, st) : launch_few_rows<float, 128>(maps, a, st);
  return D == 64 ? launch_few_rows<uint16_t, 64>(maps, a, st) : launch_few_rows<uint16_t, 128>(maps, a, st);
}

}  // namespace nt
