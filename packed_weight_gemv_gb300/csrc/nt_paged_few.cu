// nt_paged_few.cu -- paged attention of sequences with up to 8 query rows per key-value head: single tokens, and two or more
// where few heads share one.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(x_j log2(e) - m)
//
// Such a call is bound by reading keys and values once, 512 bytes a key at D 128 against 4 D products a row, so it runs on the fp32
// units: every product and sum is fp32. A warp takes 16 keys (D 64: 32) at a time, 8 dimensions a lane; the lanes' shares of the
// scores are summed while they are dealt out, so that a lane ends with R / 2 of the 8 R sums (R rows, D 128) after 7.5 R
// shuffles and takes the exponentials of these alone; the weights come back through shared memory. The reference m of a row is raised
// only when a score exceeds it by 2^8.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "nt_tree_attn.cuh"
#include "nt_paged.cuh"

namespace nt {
namespace {

constexpr int kFewWarps = 8, kFewThreads = 32 * kFewWarps;
constexpr int kFewKeys = 64;  // keys per tile of the division
constexpr int kFewStart = 1;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float4*>(p);
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(low_f(u.x), high_f(u.x), low_f(u.y), high_f(u.y));
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = v;
  else *reinterpret_cast<uint2*>(p) = make_uint2(pack_rn(v.x, v.y), pack_rn(v.z, v.w));
}

template <typename T, int D, int R, bool kExtra>
__global__ void __launch_bounds__(kFewThreads, R <= 2 ? 2 : 1) paged_few_kernel(const __grid_constant__ PaArgs a) {
  constexpr int kLanes = D / 8;            // lanes of a key
  constexpr int kAt = 32 / kLanes;         // keys of a load
  constexpr int kBlock = 8 * kAt;          // keys of a warp at a time
  constexpr int kSums = R * 8 / kLanes > 0 ? R * 8 / kLanes : 1;  // scores that end in a lane
  constexpr int kRowLanes = kLanes / R;    // lanes with scores of one row
  extern __shared__ int s_starts[];
  __shared__ __align__(16) float s_q[R][D];
  __shared__ __align__(16) float s_p[kFewWarps][kAt][R][8];
  __shared__ __align__(16) float s_o[kFewWarps][R][D];
  __shared__ float s_m[kFewWarps][R], s_l[kFewWarps][R];
  __shared__ int s_pos[R];
  __shared__ int s_last;
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31, dl = lane % kLanes, kg = lane / kLanes;
  dependent_launch_wait();
  PaWalk<kFewKeys, kFewStart> walk(a, pa_share<kFewThreads, kFewKeys, kFewStart>(a, R, s_starts), R);
  // The scores that this lane ends with: row `row`, loads j0 .. j0 + kSums - 1; `own`: the lane counts them.
  int at = 0;
  bool own = true;
  {
    int n = R * 8;
#pragma unroll
    for (int off = kLanes / 2; off; off /= 2) {
      if (n > 1) {
        n /= 2;
        if (lane & off) at += n;
      } else if (lane & off) {
        own = false;
      }
    }
  }
  const int row = at / 8, j0 = at % 8;
  int bad = 0;
  for (; walk.more();) {
    PaPiece p = walk.piece(a);
    const PaUnit& u = p.u;
    auto token = [&](int r) { return (u.mt * R + min(r, u.rows - 1)) / a.G; };  // rows behind the last one repeat it
    auto head = [&](int r) { return p.g * a.G + (u.mt * R + min(r, u.rows - 1)) % a.G; };
    __syncthreads();  // the piece before has been joined
    for (int e = i; e < R * D / 4; e += kFewThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      const T* q = static_cast<const T*>(a.q) + (int64_t)(u.t0 + token(r)) * a.q_stride + (int64_t)head(r) * D + c;
      const float4 x = load4(q);
      const float f = kExtra ? a.scale : a.scale * 1.4426950408889634f;
      *reinterpret_cast<float4*>(&s_q[r][c]) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    }
    if (i < R) s_pos[i] = u.len - u.n + token(i);
    __syncthreads();
    const int pos = s_pos[row];
    const float slope = kExtra && a.slopes ? a.slopes[head(row)] : 0.0f;
    const int hi = min(u.p1 + 1, (p.t0 + u.tile0 + p.n) * kFewKeys);            // no row sees this key or one behind it
    const int64_t sure_lo = max((int64_t)0, (int64_t)u.p1 - a.window + 1);      // every row sees from here
    const int sure_hi = u.p0;                                                   // to here
    const int key0 = (u.tile0 + p.t0) * kFewKeys;
    const int32_t* ids = a.table + (int64_t)u.s * a.width;
    float o[R][8], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < 8; ++d) o[r][d] = 0.0f;

    int base = key0 + warp * kBlock;
    int id[2];
    auto ask = [&](int b) {  // the pages of the 32 keys at b, or of 16
      id[0] = b < hi ? ids[b >> a.shift] : -1;
      id[1] = kBlock == 32 ? (b + 16 < hi ? ids[(b + 16) >> a.shift] : -1) : id[0];
    };
    ask(base);
    for (; base < hi; base += kFewWarps * kBlock) {
      uint4 k[8], v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = base + j * kAt + kg, page = id[kBlock == 32 ? j / 4 : 0];
        const bool there = key < hi && (unsigned)page < (unsigned)a.n_pages;
        if (key < hi && !there) bad = 1;
        const int64_t to = ((int64_t)p.g * a.ts + ((int64_t)page << a.shift) + (key & (a.page - 1))) * D + dl * 8;
        k[j] = there ? *reinterpret_cast<const uint4*>(a.k + to) : make_uint4(0u, 0u, 0u, 0u);
        v[j] = there ? *reinterpret_cast<const uint4*>(a.v + to) : make_uint4(0u, 0u, 0u, 0u);
      }
      ask(base + kFewWarps * kBlock);
      const bool whole = base >= sure_lo && base + kBlock - 1 <= sure_hi;  // every row sees every key
      float2 s2[R][4];  // scores of loads 2 j and 2 j + 1
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[r][j] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float2 lo[4], up[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = reinterpret_cast<const uint32_t*>(&k[2 * j])[w], y = reinterpret_cast<const uint32_t*>(&k[2 * j + 1])[w];
          lo[j] = make_float2(low_f(x), low_f(y));
          up[j] = make_float2(high_f(x), high_f(y));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 q = *reinterpret_cast<const float2*>(&s_q[r][dl * 8 + 2 * w]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s2[r][j] = fma2(make_float2(q.x, q.x), lo[j], s2[r][j]);
            s2[r][j] = fma2(make_float2(q.y, q.y), up[j], s2[r][j]);
          }
        }
      }
      float s[R * 8];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[r * 8 + 2 * j] = s2[r][j].x;
          s[r * 8 + 2 * j + 1] = s2[r][j].y;
        }
      {
        int n = R * 8;
#pragma unroll
        for (int off = kLanes / 2; off; off /= 2) {
          if (n > 1) {
            n /= 2;
            const bool upper = lane & off;
#pragma unroll
            for (int e = 0; e < R * 4; ++e) {
              if (e >= n) break;
              const float give = upper ? s[e] : s[e + n], keep = upper ? s[e + n] : s[e];
              s[e] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
          } else {
            s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
          }
        }
      }
      unsigned seen = ~0u;
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < kSums; ++e) {
        const int key = base + (j0 + e) * kAt + kg;
        if constexpr (kExtra) {
          float x = s[e];
          if (a.cap > 0.0f) x = a.cap * tanhf(x / a.cap);
          if (a.slopes) x -= slope * (float)(pos - key);
          s[e] = x * 1.4426950408889634f;
        }
        if (!whole && (key > pos || (int64_t)key + a.window <= pos)) {
          s[e] = -INFINITY;
          seen &= ~(1u << e);
        }
        mx = fmaxf(mx, s[e]);
      }
#pragma unroll
      for (int off = 1; off < kRowLanes; off *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
#pragma unroll
      for (int off = kLanes; off < 32; off *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      if (__any_sync(0xffffffffu, mx > m + kTaLazy)) {
        const float to = fmaxf(m, mx), corr = to == m ? 1.0f : ex2(m - to);
        l *= corr;
        m = to;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float c = __shfl_sync(0xffffffffu, corr, r * kRowLanes);
#pragma unroll
          for (int d = 0; d < 8; ++d) o[r][d] *= c;
        }
      }
      const float mu = m == -INFINITY ? 0.0f : m;
      __syncwarp();  // the last weights have been read
#pragma unroll
      for (int e = 0; e < kSums; ++e) {
        const float w = ex2(s[e] - mu);
        if (own) l += w;
        s_p[warp][kg][row][j0 + e] = seen >> e & 1 ? w : -1.0f;  // -1: not seen
      }
      __syncwarp();
      auto weigh = [&](auto masked) {
        constexpr bool kMasked = decltype(masked)::value;
#pragma unroll
        for (int jq = 0; jq < 2; ++jq) {
          float4 w[R];
#pragma unroll
          for (int r = 0; r < R; ++r) w[r] = *reinterpret_cast<const float4*>(&s_p[warp][kg][r][jq * 4]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t* x = reinterpret_cast<const uint32_t*>(&v[jq * 4 + j]);
#pragma unroll
            for (int d = 0; d < 8; d += 2) {
              const float2 val = make_float2(low_f(x[d / 2]), high_f(x[d / 2]));
#pragma unroll
              for (int r = 0; r < R; ++r) {
                const float wt = j == 0 ? w[r].x : j == 1 ? w[r].y : j == 2 ? w[r].z : w[r].w;
                float2 acc = make_float2(o[r][d], o[r][d + 1]);
                if constexpr (kMasked) {
                  if (wt >= 0.0f || isnan(wt)) acc = fma2(make_float2(wt, wt), val, acc);
                } else {
                  acc = fma2(make_float2(wt, wt), val, acc);
                }
                o[r][d] = acc.x;
                o[r][d + 1] = acc.y;
              }
            }
          }
        }
      };
      if (whole) weigh(std::false_type{});
      else weigh(std::true_type{});
    }

    // the warp's sums over its lanes' keys, then the warps'
#pragma unroll
    for (int off = kLanes; off < 32; off *= 2) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int d = 0; d < 8; ++d) o[r][d] += __shfl_xor_sync(0xffffffffu, o[r][d], off);
      l += __shfl_xor_sync(0xffffffffu, l, off);
    }
#pragma unroll
    for (int off = 1; off < kRowLanes; off *= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane < kLanes) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        *reinterpret_cast<float4*>(&s_o[warp][r][dl * 8]) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
        *reinterpret_cast<float4*>(&s_o[warp][r][dl * 8 + 4]) = make_float4(o[r][4], o[r][5], o[r][6], o[r][7]);
      }
      if (lane % kRowLanes == 0) {
        s_m[warp][row] = m;
        s_l[warp][row] = l;
      }
    }
    __syncthreads();
    const bool split = p.n < u.tiles;
    const int64_t slot = p.slot;
    auto write = [&](int r, int c, float4 x, float L) {
      if (r >= u.rows) return;
      const float f = L == 0.0f ? 0.0f : 1.0f / L;  // L = 0: the row sees nothing
      T* to = static_cast<T*>(a.out) + ((int64_t)(u.t0 + token(r)) * a.Hq + head(r)) * D + c;
      store4(to, make_float4(x.x * f, x.y * f, x.z * f, x.w * f));
    };
    for (int e = i; e < R * D / 4; e += kFewThreads) {
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
      if (split) {
        *reinterpret_cast<float4*>(a.part + (slot * R + r) * D + c) = x;
        if (c == 0) a.ml[slot * R + r] = make_float2(M, L);
      } else {
        write(r, c, x, L);
      }
    }
    if (split) {
      walk.parts(p);
      const int c0 = p.c0, c1 = p.c1;
      __threadfence();
      __syncthreads();
      if (i == 0) {
        const unsigned before = atomicAdd(a.count + p.job, 1u);
        s_last = before == (unsigned)(c1 - c0);
        if (s_last) a.count[p.job] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int e = i; e < R * D / 4; e += kFewThreads) {
          const int r = e / (D / 4), c = e % (D / 4) * 4;
          float M = -INFINITY, L = 0.0f;
          float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int b0 = c0; b0 <= c1; b0 += 8) {
            float4 y[8];
            float2 ml[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const int64_t from = (int64_t)walk.slot(min(b0 + b, c1)) * R + r;
              y[b] = __ldcg(reinterpret_cast<const float4*>(a.part + from * D + c));
              ml[b] = __ldcg(a.ml + from);
              if (b0 + b > c1) ml[b] = make_float2(-INFINITY, 0.0f);
            }
            float to = M;
#pragma unroll
            for (int b = 0; b < 8; ++b) to = fmaxf(to, ml[b].x);
            const float corr = M == to ? 1.0f : ex2(M - to);
            L *= corr;
            x = make_float4(x.x * corr, x.y * corr, x.z * corr, x.w * corr);
            M = to;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              if (b0 + b > c1) break;
              const float f = ml[b].x == M ? 1.0f : ex2(ml[b].x - M);
              L = fmaf(ml[b].y, f, L);
              x.x = fmaf(y[b].x, f, x.x);
              x.y = fmaf(y[b].y, f, x.y);
              x.z = fmaf(y[b].z, f, x.z);
              x.w = fmaf(y[b].w, f, x.w);
            }
          }
          write(r, c, x, L);
        }
      }
    }
    walk.next(a);
  }
  if (bad && a.n_bad) atomicAdd(a.n_bad, 1u);
}

template <typename T, int D, int R, bool kExtra>
nt_status launch_few(const PaArgs& a, cudaStream_t st) {
  const int per = R <= 2 ? 2 : 1;
  const int ctas = std::min(per * device_sm_count(), kPaFewCtas);
  const size_t smem = (size_t)a.S * sizeof(int);
  static std::atomic<int> allowed[64];
  NT_TRY(allow_smem(paged_few_kernel<T, D, R, kExtra>, kPageMaxSeqs * (int)sizeof(int), allowed));
  NT_CUDA_TRY(launch_kernel(paged_few_kernel<T, D, R, kExtra>, dim3((unsigned)ctas), dim3(kFewThreads), smem, st, true, a));
  return check_launch("paged_few_kernel");
}
template <typename T, int D, bool kExtra>
nt_status launch_few_rows(const PaArgs& a, int64_t max_rows, cudaStream_t st) {
  if (max_rows <= 1) return launch_few<T, D, 1, kExtra>(a, st);
  if (max_rows <= 2) return launch_few<T, D, 2, kExtra>(a, st);
  if (max_rows <= 4) return launch_few<T, D, 4, kExtra>(a, st);
  return launch_few<T, D, 8, kExtra>(a, st);
}

}  // namespace

nt_status launch_paged_few(const PaArgs& a, int dtype, int D, int64_t max_rows, cudaStream_t st) {
  const bool extra = a.cap > 0.0f || a.slopes;
  if (dtype == NT_F32) {
    if (D == 64) return extra ? launch_few_rows<float, 64, true>(a, max_rows, st) : launch_few_rows<float, 64, false>(a, max_rows, st);
    return extra ? launch_few_rows<float, 128, true>(a, max_rows, st) : launch_few_rows<float, 128, false>(a, max_rows, st);
  }
  if (D == 64) return extra ? launch_few_rows<uint16_t, 64, true>(a, max_rows, st) : launch_few_rows<uint16_t, 64, false>(a, max_rows, st);
  return extra ? launch_few_rows<uint16_t, 128, true>(a, max_rows, st) : launch_few_rows<uint16_t, 128, false>(a, max_rows, st);
}

}  // namespace nt
