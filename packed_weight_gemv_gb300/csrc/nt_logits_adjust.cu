// nt_logits_adjust.cu -- sampling adjustments of the logits of a batch of positions (penalties
// for repeated tokens, a bias, a grammar's allowed tokens) with the greedy choice, and the
// token counts that the penalties go by.
//
// Per value: x -> x / r or x * r by its sign, - f * count, - p where the token was used; + bias;
// -inf where it is not allowed. Every step is one fp32 rounding, in this order.
//
// A value is read once and written once, so the kernel is bound by memory if enough reads are on
// their way and the instructions per value are few. A CTA holds a chunk of 2,048 tokens -- their
// counts and biases, when the batch shares them, in registers -- and walks a group of rows over it;
// the rows' values come through shared memory by asynchronous copies, up to four rows ahead.
// Of a warp's 256 tokens a few have been used, in a text's first chunks hundreds. A few are listed and
// adjusted in shared memory, a lane each; for more the penalties are straight-line code for every
// value, two values to an instruction (with a branch around them nearly every warp took it for each of
// a lane's tokens). 64 rows of 151,936 with all adjustments (80 MB): 240 instructions per 128 values 32.5
// us, straight-line for all 24.7, listed 21.6, groups of rows that fill one wave 19.4, the ancestor bits in a
// few loads and the listed tokens in registers 19.1 = 4.2 TB/s, 62 % of the measured copy rate (15.5 where
// L2 holds the rows). Instruction issue, a row's dependent steps and the start of a CTA bound it.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "nt_adjust_plan.cuh"
#include "nt_tree.cuh"

namespace nt {
namespace {

constexpr int kAdjAhead = 4;                // rows of the ring in shared memory
constexpr int kAdjEach = 2;                 // used tokens per lane that are adjusted one by one
constexpr int kAdjFew = 32 * kAdjEach;      // so many of a warp's 256
static_assert(kTreeMaxNodes <= kAdjThreads && kAdjRows * kTreeMaxNodes / 32 <= kAdjThreads, "one thread per node, and per word");

// Workspace: the 16-byte status header, then per row the best (value, index) key and, in the first row
// of a group, the counter of CTAs done with the group; all zero between calls.
struct AdjWs {
  WsHeader head;
  struct Row {
    unsigned long long best;
    unsigned int done, pad_;
  } row[1];
};

struct AdjArgs {
  const float* x;  // [B][V]
  int B, V;
  const int32_t* counts;  // rows counts_stride apart (0: one for all), or null
  int64_t counts_stride;
  const uint32_t* tree_mask;  // [B][mask_words] ancestor bits, or null
  int mask_words;
  const int32_t* tokens;  // [B] the nodes' tokens
  float rep, freq, pres;
  float rep_inv;  // 1 / rep rounded, 0 where quotient() does not hold
  const float* bias;
  int64_t bias_stride;
  const uint32_t* allowed;  // rows allowed_stride words apart
  int64_t allowed_stride;
  float* out;       // [B][V] or null
  int32_t* argmax;  // [B] or null
  AdjWs* ws;
  int group;  // rows of a CTA, at most kAdjRows
};

// x / rep rounded to nearest, by Markstein's method (IBM J. Res. Dev. 34, 1990): with y = 1 / rep
// rounded, one step q + (x - rep q) y brings q = x y within an ulp, and a second one, whose remainder
// is exact, to the rounded quotient. It holds while the quotient is normal and the remainder's last bit is
// no less than 2^-149: for 2^-24 <= rep <= 2^24 and 2^-100 <= |x| < 2^100 the quotient is within 2^-124 and
// 2^124, and the last bits of rep and q multiply to 2^-148 at least.
struct Pair {  // two fp32 values that one instruction works on
  float x, y;
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ Pair both(float v) { return Pair{v, v}; }
__device__ __forceinline__ Pair quotient(Pair x, Pair minus_rep, Pair rep_inv) {
  Pair q = mul2(x, rep_inv);
  q = fma2(fma2(minus_rep, q, x), rep_inv, q);
  return fma2(fma2(minus_rep, q, x), rep_inv, q);
}
// Whether |x| is outside [2^-100, 2^100), as an unsigned number above kAdjRange.
constexpr uint32_t kAdjSmall = (127u - 100u) << 23, kAdjRange = (200u << 23) - 1u;
__device__ __forceinline__ uint32_t size_code(float x) { return (__float_as_uint(x) & 0x7fffffffu) - kAdjSmall; }
// The quotients of values outside that range, out of the way of the others.
__device__ __noinline__ float divide_one(float x, float rep) { return __fdiv_rn(x, rep); }

// Orders values above -inf as unsigned numbers; 0 for the others (-inf and NaN are never chosen).
__device__ __forceinline__ uint32_t choice_key(float y) {
  if (!(y > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(y + 0.0f);  // -0 as +0
  return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}

// CTA: chunk blockIdx.x of the tokens, rows group * blockIdx.y ... . With VEC = 4 a thread has two times
// four neighbouring tokens (16-byte accesses), with VEC = 1 eight that are 256 apart (rows of any alignment).
template <int VEC, bool kPenalties, bool kChoice>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const AdjArgs a) {
  constexpr int N = kAdjPer;
  __shared__ __align__(16) float ring[kAdjAhead][kAdjChunk];         // rows on their way
  __shared__ int path_tok[kTreeMaxNodes];                            // the tree's tokens inside the chunk
  __shared__ uint32_t path_rows[kTreeMaxNodes];                      // bit r: on the path of the group's row r
  __shared__ uint32_t group_mask[kAdjRows * kTreeMaxNodes / 32];     // the group's rows of ancestor bits
  __shared__ int n_path, s_last;
  __shared__ int2 used_list[kPenalties ? kAdjThreads / 32 : 1][kAdjFew];  // (place, bit 16: on a path; count)
  __shared__ unsigned long long row_best[kAdjRows][kAdjThreads / 32];
  dependent_launch_wait();
  const int i = threadIdx.x, lane = i & 31, v0 = blockIdx.x * kAdjChunk;
  const int b0 = blockIdx.y * a.group, nb = min(a.group, a.B - b0);
  // place of the thread's token e in the chunk
  auto place = [&](int e) { return VEC == 4 ? e / 4 * (4 * kAdjThreads) + 4 * i + e % 4 : e * kAdjThreads + i; };
  const int inside = a.V - v0;
  auto on = [&](int e) { return place(VEC == 4 ? e & ~3 : e) < inside; };  // with VEC = 4, V is a multiple of 4
  const bool whole = inside >= kAdjChunk;  // every token of the chunk exists
  // A thread copies its own tokens and reads no other's, so the ring needs no barrier.
  const float* next_x = a.x + (int64_t)b0 * a.V + v0;
  auto fetch = [&](int r) {
    if (r < nb) {
      float* st = ring[r % kAdjAhead];
#pragma unroll
      for (int e = 0; e < N; e += VEC)
        if (whole || on(e)) copy_async<4 * VEC>(st + place(e), next_x + place(e));
      next_x += a.V;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");  // one group per row, an empty one past the last
  };
#pragma unroll
  for (int r = 0; r < kAdjAhead; ++r) fetch(r);
  // A row's allowed bits of this thread: with VEC = 4 of its own two words, with VEC = 1 lane e loads the
  // one of all lanes' token e. Loaded a row ahead.
  const int words = (a.V + 31) / 32 - (v0 >> 5);  // from the chunk's first on
  const int w0 = VEC == 4 ? place(0) >> 5 : (i >> 5) + (lane & 7) * (kAdjThreads / 32), w1 = VEC == 4 ? place(4) >> 5 : 0;
  const uint32_t* next_word = a.allowed ? a.allowed + b0 * a.allowed_stride + (v0 >> 5) : nullptr;
  uint32_t next_allowed[2] = {~0u, ~0u};
  auto load_allowed = [&](int r) {
    if (next_word && r < nb) {
      if (w0 < words) next_allowed[0] = next_word[w0];
      if (VEC == 4 && w1 < words) next_allowed[1] = next_word[w1];
      next_word += a.allowed_stride;
    }
  };
  load_allowed(0);
  float* out = a.out ? a.out + (int64_t)b0 * a.V + v0 : nullptr;

  auto load = [&](const auto* row, auto(&x)[N], auto none) {  // this thread's part of a row of counts or biases
#pragma unroll
    for (int e = 0; e < N; e += VEC) {
      if constexpr (VEC == 4) {
        const uint4 t = on(e) ? *reinterpret_cast<const uint4*>(row + place(e)) : make_uint4(0u, 0u, 0u, 0u);
        memcpy(&x[e], &t, 16);
        if (!on(e)) x[e] = x[e + 1] = x[e + 2] = x[e + 3] = none;
      } else {
        x[e] = on(e) ? row[place(e)] : none;
      }
    }
  };
  int c[N] = {};
  float bias[N];
#pragma unroll
  for (int e = 0; e < N; ++e) bias[e] = -0.0f;  // x + -0 is x, whatever x is
  const bool row_counts = a.counts && a.counts_stride != 0, row_bias = a.bias && a.bias_stride != 0;
  if (a.counts && !row_counts) load(a.counts + v0, c, 0);
  if (a.bias && !row_bias) load(a.bias + v0, bias, -0.0f);
  int np = 0;
  if (a.tree_mask) {  // thread = node: a tree has at most kAdjThreads
    // All CTAs read these few lines at once, so a warp asks for as much as it can (with a load per row and
    // node they waited 3 us for one another's).
    const int t = i < a.B ? a.tokens[i] : -1, used_words = (a.B + 31) / 32;
    if (i < nb * used_words) group_mask[i] = a.tree_mask[(int64_t)(b0 + i / used_words) * a.mask_words + i % used_words];
    if (i == 0) n_path = 0;
    __syncthreads();
    if (t >= v0 && t - v0 < min(kAdjChunk, inside)) {
      uint32_t rows = 0;
      for (int r = 0; r < nb; ++r) rows |= (group_mask[r * used_words + (i >> 5)] >> (i & 31) & 1u) << r;
      const int at = atomicAdd(&n_path, 1);
      path_tok[at] = t - v0;
      path_rows[at] = rows;
    }
    __syncthreads();
    np = n_path;
  }
  uint32_t on_path = 0;  // bit e: token e is on some path of the group
  for (int p = 0; p < np; ++p) {
    const int t = path_tok[p], own = VEC == 4 ? t / 4 % kAdjThreads : t % kAdjThreads;
    const int e = VEC == 4 ? t / (4 * kAdjThreads) * 4 + t % 4 : t / kAdjThreads;
    if (own == i) on_path |= 1u << e;
  }
  const bool warp_path = __any_sync(0xffffffffu, on_path != 0);
  // Most warps have a few used tokens, the same ones in every row: those are listed and adjusted in
  // shared memory, a lane each, before the row is read.
  int listed = -1;  // -1: too many, or other ones in every row
  if (kPenalties && !row_counts) {
    uint32_t mine = on_path;
#pragma unroll
    for (int e = 0; e < N; ++e) mine |= (uint32_t)(c[e] > 0) << e;
    int at = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int before = __shfl_up_sync(0xffffffffu, at, o);
      at += lane >= o ? before : 0;
    }
    listed = __shfl_sync(0xffffffffu, at, 31);
    at -= __popc(mine);
    if (listed <= kAdjFew && mine) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (mine >> e & 1u) used_list[i >> 5][at++] = make_int2(place(e) | (int)(on_path >> e & 1u) << 16, c[e]);
    }
    if (listed > kAdjFew) listed = -1;
  }
  // The lane's listed tokens: place, count, on which rows' paths, and whether several nodes have it.
  int own_at[kAdjEach], own_count[kAdjEach];
  uint32_t own_rows[kAdjEach];
  bool several = false;
#pragma unroll
  for (int k = 0; k < kAdjEach; ++k) own_at[k] = own_count[k] = 0, own_rows[k] = 0u;
  if (listed > 0) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kAdjEach; ++k) {
      if (lane + 32 * k >= listed) continue;
      const int2 t = used_list[i >> 5][lane + 32 * k];
      own_at[k] = t.x & 0xffff;
      own_count[k] = t.y;
      if (t.x >> 16) {
        for (int p = 0; p < np; ++p) {
          if (path_tok[p] != own_at[k]) continue;
          several = several || own_rows[k] != 0;
          own_rows[k] |= path_rows[p];
        }
      }
    }
  }
  float less[N];      // - frequency * count
  uint32_t used = 0;  // bit e: token e has been used
  auto count = [&](const int(&n)[N]) {
    used = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      less[e] = -__fmul_rn(a.freq, __int2float_rn(n[e]));
      used |= (uint32_t)(n[e] > 0) << e;
    }
  };
  if (listed < 0) count(c);

  for (int r = 0; r < nb; ++r) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAdjAhead - 1) : "memory");  // this row is here
    float* st = ring[r % kAdjAhead];
    if (kPenalties && listed > 0) {
      __syncwarp();  // the other lanes' copies
#pragma unroll
      for (int k = 0; k < kAdjEach; ++k) {
        if (32 * k >= listed) break;
        int n = own_count[k] + (int)(own_rows[k] >> r & 1u);
        if (several && own_rows[k]) {
          n = own_count[k];
          for (int p = 0; p < np; ++p) n += path_tok[p] == own_at[k] ? (int)(path_rows[p] >> r & 1u) : 0;
        }
        if (n > 0) {
          const float x = st[own_at[k]];
          float v = quotient(Pair{x, x}, both(-a.rep), both(a.rep_inv)).x;
          if (size_code(x) > kAdjRange || a.rep_inv == 0.0f) v = divide_one(x, a.rep);
          v = x > 0.0f ? v : __fmul_rn(x, a.rep);
          st[own_at[k]] = __fsub_rn(__fsub_rn(v, __fmul_rn(a.freq, __int2float_rn(n))), a.pres);
        }
      }
      __syncwarp();
    }
    float y[N];
#pragma unroll
    for (int e = 0; e < N; e += VEC) {
      if constexpr (VEC == 4) {
        const float4 t = *reinterpret_cast<const float4*>(st + place(e));
        y[e] = t.x; y[e + 1] = t.y; y[e + 2] = t.z; y[e + 3] = t.w;
      } else {
        y[e] = st[place(e)];
      }
    }
    uint32_t allow = 0;  // bit e: token e
    if constexpr (VEC == 4) {
      allow = (next_allowed[0] >> (4 * i & 31) & 15u) | (next_allowed[1] >> (4 * i & 31) & 15u) << 4;
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) allow |= (__shfl_sync(0xffffffffu, next_allowed[0], e) >> (i & 31) & 1u) << e;
    }
    load_allowed(r + 1);
    fetch(r + kAdjAhead);
    if (row_bias) load(a.bias + (b0 + r) * a.bias_stride + v0, bias, -0.0f);
    if (kPenalties && listed < 0) {
      if (row_counts || warp_path) {
        int n[N];
        if (row_counts) load(a.counts + (b0 + r) * a.counts_stride + v0, n, 0);
#pragma unroll
        for (int e = 0; e < N; ++e) n[e] = row_counts ? n[e] : c[e];
        for (int p = 0; warp_path && p < np; ++p)
#pragma unroll
          for (int e = 0; e < N; ++e) n[e] += path_tok[p] == place(e) ? (int)(path_rows[p] >> r & 1u) : 0;
        count(n);
      }
      uint32_t code = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) code = max(code, size_code(y[e]));
      const bool rare = code > kAdjRange || a.rep_inv == 0.0f;
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const Pair x{y[e], y[e + 1]}, low = mul2(x, both(a.rep));
        Pair q = quotient(x, both(-a.rep), both(a.rep_inv));
        if (rare) q = Pair{divide_one(x.x, a.rep), divide_one(x.y, a.rep)};
        Pair v{x.x > 0.0f ? q.x : low.x, x.y > 0.0f ? q.y : low.y};
        v = add2(add2(v, Pair{less[e], less[e + 1]}), both(-a.pres));  // a - b as a + (-b): the same rounding
        y[e] = used >> e & 1u ? v.x : x.x;
        y[e + 1] = used >> (e + 1) & 1u ? v.y : x.y;
      }
    }
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const Pair v = add2(Pair{y[e], y[e + 1]}, Pair{bias[e], bias[e + 1]});
      y[e] = allow >> e & 1u ? v.x : -INFINITY;
      y[e + 1] = allow >> (e + 1) & 1u ? v.y : -INFINITY;
    }
    if (out) {
#pragma unroll
      for (int e = 0; e < N; e += VEC)
        if (whole || on(e)) {
          if constexpr (VEC == 4) __stcs(reinterpret_cast<float4*>(out + place(e)), make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]));
          else __stcs(out + place(e), y[e]);
        }
      out += a.V;
    }
    if constexpr (kChoice) {
      if (!whole) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (!on(e)) y[e] = -INFINITY;
      }
      float tops[2] = {y[0], y[1]};  // NaN is left out
#pragma unroll
      for (int e = 2; e < N; e += 2) tops[e >> 1 & 1] = max3(tops[e >> 1 & 1], y[e], y[e + 1]);
      const float top = fmaxf(tops[0], tops[1]);
      const uint32_t key = choice_key(top), most = __reduce_max_sync(0xffffffffu, key);
      uint32_t at = ~0u;  // the lowest token with that value
      if (key == most) {
#pragma unroll
        for (int e = N - 1; e >= 0; --e)
          if (y[e] == top) at = v0 + place(e);
      }
      at = __reduce_min_sync(0xffffffffu, at);
      if (lane == 0) row_best[r][i >> 5] = most ? ((unsigned long long)most << 32) | (uint32_t)~at : 0ull;
    }
  }
  if constexpr (!kChoice) return;
  __syncthreads();
  unsigned long long best = 0;
  AdjWs::Row* row = a.ws->row + b0;
  if (i < nb) {  // thread = row of the group
#pragma unroll
    for (int k = 0; k < kAdjThreads / 32; ++k) best = row_best[i][k] > best ? row_best[i][k] : best;
    if (gridDim.x > 1) {
      if (best) atomicMax(&row[i].best, best);
      __threadfence();
    }
  }
  if (gridDim.x > 1) {
    __syncthreads();
    if (i == 0) s_last = atomicAdd(&row[0].done, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (i < nb) best = atomicExch(&row[i].best, 0ull);  // the group's last CTA; back to zero for the next call
    if (i == 0) row[0].done = 0u;
  }
  if (i < nb) a.argmax[b0 + i] = best ? (int32_t)~(uint32_t)best : -1;
}

__global__ void __launch_bounds__(kAdjThreads) count_kernel(const int32_t* tokens, const int32_t* index, int n,
                                                            const int32_t* n_dev, int V, int32_t* counts, uint32_t* n_bad) {
  dependent_launch_wait();
  const int m = n_dev ? min(n, *n_dev) : n;
  for (int64_t i = blockIdx.x * kAdjThreads + threadIdx.x; i < m; i += gridDim.x * kAdjThreads) {
    const int64_t at = index ? index[i] : i;
    const int t = at >= 0 && at < n ? tokens[at] : -1;
    if (t >= 0 && t < V) atomicAdd(counts + t, 1);
    else if (n_bad) atomicAdd(n_bad, 1u);
  }
}

}  // namespace
}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_token_counts(const int32_t* tokens, const int32_t* index_opt, int n, const int32_t* n_opt, int V,
                          int32_t* counts, uint32_t* n_bad_opt, void* stream) {
  clear_error();
  if (n < 0 || V < 1) return set_error(NT_ERR_INVALID_ARG, "need n >= 0 and V >= 1");
  if (!counts || (n > 0 && !tokens)) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(tokens, 4) || !aligned(counts, 4) || (index_opt && !aligned(index_opt, 4)) ||
      (n_opt && !aligned(n_opt, 4)) || (n_bad_opt && !aligned(n_bad_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  NT_TRY(check_device());
  if (n == 0) return NT_OK;
  const int grid = (int)std::min<int64_t>(((int64_t)n + kAdjThreads - 1) / kAdjThreads, 8 * device_sm_count());
  NT_CUDA_TRY(launch_kernel(count_kernel, dim3(grid), dim3(kAdjThreads), 0, reinterpret_cast<cudaStream_t>(stream), true,
                            tokens, index_opt, n, n_opt, V, counts, n_bad_opt));
  return check_launch("count_kernel");
}

nt_status nt_logits_adjust_workspace_size(int V, int B, size_t* bytes) {
  clear_error();
  if (!bytes || V < 1 || B < 1) return set_error(NT_ERR_INVALID_ARG, "need V, B >= 1 and a result pointer");
  *bytes = sizeof(WsHeader) + sizeof(AdjWs::Row) * (size_t)B;
  return NT_OK;
}

nt_status nt_logits_adjust(const float* logits, int B, int V, const int32_t* counts_opt, int64_t counts_stride,
                           const uint32_t* tree_mask_opt, int mask_words, const int32_t* tokens_opt, float repetition,
                           float frequency, float presence, const float* bias_opt, int64_t bias_stride,
                           const uint32_t* allowed_opt, int64_t allowed_stride, float* out_opt, int32_t* argmax_opt,
                           void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (!logits || (!out_opt && !argmax_opt)) return set_error(NT_ERR_INVALID_ARG, "NULL logits, or no output at all");
  if (B < 1 || B > 65535 || V < 1 || V > INT32_MAX - 65536)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= B <= 65535 and 1 <= V <= 2^31 - 65537");
  if ((tree_mask_opt == nullptr) != (tokens_opt == nullptr))
    return set_error(NT_ERR_INVALID_ARG, "a tree needs both its mask and its tokens");
  if (tree_mask_opt && (B > kTreeMaxNodes || mask_words < (B + 31) / 32))
    return set_error(NT_ERR_INVALID_ARG, "a tree has at most 256 nodes and a mask of at least B bits per row");
  if (!(repetition > 0.0f) || !(repetition < INFINITY) || !(fabsf(frequency) < INFINITY) || !(fabsf(presence) < INFINITY))
    return set_error(NT_ERR_INVALID_ARG, "need repetition > 0 and finite penalties");
  if (counts_stride < 0 || bias_stride < 0 || allowed_stride < 0 || (counts_stride && counts_stride < V) ||
      (bias_stride && bias_stride < V) || (allowed_stride && allowed_stride < ((int64_t)V + 31) / 32))
    return set_error(NT_ERR_INVALID_ARG, "strides are 0 (one row for all) or at least a row");
  if (!aligned(logits, 4) || (counts_opt && !aligned(counts_opt, 4)) || (tree_mask_opt && !aligned(tree_mask_opt, 4)) ||
      (tokens_opt && !aligned(tokens_opt, 4)) || (bias_opt && !aligned(bias_opt, 4)) ||
      (allowed_opt && !aligned(allowed_opt, 4)) || (out_opt && !aligned(out_opt, 4)) ||
      (argmax_opt && !aligned(argmax_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "arrays must be 4-byte aligned");
  if (argmax_opt && (!ws || !aligned(ws, 16) || ws_bytes < sizeof(WsHeader) + sizeof(AdjWs::Row) * (size_t)B))
    return set_error(NT_ERR_WORKSPACE, "workspace NULL, misaligned or smaller than nt_logits_adjust_workspace_size");
  NT_TRY(check_device());
  AdjArgs a{logits, B, V, counts_opt, counts_stride, tree_mask_opt, mask_words, tokens_opt, repetition, frequency,
            presence, 0.0f, bias_opt, bias_stride, allowed_opt, allowed_stride, out_opt, argmax_opt, static_cast<AdjWs*>(ws),
            1};
  if (repetition >= 0x1p-24f && repetition <= 0x1p24f) a.rep_inv = 1.0f / repetition;
  const bool vec = V % 4 == 0 && aligned(logits, 16) && (!out_opt || aligned(out_opt, 16)) &&
                   (!counts_opt || (aligned(counts_opt, 16) && counts_stride % 4 == 0)) &&
                   (!bias_opt || (aligned(bias_opt, 16) && bias_stride % 4 == 0));
  const bool pen = counts_opt || tree_mask_opt;
  auto kern = vec ? (pen ? (argmax_opt ? adjust_kernel<4, true, true> : adjust_kernel<4, true, false>)
                         : (argmax_opt ? adjust_kernel<4, false, true> : adjust_kernel<4, false, false>))
                  : (pen ? (argmax_opt ? adjust_kernel<1, true, true> : adjust_kernel<1, true, false>)
                         : (argmax_opt ? adjust_kernel<1, false, true> : adjust_kernel<1, false, false>));
  a.group = adjust_group(B, V, device_sm_count());
  const dim3 grid((V + kAdjChunk - 1) / kAdjChunk, (B + a.group - 1) / a.group);
  NT_CUDA_TRY(launch_kernel(kern, grid, dim3(kAdjThreads), 0, reinterpret_cast<cudaStream_t>(stream), true, a));
  return check_launch("adjust_kernel");
}

}  // extern "C"
