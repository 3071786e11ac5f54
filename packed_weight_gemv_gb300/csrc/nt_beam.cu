// nt_beam.cu -- the next beams of beam search: per group of W beams the K best of their W * V continuations.
//
//   key(w, v) = ((score[w] - log S[w]) + (x[w][v] - M[w])) / (len[w] + 1)^alpha,   M[w] = max_v x[w][v],   S[w] = sum_v e^(x[w][v] - M[w])
//
// The largest logit comes off first: where a mask has put a whole row at the type's lowest value, score and log S would be lost in it (such
// a beam's keys came out as 0, above every other).
//
// Keys are compared in pairs of fp32 (a sum of two, 48 bits), ties by the lower beam and then the lower token: continuations of a beam are
// often closer than fp32 tells apart at its score's size. Between beams the order is as good as log S, which all continuations
// of a beam share: S is summed in fp32. At the very most log S is off by 2^-18 for up to 262,144 tokens and 2^-17 for more (a term that matters
// is D = log V below the largest at most; subtractions and exponents cost 2 D steps of 2^-24, three exponentials 4 each, sums 31 and
// one for every further 512 elements of a chunk), and as a rule by 2^-23 (2^-21.5 where all but one of 151,936 are alike). Weights in more than fp32 would take as long as reading the
// logits does, or longer.
//
// The first kernel reads the logits once: for every chunk of a row its maximum and the sum of e^(x - maximum), and the row's
// 1 / len^alpha beside. The second one, a CTA per group, joins the sums and then reads again only the K chunks that can hold
// the best: the K best elements stand in the K chunks that come first by maximum (ties by order), for an element of another
// chunk has the K maxima before it. So the logits cross the memory once and a group's K chunks from L2.
//
// 128 rows of 151,936 take 24 us (a fifth of the rows is finished and not read; as single cold launches the scan takes 15.0, 61 MB at 4.1 TB/s,
// and the choice 16.7); 4 rows 12 us and 48 of 32,003 with 32 best 15 us, the latency of two launches and four dependent round trips of the choice.
#include <cmath>

#include <algorithm>
#include <atomic>

#include "nt_pages.cuh"

namespace nt {
namespace {

constexpr int kBeamMax = 64;          // beams of a group, and continuations chosen
constexpr int kChunkMin = 512;        // elements of a chunk: 16 per lane of a warp
constexpr int kChunksMax = 512;       // per row
constexpr int kScanThreads = 256;
constexpr int kPickThreads = 512;
constexpr int kGroups = 128;          // sets of items whose maxima bound the K-th best
constexpr int kList = 1024;           // items that may reach the bound
constexpr int kMany = 160;            // beyond, the list is sifted: every item's rank takes as many steps as there are items

struct BeamArgs {
  const float* logits;   // [N][V]
  const float* scores;   // [N]
  const int32_t* done;   // [N] or null
  const int32_t* lens;   // [N] or null
  int32_t *parent, *token;
  float* score;
  int32_t* done_out;     // or null
  float2* chunks;        // [N][nchunks] (maximum, sum)
  double* scale;         // [N] 1 / len^alpha
  int N, V, W, K, chunk, nchunks, eos, wide;
  double alpha;
};

__device__ __forceinline__ bool row_done(const BeamArgs& a, int row) { return a.done && a.done[row] != 0; }

// e^x for x <= 0 (e^-inf = 0): log2(e) in two parts, as one part's error would be that of every term alike.
__device__ __forceinline__ float weight(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(x, 1.44269502e+0f, x * 1.92596299e-8f)));
  return y;
}

// A warp per chunk.
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamArgs a, int64_t jobs) {
  dependent_launch_wait();
  // 1 / len^alpha (at least 2^-124) of 32 rows by the first warp of each of the first CTAs: 64-bit operations take an SM 16 cycles a warp, however few
  // of its lanes want them.
  const int own = blockIdx.x * 32 + threadIdx.x;
  if (a.alpha != 0.0 && threadIdx.x < 32 && own < a.N) {
    const bool ended = row_done(a, own);
    a.scale[own] = 1.0 / pow((double)max(a.lens[own], ended ? 1 : 0) + (ended ? 0.0 : 1.0), a.alpha);
  }
  const int64_t job = (int64_t)blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);
  if (job >= jobs) return;
  const int lane = threadIdx.x & 31, row = (int)(job / a.nchunks), c = (int)(job - (int64_t)row * a.nchunks);
  const bool done = row_done(a, row);
  if (done) return;  // it has one continuation, which is known
  const float* x = a.logits + (int64_t)row * a.V;
  const int v0 = c * a.chunk, v1 = min(a.V, v0 + a.chunk);
  float m = -INFINITY, sum = 0.0f;
  for (int v = v0; v < v1; v += kChunkMin) {
    float y[16];
    if (a.wide && v + kChunkMin <= v1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(x + v) + k * 32 + lane);
        y[4 * k] = f.x; y[4 * k + 1] = f.y; y[4 * k + 2] = f.z; y[4 * k + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) y[k] = v + k * 32 + lane < v1 ? __ldcs(x + v + k * 32 + lane) : -INFINITY;
    }
    float mx = m;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      y[k] = fmaxf(y[k], -INFINITY);  // NaN counts as -inf
      mx = fmaxf(mx, y[k]);
    }
    if (mx > -INFINITY) {
      sum *= weight(m - mx);
      float more[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < 16; ++k) more[k & 3] += weight(y[k] - mx);
      sum += (more[0] + more[1]) + (more[2] + more[3]);
    }
    m = mx;
  }
  float M = m;
#pragma unroll
  for (int d = 16; d; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  sum = m > -INFINITY ? sum * weight(m - M) : 0.0f;
#pragma unroll
  for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) a.chunks[job] = make_float2(M, sum);
}

// Order of fp32 as that of unsigned integers; 0 stands for no item.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
// A row's largest logit, what is added to the logits less that, and the factor that ranks it: pairs of fp32.
struct RowKey {
  float top, add_hi, add_lo, mul_hi, mul_lo;  // add_hi NaN: the row has no continuation
};
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}
__device__ __forceinline__ void fast_two_sum(float a, float b, float& s, float& e) {  // |a| >= |b|
  s = __fadd_rn(a, b);
  e = __fsub_rn(b, __fsub_rn(s, a));
}
// (x - top) plus what the row adds; not finite where that is below the range.
__device__ __forceinline__ float2 total_of(const RowKey& r, float x) {
  float d, f, s, e;
  two_sum(x, -r.top, d, f);
  two_sum(r.add_hi, d, s, e);
  two_sum(s, __fadd_rn(e, __fadd_rn(f, r.add_lo)), s, e);
  return make_float2(s, e);
}
__device__ __forceinline__ uint64_t key_of(const RowKey& r, float x) {
  if (!(x > -INFINITY) || isnan(r.add_hi)) return 0;
  const float2 t = total_of(r, x);
  if (!isfinite(t.x)) return 0;
  float p = __fmul_rn(t.x, r.mul_hi);
  float q = __fmaf_rn(t.x, r.mul_hi, -p);
  q = __fmaf_rn(t.x, r.mul_lo, __fmaf_rn(t.y, r.mul_hi, q));
  fast_two_sum(p, q, p, q);
  q = q + 0.0f;  // -0 as +0
  p = p + 0.0f;
  return (uint64_t)ordered(p) << 32 | ordered(q);
}

struct Item {
  uint64_t key;
  int at;
};
__device__ __forceinline__ bool before(uint64_t ka, int a, uint64_t kb, int b) { return ka > kb || (ka == kb && a < b); }
__device__ __forceinline__ uint64_t shfl_max(uint64_t k, int d) {
  const uint64_t o = __shfl_xor_sync(0xffffffffu, k, d);
  return o > k ? o : k;
}

struct PickShared {
  uint64_t gmax[kGroups];
  uint64_t key[kList];
  int at[kList];
  uint64_t bound;
  int n;
  uint64_t wkey[kPickThreads / 32];
  int wat[kPickThreads / 32];
};

// An item that reaches the bound, into the list.
__device__ __forceinline__ void collect(PickShared& s, bool in, uint64_t key, int at) {
  const int lane = threadIdx.x & 31;
  const unsigned who = __ballot_sync(0xffffffffu, in);
  if (who == 0) return;
  int to = 0;
  if (lane == __ffs(who) - 1) to = atomicAdd(&s.n, __popc(who));
  to = __shfl_sync(0xffffffffu, to, __ffs(who) - 1) + __popc(who & ((1u << lane) - 1));
  if (in && to < kList) {
    s.key[to] = key;
    s.at[to] = at;
  }
}

// Every thread's best of the items dealt to it: the K-th best of the maxima of sets of four threads is a bound that K items reach, into
// s.bound (0 where there are fewer sets with an item); s.n is 0 afterwards.
__device__ void bound_of(uint64_t mine, int K, PickShared& s) {
  const int i = threadIdx.x;
#pragma unroll
  for (int d = 1; d < kPickThreads / kGroups; d *= 2) mine = shfl_max(mine, d);
  if (i % (kPickThreads / kGroups) == 0) s.gmax[i / (kPickThreads / kGroups)] = mine;
  if (i == 0) {
    s.bound = 0;
    s.n = 0;
  }
  __syncthreads();
  if (i < kGroups) {
    const uint64_t k = s.gmax[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < kGroups; ++j) rank += before(s.gmax[j], j, k, i);
    if (rank == K - 1) s.bound = k;
  }
  __syncthreads();
}

// The K best of the list, or, where it has overflowed, of all n items one after the other: (key, place), in order, into out_key and
// out_at (shared; places -1 where there are fewer). fetch(i) is item i's key; 0 is none.
template <typename F>
__device__ void best(int n, int K, F fetch, PickShared& s, uint64_t* out_key, int* out_at) {
  const int i = threadIdx.x, lane = i & 31;
  if (i < K) {
    out_key[i] = 0;
    out_at[i] = -1;
  }
  __syncthreads();
  int m = s.n;
  if (m > kMany && m <= kList) {  // by a bound of its own (one beam of 1,000 tokens, 64 best: 78 us by the ranks of all 1,000, 23 this way)
    uint64_t key[kList / kPickThreads], mine = 0;
    int at[kList / kPickThreads];
#pragma unroll
    for (int e = 0; e < kList / kPickThreads; ++e) {
      const int from = e * kPickThreads + i;
      key[e] = from < m ? s.key[from] : 0;
      at[e] = from < m ? s.at[from] : -1;
      mine = max(mine, key[e]);
    }
    __syncthreads();  // s.n has been read
    bound_of(mine, K, s);
#pragma unroll
    for (int e = 0; e < kList / kPickThreads; ++e) collect(s, key[e] != 0 && key[e] >= s.bound, key[e], at[e]);
    __syncthreads();
    m = s.n;
  }
  if (m <= kList) {  // every item's rank among those that reach the bound
    for (int e = i; e < m; e += kPickThreads) {
      const uint64_t k = s.key[e];
      const int at = s.at[e];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < m; ++j) rank += before(s.key[j], s.at[j], k, at);
      if (rank < K) {
        out_key[rank] = k;
        out_at[rank] = at;
      }
    }
    __syncthreads();
    return;
  }
  // Too many alike (a row of equal logits): one after the other.
  uint64_t last = ~0ull;
  int last_at = -1;
  for (int r = 0; r < K; ++r) {
    uint64_t top = 0;
    int at = INT32_MAX;
    for (int e = i; e < n; e += kPickThreads) {
      const uint64_t k = fetch(e);
      if (k != 0 && before(last, last_at, k, e) && before(k, e, top, at)) {
        top = k;
        at = e;
      }
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
      const uint64_t k = __shfl_xor_sync(0xffffffffu, top, d);
      const int o = __shfl_xor_sync(0xffffffffu, at, d);
      if (before(k, o, top, at)) {
        top = k;
        at = o;
      }
    }
    __syncthreads();
    if (lane == 0) {
      s.wkey[i >> 5] = top;
      s.wat[i >> 5] = at;
    }
    __syncthreads();
    for (int w = 0; w < kPickThreads / 32; ++w)
      if (w == 0 || before(s.wkey[w], s.wat[w], top, at)) {
        top = s.wkey[w];
        at = s.wat[w];
      }
    if (top == 0) break;
    if (i == 0) {
      out_key[r] = top;
      out_at[r] = at;
    }
    last = top;
    last_at = at;
  }
  __syncthreads();
}

// The K best of n items, dealt to the threads in turn.
template <typename F>
__device__ void pick(int n, int K, F fetch, PickShared& s, uint64_t* out_key, int* out_at) {
  const int i = threadIdx.x;
  uint64_t mine = 0;
#pragma unroll 1
  for (int e = i; e < n; e += kPickThreads) mine = max(mine, fetch(e));
  bound_of(mine, K, s);
  const uint64_t bound = s.bound > 0 ? s.bound : 1;
#pragma unroll 1
  for (int e0 = 0; e0 < n; e0 += kPickThreads) {
    const int e = e0 + i;
    const uint64_t k = e < n ? fetch(e) : 0;
    collect(s, k >= bound, k, e);
  }
  best(n, K, fetch, s, out_key, out_at);
}

__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamArgs a) {
  extern __shared__ float s_max[];  // [W][nchunks]
  __shared__ PickShared s;
  __shared__ RowKey s_row[kBeamMax];
  __shared__ uint64_t s_key[2][kBeamMax];
  __shared__ int s_at[2][kBeamMax];
  __shared__ unsigned char s_done[kBeamMax];
  dependent_launch_wait();
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const int row0 = blockIdx.x * a.W;
  for (int w = warp; w < a.W; w += kPickThreads / 32) {
    const int row = row0 + w;
    const bool done = row_done(a, row);
    const float2* c = a.chunks + (int64_t)row * a.nchunks;
    float M = -INFINITY, S = 0.0f;
    if (done) {
      for (int j = lane; j < a.nchunks; j += 32) s_max[w * a.nchunks + j] = j == a.eos / a.chunk ? 0.0f : -INFINITY;
      M = 0.0f;
      S = 1.0f;
    } else {
      constexpr int kMost = kChunksMax / 32;
      float2 y[kMost];  // all asked for at once
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int j = k * 32 + lane;
        y[k] = j < a.nchunks ? __ldcg(c + j) : make_float2(-INFINITY, 0.0f);
      }
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int j = k * 32 + lane;
        if (j < a.nchunks) s_max[w * a.nchunks + j] = y[k].x;
        M = fmaxf(M, y[k].x);
      }
#pragma unroll
      for (int d = 16; d; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
#pragma unroll
      for (int k = 0; k < kMost; ++k)
        if (y[k].x > -INFINITY) S += y[k].y * expf(y[k].x - M);
#pragma unroll
      for (int d = 16; d; d /= 2) S += __shfl_xor_sync(0xffffffffu, S, d);
    }
    if (lane == 0) {
      s_row[w].top = M;
      s_row[w].add_lo = S;
      s_done[w] = done;
    }
  }
  __syncthreads();
  if (i < a.W) {  // a lane per row: see above
    const float sc = a.scores[row0 + i], M = s_row[i].top, S = s_row[i].add_lo;
    const double add = s_done[i] ? (double)sc : (double)sc - log((double)S);
    RowKey r;
    r.top = M;
    r.add_hi = (float)add;
    r.add_lo = (float)(add - (double)r.add_hi);
    r.mul_hi = 1.0f;
    r.mul_lo = 0.0f;
    if (a.alpha != 0.0) {
      const double mul = a.scale[row0 + i];
      r.mul_hi = (float)mul;
      r.mul_lo = (float)(mul - (double)r.mul_hi);
    }
    // no finite score, nothing above -inf, or a logit of +inf: no continuation
    if (!isfinite(sc) || !isfinite(M) || !isfinite(r.add_hi) || !(isfinite(r.mul_hi) && r.mul_hi > 0.0f)) r.add_hi = NAN;
    s_row[i] = r;
  }
  __syncthreads();
  const int nch = a.nchunks;
  pick(a.W * nch, a.K, [&](int e) { return key_of(s_row[e / nch], s_max[e]); }, s, s_key[0], s_at[0]);
  // The elements of the chosen chunks, in the order of the chunks' places so that ties keep theirs. The K-th chunk's maximum is a bound
  // that K elements reach.
  uint64_t bound = s_key[0][a.K - 1] > 0 ? s_key[0][a.K - 1] : 1;
  if (i == 0) s.n = 0;
  if (i < a.K) {
    const int at = s_at[0][i];
    int rank = 0;
    for (int j = 0; j < a.K; ++j) rank += (unsigned)s_at[0][j] < (unsigned)at || (s_at[0][j] == at && j < i);
    s_at[1][rank] = at;  // -1, none, comes last
  }
  __syncthreads();
  const int chunk = a.chunk;
  auto element = [&](int e) -> uint64_t {
    const int place = s_at[1][e / chunk];
    if (place < 0) return 0;
    const int w = place / nch, v = (place - w * nch) * chunk + e % chunk;
    if (v >= a.V) return 0;
    if (s_done[w]) return v == a.eos ? key_of(s_row[w], 0.0f) : 0;
    return key_of(s_row[w], __ldcg(a.logits + (int64_t)(row0 + w) * a.V + v));
  };
  // A warp per 512 elements, all of them asked for at once: of a finished beam one(row, e0, e), e its one continuation's place among them
  // (outside [0, 512): none), of others all(row, e0, y), y[k] element 32 k + lane.
  auto elements = [&](auto&& one, auto&& all) {
    for (int e0 = warp * kChunkMin; e0 < a.K * chunk; e0 += kPickThreads / 32 * kChunkMin) {
      const int place = s_at[1][e0 / chunk];
      if (place < 0) continue;
      const int w = place / nch, v0 = (place - w * nch) * chunk + e0 % chunk;
      if (s_done[w]) {
        one(s_row[w], e0, a.eos - v0);
        continue;
      }
      const float* x = a.logits + (int64_t)(row0 + w) * a.V + v0;
      float y[kChunkMin / 32];
#pragma unroll
      for (int k = 0; k < kChunkMin / 32; ++k) y[k] = v0 + k * 32 + lane < a.V ? __ldcg(x + k * 32 + lane) : -INFINITY;
      all(s_row[w], e0, y);
    }
  };
  auto gather = [&] {
    elements(
        [&](const RowKey& row, int e0, int e) {
          collect(s, lane == 0 && e >= 0 && e < kChunkMin && key_of(row, 0.0f) >= bound, key_of(row, 0.0f), e0 + e);
        },
        [&](const RowKey& row, int e0, const float (&y)[kChunkMin / 32]) {
          // What is below the bound by more than fp32 can err is left out (few stay), the others' keys are formed.
          const float level = unordered((uint32_t)(bound >> 32)) / row.mul_hi,
                      least = level - row.add_hi + row.top - 1e-5f * (fabsf(level) + fabsf(row.add_hi) + fabsf(row.top));
          unsigned may = 0;
#pragma unroll
          for (int k = 0; k < kChunkMin / 32; ++k) may |= (y[k] > -INFINITY && !(y[k] < least) ? 1u : 0u) << k;
#pragma unroll 1
          while (__any_sync(0xffffffffu, may != 0)) {
            const int k = __ffs(may) - 1;
            float z = -INFINITY;
#pragma unroll
            for (int j = 0; j < kChunkMin / 32; ++j)
              if (j == k) z = y[j];
            const uint64_t key = key_of(row, z);
            collect(s, key >= bound, key, e0 + k * 32 + lane);
            may &= may - 1;
          }
        });
  };
  // With few chunks to choose from (a small vocabulary, or finished beams) the last of them says little: of 16 beams of 1,000 tokens, 32
  // best, some thousand elements reach its maximum, and a list that overflows took 660 us, of 32 beams, 64 best 2,100; now 19 and 25. There
  // the threads' best elements give a bound that some hundred reach; it is formed at once where it is sure to be wanted.
  bool sharp = a.W * nch < 4 * a.K && min(a.W * nch, a.K) * chunk > kList;
#pragma unroll 1
  while (true) {
    if (sharp) {
      uint64_t mine = 0;
      elements([&](const RowKey& row, int, int e) { if (lane == 0 && e >= 0 && e < kChunkMin) mine = max(mine, key_of(row, 0.0f)); },
               [&](const RowKey& row, int, const float (&y)[kChunkMin / 32]) {
                 float m = -INFINITY;
#pragma unroll
                 for (int k = 0; k < kChunkMin / 32; ++k) m = fmaxf(m, y[k]);
                 mine = max(mine, key_of(row, m));
               });
      bound_of(mine, a.K, s);
      bound = max(bound, s.bound);
    }
    gather();
    __syncthreads();
    if (sharp || s.n <= kList) break;
    sharp = true;
    __syncthreads();  // s.n has been read
  }
  best(a.K * chunk, a.K, element, s, s_key[0], s_at[0]);
  if (i < a.K) {
    const int e = s_at[0][i];
    const int64_t to = (int64_t)blockIdx.x * a.K + i;
    int up = -1, token = -1, fin = 0;
    float score = -INFINITY;
    if (e >= 0) {
      const int place = s_at[1][e / chunk], w = place / nch;
      token = (place - w * nch) * chunk + e % chunk;
      up = row0 + w;
      fin = s_done[w] || token == a.eos;
      score = s_done[w] ? a.scores[up] : total_of(s_row[w], a.logits[(int64_t)up * a.V + token]).x;
    }
    a.parent[to] = up;
    a.token[to] = token;
    a.score[to] = score;
    if (a.done_out) a.done_out[to] = fin;
  }
}

// ---- host -----------------------------------------------------------------------------------
int chunk_of(int V) {
  int c = kChunkMin;
  while ((V + (int64_t)c - 1) / c > kChunksMax) c *= 2;
  return c;
}
int chunks_of(int V) { return (int)((V + (int64_t)chunk_of(V) - 1) / chunk_of(V)); }
size_t beam_ws_bytes(int V, int N) { return kWsHeaderBytes + (size_t)N * (chunks_of(V) * sizeof(float2) + sizeof(double)); }

}  // namespace
}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_beam_select_workspace_size(int V, int N, size_t* bytes) {
  clear_error();
  if (!bytes || V < 1 || V > kBeamMaxVocab || N < 1 || N > kBeamMaxRows)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= V <= 2^24, 1 <= N <= 65536 and a result pointer");
  *bytes = beam_ws_bytes(V, N);
  return NT_OK;
}

nt_status nt_beam_select(const float* logits, const float* scores, int N, int W, int V, int K, const int32_t* done_opt, int eos,
                         const int32_t* lengths_opt, double alpha, int32_t* parent, int32_t* token, float* score,
                         int32_t* done_out_opt, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (!logits || !scores || !parent || !token || !score) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (V < 1 || V > kBeamMaxVocab || N < 1 || N > kBeamMaxRows) return set_error(NT_ERR_INVALID_ARG, "need 1 <= V <= 2^24 and 1 <= N <= 65536");
  if (W < 1 || W > kBeamMax || N % W != 0 || K < 1 || K > kBeamMax)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= W, K <= 64 and N a multiple of W");
  if (eos < -1 || eos >= V || (done_opt && eos < 0)) return set_error(NT_ERR_INVALID_ARG, "need -1 <= eos < V, and a token with done");
  if (!std::isfinite(alpha) || alpha < 0.0 || alpha > 4.0 || (alpha != 0.0 && !lengths_opt))
    return set_error(NT_ERR_INVALID_ARG, "need 0 <= alpha <= 4, and lengths where it is not 0");
  if (!aligned(logits, 4) || !aligned(scores, 4) || (done_opt && !aligned(done_opt, 4)) || (lengths_opt && !aligned(lengths_opt, 4)) ||
      !aligned(parent, 4) || !aligned(token, 4) || !aligned(score, 4) || (done_out_opt && !aligned(done_out_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "arrays must be 4-byte aligned");
  if (!ws || !aligned(ws, 16) || ws_bytes < beam_ws_bytes(V, N))
    return set_error(NT_ERR_WORKSPACE, "workspace NULL, misaligned or smaller than nt_beam_select_workspace_size");
  const size_t in = (size_t)N * 4, chosen = (size_t)(N / W) * K * 4;
  for (const void* o : {(const void*)parent, (const void*)token, (const void*)score, (const void*)done_out_opt})
    if (o && (overlap(o, chosen, scores, in) || (done_opt && overlap(o, chosen, done_opt, in)) || (lengths_opt && overlap(o, chosen, lengths_opt, in)) ||
              overlap(o, chosen, logits, in * V)))
      return set_error(NT_ERR_INVALID_ARG, "outputs must not overlap inputs");
  NT_TRY(check_device());
  BeamArgs a{};
  a.logits = logits;
  a.scores = scores;
  a.done = done_opt;
  a.lens = lengths_opt;
  a.parent = parent;
  a.token = token;
  a.score = score;
  a.done_out = done_out_opt;
  a.N = N;
  a.V = V;
  a.W = W;
  a.K = K;
  a.chunk = chunk_of(V);
  a.nchunks = chunks_of(V);
  a.scale = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + kWsHeaderBytes);
  a.chunks = reinterpret_cast<float2*>(a.scale + N);
  a.eos = eos;
  a.alpha = alpha;
  a.wide = V % 4 == 0 && aligned(logits, 16);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t jobs = (int64_t)N * a.nchunks;
  const int64_t ctas = std::max<int64_t>((jobs + kScanThreads / 32 - 1) / (kScanThreads / 32), (N + 31) / 32);
  NT_CUDA_TRY(launch_kernel(beam_scan_kernel, dim3((unsigned)ctas), dim3(kScanThreads), 0, st, true, a, jobs));
  NT_TRY(check_launch("beam_scan_kernel"));
  static std::atomic<int> allowed[64];
  const int smem = W * a.nchunks * (int)sizeof(float);
  if (smem > 16 * 1024) NT_TRY(allow_smem(beam_pick_kernel, kBeamMax * kChunksMax * (int)sizeof(float), allowed));
  NT_CUDA_TRY(launch_kernel(beam_pick_kernel, dim3((unsigned)(N / W)), dim3(kPickThreads), smem, st, true, a));
  return check_launch("beam_pick_kernel");
}

}  // extern "C"
