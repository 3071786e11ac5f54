// nt_logits_adjust.cu -- sampling adjustments of the logits of a batch of positions (penalties
// for repeated tokens, a bias, a grammar's allowed tokens) with the greedy choice, and the
// token counts that the penalties go by.
//
// Per value: x -> x / r or x * r by its sign, - f * count, - p where the token was used; + bias;
// -inf where it is not allowed. Every step is one fp32 rounding, in this order. A value is read
// once and written once; counts and bias rows are shared by the batch and come out of L2, so
// the kernel is bound by memory.
#include <math.h>

#include <algorithm>

#include "nt_tree.cuh"

namespace nt {
namespace {

constexpr int kAdjThreads = 256;
static_assert(kTreeMaxNodes <= kAdjThreads, "one thread per node");

// Workspace: the 16-byte status header, then per row the best (value, index) key and the
// counter of CTAs done with the row; both are zero between calls.
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
  const float* bias;
  int64_t bias_stride;
  const uint32_t* allowed;  // rows allowed_stride words apart
  int64_t allowed_stride;
  float* out;       // [B][V] or null
  int32_t* argmax;  // [B] or null
  AdjWs* ws;
  int per;  // values per CTA, a multiple of 4 * kAdjThreads
};

__device__ __forceinline__ float penalise(float x, int count, const AdjArgs& a) {
  if (count <= 0) return x;
  float y = x > 0.0f ? __fdiv_rn(x, a.rep) : __fmul_rn(x, a.rep);
  y = __fsub_rn(y, __fmul_rn(a.freq, __int2float_rn(count)));
  return __fsub_rn(y, a.pres);
}

// A key that orders values above -inf by (value, lower index first); 0 for the others.
__device__ __forceinline__ unsigned long long choice_key(float y, int v) {
  if (!(y > -INFINITY)) return 0ull;  // -inf and NaN are never chosen
  const uint32_t u = __float_as_uint(y + 0.0f);  // -0 as +0
  const uint32_t o = (u >> 31) ? ~u : u | 0x80000000u;
  return ((unsigned long long)o << 32) | (uint32_t)~v;
}

// CTA: values [blockIdx.x * per, + per) of row blockIdx.y.
template <int VEC>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const AdjArgs a) {
  __shared__ int path_tok[kTreeMaxNodes];  // tokens of the row's path inside this CTA's range
  __shared__ int n_path;
  __shared__ unsigned long long warp_best[kAdjThreads / 32];
  dependent_launch_wait();
  const int b = blockIdx.y, i = threadIdx.x;
  const int v0 = blockIdx.x * a.per, v1 = min(a.V, v0 + a.per);
  if (i == 0) n_path = 0;
  __syncthreads();
  if (a.tree_mask && i < a.B) {  // thread = node: a tree has at most kAdjThreads
    const uint32_t w = a.tree_mask[(int64_t)b * a.mask_words + (i >> 5)];
    const int t = a.tokens[i];
    if ((w >> (i & 31) & 1u) && t >= v0 && t < v1) path_tok[atomicAdd(&n_path, 1)] = t;
  }
  __syncthreads();
  const int np = n_path;
  const float* x = a.x + (int64_t)b * a.V;
  const int32_t* cnt = a.counts ? a.counts + b * a.counts_stride : nullptr;
  const float* bias = a.bias ? a.bias + b * a.bias_stride : nullptr;
  const uint32_t* allowed = a.allowed ? a.allowed + b * a.allowed_stride : nullptr;
  float* out = a.out ? a.out + (int64_t)b * a.V : nullptr;
  unsigned long long best = 0;
  for (int v = v0 + i * VEC; v < v1; v += kAdjThreads * VEC) {
    float y[VEC], bi[VEC];
    int c[VEC];
    if constexpr (VEC == 4) {
      const float4 t = __ldcs(reinterpret_cast<const float4*>(x + v));
      y[0] = t.x; y[1] = t.y; y[2] = t.z; y[3] = t.w;
      const int4 ct = cnt ? __ldg(reinterpret_cast<const int4*>(cnt + v)) : make_int4(0, 0, 0, 0);
      c[0] = ct.x; c[1] = ct.y; c[2] = ct.z; c[3] = ct.w;
      const float4 bt = bias ? __ldg(reinterpret_cast<const float4*>(bias + v)) : make_float4(0.f, 0.f, 0.f, 0.f);
      bi[0] = bt.x; bi[1] = bt.y; bi[2] = bt.z; bi[3] = bt.w;
    } else {
      y[0] = __ldcs(x + v);
      c[0] = cnt ? __ldg(cnt + v) : 0;
      bi[0] = bias ? __ldg(bias + v) : 0.0f;
    }
    const uint32_t w = allowed ? __ldg(allowed + (v >> 5)) >> (v & 31) : ~0u;
    for (int k = 0; k < np; ++k) {
      const int t = path_tok[k];
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] += t == v + e;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      y[e] = penalise(y[e], c[e], a);
      if (bias) y[e] = __fadd_rn(y[e], bi[e]);
      if (!(w >> e & 1u)) y[e] = -INFINITY;
      const unsigned long long key = choice_key(y[e], v + e);
      best = key > best ? key : best;
    }
    if (out) {
      if constexpr (VEC == 4) __stcs(reinterpret_cast<float4*>(out + v), make_float4(y[0], y[1], y[2], y[3]));
      else __stcs(out + v, y[0]);
    }
  }
  if (!a.argmax) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
    best = other > best ? other : best;
  }
  if ((i & 31) == 0) warp_best[i >> 5] = best;
  __syncthreads();
  if (i == 0) {
#pragma unroll
    for (int k = 1; k < kAdjThreads / 32; ++k) best = warp_best[k] > best ? warp_best[k] : best;
    AdjWs::Row& r = a.ws->row[b];
    if (gridDim.x > 1) {
      atomicMax(&r.best, best);
      __threadfence();
      if (atomicAdd(&r.done, 1u) != gridDim.x - 1) return;
      __threadfence();
      best = atomicExch(&r.best, 0ull);  // the row's last CTA; back to zero for the next call
      r.done = 0u;
    }
    a.argmax[b] = best ? (int32_t)~(uint32_t)best : -1;
  }
}

__global__ void __launch_bounds__(kAdjThreads) count_kernel(const int32_t* __restrict__ tokens,
                                                            const int32_t* __restrict__ index, int n,
                                                            const int32_t* __restrict__ n_dev, int V,
                                                            int32_t* __restrict__ counts, uint32_t* n_bad) {
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
            presence, bias_opt, bias_stride, allowed_opt, allowed_stride, out_opt, argmax_opt, static_cast<AdjWs*>(ws),
            4 * kAdjThreads};
  const bool vec = V % 4 == 0 && aligned(logits, 16) && (!out_opt || aligned(out_opt, 16)) &&
                   (!counts_opt || (aligned(counts_opt, 16) && counts_stride % 4 == 0)) &&
                   (!bias_opt || (aligned(bias_opt, 16) && bias_stride % 4 == 0));
  auto kern = vec ? adjust_kernel<4> : adjust_kernel<1>;
  const dim3 grid((V + a.per - 1) / a.per, B);
  NT_CUDA_TRY(launch_kernel(kern, grid, dim3(kAdjThreads), 0, reinterpret_cast<cudaStream_t>(stream), true, a));
  return check_launch("adjust_kernel");
}

}  // extern "C"
