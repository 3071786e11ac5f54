// nt_tree_attention.cu -- attention of a drafted token tree over a bf16 key-value cache: every
// node sees the sequence's cached rows and the tree rows its mask names.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "nt_kernels.cuh"

namespace nt {
namespace {

struct TreeAttnArgs {
  const void* q;  // [B][Hq][D]
  const uint16_t *kc, *vc;  // [Hkv][ts][D] bf16
  const uint32_t* mask;     // [B][words]
  void* out;                // [B][Hq][D]
  int B, Hq, Hkv, prefix, row0, ts, words;
};

__device__ __forceinline__ float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// CTA of 4 warps per (head, node): each warp walks keys w, w + 4, ... with a running maximum.
template <typename T, int D>
__global__ void __launch_bounds__(128) tree_attn_kernel(const TreeAttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  dependent_launch_wait();
  const int h = blockIdx.x, b = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = h / (a.Hq / a.Hkv);
  auto elem = [](const T* p, int e) { return sizeof(T) == 4 ? (float)p[e] : bf16_f((uint16_t)p[e]); };
  const T* q = static_cast<const T*>(a.q) + ((int64_t)b * a.Hq + h) * D + lane * E;
  float x[E], o[E];
  for (int e = 0; e < E; ++e) {
    x[e] = elem(q, e);
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const float scale = 1.0f / sqrtf((float)D);
  const uint16_t* kh = a.kc + (int64_t)g * a.ts * D + lane * E;
  const uint16_t* vh = a.vc + (int64_t)g * a.ts * D + lane * E;
  for (int t = w; t < a.prefix + a.B; t += 4) {
    const int j = t - a.prefix;
    if (j >= 0 && !(a.mask[(int64_t)b * a.words + (j >> 5)] >> (j & 31) & 1u)) continue;
    const int64_t row = (int64_t)(j >= 0 ? a.row0 + j : t) * D;
    float s = 0.0f;
    for (int e = 0; e < E; ++e) s = fmaf(x[e], bf16_f(kh[row + e]), s);
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= scale;
    const float mn = fmaxf(m, s), c = m == -INFINITY ? 0.0f : expf(m - mn), p = mn == -INFINITY ? 0.0f : expf(s - mn);
    l = l * c + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * bf16_f(vh[row + e]);
    m = mn;
  }
  if (lane == 0) {
    sm[w] = m;
    sl[w] = l;
  }
  for (int e = 0; e < E; ++e) so[w][lane * E + e] = o[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY, L = 0.0f, O = 0.0f;
    for (int k = 0; k < 4; ++k) M = fmaxf(M, sm[k]);
    for (int k = 0; k < 4; ++k) {
      const float c = sm[k] == -INFINITY ? 0.0f : expf(sm[k] - M);
      L += sl[k] * c;
      O += so[k][threadIdx.x] * c;
    }
    const float y = L > 0.0f ? O / L : L == 0.0f ? 0.0f : NAN;
    const int64_t at = ((int64_t)b * a.Hq + h) * D + threadIdx.x;
    if (sizeof(T) == 4) static_cast<float*>(a.out)[at] = y;
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  }
}

size_t tree_attn_ws_bytes(int, int, int, int, int) { return sizeof(WsHeader); }

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
  *bytes = tree_attn_ws_bytes(B, Hq, Hkv, D, prefix);
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
  if (!ws || !aligned(ws, 16) || ws_bytes < tree_attn_ws_bytes(B, Hq, Hkv, D, prefix))
    return set_error(NT_ERR_WORKSPACE, "workspace NULL, misaligned or smaller than nt_tree_attention_workspace_size");
  NT_TRY(check_device());
  const TreeAttnArgs a{q, k_cache, v_cache, mask, out, B, Hq, Hkv, prefix, tree_row0, t_stride, mask_words};
  auto kern = dtype == NT_F32 ? (D == 64 ? tree_attn_kernel<float, 64> : tree_attn_kernel<float, 128>)
                              : (D == 64 ? tree_attn_kernel<uint16_t, 64> : tree_attn_kernel<uint16_t, 128>);
  NT_CUDA_TRY(launch_kernel(kern, dim3(Hq, B), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), true, a));
  return check_launch("tree_attn_kernel");
}

}  // extern "C"
