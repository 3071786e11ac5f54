// nt_tree.cu -- the bookkeeping of a drafted token tree: ancestor bits and positions from the
// nodes' parents, acceptance of the longest drafted path that agrees with the model ("The
// Neutrino Engine", § "The 0.6B model does not get to decide", with a tree of drafts in place
// of one chain), and the move of the accepted rows behind the sequence's in every layer's cache.
// All three are small; their time is the launch and a few dependent steps: in a replayed graph
// acceptance takes 1.5 us for a chain of 8 and 1.9 for 256 nodes, the move of 5 rows in 36 layers 2.0
// and of 20 rows 3.3 (5.9 MB read and written).
#include <algorithm>

#include "nt_tree.cuh"

namespace nt {
namespace {

constexpr int kTreeWords = kTreeMaxNodes / 32;
constexpr int kCommitLayers = 128;

// One CTA, thread = node. Pointer jumping: after k rounds a node's bits cover its 2^k nearest
// ancestors (itself among them) and `up` is the one after those, so 8 rounds do for 256 nodes.
__global__ void __launch_bounds__(kTreeMaxNodes) tree_layout_kernel(const int32_t* parent, int B, int pos0, uint32_t* mask,
                                                                    int words, int32_t* pos, uint32_t* n_bad) {
  __shared__ uint32_t bits[kTreeMaxNodes][kTreeWords + 1];  // one word of padding against bank conflicts
  __shared__ int up[kTreeMaxNodes];
  dependent_launch_wait();
  const int b = threadIdx.x;
  uint32_t m[kTreeWords];
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w) bits[b][w] = m[w] = b >> 5 == w ? 1u << (b & 31) : 0u;
  int p = b < B ? parent[b] : -1;
  if (p >= b) {  // not a parent: the node stands as a root of its own
    if (n_bad) atomicAdd(n_bad, 1u);
    p = -1;
  }
  if (p < 0) p = -1;
  up[b] = p;
  __syncthreads();
  for (int span = 1; span < B; span *= 2) {
    int next = -1;
    if (p >= 0) {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w) m[w] |= bits[p][w];
      next = up[p];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) bits[b][w] = m[w];
    up[b] = p = next;
    __syncthreads();
  }
  if (b >= B) return;
  int depth = -1;
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w) {
    depth += __popc(m[w]);
    if (w < words) mask[(int64_t)b * words + w] = m[w];
  }
  for (int w = kTreeWords; w < words; ++w) mask[(int64_t)b * words + w] = 0u;
  if (pos) pos[b] = pos0 + depth;
}

// One CTA, thread = node. A node follows its parent when its token is the model's choice there
// (the lowest such child); the accepted path is the chain of those links from the root.
__global__ void __launch_bounds__(kTreeMaxNodes) tree_accept_kernel(const int32_t* parent, const int32_t* token,
                                                                    const int32_t* choice, int B, int32_t* emit,
                                                                    int32_t* path, int32_t* n_emit) {
  __shared__ int next[kTreeMaxNodes], way[kTreeMaxNodes];
  __shared__ int n_way;
  dependent_launch_wait();
  const int i = threadIdx.x;
  next[i] = kTreeMaxNodes;
  const int p = i < B ? parent[i] : -1, t = i < B ? token[i] : 0;
  __syncthreads();
  if (p >= 0 && p < i && t == choice[p]) atomicMin(&next[p], i);
  __syncthreads();
  if (i == 0) {
    int n = 0;
    for (int cur = 0; cur < kTreeMaxNodes && n < B; cur = next[cur]) way[n++] = cur;
    n_way = n;
  }
  __syncthreads();
  const int n = n_way;
  if (i < B) {
    const int at = i < n ? way[i] : -1;
    path[i] = at;
    emit[i] = at >= 0 ? choice[at] : -1;
  }
  if (i == 0) *n_emit = n;
}

struct CommitArgs {
  uint16_t* kc[kCommitLayers];
  uint16_t* vc[kCommitLayers];
  const int32_t* path;
  const int32_t* n;
  int B, Hkv, D, ts, src0, dst0;
};

// One warp per (layer, keys or values, key-value head): rows src0 + path[i] to dst0 + i in
// order, four rows loaded before any of them is stored. path rises strictly, so path[i] >= i
// and, with dst0 <= src0, a store never reaches a row that a later load still needs.
__global__ void __launch_bounds__(128) tree_commit_kernel(const __grid_constant__ CommitArgs a, int64_t jobs) {
  dependent_launch_wait();
  const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (job >= jobs) return;
  const int lane = threadIdx.x & 31, h = (int)(job % a.Hkv), lv = (int)(job / a.Hkv);
  uint16_t* base = ((lv & 1) ? a.vc[lv >> 1] : a.kc[lv >> 1]) + (int64_t)h * a.ts * a.D;
  const int n = min(*a.n, a.B);
  const int vecs = a.D / 8;  // 16-byte pieces of a row: at most one per lane
  for (int i0 = 0; i0 < n; i0 += 4) {
    uint4 v[4];
    bool move[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k, at = i < n ? a.path[i] : -1;
      move[k] = at >= i && at < a.B && lane < vecs;
      if (move[k]) v[k] = reinterpret_cast<const uint4*>(base + (int64_t)(a.src0 + at) * a.D)[lane];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (move[k]) reinterpret_cast<uint4*>(base + (int64_t)(a.dst0 + i0 + k) * a.D)[lane] = v[k];
  }
}

}  // namespace
}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_tree_layout(const int32_t* parent, int B, int pos0, uint32_t* mask, int mask_words, int32_t* pos_opt,
                         uint32_t* n_bad_opt, void* stream) {
  clear_error();
  if (!parent || !mask) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (B < 1 || B > kTreeMaxNodes || mask_words < (B + 31) / 32)
    return set_error(NT_ERR_INVALID_ARG, "need 1 <= B <= 256 and mask_words >= ceil(B / 32)");
  if (pos_opt && (int64_t)pos0 + B - 1 > INT32_MAX) return set_error(NT_ERR_INVALID_ARG, "positions leave the int range");
  if (!aligned(parent, 4) || !aligned(mask, 4) || (pos_opt && !aligned(pos_opt, 4)) || (n_bad_opt && !aligned(n_bad_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  NT_TRY(check_device());
  NT_CUDA_TRY(launch_kernel(tree_layout_kernel, dim3(1), dim3(kTreeMaxNodes), 0, reinterpret_cast<cudaStream_t>(stream),
                            true, parent, B, pos0, mask, mask_words, pos_opt, n_bad_opt));
  return check_launch("tree_layout_kernel");
}

nt_status nt_tree_accept(const int32_t* parent, const int32_t* token, const int32_t* argmax, int B, int32_t* emit,
                         int32_t* path, int32_t* n_emit, void* stream) {
  clear_error();
  if (!parent || !token || !argmax || !emit || !path || !n_emit) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (B < 1 || B > kTreeMaxNodes) return set_error(NT_ERR_INVALID_ARG, "need 1 <= B <= 256");
  if (!aligned(parent, 4) || !aligned(token, 4) || !aligned(argmax, 4) || !aligned(emit, 4) || !aligned(path, 4) ||
      !aligned(n_emit, 4))
    return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  NT_TRY(check_device());
  NT_CUDA_TRY(launch_kernel(tree_accept_kernel, dim3(1), dim3(kTreeMaxNodes), 0, reinterpret_cast<cudaStream_t>(stream),
                            true, parent, token, argmax, B, emit, path, n_emit));
  return check_launch("tree_accept_kernel");
}

nt_status nt_tree_commit(uint16_t* const* k_caches, uint16_t* const* v_caches, int n_layers, int Hkv, int D, int t_stride,
                         const int32_t* path, const int32_t* n_emit, int B, int src_row0, int dst_row0, void* stream) {
  clear_error();
  if (!k_caches || !v_caches || !path || !n_emit) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (n_layers < 1 || Hkv < 1 || Hkv > 65535 || B < 1 || B > kTreeMaxNodes)
    return set_error(NT_ERR_INVALID_ARG, "need n_layers >= 1, 1 <= Hkv <= 65535 and 1 <= B <= 256");
  if (D < 8 || D > 256 || D % 8 != 0) return set_error(NT_ERR_UNSUPPORTED, "head dimension must be a multiple of 8 up to 256");
  if (dst_row0 < 0 || src_row0 < dst_row0 || (int64_t)src_row0 + B > t_stride)
    return set_error(NT_ERR_INVALID_ARG, "need 0 <= dst_row0 <= src_row0 and src_row0 + B <= t_stride");
  if (!aligned(path, 4) || !aligned(n_emit, 4)) return set_error(NT_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  for (int i = 0; i < n_layers; ++i) {
    if (!k_caches[i] || !v_caches[i]) return set_error(NT_ERR_INVALID_ARG, "NULL cache");
    if (!aligned(k_caches[i], 16) || !aligned(v_caches[i], 16)) return set_error(NT_ERR_ALIGNMENT, "caches must be 16-byte aligned");
  }
  NT_TRY(check_device());
  for (int l0 = 0; l0 < n_layers; l0 += kCommitLayers) {
    const int L = std::min(kCommitLayers, n_layers - l0);
    CommitArgs a{};
    std::copy(k_caches + l0, k_caches + l0 + L, a.kc);
    std::copy(v_caches + l0, v_caches + l0 + L, a.vc);
    a.path = path;
    a.n = n_emit;
    a.B = B;
    a.Hkv = Hkv;
    a.D = D;
    a.ts = t_stride;
    a.src0 = src_row0;
    a.dst0 = dst_row0;
    const int64_t jobs = (int64_t)L * 2 * Hkv;
    NT_CUDA_TRY(launch_kernel(tree_commit_kernel, dim3((unsigned)((jobs + 3) / 4)), dim3(128), 0,
                              reinterpret_cast<cudaStream_t>(stream), true, a, jobs));
  }
  return check_launch("tree_commit_kernel");
}

}  // extern "C"
