// nt_paged_attention.cu -- attention of ragged chunks of new tokens over a paged bf16 cache: the call.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <string>

#include "nt_paged.cuh"

namespace nt {
namespace {

nt_status check_paged(int T, int S, int Hq, int Hkv, int D) {
  if (D != 64 && D != 128) return set_error(NT_ERR_UNSUPPORTED, "head dimension must be 64 or 128");
  if (T < 1 || T > kPagedMaxTokens || S < 1 || S > kPageMaxSeqs) return set_error(NT_ERR_INVALID_ARG, "need 1 <= T <= 1048576 and 1 <= S <= 4096");
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > kPaMaxGroup || (int64_t)T * Hq > 1 << 24)
    return set_error(NT_ERR_INVALID_ARG, "need Hq a multiple of Hkv >= 1, Hq / Hkv <= 64 and T * Hq <= 2^24");
  return NT_OK;
}

std::mutex g_paged_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_paged_encode = nullptr;

}  // namespace

nt_status paged_map(CUtensorMap* map, const uint16_t* base, int D, int box_rows, const PaArgs& a) {
  {
    std::lock_guard<std::mutex> lock(g_paged_mu);
    if (!g_paged_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      NT_CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q));
      if (q != cudaDriverEntryPointSuccess || !fn) return set_error(NT_ERR_CUDA, "cuTensorMapEncodeTiled not available");
      g_paged_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
  }
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.ts, (cuuint64_t)a.Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.ts * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_paged_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, estr,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(NT_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")");
  return NT_OK;
}

}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_paged_attention_workspace_size(int T, int S, int Hq, int Hkv, int D, size_t* bytes) {
  clear_error();
  if (!bytes) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  NT_TRY(check_paged(T, S, Hq, Hkv, D));
  *bytes = paged_layout(T, Hq, Hkv, D).bytes;
  return NT_OK;
}

nt_status nt_paged_attention(const void* q, int dtype, int64_t q_stride, const uint16_t* k_pool, const uint16_t* v_pool, int T, int S,
                             int Hq, int Hkv, int D, int page, int t_stride, const int32_t* table, int width, const int32_t* q_start,
                             const int32_t* length, int max_new, int window, float cap, const float* slopes_opt, void* out,
                             uint32_t* n_bad_opt, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (!q || !k_pool || !v_pool || !table || !q_start || !length || !out) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (dtype != NT_F32 && dtype != NT_BF16) return set_error(NT_ERR_INVALID_ARG, "dtype must be NT_F32 or NT_BF16");
  NT_TRY(check_paged(T, S, Hq, Hkv, D));
  if (!page_ok(page)) return set_error(NT_ERR_INVALID_ARG, "page must be 16, 32, 64, 128 or 256 rows");
  if (t_stride < page || width < 1) return set_error(NT_ERR_INVALID_ARG, "need t_stride >= page and width >= 1");
  if (max_new < 0 || window < 0) return set_error(NT_ERR_INVALID_ARG, "need max_new, window >= 0");
  // (twice the cap and what scores are multiplied with have to be normal numbers)
  if (cap != 0.0f && !(cap >= 0x1p-100f && cap <= 0x1p100f)) return set_error(NT_ERR_INVALID_ARG, "cap must be 0 or 2^-100 .. 2^100");
  if (q_stride % 8 != 0) return set_error(NT_ERR_ALIGNMENT, "q_stride must be a multiple of 8");
  if (T > 1 && q_stride < (int64_t)Hq * D) return set_error(NT_ERR_INVALID_ARG, "need q_stride >= Hq * D");
  if (out == q && T > 1 && q_stride != (int64_t)Hq * D) return set_error(NT_ERR_INVALID_ARG, "out may be q where q is contiguous");
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16))
    return set_error(NT_ERR_ALIGNMENT, "q, out and the pools must be 16-byte aligned");
  if (!aligned(table, 4) || !aligned(q_start, 4) || !aligned(length, 4) || (slopes_opt && !aligned(slopes_opt, 4)) ||
      (n_bad_opt && !aligned(n_bad_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "int32 and fp32 arrays must be 4-byte aligned");
  const PaLayout at = paged_layout(T, Hq, Hkv, D);
  if (!ws || !aligned(ws, 16) || ws_bytes < at.bytes)
    return set_error(NT_ERR_WORKSPACE, "workspace NULL, misaligned or smaller than nt_paged_attention_workspace_size");
  NT_TRY(check_device());
  PaArgs a{};
  a.q = q;
  a.out = out;
  a.k = k_pool;
  a.v = v_pool;
  a.table = table;
  a.q_start = q_start;
  a.length = length;
  a.slopes = slopes_opt;
  a.n_bad = n_bad_opt;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.err = reinterpret_cast<unsigned int*>(w);
  a.join = reinterpret_cast<PaJoin*>(w + at.join);
  a.count = reinterpret_cast<unsigned int*>(w + at.count);
  a.part = reinterpret_cast<float*>(w + at.part);
  a.scratch = reinterpret_cast<float*>(w + at.scratch);
  a.ml = reinterpret_cast<float2*>(w + at.ml);
  a.timeout_ns = test_fault_timeout_ns(kPaTimeoutNs);
  a.fault = test_fault() == kFaultPaged;
  a.q_stride = q_stride;
  a.most = (int64_t)T * Hq + (int64_t)S * Hkv;
  a.which = kPaAll;
  a.T = T;
  a.S = S;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.width = width;
  a.page = page;
  a.shift = page_shift(page);
  a.n_pages = t_stride / page;
  a.ts = t_stride;
  a.window = window > 0 ? window : INT32_MAX;
  a.cap = cap;
  a.scale = (float)(1.0 / std::sqrt((double)D));
  const int64_t most = (int64_t)(max_new > 0 ? std::min(max_new, T) : T) * a.G;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (most <= kPaFewRows) return launch_paged_few(a, dtype, D, most, st);
  if (S == 1) return launch_paged_many(a, dtype, D, most, st);
  // Sequences of few rows are bound by memory, and on the tensor cores each would take a tile for itself.
  if (a.G <= kPaFewRows) {
    a.which = kPaFew;
    NT_TRY(launch_paged_few(a, dtype, D, a.G, st));  // a token's rows to a tile
    a.which = kPaMany;
  }
  return launch_paged_many(a, dtype, D, most, st);
}

}  // extern "C"
