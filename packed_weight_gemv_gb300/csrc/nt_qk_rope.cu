// nt_qk_rope.cu -- norms of queries and keys per head, the rotary embedding and the append to
// the key-value cache in one pass over the projections' rows.
//
// For a head x of D dimensions at position p:  y = x * r * gamma, r = 1 / sqrt(mean(x^2) + eps);
// then each pair (a, b) of the first rotary_dim dimensions becomes (a c - b s, b c + a s) with
// (c, s) = amplitude * (cos, sin)(p * inv_freq[i]); the other dimensions pass through.
//
// Every value is read once and written once (queries to q_out, keys and values rounded to bf16
// into the cache), so the kernel is bound by memory for many tokens and by the launch for few:
// 8,191 tokens of 32 + 8 heads of 128 (fp32, 369 MB) take 60.5 us = 6.1 TB/s, 90 % of the measured
// copy rate (64.6 without the elements asked for a pass ahead); one such token 2.1 us and 64 of them in
// bf16 2.5 us in a replayed graph.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "nt_kernels.cuh"

namespace nt {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;

struct RopeArgs {
  const void *q, *k, *v;  // [B][H][D], tokens q_stride / k_stride / v_stride elements apart
  int64_t q_stride, k_stride, v_stride;
  const float *q_gamma, *k_gamma;  // [D] or null (no norm)
  float eps;
  int B, Hq, Hkv, D;
  const double* inv_freq;  // [rd / 2] radians per position
  int rd;
  float amplitude;
  const int32_t* pos;  // [B] or null: pos0 + b
  int pos0;
  const int32_t* rows;  // [B] or null: row0 + b
  int row0;
  void* q_out;  // [B][Hq][D]
  uint16_t *kc, *vc;  // [Hkv][ts][D]
  int ts;
  uint32_t* n_bad;
};

// Four neighbouring elements as they are in memory.
template <typename T>
using Raw4 = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
template <typename T>
__device__ __forceinline__ Raw4<T> raw4(const T* p) {
  return *reinterpret_cast<const Raw4<T>*>(p);
}
template <typename V>
__device__ __forceinline__ void unpack4(V v, float (&x)[4]) {
  if constexpr (sizeof(V) == 16) {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {  // bf16 is the upper half of an fp32
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
}

// Sine and cosine of p * f without a wide range reduction: f / 2 pi as a 64-bit binary fraction
// of a turn (one fp64 product per pair and CTA), times the integer position modulo one turn --
// the wrap of the 64-bit product is the reduction, and the error is |p| * 2^-64 turns next to
// the rounding of f itself. The top 32 bits as a signed number are half-turns for sincospif.
__device__ __forceinline__ void turn_sincos(double f, int pos, float* s, float* c) {
  double t = f * 0.15915494309189535;  // 1 / (2 pi)
  t -= floor(t);
  const unsigned long long frac = __double2ull_rz(t * 18446744073709551616.0);  // 2^64
  const unsigned long long turn = frac * (unsigned long long)(long long)pos;
  sincospif((float)(int)(turn >> 32) * 4.6566128730773926e-10f, s, c);  // 2^-31: half-turns in [-1, 1)
}

// CTA: token blockIdx.x and the heads of slice blockIdx.y; LPH lanes share a head, each with 8
// of its elements: unit u < rd / 8 holds pairs 4u .. 4u + 3, the units after them 8 dimensions
// that pass through.
template <typename T, bool kHalf, int LPH>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeArgs a) {
  __shared__ float cs[2][kRopeMaxD / 2];
  dependent_launch_wait();
  constexpr int kHeads = kRopeThreads / LPH;
  const int b = blockIdx.x, i = threadIdx.x, u = i % LPH;
  const int pos = a.pos ? a.pos[b] : a.pos0 + b;
  const int row = a.rows ? a.rows[b] : a.row0 + b;
  const bool rot = u < a.rd / 8, live = u < a.D / 8;
  // the unit's two groups of four elements
  const int e0 = rot && kHalf ? 4 * u : 8 * u, e1 = rot && kHalf ? a.rd / 2 + 4 * u : 8 * u + 4;
  const int heads = a.Hq + 2 * a.Hkv;
  // A pass's elements are asked for a pass ahead, the first one's before the angles are formed.
  Raw4<T> next0{}, next1{};
  auto fetch = [&](int h0) {
    const int h = h0 + i / LPH;
    if (!live || h >= heads) return;
    const bool isq = h < a.Hq, isv = h >= a.Hq + a.Hkv;
    const int g = isq ? h : isv ? h - a.Hq - a.Hkv : h - a.Hq;
    const T* x = static_cast<const T*>(isq ? a.q : isv ? a.v : a.k) +
                 (int64_t)b * (isq ? a.q_stride : isv ? a.v_stride : a.k_stride) + (int64_t)g * a.D;
    next0 = raw4(x + e0);
    next1 = raw4(x + e1);
  };
  fetch(blockIdx.y * kHeads);
  for (int p = i; p < a.rd / 2; p += kRopeThreads) {
    float s, c;
    turn_sincos(a.inv_freq[p], pos, &s, &c);
    cs[0][p] = c * a.amplitude;
    cs[1][p] = s * a.amplitude;
  }
  __syncthreads();
  const bool row_ok = row >= 0 && row < a.ts;
  if (!row_ok && a.n_bad && blockIdx.y == 0 && i == 0) atomicAdd(a.n_bad, 1u);
  for (int h0 = blockIdx.y * kHeads; h0 < heads; h0 += gridDim.y * kHeads) {
    const int h = h0 + i / LPH;
    const bool isq = h < a.Hq, isv = h >= a.Hq + a.Hkv, on = live && h < heads;
    const int g = isq ? h : isv ? h - a.Hq - a.Hkv : h - a.Hq;
    float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) {
      unpack4(next0, x0);
      unpack4(next1, x1);
    }
    fetch(h0 + gridDim.y * kHeads);
    const float* gamma = isq ? a.q_gamma : a.k_gamma;
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!on) continue;
    if (!isv) {
      if (gamma) {
        const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
        float g0[4], g1[4];
        unpack4(raw4(gamma + e0), g0);
        unpack4(raw4(gamma + e1), g1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x0[e] = x0[e] * r * g0[e];
          x1[e] = x1[e] * r * g1[e];
        }
      }
      if (rot) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float c = cs[0][4 * u + e], s = cs[1][4 * u + e];
          if (kHalf) {
            const float lo = x0[e], hi = x1[e];
            x0[e] = fmaf(lo, c, -hi * s);
            x1[e] = fmaf(hi, c, lo * s);
          } else {  // elements 2e, 2e + 1 of the unit's eight are pair 4u + e
            float& lo = e < 2 ? x0[2 * e & 3] : x1[2 * e & 3];
            float& hi = e < 2 ? x0[(2 * e & 3) + 1] : x1[(2 * e & 3) + 1];
            const float l = lo, m = hi;
            lo = fmaf(l, c, -m * s);
            hi = fmaf(m, c, l * s);
          }
        }
      }
    }
    if (isq) {
      using TO = typename std::conditional<sizeof(T) == 4, float, uint16_t>::type;
      TO* y = static_cast<TO*>(a.q_out) + ((int64_t)b * a.Hq + g) * a.D;
      store4(y + e0, x0);
      store4(y + e1, x1);
    } else if (row_ok) {
      uint16_t* y = (isv ? a.vc : a.kc) + ((int64_t)g * a.ts + row) * a.D;
      store4(y + e0, x0);
      store4(y + e1, x1);
    }
  }
}

// inv_freq[i] of a context scaling (see nt.h), in double.
__global__ void rope_frequencies_kernel(int pairs, double base, int scaling, double factor, double trained,
                                        double slow, double fast, double* __restrict__ out) {
  const int i = threadIdx.x;
  if (i >= pairs) return;
  double f = pow(base, -(double)i / pairs);
  if (scaling == NT_ROPE_LINEAR) f /= factor;
  if (scaling == NT_ROPE_WAVELENGTH) {
    const double turns = trained * f * 0.15915494309189535;
    const double w = fmin(fmax((turns - slow) / (fast - slow), 0.0), 1.0);
    f *= w + (1.0 - w) / factor;
  }
  out[i] = f;
}

template <typename T, bool kHalf>
nt_status launch_qk_rope(const RopeArgs& a, cudaStream_t st) {
  const int lph = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  const int per = kRopeThreads / lph, slices = (a.Hq + 2 * a.Hkv + per - 1) / per;
  // few tokens: a CTA per slice of heads; many: every CTA walks its token's heads
  const int want = std::max(1, 8 * device_sm_count() / a.B);
  const dim3 grid(a.B, std::min(slices, want));
  auto kern = lph == 8 ? qk_rope_kernel<T, kHalf, 8> : lph == 16 ? qk_rope_kernel<T, kHalf, 16> : qk_rope_kernel<T, kHalf, 32>;
  NT_CUDA_TRY(launch_kernel(kern, grid, dim3(kRopeThreads), 0, st, true, a));
  return check_launch("qk_rope_kernel");
}

}  // namespace
}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_rope_frequencies(int rotary_dim, double base, int scaling, double factor, int trained_len, double slow,
                              double fast, double* inv_freq, void* stream) {
  clear_error();
  if (!inv_freq) return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (rotary_dim < 8 || rotary_dim > kRopeMaxD || rotary_dim % 8 != 0 || !(base > 1.0) || !(base < 1e300))
    return set_error(NT_ERR_INVALID_ARG, "need rotary_dim a multiple of 8 in 8..256 and 1 < base < 1e300");
  if (scaling != NT_ROPE_PLAIN && scaling != NT_ROPE_LINEAR && scaling != NT_ROPE_WAVELENGTH)
    return set_error(NT_ERR_INVALID_ARG, "unknown scaling");
  if (scaling != NT_ROPE_PLAIN && !(factor > 0.0 && factor < 1e300))
    return set_error(NT_ERR_INVALID_ARG, "scaling needs a positive factor");
  if (scaling == NT_ROPE_WAVELENGTH && (trained_len < 1 || !(slow >= 0.0) || !(fast > slow) || !(fast < 1e300)))
    return set_error(NT_ERR_INVALID_ARG, "need trained_len >= 1 and 0 <= slow < fast");
  if (!aligned(inv_freq, 8)) return set_error(NT_ERR_ALIGNMENT, "inv_freq must be 8-byte aligned");
  NT_TRY(check_device());
  rope_frequencies_kernel<<<1, kRopeMaxD / 2, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      rotary_dim / 2, base, scaling, factor, trained_len, slow, fast, inv_freq);
  return check_launch("rope_frequencies_kernel");
}

nt_status nt_qk_norm_rope_append(const void* q, const void* k, const void* v, int dtype, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, const float* q_gamma_opt,
                                 const float* k_gamma_opt, float eps, int B, int Hq, int Hkv, int D,
                                 const double* inv_freq, int rotary_dim, int layout, float amplitude,
                                 const int32_t* pos_opt, int pos0, const int32_t* rows_opt, int row0, void* q_out,
                                 uint16_t* k_cache, uint16_t* v_cache, int t_stride, uint32_t* n_bad_opt,
                                 void* stream) {
  clear_error();
  if (!q || !k || !v || !q_out || !k_cache || !v_cache || (rotary_dim > 0 && !inv_freq))
    return set_error(NT_ERR_INVALID_ARG, "NULL pointer");
  if (dtype != NT_F32 && dtype != NT_BF16) return set_error(NT_ERR_INVALID_ARG, "dtype must be NT_F32 or NT_BF16");
  if (layout != NT_ROPE_HALF && layout != NT_ROPE_INTERLEAVED)
    return set_error(NT_ERR_INVALID_ARG, "layout must be NT_ROPE_HALF or NT_ROPE_INTERLEAVED");
  if (D < 8 || D > kRopeMaxD || D % 8 != 0) return set_error(NT_ERR_UNSUPPORTED, "head dimension must be a multiple of 8 up to 256");
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 8 != 0)
    return set_error(NT_ERR_INVALID_ARG, "rotary_dim must be a multiple of 8 in 0..D");
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq > 65535 || Hkv > 65535 || t_stride < 1 || !(eps >= 0.0f))
    return set_error(NT_ERR_INVALID_ARG, "need B, Hq, Hkv, t_stride >= 1 (heads up to 65535) and eps >= 0");
  if (!pos_opt && (int64_t)pos0 + B - 1 > INT32_MAX) return set_error(NT_ERR_INVALID_ARG, "positions leave the int range");
  if (!rows_opt && (row0 < 0 || (int64_t)row0 + B > t_stride))
    return set_error(NT_ERR_INVALID_ARG, "need 0 <= row0 and row0 + B <= t_stride");
  if (q_stride % 4 || k_stride % 4 || v_stride % 4)
    return set_error(NT_ERR_ALIGNMENT, "token strides must be multiples of 4 elements");
  if (B > 1 && (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D))
    return set_error(NT_ERR_INVALID_ARG, "token strides must be at least the heads' elements");
  const uintptr_t in_align = dtype == NT_F32 ? 16 : 8;
  if (!aligned(q, in_align) || !aligned(k, in_align) || !aligned(v, in_align) || !aligned(q_out, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return set_error(NT_ERR_ALIGNMENT, "q, k, v, q_out and the caches must be 16-byte aligned (bf16 inputs: 8)");
  if ((q_gamma_opt && !aligned(q_gamma_opt, 16)) || (k_gamma_opt && !aligned(k_gamma_opt, 16)) ||
      (inv_freq && !aligned(inv_freq, 8)) || (pos_opt && !aligned(pos_opt, 4)) || (rows_opt && !aligned(rows_opt, 4)) ||
      (n_bad_opt && !aligned(n_bad_opt, 4)))
    return set_error(NT_ERR_ALIGNMENT, "gammas must be 16-byte, inv_freq 8-byte, int32 arrays 4-byte aligned");
  NT_TRY(check_device());
  const RopeArgs a{q, k, v, q_stride, k_stride, v_stride, q_gamma_opt, k_gamma_opt, eps, B, Hq, Hkv, D, inv_freq,
                   rotary_dim, amplitude, pos_opt, pos0, rows_opt, row0, q_out, k_cache, v_cache, t_stride, n_bad_opt};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == NT_F32)
    return layout == NT_ROPE_HALF ? launch_qk_rope<float, true>(a, st) : launch_qk_rope<float, false>(a, st);
  return layout == NT_ROPE_HALF ? launch_qk_rope<uint16_t, true>(a, st) : launch_qk_rope<uint16_t, false>(a, st);
}

}  // extern "C"
