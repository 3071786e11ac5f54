// nt_tree_attn.cuh -- what the two kernels of the tree attention share: arguments, barriers, TMA, tcgen05
// and the cutting of fp32 values into bf16 terms.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "nt_tree.cuh"
#include "nt_tree_plan.cuh"

namespace nt {

struct TaArgs {
  const void* q;            // [B][Hq][D]
  void* out;                // [B][Hq][D]
  const uint32_t* mask;     // [B][words]
  const uint16_t* vtree;    // the tree's first value row of head 0
  int64_t head_stride;      // elements between heads of a cache
  float* part;              // [slots][rows][D] weighted sums of a split
  float2* ml;               // [slots][rows] (m, sum)
  unsigned int* err;        // the workspace's status header [code, CTA]
  uint64_t timeout_ns;
  int fault;
  int B, Hq, G, R, words;   // R = B * G rows per key-value head
  int prefix, pre_tiles, tiles;  // 64-key tiles of the sequence, and with the tree's
  int nsplit, mtiles;       // splits of a tile of rows (0: every CTA an equal share of all tiles), tiles of rows per head
  int groups, ctas;         // tiles of rows of all heads; CTAs of the first kernel
  int cluster;              // few rows: whether a cluster holds the splits of a head
  float scale_log2;         // log2(e) / sqrt(D)
  float inv_g;              // 1 / G
};
struct TaMaps {
  CUtensorMap kp, vp, kt, vt;  // sequence and tree rows of keys and values
};

namespace {

// Warps: the issuers come first, as the scheduler prefers older warps and each of them holds up all others.
constexpr int kTaKeyLoad = 0, kTaScore = 1, kTaValue = 2, kTaValueLoad = 3, kTaFirstSoftmax = 4;
constexpr int kTaSoftmax = 256;         // two groups of 128 threads = tensor-memory lanes (rows)
constexpr int kTaThreads = 32 * kTaFirstSoftmax + kTaSoftmax;
constexpr int kTaTmemCols = 512;
constexpr int kTaFirst = 3;             // ring slots filled before the queries have arrived
constexpr float kTaLazy = 8.0f;         // a maximum is raised once a score exceeds it by 2^8
constexpr uint64_t kTaTimeoutNs = 2000000000ull;
constexpr unsigned int kTaErrWait = 18;  // status code of a wait that ran out

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait; false after the timeout or once another role of the CTA has given up. The clock
// is first read after 256 polls: reading it before the first one cost every short wait 300 cycles.
__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* fail, uint64_t timeout_ns) {
  uint64_t deadline = 0;
  for (uint32_t it = 1;; ++it) {
    if (bar_try(bar, parity)) return true;
    if ((it & 255u) != 0u) continue;
    const uint64_t now = globaltimer_ns();
    if (deadline == 0) deadline = now + timeout_ns;
    if (*fail || now > deadline) {
      *fail = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* fail, uint64_t timeout_ns) {
  return bar_try(bar, parity) || bar_wait_slow(bar, parity, fail, timeout_ns);
}
// One arrival for a warp (32 separate ones, times eight warps, held a tile up by 350 cycles).
__device__ __forceinline__ void bar_arrive_warp(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) bar_arrive(bar);
}
// The same for a whole warp: every lane gets one answer, so the warp stays together.
__device__ __forceinline__ bool bar_wait_warp(uint32_t bar, uint32_t parity, volatile int* fail, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, fail, timeout_ns));
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Shared-memory operand with the 128-byte swizzle, as the TMA boxes of 64 elements x 64 rows
// write it: 8-row groups 1,024 bytes apart. K-major for the keys (rows = keys, 64 dimensions of
// the reduction in a row); for the values rows are the reduction and the second 64 dimensions
// stand `lead` bytes on.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lead) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lead >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version (sm_100)
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}
// kind::f16, A = B = bf16, D = fp32, M = 128, N = n; B K-major, or with the reduction along rows; A's sign turned.
__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool b_rows, bool minus_a = false) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (minus_a ? 1u << 13 : 0u) | (b_rows ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One lane of a converged warp, the same one every time: code under it stays uniform for the
// compiler, which feeds the MMAs from uniform registers (measured: 29 cycles to issue a 128 x 64 x 16
// MMA instead of 45 under `lane == 0`; its execution takes 32).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_smem_a(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Tensor memory, by one whole warp; its address goes to shared memory.
__device__ __forceinline__ void tm_alloc(uint32_t slot, int cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_free(uint32_t tmem, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// Columns of this lane. The wait stands in the same statement as the load: registers of a load on
// its way must not be moved or spilled.
__device__ __forceinline__ void tm_ld16(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16]; tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32]; tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tm_load(uint32_t addr, float (&r)[N]) {
  if constexpr (N == 16) {
    tm_ld16(addr, r);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 32) tm_ld32(addr + i, r + i);
  }
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <int N>
__device__ __forceinline__ void tm_store(uint32_t addr, const uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) tm_st8(addr + i, r + i);
}
__device__ __forceinline__ void tm_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {  // 2^x (2^-inf = +0)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_rn(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Tiles are decided on in order, quarter of the lanes by quarter: the group that has decided on a
// tile lets the other one, which has the next tile, go on.
__device__ __forceinline__ void turn_wait(int quarter, int group) {
  asm volatile("bar.sync %0, 64;" ::"r"(1 + 2 * quarter + group) : "memory");
}
__device__ __forceinline__ void turn_pass(int quarter, int group) {
  asm volatile("bar.arrive %0, 64;" ::"r"(1 + 2 * quarter + (group ^ 1)) : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
// The bf16 pair in w less two values: w.lo - x, w.hi - y, each one rounding (here exact).
__device__ __forceinline__ float2 less2(uint32_t w, float x, float y) {
  float2 r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n sub.f32.bf16 %0, l, %3;\n sub.f32.bf16 %1, h, %4;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "r"(w), "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two values as pairs of bf16 terms, term t of both in w[t], the second one with its sign turned: with
// three terms the leading 8, next 8 and last 8 bits of the significand, cut off one after the other, so
// nothing is lost (a value below 2^-110 aside); with two, each the rest so far, rounded. (With masks and
// fp32 differences in place of less2, the half-rate logic operations bound the softmax.)
template <int N>
__device__ __forceinline__ void split(float x, float y, uint32_t (&w)[N]) {
  if constexpr (N == 3) {
    w[0] = prmt(__float_as_uint(x), __float_as_uint(y), 0x7632u);
    const float2 r = less2(w[0], x, y);  // - the rest
    w[1] = prmt(__float_as_uint(r.x), __float_as_uint(r.y), 0x7632u);
    const float2 q = less2(w[1], r.x, r.y);  // the rest's rest
    w[2] = prmt(__float_as_uint(q.x), __float_as_uint(q.y), 0x7632u);
  } else {
    static_assert(N == 2, "terms");
    w[0] = pack_rn(x, y);
    const float2 r = less2(w[0], x, y);
    w[1] = pack_rn(r.x, r.y);
  }
}
// Whether a word holds a bf16 that is not finite.
__device__ __forceinline__ bool word_bad(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Node of a row, row / G: exact for rows up to 2^20 (half a row is more than the product's error).
__device__ __forceinline__ int node_of(int row, float inv_g) { return (int)(((float)row + 0.5f) * inv_g); }

}  // namespace

// Before a call with up to kTaFewNodes nodes or kTaFewRows rows is planned. *clusters: how many run at a time.
nt_status set_up_tree_few(int R, int dtype, int D, int* clusters);
nt_status launch_tree_few(const TaMaps& maps, const TaArgs& a, int dtype, int D, cudaStream_t st);

}  // namespace nt
