// nt_paged_many.cu -- paged attention of chunks of new tokens on the tensor cores.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(x_j log2(e) - m)
//
// The query rows of a tile (128 rows: tokens x the G heads of a key-value head) are the M side of tcgen05.mma. 128 keys at a time
// are the N side of the scores S = Q K^T; the softmax turns S into weights P in the place of S in tensor memory, and P is the A operand of
// O += P V. Two groups of 128 threads (thread = row = tensor-memory lane) take turns, so that one's exponentials run under
// the other's products: each has a tile of rows of its own over the same keys (bf16 queries, more than 128 rows: 256 rows to a CTA), or both have
// the same rows and every other tile of keys, with sums of their own that are joined at the end (fp32 queries, whose three bf16 terms
// take the shared memory of three tiles; and up to 128 rows).
//
// CTA (384 threads): warps 0 and 2 ask for the pages of keys and values (TMA boxes of one page each, 128-byte swizzle) into a ring of tiles; one lane of
// warp 1 issues all MMAs, in the order S(1st), S(2nd), { O, next S } of the groups in turn, so the tensor pipe has one group's products
// while the other group's weights are formed, and a commit behind an S also tells that the O before it is done; warps 4-7 and 8-11 are
// the groups. S of the next tile goes where P of the last one stood: MMAs of one thread run in the order they are issued in.
//
// fp32 queries enter as three bf16 terms without loss. Weights enter as two rounded bf16 terms (2^-17), those of fp32 queries with D 64
// as three without loss. For bf16 queries one term would do with two products in place of three (ragged prompts of 8,000 tokens 626 us
// instead of 776, 257 among decoding sequences 93 instead of 94, 32 over 8,000 25.3 instead of 26.9), but its 2^-8 stands beside the
// output's own: 1.28 to 1.41 times the error of rounding the output alone, which is all that two terms leave, and a token would be less
// exact in a chunk than by itself. The tensor core cuts its fp32 sums off instead of rounding them, so O is taken off it every kFlush
// tiles of a group, into sums in the workspace that round to nearest.
//
// Bound by the tensor pipe, the more so the longer the keys: 2,049 bf16 tokens over 16,000, 32 / 8 heads of 128, take 549 us (three products for
// two, 1,560 TFLOP/s of them), ragged prompts of 8,000 tokens together 776 us (1,430), 511 fp32 tokens over 7,489 124
// us (127 cold; five products for two, 1,310 of them). Of the bf16 times keys and values from L2 alone would take four
// tenths, the exponentials six. What a call pays besides is about 25 us: 13 to the end of a first tile, 6 for the join of parts.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "nt_tree_attn.cuh"
#include "nt_paged.cuh"

namespace nt {
namespace {

constexpr int kPmKeys = 128;
constexpr int kPmKeyLoad = 0, kPmMma = 1, kPmValueLoad = 2, kPmFirstSoftmax = 4;
constexpr int kPmSoftmax = 256;  // two groups of 128 threads
constexpr int kPmThreads = 32 * kPmFirstSoftmax + kPmSoftmax;
constexpr int kPmNear = 1;
constexpr float kPmLazy = 32.0f;  // a reference is raised once a score exceeds it by 2^32: weights that large lose nothing in fp32 or bf16
constexpr int kPmSmem = 224 * 1024;
// Registers of a thread: launched with 168; the first four warps give some of theirs to the softmax (128 x 88 + 256 x 208 = 384 x 168).
constexpr int kPmRegsIssue = 88, kPmRegsSoftmax = 208;

struct PmMaps {
  CUtensorMap k, v;  // boxes of 64 dimensions x a page (at most 128 rows)
};

template <typename T, int D, bool kPair>
struct PmShape {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kTermsQ = kF32 ? 3 : 1, kTermsP = kF32 && D == 64 ? 3 : 2;
  static constexpr int kScoreCols = std::max(kPmKeys, kTermsP * kPmKeys / 2);  // of a group: its weights' terms stand in the place of its scores
  static constexpr int kRows = kPair ? 256 : 128;
  static constexpr int kSlot = kPmKeys * D * 2;
  static constexpr int kQTile = 128 * D * 2;  // one term of 128 rows
  static constexpr int kQBytes = kQTile * kTermsQ * (kPair ? 2 : 1);
  static constexpr int kStages = std::min(8, (kPmSmem - kQBytes) / kSlot);
  static constexpr int kAhead = kPair ? 1 : 2;  // tiles whose scores are formed before the first weights
  // What a piece's start and end cost in tiles. Measured, bf16 in pairs: ragged prompts 817 us with 4, 776 with 5, 780 with 6, 794 with 8, 808
  // with 10; a chunk among decoding sequences 91, 94, 95, 96, 99. fp32: 511 tokens over 7,489 123 us with 3, 127 with 6.
  static constexpr int kStart = kPair ? 5 : 3;
  static constexpr int kColO = 0, kColS = 2 * D;
  // A tile costs a sum at most 8 cuts of 2^-23 for every term of the weights: 2^-16 over 8 tiles (three terms: 4), 2^-13 over 64. (fp32, 511
  // tokens over 7,489. D 64: 81 us and 3.3e-6 off with two terms, 98 us and 1.7e-6 with three, as torch's own products in fp32. D 128: 124
  // us and 3.3e-6; every 4 tiles 135 and 2.7e-6, every 2 155 and 2.5e-6, as the two terms are left; a third has no place, 192 columns for P next
  // to S and O of two groups, but with tiles of 64 keys, whose scores read the queries' terms twice as often: 172 us and 1.9e-6.)
  static constexpr int kFlush = kF32 ? (kTermsP == 3 ? 4 : 8) : 64;
  static constexpr int kSmem = kQBytes + kStages * kSlot + 1024;
  static_assert(kStages >= 4, "ring");
  static_assert(kColS + 2 * kScoreCols <= kTaTmemCols, "tensor-memory columns");
  static_assert(kPageMaxSeqs * 4 <= kStages * kSlot, "the division's scratch stands in the ring");
};

// bar_wait in one piece: a call would fix the registers that setmaxnreg moves.
__device__ __forceinline__ bool pm_wait(uint32_t bar, uint32_t parity, volatile int* fail, uint64_t timeout_ns) {
  if (bar_try(bar, parity)) return true;
  uint64_t deadline = 0;
#pragma unroll 1
  for (uint32_t it = 1; !bar_try(bar, parity); ++it) {
    if ((it & 255u) != 0u) continue;
    const uint64_t now = globaltimer_ns();
    if (deadline == 0) deadline = now + timeout_ns;
    if (*fail || now > deadline) {
      *fail = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool pm_wait_warp(uint32_t bar, uint32_t parity, volatile int* fail, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, pm_wait(bar, parity, fail, timeout_ns));
}

// 128 columns of this lane: four loads under way together, and the wait.
__device__ __forceinline__ void tm_ld128(uint32_t addr, float (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31]),
        "=f"(r[32]), "=f"(r[33]), "=f"(r[34]), "=f"(r[35]), "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]),
        "=f"(r[40]), "=f"(r[41]), "=f"(r[42]), "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]),
        "=f"(r[48]), "=f"(r[49]), "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]),
        "=f"(r[56]), "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]), "=f"(r[63]),
        "=f"(r[64]), "=f"(r[65]), "=f"(r[66]), "=f"(r[67]), "=f"(r[68]), "=f"(r[69]), "=f"(r[70]), "=f"(r[71]),
        "=f"(r[72]), "=f"(r[73]), "=f"(r[74]), "=f"(r[75]), "=f"(r[76]), "=f"(r[77]), "=f"(r[78]), "=f"(r[79]),
        "=f"(r[80]), "=f"(r[81]), "=f"(r[82]), "=f"(r[83]), "=f"(r[84]), "=f"(r[85]), "=f"(r[86]), "=f"(r[87]),
        "=f"(r[88]), "=f"(r[89]), "=f"(r[90]), "=f"(r[91]), "=f"(r[92]), "=f"(r[93]), "=f"(r[94]), "=f"(r[95]),
        "=f"(r[96]), "=f"(r[97]), "=f"(r[98]), "=f"(r[99]), "=f"(r[100]), "=f"(r[101]), "=f"(r[102]), "=f"(r[103]),
        "=f"(r[104]), "=f"(r[105]), "=f"(r[106]), "=f"(r[107]), "=f"(r[108]), "=f"(r[109]), "=f"(r[110]), "=f"(r[111]),
        "=f"(r[112]), "=f"(r[113]), "=f"(r[114]), "=f"(r[115]), "=f"(r[116]), "=f"(r[117]), "=f"(r[118]), "=f"(r[119]),
        "=f"(r[120]), "=f"(r[121]), "=f"(r[122]), "=f"(r[123]), "=f"(r[124]), "=f"(r[125]), "=f"(r[126]), "=f"(r[127])
      : "r"(addr), "r"(addr + 32), "r"(addr + 64), "r"(addr + 96)
      : "memory");
}

template <typename T, int D, bool kPair, bool kExtra>
__global__ void __launch_bounds__(kPmThreads, 1) paged_many_kernel(const __grid_constant__ PmMaps maps, const __grid_constant__ PaArgs a) {
  using S = PmShape<T, D, kPair>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* q_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = q_smem + S::kQBytes;
  constexpr int kBars = 2 * S::kStages + 6;
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_fail, s_bad;
  volatile int* fail = &s_fail;
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S::kStages, sfull0 = empty0 + 8 * S::kStages, pfull0 = sfull0 + 16,
                 qfull = pfull0 + 16, drain = qfull + 8;
  if (i < kBars) {
    const int b = i - 2 * S::kStages;  // a group's four warps arrive at pfull, all eight at qfull
    bar_init(full0 + 8 * i, b == 2 || b == 3 ? 4 : b == 4 ? 8 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (i == 0) s_fail = s_bad = 0;
  if (warp == kPmMma) tm_alloc(smem_u32(&tmem_slot), kTaTmemCols);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = tmem_slot;
  dependent_launch_wait();
  PaWalk<kPmKeys, S::kStart> walk(a, pa_share<kPmThreads, kPmKeys, S::kStart>(a, S::kRows, kPmNear, reinterpret_cast<int*>(ring)), S::kRows);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before copies over the division's scratch
  __syncthreads();
  auto full = [&](int k) { return full0 + 8 * (k % S::kStages); };
  auto empty = [&](int k) { return empty0 + 8 * (k % S::kStages); };
  auto turn = [&](int k) { return (uint32_t)(k / S::kStages) & 1u; };
  auto slot = [&](int k) { return smem_u32(ring) + (k % S::kStages) * S::kSlot; };
  auto wait = [&](uint32_t bar, uint32_t parity) { return pm_wait(bar, parity, fail, a.timeout_ns); };
  // Ring order of a piece of n tiles: the keys of the first kAhead, then values j and keys j + kAhead in turn.
  auto ring_val = [&](int j, int n) { return min(S::kAhead, n) + j + min(j, max(n - S::kAhead, 0)); };
  auto ring_key = [&](int j) { return j < S::kAhead ? j : 2 * j - S::kAhead + 1; };
  int k0 = 0;  // tiles of the pieces before

  // (in every branch: code behind a join of the two would be held to the smaller number)
  auto give = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPmRegsIssue)); };
  if (warp == kPmKeyLoad || warp == kPmValueLoad) {
    give();
    const bool val = warp == kPmValueLoad;
    const CUtensorMap* map = val ? &maps.v : &maps.k;
    const int per = min(a.page, kPmKeys), boxes = kPmKeys / per;  // rows of a box; boxes of 64 dimensions of a tile
    const int box = lane % boxes, half = lane / boxes;
    const bool mine = half < D / 64;
    bool ok = a.fault == 0;
    int bad = 0, issued = -1;
    for (; walk.more() && ok; walk.next(a)) {
      const PaPiece p = walk.piece(a);
      // Whether any row sees a key of a box. (The first tile begins before the first key that is seen: pages that a window has left behind
      // may be gone.)
      auto there = [&](int key) { return key <= p.u.p1 && key + per - 1 >= p.u.lo; };
      const int32_t* ids = a.table + (int64_t)p.u.s * a.width;
      const int first = (p.u.tile0 + p.t0) * kPmKeys + box * per;
      // The page of this lane's box of tile j. Asked for three tiles before it is looked at: the loads would otherwise wait for it, a
      // round trip to L2 for every tile.
      auto ask = [&](int j) {
        const int key = first + j * kPmKeys;
        return j < p.n && there(key) ? ids[key >> a.shift] : -1;
      };
      constexpr int kAsk = 3;
      int id[kAsk];
#pragma unroll
      for (int j = 0; j < kAsk; ++j) id[j] = ask(j);
      for (int j = 0; ok && j < p.n; ++j) {
        const int key = first + j * kPmKeys, page = id[0];
        int y = a.ts;  // behind the pool (zeros) where nothing is seen, or nothing is there
        if (there(key)) {
          if ((unsigned)page < (unsigned)a.n_pages) y = (page << a.shift) + (key & (a.page - 1));
          else bad = 1;
        }
#pragma unroll
        for (int e = 0; e + 1 < kAsk; ++e) id[e] = id[e + 1];
        id[kAsk - 1] = ask(j + kAsk);
        const int k = k0 + (val ? ring_val(j, p.n) : ring_key(j));
        if (k >= S::kStages) ok = pm_wait_warp(empty(k), turn(k) ^ 1u, fail, a.timeout_ns);
        if (!ok) break;
        if (lane == 0) bar_expect_tx(full(k), S::kSlot);
        __syncwarp();
        if (mine) tma_3d(slot(k) + half * (kPmKeys * 128) + box * per * 128, map, half * 64, y, p.g, full(k));
        issued = k;
      }
      k0 += 2 * p.n;
    }
    if (!ok) {  // every copy must land before the CTA may exit
      const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
      // (the places of the last kStages that this warp has filled are among these; a wait for the other warp's ends as well)
      for (int k = max(0, issued - S::kStages + 1); k <= issued; ++k)
        while (!bar_try(full(k), turn(k)))
          if (globaltimer_ns() > deadline) break;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0 && bad && !val && a.n_bad) atomicAdd(a.n_bad, 1u);
  } else if (warp == kPmMma) {
    give();
    if (elect_one()) {
      bool ok = true;
      int piece = 0, steps[2] = {0, 0};  // steps of the groups so far
      for (; walk.more() && ok; ++piece) {
        PaPiece p = walk.piece(a);
        const int n = p.n;
        auto scores = [&](int x, int k) {
          const uint32_t d = tmem + S::kColS + x * S::kScoreCols;
          const uint64_t bd = sdesc(slot(k), 16);
          // the smallest terms first: the tensor core cuts its sums off, so a sum loses least while it is small
#pragma unroll
          for (int t = S::kTermsQ - 1; t >= 0; --t) {
            const uint64_t ad = sdesc(smem_u32(q_smem) + ((kPair ? x : 0) * S::kTermsQ + t) * S::kQTile, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t at = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16;
              mma_smem_a(d, ad + at, bd + at, idesc_bf16(kPmKeys, false), t < S::kTermsQ - 1 || kk > 0);
            }
          }
        };
        ok = wait(qfull, piece & 1);
        tm_fence_after();
        int c[2] = {0, 0};  // steps of the groups in this piece
        if constexpr (kPair) {
          ok = ok && wait(full(k0), turn(k0));
          tm_fence_after();
          if (ok) {
            scores(0, k0);
            mma_commit(sfull0);
            scores(1, k0);
            mma_commit(sfull0 + 8);
            mma_commit(empty(k0));
          }
        } else {
          for (int x = 0; x < 2 && x < n && ok; ++x) {
            ok = wait(full(k0 + x), turn(k0 + x));
            tm_fence_after();
            if (!ok) break;
            scores(x, k0 + x);
            mma_commit(sfull0 + 8 * x);
            mma_commit(empty(k0 + x));
          }
        }
        for (int s = 0; ok && s < (kPair ? 2 * n : n); ++s) {
          const int x = s & 1, j = kPair ? s >> 1 : s, kv = k0 + ring_val(j, n), next = j + S::kAhead, kk0 = k0 + ring_key(next);
          const bool first = !kPair || x == 0, last = !kPair || x == 1;
          if (first) ok = wait(full(kv), turn(kv));
          ok = ok && wait(pfull0 + 8 * x, steps[x] & 1);
          if (!ok) break;
          tm_fence_after();
          const uint64_t bd = sdesc(slot(kv), kPmKeys * 128);
          const bool fresh = c[x] % S::kFlush == 0;
#pragma unroll
          for (int t = S::kTermsP - 1; t >= 0; --t)
#pragma unroll
            for (int kk = 0; kk < kPmKeys / 16; ++kk)  // 16 keys: 2,048 bytes of each 64 dimensions
              mma_tmem_a(tmem + S::kColO + x * D, tmem + S::kColS + x * S::kScoreCols + t * (kPmKeys / 2) + 8 * kk, bd + kk * 2048 / 16,
                         idesc_bf16(D, true, t == 1), t < S::kTermsP - 1 || kk > 0 || !fresh);
          if (last) mma_commit(empty(kv));
          if (next < n) {
            if (first) ok = wait(full(kk0), turn(kk0));
            if (!ok) break;
            tm_fence_after();
            scores(x, kk0);
          }
          if (last && next < n) mma_commit(empty(kk0));
          mma_commit(sfull0 + 8 * x);  // the last word of a piece: nothing is under way behind it
          ++steps[x];
          ++c[x];
        }
        k0 += 2 * n;
        walk.next(a);
      }
      if (!ok) {
        mma_commit(drain);
        const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
        while (!bar_try(drain, 0))
          if (globaltimer_ns() > deadline) break;
      }
    }
    __syncwarp();
  } else if (warp < kPmFirstSoftmax) {
    give();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPmRegsSoftmax));
    const int quarter = warp & 3, x = (warp - kPmFirstSoftmax) >> 2, ln = quarter * 32 + lane;  // group, tensor-memory lane
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    float* scratch = a.scratch + ((int64_t)blockIdx.x * 2) * D * 128 + ln;  // [2][D][128]
    float4* s_stat = reinterpret_cast<float4*>(q_smem);  // [2][128], when the queries have been read
    const float inv_g = 1.0f / (float)a.G;
    constexpr int kChunk = 16;  // keys whose weights are formed together
    bool ok = true, left_part = false;
    uint32_t phase = 0;  // of sfull
    auto meet = [&] { asm volatile("bar.sync 9, %0;" ::"n"(kPmSoftmax) : "memory"); };
    // This thread's part of a piece's queries, asked for before the end of the piece before: 8 dimensions each of kLoads rows.
    constexpr int kLanes = D / 8, kAt = 32 / kLanes, kRowsMine = kPair ? 32 : 16, kLoads = kRowsMine / kAt, kVecs = S::kF32 ? 2 : 1;
    uint4 f[kLoads][kVecs];
    auto queries = [&](const PaPiece& p) {
      const int row0 = p.u.mt * S::kRows, first = row0 / a.G, rest = row0 - first * a.G;
      const int r0 = (kPair ? x * 128 : x * kRowsMine) + quarter * 32 + lane / kLanes;
      const T* q0 = static_cast<const T*>(a.q) + (int64_t)(p.u.t0 + first) * a.q_stride + (int64_t)(p.g * a.G + rest) * D + lane % kLanes * 8;
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        const int ru = r0 + e * kAt, away = node_of(rest + ru, inv_g);
        const T* q = q0 + (int64_t)away * a.q_stride + (ru - away * a.G) * D;
#pragma unroll
        for (int y = 0; y < kVecs; ++y) f[e][y] = ru < p.u.rows ? reinterpret_cast<const uint4*>(q)[y] : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    {
      PaPiece ahead{};
      if (walk.more()) ahead = walk.piece(a);
      queries(ahead);
    }
    for (; walk.more(); walk.next(a)) {
      const PaPiece p = walk.piece(a);
      const PaUnit& u = p.u;
      const int n = p.n;
      // Row r of the tile is token tok0 + token_of(r), head head0 + r - G token_of(r).
      const int row0 = u.mt * S::kRows, first = row0 / a.G, rest = row0 - first * a.G;
      const int tok0 = u.t0 + first, head0 = p.g * a.G + rest;
      auto token_of = [&](int r) { return node_of(rest + r, inv_g); };
      {  // the queries' terms into shared memory, rows of 64 dimensions with the 128-byte swizzle
        const int c = lane % kLanes, r0 = quarter * 32 + (kPair ? 0 : x * kRowsMine) + lane / kLanes;
        uint8_t* to = q_smem + (kPair ? x * S::kTermsQ * S::kQTile : 0) + (c >> 3) * (128 * 128);
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int r = r0 + e * kAt;
          uint4 w[S::kTermsQ];
          if constexpr (S::kF32) {
            uint32_t t0[3], t1[3], t2[3], t3[3];
            split(__uint_as_float(f[e][0].x), __uint_as_float(f[e][0].y), t0);
            split(__uint_as_float(f[e][0].z), __uint_as_float(f[e][0].w), t1);
            split(__uint_as_float(f[e][1].x), __uint_as_float(f[e][1].y), t2);
            split(__uint_as_float(f[e][1].z), __uint_as_float(f[e][1].w), t3);
#pragma unroll
            for (int t = 0; t < 3; ++t) {
              const uint32_t sign = t == 1 ? 0x80008000u : 0u;
              w[t] = make_uint4(t0[t] ^ sign, t1[t] ^ sign, t2[t] ^ sign, t3[t] ^ sign);
            }
          } else {
            w[0] = f[e][0];
          }
#pragma unroll
          for (int t = 0; t < S::kTermsQ; ++t) *reinterpret_cast<uint4*>(to + t * S::kQTile + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w[t];
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        bar_arrive_warp(qfull, lane);
      }
      const int ru = (kPair ? x * 128 : 0) + ln;           // row of the unit
      const bool live = ru < u.rows, idle = ru - lane >= u.rows;  // warps of rows past the last one only keep the barriers going
      const int rl = min(ru, u.rows - 1), tok = token_of(rl), h = head0 + rl - tok * a.G;
      const int pos = u.len - u.n + first + tok;
      const int lo = (int)max((int64_t)0, (int64_t)pos - a.window + 1);
      const int sure_lo = (int)max((int64_t)0, (int64_t)u.p1 - a.window + 1);  // every row sees from here to u.p0
      const float slope = kExtra && a.slopes ? a.slopes[h] : 0.0f;
      const int cnt = kPair ? n : (n + 1 - x) / 2;
      const int key_first = (u.tile0 + p.t0) * kPmKeys;
      auto partial = [&](int key) { return key + kPmKeys - 1 > u.p0 || key < sure_lo; };
      const uint32_t scol = tl + S::kColS + x * S::kScoreCols, ocol = tl + S::kColO + x * D;
      float m = -INFINITY, l = 0.0f, sums_m = -INFINITY;
      bool summed = false;
      for (int c = 0; c < cnt; ++c) {
        const int j = kPair ? c : 2 * c + x, key0 = key_first + j * kPmKeys;
        const bool fresh = c % S::kFlush == 0;
        if (fresh && c > 0) {  // O to the sums, which are in units of a reference of their own and asked for before the wait
          float* to = scratch + (int64_t)x * D * 128;
          float old[D];
          if (summed) {
#pragma unroll
            for (int d = 0; d < D; ++d) old[d] = to[d * 128];
          } else {
#pragma unroll
            for (int d = 0; d < D; ++d) old[d] = 0.0f;
          }
          ok = ok && pm_wait_warp(sfull0 + 8 * x, phase & 1, fail, a.timeout_ns);
          tm_fence_after();
          if (ok && !idle) {
            const float scale = sums_m == m ? 1.0f : ex2(sums_m - m);
#pragma unroll
            for (int d = 0; d < D; d += 16) {
              float o[16];
              tm_load(ocol + d, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) to[(d + e) * 128] = summed ? fmaf(old[d + e], scale, o[e]) : o[e];
            }
            sums_m = m;
            summed = true;
          }
        }
        ok = ok && pm_wait_warp(sfull0 + 8 * x, phase & 1, fail, a.timeout_ns);
        ++phase;
        tm_fence_after();
        const bool part = partial(key0);
        if (part) {  // values that are not finite are taken out: some row may not see them
          const int k = k0 + ring_val(j, n);
          ok = ok && pm_wait_warp(full(k), turn(k), fail, a.timeout_ns);
          uint4* at = reinterpret_cast<uint4*>(ring + (k % S::kStages) * S::kSlot) + ln;
          bool bad = false;
#pragma unroll 4
          for (int e = 0; e < S::kSlot / 16; e += 128) {
            const uint4 v = at[e];
            bad |= word_bad(v.x) || word_bad(v.y) || word_bad(v.z) || word_bad(v.w);
          }
          if (bad && ok) {
#pragma unroll 1
            for (int e = 0; e < S::kSlot / 16; e += 128) {
              uint16_t* w = reinterpret_cast<uint16_t*>(at + e);
              for (int y = 0; y < 8; ++y)
                if ((w[y] & 0x7f80u) == 0x7f80u) w[y] = 0;
            }
            s_bad = 1;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        if constexpr (kExtra) {
          // Cap and bias, from tensor memory and back: 32 keys at a time in a loop, as code for 128 in a row is fetched more slowly than
          // it runs (300 fp32 tokens over 4,000, capped: 73 us, 22 more in a row; bf16, 257 among decoding sequences: 2 us more).
          const float f = a.cap > 0.0f ? a.scale / a.cap : a.scale;
          if (ok && !idle) {
#pragma unroll 1
            for (int c = 0; c < kPmKeys; c += 32) {
              float r[32];
              tm_load(scol + c, r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] *= f;
              if (a.cap > 0.0f) {
                bool big = !S::kF32 && a.cap <= 256.0f;  // 2^-21 of it is nothing next to a bf16 output, and the series takes as long
#pragma unroll
                for (int e = 0; e < 32; ++e) big |= !(fabsf(r[e]) < kCapSmall);
                if (__any_sync(0xffffffffu, big)) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) {
                    const float t = cap_whole(r[e], a.cap);
                    r[e] = (S::kF32 || a.cap > 256.0f) && fabsf(r[e]) < kCapSmall ? cap_series(r[e], a.cap) : t;
                  }
                } else {
#pragma unroll
                  for (int e = 0; e < 32; ++e) r[e] = cap_series(r[e], a.cap);
                }
              }
              if (a.slopes) {
                const float away = (float)(pos - key0 - c);
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = fmaf(slope, (float)e - away, r[e]);
              }
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(r[e]);
              tm_store(scol + c, w);
            }
            tm_st_wait();
          }
        }
        float s[kPmKeys];
        if (ok && !idle) {
          tm_ld128(scol, s);
        } else {
#pragma unroll
          for (int e = 0; e < kPmKeys; ++e) s[e] = 0.0f;
        }
        if (part) {
          const int to = pos - key0, from = lo - key0;
#pragma unroll
          for (int e = 0; e < kPmKeys; ++e)
            if (e > to || e < from) s[e] = -INFINITY;
        }
        const float f = kExtra ? 1.4426950408889634f : a.scale * 1.4426950408889634f;
        float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int e = 4; e + 1 < kPmKeys; e += 2) mx4[e >> 1 & 3] = max3(mx4[e >> 1 & 3], s[e], s[e + 1]);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * f;
        if (__any_sync(0xffffffffu, ok && !idle && mx > m + kPmLazy)) {
          const float to = fmaxf(m, mx), corr = to == m ? 1.0f : ex2(m - to);
          l *= corr;
          m = to;
          if (!fresh && ok && !idle) {
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
              float o[16];
              tm_load(ocol + d, o);
              uint32_t v[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[e] * corr);
              tm_store(ocol + d, v);
            }
          }
        }
        if (!idle && ok) {
          const float mu = m == -INFINITY ? 0.0f : m;  // nothing seen so far: every weight is 2^-inf
          const float2 sc = make_float2(f, f), mm = make_float2(-mu, -mu);
          float2 ls = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int ch = 0; ch < kPmKeys; ch += kChunk) {
            uint32_t w[S::kTermsP][kChunk / 2];
#pragma unroll
            for (int e = 0; e < kChunk; e += 2) {
              const float2 y = fma2(make_float2(s[ch + e], s[ch + e + 1]), sc, mm);
              const float2 pp = make_float2(ex2(y.x), ex2(y.y));
              ls = add2(ls, pp);
              uint32_t term[S::kTermsP];
              split(pp.x, pp.y, term);
#pragma unroll
              for (int t = 0; t < S::kTermsP; ++t) w[t][e / 2] = term[t];
            }
#pragma unroll
            for (int t = 0; t < S::kTermsP; ++t) tm_store(scol + t * (kPmKeys / 2) + ch / 2, w[t]);
          }
          l += ls.x + ls.y;
        }
        tm_st_wait();
        tm_fence_before();
        if (ok) bar_arrive_warp(pfull0 + 8 * x, lane);
      }
      {
        PaWalk<kPmKeys, S::kStart> after = walk;
        after.next(a);
        PaPiece ahead{};
        if (after.more()) ahead = after.piece(a);
        queries(ahead);  // (of none, zeros: what is only set at times would take registers all along)
      }
      if (cnt > 0) {  // the last products
        ok = ok && pm_wait_warp(sfull0 + 8 * x, phase & 1, fail, a.timeout_ns);
        ++phase;
      }
      // The row's sums: its own, or those of both groups. (A group without a tile leaves the place of its statistics
      // alone: the other one's scores may still read the queries there.)
      if (!kPair && cnt > 0) s_stat[x * 128 + ln] = make_float4(m, l, sums_m, summed ? 1.0f : 0.0f);
      tm_fence_before();
      meet();
      tm_fence_after();
      float M, L, f_own[2] = {1.0f, 0.0f}, f_sum[2] = {0.0f, 0.0f};
      bool use[2] = {true, false}, more[2] = {false, false};
      {
        const float4 none = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
        const float4 t0 = kPair ? make_float4(m, l, sums_m, summed ? 1.0f : 0.0f) : s_stat[ln], t1 = !kPair && n > 1 ? s_stat[128 + ln] : none;
        M = fmaxf(t0.x, t1.x);
        auto rel = [&](float r) { return r == M ? 1.0f : ex2(r - M); };
        f_own[0] = rel(t0.x);
        f_sum[0] = rel(t0.z);
        more[0] = t0.w != 0.0f;
        L = t0.y * f_own[0];
        if (!kPair && n > 1) {
          f_own[1] = rel(t1.x);
          f_sum[1] = rel(t1.z);
          use[1] = true;
          more[1] = t1.w != 0.0f;
          L = fmaf(t1.y, f_own[1], L);
        }
      }
      if (!kPair) meet();  // the statistics have been read: rows are staged there
      const bool split_up = n < u.tiles;
      if (ok && !idle) {
        // Rows pass through the queries' place, 32 of a warp at a time, so that they are written in pieces of up to 128 bytes: a thread
        // that wrote its own row took 4 us for what now takes one.
        constexpr int kOut = kPair ? D : D / 2;  // dimensions of a thread
        const float f = split_up || L == 0.0f ? (split_up ? 1.0f : 0.0f) : 1.0f / L;  // L = 0: the row sees nothing
        const bool fix = s_bad;
        const int d0 = kPair ? 0 : x * kOut;
        const bool wide = sizeof(T) == 4 || split_up;  // fp32 rows
        constexpr int kStage = std::min(S::kQBytes / 8, 4096);  // of a warp
        const int size = wide ? 4 : 2, seg = min(kStage / 32, kOut * size), per = seg / size, chunks = seg / 16;
        uint8_t* stage = q_smem + (warp - kPmFirstSoftmax) * kStage;
        // where this thread's row goes; the lanes that write it ask for it
        uint8_t* own = split_up ? reinterpret_cast<uint8_t*>(a.part + ((int64_t)p.slot * S::kRows + ru) * D)
                                : reinterpret_cast<uint8_t*>(static_cast<T*>(a.out) + ((int64_t)(tok0 + tok) * a.Hq + h) * D);
        const int left = u.rows - (ru - lane);  // live rows of the warp
#pragma unroll 1
        for (int ds = d0; ds < d0 + kOut; ds += per) {
#pragma unroll 1
          for (int d = ds; d < ds + per; d += 16) {
            __syncwarp();
            float o[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0.0f;
#pragma unroll
            for (int y = 0; y < (kPair ? 1 : 2); ++y) {
              const int gr = kPair ? x : y;
              float t[16];
              if (use[y]) {
                tm_load(tl + S::kColO + gr * D + d, t);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = fmaf(t[e], f_own[y], o[e]);
              }
              if (more[y]) {
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = fmaf(scratch[((int64_t)gr * D + d + e) * 128], f_sum[y], o[e]);
              }
            }
            if (fix && live) {  // values that are not finite, for the rows that see them
#pragma unroll 1
              for (int j = 0; j < n; ++j) {
                const int key0 = key_first + j * kPmKeys;
                if (!partial(key0)) continue;
#pragma unroll 1
                for (int key = max(key0, lo); key < min(key0 + kPmKeys, pos + 1); ++key) {
                  const int id = a.table[(int64_t)u.s * a.width + (key >> a.shift)];
                  if ((unsigned)id >= (unsigned)a.n_pages) continue;
                  const uint32_t* v = reinterpret_cast<const uint32_t*>(
                      a.v + ((int64_t)p.g * a.ts + ((int64_t)id << a.shift) + (key & (a.page - 1))) * D + d);
#pragma unroll
                  for (int e = 0; e < 16; e += 2) {
                    const uint32_t w = v[e / 2];
                    if (!isfinite(low_f(w))) o[e] += low_f(w);
                    if (!isfinite(high_f(w))) o[e + 1] += high_f(w);
                  }
                }
              }
            }
            const int c0 = (d - ds) * size / 16;  // 16-byte pieces, in an order that keeps a column of rows off one bank
            auto put = [&](int c, uint4 v) { *reinterpret_cast<uint4*>(stage + lane * seg + ((c ^ (lane & (chunks - 1))) << 4)) = v; };
            if (wide) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                put(c0 + e / 4, make_uint4(__float_as_uint(o[e] * f), __float_as_uint(o[e + 1] * f), __float_as_uint(o[e + 2] * f),
                                           __float_as_uint(o[e + 3] * f)));
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                put(c0 + e / 8, make_uint4(pack_rn(o[e] * f, o[e + 1] * f), pack_rn(o[e + 2] * f, o[e + 3] * f),
                                           pack_rn(o[e + 4] * f, o[e + 5] * f), pack_rn(o[e + 6] * f, o[e + 7] * f)));
            }
          }
          __syncwarp();
          const int c = lane & (chunks - 1), step = 32 / chunks;
          uint8_t* at = own + ds * size;
#pragma unroll 4
          for (int r0 = 0; r0 < 32; r0 += step) {
            const int r = r0 + lane / chunks;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + r * seg + ((c ^ (r & (chunks - 1))) << 4));
            uint8_t* to = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(at), r));
            if (r < left) *reinterpret_cast<uint4*>(to + c * 16) = v;
          }
        }
        if (split_up && live && d0 == 0) a.ml[(int64_t)p.slot * S::kRows + ru] = make_float2(M, L);
      }
      if (i == 32 * kPmFirstSoftmax && split_up && p.t0 == 0) {  // the first part of a unit: what the join has to know
        PaPiece part = p;
        walk.parts(part);
        PaJoin* to = a.join + blockIdx.x;
        to->tok0 = tok0;
        to->head0 = head0;
        to->rest = rest;
        to->rows = ok ? u.rows : 0;
        to->last = part.c1;
        left_part = true;
      }
      tm_fence_before();
      meet();  // all has been read: tensor memory, the statistics, s_bad
      if (i == 32 * kPmFirstSoftmax) s_bad = 0;
      k0 += 2 * n;
    }
    if (i == 32 * kPmFirstSoftmax && !left_part) a.join[blockIdx.x].rows = 0;
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == kPmMma) tm_free(tmem, kTaTmemCols);
  if (*fail && i == 0 && atomicCAS(a.err, 0u, kTaErrWait) == 0u) a.err[1] = blockIdx.x;
}

// Joins the parts of the units that were split: a warp per row, four (D 64: two) dimensions a lane. Statistics come first, a part to a
// lane, so that nothing waits between the parts themselves (a warp with two rows and running statistics took 15 us for 128 rows of
// 19 parts). The live rows of all units, in order, are dealt to warps: most CTAs of the first kernel leave no rows to join, and a grid of
// a CTA for every four rows there could be took 10 us to start and end.
constexpr int kJoinWarps = 8, kJoinCtas = 4;  // CTAs per CTA of the first kernel
template <typename T, int D, int kRows>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const __grid_constant__ PaArgs a, int jobs) {
  constexpr int E = D / 32;
  using V = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ int s_rows[kPaManyCtas + 1];  // rows of the units before
  dependent_launch_wait();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    constexpr int kEach = (kPaManyCtas + 31) / 32;
    int n[kEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) n[e] = lane * kEach + e < jobs ? a.join[lane * kEach + e].rows : 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) sum += n[e];
    int before = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, before, d);
      before += lane < d ? 0 : x;
    }
    before -= sum;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (lane * kEach + e <= kPaManyCtas) s_rows[lane * kEach + e] = before;
      before += n[e];
    }
    if (lane == 31) s_rows[kPaManyCtas] = before;
  }
  __syncthreads();
  const int total = s_rows[kPaManyCtas];
#pragma unroll 1
  for (int item = blockIdx.x * kJoinWarps + (threadIdx.x >> 5); item < total; item += gridDim.x * kJoinWarps) {
    int c0 = 0;  // the last unit that begins at or before this row
#pragma unroll
    for (int d = 128; d; d /= 2)
      if (c0 + d < kPaManyCtas && s_rows[c0 + d] <= item) c0 += d;
    const PaJoin job = a.join[c0];
    const int r = item - s_rows[c0];
    const V* part = reinterpret_cast<const V*>(a.part + (int64_t)r * D) + lane;
    auto place = [&](int c) { return (int64_t)(2 * c + (c == c0)) * kRows; };
    float M = -INFINITY, L = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 1
    for (int b0 = c0; b0 <= job.last; b0 += 32) {  // 32 parts at a time
      const float2 ml = b0 + lane <= job.last ? __ldcg(a.ml + place(b0 + lane) + r) : make_float2(-INFINITY, 0.0f);
      float to = ml.x;
#pragma unroll
      for (int d = 16; d; d /= 2) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
      to = fmaxf(to, M);
      const float corr = M == to ? 1.0f : ex2(M - to), mine = ml.x == to ? 1.0f : ex2(ml.x - to);
      float sum = ml.y * mine;
#pragma unroll
      for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      L = fmaf(L, corr, sum);
      M = to;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= corr;
      const int n = min(32, job.last - b0 + 1);
#pragma unroll 16
      for (int b = 0; b < n; ++b) {
        const V y = __ldcg(part + place(b0 + b) * (D / E));
        const float g = __shfl_sync(0xffffffffu, mine, b);
        const float* ye = reinterpret_cast<const float*>(&y);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(ye[e], g, o[e]);
      }
    }
    const float g = L == 0.0f ? 0.0f : 1.0f / L;
    const int away = node_of(job.rest + r, 1.0f / (float)a.G);
    T* out = static_cast<T*>(a.out) + ((int64_t)(job.tok0 + away) * a.Hq + job.head0 + r - away * a.G) * D + lane * E;
    if constexpr (sizeof(T) == 4) {
      if constexpr (E == 4) *reinterpret_cast<float4*>(out) = make_float4(o[0] * g, o[1] * g, o[2] * g, o[3] * g);
      else *reinterpret_cast<float2*>(out) = make_float2(o[0] * g, o[1] * g);
    } else {
      uint32_t w[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) w[e / 2] = pack_rn(o[e] * g, o[e + 1] * g);
      if constexpr (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(out) = w[0];
    }
  }
}

// ---- host -----------------------------------------------------------------------------------
template <typename T, int D, bool kPair, bool kExtra>
nt_status launch_many(const PmMaps& maps, const PaArgs& a, cudaStream_t st) {
  constexpr int smem = PmShape<T, D, kPair>::kSmem;
  static std::atomic<int> allowed[64];
  NT_TRY(allow_smem(paged_many_kernel<T, D, kPair, kExtra>, smem, allowed));
  const int ctas = std::min(device_sm_count(), kPaManyCtas);
  NT_CUDA_TRY(launch_kernel(paged_many_kernel<T, D, kPair, kExtra>, dim3((unsigned)ctas), dim3(kPmThreads), smem, st, true, maps, a));
  NT_TRY(check_launch("paged_many_kernel"));
  NT_CUDA_TRY(launch_kernel(paged_join_kernel<T, D, PmShape<T, D, kPair>::kRows>, dim3((unsigned)(ctas * kJoinCtas)), dim3(32 * kJoinWarps), 0, st, true, a, ctas));
  return check_launch("paged_join_kernel");
}
template <typename T, int D, bool kPair>
nt_status launch_many_extra(const PmMaps& maps, const PaArgs& a, cudaStream_t st) {
  return a.cap > 0.0f || a.slopes ? launch_many<T, D, kPair, true>(maps, a, st) : launch_many<T, D, kPair, false>(maps, a, st);
}

}  // namespace

nt_status launch_paged_many(const PaArgs& a, int dtype, int D, int64_t max_rows, cudaStream_t st) {
  PmMaps maps;
  NT_TRY(paged_map(&maps.k, a.k, D, std::min(a.page, kPmKeys), a));
  NT_TRY(paged_map(&maps.v, a.v, D, std::min(a.page, kPmKeys), a));
  if (dtype == NT_F32) return D == 64 ? launch_many_extra<float, 64, false>(maps, a, st) : launch_many_extra<float, 128, false>(maps, a, st);
  if (max_rows <= 128)
    return D == 64 ? launch_many_extra<uint16_t, 64, false>(maps, a, st) : launch_many_extra<uint16_t, 128, false>(maps, a, st);
  return D == 64 ? launch_many_extra<uint16_t, 64, true>(maps, a, st) : launch_many_extra<uint16_t, 128, true>(maps, a, st);
}

}  // namespace nt
