// What the two kernels of idx_tree_mla share: the call's parameters, how its work
// is dealt to the CTAs, the planner warp that walks a CTA's share, the join of
// items that shares cut, and inline PTX.
//
// Work: an item is a group of M rows of a sequence (of a token, where each token
// has its own selection) with all keys that they see, in tiles of KT keys.  The
// tiles of all items are numbered through and dealt in equal contiguous shares to
// teams of CTAs, one persistent CTA per SM (a team is one CTA, or the two that
// share a row's output columns); so ragged lengths and counts cost nothing.
// Groups of one sequence lie side by side in that order, so that teams near each
// other read its rows, but a team's next group reads them again, and where the
// caches of all sequences exceed L2 that costs HBM reads (eight groups over 208 MB:
// 692 MB read, a quarter of what HBM delivers meanwhile).  An item that a share's
// end cuts leaves partial (O, maximum, sum) in the workspace, and
// tree_mla_join_kernel adds them in a fixed order.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "api_internal.h"
#include "ptx.cuh"

namespace idx {
namespace tree {

constexpr int kLat = 512, kRow = 576;
// Keys per share below which work is not split further: a tile of 128 keys (one
// sequence of 2 048 positions, 64 heads, calls in a CUDA graph: 18.8 us, with 256 25.6,
// with 512 31.2; 128 heads 19.7, 23.5, 26.8).  Up to two of them an item stays whole,
// which saves the join's launch: 256 positions, 16 heads take 13.7 us then and 11.7
// cut in two, 128 heads 16.8 and 17.9.
constexpr int kMinShare = 128;
constexpr int kAhead = 4;                     // tiles that the planner may be ahead of its readers
constexpr float kRaise = 8.f;                 // log2 margin of the reference maximum
constexpr float kNone = -3.4028235e38f;       // stands for a reference maximum of −inf: any score passes it
// A weight is 2^(s · scale − m), one fused operation, with m = fl(s_max · scale): what
// that product was rounded by, half a step of m at most, multiplies all weights of a
// row alike.  Beyond 2^28 (a step of 2^4 and more) that may be more than an exponent
// holds, and scores that differ at all differ by 2^4: there the weight is 1 where
// fl(s · scale) reaches m and 0 elsewhere.  Such rows are looked at in every tile.
constexpr float kFar = 268435456.f;
constexpr int kFaultScores = 1;               // the scores of a piece's last tile
constexpr int kFaultEnd = 4;                  // one of the softmax warps that share rows, at its list's end
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Piece {                                // what the CTA does next: tiles [t0, t1) of an item
  int t0, t1;
  int rows;                                   // valid rows
  int slot;                                   // −1: the whole item; else partial slot 0 or 1
  int mixed;                                  // the rows belong to several tokens
  int nkeys;                                  // keys before the drafts
  int64_t row0;                               // global row of the first
};

struct Cut {                                  // an item that begins in a share and ends in another
  int64_t row0;
  int rows, pieces;                           // pieces after the first; 0: nothing to join
};

struct TreeParams {
  const uint16_t *q, *cache;
  const int32_t* table;
  int max_pages, num_pages, page_size;
  uint32_t div_mul;                           // x / page_size = x · div_mul >> div_shift for x < 2^31
  int div_shift;
  const int32_t *lengths, *counts;
  int B, n, H, max_len;
  const uint64_t* mask;
  const int32_t* indices;
  int k;
  float scale_log2;
  void* out;
  int out_bf16;
  float* lse;
  int M, halves;                              // rows per CTA; CTAs (a team) that share the output columns of a row
  int teams, whole;                           // whole: items are not cut
  float* part;                                // [CTA][2] partial slots: M · (512 / halves) outputs, M maxima, M sums
  Cut* cuts;                                  // [CTA]
  unsigned long long budget_ns;               // bound of every wait
  int fault;                                  // tests: who waits for a barrier that nothing signals
  unsigned int* err;
};

int launch_tree_mla_wide(const CUtensorMap& tmap_q, const TreeParams& p, int ctas, cudaStream_t stream);

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}
// 16 bytes into shared memory, zeros where bytes = 0; cp_async_arrive makes the
// barrier count this thread once its copies so far have landed
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// the same for what is read once: its line in L2 is the next to be given up
__device__ __forceinline__ uint64_t once_policy() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void cp_async16_once(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* src) { asm volatile("prefetch.global.L2 [%0];" ::"l"(src)); }
__device__ __forceinline__ void prefetch_l2_row(const void* src) {   // a cache row, 16-byte aligned
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "n"(2 * kRow) : "memory");
}
// 32 bytes of one thread: a whole sector (32-byte aligned)
__device__ __forceinline__ void st_global32(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// the same with A read from TMEM (row m in lane m, two bf16 per 32-bit column)
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f16, A = B = bf16, D = f32, M = 128; a_mn, b_mn: operand MN-major
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? (1u << 15) : 0u) | (b_mn ? (1u << 16) : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
constexpr uint32_t kNegateA = 1u << 13;       // the product with A's signs turned
// MN-major operand, 128-byte swizzle: 64 elements along MN per 128-byte row, 8-row
// atoms along K; `mn_stride` bytes to the next 64 elements along MN
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t mn_stride) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | static_cast<uint64_t>((mn_stride >> 4) & 0x3FFF) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two weights (≥ 0) rounded to bf16, ties away from zero: on the integer pipe,
// since the conversion instruction shares its pipe with ex2 and 8 192 of each per
// tile are what the softmax would wait for.  A NaN weight may be lost here; its
// row's sum keeps it.
__device__ __forceinline__ uint32_t bf_pack_weights(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo) + 0x8000u, __float_as_uint(hi) + 0x8000u, 0x7632);
}
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > kFar && m > -INFINITY; }
// a score of a row beyond kFar as what stands in for it, with 0 for m: 0 or −inf (NaN where m is infinite)
__device__ __forceinline__ float far_score(float z, float scale, float m) {
  const float d = __fmul_rn(z, scale) - m;    // (not fused: m is such a product)
  return d < 0.f ? -INFINITY : d;
}
// `count` threads meet; whether any of them says v
__device__ __forceinline__ bool bar_named_any(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}
// The softmax warps that share rows meet at one named barrier, always by vote().
// The meetings are not bounded in time, so every warp takes its place once more on
// its way out (part): one that gives up writes the number of that meeting first and
// says true, and the others, wherever they then meet, see the number and go too.
// The meeting after the list's end is there for a warp that gave up while the
// others came to the end: all of them have met equally often, so its last meeting
// is theirs.  (A warp can give up only between meetings that end a wait; the number
// tells this meeting from a later one.)
struct Meeting {
  int id, count, number;
  volatile int* left_at;
  __device__ __forceinline__ bool vote(bool v) {
    ++number;
    return bar_named_any(id, count, v);
  }
  __device__ __forceinline__ bool left() const { return __any_sync(0xFFFFFFFFu, *left_at == number); }
  __device__ __forceinline__ void part(bool ok) {
    if (!ok) *left_at = number + 1;
    vote(!ok);
  }
};

// A warp's wait for a phase of an mbarrier, for at most budget_ns; false once this
// CTA has given up.  The global timer, whose read takes about 1 000 cycles, is
// looked at every 256 polls only: a wait that succeeds at once costs some 60
// cycles instead of 300, and there are a dozen per tile on the critical path.
// The vote makes the answer uniform for the compiler, so that what the MMA issue
// computes stays in uniform registers.  nap: about 50 ns between polls, where
// nobody waits for this warp, so that the shared-memory queue stays free.
struct Waits {
  uint64_t budget_ns;
  volatile int* abort_flag;
  unsigned int* err;
  template <bool kNap>
  __device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity) const {
    uint64_t t0 = 0;
    for (uint32_t i = 1; !__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)); ++i) {
      if ((i & 255) == 0 && gave_up(t0)) return false;
      if (kNap) __nanosleep(40);
    }
    return true;
  }
  __device__ __noinline__ bool gave_up(uint64_t& t0) const {
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    const bool late = __any_sync(0xFFFFFFFFu, now - t0 > budget_ns);
    if (late && !*abort_flag) raise_error(err, IDX_DEV_ERR_TIMEOUT);
    if (late) *abort_flag = 1;
    return __any_sync(0xFFFFFFFFu, *abort_flag);
  }
  __device__ __forceinline__ bool test(uint64_t* bar, uint32_t parity) const {
    uint32_t ok;                              // (try_wait would suspend the thread for a while)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xFFFFFFFFu, ok != 0);
  }
  __device__ __forceinline__ bool nap(uint64_t* bar, uint32_t parity) const { return poll<true>(bar, parity); }
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const { return poll<false>(bar, parity); }
  // during teardown: whatever happened before, wait (the whole warp) for what is in
  // flight; 10 ms at least, however small the budget, since memory goes back behind it
  __device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) const {
    const uint64_t t0 = globaltimer_ns(), limit = max(budget_ns, uint64_t{10000000});
    while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity) || globaltimer_ns() - t0 > limit)) {}
  }
};

// NC consecutive 32-bit columns of this warp's 32 lanes
template <int NC>
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t* r);
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
template <int NC>
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t* r);
template <>
__device__ __forceinline__ void tmem_st<8>(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t a, const uint32_t* r) {
  tmem_st<8>(a, r);
  tmem_st<8>(a + 8, r + 8);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// ties loaded registers to a point after tmem_wait()
template <int NC>
__device__ __forceinline__ void regs_ready(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < NC; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// ------------------------------------------------------------------ work
struct Seq {
  int len, cnt, ctx, groups, items, tiles;    // row groups (of a token, where each has its selection); tiles per item
};
template <int M, int KT>
__device__ __forceinline__ Seq seq_info(const TreeParams& p, int b, bool report) {
  Seq s;
  s.cnt = p.counts ? __ldg(p.counts + b) : p.n;
  s.len = __ldg(p.lengths + b);
  if (s.cnt < 0 || s.cnt > p.n || s.len < s.cnt || s.len > p.max_len) {
    if (report) raise_error(p.err, IDX_DEV_ERR_LENGTH);
    s.cnt = s.len = 0;
  }
  s.ctx = s.len - s.cnt;
  s.groups = static_cast<int>(((p.indices ? 1 : s.cnt) * static_cast<int64_t>(p.H) + M - 1) / M);
  s.items = p.indices ? s.cnt * s.groups : s.groups;
  s.tiles = (static_cast<int>(p.indices ? p.k + s.cnt : s.len) + KT - 1) / KT;
  return s;
}

// drafts that a token's rows see
__device__ __forceinline__ uint64_t draft_mask(const TreeParams& p, int b, int i, int cnt) {
  const uint64_t all = cnt >= 64 ? ~0ull : (1ull << cnt) - 1;
  const uint64_t m = p.mask ? __ldg(reinterpret_cast<const unsigned long long*>(p.mask) + static_cast<int64_t>(b) * p.n + i)
                            : (2ull << i) - 1;
  return m & all;
}

// Shared state of the planner and the warps that follow it; M rows, KT keys a tile.
template <int M, int KT, int kWarps>
struct PlanState {
  uint64_t mask[2][M];                        // per piece parity: drafts each row sees
  unsigned long long wild[2];                 // drafts that were taken out of V, their rows not being finite
  alignas(16) uint8_t kind[kAhead][KT];       // per tile (mod kAhead) and key: 0 unseen, 1 context, 2 + j draft j
  alignas(16) int row[kAhead][KT];            // cache rows of the keys, −1: none
  int last[kAhead];                           // no tile: the list has ended
  Piece piece[2];
  long long scan[kWarps];
  long long start_off;
  int start_b;
  int abort_flag;
  uint32_t tmem;
  uint64_t never;                             // nothing signals it
  uint64_t tile_full[kAhead], tile_read[kAhead], piece_full[2], piece_empty[2], q_full, q_empty;

  __device__ void init(int B, int tile_readers, int piece_readers) {
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&tile_full[i], 1);
      mbar_init(&tile_read[i], tile_readers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], piece_readers);
    }
    mbar_init(&never, 1);
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    abort_flag = 0;
    start_b = B;
    start_off = 0;
  }
};

// a / b for a ≥ 0 whose result fits an int (a 64-bit division takes some 500 cycles)
__device__ __forceinline__ int quotient(long long a, int b) {
  return a <= 0x7FFFFFFF ? static_cast<int>(a) / b : static_cast<int>(a / b);
}

struct Share {
  long long size, begin, end;                 // in tiles (in items where they are not cut)
};
// Where this team's share lies: every thread of the CTA adds up a run of
// sequences, then the one whose run holds the share's begin looks for it.  Two
// CTA barriers; what was written before the first is visible after it.
template <int M, int KT, int kThreads, class State>
__device__ __forceinline__ Share find_share(const TreeParams& p, State& ms, int team) {
  if (!p.whole) asm volatile("griddepcontrol.launch_dependents;");   // the join may be placed as SMs become free
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, static_cast<int>(threadIdx.x) * per), b_hi = min(p.B, b_lo + per);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s = seq_info<M, KT>(p, b, blockIdx.x == 0);
    mine += static_cast<long long>(s.items) * (p.whole ? 1 : s.tiles);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) ms.scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0, before = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += ms.scan[w];
    total += ms.scan[w];
  }
  Share sh;
  sh.size = max(static_cast<long long>(p.whole ? 1 : kMinShare / KT), (total + p.teams - 1) / p.teams);
  sh.begin = min(total, sh.size * team);
  sh.end = min(total, sh.begin + sh.size);
  if (sh.begin < sh.end && before + incl - mine <= sh.begin && sh.begin < before + incl) {
    long long at = before + incl - mine;
    for (int b = b_lo; b < b_hi; ++b) {
      const Seq s = seq_info<M, KT>(p, b, false);
      const long long w = static_cast<long long>(s.items) * (p.whole ? 1 : s.tiles);
      if (sh.begin < at + w) {
        ms.start_b = b;
        ms.start_off = sh.begin - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  return sh;
}

// The planner warp: walks the share, publishes each piece (tile range, what its
// rows see of the drafts) and each tile (cache rows of its keys), and has the
// piece's queries loaded: load_q(row0) issues them on ms.q_full.
template <int M, int KT, class State, class LoadQ>
__device__ __forceinline__ void plan(const TreeParams& p, State& ms, const Share& sh, const Waits& waits, LoadQ load_q) {
  constexpr int E = KT / 32;                  // keys per lane
  const int lane = threadIdx.x & 31;
  bool ok = true;
  int tiles = 0, pieces = 0;                  // running counts
  long long cur = sh.begin;
  int b = ms.start_b;
  long long off = ms.start_off;
  Cut cut{0, 0, 0};
  Seq s{}, ahead{};                           // this sequence, the next one
  if (b < p.B) s = seq_info<M, KT>(p, b, false);
  if (b + 1 < p.B) ahead = seq_info<M, KT>(p, b + 1, false);
  while (ok && cur < sh.end) {
    const int weight = p.whole ? 1 : s.tiles;
    if (off >= static_cast<long long>(s.items) * weight) {
      if (++b >= p.B) break;
      s = ahead;
      if (b + 1 < p.B) ahead = seq_info<M, KT>(p, b + 1, false);
      off = 0;
      continue;
    }
    const int item = p.whole ? static_cast<int>(off) : quotient(off, weight);
    const int t0 = p.whole ? 0 : static_cast<int>(off - static_cast<long long>(item) * weight);
    const int t1 = p.whole ? s.tiles : static_cast<int>(min(static_cast<long long>(s.tiles), t0 + (sh.end - cur)));
    const int step = p.whole ? 1 : t1 - t0;
    off += step;
    cur += step;
    // this CTA's rows: M flattened (token, head) rows of the sequence, or M heads
    // of one token where each token has its selection
    const int tok = p.indices ? item / s.groups : 0;
    const int64_t lo = static_cast<int64_t>(p.indices ? item % s.groups : item) * M;
    const int64_t have = p.indices ? p.H : static_cast<int64_t>(s.cnt) * p.H;
    const int rows = static_cast<int>(min(static_cast<int64_t>(M), have - lo));
    const int64_t row0 = (static_cast<int64_t>(b) * p.n + tok) * p.H + lo;
    const int slot = t0 == 0 && t1 == s.tiles ? -1 : t0 == 0 ? 1 : 0;
    if (slot == 1) {
      cut.row0 = row0;
      cut.rows = rows;
      cut.pieces = sh.size >= s.tiles ? 1 : (s.tiles - t1 + static_cast<int>(sh.size) - 1) / static_cast<int>(sh.size);
    }
    const int nkeys = p.indices ? p.k : s.ctx;
    // Its tiles' keys, lane ↔ keys E·lane …: the positions of tile t + 2 and the page
    // numbers of tile t + 1 are fetched while tile t is published, and those of the
    // first two before anything else of the piece (0.1 - 0.3 us off a short call)
    const int32_t* sel = p.indices ? p.indices + (static_cast<int64_t>(b) * p.n + tok) * p.k : nullptr;
    const int32_t* pages = p.table + static_cast<int64_t>(b) * p.max_pages;
    uint64_t any = 0;                         // drafts that some row sees
    auto page_of = [&](int pos) {
      return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(pos)) * p.div_mul >> p.div_shift);
    };
    auto position = [&](int t, int e) {       // position of a key, −1 (or beyond the context) where it selects nothing
      const int v = t * KT + E * lane + e;
      if (v >= nkeys) return v - nkeys < s.cnt ? s.ctx + v - nkeys : -1;
      if (!sel) return v;
      return t < t1 ? __ldg(sel + v) : -1;
    };
    auto valid = [&](int t, int e, int pos) {  // a selection names context positions only
      return pos >= 0 && (t * KT + E * lane + e >= nkeys || pos < s.ctx);
    };
    auto seen = [&](int t, int e) {
      const int v = t * KT + E * lane + e - nkeys;
      return v < 0 || v >= 64 || ((any >> v) & 1);
    };
    int pos_next[E], page_next[E], pos_far[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      pos_next[e] = position(t0, e);
      if (!valid(t0, e, pos_next[e])) pos_next[e] = -1;
      pos_far[e] = position(t0 + 1, e);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) page_next[e] = pos_next[e] >= 0 ? __ldg(pages + page_of(pos_next[e])) : 0;
    const int pb = pieces & 1;
    if (pieces >= 2 && !(ok = waits.nap(&ms.piece_empty[pb], ((pieces >> 1) - 1) & 1))) break;
    for (int c = lane; c < M; c += 32) {
      const uint64_t m = c < rows ? draft_mask(p, b, p.indices ? tok : quotient(lo + c, p.H), s.cnt) : 0;
      ms.mask[pb][c] = m;
      any |= m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) any |= __shfl_xor_sync(0xFFFFFFFFu, any, o);
    if (lane == 0) {
      Piece& pc = ms.piece[pb];
      pc.t0 = t0;
      pc.t1 = t1;
      pc.rows = rows;
      pc.slot = slot;
      pc.mixed = !p.indices && quotient(lo, p.H) != quotient(lo + rows - 1, p.H);
      pc.nkeys = nkeys;
      pc.row0 = row0;
      ms.wild[pb] = 0;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.piece_full[pb]);
    // ---- its tiles
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (!seen(t0, e)) pos_next[e] = -1;
    for (int t = t0; t < t1; ++t) {
      int row[E];
      uint32_t kinds = 0;
      bool bad = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int v = t * KT + E * lane + e;
        row[e] = -1;
        if (pos_next[e] >= 0) {
          if (page_next[e] < 0 || page_next[e] >= p.num_pages) {
            bad = true;
          } else {
            row[e] = (page_next[e] - page_of(pos_next[e])) * p.page_size + pos_next[e];
            kinds |= static_cast<uint32_t>(v < nkeys ? 1 : 2 + v - nkeys) << (8 * e);
          }
        }
      }
      if (bad) raise_error(p.err, IDX_DEV_ERR_PAGE);
      if (t + 1 < t1) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          pos_next[e] = valid(t + 1, e, pos_far[e]) && seen(t + 1, e) ? pos_far[e] : -1;
          page_next[e] = pos_next[e] >= 0 ? __ldg(pages + page_of(pos_next[e])) : 0;
          pos_far[e] = position(t + 2, e);
        }
      }
      const int par = tiles % kAhead;
      // free once the copies and the softmax have read what it said kAhead tiles ago
      if (tiles >= kAhead && !(ok = waits.nap(&ms.tile_read[par], (tiles / kAhead - 1) & 1))) break;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        ms.kind[par][E * lane + e] = static_cast<uint8_t>(kinds >> (8 * e));
        ms.row[par][E * lane + e] = row[e];
      }
      if (lane == 0) ms.last[par] = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.tile_full[par]);
      ++tiles;
      if (t == t0) {                          // its queries, once the last piece's are no longer read
        if (pieces >= 1 && !(ok = waits.nap(&ms.q_empty, (pieces - 1) & 1))) break;
        if (elect_one()) load_q(static_cast<int>(row0));
        __syncwarp();
        ++pieces;
      }
    }
  }
  // the end of the list
  if (ok) {
    const int pb = pieces & 1;
    if (pieces >= 2) ok = waits.nap(&ms.piece_empty[pb], ((pieces >> 1) - 1) & 1);
    if (ok && lane == 0) {
      ms.piece[pb].t0 = ms.piece[pb].t1 = 0;
      mbar_arrive(&ms.piece_full[pb]);
    }
    const int par = tiles % kAhead;
    if (ok && tiles >= kAhead) ok = waits.nap(&ms.tile_read[par], (tiles / kAhead - 1) & 1);
    if (ok && lane == 0) {
      ms.last[par] = 1;
      mbar_arrive(&ms.tile_full[par]);
    }
  }
  if (!p.whole && lane == 0) p.cuts[blockIdx.x] = cut;
  if (pieces) waits.drain(&ms.q_full, (pieces - 1) & 1);   // landed before the memory goes
}

// A draft whose latent features are not all finite, in a group of rows of which some
// do not see it: it is taken out of V, since 0 · NaN would reach those rows too.
// Rows that see it have its score, which is not finite either.  NaN and +∞ make
// their weights NaN, and their sums say so; −∞ makes a weight of 0, and what
// 0 · (what is not finite) would have put into the output is put there after the
// product (spoil), where the draft's row is read once more.
__device__ __forceinline__ bool not_finite(uint16_t bf) { return (bf & 0x7F80u) == 0x7F80u; }
__device__ __forceinline__ bool not_finite(const uint4& x) {       // any of eight
  const uint32_t e[4] = {x.x, x.y, x.z, x.w};
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= (e[i] & 0x7F80u) == 0x7F80u || (e[i] & 0x7F800000u) == 0x7F800000u;
  return r;
}
// cache row of draft j of the sequence that the group's first row belongs to; some
// row sees it, so its page was one (checked again: the table is read anew)
__device__ __forceinline__ const uint16_t* draft_row(const TreeParams& p, const Piece& pc, int j) {
  const int64_t b = pc.row0 / (static_cast<int64_t>(p.n) * p.H);
  const int pos = pc.nkeys + j, at = pos / p.page_size;
  const int page = min(max(__ldg(p.table + b * p.max_pages + at), 0), p.num_pages - 1);
  return p.cache + (static_cast<int64_t>(page) * p.page_size + (pos - at * p.page_size)) * kRow;
}
// NaN for output feature d of row `row0 + row`, or of a partial result (`part`: its place)
__device__ __forceinline__ void spoil(const TreeParams& p, const Piece& pc, int row, int d, float* part) {
  const float nan = __int_as_float(0x7FFFFFFF);
  if (part)
    *part = nan;
  else if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.out)[(pc.row0 + row) * kLat + d] = __float2bfloat16_rn(nan);
  else
    static_cast<float*>(p.out)[(pc.row0 + row) * kLat + d] = nan;
}

__device__ __forceinline__ float lse_of(float m, float z) {    // m in log2 units
  return m == -INFINITY && z == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * kLn2) + logf(z);
}

// partial slot of a CTA: M rows of D outputs (as [M][D], in runs of eight as
// [D / 8][M][8] where a row's outputs are split over two CTAs), M maxima, M sums
__device__ __forceinline__ float* part_slot(const TreeParams& p, int64_t cta, int slot) {
  return p.part + (cta * 2 + slot) * (static_cast<int64_t>(p.M) * (kLat / p.halves + 2));
}

}  // namespace tree
}  // namespace idx
