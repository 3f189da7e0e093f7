// Latent attention of drafted token trees over the paged cache (idx_tree_mla):
//   S = q · Kᵀ over 576 features, a softmax over the positions each row sees,
//   O = P · V with V the first 512 features of the same cache rows.
//
// Everything is computed transposed: Sᵀ = K · qᵀ (M = 128 keys, N rows) and
// Oᵀ = Vᵀ · Pᵀ (M = 128 output features, four times; K = 128 keys).  The cache
// tile is the A operand of both products (K-major for the scores, MN-major for
// the output: the same shared-memory bytes), and a row (token, head) is a
// column of the accumulators.  So a few rows (16 heads of one token) need
// N = 16 columns instead of a 128-row tile that is mostly padding, and 64 rows
// keep Oᵀ (4 · N columns) and Sᵀ in TMEM together.  A tcgen05.mma of M = 128,
// K = 16 costs 40 / 41 / 48 cycles at N = 16 / 32 / 64 (shared-memory reads of
// A, 4 KB, and B; the tensor cores alone need 8 / 16 / 32), so a 128-key tile
// costs 68 MMAs ≈ 2 700 – 3 300 cycles, against 147 KB of cache rows that HBM
// delivers to one SM in about 6 500: small N is bound by HBM, N = 64 by the MMAs.
//
// Work: the (sequence, row block) items' 128-key tiles are numbered through and
// dealt in equal contiguous shares to teams of CTAs, one persistent CTA per SM;
// the CTAs of a team walk the same tiles with different row groups (the rows of
// a cache tile come from HBM once and from L2 after that).  An item cut by a
// share's end leaves partial (O, max, sums) in the workspace; a second kernel
// joins them in a fixed order.
//
// One CTA, 12 warps (20 for N = 64):
//   warp 0     walks the share: publishes each piece (item, tile range, row masks),
//              loads its queries, and streams the tiles' rows by TMA — boxes of
//              whole page runs for dense tiles, tile::gather4 by row number for
//              selections and ragged tiles, where a row that no one sees has row
//              number −1 and arrives as zeros (never as what memory holds);
//   warp 1     issues the MMAs: scores of tile t, then its product, so that tile
//              t + 1 streams into the parts of the buffer that the product has freed;
//   warps 2, 3 issue two thirds of the copies (a selection's tile is 288 of them);
//   warps 4 …  softmax: thread ↔ (key, part of the rows); the column maxima by a
//              transposing butterfly across lanes and shared memory across warps; a
//              running reference maximum per row, raised only when a tile passes it by
//              2^8 (then O in TMEM is rescaled); P = 2^(s − m) in bf16 for the tensor
//              cores (a relative 2^-8 per weight; the sum that divides O adds the
//              rounded weights, the one behind lse the unrounded); O / Σ at the end.
// Every wait is bounded; a CTA that gives up raises IDX_DEV_ERR_TIMEOUT, waits for
// its copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "api_internal.h"
#include "ptx.cuh"

namespace idx {
namespace {

constexpr int kLat = 512, kRow = 576;
constexpr int kTile = 128;                    // keys per tile
constexpr int kPair = 32768;                  // 128 keys × 128 latent features: two 64-feature chunks
constexpr int kChunk = 16384;                 // 128 keys × 64 features
constexpr int kMaxTeam = 16;
constexpr int kMinShare = 2;                  // tiles per team below which work is not split further
constexpr int kCopyWarps = 4;                 // warps that copy the tiles
constexpr int kFirstSoft = 2 + kCopyWarps;    // planner, MMA issuer, copies, then the softmax
constexpr float kRaise = 8.f;                 // log2 margin of the reference maximum
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int N>
struct Cfg {
  static constexpr int kSoftWarps = N == 64 ? 16 : 8;
  static constexpr int kParts = kSoftWarps / 4;             // row parts, each of four warps (128 keys)
  static constexpr int kNC = N / kParts;                    // rows per softmax thread
  static constexpr int kThreads = (kFirstSoft + kSoftWarps) * 32;
  static constexpr int kPairs = N == 16 ? 5 : 4;            // latent buffers
  static constexpr int kRopes = N == 32 ? 2 : 1;            // rotary-chunk buffers
  static constexpr bool kAliasP = N == 64;                  // P takes the rotary chunk's place after the scores
  static constexpr int kOffRope = kPairs * kPair;
  static constexpr int kOffP = kAliasP ? kOffRope : kOffRope + kRopes * kChunk;
  static constexpr int kOffQ = kOffRope + (kRopes + (kAliasP ? 0 : 1)) * kChunk;
  static constexpr int kOffMisc = kOffQ + 9 * N * 128;
  static constexpr uint32_t kTmemCols = N == 16 ? 128 : N == 32 ? 256 : 512;
};

struct Piece {                                // what the CTA does next: tiles [t0, t1) of an item
  int t0, t1;
  int rows;                                   // valid columns
  int slot;                                   // −1: the whole item; else partial slot 0 or 1
  int mixed;                                  // the columns span several tokens
  int pad;
  int64_t row0;                               // global row of column 0
};

struct Cut {                                  // an item that begins in a share and ends in another
  int64_t row0;
  int rows, pieces;                           // pieces after the first; 0: nothing to join
};

template <int N>
struct Misc {
  uint64_t mask[2][N];                        // per piece parity: drafts each column sees
  float wmax[2][Cfg<N>::kParts][4][Cfg<N>::kNC];   // per tile parity, row part, warp: column maxima
  float m[Cfg<N>::kSoftWarps][Cfg<N>::kNC], alpha[Cfg<N>::kSoftWarps][Cfg<N>::kNC];
  float sum[Cfg<N>::kParts][4][Cfg<N>::kNC];  // row part, warp
  alignas(16) uint8_t kind[2][kTile];         // per tile parity and key: 0 unseen, 1 context, 2 + j draft j
  alignas(16) int row[2][kTile];              // per tile parity: cache rows of the keys, −1: none
  int last[2];                                // per tile parity: no tile, the list has ended
  Piece piece[2];
  long long scan[Cfg<N>::kThreads / 32];
  long long start_off, total;
  int start_b;
  uint64_t pair_full[5], pair_empty[5], rope_full[2], rope_empty[2];
  uint64_t q_full, q_empty, s_full, p_full, o_full, o_free, drain;
  uint64_t tile_full[2], tile_read[2], piece_full[2], piece_empty[2];
  uint32_t tmem;
  int abort_flag;
};

struct TreeParams {
  const int32_t* table;
  const uint16_t* cache;
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
  int team, blocks;                           // CTAs per team, row blocks (of `team` groups) per token set
  int teams, whole;                           // whole: items are not cut
  float* part;                                // [CTA][2] partial slots of N·(512 + 2) floats
  Cut* cuts;                                  // [CTA]
  unsigned long long budget_ns;
  unsigned int* err;
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}
// mbar_wait that polls 256 times before it looks at the clock: a read of the
// global timer takes about 1 000 cycles, which every wait that does not succeed
// at once would add to its hand-off
__device__ __forceinline__ bool mbar_wait_polling(uint64_t* bar, uint32_t parity, uint64_t budget_ns,
                                                  volatile int* abort_flag, unsigned int* err) {
  for (int i = 0; i < 256; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, budget_ns, abort_flag, err);
}
// 16 bytes into shared memory, zeros where bytes = 0; cp_async_arrive makes the
// barrier count this thread once its copies so far have landed
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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
// kind::f16, A = B = bf16, D = f32, M = 128; mn: both operands MN-major
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? (3u << 15) : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (8u << 24);
}
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
__device__ __forceinline__ void bar_part(int part) {            // the 128 softmax threads of a row part
  asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");
}

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

// Column reduction of v[NC] over the warp's 32 lanes by a transposing butterfly;
// returns the result of column lane >> (5 − log2 NC).  v is overwritten.
template <int NC, bool kMax>
__device__ __forceinline__ float reduce_columns(float* v, int lane) {
  int off = 16;
#pragma unroll
  for (int m = NC; m > 1; m >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < m / 2; ++i) {
      const float keep = up ? v[i + m / 2] : v[i];
      const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + m / 2], off);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
    off >>= 1;
  }
  float r = v[0];
  for (; off > 0; off >>= 1) {
    const float got = __shfl_xor_sync(0xFFFFFFFFu, r, off);
    r = kMax ? fmaxf(r, got) : r + got;
  }
  return r;
}

// ------------------------------------------------------------------ work
struct Seq {
  int len, cnt, ctx, items, tiles;            // items: row blocks to serve; tiles per item
};
__device__ __forceinline__ Seq seq_info(const TreeParams& p, int b, bool report) {
  Seq s;
  s.cnt = p.counts ? __ldg(p.counts + b) : p.n;
  s.len = __ldg(p.lengths + b);
  if (s.cnt < 0 || s.cnt > p.n || s.len < s.cnt || s.len > p.max_len) {
    if (report) raise_error(p.err, IDX_DEV_ERR_LENGTH);
    s.cnt = s.len = 0;
  }
  s.ctx = s.len - s.cnt;
  s.items = p.indices ? s.cnt * p.blocks : s.cnt > 0 ? p.blocks : 0;
  s.tiles = (static_cast<int>(p.indices ? p.k + s.cnt : s.len) + kTile - 1) / kTile;
  return s;
}

// drafts that a token's rows see
__device__ __forceinline__ uint64_t draft_mask(const TreeParams& p, int b, int i, int cnt) {
  const uint64_t all = cnt >= 64 ? ~0ull : (1ull << cnt) - 1;
  const uint64_t m = p.mask ? __ldg(reinterpret_cast<const unsigned long long*>(p.mask) + static_cast<int64_t>(b) * p.n + i)
                            : (2ull << i) - 1;
  return m & all;
}

template <int N>
__global__ void __launch_bounds__(Cfg<N>::kThreads, 1)
    tree_mla_kernel(const __grid_constant__ CUtensorMap tmap_q, const TreeParams p) {
  using C = Cfg<N>;
  constexpr int NC = C::kNC, kThreads = C::kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc<N>& ms = *reinterpret_cast<Misc<N>*>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / p.team, rank = blockIdx.x % p.team;
  const uint64_t budget = p.budget_ns;
  volatile int* abort_flag = &ms.abort_flag;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kPairs; ++i) {
      mbar_init(&ms.pair_full[i], kCopyWarps * 32);
      mbar_init(&ms.pair_empty[i], 1);
    }
    for (int i = 0; i < C::kRopes; ++i) {
      mbar_init(&ms.rope_full[i], kCopyWarps * 32);
      mbar_init(&ms.rope_empty[i], 1);
    }
    mbar_init(&ms.q_full, 1);
    mbar_init(&ms.q_empty, 1);
    mbar_init(&ms.s_full, 1);
    mbar_init(&ms.p_full, C::kSoftWarps);
    mbar_init(&ms.o_full, 1);
    mbar_init(&ms.o_free, C::kSoftWarps);
    mbar_init(&ms.drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.tile_full[i], 1);
      mbar_init(&ms.tile_read[i], kCopyWarps + C::kSoftWarps);
      mbar_init(&ms.piece_full[i], 1);
      mbar_init(&ms.piece_empty[i], C::kSoftWarps + 1);
    }
    ms.abort_flag = 0;
    ms.start_b = p.B;
    ms.start_off = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == 1) tmem_alloc(&ms.tmem, C::kTmemCols);

  // ---- where this team's share begins: every thread adds up a run of sequences
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, static_cast<int>(threadIdx.x) * per), b_hi = min(p.B, b_lo + per);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s = seq_info(p, b, blockIdx.x == 0);
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
  const long long share = max(static_cast<long long>(p.whole ? 1 : kMinShare), (total + p.teams - 1) / p.teams);
  const long long begin = min(total, share * team), end = min(total, begin + share);
  if (begin < end && before + incl - mine <= begin && begin < before + incl) {
    long long at = before + incl - mine;
    for (int b = b_lo; b < b_hi; ++b) {
      const Seq s = seq_info(p, b, false);
      const long long w = static_cast<long long>(s.items) * (p.whole ? 1 : s.tiles);
      if (begin < at + w) {
        ms.start_b = b;
        ms.start_off = begin - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  const uint32_t tmem = ms.tmem;
  const uint32_t smem_base = smem_u32(smem);
  if (warp == 0) {
    // ================================================================ planner
    bool ok = true;
    int tiles = 0, pieces = 0;                             // running counts
    long long cur = begin;
    int b = ms.start_b;
    long long off = ms.start_off;
    Cut cut{0, 0, 0};
    // waits of the whole warp: lane 0 polls
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      int w = 1;
      if (lane == 0) w = mbar_wait_polling(bar, parity, budget, abort_flag, p.err) ? 1 : 0;
      w = __shfl_sync(0xFFFFFFFFu, w, 0);
      __syncwarp();
      return w != 0;
    };
    Seq s{};
    if (b < p.B) s = seq_info(p, b, false);
    while (ok && cur < end) {
      const int weight = p.whole ? 1 : s.tiles;
      if (off >= static_cast<long long>(s.items) * weight) {
        ++b;
        if (b >= p.B) break;                               // (the share ends inside the batch)
        s = seq_info(p, b, false);
        off = 0;
        continue;
      }
      const int item = static_cast<int>(off / weight);
      const int t0 = p.whole ? 0 : static_cast<int>(off - static_cast<long long>(item) * weight);
      const int t1 = p.whole ? s.tiles : static_cast<int>(min(static_cast<long long>(s.tiles), t0 + (end - cur)));
      const int step = p.whole ? 1 : t1 - t0;
      off += step;
      cur += step;
      // the rows of this CTA: group of N flattened (token, head) rows of the
      // sequence, or of heads of one token where each token has its selection
      const int tok = p.indices ? item / p.blocks : 0;
      const int blk = p.indices ? item % p.blocks : item;
      const int64_t lo = (static_cast<int64_t>(blk) * p.team + rank) * N;
      const int64_t have = p.indices ? p.H : static_cast<int64_t>(s.cnt) * p.H;
      const int rows = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(N), have - lo)));
      const int64_t row0 = (static_cast<int64_t>(b) * p.n + tok) * p.H + lo;
      const int slot = t0 == 0 && t1 == s.tiles ? -1 : t0 == 0 ? 1 : 0;
      if (slot == 1) {
        cut.row0 = row0;
        cut.rows = rows;
        cut.pieces = static_cast<int>((s.tiles - t1 + share - 1) / share);
      }
      if (rows == 0) continue;                             // fewer rows than the team has groups
      // ---- publish the piece: what each column sees of the drafts
      const int pb = pieces & 1;
      if (pieces >= 2 && !(ok = wait(&ms.piece_empty[pb], ((pieces >> 1) - 1) & 1))) break;
      uint64_t any = 0;
      for (int c = lane; c < N; c += 32) {
        const uint64_t m =
            c < rows ? draft_mask(p, b, p.indices ? tok : static_cast<int>((lo + c) / p.H), s.cnt) : 0;
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
        pc.mixed = !p.indices && lo / p.H != (lo + rows - 1) / p.H;
        pc.row0 = row0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.piece_full[pb]);
      // ---- its tiles: lane ↔ keys 4·lane … 4·lane + 3.  The positions of tile
      // t + 2 and the page numbers of tile t + 1 are fetched while tile t is issued
      const int32_t* sel = p.indices ? p.indices + (static_cast<int64_t>(b) * p.n + tok) * p.k : nullptr;
      const int32_t* pages = p.table + static_cast<int64_t>(b) * p.max_pages;
      const int nkeys = p.indices ? p.k : s.ctx;           // keys before the drafts
      auto page_of = [&](int pos) {
        return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(pos)) * p.div_mul >> p.div_shift);
      };
      auto position = [&](int t, int e) {                  // position of a key, −1 where it selects nothing
        const int v = t * kTile + 4 * lane + e;
        if (v >= nkeys) return v - nkeys < s.cnt && ((any >> (v - nkeys)) & 1) ? s.ctx + v - nkeys : -1;
        if (!sel) return v;
        return t < t1 ? __ldg(sel + v) : -1;
      };
      auto valid = [&](int t, int e, int pos) {            // a selection names context positions only
        return pos >= 0 && (t * kTile + 4 * lane + e >= nkeys || pos < s.ctx);
      };
      int pos_next[4], page_next[4], pos_far[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pos_next[e] = position(t0, e);
        if (!valid(t0, e, pos_next[e])) pos_next[e] = -1;
        pos_far[e] = position(t0 + 1, e);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        page_next[e] = pos_next[e] >= 0 ? __ldg(pages + page_of(pos_next[e])) : 0;
      for (int t = t0; t < t1 && ok; ++t) {
        int row[4];
        uint32_t kinds = 0;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = t * kTile + 4 * lane + e;
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
          for (int e = 0; e < 4; ++e) {
            pos_next[e] = valid(t + 1, e, pos_far[e]) ? pos_far[e] : -1;
            page_next[e] = pos_next[e] >= 0 ? __ldg(pages + page_of(pos_next[e])) : 0;
            pos_far[e] = position(t + 2, e);
          }
        }
        const int par = tiles & 1;
        // free once the copies and the softmax have read what it said two tiles ago
        if (tiles >= 2 && !(ok = wait(&ms.tile_read[par], ((tiles >> 1) - 1) & 1))) break;
        *reinterpret_cast<uint32_t*>(&ms.kind[par][4 * lane]) = kinds;
        *reinterpret_cast<int4*>(&ms.row[par][4 * lane]) = make_int4(row[0], row[1], row[2], row[3]);
        if (lane == 0) ms.last[par] = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.tile_full[par]);
        ++tiles;
        if (t == t0) {                                     // its queries, once the last piece's are no longer read
          if (pieces >= 1 && !(ok = wait(&ms.q_empty, (pieces - 1) & 1))) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&ms.q_full, 9 * N * 128);
            for (int c = 0; c < 9; ++c)
              tma_box(smem_base + C::kOffQ + c * N * 128, &tmap_q, smem_u32(&ms.q_full), c * 64, static_cast<int>(row0));
          }
          __syncwarp();
          ++pieces;
        }
      }
    }
    // the end of the list
    if (ok) {
      const int pb = pieces & 1;
      if (pieces >= 2) ok = wait(&ms.piece_empty[pb], ((pieces >> 1) - 1) & 1);
      if (ok && lane == 0) {
        ms.piece[pb].t0 = ms.piece[pb].t1 = 0;
        mbar_arrive(&ms.piece_full[pb]);
      }
      const int par = tiles & 1;
      if (ok && tiles >= 2) ok = wait(&ms.tile_read[par], ((tiles >> 1) - 1) & 1);
      if (ok && lane == 0) {
        ms.last[par] = 1;
        mbar_arrive(&ms.tile_full[par]);
      }
    }
    if (!p.whole && lane == 0) p.cuts[blockIdx.x] = cut;
    if (lane == 0 && pieces) {                             // the queries have landed before the memory goes
      int dummy = 0;
      mbar_wait(&ms.q_full, (pieces - 1) & 1, budget, &dummy, p.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    constexpr uint32_t id_s = idesc_bf16(N, false), id_o = idesc_bf16(N, true);
    const uint32_t d_s = tmem + 4 * N;
    const uint64_t q_desc = smem_desc_k128_sw128(smem_base + C::kOffQ);
    const uint64_t k_desc = smem_desc_k128_sw128(smem_base);
    const uint64_t v_desc = desc_mn(smem_base, kChunk);
    const uint64_t p_desc = desc_mn(smem_base + C::kOffP, kChunk);
    bool ok = true, issued = false;
    int pairs = 0, ropes = 0, tiles = 0, pieces = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_polling(bar, parity, budget, abort_flag, p.err); };
    while (true) {
      const int pb = pieces & 1;
      if (!(ok = wait(&ms.piece_full[pb], (pieces >> 1) & 1))) break;
      const int t0 = ms.piece[pb].t0, t1 = ms.piece[pb].t1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.piece_empty[pb]);
      if (t0 == t1) break;
      if (!(ok = wait(&ms.q_full, pieces & 1))) break;
      for (int t = t0; t < t1 && ok; ++t) {
        // Sᵀ = K · qᵀ
        const int first = pairs;
        for (int u = 0; u < 4 && ok; ++u) {
          const int sl = (first + u) % C::kPairs;
          if (!(ok = wait(&ms.pair_full[sl], ((first + u) / C::kPairs) & 1))) break;
          fence_proxy_async_smem();                        // the copies wrote through the generic proxy
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a = k_desc + static_cast<uint64_t>(sl * (kPair >> 4));
            const uint64_t q = q_desc + static_cast<uint64_t>(u * (2 * N * 128 >> 4));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_f16(d_s, a + static_cast<uint64_t>((i >> 2) * (kChunk >> 4) + (i & 3) * 2),
                      q + static_cast<uint64_t>((i >> 2) * (N * 128 >> 4) + (i & 3) * 2), id_s, (u > 0 || i > 0) ? 1u : 0u);
          }
          issued = true;
          __syncwarp();
        }
        if (!ok) break;
        const int rs = ropes % C::kRopes;
        if (!(ok = wait(&ms.rope_full[rs], (ropes / C::kRopes) & 1))) break;
        fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = k_desc + static_cast<uint64_t>((C::kOffRope + rs * kChunk) >> 4);
          const uint64_t q = q_desc + static_cast<uint64_t>(8 * N * 128 >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_f16(d_s, a + i * 2, q + i * 2, id_s, 1u);
          mma_commit(&ms.s_full);
          if (!C::kAliasP) mma_commit(&ms.rope_empty[rs]);
          if (t == t1 - 1) mma_commit(&ms.q_empty);
        }
        __syncwarp();
        // Oᵀ += Vᵀ · Pᵀ
        if (!(ok = wait(&ms.p_full, tiles & 1))) break;
        if (t == t0 && pieces > 0 && !(ok = wait(&ms.o_free, (pieces - 1) & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t acc = t > t0 ? 1u : 0u;
          for (int u = 0; u < 4; ++u) {
            const int sl = (first + u) % C::kPairs;
            const uint64_t a = v_desc + static_cast<uint64_t>(sl * (kPair >> 4));
#pragma unroll
            for (int i = 0; i < 8; ++i)                    // 16 keys per instruction: two 8-row atoms
              mma_f16(tmem + u * N, a + i * (2048 >> 4), p_desc + i * (2048 >> 4), id_o, i > 0 ? 1u : acc);
            mma_commit(&ms.pair_empty[sl]);
          }
          if (C::kAliasP) mma_commit(&ms.rope_empty[rs]);
          if (t == t1 - 1) mma_commit(&ms.o_full);
        }
        __syncwarp();
        pairs += 4;
        ++ropes;
        ++tiles;
      }
      if (!ok) break;
      ++pieces;
    }
    if (issued) {
      if (elect_one()) mma_commit(&ms.drain);
      __syncwarp();
      int dummy = 0;
      mbar_wait(&ms.drain, 0, budget, &dummy, p.err);
    }
    __syncwarp();
  } else if (warp < 2 + kCopyWarps) {
    // ================================================================ copies
    // A warp instruction copies 256 bytes of two rows: lanes 0-15 key 2·w + 8·j,
    // lanes 16-31 the next; piece c of row r goes to (c mod 8) ^ (r mod 8) of its
    // 128-byte row, the swizzle that the descriptors name
    const int key0 = 2 * (warp - 2) + (lane >> 4);
    const int piece = lane & 15;
    const uint32_t to_pair = smem_base + (piece >> 3) * kChunk + key0 * 128 + (((piece & 7) ^ (key0 & 7)) << 4);
    // rotary chunk: lanes ↔ four rows of 8 pieces
    const int key1 = 4 * (warp - 2) + (lane >> 3);
    const uint32_t to_rope = smem_base + C::kOffRope + key1 * 128 + (((lane & 7) ^ (key1 & 7)) << 4);
    const uint8_t* from = reinterpret_cast<const uint8_t*>(p.cache);
    int pairs = 0, ropes = 0, tiles = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      int w = 1;
      if (lane == 0) w = mbar_wait_polling(bar, parity, budget, abort_flag, p.err) ? 1 : 0;
      w = __shfl_sync(0xFFFFFFFFu, w, 0);
      __syncwarp();
      return w != 0;
    };
    bool ok = true;
    while (ok) {
      const int par = tiles & 1;
      if (!wait(&ms.tile_full[par], (tiles >> 1) & 1) || ms.last[par]) break;
      int row[kTile / 8], rope_row[kTile / 16];
#pragma unroll
      for (int j = 0; j < kTile / 8; ++j) row[j] = ms.row[par][key0 + 8 * j];
#pragma unroll
      for (int j = 0; j < kTile / 16; ++j) rope_row[j] = ms.row[par][key1 + 16 * j];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.tile_read[par]);
      for (int u = 0; u < 4; ++u) {
        const int sl = pairs % C::kPairs;
        if (pairs >= C::kPairs && !(ok = wait(&ms.pair_empty[sl], (pairs / C::kPairs - 1) & 1))) break;
        const uint32_t to = to_pair + sl * kPair;
        const uint8_t* src = from + u * 256 + piece * 16;
#pragma unroll
        for (int j = 0; j < kTile / 8; ++j)
          cp_async16(to + j * 1024, src + static_cast<int64_t>(max(row[j], 0)) * (2 * kRow), row[j] >= 0 ? 16 : 0);
        cp_async_arrive(&ms.pair_full[sl]);
        ++pairs;
      }
      if (!ok) break;
      const int sl = ropes % C::kRopes;
      if (ropes >= C::kRopes && !(ok = wait(&ms.rope_empty[sl], (ropes / C::kRopes - 1) & 1))) break;
      const uint32_t to = to_rope + sl * kChunk;
      const uint8_t* src = from + 2 * kLat + (lane & 7) * 16;
#pragma unroll
      for (int j = 0; j < kTile / 16; ++j)
        cp_async16(to + j * 2048, src + static_cast<int64_t>(max(rope_row[j], 0)) * (2 * kRow), rope_row[j] >= 0 ? 16 : 0);
      cp_async_arrive(&ms.rope_full[sl]);
      ++ropes;
      ++tiles;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");       // they have landed before the memory goes
  } else if (warp >= kFirstSoft) {
    // ================================================================ softmax
    constexpr int kColShift = NC == 16 ? 1 : 2;
    const int sw = warp - kFirstSoft, quad = warp & 3, part_id = sw >> 2;
    const int key = quad * 32 + lane;
    const int my_col = lane >> kColShift;                  // the column this lane keeps statistics of
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_addr = lanes + 4 * N + part_id * NC;
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80000000u : 0u;
    const float scale = fmaxf(fabsf(p.scale_log2), 1.1754944e-38f);   // (never 0 · −inf)
    uint8_t* p_row = smem + C::kOffP + key * 128;
    bool ok = true;
    int tiles = 0, pieces = 0, pairs = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      int w = 1;
      if (lane == 0) w = mbar_wait_polling(bar, parity, budget, abort_flag, p.err) ? 1 : 0;
      w = __shfl_sync(0xFFFFFFFFu, w, 0);
      __syncwarp();
      return w != 0;
    };
    while (true) {
      const int pb = pieces & 1;
      if (!(ok = wait(&ms.piece_full[pb], (pieces >> 1) & 1))) break;
      const Piece pc = ms.piece[pb];
      if (pc.t0 == pc.t1) break;
      float m = -INFINITY;                                 // reference maximum of column my_col, log2 units
      float l[NC];                                         // sums of this key's weights, before their rounding
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;
      ms.m[sw][my_col] = 0.f;
      for (int t = pc.t0; t < pc.t1; ++t, ++tiles, pairs += 4) {
        if (!(ok = wait(&ms.tile_full[tiles & 1], (tiles >> 1) & 1))) break;
        const int kind = ms.kind[tiles & 1][key];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.tile_read[tiles & 1]);
        const bool all_seen = __all_sync(0xFFFFFFFFu, kind == 1);
        const bool drafts = __any_sync(0xFFFFFFFFu, kind >= 2);
        if (!(ok = wait(&ms.s_full, tiles & 1))) break;
        tc_fence_after();
        uint32_t r[NC];
        tmem_ld<NC>(s_addr, r);
        tmem_wait();
        regs_ready<NC>(r);
        // the scores of a negative scale are compared with their signs turned
        float z[NC], v[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) z[c] = __uint_as_float(r[c] ^ flip);
        if (!all_seen) {
          if (kind == 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c) z[c] = -INFINITY;
          }
          if (drafts) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const uint64_t bits = ms.mask[pb][part_id * NC + c];
              if (kind >= 2 && !((bits >> (kind - 2)) & 1)) z[c] = -INFINITY;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) v[c] = z[c];
        const float wm = reduce_columns<NC, true>(v, lane);
        ms.wmax[tiles & 1][part_id][quad][my_col] = wm;
        bar_part(part_id);
        float top = ms.wmax[tiles & 1][part_id][0][my_col];
#pragma unroll
        for (int w = 1; w < 4; ++w) top = fmaxf(top, ms.wmax[tiles & 1][part_id][w][my_col]);
        top = top == -INFINITY ? top : top * scale;
        const bool raise = top > m + kRaise || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(0xFFFFFFFFu, raise)) {              // the same in the part's four warps
          const float a = !raise ? 1.f : m == -INFINITY ? 0.f : ex2(m - top);
          if (raise) m = top;
          ms.alpha[sw][my_col] = a;
          ms.m[sw][my_col] = m == -INFINITY ? 0.f : m;
          __syncwarp();
#pragma unroll
          for (int c = 0; c < NC; ++c) l[c] *= ms.alpha[sw][c];
          if (t > pc.t0) {                                 // (the scores' arrival implies the last product's end)
#pragma unroll 1
            for (int blk = 0; blk < 4; ++blk) {
              uint32_t o[NC];
              const uint32_t oa = lanes + blk * N + part_id * NC;
              tmem_ld<NC>(oa, o);
              tmem_wait();
              regs_ready<NC>(o);
#pragma unroll
              for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * ms.alpha[sw][c]);
              tmem_st<NC>(oa, o);
            }
            tmem_wait_st();
          }
        }
        // P row of this key: NC bf16, 128-byte swizzle
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          uint32_t w[4];
          const float4 m0 = *reinterpret_cast<const float4*>(&ms.m[sw][c]);
          const float4 m1 = *reinterpret_cast<const float4*>(&ms.m[sw][c + 4]);
          const float mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p0 = ex2(fmaf(z[c + 2 * e], scale, -mm[2 * e]));
            const float p1 = ex2(fmaf(z[c + 2 * e + 1], scale, -mm[2 * e + 1]));
            w[e] = bf_pack(p0, p1);
            l[c + 2 * e] += p0;
            l[c + 2 * e + 1] += p1;
          }
          *reinterpret_cast<uint4*>(p_row + (((part_id * NC + c) / 8) ^ (key & 7)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // a draft's row that only some columns see must not reach the others as
        // 0 · NaN: where it is not finite it becomes zero (the columns that see
        // it have it in their weights already)
        if (pc.mixed && drafts && part_id == 0) {
          for (int u = 0; u < 4 && ok; ++u)
            ok = wait(&ms.pair_full[(pairs + u) % C::kPairs], ((pairs + u) / C::kPairs) & 1);
          if (!ok) break;
          if (kind >= 2) {
            bool wild = false;
            for (int j = 0; j < 64; ++j) {
              const uint4 x = *reinterpret_cast<const uint4*>(smem + ((pairs + (j >> 4)) % C::kPairs) * kPair +
                                                              ((j >> 3) & 1) * kChunk + key * 128 + (j & 7) * 16);
              const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                wild |= (e[i] & 0x7F80u) == 0x7F80u || (e[i] & 0x7F800000u) == 0x7F800000u;
            }
            if (wild)
              for (int j = 0; j < 64; ++j)
                *reinterpret_cast<uint4*>(smem + ((pairs + (j >> 4)) % C::kPairs) * kPair + ((j >> 3) & 1) * kChunk +
                                          key * 128 + (j & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full);
      }
      if (!ok) break;
      // ---- the sums over all keys
      ms.sum[part_id][quad][my_col] = reduce_columns<NC, false>(l, lane);
      bar_part(part_id);
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) z += ms.sum[part_id][w][my_col];
      const bool whole = pc.slot < 0;
      float* part = whole ? nullptr : p.part + (static_cast<int64_t>(blockIdx.x) * 2 + pc.slot) * (N * (kLat + 2));
      ms.alpha[sw][my_col] = whole ? (z == 0.f ? 0.f : 1.f / z) : 1.f;
      if (quad == 0 && (lane & ((1 << kColShift) - 1)) == 0) {
        const int c = part_id * NC + my_col;
        if (!whole) {
          part[N * kLat + c] = m;
          part[N * kLat + N + c] = z;
        } else if (p.lse && c < pc.rows) {
          p.lse[pc.row0 + c] = m == -INFINITY && z == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * kLn2) + logf(z);
        }
      }
      __syncwarp();
      if (!(ok = wait(&ms.o_full, pieces & 1))) break;
      tc_fence_after();
#pragma unroll 1
      for (int blk = 0; blk < 4; ++blk) {
        uint32_t o[NC];
        tmem_ld<NC>(lanes + blk * N + part_id * NC, o);
        tmem_wait();
        regs_ready<NC>(o);
        const int d = blk * 128 + key;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float x = __uint_as_float(o[c]) * ms.alpha[sw][c];
          const int col = part_id * NC + c;
          if (!whole) {
            part[col * kLat + d] = x;
          } else if (col < pc.rows) {
            if (p.out_bf16)
              static_cast<__nv_bfloat16*>(p.out)[(pc.row0 + col) * kLat + d] = __float2bfloat16_rn(x);
            else
              static_cast<float*>(p.out)[(pc.row0 + col) * kLat + d] = x;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.o_free);
        mbar_arrive(&ms.piece_empty[pb]);
      }
      ++pieces;
    }
  }
  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the pieces of the items that shares cut: CTA (x, y) takes rows y, y + 8, …
// of the item that begins in CTA x's share and goes on in the next teams'.  Four
// groups of 128 threads walk every fourth piece, lane ↔ four output features;
// their sums are added in a fixed order.
constexpr int kJoinGroups = 4, kJoinY = 8;
template <int N>
__global__ void __launch_bounds__(kJoinGroups * 128) tree_mla_join_kernel(const TreeParams p) {
  __shared__ float4 acc[kJoinGroups][128];
  __shared__ float sums[kJoinGroups];
  const Cut cut = p.cuts[blockIdx.x];
  if (!cut.pieces) return;
  const int group = threadIdx.x >> 7, d = threadIdx.x & 127;
  const int team = blockIdx.x / p.team, rank = blockIdx.x % p.team;
  auto slot = [&](int i) {                     // piece 0 is this team's slot 1, the others the next teams' slot 0
    return p.part + (static_cast<int64_t>((team + i) * p.team + rank) * 2 + (i == 0 ? 1 : 0)) * (N * (kLat + 2));
  };
  for (int c = blockIdx.y; c < cut.rows; c += kJoinY) {
    float top = -INFINITY;
    for (int i = 0; i <= cut.pieces; ++i) top = fmaxf(top, slot(i)[N * kLat + c]);
    const float base = top == -INFINITY ? 0.f : top;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float z = 0.f;
#pragma unroll 4
    for (int i = group; i <= cut.pieces; i += kJoinGroups) {
      const float* s = slot(i);
      const float w = ex2(s[N * kLat + c] - base);
      const float4 x = *reinterpret_cast<const float4*>(s + c * kLat + d * 4);
      o.x += w * x.x;
      o.y += w * x.y;
      o.z += w * x.z;
      o.w += w * x.w;
      z += w * s[N * kLat + N + c];
    }
    acc[group][d] = o;
    if (d == 0) sums[group] = z;
    __syncthreads();
    if (group == 0) {
      z = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kJoinGroups; ++g) {
        const float4 x = acc[g][d];
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
        z += sums[g];
      }
      const float inv = z == 0.f ? 0.f : 1.f / z;
      const int64_t at = (cut.row0 + c) * kLat + d * 4;
      if (p.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
            make_uint2(bf_pack(o.x * inv, o.y * inv), bf_pack(o.z * inv, o.w * inv));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (p.lse && d == 0) p.lse[cut.row0 + c] = top == -INFINITY && z == 0.f ? -INFINITY : base * kLn2 + logf(z);
    }
    __syncthreads();
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// How a call's rows and tiles are dealt: N rows per CTA (the fewest columns that
// hold the rows which share keys, at most 64), teams of CTAs over the row groups.
struct Plan {
  int N, team, blocks, teams, whole;
  size_t ws;
};
Plan plan_for(int n, int H, int max_len, int k, int sms) {
  Plan pl;
  const int64_t rows = k ? H : static_cast<int64_t>(n) * H;
  pl.N = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  const int64_t groups = (rows + pl.N - 1) / pl.N;
  pl.blocks = static_cast<int>((groups + kMaxTeam - 1) / kMaxTeam);
  pl.team = static_cast<int>((groups + pl.blocks - 1) / pl.blocks);
  pl.teams = sms / pl.team > 0 ? sms / pl.team : 1;
  const int64_t tiles = ((k ? static_cast<int64_t>(k) + n : max_len) + kTile - 1) / kTile;
  pl.whole = tiles <= kMinShare || pl.teams == 1;
  const size_t ctas = static_cast<size_t>(pl.teams) * pl.team;
  pl.ws = pl.whole ? 0 : ctas * 2 * pl.N * (kLat + 2) * sizeof(float) + ctas * sizeof(Cut);
  return pl;
}

template <int N>
int launch(const CUtensorMap& tq, const TreeParams& p, int ctas, cudaStream_t stream) {
  constexpr int smem = 1024 + Cfg<N>::kOffMisc + static_cast<int>(sizeof(Misc<N>));
  static_assert(smem <= 227 * 1024, "shared memory");
  if (const int r = ensure_smem_limit(reinterpret_cast<const void*>(tree_mla_kernel<N>), smem)) return r;
  tree_mla_kernel<N><<<static_cast<unsigned>(ctas), Cfg<N>::kThreads, smem, stream>>>(tq, p);
  if (const int r = check_launch()) return r;
  if (p.whole) return IDX_OK;
  tree_mla_join_kernel<N><<<dim3(static_cast<unsigned>(ctas), kJoinY), kJoinGroups * 128, 0, stream>>>(p);
  return check_launch();
}

}  // namespace
}  // namespace idx

using namespace idx;

extern "C" size_t idx_tree_mla_workspace_size(int B, int n, int H, int max_len, int k) {
  if (B <= 0 || n <= 0 || n > IDX_MAX_DRAFTS || H <= 0 || max_len <= 0 || k < 0) return 0;
  return plan_for(n, H, max_len, k, num_sms()).ws;
}

extern "C" int idx_tree_mla(const uint16_t* q, const uint16_t* cache, const int32_t* page_table, int max_pages,
                            int num_pages, int page_size, const int32_t* lengths, const int32_t* counts, int B, int n,
                            int H, int max_len, const uint64_t* tree_mask, const int32_t* indices, int k,
                            float softmax_scale, void* out, int out_dtype, float* lse, void* ws, size_t ws_bytes,
                            idx_stream_t stream) {
  constexpr int64_t kMaxRows = 0x7FFFFFFF;
  if (out_dtype != IDX_OUT_F32 && out_dtype != IDX_OUT_BF16) return IDX_ERR_FMT;
  if (B < 0 || n < 0 || n > IDX_MAX_DRAFTS || H <= 0 || k < 0 || k > kMaxRows - kTile - IDX_MAX_DRAFTS ||
      !std::isfinite(softmax_scale))
    return IDX_ERR_SHAPE;
  if (B == 0 || n == 0) return IDX_OK;
  if (max_pages <= 0 || num_pages <= 0 || page_size <= 0 || static_cast<int64_t>(num_pages) * page_size > kMaxRows ||
      static_cast<int64_t>(max_pages) * page_size > kMaxRows)
    return IDX_ERR_SHAPE;
  if (max_len <= 0 || max_len > static_cast<int64_t>(max_pages) * page_size || max_len > kMaxRows - 2 * kTile)
    return IDX_ERR_SHAPE;
  if ((k > 0) != (indices != nullptr)) return indices ? IDX_ERR_K : IDX_ERR_NULL;
  if (!q || !cache || !page_table || !lengths || !out) return IDX_ERR_NULL;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(ws, 16) || !aligned(tree_mask, 8))
    return IDX_ERR_ALIGN;
  const int64_t rows = static_cast<int64_t>(B) * n;
  if (rows > kMaxRows / H) return IDX_ERR_SHAPE;
  const Plan pl = plan_for(n, H, max_len, k, num_sms());
  if (pl.ws > 0 && !ws) return IDX_ERR_NULL;
  if (ws_bytes < pl.ws) return IDX_ERR_SCRATCH;
  const int ctas = pl.teams * pl.team;
  CUtensorMap tq;
  if (!make_tmap_2d_bf16_sw128(&tq, q, kRow, static_cast<uint64_t>(rows) * H, static_cast<uint32_t>(pl.N)))
    return IDX_ERR_UNSUPPORTED;
  TreeParams p;
  p.table = page_table;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.cache = cache;
  // s = ⌈log2 d⌉, m = ⌊2^(31+s)/d⌋ + 1: x·m >> (31+s) is x / d for every x < 2^31
  int sh = 0;
  while ((int64_t{1} << sh) < page_size) ++sh;
  p.div_mul = static_cast<uint32_t>((uint64_t{1} << (31 + sh)) / static_cast<uint64_t>(page_size) + 1);
  p.div_shift = 31 + sh;
  p.lengths = lengths;
  p.counts = counts;
  p.B = B;
  p.n = n;
  p.H = H;
  p.max_len = max_len;
  p.mask = tree_mask;
  p.indices = indices;
  p.k = k;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = out;
  p.out_bf16 = out_dtype == IDX_OUT_BF16;
  p.lse = lse;
  p.team = pl.team;
  p.blocks = pl.blocks;
  p.teams = pl.teams;
  p.whole = pl.whole;
  p.part = static_cast<float*>(ws);
  p.cuts = reinterpret_cast<Cut*>(static_cast<uint8_t*>(ws) +
                                  static_cast<size_t>(ctas) * 2 * pl.N * (kLat + 2) * sizeof(float));
  p.budget_ns = debug_state().budget_ns;
  p.err = device_error_word();
  if (!p.err) return check_launch();
  auto* s = reinterpret_cast<cudaStream_t>(stream);
  return pl.N == 16   ? launch<16>(tq, p, ctas, s)
         : pl.N == 32 ? launch<32>(tq, p, ctas, s)
                      : launch<64>(tq, p, ctas, s);
}
