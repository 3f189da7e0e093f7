// Latent attention of drafted token trees over the paged cache (idx_tree_mla),
// for at most 64 rows (tokens · heads, or heads where each token has its own
// selection) per set of keys:
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
// delivers to one SM in about 5 700.  Rows from HBM bind small N (16 x 131 000
// positions, 16 heads: 86% of its rate); rows from L2 leave the chain of one tile, its
// last copy, scores, softmax and product, 5 400 cycles, since shared memory holds one
// tile and a quarter.
//
// One CTA, 15 warps (23 for N = 64):
//   warp 0     the planner (tree_mla.cuh);
//   warps 1, 2 issue the MMAs of the scores and of the products (two warps, since what
//              one asks of a barrier waits behind the MMAs that it has queued): the
//              product of tile t frees the latent buffers one by one, and tile t + 1
//              streams into them and through the scores;
//   warps 3-6  copy the tiles' rows by cp.async, 16 bytes a lane; a key that no row
//              sees arrives as zeros, never as what memory holds.  (TMA delivers these
//              1 152-byte rows at 25 B/clk per SM in boxes and 9 – 20 gathered, cp.async
//              at 34 – 70 with 4 – 16 warps from L2 and 26 from HBM, its limit.  Asking
//              for selected rows in L2 ahead of the copies was measured, up to four tiles
//              ahead, by lines and by rows: 5 – 10% less time where HBM is idle (16 x 7
//              tokens), up to 17% more where it is not (128 tokens with rows of their own).)
//              A key set's rows are read by one CTA (tokens of a sequence may share
//              selected rows), so they are the first to leave L2: 128 tokens of 2 048 rows 84 -> 74 us, 16 x 131 000 positions
//              242 -> 239; in the wide kernel, where two CTAs read them, 139 -> 150;
//   warps 7 …  softmax: thread ↔ (key, part of the rows).  Scores are compared with
//              a running reference maximum per row as it is; only where one passes it
//              by 2^8 (a piece's first tile always) the column maxima are reduced, by a
//              transposing butterfly across lanes and shared memory across warps, the
//              reference is raised and O in TMEM rescaled.  P = 2^(s − m) in bf16 for
//              the tensor cores (a relative 2^-8 per weight); the sum that divides O and
//              stands behind lse adds the weights before that rounding, in fp32.
// Every wait is bounded; a CTA that gives up raises IDX_DEV_ERR_TIMEOUT, waits for
// its copies and MMAs, frees TMEM and returns.
#include "tree_mla.cuh"

namespace idx {
namespace {

using namespace tree;

constexpr int kTile = 128;                    // keys per tile
constexpr int kPair = 32768;                  // 128 keys × 128 latent features: two 64-feature chunks
constexpr int kChunk = 16384;                 // 128 keys × 64 features
constexpr int kCopyWarps = 4;                 // warps that copy the tiles
constexpr int kFirstCopy = 3;                 // planner, the two MMA issuers, copies, then the softmax
constexpr int kFirstSoft = kFirstCopy + kCopyWarps;

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

template <int N>
struct Misc : PlanState<N, kTile, Cfg<N>::kThreads / 32> {
  alignas(16) float wmax[Cfg<N>::kParts][4][Cfg<N>::kNC];   // row part, warp: column maxima
  alignas(16) float m[Cfg<N>::kSoftWarps][Cfg<N>::kNC];     // reference maxima (0 beyond kFar), a copy per softmax warp
  alignas(16) float alpha[Cfg<N>::kSoftWarps][Cfg<N>::kNC];
  alignas(16) float sum[Cfg<N>::kParts][4][Cfg<N>::kNC];
  uint64_t pair_full[5], pair_empty[5], rope_full[2], rope_empty[2];
  uint64_t s_full, s_free, p_full, p_free, o_full, o_free, drain_bar[2];
  int left_at[Cfg<N>::kParts];
};

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

// Draft j's row at `at` of the four latent buffers from `first` on: zeros where it is not finite
__device__ __forceinline__ void clear_wild(uint8_t* at, int first, int buffers, unsigned long long* wild, int j) {
  auto piece = [&](int i) {
    const int b = first + (i >> 4);
    return reinterpret_cast<uint4*>(at + (b < buffers ? b : b - buffers) * kPair + ((i >> 3) & 1) * kChunk + (i & 7) * 16);
  };
  bool any = false;
  for (int i = 0; i < 64; ++i) any |= not_finite(*piece(i));
  if (!any) return;
  atomicOr(wild, 1ull << j);
  for (int i = 0; i < 64; ++i) *piece(i) = make_uint4(0, 0, 0, 0);
}
// NaN into outputs key, 128 + key … of columns [c0, c0 + nc) that see a wild draft, where its features are not finite
__device__ __noinline__ void spoil_columns(const TreeParams& p, const Piece& pc, const uint64_t* mask, uint64_t wild,
                                           int key, int c0, int nc) {
  for (; wild; wild &= wild - 1) {
    const int j = __ffsll(static_cast<long long>(wild)) - 1;
    const uint16_t* src = draft_row(p, pc, j);
    for (int d = key; d < kLat; d += kTile) {
      if (!not_finite(src[d])) continue;
      for (int c = c0; c < min(c0 + nc, pc.rows); ++c)
        if ((mask[c] >> j) & 1)
          spoil(p, pc, c, d, pc.slot < 0 ? nullptr : part_slot(p, blockIdx.x, pc.slot) + c * kLat + d);
    }
  }
}

template <int N>
__global__ void __launch_bounds__(Cfg<N>::kThreads, 1)
    tree_mla_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ TreeParams p) {
  using C = Cfg<N>;
  constexpr int NC = C::kNC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc<N>& ms = *reinterpret_cast<Misc<N>*>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / p.halves;
  const Waits waits{p.budget_ns, &ms.abort_flag, p.err};

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kPairs; ++i) {
      mbar_init(&ms.pair_full[i], kCopyWarps * 32);
      mbar_init(&ms.pair_empty[i], 1);
    }
    for (int i = 0; i < C::kRopes; ++i) {
      mbar_init(&ms.rope_full[i], kCopyWarps * 32);
      mbar_init(&ms.rope_empty[i], 1);
    }
    mbar_init(&ms.s_full, 1);
    mbar_init(&ms.s_free, C::kSoftWarps);
    mbar_init(&ms.p_full, C::kSoftWarps);
    mbar_init(&ms.p_free, 1);
    mbar_init(&ms.o_full, 1);
    mbar_init(&ms.o_free, C::kSoftWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&ms.drain_bar[i], 1);
    for (int i = 0; i < C::kParts; ++i) ms.left_at[i] = 0;
    ms.init(p.B, kCopyWarps + C::kSoftWarps, C::kSoftWarps + 2);
    fence_barrier_init();
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == 1) tmem_alloc(&ms.tmem, C::kTmemCols);
  const Share share = find_share<N, kTile, C::kThreads>(p, ms, team);
  const uint32_t tmem = ms.tmem;
  const uint32_t smem_base = smem_u32(smem);

  if (warp == 0) {
    plan<N, kTile>(p, ms, share, waits, [&](int row0) {
      mbar_arrive_expect_tx(&ms.q_full, 9 * N * 128);
      for (int c = 0; c < 9; ++c)
        tma_box(smem_base + C::kOffQ + c * N * 128, &tmap_q, smem_u32(&ms.q_full), c * 64, row0);
    });
  } else if (warp == 1) {
    // ================================================================ scores
    // a negative scale turns the scores' signs here, so that the softmax sees a positive one
    const uint32_t id_s = idesc_bf16(N, false, false) | (p.scale_log2 < 0.f ? kNegateA : 0u);
    const uint32_t d_s = tmem + 4 * N;
    const uint64_t q_desc = smem_desc_k128_sw128(smem_base + C::kOffQ);
    const uint64_t k_desc = smem_desc_k128_sw128(smem_base);
    bool ok = true, issued = false;
    int slot = 0, lap = 0, tiles = 0, pieces = 0;          // latent buffer, times around; running counts
    while (true) {
      const int pb = pieces & 1;
      if (!(ok = waits(&ms.piece_full[pb], (pieces >> 1) & 1))) break;
      const int n = __reduce_max_sync(0xFFFFFFFFu, ms.piece[pb].t1 - ms.piece[pb].t0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.piece_empty[pb]);
      if (n == 0) break;
      if (!(ok = waits(&ms.q_full, pieces & 1))) break;
      for (int c = 0; c < n && ok; ++c) {
        // Sᵀ = K · qᵀ, once the softmax has read the last S, chunk by chunk as they land
        if (tiles >= 1 && !(ok = waits(&ms.s_free, (tiles - 1) & 1))) break;
        if ((p.fault & kFaultScores) && c == n - 1 && !(ok = waits(&ms.never, 0))) break;
        // (the rotary chunk first where its place is free since the last scores, so that
        // less follows the last copy; last where P held it)
        const int rs = tiles % C::kRopes;
        auto rope_scores = [&] {
          if (!(ok = waits(&ms.rope_full[rs], (tiles / C::kRopes) & 1))) return;
          fence_proxy_async_smem();                        // the copies wrote through the generic proxy
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a = k_desc + static_cast<uint64_t>((C::kOffRope + rs * kChunk) >> 4);
            const uint64_t q = q_desc + static_cast<uint64_t>(8 * N * 128 >> 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_f16(d_s, a + i * 2, q + i * 2, id_s, (C::kAliasP || i > 0) ? 1u : 0u);
            if (!C::kAliasP) mma_commit(&ms.rope_empty[rs]);
          }
          issued = true;
          __syncwarp();
        };
        if (!C::kAliasP) rope_scores();
        for (int u = 0; u < 4 && ok; ++u) {
          if (!(ok = waits(&ms.pair_full[slot], lap & 1))) break;
          fence_proxy_async_smem();
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a = k_desc + static_cast<uint64_t>(slot * (kPair >> 4));
            const uint64_t q = q_desc + static_cast<uint64_t>(u * (2 * N * 128 >> 4));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_f16(d_s, a + static_cast<uint64_t>((i >> 2) * (kChunk >> 4) + (i & 3) * 2),
                      q + static_cast<uint64_t>((i >> 2) * (N * 128 >> 4) + (i & 3) * 2), id_s,
                      (!C::kAliasP || u > 0 || i > 0) ? 1u : 0u);
          }
          issued = true;
          __syncwarp();
          if (++slot == C::kPairs) slot = 0, ++lap;
        }
        if (ok && C::kAliasP) rope_scores();
        if (!ok) break;
        if (elect_one()) {
          mma_commit(&ms.s_full);
          if (c == n - 1) mma_commit(&ms.q_empty);
        }
        __syncwarp();
        ++tiles;
      }
      if (!ok) break;
      ++pieces;
    }
    if (issued) {
      if (elect_one()) mma_commit(&ms.drain_bar[0]);
      __syncwarp();
      waits.drain(&ms.drain_bar[0], 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ================================================================ products
    constexpr uint32_t id_o = idesc_bf16(N, true, true);
    const uint64_t v_desc = desc_mn(smem_base, kChunk);
    const uint64_t p_desc = desc_mn(smem_base + C::kOffP, kChunk);
    bool ok = true, issued = false;
    int slot = 0, tiles = 0, pieces = 0;
    while (true) {
      const int pb = pieces & 1;
      if (!(ok = waits(&ms.piece_full[pb], (pieces >> 1) & 1))) break;
      const int n = __reduce_max_sync(0xFFFFFFFFu, ms.piece[pb].t1 - ms.piece[pb].t0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.piece_empty[pb]);
      if (n == 0) break;
      for (int c = 0; c < n; ++c) {
        // Oᵀ += Vᵀ · Pᵀ (the tile's scores, and so its V, were complete before its P)
        if (c == 0 && pieces > 0 && !(ok = waits(&ms.o_free, (pieces - 1) & 1))) break;
        if (!(ok = waits(&ms.p_full, tiles & 1))) break;
        fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          int sl = slot;
#pragma unroll 1
          for (int u = 0; u < 4; ++u) {
            const uint64_t a = v_desc + static_cast<uint64_t>(sl * (kPair >> 4));
#pragma unroll
            for (int i = 0; i < 8; ++i)                    // 16 keys per instruction: two 8-row atoms
              mma_f16(tmem + u * N, a + i * (2048 >> 4), p_desc + i * (2048 >> 4), id_o, (c > 0 || i > 0) ? 1u : 0u);
            mma_commit(&ms.pair_empty[sl]);
            if (++sl == C::kPairs) sl = 0;
          }
          mma_commit(&ms.p_free);
          if (C::kAliasP) mma_commit(&ms.rope_empty[tiles % C::kRopes]);
          if (c == n - 1) mma_commit(&ms.o_full);
        }
        issued = true;
        __syncwarp();
        slot = (slot + 4) % C::kPairs;
        ++tiles;
      }
      if (!ok) break;
      ++pieces;
    }
    if (issued) {
      if (elect_one()) mma_commit(&ms.drain_bar[1]);
      __syncwarp();
      waits.drain(&ms.drain_bar[1], 0);
    }
    __syncwarp();
  } else if (warp < kFirstSoft) {
    // ================================================================ copies
    // A warp instruction copies 256 bytes of two rows: lanes 0-15 key 2·w + 8·j,
    // lanes 16-31 the next; piece c of row r goes to (c mod 8) ^ (r mod 8) of its
    // 128-byte row, the swizzle that the descriptors name.  The rotary chunk: 128
    // bytes of four rows, 16 rows a step.
    constexpr int kStep = 2 * kCopyWarps, kRopeStep = 4 * kCopyWarps;
    constexpr int kRuns = kTile / kStep, kRopeRuns = kTile / kRopeStep;
    static_assert(kStep % 8 == 0 && kTile % kRopeStep == 0, "the swizzle of later runs");
    const int w = warp - kFirstCopy;
    const int key0 = 2 * w + (lane >> 4);
    const int piece = lane & 15;
    const uint32_t to_pair = smem_base + (piece >> 3) * kChunk + key0 * 128 + (((piece & 7) ^ (key0 & 7)) << 4);
    const int key1 = 4 * w + (lane >> 3);
    const uint32_t to_rope = smem_base + C::kOffRope + key1 * 128 + (((lane & 7) ^ (key1 & 7)) << 4);
    const uint8_t* from = reinterpret_cast<const uint8_t*>(p.cache);
    const uint64_t once = once_policy();
    int pairs = 0, ropes = 0, tiles = 0;
    bool ok = true;
    while (ok) {
      const int par = tiles % kAhead;
      if (!waits.nap(&ms.tile_full[par], (tiles / kAhead) & 1) || ms.last[par]) break;
      int row[kRuns], rope_row[kRopeRuns];
#pragma unroll
      for (int j = 0; j < kRuns; ++j) row[j] = ms.row[par][key0 + kStep * j];
#pragma unroll
      for (int j = 0; j < kRopeRuns; ++j) rope_row[j] = ms.row[par][key1 + kRopeStep * j];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.tile_read[par]);
      auto copy_rope = [&] {
        const int sl = ropes % C::kRopes;
        if (ropes >= C::kRopes && !(ok = waits.nap(&ms.rope_empty[sl], (ropes / C::kRopes - 1) & 1))) return;
        const uint32_t to = to_rope + sl * kChunk;
        const uint8_t* src = from + 2 * kLat + (lane & 7) * 16;
#pragma unroll
        for (int j = 0; j < kRopeRuns; ++j)
          cp_async16_once(to + j * (kRopeStep * 128), src + static_cast<int64_t>(max(rope_row[j], 0)) * (2 * kRow),
                     rope_row[j] >= 0 ? 16 : 0, once);
        cp_async_arrive(&ms.rope_full[sl]);
        ++ropes;
      };
      if (!C::kAliasP) copy_rope();
      for (int u = 0; u < 4 && ok; ++u) {
        const int sl = pairs % C::kPairs;
        if (pairs >= C::kPairs && !(ok = waits.nap(&ms.pair_empty[sl], (pairs / C::kPairs - 1) & 1))) break;
        const uint32_t to = to_pair + sl * kPair;
        const uint8_t* src = from + u * 256 + piece * 16;
#pragma unroll
        for (int j = 0; j < kRuns; ++j)
          cp_async16_once(to + j * (kStep * 128), src + static_cast<int64_t>(max(row[j], 0)) * (2 * kRow), row[j] >= 0 ? 16 : 0, once);
        cp_async_arrive(&ms.pair_full[sl]);
        ++pairs;
      }
      if (!ok) break;
      if (C::kAliasP) copy_rope();
      ++tiles;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");       // they have landed before the memory goes
  } else {
    // ================================================================ softmax
    constexpr int kColShift = NC == 16 ? 1 : 2;
    const int sw = warp - kFirstSoft, quad = warp & 3, part_id = sw >> 2;
    const int key = quad * 32 + lane;
    const int my_col = lane >> kColShift;                  // the column this lane keeps statistics of
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_addr = lanes + 4 * N + part_id * NC;
    const float scale = fmaxf(fabsf(p.scale_log2), 1.1754944e-38f);   // (never 0 · −inf)
    uint8_t* p_row = smem + C::kOffP + key * 128;
    bool ok = true, gone = false;                          // gone: another warp of the part has given up
    Meeting meeting{1 + part_id, 128, 0, &ms.left_at[part_id]};
    int tiles = 0, pieces = 0, pairs = 0;
    while (true) {
      const int pb = pieces & 1;
      if (!(ok = waits(&ms.piece_full[pb], (pieces >> 1) & 1))) break;
      const Piece pc = ms.piece[pb];
      if (pc.t0 == pc.t1) break;
      float m = -INFINITY;                                 // reference maximum of column my_col, log2 units
      bool check = true;                                   // first tile, or a column's maximum is beyond kFar
      float l[NC];                                         // sums of this key's weights, before their rounding
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;
      ms.m[sw][my_col] = kNone;
      for (int t = pc.t0; t < pc.t1; ++t, ++tiles, pairs += 4) {
        if (!(ok = waits(&ms.tile_full[tiles % kAhead], (tiles / kAhead) & 1))) break;
        const int kind = ms.kind[tiles % kAhead][key];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.tile_read[tiles % kAhead]);
        const bool all_seen = __all_sync(0xFFFFFFFFu, kind == 1);
        const bool drafts = __any_sync(0xFFFFFFFFu, kind >= 2);
        if (!(ok = waits(&ms.s_full, tiles & 1))) break;
        tc_fence_after();
        uint32_t r[NC];
        tmem_ld<NC>(s_addr, r);
        tmem_wait();
        regs_ready<NC>(r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.s_free);
        float z[NC];                                       // scores, then their logarithms' distances from m
#pragma unroll
        for (int c = 0; c < NC; ++c) z[c] = __uint_as_float(r[c]);
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
        // Against the reference maxima as they are: only where some score passes
        // its column's by 2^8 (the first tile of a piece always) is there anything
        // to reduce; one barrier tells the part's four warps alike
        bool over = check;
        float far = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 mc = *reinterpret_cast<const float4*>(&ms.m[sw][c]);
          far = fmaxf(far, fmaxf(fmaf(z[c], scale, -mc.x), fmaf(z[c + 1], scale, -mc.y)));
          far = fmaxf(far, fmaxf(fmaf(z[c + 2], scale, -mc.z), fmaf(z[c + 3], scale, -mc.w)));
        }
        over |= far > kRaise;
        if (meeting.vote(over)) {
          if ((gone = meeting.left())) break;
          float v[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) v[c] = z[c];
          ms.wmax[part_id][quad][my_col] = reduce_columns<NC, true>(v, lane);
          meeting.vote(false);
          float top = ms.wmax[part_id][0][my_col];
#pragma unroll
          for (int w = 1; w < 4; ++w) top = fmaxf(top, ms.wmax[part_id][w][my_col]);
          top = top == -INFINITY ? top : __fmul_rn(top, scale);
          const bool raise = top > m + kRaise || (m == -INFINITY && top > -INFINITY);
          const float a = !raise ? 1.f : m == -INFINITY ? 0.f : ex2(m - top);
          if (raise) m = top;
          ms.alpha[sw][my_col] = a;
          ms.m[sw][my_col] = m == -INFINITY ? kNone : is_far(m) ? 0.f : m;
          check = __any_sync(0xFFFFFFFFu, is_far(m));
          if (check) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float mc = __shfl_sync(0xFFFFFFFFu, m, c << kColShift);
              if (is_far(mc)) z[c] = far_score(z[c], scale, mc);
            }
          }
          __syncwarp();
#pragma unroll
          for (int c = 0; c < NC; ++c) l[c] *= ms.alpha[sw][c];
          if (t > pc.t0) {
            if (!(ok = waits(&ms.p_free, (tiles - 1) & 1))) break;   // the last product has ended
            tc_fence_after();
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
        // P row of this key: NC bf16, 128-byte swizzle, once the last product has read its P
        uint32_t w[NC / 2];
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          const float4 m0 = *reinterpret_cast<const float4*>(&ms.m[sw][c]);
          const float4 m1 = *reinterpret_cast<const float4*>(&ms.m[sw][c + 4]);
          const float mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p0 = ex2(fmaf(z[c + 2 * e], scale, -mm[2 * e]));
            const float p1 = ex2(fmaf(z[c + 2 * e + 1], scale, -mm[2 * e + 1]));
            w[c / 2 + e] = bf_pack_weights(p0, p1);
            l[c + 2 * e] += p0;
            l[c + 2 * e + 1] += p1;
          }
        }
        if (tiles >= 1 && !(ok = waits(&ms.p_free, (tiles - 1) & 1))) break;
#pragma unroll
        for (int c = 0; c < NC / 8; ++c)
          *reinterpret_cast<uint4*>(p_row + ((part_id * NC / 8 + c) ^ (key & 7)) * 16) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        // a draft's row that only some columns see must not reach the others as
        // 0 · NaN: where it is not finite it becomes zero (see spoil for the columns
        // that see it)
        if (pc.mixed && drafts && part_id == 0) {
          for (int u = 0; u < 4 && ok; ++u)
            ok = waits(&ms.pair_full[(pairs + u) % C::kPairs], ((pairs + u) / C::kPairs) & 1);
          if (!ok) break;
          if (kind >= 2) clear_wild(smem + key * 128, pairs % C::kPairs, C::kPairs, &ms.wild[pb], kind - 2);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full);
      }
      if (!ok || gone) break;
      // ---- the sums over all keys
      ms.sum[part_id][quad][my_col] = reduce_columns<NC, false>(l, lane);
      if (meeting.vote(false) && (gone = meeting.left())) break;
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) z += ms.sum[part_id][w][my_col];
      const bool whole = pc.slot < 0;
      float* part = whole ? nullptr : part_slot(p, blockIdx.x, pc.slot);
      ms.alpha[sw][my_col] = whole ? (z == 0.f ? 0.f : 1.f / z) : 1.f;
      if (quad == 0 && (lane & ((1 << kColShift) - 1)) == 0) {
        const int c = part_id * NC + my_col;
        if (!whole) {
          part[N * kLat + c] = m;
          part[N * kLat + N + c] = z;
        } else if (p.lse && c < pc.rows) {
          p.lse[pc.row0 + c] = lse_of(m, z);
        }
      }
      __syncwarp();
      if (!(ok = waits(&ms.o_full, pieces & 1))) break;
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
      if (const uint64_t wild = ms.wild[pb])
        spoil_columns(p, ms.piece[pb], ms.mask[pb], wild, key, part_id * NC, NC);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.o_free);
        mbar_arrive(&ms.piece_empty[pb]);
      }
      ++pieces;
    }
    if (!gone) {
      if (ok && (p.fault & kFaultEnd) && quad == 0) ok = waits(&ms.never, 0);
      meeting.part(ok);
    }
  }
  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the pieces of the items that shares cut.  A unit is 32 runs of eight output
// features of such an item, a lane each, walking the pieces with a running maximum.
// CTA (x, y) takes every kJoinY-th eight units, a warp each, of the item that begins
// in CTA x's share, where it has few pieces.  Items of kJoinSplit pieces and more
// (one long sequence over all SMs is one item) are dealt to all CTAs: one unit at a
// time, whose pieces the CTA's eight warps share; their results are added in a
// fixed order (64 heads over one sequence of 131 072, L2 flushed before each call:
// 69 us, 147 when CTA x alone took its item).  Reads what the pieces wrote, from L2 as far as it is
// still there; two pieces of each of 128 items of 128 rows, 38 MB: 6 us.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinY = 8, kJoinSplit = 8;
struct Joined {
  float o[8], top, z;
};
__device__ __forceinline__ void join_add(Joined& a, float m, float z, const float* x) {
  const float up = fmaxf(a.top, m), base = up == -INFINITY ? 0.f : up;
  const float keep = ex2(a.top - base), w = ex2(m - base);
#pragma unroll
  for (int i = 0; i < 8; ++i) a.o[i] = a.o[i] * keep + w * x[i];
  a.z = a.z * keep + w * z;
  a.top = up;
}
// pieces first, first + step … ≤ last of a run, K of them in flight at a time
struct PieceRun {
  const float *head, *next;                   // piece 0; piece i > 0 lies at next + i · stride
  int64_t stride;
  int at, at_m, at_z;
};
template <int K>
__device__ __forceinline__ Joined join_pieces(const PieceRun& r, int first, int step, int last) {
  Joined a{{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, -INFINITY, 0.f};
  for (int i = first; i <= last; i += K * step) {
    float m[K], z[K];
    float4 x[K][2];
#pragma unroll
    for (int h = 0; h < K; ++h) {
      const int piece = min(i + h * step, last);
      const float* s = piece == 0 ? r.head : r.next + piece * r.stride;
      m[h] = s[r.at_m];
      z[h] = s[r.at_z];
      x[h][0] = *reinterpret_cast<const float4*>(s + r.at);
      x[h][1] = *reinterpret_cast<const float4*>(s + r.at + 4);
    }
#pragma unroll
    for (int h = 0; h < K; ++h)
      if (i + h * step <= last) join_add(a, m[h], z[h], reinterpret_cast<const float*>(x[h]));
  }
  return a;
}
struct Unit {                                 // a lane's run of an item
  int row, feature, valid;
  PieceRun run;
};
__device__ __forceinline__ Unit join_unit(const TreeParams& p, const Cut& cut, int cta, int unit, int lane) {
  const int D = kLat / p.halves, D8 = D / 8, count = cut.rows * D8;   // output features per slot row
  // neighbours in memory are neighbours in the warp: features of a row, or rows
  const int e = min(unit * 32 + lane, count - 1);
  const int c = p.halves == 1 ? e / D8 : e % cut.rows, d = p.halves == 1 ? e % D8 : e / cut.rows;
  Unit u;
  u.row = c;
  u.feature = cta % p.halves * D + d * 8;
  u.valid = unit * 32 + lane < count;
  u.run.head = part_slot(p, cta, 1);           // it begins in this share; the next teams' slots 0 go on
  u.run.next = part_slot(p, cta, 0);
  u.run.stride = static_cast<int64_t>(p.halves) * 2 * p.M * (D + 2);
  u.run.at = p.halves == 1 ? c * D + d * 8 : (d * p.M + c) * 8;
  u.run.at_m = p.M * D + c;
  u.run.at_z = u.run.at_m + p.M;
  return u;
}
__device__ __forceinline__ void join_store(const TreeParams& p, const Cut& cut, const Unit& u, Joined& a) {
  if (!u.valid) return;
  const float inv = a.z == 0.f ? 0.f : 1.f / a.z;
  const int64_t to = (cut.row0 + u.row) * kLat + u.feature;
#pragma unroll
  for (int i = 0; i < 8; ++i) a.o[i] *= inv;
  if (p.out_bf16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to) =
        make_uint4(bf_pack(a.o[0], a.o[1]), bf_pack(a.o[2], a.o[3]), bf_pack(a.o[4], a.o[5]), bf_pack(a.o[6], a.o[7]));
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + to);
    dst[0] = make_float4(a.o[0], a.o[1], a.o[2], a.o[3]);
    dst[1] = make_float4(a.o[4], a.o[5], a.o[6], a.o[7]);
  }
  if (p.lse && u.feature == 0) p.lse[cut.row0 + u.row] = lse_of(a.top, a.z);
}
__global__ void __launch_bounds__(kJoinThreads) tree_mla_join_kernel(const TreeParams p) {
  __shared__ Joined part[kJoinThreads];
  __shared__ Cut cuts[kJoinThreads];
  __shared__ int sums[kJoinWarps], found, found_at;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched under the end of the main kernel: its results first
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D8 = kLat / p.halves / 8;
  const Cut own = p.cuts[blockIdx.x];
  Cut mine{0, 0, 0};                           // thread ↔ CTA of the main kernel
  if (threadIdx.x < gridDim.x) mine = p.cuts[threadIdx.x];
  if (own.pieces < kJoinSplit && own.pieces > 0)
    for (int unit = blockIdx.y * kJoinWarps + warp; unit * 32 < own.rows * D8; unit += kJoinY * kJoinWarps) {
      const Unit u = join_unit(p, own, blockIdx.x, unit, lane);
      Joined a = join_pieces<2>(u.run, 0, 1, own.pieces);
      join_store(p, own, u, a);
    }
  if (!__syncthreads_or(mine.pieces >= kJoinSplit)) return;
  cuts[threadIdx.x] = mine;
  const int units = mine.pieces >= kJoinSplit ? (mine.rows * D8 + 31) / 32 : 0;
  int end = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, end, o);
    if (lane >= o) end += v;
  }
  if (lane == 31) sums[warp] = end;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) end += sums[w];
    total += sums[w];
  }
  for (int j = blockIdx.y * gridDim.x + blockIdx.x; j < total; j += gridDim.x * kJoinY) {
    if (end - units <= j && j < end) {
      found = threadIdx.x;
      found_at = j - (end - units);
    }
    __syncthreads();
    const Cut cut = cuts[found];
    const Unit u = join_unit(p, cut, found, found_at, lane);
    Joined a = join_pieces<4>(u.run, warp, kJoinWarps, cut.pieces);
    part[threadIdx.x] = a;
    __syncthreads();
    if (warp == 0) {
      for (int g = 1; g < kJoinWarps; ++g) {
        const Joined& b = part[g * 32 + lane];
        join_add(a, b.top, b.z, b.o);
      }
      join_store(p, cut, u, a);
    }
    __syncthreads();
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// How a call's rows and tiles are dealt.  Rows that share keys: up to 64 go to the
// transposed kernel above with the fewest columns that hold them (16, 32, 64; 16
// heads over 16 x 30 000 positions: 113 us with 16 columns, 121 with 32; 32 rows over
// 32 x 16 000: 129 with 32, 166 with 64); more to the wide kernel (tree_mla_wide.cu) in
// groups of 128, two CTAs each.  Both sides, the wide kernel and groups of 64 here, in us
// in a CUDA graph:
//   64 x 6 000 positions, one token of 65 / 96 / 128 / 144 / 160 / 192 / 256 heads:
//     160 / 175 / 172 / 314 / 332 / 313 / 365 and 221 / 230 / 231 / 352 / 343 / 368 / 478;
//   48 x 3 000, tokens of 16 heads, 5 / 6 / 8 / 9 / 10 / 13 / 16 of them:
//     99 / 101 / 83 / 128 / 133 / 141 / 147 and 115 / 111 / 108 / 125 / 124 / 184 / 188.
// (Groups of 64 win by 3 - 7% only at 144 and 160 rows of few keys, and the other way
// round: 128 tokens of 64 heads, 2 048 of 16 000 positions take 113 us here, 127 there.)
struct Plan {
  int M, halves, teams, whole;
  size_t part_bytes, ws;
};
Plan plan_for(int B, int n, int H, int max_len, int k, int sms) {
  Plan pl;
  sms = sms < kJoinThreads ? sms : kJoinThreads;   // (the join has a thread per CTA)
  const int64_t rows = k ? H : static_cast<int64_t>(n) * H;
  pl.M = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  pl.halves = pl.M == 128 ? 2 : 1;
  const int64_t keys = k ? static_cast<int64_t>(k) + n : max_len;
  const int most = sms / pl.halves > 0 ? sms / pl.halves : 1;
  pl.whole = keys <= 2 * kMinShare || most == 1;
  // no more teams than the call can have shares (one sequence of 2 048 positions, 64
  // heads, in a CUDA graph: 18.5 us with 16 CTAs, 19.9 with 148, most of them for nothing)
  const int64_t items = (k ? n : 1) * ((rows + pl.M - 1) / pl.M) * B;
  const int64_t per_item = pl.whole ? 1 : (keys + kMinShare - 1) / kMinShare;
  pl.teams = items < most && items * per_item < most ? static_cast<int>(items * per_item) : most;
  const size_t ctas = static_cast<size_t>(pl.teams) * pl.halves;
  pl.part_bytes = ctas * 2 * pl.M * (kLat / pl.halves + 2) * sizeof(float);
  pl.ws = pl.whole ? 0 : pl.part_bytes + ctas * sizeof(Cut);
  return pl;
}

template <int N>
int launch(const CUtensorMap& tq, const TreeParams& p, int ctas, cudaStream_t stream) {
  constexpr int smem = 1024 + Cfg<N>::kOffMisc + static_cast<int>(sizeof(Misc<N>));
  static_assert(smem <= 227 * 1024, "shared memory");
  if (const int r = ensure_smem_limit(reinterpret_cast<const void*>(tree_mla_kernel<N>), smem)) return r;
  tree_mla_kernel<N><<<static_cast<unsigned>(ctas), Cfg<N>::kThreads, smem, stream>>>(tq, p);
  return check_launch();
}

}  // namespace
}  // namespace idx

using namespace idx;
extern "C" size_t idx_tree_mla_workspace_size(int B, int n, int H, int max_len, int k) {
  if (B <= 0 || n <= 0 || n > IDX_MAX_DRAFTS || H <= 0 || max_len <= 0 || k < 0) return 0;
  if (static_cast<int64_t>(B) * n > 0x7FFFFFFF / H) return 0;     // (idx_tree_mla refuses it)
  return plan_for(B, n, H, max_len, k, num_sms()).ws;
}

extern "C" int idx_tree_mla(const uint16_t* q, const uint16_t* cache, const int32_t* page_table, int max_pages,
                            int num_pages, int page_size, const int32_t* lengths, const int32_t* counts, int B, int n,
                            int H, int max_len, const uint64_t* tree_mask, const int32_t* indices, int k,
                            float softmax_scale, void* out, int out_dtype, float* lse, void* ws, size_t ws_bytes,
                            idx_stream_t stream) {
  using namespace tree;
  constexpr int64_t kMaxRows = 0x7FFFFFFF;
  if (out_dtype != IDX_OUT_F32 && out_dtype != IDX_OUT_BF16) return IDX_ERR_FMT;
  if (B < 0 || n < 0 || n > IDX_MAX_DRAFTS || H <= 0 || k < 0 || k > kMaxRows - 2 * kTile - IDX_MAX_DRAFTS ||
      !std::isfinite(softmax_scale * kLog2e))
    return IDX_ERR_SHAPE;
  if (B == 0 || n == 0) return IDX_OK;
  if (max_pages <= 0 || num_pages <= 0 || page_size <= 0 || static_cast<int64_t>(num_pages) * page_size > kMaxRows ||
      static_cast<int64_t>(max_pages) * page_size > kMaxRows)
    return IDX_ERR_SHAPE;
  if (max_len <= 0 || max_len > static_cast<int64_t>(max_pages) * page_size || max_len > kMaxRows - 2 * kTile)
    return IDX_ERR_SHAPE;
  if ((k > 0) != (indices != nullptr)) return indices ? IDX_ERR_K : IDX_ERR_NULL;
  if (!q || !cache || !page_table || !lengths || !out) return IDX_ERR_NULL;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 32) || !aligned(ws, 32) || !aligned(tree_mask, 8))
    return IDX_ERR_ALIGN;
  const int64_t rows = static_cast<int64_t>(B) * n;
  if (rows > kMaxRows / H) return IDX_ERR_SHAPE;
  const Plan pl = plan_for(B, n, H, max_len, k, num_sms());
  if (pl.ws > 0 && !ws) return IDX_ERR_NULL;
  if (ws_bytes < pl.ws) return IDX_ERR_SCRATCH;
  const int ctas = pl.teams * pl.halves;
  CUtensorMap tq;
  if (!make_tmap_2d_bf16_sw128(&tq, q, kRow, static_cast<uint64_t>(rows) * H, static_cast<uint32_t>(pl.M)))
    return IDX_ERR_UNSUPPORTED;
  TreeParams p;
  p.table = page_table;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.q = q;
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
  p.M = pl.M;
  p.halves = pl.halves;
  p.teams = pl.teams;
  p.whole = pl.whole;
  p.part = static_cast<float*>(ws);
  p.cuts = reinterpret_cast<Cut*>(static_cast<uint8_t*>(ws) + pl.part_bytes);
  const DebugState dbg = debug_state();
  p.budget_ns = dbg.budget_ns;
  p.fault = dbg.flags & (kFaultScores | kFaultEnd);
  p.err = device_error_word();
  if (!p.err) return check_launch();
  auto* s = reinterpret_cast<cudaStream_t>(stream);
  const int r = pl.M == 16   ? launch<16>(tq, p, ctas, s)
                : pl.M == 32 ? launch<32>(tq, p, ctas, s)
                : pl.M == 64 ? launch<64>(tq, p, ctas, s)
                             : launch_tree_mla_wide(tq, p, ctas, s);
  if (r || p.whole) return r;
  // a programmatic dependent launch: the join's blocks are placed while the main
  // kernel's last ones still run, and wait there for the whole of it
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(static_cast<unsigned>(ctas), kJoinY);
  config.blockDim = dim3(kJoinThreads);
  config.stream = s;
  config.attrs = &attr;
  config.numAttrs = 1;
  cudaLaunchKernelEx(&config, tree_mla_join_kernel, p);
  return check_launch();
}
