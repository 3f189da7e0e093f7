// Latent attention of drafted token trees over the paged cache (idx_tree_mla),
// for more than 64 rows per set of keys (tokens · heads, or heads where each
// token has its own selection): groups of 128 rows.
//
// A row is an accumulator lane: S = q · Kᵀ (M = 128 rows, N = 64 keys, K = 576)
// and O = P · V (N = 256 output features, K = 64 keys).  TMEM holds 512 columns,
// and a full O of 512 would leave none for S, so two CTAs share a row group: both
// compute all its scores (36 MMAs per tile: 24 with the queries in TMEM at 32
// cycles, 12 with them in shared memory at 48) and each accumulates its half of
// the output features (4 MMAs at 128), 1 860 cycles per 64 keys where one CTA
// with a whole S and O would need 2 180 of the tensor cores.
//
// The tile's nine 64-feature chunks live in two rings: the four that are also
// this CTA's V (three buffers: free after the product) and the five others (a ring
// of seven: free after the scores).  So the copies of the next tile wait neither
// for this tile's softmax nor for its product, and the scores of tile t + 1 run while
// the softmax of t does.  Scores and products are issued by two warps: what a warp asks of
// a barrier waits behind the MMAs that it has queued (some 400 cycles of them).
// Trees of 8 drafts of 128 heads over 32 x <= 8 192 positions: 2 460 cycles a tile, 14 500
// from a piece's last tile to the next one's first, at 1.56 - 1.70 GHz under this load; of
// a CTA's life 86% are inside pieces, 7.5% between them, 4.5% before the first scores.
//
// One CTA, 20 warps:
//   warp 0       the planner (tree_mla.cuh);
//   warps 1, 2   issue the MMAs of the scores and of the products;
//   warps 3-10   copy the rows by cp.async, 16 bytes a lane (a key that no row sees
//                arrives as zeros);
//   warps 11-18  softmax: thread ↔ (row, half of the keys), the row's reference
//                maximum in a register, raised only where a score passes it by 2^8
//                (then the two threads of a row agree through shared memory and O
//                in TMEM is rescaled); P = 2^(s − m) in bf16 in shared memory;
//                between pieces they put the next queries' first six chunks into
//                TMEM while the last product runs;
//   warp 19      asks for the tiles' rows in L2 a few tiles ahead of the copies (the
//                rings hold a tile and a half, less than the latency of HBM).
// Rounding, bounded waits and the way out as in tree_mla.cu.
#include "tree_mla.cuh"

namespace idx {
namespace {

using namespace tree;

constexpr int kRows = 128;                    // rows per CTA
constexpr int kKeys = 64;                     // keys per tile
constexpr int kHalf = 256;                    // output features per CTA
constexpr int kCopyWarps = 8, kSoftWarps = 8;
constexpr int kFirstCopy = 3, kFirstSoft = kFirstCopy + kCopyWarps;
constexpr int kPrefetchWarp = kFirstSoft + kSoftWarps;
constexpr int kThreads = (kPrefetchWarp + 1) * 32;
constexpr int kChunk = kKeys * 128;           // 64 keys × 64 features
constexpr int kV = 4 * kChunk;                // a V buffer
constexpr int kVs = 3, kXs = 7;               // buffers of V, and of the other chunks
constexpr int kQTmem = 6;                     // query chunks in TMEM; the other three in shared memory
constexpr int kQChunk = kRows * 128;

constexpr int kOffX = kVs * kV;
constexpr int kOffQ = kOffX + kXs * kChunk;
constexpr int kOffP = kOffQ + 3 * kQChunk;
constexpr int kOffMisc = kOffP + kRows * 128;
constexpr uint32_t kColS = kQTmem * 32, kColO = 256;
static_assert(kColS + kKeys <= kColO, "TMEM columns");

struct WideState : PlanState<kRows, kKeys, kThreads / 32> {
  float top[2][kRows], sum[2][kRows];         // per half of the keys
  int left_at[4];                             // per quarter of the rows
  uint64_t v_full[kVs], v_empty[kVs], x_full[2];
  uint64_t x_head, x_tail[2];                 // scores: the first three chunks done, all five
  uint64_t q_ready, s_issued[2], s_full, s_free, p_full, p_free, o_full, o_free, drain_bar[2];
};
constexpr int kSmem = 1024 + kOffMisc + static_cast<int>(sizeof(WideState));
static_assert(kSmem <= 227 * 1024, "shared memory");

// The chunks in the order the scores take them: the four latent chunks of the
// other half, the rotary chunk, the four of this half.
__device__ __forceinline__ int feature_chunk(int pos, int half) {
  return pos < 4 ? 4 * (1 - half) + pos : pos == 4 ? 8 : 4 * half + pos - 5;
}

// 64 features of draft j: zeros where one of them is not finite
__device__ __noinline__ void clear_wild(uint8_t* at, unsigned long long* wild, int j) {
  uint4* x = reinterpret_cast<uint4*>(at);
  bool any = false;
  for (int i = 0; i < 8; ++i) any |= not_finite(x[i]);
  if (!any) return;
  atomicOr(wild, 1ull << j);
  for (int i = 0; i < 8; ++i) x[i] = make_uint4(0, 0, 0, 0);
}
// NaN into this thread's 128 outputs where a wild draft's features are not finite
__device__ __noinline__ void spoil_half(const TreeParams& p, const Piece& pc, uint64_t wild, int r_id, int half, int part) {
  for (; wild; wild &= wild - 1) {
    const uint16_t* src = draft_row(p, pc, __ffsll(static_cast<long long>(wild)) - 1) + half * kHalf;
    for (int c = part * (kHalf / 2); c < (part + 1) * (kHalf / 2); ++c)
      if (not_finite(src[c]))
        spoil(p, pc, r_id, half * kHalf + c,
              pc.slot < 0 ? nullptr : part_slot(p, blockIdx.x, pc.slot) + (c >> 3) * 8 * kRows + r_id * 8 + (c & 7));
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    tree_mla_wide_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  WideState& ms = *reinterpret_cast<WideState*>(smem + kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / p.halves, half = blockIdx.x % p.halves;
  const Waits waits{p.budget_ns, &ms.abort_flag, p.err};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kVs; ++i) {
      mbar_init(&ms.v_full[i], kCopyWarps * 32);
      mbar_init(&ms.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&ms.x_full[i], kCopyWarps * 32);
    mbar_init(&ms.x_head, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ms.x_tail[i], 1);
    mbar_init(&ms.q_ready, kSoftWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&ms.s_issued[i], 1);
    mbar_init(&ms.s_full, 1);
    mbar_init(&ms.s_free, kSoftWarps);
    mbar_init(&ms.p_full, kSoftWarps);
    mbar_init(&ms.p_free, 1);
    mbar_init(&ms.o_full, 1);
    mbar_init(&ms.o_free, kSoftWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&ms.drain_bar[i], 1);
    for (int i = 0; i < 4; ++i) ms.left_at[i] = 0;
    ms.init(p.B, kCopyWarps + kSoftWarps + 1, kSoftWarps + 2);
    fence_barrier_init();
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == 1) tmem_alloc(&ms.tmem, 512);
  const Share share = find_share<kRows, kKeys, kThreads>(p, ms, team);
  const uint32_t tmem = ms.tmem;
  const uint32_t smem_base = smem_u32(smem);

  if (warp == 0) {
    plan<kRows, kKeys>(p, ms, share, waits, [&](int row0) {
      mbar_arrive_expect_tx(&ms.q_full, 3 * kQChunk);
      for (int c = 0; c < 3; ++c)
        tma_box(smem_base + kOffQ + c * kQChunk, &tmap_q, smem_u32(&ms.q_full), feature_chunk(kQTmem + c, half) * 64,
                row0);
    });
  } else if (warp == 1) {
    // ================================================================ scores
    const uint32_t id_s = idesc_bf16(kKeys, false, false) | (p.scale_log2 < 0.f ? kNegateA : 0u);
    const uint32_t d_s = tmem + kColS;
    const uint64_t k_desc = smem_desc_k128_sw128(smem_base);
    const uint64_t q_desc = smem_desc_k128_sw128(smem_base + kOffQ);
    bool ok = true, issued = false;
    int xs = 0, tiles = 0, pieces = 0;         // next x buffer; running counts
    while (true) {
      const int pb = pieces & 1;
      if (!(ok = waits(&ms.piece_full[pb], (pieces >> 1) & 1))) break;
      const int n = __reduce_max_sync(0xFFFFFFFFu, ms.piece[pb].t1 - ms.piece[pb].t0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.piece_empty[pb]);
      if (n == 0) break;
      if (!(ok = waits(&ms.q_full, pieces & 1)) || !(ok = waits(&ms.q_ready, pieces & 1))) break;
      for (int c = 0; c < n; ++c) {
        // S = q · Kᵀ of tile c, once the softmax has read the last S
        const int sl = tiles % kVs;
        if (!(ok = waits(&ms.x_full[tiles & 1], (tiles >> 1) & 1))) break;
        if (!(ok = waits(&ms.v_full[sl], (tiles / kVs) & 1))) break;
        fence_proxy_async_smem();              // the copies wrote through the generic proxy
        if (tiles >= 1 && !(ok = waits(&ms.s_free, (tiles - 1) & 1))) break;
        if ((p.fault & kFaultScores) && c == n - 1 && !(ok = waits(&ms.never, 0))) break;
        tc_fence_after();
        if (elect_one()) {
          int x = xs;
#pragma unroll 1
          for (int u = 0; u < 5; ++u) {
            const uint64_t b = k_desc + static_cast<uint64_t>((kOffX >> 4) + x * (kChunk >> 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_f16_ta(d_s, tmem + u * 32 + i * 8, b + i * 2, id_s, (u > 0 || i > 0) ? 1u : 0u);
            if (u == 2) mma_commit(&ms.x_head);
            x = x == kXs - 1 ? 0 : x + 1;
          }
          mma_commit(&ms.x_tail[tiles & 1]);
          const uint64_t b = k_desc + static_cast<uint64_t>(sl * (kV >> 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_f16_ta(d_s, tmem + 5 * 32 + i * 8, b + i * 2, id_s, 1u);
#pragma unroll 1
          for (int u = 0; u < 3; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16(d_s, q_desc + static_cast<uint64_t>(u * (kQChunk >> 4) + i * 2),
                      b + static_cast<uint64_t>((u + 1) * (kChunk >> 4) + i * 2), id_s, 1u);
          mma_commit(&ms.s_full);
          if (c == n - 1) mma_commit(&ms.q_empty);
        }
        issued = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.s_issued[tiles & 1]);   // (reaches the barrier as the queued MMAs drain)
        xs = (xs + 5) % kXs;
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
    constexpr uint32_t id_o = idesc_bf16(kHalf, false, true);
    const uint32_t d_o = tmem + kColO;
    const uint64_t p_desc = smem_desc_k128_sw128(smem_base + kOffP);
    const uint64_t v_desc = desc_mn(smem_base, kChunk);
    bool ok = true, issued = false;
    int tiles = 0, pieces = 0;
    while (true) {
      const int pb = pieces & 1;
      if (!(ok = waits(&ms.piece_full[pb], (pieces >> 1) & 1))) break;
      const int n = __reduce_max_sync(0xFFFFFFFFu, ms.piece[pb].t1 - ms.piece[pb].t0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.piece_empty[pb]);
      if (n == 0) break;
      for (int c = 0; c < n; ++c) {
        // O += P · V of tile c (its scores, and so its V, were complete before its P),
        // behind the scores of tile c + 1: it then runs while the softmax reads those
        // out of TMEM, when the tensor cores would wait for the buffer
        const int sl = tiles % kVs;
        if (c == 0 && pieces > 0 && !(ok = waits(&ms.o_free, (pieces - 1) & 1))) break;
        if (!(ok = waits(&ms.p_full, tiles & 1))) break;
        if (c < n - 1 && !(ok = waits(&ms.s_issued[(tiles + 1) & 1], ((tiles + 1) >> 1) & 1))) break;
        fence_proxy_async_smem();              // P was written through the generic proxy
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = v_desc + static_cast<uint64_t>(sl * (kV >> 4));
#pragma unroll
          for (int i = 0; i < 4; ++i)           // 16 keys per instruction: two 8-row atoms
            mma_f16(d_o, p_desc + i * 2, b + i * (2048 >> 4), id_o, (c > 0 || i > 0) ? 1u : 0u);
          mma_commit(&ms.p_free);
          mma_commit(&ms.v_empty[sl]);
          if (c == n - 1) mma_commit(&ms.o_full);
        }
        issued = true;
        __syncwarp();
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
    // V: a warp instruction copies 512 bytes of key w + 8·j.  The other chunks:
    // 128 bytes of the four keys 4·w + 32·j ….  Piece c of row r goes to
    // (c mod 8) ^ (r mod 8) of its 128-byte row, as the descriptors say.
    const int w = warp - kFirstCopy;
    const uint32_t to_v = smem_base + (lane >> 3) * kChunk + w * 128 + (((lane & 7) ^ (w & 7)) << 4);
    const int key1 = 4 * w + (lane >> 3);
    const uint32_t to_x = smem_base + kOffX + key1 * 128 + (((lane & 7) ^ (key1 & 7)) << 4);
    const uint8_t* from = reinterpret_cast<const uint8_t*>(p.cache);
    int xs = 0, tiles = 0;
    bool ok = true;
    while (ok) {
      const int par = tiles % kAhead;
      if (!waits.nap(&ms.tile_full[par], (tiles / kAhead) & 1) || ms.last[par]) break;
      int row[8], xrow[2];
#pragma unroll
      for (int j = 0; j < 8; ++j) row[j] = ms.row[par][w + 8 * j];
#pragma unroll
      for (int j = 0; j < 2; ++j) xrow[j] = ms.row[par][key1 + 32 * j];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.tile_read[par]);
      // In the order in which places become free: chunk 5·t + u takes the place of
      // the one seven earlier — the first two of tile t − 2's last two, the others of
      // tile t − 1's first three, whose scores are the last thing to wait for — and V
      // that of tile t − 3
      auto copy_x = [&](int u) {
        const uint8_t* src = from + feature_chunk(u, half) * 128 + (lane & 7) * 16;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          cp_async16(to_x + xs * kChunk + j * 4096, src + static_cast<int64_t>(max(xrow[j], 0)) * (2 * kRow),
                     xrow[j] >= 0 ? 16 : 0);
        xs = xs == kXs - 1 ? 0 : xs + 1;
      };
      if (tiles >= 2 && !(ok = waits.nap(&ms.x_tail[tiles & 1], ((tiles >> 1) - 1) & 1))) break;
      copy_x(0);
      copy_x(1);
      const int sl = tiles % kVs;
      if (tiles >= kVs && !(ok = waits.nap(&ms.v_empty[sl], (tiles / kVs - 1) & 1))) break;
      const uint8_t* src = from + half * 512 + lane * 16;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        cp_async16(to_v + sl * kV + j * 1024, src + static_cast<int64_t>(max(row[j], 0)) * (2 * kRow), row[j] >= 0 ? 16 : 0);
      cp_async_arrive(&ms.v_full[sl]);
      if (tiles >= 1 && !(ok = waits(&ms.x_head, (tiles - 1) & 1))) break;
      copy_x(2);
      copy_x(3);
      copy_x(4);
      cp_async_arrive(&ms.x_full[tiles & 1]);
      ++tiles;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");       // they have landed before the memory goes
  } else if (warp == kPrefetchWarp) {
    // ================================================================ prefetch
    // this CTA's half of the rows, one bulk request each (128 x 2 048 selected positions
    // of 16 384, 128 heads: 139 us, 149 without the warp; 8 drafts of 128 heads over
    // 32 x 8 192: 332 and 345)
    const uint8_t* from = reinterpret_cast<const uint8_t*>(p.cache);
    for (int tiles = 0;; ++tiles) {
      const int at = tiles % kAhead;
      if (!waits.nap(&ms.tile_full[at], (tiles / kAhead) & 1) || ms.last[at]) break;
      const int r = ms.row[at][half * 32 + lane];
      if (r >= 0) prefetch_l2_row(from + static_cast<int64_t>(r) * (2 * kRow));
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.tile_read[at]);
    }
  } else {
    // ================================================================ softmax
    const int sw = warp - kFirstSoft, quad = warp & 3, part = sw >> 2;
    const int r_id = quad * 32 + lane;                     // row within the group (TMEM lane)
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float scale = fmaxf(fabsf(p.scale_log2), 1.1754944e-38f);   // (never 0 · −inf)
    uint8_t* p_row = smem + kOffP + r_id * 128;
    bool ok = true, gone = false;                          // gone: the other warp of these rows has given up
    Meeting meeting{1 + quad, 64, 0, &ms.left_at[quad]};
    int tiles = 0, pieces = 0;
    // Three of the six query chunks that live in TMEM, into this warp's lanes: read
    // as 64-byte runs of eight rows (a lane reading its own row would touch 32
    // lines per instruction), turned through the warp's 2 KB of the P buffer, which
    // the last product must have left
    uint8_t* stage = smem + kOffP + sw * 2048;
    auto load_q = [&](const Piece& pc, uint64_t* p_left, uint32_t parity) {
      const int r0 = quad * 32 + (lane >> 2), pc16 = lane & 3;
      const uint16_t* src = p.q + (pc.row0 + r0) * kRow + pc16 * 8;
      uint4 x[3][4];
      auto fetch = [&](int h) {                            // half chunk h of six
        const int f = feature_chunk(part * 3 + h / 2, half) * 64 + (h & 1) * 32;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[h % 3][j] = r0 + 8 * j < pc.rows ? __ldg(reinterpret_cast<const uint4*>(src + 8 * j * kRow + f)) : make_uint4(0, 0, 0, 0);
      };
#pragma unroll
      for (int h = 0; h < 3; ++h) fetch(h);
      if (p_left && !waits(p_left, parity)) return false;
#pragma unroll
      for (int h = 0; h < 6; ++h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (lane >> 2) + 8 * j;
          *reinterpret_cast<uint4*>(stage + r * 64 + ((pc16 ^ (r >> 1)) & 3) * 16) = x[h % 3][j];
        }
        if (h + 3 < 6) fetch(h + 3);
        __syncwarp();
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 y = *reinterpret_cast<const uint4*>(stage + lane * 64 + ((j ^ (lane >> 1)) & 3) * 16);
          w[4 * j] = y.x;
          w[4 * j + 1] = y.y;
          w[4 * j + 2] = y.z;
          w[4 * j + 3] = y.w;
        }
        tmem_st<16>(lanes + (part * 3 + h / 2) * 32 + (h & 1) * 16, w);
        __syncwarp();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_ready);
      return true;
    };
    ok = waits(&ms.piece_full[0], 0);
    if (ok && ms.piece[0].t0 != ms.piece[0].t1) load_q(ms.piece[0], nullptr, 0);
    while (ok) {
      const int pb = pieces & 1;
      const Piece pc = ms.piece[pb];
      if (pc.t0 == pc.t1) break;
      const uint64_t drafts = ms.mask[pb][r_id];
      float m = -INFINITY, l = 0.f;                        // reference maximum (log2 units), sum of this half's weights
      bool check = true;                                   // first tile, or a row's maximum is beyond kFar
      // what this row sees of a tile's keys: the context, and its drafts (draft j is
      // key nkeys + j); read a tile ahead, while the last product runs
      uint32_t next_sees = 0;
      auto look = [&](int t, int tile) {
        if (!waits(&ms.tile_full[tile % kAhead], (tile / kAhead) & 1)) return false;
        const int kind = ms.kind[tile % kAhead][part * 32 + lane];
        next_sees = __ballot_sync(0xFFFFFFFFu, kind == 1);
        const uint32_t dr = __ballot_sync(0xFFFFFFFFu, kind >= 2);
        if (dr) {
          const int sh = pc.nkeys - (t * kKeys + part * 32);   // key of draft 0 in these 32
          const uint64_t at = sh >= 0 ? (sh < 64 ? drafts << sh : 0) : (sh > -64 ? drafts >> -sh : 0);
          next_sees |= static_cast<uint32_t>(at) & dr;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.tile_read[tile % kAhead]);
        return true;
      };
      if (!(ok = look(pc.t0, tiles))) break;
      for (int t = pc.t0; t < pc.t1; ++t, ++tiles) {
        const uint32_t sees = next_sees;
        if (t == pc.t1 - 1 && waits.test(&ms.piece_full[pb ^ 1], ((pieces + 1) >> 1) & 1)) {
          const Piece& next = ms.piece[pb ^ 1];            // its queries into L2 (load_q reads them soon)
          if (next.t0 != next.t1 && r_id < next.rows)
            for (int i = 0; i < 3; ++i)
              prefetch_l2(p.q + (next.row0 + r_id) * kRow + feature_chunk(part * 3 + i, half) * 64);
        }
        if (!(ok = waits(&ms.s_full, tiles & 1))) break;
        tc_fence_after();
        uint32_t r[32];
        tmem_ld<16>(lanes + kColS + part * 32, r);
        tmem_ld<16>(lanes + kColS + part * 32 + 16, r + 16);
        tmem_wait();
        regs_ready<32>(r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.s_free);
        float z[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) z[c] = __uint_as_float(r[c]);
        if (__any_sync(0xFFFFFFFFu, sees != 0xFFFFFFFFu)) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((sees >> c) & 1)) z[c] = -INFINITY;
        }
        float far = -INFINITY;
#pragma unroll
        for (int c = 0; c < 32; ++c) far = fmaxf(far, z[c]);
        const float mu = m == -INFINITY ? kNone : m;
        const bool raised = meeting.vote(check || fmaf(far, scale, -mu) > kRaise);
        float a = 1.f;
        if (raised) {                                      // the same in both warps of these rows
          if ((gone = meeting.left())) break;
          ms.top[part][r_id] = far;
          meeting.vote(false);
          float top = fmaxf(far, ms.top[1 - part][r_id]);
          top = top == -INFINITY ? top : __fmul_rn(top, scale);
          const bool raise = top > m + kRaise || (m == -INFINITY && top > -INFINITY);
          if (raise) {
            a = m == -INFINITY ? 0.f : ex2(m - top);
            m = top;
          }
          l *= a;
          check = __any_sync(0xFFFFFFFFu, is_far(m));
          if (is_far(m))
#pragma unroll
            for (int c = 0; c < 32; ++c) z[c] = far_score(z[c], scale, m);
          meeting.vote(false);                             // (top may be written again)
        }
        const float base = fabsf(m) > kFar ? 0.f : m;      // (−inf: the row has seen nothing, all its scores are −inf)
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float p0 = ex2(fmaf(z[2 * c], scale, -base)), p1 = ex2(fmaf(z[2 * c + 1], scale, -base));
          w[c] = bf_pack_weights(p0, p1);
          l += p0 + p1;
        }
        if (t + 1 < pc.t1 && !(ok = look(t + 1, tiles + 1))) break;
        // P and O are free once the last product has ended
        if (tiles >= 1 && !(ok = waits(&ms.p_free, (tiles - 1) & 1))) break;
        tc_fence_after();
        if (raised && t > pc.t0) {
#pragma unroll 1
          for (int q = 0; q < kHalf / 32; q += 2) {
            uint32_t o[16];
            const uint32_t oa = lanes + kColO + part * (kHalf / 2) + q * 16;
            tmem_ld<16>(oa, o);
            tmem_wait();
            regs_ready<16>(o);
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a);
            tmem_st<16>(oa, o);
            tmem_ld<16>(oa + 16, o);
            tmem_wait();
            regs_ready<16>(o);
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a);
            tmem_st<16>(oa + 16, o);
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(p_row + ((part * 4 + c) ^ (r_id & 7)) * 16) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        // a draft's row that only some rows see must not reach the others as
        // 0 · NaN: where it is not finite it becomes zero (see spoil for the rows that
        // see it)
        if (pc.mixed && pc.nkeys < (t + 1) * kKeys) {
          const int sl = tiles % kVs;
          if (!(ok = waits(&ms.v_full[sl], (tiles / kVs) & 1))) break;
          const int id = threadIdx.x - kFirstSoft * 32, key = id >> 2;
          if (t * kKeys + key >= pc.nkeys)                 // (a key past the last draft is zeros)
            clear_wild(smem + sl * kV + (id & 3) * kChunk + key * 128, &ms.wild[pb], t * kKeys + key - pc.nkeys);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full);
      }
      if (!ok || gone) break;
      // ---- the next piece's queries, once the last product has read P
      const int nb = pb ^ 1;
      if (!(ok = waits(&ms.piece_full[nb], ((pieces + 1) >> 1) & 1))) break;
      if (ms.piece[nb].t0 != ms.piece[nb].t1 && !(ok = load_q(ms.piece[nb], &ms.o_full, pieces & 1))) break;
      if (!(ok = waits(&ms.o_full, pieces & 1))) break;
      // ---- the sum over all keys, and this thread's 128 outputs
      ms.sum[part][r_id] = l;
      if (meeting.vote(false) && (gone = meeting.left())) break;
      const float z = ms.sum[0][r_id] + ms.sum[1][r_id];
      const bool whole = pc.slot < 0, have = r_id < pc.rows;
      float* slot = whole ? nullptr : part_slot(p, blockIdx.x, pc.slot);
      if (part == 0) {
        if (!whole) {
          slot[kRows * kHalf + r_id] = m;
          slot[kRows * kHalf + kRows + r_id] = z;
        } else if (p.lse && half == 0 && have) {
          p.lse[pc.row0 + r_id] = lse_of(m, z);
        }
      }
      const float inv = whole ? (z == 0.f ? 0.f : 1.f / z) : 1.f;
      tc_fence_after();
      const int64_t at = (pc.row0 + r_id) * kLat + half * kHalf + part * (kHalf / 2);
      float* mine = slot + (part * (kHalf / 2) * kRows + r_id * 8);   // [output / 8][row][8]: a warp's rows lie together
#pragma unroll 1
      for (int q = 0; q < kHalf / 2; q += 32) {
        uint32_t o[32];
        tmem_ld<16>(lanes + kColO + part * (kHalf / 2) + q, o);
        tmem_ld<16>(lanes + kColO + part * (kHalf / 2) + q + 16, o + 16);
        tmem_wait();
        regs_ready<32>(o);
        if (!have) {
          // (the loads are for all lanes)
        } else if (!whole || !p.out_bf16) {
          float* dst = whole ? static_cast<float*>(p.out) + at + q : mine + q * kRows;
          const int next = whole ? 8 : 8 * kRows;
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv);
#pragma unroll
          for (int c = 0; c < 4; ++c) st_global32(dst + c * next, o + 8 * c);
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + at + q;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            o[c] = bf_pack(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv);
          st_global32(dst, o);
          st_global32(dst + 16, o + 8);
        }
        __syncwarp();
      }
      if (const uint64_t wild = ms.wild[pb] & ms.mask[pb][r_id])     // (no mask past the last row)
        spoil_half(p, ms.piece[pb], wild, r_id, half, part);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.o_free);
        mbar_arrive(&ms.piece_empty[pb]);
      }
      ++pieces;
    }
    if (!gone) {
      if (ok && (p.fault & kFaultEnd) && part == 0) ok = waits(&ms.never, 0);
      meeting.part(ok);
    }
  }
  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

namespace tree {

int launch_tree_mla_wide(const CUtensorMap& tmap_q, const TreeParams& p, int ctas, cudaStream_t stream) {
  if (const int r = ensure_smem_limit(reinterpret_cast<const void*>(tree_mla_wide_kernel), kSmem)) return r;
  tree_mla_wide_kernel<<<static_cast<unsigned>(ctas), kThreads, kSmem, stream>>>(tmap_q, p);
  return check_launch();
}

}  // namespace tree
}  // namespace idx
