// Append to the paged latent cache (idx_latent_append): per new token the
// RMSNorm of its 512 latent features and the rotation of its 64 rotary
// features, written to the token's cache row; per query head the rotation of
// its 64 rotary features, written into the joined query.
//
// Memory-bound for prompts, latency-bound for decode steps: each output is a
// function of one token, nothing is read twice.  One warp is a task: a token's
// cache row (lane ↔ 16 latent features and one rotary pair, the sum of squares
// by shuffles), or 16 of its query heads (8 lanes ↔ one head's 128 bytes, four
// 16-byte loads in flight per lane), so that a decode step spreads over the SMs
// and every access is a 16-byte piece of a contiguous run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "api_internal.h"
#include "ptx.cuh"

namespace idx {
namespace {

constexpr int kLat = 512, kRot = 64, kRow = kLat + kRot;
constexpr int kTaskHeads = 16;             // query heads per warp
constexpr int kAppendThreads = 128;

struct AppendParams {
  const uint16_t* kv;
  int64_t kv_seq, kv_tok;
  const float* gain;
  float eps;
  const float *rope_cos, *rope_sin;
  const int32_t *positions, *counts, *table;
  int max_pages, B, n;
  uint16_t* cache;
  int num_pages, page_size;
  const uint16_t* q_pe;
  int64_t q_seq, q_tok, q_head;
  int H;
  uint16_t* q_out;
  int tasks_per_token;
  unsigned int* err;
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16);
}

// Eight consecutive rotary features (piece `sub` of a head's eight) turned.
// Half-split pairs (i, i + 32) lie four lanes apart: the partner's piece comes
// by shuffle, so all 32 lanes of the warp call this together.
template <bool kInterleaved>
__device__ __forceinline__ uint4 rotate8(uint4 v, const float* cs, const float* sn, int sub) {
  uint32_t x[4] = {v.x, v.y, v.z, v.w}, y[4];
  if (kInterleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = bf_lo(x[j]), b = bf_hi(x[j]);
      y[j] = bf_pack(a * cs[j] - b * sn[j], a * sn[j] + b * cs[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, x[j], 4);
      const float sign = sub < 4 ? -1.f : 1.f;      // first half: a·cos − b·sin, second: b·cos + a·sin
      y[j] = bf_pack(bf_lo(x[j]) * cs[2 * j] + sign * (bf_lo(o) * sn[2 * j]),
                     bf_hi(x[j]) * cs[2 * j + 1] + sign * (bf_hi(o) * sn[2 * j + 1]));
    }
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int64_t token = task / p.tasks_per_token;
  const int part = static_cast<int>(task - token * p.tasks_per_token);
  if (token >= static_cast<int64_t>(p.B) * p.n) return;
  const int b = static_cast<int>(token / p.n);
  const int i = static_cast<int>(token - static_cast<int64_t>(b) * p.n);
  const int cnt = p.counts ? __ldg(p.counts + b) : p.n;
  const int64_t first = __ldg(p.positions + b);
  const int64_t slots = static_cast<int64_t>(p.max_pages) * p.page_size;
  if (cnt < 0 || cnt > p.n) {
    if (i == 0 && part == 0 && lane == 0) raise_error(p.err, IDX_DEV_ERR_LENGTH);
    return;
  }
  if (i >= cnt) return;
  if (first < 0 || first + cnt > slots) {
    if (i == 0 && part == 0 && lane == 0) raise_error(p.err, IDX_DEV_ERR_POSITION);
    return;
  }
  const float* cs_row = p.rope_cos + token * (kRot / 2);
  const float* sn_row = p.rope_sin + token * (kRot / 2);

  if (part == 0) {
    // ---- the token's cache row
    const uint16_t* src = p.kv + b * p.kv_seq + i * p.kv_tok;
    const int64_t slot = first + i;
    const int page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + slot / p.page_size);
    // lane ↔ latent features 8·lane … + 7 and 256 + 8·lane … + 7
    uint4 v[2];
    float4 g[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[h] = __ldg(reinterpret_cast<const uint4*>(src) + h * 32 + lane);
      g[2 * h] = __ldg(reinterpret_cast<const float4*>(p.gain) + h * 64 + lane * 2);
      g[2 * h + 1] = __ldg(reinterpret_cast<const float4*>(p.gain) + h * 64 + lane * 2 + 1);
    }
    const float c = __ldg(cs_row + lane), s = __ldg(sn_row + lane);
    // lane ↔ rotary pair `lane`
    float a, w;
    if (kInterleaved) {
      const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(src + kLat) + lane);
      a = bf_lo(r);
      w = bf_hi(r);
    } else {
      a = bf_lo(__ldg(src + kLat + lane));
      w = bf_lo(__ldg(src + kLat + 32 + lane));
    }
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t x[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += bf_lo(x[j]) * bf_lo(x[j]) + bf_hi(x[j]) * bf_hi(x[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float r = 1.f / sqrtf(sum * (1.f / kLat) + p.eps);
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) raise_error(p.err, IDX_DEV_ERR_PAGE);
      return;
    }
    uint16_t* dst = p.cache + (static_cast<int64_t>(page) * p.page_size + slot % p.page_size) * kRow;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 g0 = g[2 * h], g1 = g[2 * h + 1];
      uint4 y;
      y.x = bf_pack(bf_lo(v[h].x) * r * g0.x, bf_hi(v[h].x) * r * g0.y);
      y.y = bf_pack(bf_lo(v[h].y) * r * g0.z, bf_hi(v[h].y) * r * g0.w);
      y.z = bf_pack(bf_lo(v[h].z) * r * g1.x, bf_hi(v[h].z) * r * g1.y);
      y.w = bf_pack(bf_lo(v[h].w) * r * g1.z, bf_hi(v[h].w) * r * g1.w);
      *(reinterpret_cast<uint4*>(dst) + h * 32 + lane) = y;
    }
    const uint32_t out = bf_pack(a * c - w * s, a * s + w * c);
    if (kInterleaved) {
      *(reinterpret_cast<uint32_t*>(dst + kLat) + lane) = out;
    } else {
      dst[kLat + lane] = static_cast<uint16_t>(out);
      dst[kLat + 32 + lane] = static_cast<uint16_t>(out >> 16);
    }
    return;
  }

  // ---- 16 query heads: 8 lanes per head, four heads per step
  const int sub = lane & 7;
  const int h0 = (part - 1) * kTaskHeads + (lane >> 3);
  const uint16_t* src = p.q_pe + b * p.q_seq + i * p.q_tok + sub * 8;
  uint4 v[kTaskHeads / 4];
#pragma unroll
  for (int j = 0; j < kTaskHeads / 4; ++j) {
    const int h = h0 + 4 * j;
    v[j] = h < p.H ? __ldg(reinterpret_cast<const uint4*>(src + h * p.q_head)) : make_uint4(0, 0, 0, 0);
  }
  // the angles of this lane's features: 4 pairs (interleaved), or 8 features of a half
  float cs[8], sn[8];
  constexpr int kAngles = kInterleaved ? 4 : 8;
  const int first_angle = kInterleaved ? 4 * sub : 8 * (sub & 3);
#pragma unroll
  for (int j = 0; j < kAngles; j += 4) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs_row + first_angle + j));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(sn_row + first_angle + j));
    cs[j] = c4.x, cs[j + 1] = c4.y, cs[j + 2] = c4.z, cs[j + 3] = c4.w;
    sn[j] = s4.x, sn[j + 1] = s4.y, sn[j + 2] = s4.z, sn[j + 3] = s4.w;
  }
  uint16_t* dst = p.q_out + token * p.H * kRow + kLat + sub * 8;
#pragma unroll
  for (int j = 0; j < kTaskHeads / 4; ++j) {
    const int h = h0 + 4 * j;
    const uint4 y = rotate8<kInterleaved>(v[j], cs, sn, sub);
    if (h < p.H) *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(h) * kRow) = y;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace idx

using namespace idx;

extern "C" int idx_latent_append(const uint16_t* kv_proj, int64_t kv_seq_pitch, int64_t kv_tok_pitch,
                                 const float* gain, float eps, const float* rope_cos, const float* rope_sin,
                                 int interleaved, const int32_t* positions, const int32_t* counts,
                                 const int32_t* page_table, int max_pages, int B, int n, uint16_t* cache,
                                 int num_pages, int page_size, const uint16_t* q_pe, int64_t q_seq_pitch,
                                 int64_t q_tok_pitch, int64_t q_head_pitch, int H, uint16_t* q_out,
                                 idx_stream_t stream) {
  constexpr int64_t kMaxRows = 0x7FFFFFFF;
  if (B < 0 || n < 0 || H < 0 || !(eps >= 0.f) || std::isinf(eps) || (interleaved != 0 && interleaved != 1))
    return IDX_ERR_SHAPE;
  if (B == 0 || n == 0) return IDX_OK;
  if (max_pages <= 0 || num_pages <= 0 || page_size <= 0 || static_cast<int64_t>(num_pages) * page_size > kMaxRows ||
      static_cast<int64_t>(max_pages) * page_size > kMaxRows)
    return IDX_ERR_SHAPE;
  if (!kv_proj || !gain || !rope_cos || !rope_sin || !positions || !page_table || !cache) return IDX_ERR_NULL;
  if (H > 0 && (!q_pe || !q_out)) return IDX_ERR_NULL;
  if (!aligned16(kv_proj) || !aligned16(gain) || !aligned16(rope_cos) || !aligned16(rope_sin) || !aligned16(cache) ||
      ((kv_seq_pitch | kv_tok_pitch) & 7))
    return IDX_ERR_ALIGN;
  if (H > 0 && (!aligned16(q_pe) || !aligned16(q_out) || ((q_seq_pitch | q_tok_pitch | q_head_pitch) & 7)))
    return IDX_ERR_ALIGN;
  AppendParams p;
  p.kv = kv_proj;
  p.kv_seq = kv_seq_pitch;
  p.kv_tok = kv_tok_pitch;
  p.gain = gain;
  p.eps = eps;
  p.rope_cos = rope_cos;
  p.rope_sin = rope_sin;
  p.positions = positions;
  p.counts = counts;
  p.table = page_table;
  p.max_pages = max_pages;
  p.B = B;
  p.n = n;
  p.cache = cache;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.q_pe = q_pe;
  p.q_seq = q_seq_pitch;
  p.q_tok = q_tok_pitch;
  p.q_head = q_head_pitch;
  p.H = H;
  p.q_out = q_out;
  p.tasks_per_token = 1 + static_cast<int>((static_cast<int64_t>(H) + kTaskHeads - 1) / kTaskHeads);
  const int64_t tokens = static_cast<int64_t>(B) * n;
  constexpr int kWarps = kAppendThreads / 32;
  if (tokens > (kMaxRows - 1) * kWarps / p.tasks_per_token) return IDX_ERR_SHAPE;
  const int64_t blocks = (tokens * p.tasks_per_token + kWarps - 1) / kWarps;
  p.err = device_error_word();
  if (!p.err) return check_launch();
  auto* s = reinterpret_cast<cudaStream_t>(stream);
  if (interleaved)
    latent_append_kernel<true><<<static_cast<unsigned>(blocks), kAppendThreads, 0, s>>>(p);
  else
    latent_append_kernel<false><<<static_cast<unsigned>(blocks), kAppendThreads, 0, s>>>(p);
  return check_launch();
}
