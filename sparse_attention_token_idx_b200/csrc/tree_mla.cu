// Latent attention of drafted token trees over the paged cache (idx_tree_mla).
// One CTA per (sequence, row, head); each warp walks every eighth key with a
// running maximum and sum, lane ↔ 18 features of the score and 16 of the output;
// the eight partial results are joined at the end.  fp32 on the CUDA cores.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "api_internal.h"
#include "ptx.cuh"

namespace idx {
namespace {

constexpr int kLat = 512, kRow = 576;
constexpr int kWarps = 8;

struct TreeParams {
  const uint16_t *q, *cache;
  const int32_t* table;
  int max_pages, num_pages, page_size;
  const int32_t *lengths, *counts;
  int B, n, H, max_len;
  const uint64_t* mask;
  const int32_t* indices;
  int k;
  float scale;
  void* out;
  int out_bf16;
  float* lse;
  unsigned int* err;
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__global__ void __launch_bounds__(kWarps * 32) tree_mla_kernel(const TreeParams p) {
  __shared__ float so[kWarps][kLat];
  __shared__ float sm[kWarps], sl[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;                       // (b·n + i)·H + h
  const int64_t bi = row / p.H;
  const int b = static_cast<int>(bi / p.n), i = static_cast<int>(bi % p.n);
  const int cnt = p.counts ? p.counts[b] : p.n;
  const int len = p.lengths[b];
  if (cnt < 0 || cnt > p.n || len < cnt || len > p.max_len) {
    if (threadIdx.x == 0) raise_error(p.err, IDX_DEV_ERR_LENGTH);
    return;
  }
  if (i >= cnt) return;
  const int ctx = len - cnt;
  const uint64_t bits = p.mask ? p.mask[bi] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1);
  const int first = p.indices ? p.k : ctx;              // keys before the drafts
  float q[18], o[16];
  const uint32_t* q32 = reinterpret_cast<const uint32_t*>(p.q + row * kRow);
#pragma unroll
  for (int j = 0; j < 9; ++j) {
    const uint32_t v = q32[j * 32 + lane];
    q[2 * j] = bf_lo(v);
    q[2 * j + 1] = bf_hi(v);
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int t = warp; t < first + cnt; t += kWarps) {
    int pos = t;
    if (t >= first) {
      if (!((bits >> (t - first)) & 1)) continue;
      pos = ctx + t - first;
    } else if (p.indices) {
      pos = p.indices[bi * p.k + t];
      if (pos < 0 || pos >= ctx) continue;
    }
    const int page = p.table[static_cast<int64_t>(b) * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) raise_error(p.err, IDX_DEV_ERR_PAGE);
      continue;
    }
    const uint32_t* kv = reinterpret_cast<const uint32_t*>(
        p.cache + (static_cast<int64_t>(page) * p.page_size + pos % p.page_size) * kRow);
    uint32_t v[9];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      v[j] = kv[j * 32 + lane];
      s = fmaf(q[2 * j], bf_lo(v[j]), s);
      s = fmaf(q[2 * j + 1], bf_hi(v[j]), s);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= p.scale;
    const float m_new = fmaxf(m, s);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float a = expf(m - base), w = expf(s - base);
    l = l * a + w;
    m = m_new;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[2 * j] = fmaf(w, bf_lo(v[j]), o[2 * j] * a);
      o[2 * j + 1] = fmaf(w, bf_hi(v[j]), o[2 * j + 1] * a);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    so[warp][(j * 32 + lane) * 2] = o[2 * j];
    so[warp][(j * 32 + lane) * 2 + 1] = o[2 * j + 1];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  const float base = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) sum += sl[w] * expf(sm[w] - base);
  for (int c = threadIdx.x; c < kLat; c += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += so[w][c] * expf(sm[w] - base);
    x = sum == 0.f ? 0.f : x / sum;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[row * kLat + c] = __float2bfloat16_rn(x);
    else
      static_cast<float*>(p.out)[row * kLat + c] = x;
  }
  if (p.lse && threadIdx.x == 0) p.lse[row] = base == 0.f && sum == 0.f ? -INFINITY : base + logf(sum);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace idx

using namespace idx;

extern "C" size_t idx_tree_mla_workspace_size(int B, int n, int H, int max_len, int k) {
  (void)B, (void)n, (void)H, (void)max_len, (void)k;
  return 0;
}

extern "C" int idx_tree_mla(const uint16_t* q, const uint16_t* cache, const int32_t* page_table, int max_pages,
                            int num_pages, int page_size, const int32_t* lengths, const int32_t* counts, int B, int n,
                            int H, int max_len, const uint64_t* tree_mask, const int32_t* indices, int k,
                            float softmax_scale, void* out, int out_dtype, float* lse, void* ws, size_t ws_bytes,
                            idx_stream_t stream) {
  constexpr int64_t kMaxRows = 0x7FFFFFFF;
  if (out_dtype != IDX_OUT_F32 && out_dtype != IDX_OUT_BF16) return IDX_ERR_FMT;
  if (B < 0 || n < 0 || n > IDX_MAX_DRAFTS || H <= 0 || k < 0 || !std::isfinite(softmax_scale)) return IDX_ERR_SHAPE;
  if (B == 0 || n == 0) return IDX_OK;
  if (max_pages <= 0 || num_pages <= 0 || page_size <= 0 || static_cast<int64_t>(num_pages) * page_size > kMaxRows ||
      static_cast<int64_t>(max_pages) * page_size > kMaxRows)
    return IDX_ERR_SHAPE;
  if (max_len <= 0 || max_len > static_cast<int64_t>(max_pages) * page_size) return IDX_ERR_SHAPE;
  if ((k > 0) != (indices != nullptr)) return indices ? IDX_ERR_K : IDX_ERR_NULL;
  if (!q || !cache || !page_table || !lengths || !out) return IDX_ERR_NULL;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(ws, 16) || !aligned(tree_mask, 8))
    return IDX_ERR_ALIGN;
  const int64_t rows = static_cast<int64_t>(B) * n * H;
  if (rows > kMaxRows) return IDX_ERR_SHAPE;
  if (ws_bytes < idx_tree_mla_workspace_size(B, n, H, max_len, k)) return IDX_ERR_SCRATCH;
  TreeParams p{q,       cache, page_table, max_pages, num_pages, page_size,     lengths, counts,
               B,       n,     H,          max_len,   tree_mask, indices,       k,       softmax_scale,
               out,     out_dtype == IDX_OUT_BF16, lse, nullptr};
  p.err = device_error_word();
  if (!p.err) return check_launch();
  tree_mla_kernel<<<static_cast<unsigned>(rows), kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return check_launch();
}
