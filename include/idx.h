/*
 * idx.h — C ABI of libidx.so, a B200 (sm_100a) implementation of the
 * DeepSeek-V3.2 lightning indexer's hot path:
 *
 *   keys:    rotate (scaled Hadamard-128) → block-FP8 quantise → append to the
 *            per-sequence FP8 key cache;
 *   scores:  S[t,s] = k_scale[s] · Σ_{h<64} w[t,h] · ReLU(q_fp8[t,h] · k_fp8[s]);
 *   select:  the min(k, visible) highest-scoring cached positions per query row.
 *
 * Around that path: the front end before it (the three projections on the
 * tensor cores: idx_project; query RoPE, key LayerNorm + RoPE, fused with the
 * quantiser: idx_front_quant_append), the attention after it
 * (sparse latent attention over the selected positions: idx_sparse_mla_decode),
 * and split-T selection of one sequence over several GPUs (idx_gather_scores,
 * idx_merge_topk).
 *
 * Sources (web pages on DeepSeek-V3.2-Exp's lightning indexer):
 *   "Index scores"          — score equation S^I, fp8_index docstring, Indexer.forward excerpt;
 *   "Index key cache"       — k_cache / k_scale_cache buffers, append before scoring;
 *   "Hadamard rotation"     — rotation equation and orthonormality note;
 *   NKI "DeepSeek-V3.2 Sparse Indexer Kernel API Reference" — caller-owned cache written in
 *                             place, int32 positions, int32 unordered top-k set, finite mask
 *                             bound, front-end parameters (cos / sin tables, LayerNorm gain, bias);
 *   "Join query parts"      — MQA decode excerpt: the attention that consumes the selection.
 *
 * Conventions for every call below.
 *   - All array arguments are DEVICE pointers to row-major, contiguous memory
 *     owned by the caller.  The library never allocates device memory and never
 *     synchronises in these calls; work is enqueued on `stream` (a cudaStream_t;
 *     NULL = the legacy default stream) and runs asynchronously.
 *   - bf16 arrays are passed as uint16_t bit patterns; FP8 arrays hold e4m3fn
 *     codes as uint8_t.
 *   - Index head count H = 64 and head dimension D = 128 are fixed.
 *   - Return value: IDX_OK (0) when the work was enqueued, or a negative IDX_ERR_*
 *     for an argument error detected on the host (nothing is enqueued then).
 *     Errors that depend on device data (positions, lengths) are detected in the
 *     kernels, which then skip the offending sequence and set a bit in a device
 *     error word; idx_status() reports and clears it.
 *   - Query row i (0 ≤ i < n) of sequence b sits at position lengths[b] − n + i
 *     (the call's new rows are the last n cached positions).  Key s is visible to
 *     that row iff s < lengths[b] and, when causal != 0, s ≤ its position.
 *     visible(b,i) = causal ? lengths[b] − n + i + 1 : lengths[b].
 *   - Scale format `fmt`: IDX_FMT_FP32 stores scale = fl32(max(amax,1e-4)/448);
 *     IDX_FMT_UE8M0 rounds that up to a power of two.  Both store float32.
 */
#ifndef IDX_H_
#define IDX_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define IDX_API __attribute__((visibility("default")))
#else
#define IDX_API
#endif

typedef struct CUstream_st* idx_stream_t;

#define IDX_HEADS 64
#define IDX_DIM 128
#define IDX_ROPE_DIM 64    /* leading features the rotary embedding turns */
#define IDX_MAX_LEN 131072 /* largest lengths[b] / max_len a score call accepts */

enum idx_fmt { IDX_FMT_FP32 = 0, IDX_FMT_UE8M0 = 1 };

/* Key-scale storage read by the *_ex score calls: fp32 values, or one e8m0
 * byte per key (OCP MX scale format: value 2^(byte − 127)), as written by
 * idx_quant_append_e8 — 129 instead of 132 cache bytes per key. */
enum idx_scale_storage { IDX_SCALE_F32 = 0, IDX_SCALE_E8M0 = 1 };

/* Score element type written by idx_score_ex. */
enum idx_score_dtype { IDX_SCORE_F32 = 0, IDX_SCORE_BF16 = 1 };

/* The most negative finite bfloat16, −(2 − 2^−7)·2^127: a finite mask value a
 * bf16 consumer reads unchanged ("DeepSeek-V3.2 Sparse Indexer Kernel API
 * Reference" page, Notes: masked slots are clamped to a finite bound because a
 * bf16 max-select turns −inf into NaN).  Exact in fp32. */
#define IDX_MASK_BOUND_BF16 (-3.38953138925153547590470800371487866880e+38f)

enum idx_status_code {
  IDX_OK = 0,
  IDX_ERR_NULL = -1,        /* a required pointer is NULL */
  IDX_ERR_SHAPE = -2,       /* a size is negative, zero where it must not be, or too large */
  IDX_ERR_FMT = -3,         /* fmt is not IDX_FMT_FP32 / IDX_FMT_UE8M0 */
  IDX_ERR_K = -4,           /* k <= 0 */
  IDX_ERR_ALIGN = -5,       /* a pointer is not 16-byte aligned where required */
  IDX_ERR_LAUNCH = -6,      /* the CUDA launch failed (the CUDA error is in idx_last_cuda_error) */
  IDX_ERR_DEVICE = -7,      /* idx_status: a kernel set the device error word */
  IDX_ERR_CUDA = -8,        /* idx_status: the stream itself reported a CUDA error */
  IDX_ERR_UNSUPPORTED = -9, /* no device code for this GPU (not sm_100) */
  IDX_ERR_SCRATCH = -10     /* the scratch is too small: idx_score_topk_noalloc's fixed scratch, idx_project's and
                               idx_tree_mla's ws */
};

/* Bits of the device error word (returned by idx_device_error_bits). */
#define IDX_DEV_ERR_TIMEOUT 0x1u  /* a bounded wait inside a kernel gave up */
#define IDX_DEV_ERR_POSITION 0x2u /* idx_quant_append: positions[b] < 0 or positions[b] + n > T_cap */
#define IDX_DEV_ERR_LENGTH 0x4u   /* score/top-k: lengths[b] < n (< 0 where causal = 0) or > max_len; the paged calls:
                                     a count or a length out of range */
#define IDX_DEV_ERR_PAGE 0x8u     /* the paged calls: a page number outside [0, num_pages) */

/*
 * idx_quant — "Hadamard rotation" page (rotation equation) followed by the
 * block-FP8 quantisation of groups of 128 features.
 *   x_bf16  [rows, 128]  bf16 input rows.
 *   x_fp8   [rows, 128]  out: e4m3 codes of fl32(y / scale), y = bf16(H·x/√128).
 *   x_scale [rows]       out: float32 scale per row.
 * rows may be 0 (nothing is enqueued).  x_bf16 and x_fp8 must be 16-byte aligned.
 */
IDX_API int idx_quant(const uint16_t* x_bf16, int64_t rows, uint8_t* x_fp8, float* x_scale, int fmt,
              idx_stream_t stream);

/*
 * idx_quant_queries — queries of `tokens` rows of 64 heads: the same rotation
 * and quantisation per (token, head), and the head weights folded as on the
 * "Index scores" page (1/√64 into the weights, 1/√128 with the query's scale):
 *   w[t,h] = fl32(fl32(fl32(w_raw[t,h]·0.125)·q_scale[t,h])·fl32(128^-1/2)).
 *   q_bf16 [tokens, 64, 128], w_raw [tokens, 64] float32 in;
 *   q_fp8 [tokens, 64, 128] out; w [tokens, 64] float32 out (the folded weights
 *   idx_score / idx_score_topk take).  The query scales are not stored.
 *   q_bf16 and q_fp8 must be 16-byte aligned.
 */
IDX_API int idx_quant_queries(const uint16_t* q_bf16, const float* w_raw, int64_t tokens, uint8_t* q_fp8, float* w,
                      int fmt, idx_stream_t stream);

/*
 * idx_quant_append — "Index key cache" page: rotate and quantise n new keys of
 * each of B sequences and write them in place at slots positions[b] … +n−1.
 *   k_bf16        [B, n, 128] bf16.
 *   positions     [B] int32 first slot per sequence.
 *   k_cache       [B, T_cap, 128] uint8 (e4m3), written in place.
 *   k_scale_cache [B, T_cap] float32, written in place.
 * A sequence with positions[b] < 0 or positions[b] + n > T_cap is skipped and
 * IDX_DEV_ERR_POSITION is raised.  k_bf16 and k_cache must be 16-byte aligned.
 */
IDX_API int idx_quant_append(const uint16_t* k_bf16, const int32_t* positions, int B, int n, uint8_t* k_cache,
                     float* k_scale_cache, int T_cap, int fmt, idx_stream_t stream);

/*
 * idx_quant_append_e8 — idx_quant_append with fmt = IDX_FMT_UE8M0 and each key's
 * power-of-two scale stored as its e8m0 byte (2^(byte − 127); the byte is the
 * fp32 exponent field of the scale) in k_scale_e8 [B, T_cap] uint8 — the "e8m0"
 * of the fp8_index docstring ("Index scores" page).  Read by the *_ex score
 * calls with IDX_SCALE_E8M0.  Arguments, alignment and errors as idx_quant_append.
 */
IDX_API int idx_quant_append_e8(const uint16_t* k_bf16, const int32_t* positions, int B, int n, uint8_t* k_cache,
                                uint8_t* k_scale_e8, int T_cap, idx_stream_t stream);

/*
 * idx_quant_queries_append — idx_quant_queries and idx_quant_append of one
 * indexer call in a single launch (the two are independent row sets of the
 * same rotation + quantisation).  Arguments as in the two calls; either part
 * may be empty (tokens = 0, or B = 0 / n = 0).
 */
IDX_API int idx_quant_queries_append(const uint16_t* q_bf16, const float* w_raw, int64_t tokens, uint8_t* q_fp8,
                                     float* w, const uint16_t* k_bf16, const int32_t* positions, int B, int n,
                                     uint8_t* k_cache, float* k_scale_cache, int T_cap, int fmt,
                                     idx_stream_t stream);

/*
 * idx_front_quant_append — the indexer's front end after its projections, in
 * the order of the Indexer.forward excerpt, fused with idx_quant_queries_append:
 * queries get the rotary embedding; keys get the LayerNorm (k_norm), then the
 * rotary embedding; both are then rotated and quantised, the keys appended and
 * the weights folded as in idx_quant_queries_append.
 *   q_proj [B, n, 64, 128] bf16: the query projection (wq_b of the low-rank
 *          query), 16-byte aligned.
 *   w_raw [B, n, 64] fp32: the weight projection of the hidden state.
 *   k_proj [B, n, 128] bf16: the key projection (wk of the hidden state), 16-byte aligned.
 *   rope_cos, rope_sin [B, n, IDX_ROPE_DIM / 2] fp32: cos θ_i and sin θ_i of
 *          each token's position (the NKI page's cos / sin tables); feature
 *          i and i + 32 (i < 32) are the pair turned by θ_i (not interleaved);
 *          features 64 … 127 are not turned.
 *   ln_gain, ln_bias [128] fp32, ln_eps ≥ 0: the key LayerNorm (biased
 *          variance, eps under the square root).
 *   positions, B, n, q_fp8, w, k_cache, k_scale_cache, T_cap, fmt: as in
 *          idx_quant_queries_append (tokens = B·n).
 * Arithmetic: float64 with one rounding per operation (sums over features in
 * feature order), each step's result rounded to bf16, then the rotation and
 * quantisation of idx_quant.  Errors as idx_quant_queries_append, plus
 * IDX_ERR_SHAPE for a negative, infinite or NaN ln_eps.
 */
IDX_API int idx_front_quant_append(const uint16_t* q_proj, const float* w_raw, const uint16_t* k_proj,
                                   const float* rope_cos, const float* rope_sin, const float* ln_gain,
                                   const float* ln_bias, float ln_eps, const int32_t* positions, int B, int n,
                                   uint8_t* q_fp8, float* w, uint8_t* k_cache, float* k_scale_cache, int T_cap,
                                   int fmt, idx_stream_t stream);

/*
 * idx_project — the three projections that open the Indexer.forward excerpt
 * ("Index scores" page): q = wq_b(qr) viewed as 64 heads of 128 features,
 * k = wk(x), and the head weights weights_proj(x.float()).
 *   x      [tokens, hidden] bf16 (hidden a multiple of 64), the hidden state.
 *   qr     [tokens, q_lora] bf16 (q_lora a multiple of 64), the low-rank query.
 *   wq_b   [64·128, q_lora] bf16, wk [128, hidden] bf16: Linear weights [out, in].
 *   w_proj [64, hidden] fp32.
 *   q_proj [tokens, 64, 128] bf16 out, k_proj [tokens, 128] bf16 out: the fp32
 *          products (tensor cores, fp32 accumulation) rounded to nearest-even bf16;
 *          ready for idx_front_quant_append.
 *   w_raw  [tokens, 64] fp32 out: Σ_k x·w_proj in fp32 on the tensor cores, with
 *          w_proj split into three bf16 parts hi + mid + lo (equal to it within
 *          2^-24 relative), each part's products summed in fp32, the three sums
 *          added (lo + mid) + hi.
 *   ws / ws_bytes: scratch of at least idx_project_workspace_size(tokens, hidden,
 *          q_lora) bytes (16-byte aligned, required): the three bf16 parts of
 *          w_proj (written every call) and the fp32 partial sums of products split
 *          over K when few tokens cannot fill the GPU (added in a fixed order).
 * All pointers except w_proj must be 16-byte aligned.  Errors: IDX_ERR_SHAPE,
 * IDX_ERR_NULL (ws included), IDX_ERR_ALIGN, IDX_ERR_SCRATCH (ws_bytes too small).
 */
IDX_API size_t idx_project_workspace_size(int64_t tokens, int hidden, int q_lora);
IDX_API int idx_project(const uint16_t* x, const uint16_t* qr, int64_t tokens, int hidden, int q_lora,
                        const uint16_t* wq_b, const uint16_t* wk, const float* w_proj, uint16_t* q_proj,
                        uint16_t* k_proj, float* w_raw, void* ws, size_t ws_bytes, idx_stream_t stream);

/*
 * idx_score — "Index scores" page: score equation and fp8_index docstring
 * (FP8 q·k → fp32 logits, ReLU, × head weight, sum over heads, × key scale),
 * with the causal mask of the Indexer.forward excerpt.
 *   q_fp8  [B, n, 64, 128] e4m3 codes; w [B, n, 64] folded weights (idx_quant_queries).
 *   k_cache [B, T_cap, 128], k_scale_cache [B, T_cap]; lengths [B] int32.
 *   causal = 1: the n rows are the sequence's last n keys, row i sees the keys up
 *            to its own: n ≤ lengths[b].  causal = 0: every row sees all lengths[b]
 *            keys, be they more than n, fewer or none (rows that are not cached).
 *   max_len: host-side upper bound on lengths[b], at least n (1 where causal = 0)
 *            and at most min(T_cap, IDX_MAX_LEN); it sizes the launch.
 *   scores [B, n, ld] float32 out: S for visible keys, −inf for every other column < ld.
 *          ld ≥ 1; columns ≥ ld are not computed.
 * q_fp8 and k_cache must be 16-byte aligned (they are read by TMA).
 */
IDX_API int idx_score(const uint8_t* q_fp8, const float* w, const uint8_t* k_cache, const float* k_scale_cache,
              const int32_t* lengths, int B, int n, int T_cap, int max_len, int causal, float* scores, int64_t ld,
              idx_stream_t stream);

/*
 * idx_score_ex — idx_score with the storage and output options of the NKI
 * indexer page (its Notes on the finite mask bound) and of the fp8_index
 * docstring (the key scale "e8m0 here"):
 *   k_scale      [B, T_cap] key scales: float32 (scale_fmt = IDX_SCALE_F32) or
 *                uint8 e8m0 bytes (IDX_SCALE_E8M0; T_cap a multiple of 16),
 *                16-byte aligned.
 *   scores       [B, n, ld] of score_dtype: IDX_SCORE_F32, or IDX_SCORE_BF16
 *                (each fp32 score rounded to nearest even).
 *   mask_value   written to every masked column: −inf as idx_score, or a
 *                finite bound such as IDX_MASK_BOUND_BF16 (NaN is rejected).
 * An e8m0 scale is the same power of two as the fp32 ue8m0 scale, so the
 * scores equal idx_score's on a cache filled with IDX_FMT_UE8M0.
 * Returns IDX_ERR_FMT for an unknown scale_fmt or score_dtype.
 */
IDX_API int idx_score_ex(const uint8_t* q_fp8, const float* w, const uint8_t* k_cache, const void* k_scale,
                         int scale_fmt, const int32_t* lengths, int B, int n, int T_cap, int max_len, int causal,
                         void* scores, int64_t ld, int score_dtype, float mask_value, idx_stream_t stream);

/*
 * idx_score_visible — the scores of idx_score for the visible keys only, as
 * the score + top-k path computes them into its workspace: one persistent CTA
 * per SM, each streaming an equal share of all (row block, 128-key tile)
 * pairs of the call.
 *   Arguments as in idx_score, with ld ≥ max_len and w 16-byte aligned.
 *   scores [B, n, ld]: S for visible keys, −inf from each row's visible count
 *          up to the end of its last 128-key tile; columns past that tile are
 *          left unwritten (their contents are unspecified).
 * Calls with more than 4096 blocks of query rows are served by idx_score.
 */
IDX_API int idx_score_visible(const uint8_t* q_fp8, const float* w, const uint8_t* k_cache,
                              const float* k_scale_cache, const int32_t* lengths, int B, int n, int T_cap,
                              int max_len, int causal, float* scores, int64_t ld, idx_stream_t stream);

/*
 * idx_topk — Indexer.forward excerpt (top min(index_topk, ·) per row) and the
 * NKI page's output convention (int32, unordered set), on scores already in memory.
 *   scores [B, n, ld] float32 (finite for visible keys); lengths [B]; causal as above.
 *   indices [B, n, k] int32 out: the k_t = min(k, visible(b,i)) positions with the
 *   highest scores, in unspecified order, in columns 0 … k_t−1; columns k_t … k−1
 *   hold −1.  Ties at the k_t-th score are broken arbitrarily.
 *   max_len as in idx_score (and ≤ ld).  ws / ws_bytes: not used, pass NULL / 0.
 */
IDX_API int idx_topk(const float* scores, const int32_t* lengths, int B, int n, int64_t ld, int max_len, int causal, int k,
             int32_t* indices, void* ws, size_t ws_bytes, idx_stream_t stream);

/*
 * Split-T selection: one sequence's keys split over G GPUs (or G slices on one
 * GPU).  The Indexer.forward excerpt selects the row's top min(index_topk, ·)
 * and then checks with a broadcast that every rank agrees; here each rank
 * selects the k best of its own slice (idx_topk on its scores), turns them into
 * (score, global position) pairs with idx_gather_scores, the ranks exchange the
 * pairs (one all-gather of k·8 bytes per row), and idx_merge_topk selects the
 * row's k best among the G·k candidates.  Exact: a key of the row's top k is in
 * its own slice's top k.
 */
typedef struct {
  float score;   /* the key's score */
  int32_t pos;   /* its position in the whole sequence; −1 marks an empty slot */
} idx_cand_t;    /* 8 bytes */

/*
 * idx_gather_scores
 *   scores [rows, ld] float32 (device): this slice's scores, row r at r·ld.
 *   idx [rows, k] int32 (device): slice-local positions from idx_topk, −1 = empty.
 *   counts [rows] int32 (device) or NULL: keys of row r held in this slice;
 *          positions ≥ counts[r] count as empty.  (A slice holding none of a
 *          row's keys is scored and selected with a length of 1 — the scorer
 *          requires lengths ≥ n — and its one position is dropped here.)
 *   offset: the slice's first global position (added to every valid position).
 *   cand [rows, k] idx_cand_t (device, caller-owned, 8-byte aligned) out:
 *   (scores[r·ld + idx], idx + offset); empty slots give (−inf, −1).
 *   Errors: IDX_ERR_SHAPE (rows, k < 0 or ld ≤ 0), IDX_ERR_NULL; nothing to do
 *   when rows·k = 0.
 */
IDX_API int idx_gather_scores(const float* scores, int64_t ld, const int32_t* idx, int64_t rows, int k,
                              const int32_t* counts, int32_t offset, idx_cand_t* cand, idx_stream_t stream);

/*
 * idx_merge_topk
 *   cand [G, rows, kin] idx_cand_t (device): rank g's candidates of row r at
 *   (g·rows + r)·kin — the layout of an all-gather of the per-rank [rows, kin]
 *   outputs of idx_gather_scores.  Empty slots (pos −1) are skipped; the others
 *   need finite scores and distinct positions.
 *   out [rows, k] int32 (device, caller-owned): the positions of the
 *   k_t = min(k, valid candidates) highest scores in columns 0 … k_t−1 (a set,
 *   ties at the k_t-th score broken arbitrarily), −1 after.
 *   Limits: G·kin ≤ 16384.  Errors: IDX_ERR_SHAPE, IDX_ERR_K (k ≤ 0), IDX_ERR_NULL.
 *   One CTA per row.
 */
IDX_API int idx_merge_topk(const idx_cand_t* cand, int G, int64_t rows, int kin, int k, int32_t* out,
                           idx_stream_t stream);

/*
 * idx_sparse_mla_decode — the attention that consumes the selection ("Join
 * query parts" page, MQA decode excerpt): for one decode token per sequence,
 * each head scores the selected cache rows, takes the softmax over them and
 * returns the latent output.
 *   q [B, H, 576] bf16: per head the absorbed content query (512) followed by
 *          the rotary query (64); H a multiple of 16.
 *   kv [B, T_cap, 576] bf16 (16-byte aligned): per position the latent (512)
 *          followed by the rotary key (64).
 *   indices [B, k] int32: the selected positions (the indexer's output for the
 *          token); entries < 0 or ≥ T_cap select nothing.
 *   softmax_scale: finite; s = softmax_scale · q·kv.
 *   out [B, H, 512] fp32 (caller-owned): Σ_t softmax(s)_t · kv[t, 0:512]
 *          over the selected t; 0 for a row that selects nothing.
 * Arithmetic: when H is a multiple of 128 (and q 16-byte aligned), on the
 * tensor cores — bf16 products accumulated in fp32, the softmax weights
 * rounded to bf16 for the weighted sum (their sum taken as rounded), chunks of
 * 64 positions; otherwise fp32 on the CUDA cores (online softmax over chunks
 * of 32 positions).  Errors: IDX_ERR_SHAPE (B < 0, H not a positive multiple of 16,
 * T_cap ≤ 0, a non-finite scale), IDX_ERR_K (k ≤ 0), IDX_ERR_NULL, IDX_ERR_ALIGN.
 */
IDX_API int idx_sparse_mla_decode(const uint16_t* q, const uint16_t* kv, const int32_t* indices, int B, int H,
                                  int64_t T_cap, int k, float softmax_scale, float* out, idx_stream_t stream);

/*
 * The paged latent cache: cache [num_pages, page_size, 576] bf16, one row per
 * position (512 latent features, then the 64 rotated ones).  Position t of
 * sequence b is row t mod page_size of page page_table[b, t / page_size]
 * (page_table [B, max_pages] int32; entries past a sequence's last position are
 * not read).  page_size is any number ≥ 1; sequences may share pages that
 * neither of them writes.  num_pages · page_size < 2^31, max_pages · page_size < 2^31.
 *
 * idx_latent_append — the new tokens' rows: the latent's RMSNorm, the rotation
 * of the shared rotary key, and the write into the paged cache; and, in the
 * same launch, the rotation of the queries' rotary part into the joined queries
 * that idx_tree_mla reads.
 *   kv_proj  [B, n, 576] bf16: the latent and the rotary key as projected, in
 *            rows kv_tok_pitch elements apart, sequences kv_seq_pitch apart (the
 *            tail of a wider projection is read in place); 16-byte aligned,
 *            pitches multiples of 8.
 *   gain     [512] fp32, eps ≥ 0: latent[j] = bf16(x[j] · (Σx²/512 + eps)^-1/2 · gain[j]).
 *   rope_cos, rope_sin [B, n, 32] fp32 of each token's position (for a tree of
 *            drafts its depth after the context, not its slot).  interleaved = 1:
 *            features 2i and 2i + 1 are the pair turned by θ_i; 0: features i and
 *            i + 32.
 *   positions [B] int32: slot of each sequence's first new token; token i goes
 *            to slot positions[b] + i.
 *   counts   [B] int32 or NULL (all n): sequence b has counts[b] ≤ n new tokens;
 *            nothing is read, written or checked for the rows behind them.
 *   q_pe     [B, n, H, 64] bf16 or NULL (H = 0), with pitches in elements as
 *            kv_proj's; q_out [B, n, H, 576] bf16: features 512 … 575 are written,
 *            the first 512 (the absorbed content query) are left alone.
 * fp32 arithmetic, one rounding to bf16 per output.  All pointers but positions,
 * counts and page_table are 16-byte aligned.  A sequence whose slots are
 * negative or pass max_pages · page_size raises IDX_DEV_ERR_POSITION and one
 * with counts[b] outside [0, n] IDX_DEV_ERR_LENGTH: neither writes anything (its
 * queries included).  A token whose page number is outside [0, num_pages)
 * raises IDX_DEV_ERR_PAGE and its cache row is not written.  Two tokens of a call
 * that share a slot (of sequences that share its page) leave features of both there.
 */
IDX_API int idx_latent_append(const uint16_t* kv_proj, int64_t kv_seq_pitch, int64_t kv_tok_pitch, const float* gain,
                              float eps, const float* rope_cos, const float* rope_sin, int interleaved,
                              const int32_t* positions, const int32_t* counts, const int32_t* page_table,
                              int max_pages, int B, int n, uint16_t* cache, int num_pages, int page_size,
                              const uint16_t* q_pe, int64_t q_seq_pitch, int64_t q_tok_pitch, int64_t q_head_pitch,
                              int H, uint16_t* q_out, idx_stream_t stream);

/* Element type of idx_tree_mla's out. */
enum idx_out_dtype { IDX_OUT_F32 = 0, IDX_OUT_BF16 = 1 };
#define IDX_MAX_DRAFTS 64 /* rows per sequence of idx_tree_mla: the bits of a tree mask */

/*
 * idx_tree_mla — latent attention of each sequence's last rows over its paged
 * cache: a tree of drafted tokens (speculative decoding), a chain of new tokens,
 * or one decode token (n = 1); over the whole context, or over the positions
 * that the indexer selected for each row.  The rows' own cache rows are appended
 * first (idx_latent_append).
 *   q        [B, n, H, 576] bf16, 1 ≤ n ≤ IDX_MAX_DRAFTS, H ≥ 1.
 *   lengths  [B] int32: cached positions including the drafts; counts [B] int32
 *            or NULL (all n).  Row i < counts[b] is draft i, at slot ctx + i with
 *            ctx = lengths[b] − counts[b].  Outputs of rows behind counts[b] are
 *            left as they were.
 *   max_len  host bound: lengths[b] ≤ max_len ≤ max_pages · page_size.
 *   tree_mask [B, n] uint64 or NULL (a chain: row i sees drafts 0 … i): row i
 *            sees draft j < counts[b] iff bit j of tree_mask[b, i] is set.
 *   indices  [B, n, k] int32 or NULL (the whole context, k = 0): the context
 *            positions row i attends to, in any order, as idx_score_topk gives
 *            them; entries outside [0, ctx) select nothing, a position named
 *            twice counts twice.  The drafts are seen as by tree_mask either way.
 *   s[t] = softmax_scale · Σ_d q[d] · row_t[d];  p = softmax of s over the row's positions
 *   out      [B, n, H, 512] of out_dtype: Σ_t p[t] · row_t[0:512].
 *   lse      [B, n, H] fp32 or NULL: ln Σ_t exp(s[t]) (joins results over other keys).
 *   A row that sees nothing gives out = 0, lse = −inf.  Cache rows that a
 *   sequence does not hold are never read as numbers.
 *   ws / ws_bytes: at least idx_tree_mla_workspace_size(B, n, H, max_len, k)
 *            bytes, 32-byte aligned (may be NULL where that is 0).  It holds
 *            partial results inside the call: calls (or captured graphs) that may
 *            run at the same time need one each.
 * q, cache: 16-byte aligned; out, ws 32; tree_mask 8.  Scores, the sum of the
 * weights (lse), and the output's sums are fp32; the weights themselves are rounded
 * to bf16 before they are multiplied with the rows, for the tensor cores: 2^-8 of
 * each at most, which out carries in both of its types, IDX_OUT_F32 too.
 * softmax_scale may be negative or 0; |softmax_scale| · log2 e must be finite in fp32.
 * A score beyond 2^128 · ln 2 = 2.36e38 in size counts as infinite.
 * Errors: IDX_ERR_SHAPE, IDX_ERR_NULL, IDX_ERR_ALIGN, IDX_ERR_FMT (out_dtype),
 * IDX_ERR_SCRATCH.  counts[b] outside [0, n], lengths[b] < counts[b] or
 * lengths[b] > max_len raise IDX_DEV_ERR_LENGTH and leave the sequence's outputs as
 * they were; a page number outside [0, num_pages) raises IDX_DEV_ERR_PAGE and its
 * positions are not seen.
 */
IDX_API size_t idx_tree_mla_workspace_size(int B, int n, int H, int max_len, int k);
IDX_API int idx_tree_mla(const uint16_t* q, const uint16_t* cache, const int32_t* page_table, int max_pages,
                         int num_pages, int page_size, const int32_t* lengths, const int32_t* counts, int B, int n,
                         int H, int max_len, const uint64_t* tree_mask, const int32_t* indices, int k,
                         float softmax_scale, void* out, int out_dtype, float* lse, void* ws, size_t ws_bytes,
                         idx_stream_t stream);

/*
 * idx_score_topk — scores and top-k in one call, arguments as in idx_score /
 * idx_topk.  Decode-shaped calls (n ≤ 2) run one kernel in which a row's scores
 * never leave on-chip memory.  Prefill-shaped calls (n > 2) given a workspace of
 * at least idx_workspace_size(B, n, max_len, k) bytes (16-byte aligned) write
 * the scores there and select with the top-k kernel (faster: selections of
 * different rows overlap); without one they use the single-kernel path.
 */
IDX_API int idx_score_topk(const uint8_t* q_fp8, const float* w, const uint8_t* k_cache, const float* k_scale_cache,
                   const int32_t* lengths, int B, int n, int T_cap, int max_len, int causal, int k,
                   int32_t* indices, void* ws, size_t ws_bytes, idx_stream_t stream);

/*
 * idx_score_topk_ex — idx_score_topk with the key scales stored as fp32
 * (scale_fmt = IDX_SCALE_F32) or as e8m0 bytes (IDX_SCALE_E8M0, T_cap a
 * multiple of 16).  The selected set equals idx_score_topk's on a cache filled
 * with IDX_FMT_UE8M0.
 */
IDX_API int idx_score_topk_ex(const uint8_t* q_fp8, const float* w, const uint8_t* k_cache, const void* k_scale,
                              int scale_fmt, const int32_t* lengths, int B, int n, int T_cap, int max_len,
                              int causal, int k, int32_t* indices, void* ws, size_t ws_bytes, idx_stream_t stream);

/*
 * idx_score_topk_noalloc — idx_score_topk for callers that cannot allocate
 * device memory when they call (for example while their stream is being
 * captured into a CUDA graph, or inside a plugin enqueue step that must not
 * allocate).  The pages have no counterpart: this is a deployment variant.
 * Prefill-shaped calls keep their score workspace in a buffer the library
 * owns: a file-scope device array of 64 MiB (B·n·max_len ≤ 16 Mi scores),
 * held on every GPU that loads the library until the process exits.  Larger
 * calls return IDX_ERR_SCRATCH before anything is enqueued — for example two
 * sequences of 2048 new rows over 16 384 keys (256 MiB of scores): call
 * idx_score_topk with a workspace for those.  Decode-shaped calls need no scratch.
 *   - The first call on a device, of any shape, looks up the buffer's device
 *     address (no allocation); make that first call before any stream capture.
 *   - Every call reuses the same buffer and rewrites all of the part it uses,
 *     so nothing needs clearing, but calls that overlap on the GPU (other
 *     streams, other threads) race on it: serialise them.
 *   - It calls no cudaMalloc / cudaFree; arguments otherwise as idx_score_topk.
 */
IDX_API int idx_score_topk_noalloc(const uint8_t* q_fp8, const float* w, const uint8_t* k_cache,
                                   const float* k_scale_cache, const int32_t* lengths, int B, int n, int T_cap,
                                   int max_len, int causal, int k, int32_t* indices, idx_stream_t stream);

/* Workspace bytes idx_score_topk uses for these sizes: 0 for decode-shaped
 * calls (n ≤ 2), B·n·max_len·4 (fp32 scores) for prefill-shaped ones. */
IDX_API size_t idx_workspace_size(int B, int n, int max_len, int k);

/*
 * idx_status — synchronises `stream`, then reads and clears the device error
 * word.  Returns IDX_OK, IDX_ERR_DEVICE (bits available from
 * idx_device_error_bits) or IDX_ERR_CUDA.
 */
IDX_API int idx_status(idx_stream_t stream);
IDX_API unsigned int idx_device_error_bits(void); /* bits seen by the last idx_status call */
IDX_API const char* idx_error_string(int code);
IDX_API int idx_last_cuda_error(void); /* cudaError_t of the last failed launch, 0 if none */

/*
 * idx_e4m3_encode — the float32 → e4m3fn conversion the quantiser uses (round to
 * nearest even, saturate to ±448, sign of zero kept), exposed so that it can be
 * checked value by value.  x [count] float32 in, out [count] uint8 codes.
 */
IDX_API int idx_e4m3_encode(const float* x, int64_t count, uint8_t* out, idx_stream_t stream);

/*
 * Fault-injection control for tests: when `flags` has bit 0 set, the next score
 * and idx_tree_mla launches make one bounded wait in each CTA wait for a barrier
 * that nothing signals, with the wait budget set to `budget_ns`; the kernels then
 * report IDX_DEV_ERR_TIMEOUT and return.  Bit 2: in idx_tree_mla launches, one of
 * the softmax warps that share rows waits so where its CTA's work has ended (its
 * results are written by then).  idx_debug_set(0, 0) restores normal operation (2 s
 * wait budget).
 */
IDX_API void idx_debug_set(unsigned int flags, unsigned long long budget_ns);

/*
 * Profiling aid: when the debug flags have bit 1 set, score launches record per
 * CTA (first 8192 CTAs) 16 words: [0] entry, [1] set-up done, [2] first
 * accumulator ready, [3] key stream done, [4] selection done, [5] exit
 * (globaltimer ns), [7] SM id, [8..14] steps inside the first row's
 * selection, [15] its candidate count.  idx_debug_trace copies them to
 * host_out (max_ctas × 16 words) after synchronising the device.
 */
IDX_API int idx_debug_trace(unsigned long long* host_out, int max_ctas);

#ifdef __cplusplus
}
#endif

#endif /* IDX_H_ */
