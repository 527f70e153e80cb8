/*
 * v4a — one layer of DeepSeek-V4-style hybrid compressed attention on one GB300 (sm_103a).
 *
 * C ABI of the library. Every call is asynchronous on the caller's CUDA stream, allocates
 * nothing, keeps no state between calls and may be called from several host threads.
 * All pointers named "device" point to device memory owned by the caller; the library
 * never frees or retains them after the call returns (the kernels it enqueued may still
 * be reading them until the stream reaches that point). Structs passed by pointer
 * (v4a_layer_cfg, v4a_cache) live in host memory and are copied during the call.
 *
 * Sources (page title, section):
 *   [notes] "DeepSeek V4 in vLLM 技术博客详尽笔记" (vllm-deepseek-v4-notes.pages.dev)
 *   [blog]  "vLLM DeepSeek V4 支援：高效長上下文注意力" (agentlenshq.com)
 *   [serve] "DeepSeek-V4服务：百万token上下文成为推理系统难题" (ai-pulse-lab.com)
 *
 * Paged layout ([notes] 解决方案一：统一逻辑块大小): every cache is split into logical
 * blocks of 256 native token positions. A block of a c4a entry cache holds 64 entries,
 * a block of a c128a entry cache holds 2 entries, a block of a token cache (sliding
 * window, compressor residual) holds 256 tokens. Row r of sequence b (a token position or
 * an entry index) lives in logical block r / R (R = rows per block), whose physical page
 * is block_table[b * max_blocks + r / R]; its pool row ("slot") is page * R + r % R.
 * A page of -1 means the block is not allocated.
 *
 * Error behaviour: every call first validates its host-visible arguments and returns
 * V4A_ERR_ARG or V4A_ERR_UNSUPPORTED without enqueuing anything. A failed launch returns
 * V4A_ERR_CUDA. Problems only the device can see (a needed row whose block has no page, a
 * page id outside the pool, a top-k entry that is not visible to its query) are OR-ed
 * into the caller's device error word `dev_err` (may be NULL to ignore them); the affected
 * row or query is skipped or zeroed, never read out of bounds. v4a_get_error() reads and
 * clears that word.
 */
#ifndef V4A_H
#define V4A_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* v4a_stream_t; /* a cudaStream_t; NULL = legacy default stream */

/* return codes */
#define V4A_OK 0
#define V4A_ERR_ARG (-1)          /* NULL pointer, misaligned pointer, inconsistent sizes */
#define V4A_ERR_UNSUPPORTED (-2)  /* dims / dtype / kind without a kernel */
#define V4A_ERR_CUDA (-3)         /* a CUDA launch or runtime call failed */
#define V4A_ERR_DEVICE (-4)       /* v4a_get_error found device-side error bits */
#define V4A_ERR_TOO_LARGE (-5)    /* the request exceeds the fixed scratch of v4a_index_topk_noalloc */

/* device error word bits */
#define V4A_DEV_MISSING_PAGE 1u   /* a row the computation needs is in a block with no page */
#define V4A_DEV_BAD_PAGE 2u       /* a block table names a page >= n_pages */
#define V4A_DEV_BAD_INDEX 4u      /* a top-k list names an entry its query may not see */
#define V4A_DEV_BAD_POS 8u        /* a query position above the max_pos the call was sized for;
                                     the query's rows beyond that bound are ignored */
#define V4A_DEV_TIMEOUT 16u       /* a bounded wait inside a kernel gave up (about 1 s); the
                                     kernel drained its copies, released its tensor memory and
                                     returned; its outputs are incomplete */
#define V4A_DEV_NO_PAGE 32u       /* the pool has no free page left for a block that needs one */

/* layer kinds ([notes] 四大核心技术; 数学附录精要) */
#define V4A_C4A 0                 /* entry = weighted sum of 8 tokens at stride 4 */
#define V4A_C128A 1               /* entry = weighted sum of 128 tokens at stride 128 */

/* arithmetic / storage */
#define V4A_FP32 0                /* fp32 inputs, fp32 caches, fp32 output */
#define V4A_BF16_FP8 1            /* bf16 inputs, fp8 e4m3 caches + fp32 row scale, bf16 output */
#define V4A_BF16 2                /* bf16 inputs, bf16 caches, bf16 output (v4a_rope, v4a_latent_*) */

/* indexer-cache formats (v4a_layer_cfg.idx_format) */
#define V4A_IDX_DEFAULT 0         /* the layer's cache type: fp8 e4m3 (BF16_FP8) or fp32 (FP32) */
#define V4A_IDX_FP4 1             /* e2m1 codes, two per byte (element 2i in the low nibble), and
                                     one fp32 scale per row: scale = max|y| / 6 (1 for a zero row),
                                     code = round-to-nearest-even of y / scale saturated to +-6
                                     ([notes] 四大核心技术 and [blog] KV 快取記憶體管理: the fp4
                                     indexer cache; the block of one scale is the whole row).
                                     BF16_FP8 layers with d_I = 128 only. */

typedef struct v4a_layer_cfg {
  int32_t kind;          /* V4A_C4A or V4A_C128A */
  int32_t dtype;         /* V4A_FP32 or V4A_BF16_FP8 */
  int32_t head_dim;      /* D: dim of the shared K=V head and of each query head */
  int32_t rope_dim;      /* d_r: the last d_r dims are rotated, as adjacent pairs */
  int32_t n_heads;       /* H: query heads */
  int32_t idx_heads;     /* H_I: indexer heads (c4a) */
  int32_t idx_dim;       /* d_I: indexer head dim (c4a) */
  int32_t window;        /* W: tokens per entry (8 for c4a, 128 for c128a) */
  int32_t stride;        /* S: tokens between entries (4 / 128) */
  int32_t win_off;       /* entry j covers S*j+win_off .. S*j+win_off+W-1, win_off in (-W, 0] */
  int32_t swa;           /* sliding window: a query at p sees tokens [p-swa+1, p] */
  float rope_base;       /* theta_i = rope_base^(-2i/d_r) */
  float rms_eps;         /* RMSNorm epsilon of compressed entries */
  float softmax_scale;   /* logit scale, usually 1/sqrt(D) */
  int32_t idx_format;    /* V4A_IDX_DEFAULT or V4A_IDX_FP4 (c4a indexer cache) */
} v4a_layer_cfg;

typedef struct v4a_cache {
  void* data;                  /* device: [n_pages*rows_per_block, row_width] elements; e4m3
                                  bytes for fp8 pools, fp32 or bf16 for the others */
  float* scale;                /* device: [n_pages*rows_per_block] row scales (fp8 pools), else NULL */
  const int32_t* block_table;  /* device: [n_seq, max_blocks] physical page per logical block, -1 = none */
  int32_t max_blocks;          /* columns of block_table */
  int32_t rows_per_block;      /* 64 (c4a entries), 2 (c128a entries), 256 (token caches) */
  int64_t n_pages;             /* pages in the pool (bounds check of block-table values) */
  int32_t row_width;           /* elements per row (an fp4 row holds two per byte) */
  int32_t reserved;            /* must be 0 */
} v4a_cache;

/*
 * v4a_compress_insert — insert one step's new tokens of every sequence (steps a1-a5).
 *
 * [blog] GPU 計算飽和度 / [notes] 优化一：三大内核融合 (fusion 1: compressor + RMSNorm +
 * RoPE + cache insert; fusion 3's KV RoPE + K insert) and [notes] 解决方案二 (the compressor
 * state kept as sliding-window KV).
 *
 * Sequence b owns input rows cu_tokens[b] .. cu_tokens[b+1]-1 at positions
 * start_pos[b] + (row - cu_tokens[b]). For every new token t:
 *   - swa row t      = RoPE(kv_t, t), stored (fp8: per-row scale amax/448, e4m3 RNE);
 *   - state row t    = raw (kv_t | s_t | ik_t | is_t) if t is among the last W positions of
 *                      the sequence's new tokens (what later calls can still need);
 *   - if t completes entry j (t = S*j + win_off + W - 1, j >= 0):
 *       attn row j   = RoPE(RMSNorm(sum_o softmax_o(s + bias[o]) * kv) * gamma, S*j),
 *       idx row j    = sum_o softmax_o(is + ibias[o]) * ik (c4a only; no norm, no RoPE),
 *     where the window's tokens before start_pos[b] are read from the state cache.
 * Rows whose block has no page are not written (a needed state row without a page sets
 * V4A_DEV_MISSING_PAGE and the entry is skipped).
 *
 * kv, score:    device [n_tokens, D]    (fp32 or bf16 per cfg->dtype)
 * ikv, iscore:  device [n_tokens, d_I]  (c4a; NULL for c128a)
 * bias:         device fp32 [W, D];  gamma: device fp32 [D];  ibias: device fp32 [W, d_I] (c4a)
 * cu_tokens:    device int32 [n_seq+1], non-decreasing, cu_tokens[n_seq] == n_tokens
 * start_pos:    device int64 [n_seq]
 * attn:  entry cache (rows_per_block = 256/S, row_width = D)
 * idx:   indexer-key cache (c4a: rows_per_block 64, row_width d_I; NULL for c128a)
 * swa:   token cache (rows_per_block 256, row_width D)
 * state: token cache of raw rows (rows_per_block 256, row_width 2D (+2 d_I for c4a)),
 *        element type of the inputs.
 * Pool data pointers and kv, score, ikv, iscore, bias, gamma, ibias must be 16-byte
 * aligned (V4A_ERR_ARG otherwise).
 */
int v4a_compress_insert(const v4a_layer_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                        const int32_t* cu_tokens, const int64_t* start_pos,
                        const void* kv, const void* score, const float* bias,
                        const float* gamma, const void* ikv, const void* iscore,
                        const float* ibias, const v4a_cache* attn, const v4a_cache* idx,
                        const v4a_cache* swa, const v4a_cache* state, int32_t* dev_err,
                        v4a_stream_t stream);

/*
 * v4a_compress_insert_qnorm — v4a_compress_insert plus the per-head query RMSNorm of the
 * step's queries, in the same launch.
 *
 * [notes] 优化一：三大内核融合, fusion 3 (Q Norm + KV RoPE + K Insert, static warp-ID
 * dispatch: every warp handles one Q head or one K row on its own). The launch's first
 * n_tokens warps do exactly what v4a_compress_insert does; each of the next n_q * H warps
 * takes one (query, head) row:
 *   q_out[i, h, :] = q_gamma * q[i, h, :] / sqrt(mean(q[i, h, :]^2) + cfg->rms_eps),
 * computed in fp32 and stored in the input type (bf16 round-to-nearest-even or fp32).
 *
 * n_q:      queries (>= 0); n_q = 0 makes the call v4a_compress_insert
 * q:        device [n_q, H, D] (fp32 or bf16 per cfg->dtype), 16-byte aligned
 * q_gamma:  device fp32 [D], 16-byte aligned, shared by the heads
 * q_out:    device [n_q, H, D], same type, 16-byte aligned; q_out == q normalises in place,
 *           any other overlap with q returns V4A_ERR_ARG
 * The insert arguments are checked only when n_tokens > 0, so n_tokens = 0 runs the norm
 * alone. Errors: as v4a_compress_insert, plus V4A_ERR_ARG for a NULL, misaligned or
 * partially overlapping query buffer.
 */
int v4a_compress_insert_qnorm(const v4a_layer_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                              const int32_t* cu_tokens, const int64_t* start_pos,
                              const void* kv, const void* score, const float* bias,
                              const float* gamma, const void* ikv, const void* iscore,
                              const float* ibias, const v4a_cache* attn, const v4a_cache* idx,
                              const v4a_cache* swa, const v4a_cache* state, int32_t n_q,
                              const void* q, const float* q_gamma, void* q_out,
                              int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_index_topk — indexer scores and top-k selection of c4a entries (steps a6, a7).
 *
 * [blog] DeepSeek Sparse Attention (DSA) and [notes] 压缩参数细节 (C4A top-k 512).
 * For query i of sequence q_seq[i] at position p = q_pos[i], over the visible entries
 * j (every position S*j+win_off+o they cover is < p; [notes] 因果性条件):
 *   score_j = sum_h w[i,h] * max(0, q_idx[i,h,:] . k_j)
 * with k_j the dequantised indexer key. If at most k entries are visible, all are kept;
 * otherwise the k largest scores, ties to the smaller j. topk_out[i, :] lists the kept j
 * in ascending order, padded with -1.
 *
 * q_idx:    device [n_q, H_I, d_I] (fp32 or bf16)
 * w:        device fp32 [n_q, H_I]
 * q_seq:    device int32 [n_q];  q_pos: device int64 [n_q], every q_pos <= max_pos
 * topk_out: device int32 [n_q, k]
 * workspace: device, >= v4a_index_topk_workspace_size(...) bytes, 256-byte aligned.
 */
size_t v4a_index_topk_workspace_size(const v4a_layer_cfg* cfg, int32_t n_q, int64_t max_pos);
int v4a_index_topk(const v4a_layer_cfg* cfg, int32_t n_q, const int32_t* q_seq,
                   const int64_t* q_pos, int64_t max_pos, const void* q_idx, const float* w,
                   const v4a_cache* idx, int32_t k, int32_t* topk_out, void* workspace,
                   size_t workspace_bytes, int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_index_scores — the indexer scores alone (step a6), as v4a_index_topk computes them
 * before its selection ([blog] DeepSeek Sparse Attention: score_j = sum_h w_h ReLU(q_h . k_j)).
 * Same arguments and checks as v4a_index_topk without k and the output list. Row i of
 * `scores` holds score_j of query i in column j for every visible j (j < visible(q_pos[i]));
 * the other columns of the row are not written.
 *
 * scores:       device fp32 [n_q, v4a_index_scores_row_stride(cfg, max_pos)], 16-byte
 *               aligned, caller-owned; scores_bytes its size (V4A_ERR_ARG if too small)
 * row stride:   visible(max_pos) rounded up to a multiple of 4 floats (0 for a bad cfg)
 */
int64_t v4a_index_scores_row_stride(const v4a_layer_cfg* cfg, int64_t max_pos);
int v4a_index_scores(const v4a_layer_cfg* cfg, int32_t n_q, const int32_t* q_seq,
                     const int64_t* q_pos, int64_t max_pos, const void* q_idx, const float* w,
                     const v4a_cache* idx, float* scores, size_t scores_bytes, int32_t* dev_err,
                     v4a_stream_t stream);

/*
 * v4a_index_topk_noalloc — v4a_index_topk without a workspace argument, for callers that
 * cannot allocate device memory and have none to lend: for example a library embedded in
 * a framework or serving runtime that owns all device memory and gives its kernels no
 * scratch, or a code path where an allocation would synchronise the device or exceed a
 * memory budget fixed in advance. The pages have no counterpart to this call; it exists
 * for such callers only.
 *
 * Same arguments, meaning and results as v4a_index_topk, minus workspace and
 * workspace_bytes. The score rows live in a fixed 8 MiB array inside the library's device
 * image (held by every GPU that loads the library until the process exits), so
 * n_q * visible(max_pos), with visible(max_pos) rounded up to a multiple of 4 (score rows
 * start on 16-byte boundaries), must not exceed v4a_index_topk_noalloc_capacity() floats
 * (2,097,152; e.g. 64 queries at positions up to 131,072); larger requests return
 * V4A_ERR_TOO_LARGE without enqueuing anything. The call itself allocates nothing.
 * The first call on each device looks up the array's device address while that device
 * is current and keeps it for the life of the process; make that first call before any
 * stream capture. A device reset (cudaDeviceReset) unloads the library's device image and
 * makes the kept address invalid: do not call this entry point on a device after resetting
 * it. The host checks and their return codes are those of v4a_index_topk. All calls share the array
 * and it keeps the previous call's contents (each call writes every score it reads, so no
 * clearing is needed); calls that overlap on the GPU, e.g. on two unordered streams, race
 * on it and must be serialised by the caller.
 */
size_t v4a_index_topk_noalloc_capacity(void);
int v4a_index_topk_noalloc(const v4a_layer_cfg* cfg, int32_t n_q, const int32_t* q_seq,
                           const int64_t* q_pos, int64_t max_pos, const void* q_idx,
                           const float* w, const v4a_cache* idx, int32_t k, int32_t* topk_out,
                           int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_attn_decode / v4a_attn_prefill — shared-K=V attention with inverse RoPE (a8, a9).
 *
 * [notes] Inverse RoPE 的数学原理: out = (sum softmax(q K^T) V) R^-1(theta_p), K = V;
 * [blog] 短滑動窗口 (window of 128 uncompressed tokens).
 * For query i at p = q_pos[i] of sequence b = q_seq[i]:
 *   keys  = { attn row j : j in topk[i, :], j >= 0 }   (topk != NULL, c4a)
 *         | { attn row j : j visible at p }             (topk == NULL, dense, c128a)
 *         + { swa row t : max(0, p-swa+1) <= t <= p }
 *   out_h = R^-1(p) * sum_x softmax_x(scale * RoPE(q_h, p) . key_x) * key_x
 * Both calls compute the same function; decode splits each query's keys over several
 * CTAs (few queries, one per sequence), prefill gives each query one CTA (many queries).
 *
 * q:    device [n_q, H, D] (fp32 or bf16);  out: device [n_q, H, D] (fp32 or bf16)
 * topk: device int32 [n_q, k] or NULL
 * attn: entry cache;  swa: token cache
 * workspace: device, >= v4a_attn_workspace_size(...) bytes, 256-byte aligned.
 */
size_t v4a_attn_workspace_size(const v4a_layer_cfg* cfg, int32_t n_q, int64_t max_pos,
                               int32_t k, int32_t prefill);
int v4a_attn_decode(const v4a_layer_cfg* cfg, int32_t n_q, const int32_t* q_seq,
                    const int64_t* q_pos, int64_t max_pos, const void* q, const int32_t* topk,
                    int32_t k, const v4a_cache* attn, const v4a_cache* swa, void* out,
                    void* workspace, size_t workspace_bytes, int32_t* dev_err,
                    v4a_stream_t stream);
/* v4a_attn_plan — how v4a_attn_decode (prefill = 0) or v4a_attn_prefill (prefill = 1) of
 * this shape runs on the current device: *n_split = key ranges per query (1 = no split),
 * *n_kernels = kernels the call launches (0 for n_q = 0; 1, or 2 when a split is combined
 * by the merge kernel). Host only, enqueues nothing. Returns V4A_ERR_ARG for NULL outputs
 * or negative sizes. */
int v4a_attn_plan(const v4a_layer_cfg* cfg, int32_t n_q, int64_t max_pos, int32_t k,
                  int32_t prefill, int32_t* n_split, int32_t* n_kernels);

/* v4a_attn_decode_q8 — v4a_attn_decode whose epilogue also quantises the output for an fp8
 * output projection ([notes] 优化一, 融合 2：Inverse RoPE + FP8 Quant: the attention output goes
 * through the inverse RoPE and straight into an fp8 batched matmul; [blog] GPU 計算飽和度).
 *   out_codes  [n_q, H, D] e4m3 bytes, 16-byte aligned (caller-owned)
 *   out_scale  [n_q, H] fp32 (caller-owned)
 * Per (query, head) row y of R^-1(p) o_h: scale = max|y| / 448 (1 for a zero row) and
 * code = e4m3 round-to-nearest-even, saturating, of y / scale: the rule of the fp8 caches.
 * bf16 layers (V4A_BF16_FP8) only, else V4A_ERR_UNSUPPORTED. The keys of a query are always
 * split into at least two ranges (the quantisation runs where the ranges are merged), so the
 * workspace is v4a_attn_q8_workspace_size(cfg, n_q, max_pos, k), 256-byte aligned. Other
 * arguments, errors and the device error word as for v4a_attn_decode. */
size_t v4a_attn_q8_workspace_size(const v4a_layer_cfg* cfg, int32_t n_q, int64_t max_pos, int32_t k);
int v4a_attn_decode_q8(const v4a_layer_cfg* cfg, int32_t n_q, const int32_t* q_seq,
                       const int64_t* q_pos, int64_t max_pos, const void* q, const int32_t* topk,
                       int32_t k, const v4a_cache* attn, const v4a_cache* swa, uint8_t* out_codes,
                       float* out_scale, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                       v4a_stream_t stream);
int v4a_attn_prefill(const v4a_layer_cfg* cfg, int32_t n_q, const int32_t* q_seq,
                     const int64_t* q_pos, int64_t max_pos, const void* q,
                     const int32_t* topk, int32_t k, const v4a_cache* attn,
                     const v4a_cache* swa, void* out, void* workspace, size_t workspace_bytes,
                     int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_slot_mapping — pool rows of logical rows ([notes] 解决方案一: slot mapping in the
 * unit of the 256-position block). slots[i] = page * R + row[i] % R with
 * page = block_table[seq[i], row[i] / R], or -1 if the block has no page or lies beyond
 * max_blocks (a page >= n_pages also gives -1 and sets V4A_DEV_BAD_PAGE).
 * seq: device int32 [n]; row: device int64 [n]; slots: device int32 [n].
 */
int v4a_slot_mapping(const v4a_cache* cache, int32_t n, const int32_t* seq,
                     const int64_t* row, int32_t* slots, int32_t* dev_err,
                     v4a_stream_t stream);

/*
 * Latent attention: the layer whose cache holds one shared vector a token, a latent of
 * latent_dim values and a rotary key of rope.dim values, from which every head's key and
 * value are projections ([notes] 压缩参数细节 and 8.7x 节省的算术推导: the V3.2 stack that the
 * compressed layer is compared with, 576 bf16 values a token). v4a_latent_insert writes the
 * cache, v4a_latent_attn reads it in the absorbed form (the key projection applied to the
 * query, the value projection to the output: one shared key row for all heads),
 * v4a_latent_gather copies cached rows out for the projections of the expanded form, and
 * v4a_latent_attn_expanded attends with projected keys and values. v4a_rope rotates the
 * query's rotary part (and anything else that needs it).
 *
 * These calls describe a batch as v4a_compress_insert does: sequence b owns rows
 * cu[b] .. cu[b+1]-1 of the packed inputs, at positions start_pos[b] + (row - cu[b]).
 * cu is non-decreasing; rows at or behind cu[n_seq] belong to no sequence: inputs there are
 * not used and outputs there are left as they were. At most V4A_MAX_SEQ sequences a call.
 * Every call reads its inputs only after the kernels enqueued before it on the stream have
 * completed. A call may enqueue several kernels that meet in its workspace: calls share a
 * workspace only if they are on one stream and each is made after the one before it has
 * returned. Calls on different streams, and calls that two threads make at once (on one
 * stream too), need workspaces of their own.
 * Numerics of both attention forms: logits, softmax statistics, sums and accumulators in fp32,
 * the result rounded once. On the tensor cores (the bf16 shapes named at the calls) each softmax
 * weight is also rounded once, to bf16, before it multiplies its value, while the sum of weights
 * takes it unrounded; every other shape keeps its weights in fp32. Sums of w v are formed with
 * weights w of at most 1 and divided at the end by the sum of w: a result is lost to overflow only
 * where such a sum in 32 bits is (|v| above 2^128 / keys), and values below 2^-110 may be lost
 * beside 0.
 * A call counts its steps, (rows, keys) tiles, in 31 bits: it may return V4A_ERR_UNSUPPORTED where
 * the sizes that it is given, max_pos or n_k among them, allow 2^30 of them or more (tiles of 64 x
 * 128 (token, head) rows x keys absorbed, of 512 queries of a head x 128 keys expanded; 16 x 32 for
 * absorbed shapes on CUDA cores), or 2^30 (token, head) rows. Size max_pos by the batch.
 */
#define V4A_MAX_SEQ 1024
#define V4A_MAX_POS ((int64_t)1 << 36)  /* positions are below this */

/* pairs of a rotation: (2i, 2i+1) or (i, i + dim/2) */
#define V4A_ROPE_INTERLEAVED 0
#define V4A_ROPE_HALF 1

/* how the turning rates theta_i = base^(-2i/dim) are scaled for long contexts. With
 * turns_i = orig_max_pos * theta_i / (2 pi), every rate is theta_i (t_i + (1 - t_i) / factor):
 *   NONE      t_i = 1
 *   LINEAR    t_i = 0 (position interpolation)
 *   BY_PARTS  t_i = clamp((turns_i - low) / (high - low), 0, 1): a ramp in the turns
 *   YARN      t_i = 1 - clamp((i - a) / (b - a), 0, 1): a ramp in the pair index, where
 *             pair(t) = dim ln(orig_max_pos / (2 pi t)) / (2 ln base) is the index of the
 *             pair that makes t turns, a = max(floor(pair(high)), 0),
 *             b = min(ceil(pair(low)), dim - 1), and b - a is at least 1e-3
 * (the "by parts" interpolation of Peng et al., "YaRN: Efficient Context Window Extension of
 * Large Language Models", 2023, with both ramps in use for it). */
#define V4A_ROPE_SCALE_NONE 0
#define V4A_ROPE_SCALE_LINEAR 1
#define V4A_ROPE_SCALE_BY_PARTS 2
#define V4A_ROPE_SCALE_YARN 3

typedef struct v4a_rope_cfg {
  int32_t dim;           /* rotated dims: even, 2 .. 256 */
  int32_t layout;        /* V4A_ROPE_INTERLEAVED or V4A_ROPE_HALF */
  int32_t scaling;       /* V4A_ROPE_SCALE_* */
  int32_t reserved;      /* must be 0 */
  float base;            /* > 0; > 1 for YARN */
  float factor;          /* > 0; unused for NONE */
  float orig_max_pos;    /* BY_PARTS, YARN: > 0 */
  float low, high;       /* BY_PARTS, YARN: turns, 0 < low < high */
  float amplitude;       /* > 0, on cosine and sine alike (1 = a rotation) */
} v4a_rope_cfg;

/* Cache formats of a latent layer (v4a_latent_cfg.cache_format).
 * PLAIN: rows of latent_dim + rope.dim elements of the layer's type, no scales.
 * FP4:   the latent part in 4 bits (latent_dim a multiple of 32), whatever the layer's type. A pool
 *   row is V4A_LATENT_FP4_ROW_BYTES(latent_dim, rope.dim) bytes: latent_dim / 2 bytes of e2m1 codes
 *   (element 2i in the low nibble of byte i, codes as for V4A_IDX_FP4), rope.dim f16 numbers h,
 *   latent_dim / 16 e4m3 block scales B, padding up to a multiple of 16; v4a_cache.scale holds one
 *   fp32 scale s a row, and v4a_cache.row_width is latent_dim + rope.dim. The row stands for
 *     s * (B[i / 16] * code_i)  and  s * h_j.
 *   v4a_latent_insert chooses them in fp32, r = 1 / sqrt(mean(c^2) + rms_eps) (1 without gamma),
 *   z = gamma * c, k = rope(k_pe):
 *     u = max|z| * (1 / 2688), s = r * u; where s is below least = max(max|k| / 32768, 2^-100):
 *     s = least, u = s / r. Then t = z * (1 / u), B = e4m3(max|t| of the block * (1 / 6)),
 *     code = e2m1(t * (1 / B)) (0 where B = 0), h = f16(k * (1 / s)), all round to nearest even and
 *     saturating. (2688 = 6 * 448: the row's largest element uses both formats to their ends. The
 *     rotary part stays in 16 bits: it carries the positions and is a ninth of the row. The row
 *     scale takes the norm's r, so which code a value gets does not depend on how the mean square
 *     is summed.) A row with an element that is not finite is not finite. */
#define V4A_LATENT_PLAIN 0
#define V4A_LATENT_FP4 1
#define V4A_LATENT_FP4_ROW_BYTES(latent_dim, rope_dim) \
  (((latent_dim) / 2 + 2 * (rope_dim) + (latent_dim) / 16 + 15) / 16 * 16)

typedef struct v4a_latent_cfg {
  int32_t dtype;         /* V4A_BF16 or V4A_FP32: inputs, cache and outputs */
  int32_t n_heads;       /* H */
  int32_t latent_dim;    /* C: a multiple of 8, 8 .. 1024 */
  int32_t nope_dim;      /* dims of an expanded key before its rotary part: multiple of 8, .. 256 */
  int32_t v_dim;         /* dims of an expanded value: multiple of 8, 8 .. 256 */
  __extension__ union {
    int32_t cache_format; /* V4A_LATENT_PLAIN (0) or V4A_LATENT_FP4 */
    int32_t reserved;     /* the field's name before it had a meaning */
  };
  float rms_eps;         /* of v4a_latent_insert's norm */
  float softmax_scale;   /* > 0, of both attention forms */
  v4a_rope_cfg rope;     /* rope.dim: a multiple of 8, 8 .. 128 */
} v4a_latent_cfg;

/*
 * v4a_rope — rotate rows of n_heads x rope->dim values by their token's position.
 *   y_pair = amplitude * (x0 c - x1 s, x0 s + x1 c), (c, s) = (cos, sin)(pos[t] * rate_i)
 * inverse != 0 turns the other way (s -> -s): with amplitude 1 the inverse, and for any
 * amplitude the gradient of the forward call with respect to x.
 * The rotated part of a wider head is given by its pointer and strides.
 *
 * dtype: V4A_FP32 or V4A_BF16 (computed in fp32, the angle reduced exactly, rounded once).
 *        Cosine and sine are good to a few 2^-24 for positions below 2^28; beyond, the rates,
 *        64-bit numbers, add up to pos * 2^-49
 * pos:   device int64 [n_tokens], each in [0, V4A_MAX_POS); a token outside it is left
 *        unwritten and sets V4A_DEV_BAD_POS
 * x, y:  device, element (t, h, d) at t * token_stride + h * head_stride + d (strides in
 *        elements, >= 0; y's rows must not overlap one another); y == x with equal strides
 *        rotates in place, any other element of y must not be an element of x
 * Rows on 16-byte boundaries take 16-byte accesses, others single elements.
 */
int v4a_rope(const v4a_rope_cfg* rope, int32_t dtype, int32_t n_tokens, int32_t n_heads,
             const int64_t* pos, const void* x, int64_t x_token_stride, int64_t x_head_stride,
             void* y, int64_t y_token_stride, int64_t y_head_stride, int32_t inverse,
             int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_latent_insert — write the cache rows of new tokens:
 *   row = [ gamma * c / sqrt(mean(c^2) + rms_eps) | rope(k_pe, pos) ],
 * computed in fp32 and rounded once; gamma == NULL stores c as it is.
 *
 * c:     device [n_tokens, C] with c_stride elements between tokens; k_pe: device
 *        [n_tokens, rope.dim], k_stride apart (two parts of one projection's output, say).
 *        Pointers on 16-byte boundaries, strides multiples of 16 bytes.
 * gamma: device fp32 [C], 16-byte aligned, or NULL
 * cache: rows_per_block 256, row_width C + rope.dim, no scales (FP4: rows and scales as stated at
 *        V4A_LATENT_FP4; a row's padding is left as it was)
 * Tokens without a page or with a position outside [0, V4A_MAX_POS) are not written and set
 * V4A_DEV_MISSING_PAGE / V4A_DEV_BAD_PAGE / V4A_DEV_BAD_POS.
 */
int v4a_latent_insert(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                      const int32_t* cu_tokens, const int64_t* start_pos, const void* c,
                      int64_t c_stride, const void* k_pe, int64_t k_stride, const float* gamma,
                      const v4a_cache* cache, int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_latent_gather — copy cached rows out: out row cu_rows[b] + i = the cache's row of
 * position start_pos[b] + i of sequence b (FP4: the values that it stands for, computed in fp32 and
 * rounded once to the layer's type). out: device [n_rows, C + rope.dim], 16-byte
 * aligned. A row without a page (or at a negative position) is zeroed and sets
 * V4A_DEV_MISSING_PAGE / V4A_DEV_BAD_PAGE.
 */
int v4a_latent_gather(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_rows,
                      const int32_t* cu_rows, const int64_t* start_pos, const v4a_cache* cache,
                      void* out, int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_latent_attn — absorbed latent attention of each sequence's newest tokens (one or many)
 * over its cached rows, their own included (insert them first):
 *   out[t, h] = sum_x softmax_x(softmax_scale * q[t, h] . row_x) row_x[0:C],  x <= pos(t).
 *
 * q:     device [n_tokens, H, C + rope.dim], the rotary part already rotated, 16-byte aligned
 * out:   device [n_tokens, H, C], 16-byte aligned
 * max_pos: no position of the call is above it; a token beyond it sees the keys up to it and
 *        sets V4A_DEV_BAD_POS
 * workspace: device, >= v4a_latent_attn_workspace_size(...) bytes, 256-byte aligned (may be
 *        NULL where that is 0)
 * Keys in a block without a page are left out (and set the error word); a token that sees no
 * key gives zeros. Rows of the cache behind a sequence's last token are not used, whatever
 * they hold. A key that is not finite makes the outputs of the tokens that see it not finite, and
 * may do so to other tokens of its sequence in the same call.
 * bf16 with C = 512 and rope.dim = 64 runs on the tensor cores; other shapes on CUDA cores, about
 * 16 times slower where the products decide (14-17 TFLOP/s for C of 256 and 512, 6 for 128).
 * FP4 caches: rows are the values that they stand for (scales 0 < s <= 2^126; a row with s = 0 is a
 * row of zeros). On the tensor cores the products take B * code exactly and q but for elements below 2^-32 of
 * the largest |q| of up to 64 neighbouring (token, head) rows, and each weight times its row's scale is
 * rounded once, to f16 (11 bits down to 2^-20 of the largest such product of a head so far, fewer below;
 * rows whose scales are 2^126 apart are not told from nothing). Against a plain cache: a third of the
 * bytes; 192 against 196 us at 32 x 32,768 tokens and 64 heads.
 */
size_t v4a_latent_attn_workspace_size(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                                      int64_t max_pos);
int v4a_latent_attn(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                    const int32_t* cu_tokens, const int64_t* start_pos, int64_t max_pos,
                    const void* q, const v4a_cache* cache, void* out, void* workspace,
                    size_t workspace_bytes, int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_latent_attn_window — v4a_latent_attn in which a token at position p sees, of the keys x <= p,
 * those of a sliding window and the sequence's first ones:
 *   x > p - window  or  x < sinks.
 * Blocks that no token of the call sees into are not looked up: their pages may have been given
 * back. window >= 1, sinks >= 0; window > max_pos is v4a_latent_attn. The work of a token is
 * window + sinks keys, whatever its position. Other arguments, numerics and errors as there.
 */
size_t v4a_latent_attn_window_workspace_size(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                                             int64_t max_pos, int64_t window, int64_t sinks);
int v4a_latent_attn_window(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                           const int32_t* cu_tokens, const int64_t* start_pos, int64_t max_pos,
                           int64_t window, int64_t sinks, const void* q, const v4a_cache* cache,
                           void* out, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                           v4a_stream_t stream);

/*
 * v4a_latent_attn_expanded — latent attention with projected keys and values, for prompts:
 * sequence b has query rows cu_q[b] .. cu_q[b+1]-1 and key rows cu_k[b] .. cu_k[b+1]-1,
 *   s = softmax_scale * (q[i, h, 0:nope] . k[x, h] + q[i, h, nope:] . k_pe[x])
 *   out[i, h] = sum_x softmax_x(s) v[x, h].
 * causal != 0: the sequence's last query sees its last key, each query before it one key
 * fewer; causal == 0: every query sees every key. A query that sees no key gives zeros.
 *
 * q:    device [n_q, H, nope + rope.dim] (rotary part last, rotated); out: device [n_q, H, v_dim]
 * k, v: device, element (x, h, d) at x * token_stride + h * head_stride + d (strides in
 *       elements, so k and v may be parts of one projection's output); k_pe: device
 *       [n_k, rope.dim], k_pe_stride elements between tokens, shared by the heads
 * workspace: device, >= v4a_latent_attn_expanded_workspace_size(...) bytes, 256-byte aligned
 *       (may be NULL where that is 0)
 * All pointers on 16-byte boundaries, strides positive multiples of 16 bytes.
 * Key and value rows at or behind cu_k[n_seq], and other sequences' rows, are not used,
 * whatever they hold. A value that is not finite may reach queries of its sequence that do
 * not see it. dev_err: V4A_DEV_TIMEOUT only (nothing here is looked up).
 * bf16 with nope = 128, rope.dim = 64 and v_dim = 128 runs on the tensor cores; other shapes
 * on CUDA cores, 50 times slower and more (5-9 TFLOP/s; a 2,048-token prompt of 16 heads 2.3-2.9 ms
 * against 44 us).
 */
size_t v4a_latent_attn_expanded_workspace_size(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_q,
                                               int32_t n_k);
int v4a_latent_attn_expanded(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_q,
                             const int32_t* cu_q, int32_t n_k, const int32_t* cu_k, const void* q,
                             const void* k, int64_t k_token_stride, int64_t k_head_stride,
                             const void* k_pe, int64_t k_pe_stride, const void* v,
                             int64_t v_token_stride, int64_t v_head_stride, int32_t causal,
                             void* out, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                             v4a_stream_t stream);

/*
 * Pages. Pools whose sequences grow together (the layers of a model, say) share one block table and
 * one count of references per page: refs[page] is the number of the table's entries that name the
 * page, 0 where it is free. The calls below keep both, and move rows, on the device and in stream
 * order; what they choose depends on the table and the counts alone (pages are taken lowest number
 * first), so a run repeats exactly. Nothing is synchronised, and no list of free pages is kept.
 *
 * At most V4A_MAX_SEQ rows of a table, V4A_MAX_POOLS pools and 2^23 pages a call. A page of -1 is
 * none; a table entry outside [-1, n_pages) sets V4A_DEV_BAD_PAGE and is taken for none (v4a_pages_free
 * clears it). Counts below 0 are taken for 0. workspace: device, >= v4a_pages_workspace_size(table)
 * bytes, 256-byte aligned; calls share one under the rule of the latent calls. The table, counts and
 * lists must not overlap one another, the pools or the workspace.
 */
#define V4A_MAX_POOLS 64

typedef struct v4a_page_table {
  int32_t* block_table;  /* device [n_seq, max_blocks] */
  int32_t* refs;         /* device [n_pages], 16-byte aligned */
  int32_t n_seq;
  int32_t max_blocks;
  int64_t n_pages;
} v4a_page_table;

typedef struct v4a_pool {
  void* data;              /* device [n_pages * rows_per_block][row_bytes], 16-byte aligned */
  float* scale;            /* device fp32 [n_pages * rows_per_block], or NULL */
  int64_t row_bytes;       /* a positive multiple of 16 */
  int32_t rows_per_block;  /* 1 .. 256 */
  int16_t late;            /* 0 .. 255: up to this many tokens behind a block's last position still
                              write into its rows. 0 for token caches; max(0, W - S + win_off) for
                              the entry caches (attn, idx) of a compressed layer: 4 for c4a and 0 for
                              c128a at win_off 0 */
  int16_t reserved;        /* must be 0 */
} v4a_pool;

size_t v4a_pages_workspace_size(const v4a_page_table* table);

/*
 * v4a_pages_free — give back blocks first[b] .. last[b] - 1 of every row b of the table (first,
 * last: device int32 [n_seq], clamped to [0, max_blocks]; empty where last <= first): each entry
 * becomes -1 and its page's count falls by 1. A page whose count was 0 sets V4A_DEV_BAD_PAGE and
 * stays at 0. Contents are left as they are.
 */
int v4a_pages_free(const v4a_page_table* table, const int32_t* first, const int32_t* last,
                   int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_pages_grow — give every block first[b] .. last[b] - 1 of row b that has no page the lowest free
 * page, in the order of rows and blocks, with a count of 1. Where the free pages do not suffice, the
 * blocks last in that order stay without one and V4A_DEV_NO_PAGE is set.
 */
int v4a_pages_grow(const v4a_page_table* table, const int32_t* first, const int32_t* last,
                   void* workspace, size_t workspace_bytes, int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_pages_fork — row dst[i] of the table takes over the first length[i] positions of row src[i],
 * for i < n (device int32 [n], int32 [n], int64 [n]; n <= V4A_MAX_SEQ). Blocks into which no later
 * token writes are shared (the same page, its count one higher; -1 stays -1): those wholly below
 * length[i], but for the last of them where length[i] % 256 is below some pool's `late`. That one and
 * the block that length[i] cuts get the lowest free pages, in the order of i and of blocks. The rows
 * are copied in every pool: of the first all, of the cut block those of its positions below length[i]
 * (a pool with R rows a block: its first ceil(R * cut / 256)); the page's other rows are left as they
 * were. So neither row writes into the other's tokens when both go on. (A compressed layer goes on
 * from the residual rows of the last W - 1 positions below length[i]. v4a_compress_insert has written
 * those where one of its calls ended at length[i], or each of them was among the last W of its call.)
 * dst's row must hold no page, and its blocks behind length[i] stay without. A row may have several
 * children. An entry that is not so is left out whole and sets V4A_DEV_BAD_INDEX: a row outside the
 * table, src == dst, dst named by another entry as src or dst, a dst that holds a page, a length
 * below 0 or beyond the table. Where no page is left for a block it stays without and
 * V4A_DEV_NO_PAGE is set.
 */
int v4a_pages_fork(const v4a_page_table* table, const v4a_pool* pools, int32_t n_pools, int32_t n,
                   const int32_t* src, const int32_t* dst, const int64_t* length, void* workspace,
                   size_t workspace_bytes, int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_pages_copy — copy whole pages src[i] -> dst[i] (device int32 [n], n <= 2^20) in every pool;
 * the table is not read. A page that is written may be neither read nor written by another entry.
 * An entry outside [0, n_pages) is left out and sets V4A_DEV_BAD_PAGE.
 */
int v4a_pages_copy(const v4a_page_table* table, const v4a_pool* pools, int32_t n_pools, int32_t n,
                   const int32_t* src, const int32_t* dst, int32_t* dev_err, v4a_stream_t stream);

/*
 * v4a_pages_compact — move the used pages to the front: with U used pages (counts above 0), the k-th
 * used page at or behind U moves to the k-th free page below U, in every pool, and the table and
 * the counts follow. Pages behind U are then free, so a server may keep (or copy out) the first U.
 * n_used: device int32 [1], receives U. moved: device int32 [n_pages] or NULL, receives every page's
 * new number (its own where it stays, -1 where it was free), for holders of pages besides the table.
 */
int v4a_pages_compact(const v4a_page_table* table, const v4a_pool* pools, int32_t n_pools,
                      int32_t* n_used, int32_t* moved, void* workspace, size_t workspace_bytes,
                      int32_t* dev_err, v4a_stream_t stream);

/* Synchronise `stream`, read the device error word, clear it. *flags_out (may be NULL)
 * receives the bits. Returns V4A_OK, V4A_ERR_DEVICE if any bit was set, or V4A_ERR_CUDA. */
int v4a_get_error(int32_t* dev_err, v4a_stream_t stream, int32_t* flags_out);

/* Library version, raised whenever an entry point or a kernel changes (profiles and the
 * binding compare against it). */
int32_t v4a_version(void);

#ifdef __cplusplus
}
#endif
#endif /* V4A_H */
