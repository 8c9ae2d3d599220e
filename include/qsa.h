/*
 * qsa.h — C ABI of the GB300 (sm_103a) indexer-driven sparse attention library (libqsa.so).
 *
 * The method (Qwen Sparse Attention style), as stated on
 * "3090x3で 314 万コンテキスト; KVキャッシュをホストRAMに置けるアーキテクチャの偉大さ":
 *   section "なぜ": an indexer scores every pooled 4-token block of the history
 *     (indexer_compress_ratio = 4) and keeps a fixed budget of 2048 tokens
 *     (indexer_budget = 2048, i.e. the top 512 blocks); up to 4*512+3 = 2051
 *     tokens of context everything is read;
 *   section "VRAM に残す必要があるもの": the pooled key of a block is 128 x bf16 and
 *     the indexer scans all of them every step;
 *   section "カーネルを書き換えずに済む": the gather kernel addresses
 *     K/V as (tok * n_kv_heads + kv_head) * head_dim + d;
 *   section "ちなみにこの欠点": prefill walks the history in fixed intervals
 *     (outer loop) with all chunk tokens inside (inner loop), merging softmax
 *     partials across intervals.
 * Partial results over disjoint token sets are merged by log-sum-exp
 * ("GLM-5.3 最適化 第2部：16基のH200上でのPCP、DCP、およびHybrid HiSparse", section "DCP").
 *
 * Conventions for every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller. The library
 *    never allocates, never frees, never keeps a pointer after returning and never
 *    synchronises, except qsa_read_device_status, which synchronises the stream it is given.
 *  - The K/V cache (k_cache, v_cache) of the attention calls, and raw_idx_k of
 *    qsa_decode_step, may instead live in pinned host memory mapped into the device's
 *    address space (cudaHostAlloc, or cudaHostRegister with cudaHostRegisterMapped): the
 *    kernels then gather the selected rows over the host link ("3090x3で 314 万コンテキスト",
 *    section "VRAM に残す必要があるもの": only the pooled keys must stay on the GPU). A pointer
 *    the device cannot read at the same address returns QSA_ERR_INVALID_ARGUMENT.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *    stream). Nothing else is launched, so the calls can be captured in a CUDA graph.
 *  - Row-major layouts; bf16 values are passed as raw 16-bit patterns (qsa_bf16).
 *  - Ragged batches are flat token arrays with int32 offsets (tok_off[s] .. tok_off[s+1]).
 *  - Host-side validation failures return immediately with nothing enqueued.
 *    A failed launch returns QSA_ERR_CUDA. Errors found on the device (an index out
 *    of range, a bounded wait that gave up) never trap: the kernel skips the access,
 *    records the first error in the workspace's status word and returns; read it
 *    with qsa_read_device_status. The status word is sticky until qsa_workspace_init.
 *  - Supported geometry: head_dim 256, idx_dim 128, indexer_compress_ratio 4,
 *    indexer_budget 2048, n_q_heads % n_kv_heads == 0, n_q_heads / n_kv_heads <= 16.
 *    Anything else returns QSA_ERR_UNSUPPORTED.
 *  - Per-thread detail of the last host-side error: qsa_last_error().
 */
#ifndef QSA_H
#define QSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define QSA_API __attribute__((visibility("default")))
#else
#define QSA_API
#endif

typedef enum {
    QSA_OK = 0,
    QSA_ERR_INVALID_ARGUMENT = 1,   /* null/misaligned pointer, negative size, bad stride */
    QSA_ERR_UNSUPPORTED = 2,        /* geometry outside the supported set */
    QSA_ERR_WORKSPACE_TOO_SMALL = 3,
    QSA_ERR_CUDA = 4,               /* a CUDA launch or runtime call failed */
    QSA_ERR_DEVICE_TIMEOUT = 5,     /* a bounded device-side wait gave up */
    QSA_ERR_DEVICE_BOUNDS = 6       /* a device-side index/offset check failed */
} qsa_status;

typedef enum {
    QSA_OP_POOL_KEYS = 0,
    QSA_OP_INDEX_SCORE = 1,
    QSA_OP_TOPK_BLOCKS = 2,
    QSA_OP_SPARSE_DECODE = 3,
    QSA_OP_SPARSE_PREFILL_CHUNK = 4,
    QSA_OP_DECODE_STEP = 5,
    QSA_OP_PREFILL_SELECT = 6
} qsa_op;

/* Geometry. Field names follow the model config the page quotes
 * (indexer_budget, indexer_compress_ratio, section "なぜ"). */
typedef struct {
    int32_t n_q_heads;              /* query heads (8 or 16 in the workloads) */
    int32_t n_kv_heads;             /* KV heads (2); query head h reads KV head h / (n_q_heads/n_kv_heads) */
    int32_t head_dim;               /* 256 */
    int32_t idx_dim;                /* 128: width of raw/pooled indexer keys and indexer queries */
    int32_t indexer_compress_ratio; /* 4 tokens per pooled block */
    int32_t indexer_budget;         /* 2048 tokens = 512 blocks kept per query */
    float softmax_scale;            /* <= 0 selects 1/sqrt(head_dim) */
} qsa_config;

typedef uint16_t qsa_bf16;          /* raw bf16 bits */
typedef void *qsa_stream;           /* cudaStream_t */

/* Workspace bytes an op needs for the given sizes (0 on unsupported geometry).
 * n_rows: queries (index_score/topk), sequences (decode), chunk queries (prefill).
 * max_blocks: the largest number of visible blocks of any row (topk: the scores' ld).
 * Every workspace starts with a 256-byte status block; it must be zeroed once with
 * qsa_workspace_init before first use (and after a device error). One workspace
 * may be reused by consecutive calls on the same stream; calls that run
 * concurrently need separate workspaces. */
QSA_API size_t qsa_workspace_size(int32_t op, const qsa_config *cfg, int32_t n_rows, int64_t max_blocks);

/* Zero `ws_bytes` bytes of the workspace on `stream` (clears the status word). */
QSA_API qsa_status qsa_workspace_init(void *ws, size_t ws_bytes, qsa_stream stream);

/* Synchronise `stream`, then copy the workspace's status word to *out and the
 * kernel-specific detail (e.g. the offending row) to *detail (may be NULL). */
QSA_API qsa_status qsa_read_device_status(const void *ws, qsa_stream stream, qsa_status *out, int32_t *detail);

/* Input staging helper (not a step of the method): copies n_rows rows of row_bytes bytes
 * from src (rows src_pitch bytes apart) to dst (rows dst_pitch bytes apart), host or device
 * memory on either side, asynchronously on `stream` (one strided copy, no kernel). Used
 * to append a new token's rows to per-layer caches stacked with a fixed layer stride.
 * Host memory should be pinned for the copy to be asynchronous. Errors: NULL pointers,
 * row_bytes larger than either pitch -> QSA_ERR_INVALID_ARGUMENT; n_rows == 0 copies
 * nothing. */
QSA_API qsa_status qsa_copy_rows(void *dst, size_t dst_pitch, const void *src, size_t src_pitch, size_t row_bytes,
                                 size_t n_rows, qsa_stream stream);

/* a1 — Pool indexer keys ("VRAM に残す必要があるもの": one pooled 128 x bf16 key per
 * 4-token block). For each sequence s < B and each block b in [blk_begin[s], blk_end[s]):
 *   pooled[blk_off[s] + b][d] = bf16_rne( (raw[t0][d] + raw[t0+1][d] + raw[t0+2][d] + raw[t0+3][d]) / 4 ),
 *   t0 = tok_off[s] + 4 b,
 * with the sum exact (accumulated in fp64) and a single round-to-nearest-even.
 *   raw_idx_k  [n_tokens_total, idx_dim] bf16, 16-byte aligned
 *   tok_off    [B+1] int32 (device), blk_off [B+1] int32, blk_begin [B], blk_end [B] int32
 *   pooled     [n_pooled_total, idx_dim] bf16 (written), 16-byte aligned
 *   max_blocks_per_seq: host upper bound of blk_end[s] - blk_begin[s] (sizes the grid)
 * Device checks: 0 <= blk_begin <= blk_end, blk_end - blk_begin <= max_blocks_per_seq,
 * 4*blk_end <= tokens of s, blk_off[s] + blk_end <= n_pooled_total; a failing sequence
 * is skipped and QSA_ERR_DEVICE_BOUNDS recorded. Only complete blocks are pooled. */
QSA_API qsa_status qsa_pool_keys(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, int64_t n_tokens_total,
                                 const int32_t *tok_off, const int32_t *blk_off, const int32_t *blk_begin,
                                 const int32_t *blk_end, int32_t B, int64_t max_blocks_per_seq,
                                 qsa_bf16 *pooled, int64_t n_pooled_total,
                                 void *ws, size_t ws_bytes, qsa_stream stream);

/* a2 — Indexer scores ("なぜ", "VRAM に残す必要があるもの": every pooled block is scored
 * every step). For query r < Nq with p = q_pos[r] history tokens and nb = p / 4:
 *   scores[r * ld + b] = sum_d q_idx[r][d] * pooled[blk_off[q_seq[r]] + b][d],  b < nb,
 * fp32 accumulation of exact bf16 products. Entries b >= nb are not written.
 *   q_idx [Nq, idx_dim] bf16; q_seq [Nq], q_pos [Nq] int32; pooled as above;
 *   blk_off [B+1] int32 (per-sequence pooled offsets); scores [Nq, ld] fp32.
 * q_seq may be NULL: every query then belongs to sequence 0 (a prefill chunk). With
 * Nq >= 128 and n_pooled_total >= 256 that case runs as one tensor-core GEMM ("GLM-5.3
 * 最適化 第2部": prefill scoring is quadratic) in tiles of 128 queries x 256 blocks, the
 * products summed in fp32 in the tensor core's order; otherwise one query at a time.
 * Device checks: nb <= ld, blk_off[s] + nb <= n_pooled_total. */
QSA_API qsa_status qsa_index_score(const qsa_config *cfg, const qsa_bf16 *q_idx, const int32_t *q_seq,
                                   const int32_t *q_pos, int32_t Nq, const qsa_bf16 *pooled,
                                   int64_t n_pooled_total, const int32_t *blk_off, float *scores, int64_t ld,
                                   void *ws, size_t ws_bytes, qsa_stream stream);

/* a1 with FP8 keys — pooled indexer keys stored as 128 FP8 (E4M3) codes plus one fp32 scale
 * per block ("GLM-5.3 最適化 第2部：16基のH200上でのPCP、DCP、およびHybrid HiSparse", footnote on
 * the indexer cache: 128 FP8 values and a 4-byte scale per key), so the scan of every pooled
 * block reads 132 bytes instead of 256. For each block the call first forms the bf16 pooled
 * key exactly as qsa_pool_keys does (key[d]), then
 *   scales[i] = amax / 448 (fp32 IEEE division, amax = max_d |key[d]|),
 *   codes[i][d] = E4M3(key[d] / scales[i]) (fp32 IEEE division; nearest, ties to even;
 *                 saturating at +-448),
 * with i = blk_off[s] + b; a block whose key is all zero (scale 0) gets zero codes.
 *   codes [n_pooled_total, idx_dim] uint8 (written), 16-byte aligned;
 *   scales [n_pooled_total] fp32 (written), 4-byte aligned.
 * Other arguments, the workspace (QSA_OP_POOL_KEYS) and the device checks as qsa_pool_keys. */
QSA_API qsa_status qsa_pool_keys_fp8(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, int64_t n_tokens_total,
                                     const int32_t *tok_off, const int32_t *blk_off, const int32_t *blk_begin,
                                     const int32_t *blk_end, int32_t B, int64_t max_blocks_per_seq, uint8_t *codes,
                                     float *scales, int64_t n_pooled_total, void *ws, size_t ws_bytes,
                                     qsa_stream stream);

/* a2 with FP8 keys — indexer scores against the keys qsa_pool_keys_fp8 writes. For query r
 * with nb = q_pos[r] / 4 and i = blk_off[q_seq[r]] + b:
 *   scores[r * ld + b] = scales[i] * sum_d q_idx[r][d] * codes[i][d],  b < nb,
 * with exact products and an fp32 sum, then one fp32 multiply by the scale. Entries b >= nb
 * are not written. q_seq may be NULL (every query in sequence 0). An HBM stream (no
 * tensor-core path): the CTAs resident in one wave are shared over the queries, each
 * streaming an equal range of its query's blocks. The first call on a device queries that
 * occupancy and should precede stream capture. Workspace QSA_OP_INDEX_SCORE. Device checks:
 * nb <= ld, blk_off[s] + nb <= n_pooled_total. The scores feed qsa_topk_blocks unchanged. */
QSA_API qsa_status qsa_index_score_fp8(const qsa_config *cfg, const qsa_bf16 *q_idx, const int32_t *q_seq,
                                       const int32_t *q_pos, int32_t Nq, const uint8_t *codes, const float *scales,
                                       int64_t n_pooled_total, const int32_t *blk_off, float *scores, int64_t ld,
                                       void *ws, size_t ws_bytes, qsa_stream stream);

/* a2 + a3 fused for a prefill chunk (one sequence, q_seq NULL): the same blocks and counts
 * as qsa_index_score followed by qsa_topk_blocks, without writing the score matrix
 * ("GLM-5.3 最適化 第2部": prefill scoring is quadratic; "なぜ": top-512 per query). The
 * scoring GEMM runs twice: first it keeps each row's maximum over every 64 consecutive
 * visible blocks, whose 512th largest is a floor that at least 512 scores reach; then its
 * epilogue keeps every visible score at or above the floor (exact fp32 scores, as
 * qsa_index_score computes them) and the top-k takes each row's top 512 from those. A row
 * whose candidates overflow (more than 32 in a tile of 256 blocks, e.g. many equal scores)
 * or fall short is finished on the exact path: the full scores are then written to
 * `scores` [Nq, ld] and that row streamed as by qsa_topk_blocks; otherwise `scores` is
 * not touched. Arguments as for those two calls; workspace
 * qsa_workspace_size(QSA_OP_PREFILL_SELECT, cfg, Nq, ld) (about 300 MB for 4096 queries
 * over 66,560 blocks). Needs Nq >= 128, n_pooled_total >= 256, ld <= 524288, else
 * QSA_ERR_UNSUPPORTED. */
QSA_API qsa_status qsa_prefill_select(const qsa_config *cfg, const qsa_bf16 *q_idx, const int32_t *q_pos, int32_t Nq,
                                      const qsa_bf16 *pooled, int64_t n_pooled_total, const int32_t *blk_off,
                                      float *scores, int64_t ld, int32_t *blocks, int32_t *count, void *ws,
                                      size_t ws_bytes, qsa_stream stream);

/* a3 — Fixed-budget block selection ("なぜ": exactly 2048 tokens = 512 blocks beyond 2051
 * tokens of context; all blocks below). For row r with nb = q_pos[r] / 4, k = budget/ratio:
 * the min(k, nb) blocks with the largest scores, ties to the lower block id
 * ("125B MoE を 3090 3 枚で運用する vLLM 最適化編" section 3.3 uses the same rule), written
 * to blocks[r * k ...] in ASCENDING id order; the rest of the row is set to -1;
 * count[r] = min(k, nb). NaN scores rank below every number; -0 equals +0.
 *   scores [Nq, ld] fp32 (only b < nb read); q_pos [Nq]; blocks [Nq, k] int32; count [Nq] int32. */
QSA_API qsa_status qsa_topk_blocks(const qsa_config *cfg, const float *scores, int64_t ld, const int32_t *q_pos,
                                   int32_t Nq, int32_t *blocks, int32_t *count,
                                   void *ws, size_t ws_bytes, qsa_stream stream);

/* a4 + a5 — Sparse GQA decode over the selected blocks with split partials merged by
 * log-sum-exp ("なぜ": 4 MiB of K/V per layer whatever the context; "カーネルを
 * 書き換えずに済む": K/V addressing; "GLM-5.3 最適化 第2部" section DCP: LSE merge).
 * Sequence s has its query at position p = ctx_len[s]; its tokens live at
 * tok_off[s] .. tok_off[s+1]-1 and the current token's K/V is already at index p.
 * Attended tokens J = {4b .. 4b+3 : b in blocks[s][0 .. count[s])} U {4*(p/4) .. p}.
 * For query head h (KV head h / (Hq/Hkv)):
 *   out[s][h] = sum_{j in J} softmax_j(scale * q[s][h] . K[j]) V[j],   lse[s][h] = ln sum_j e^(scale q.K[j])
 *   q [B, Hq, D] bf16; k_cache, v_cache [n_tokens_total, Hkv, D] bf16 (token-major);
 *   blocks [B, k] int32 (as written by qsa_topk_blocks; any order, no duplicates), count [B];
 *   out [B, Hq, D] bf16; lse [B, Hq] fp32 or NULL.
 * Device checks: p + 1 <= tokens of s, count <= min(k, p/4), 0 <= block < p/4. */
QSA_API qsa_status qsa_sparse_decode(const qsa_config *cfg, const qsa_bf16 *q, const qsa_bf16 *k_cache,
                                     const qsa_bf16 *v_cache, int64_t n_tokens_total, const int32_t *tok_off,
                                     const int32_t *ctx_len, int32_t B, const int32_t *blocks,
                                     const int32_t *count, qsa_bf16 *out, float *lse,
                                     void *ws, size_t ws_bytes, qsa_stream stream);

/* a6 — Prefill chunk ("ちなみにこの欠点": each chunk token selects its own 2048 tokens;
 * the history is walked interval by interval with a softmax merge). Chunk query i
 * (0 <= i < Nc) sits at p_i = p0 + i of one sequence whose K/V (history and chunk)
 * occupy tokens 0 .. p0+Nc-1; it attends exactly what qsa_sparse_decode would for
 * p = p_i with its own blocks[i] / count[i]. interval_tokens (a positive multiple of
 * 128) sets the evaluation order only, not the result.
 *   q [Nc, Hq, D] bf16; k_cache, v_cache [p0+Nc, Hkv, D] bf16;
 *   blocks [Nc, k] int32, 16-byte aligned, each row's first count[i] entries strictly
 *   ascending (as qsa_topk_blocks writes them); count [Nc]; out [Nc, Hq, D] bf16;
 *   lse [Nc, Hq] fp32 or NULL. q, k_cache, v_cache and out are 16-byte aligned.
 * With 8 or 16 query heads per KV head the chunk runs on the tensor cores in tiles of
 * 128 (query, head) rows that share each interval's union of selected blocks; a row out
 * of order there is recorded as QSA_ERR_DEVICE_BOUNDS and its tile's outputs are not
 * written. The workspace (qsa_workspace_size) then holds the tiles' chunk plan, about
 * 197 KB per 16 queries. Other head ratios run one CTA per
 * (query, KV head) on the CUDA cores. Requires (p0 + Nc) / 4 < 524288 on the tensor-core
 * path (else QSA_ERR_UNSUPPORTED). */
QSA_API qsa_status qsa_sparse_prefill_chunk(const qsa_config *cfg, const qsa_bf16 *q, int32_t p0, int32_t Nc,
                                            const qsa_bf16 *k_cache, const qsa_bf16 *v_cache,
                                            const int32_t *blocks, const int32_t *count, int32_t interval_tokens,
                                            qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes,
                                            qsa_stream stream);

/* a6 staged, for K/V in host memory ("3090x3で 314 万コンテキスト", section "ちなみにこの欠点":
 * the prefill copies the history over the link into a device staging arena and computes
 * from there, so each row crosses the link once instead of once per tile that gathers it).
 * Rows [0, p0 + Nc) of k_cache and v_cache (any memory the copy engine reaches, pinned host
 * memory for an asynchronous copy) are copied into `stage` (K rows, then V rows:
 * 2 (p0 + Nc) n_kv_heads head_dim x 2 bytes, device memory, 16-byte aligned), then
 * qsa_sparse_prefill_chunk runs on the staged rows: the results are bit-identical to running
 * it on device-resident K/V. A stage shorter than needed -> QSA_ERR_WORKSPACE_TOO_SMALL;
 * a NULL or misaligned stage -> QSA_ERR_INVALID_ARGUMENT. Other arguments and errors as
 * qsa_sparse_prefill_chunk. The caller keeps the stage (an arena it may reuse for every layer). */
QSA_API qsa_status qsa_sparse_prefill_chunk_staged(const qsa_config *cfg, const qsa_bf16 *q, int32_t p0, int32_t Nc,
                                                   const qsa_bf16 *k_cache, const qsa_bf16 *v_cache,
                                                   const int32_t *blocks, const int32_t *count, int32_t interval_tokens,
                                                   qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, void *stage,
                                                   size_t stage_bytes, qsa_stream stream);

/* a6 over FP8 K/V rows (the row format of qsa_quantize_kv_fp8; "GLM-5.3 最適化 第2部", footnote 1).
 * The prefill multiplies bf16 tiles on the tensor cores, so rows [0, p0 + Nc) of the K and V
 * caches are first dequantised into `stage` as qsa_dequantize_kv_fp8 does (K rows, then V
 * rows: 2 (p0 + Nc) n_kv_heads x 512 bytes of device memory, 16-byte aligned), then
 * qsa_sparse_prefill_chunk runs on the staged rows: the results are bit-identical to running it
 * on the dequantised bf16 caches. Each element is thus code x scale rounded once to bf16 (at
 * most 2^-8 of its magnitude off the exact value) before the attention.
 *   k_codes, v_codes [p0 + Nc][n_kv_heads][256] uint8, 16-byte aligned; k_scales, v_scales
 *   [p0 + Nc][n_kv_heads][2] fp32, 8-byte aligned (device memory or mapped pinned host memory).
 * A stage shorter than needed -> QSA_ERR_WORKSPACE_TOO_SMALL; a NULL or misaligned stage or
 * row pointer -> QSA_ERR_INVALID_ARGUMENT. Other arguments and errors as
 * qsa_sparse_prefill_chunk. The caller keeps the stage (an arena it may reuse for every layer). */
QSA_API qsa_status qsa_sparse_prefill_chunk_fp8kv(const qsa_config *cfg, const qsa_bf16 *q, int32_t p0, int32_t Nc,
                                                  const uint8_t *k_codes, const float *k_scales,
                                                  const uint8_t *v_codes, const float *v_scales,
                                                  const int32_t *blocks, const int32_t *count, int32_t interval_tokens,
                                                  qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, void *stage,
                                                  size_t stage_bytes, qsa_stream stream);

/* a1-a5 fused — one decode layer-step for a batch of B <= 64 sequences in a single
 * cooperative launch ("なぜ", "VRAM に残す必要があるもの", "カーネルを書き換えずに済む";
 * LSE merge from "GLM-5.3 最適化 第2部" section DCP). For sequence s with p = ctx_len[s],
 * nb = p / 4:
 *   1. pooled[blk_off[s] + nb - 1] is (re)computed from raw_idx_k as in qsa_pool_keys (the
 *      newest block the query scores; blocks below it must already be pooled);
 *   2. every block b < nb is scored as in qsa_index_score (fp32 accumulation);
 *   3. the selection of qsa_topk_blocks is written to blocks[s] (ascending, -1 padded) and
 *      count[s];
 *   4. out[s] and lse[s] are computed as in qsa_sparse_decode over that selection.
 * Arguments have the meaning, layout and alignment they have in those calls.
 * max_blocks: host upper bound of nb over the batch (sizes the workspace:
 * qsa_workspace_size(QSA_OP_DECODE_STEP, cfg, B, max_blocks)). Requires n_kv_heads <= 2 and
 * a batch whose blocks fit the kernel's on-chip limit per CTA (else QSA_ERR_UNSUPPORTED;
 * use the separate calls then). Device errors (bounds, a bounded wait that gave up) go to
 * the workspace status word. The launch is cooperative; the first call on a device sizes
 * the grid and should precede stream capture. */
QSA_API qsa_status qsa_decode_step(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, qsa_bf16 *pooled,
                                   int64_t n_pooled_total, const int32_t *blk_off, const qsa_bf16 *q_idx,
                                   const qsa_bf16 *q, const qsa_bf16 *k_cache, const qsa_bf16 *v_cache,
                                   int64_t n_tokens_total, const int32_t *tok_off, const int32_t *ctx_len, int32_t B,
                                   int64_t max_blocks, int32_t *blocks, int32_t *count, qsa_bf16 *out, float *lse,
                                   void *ws, size_t ws_bytes, qsa_stream stream);

/* a1-a5 fused with FP8 keys — qsa_decode_step over the keys qsa_pool_keys_fp8 writes
 * (128 E4M3 codes + an fp32 scale per block; "GLM-5.3 最適化 第2部：16基のH200上でのPCP、DCP、
 * およびHybrid HiSparse", footnote on the indexer cache), so the scan reads 132 bytes per block
 * instead of 256. For sequence s with p = ctx_len[s], nb = p / 4:
 *   1. block blk_off[s] + nb - 1 is (re)pooled from raw_idx_k and quantised as by
 *      qsa_pool_keys_fp8 (codes and scale written);
 *   2. every block b < nb is scored as by qsa_index_score_fp8 (same products, fp32 sum order
 *      and scale multiply, hence the same fp32 scores);
 *   3.-4. selection and attention as in qsa_decode_step.
 *   codes [n_pooled_total, idx_dim] uint8, 16-byte aligned; scales [n_pooled_total] fp32,
 *   16-byte aligned. n_pooled_total must be a multiple of 4 (the scan copies whole
 *   16-byte groups of scales): pad both arrays to it. Else QSA_ERR_INVALID_ARGUMENT.
 * Other arguments, the workspace (QSA_OP_DECODE_STEP), limits and errors as qsa_decode_step. */
QSA_API qsa_status qsa_decode_step_fp8(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, uint8_t *codes,
                                       float *scales, int64_t n_pooled_total, const int32_t *blk_off,
                                       const qsa_bf16 *q_idx, const qsa_bf16 *q, const qsa_bf16 *k_cache,
                                       const qsa_bf16 *v_cache, int64_t n_tokens_total, const int32_t *tok_off,
                                       const int32_t *ctx_len, int32_t B, int64_t max_blocks, int32_t *blocks,
                                       int32_t *count, qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes,
                                       qsa_stream stream);

/* FP8 K/V rows — the KV-row format of "GLM-5.3 最適化 第2部：16基のH200上でのPCP、DCP、および
 * Hybrid HiSparse" (footnote 1: E4M3 codes in groups of 128 dims, one fp32 scale per group)
 * applied to the GQA cache of this library. Each 256-dim row (one token's K, or V, of one KV
 * head) is two groups; for group g of row r:
 *   scales[r][g] = max_d |x[r][128 g + d]| / 448 (an fp32 IEEE division);
 *   codes[r][128 g + d] = E4M3(x[r][128 g + d] / scales[r][g]) (fp32 IEEE division, nearest
 *   even, saturated at +-448); a group of zeros has scale 0 and zero codes.
 *   x [n_rows][256] bf16, 16-byte aligned (a cache [T][Hkv][256] is n_rows = T x Hkv);
 *   codes [n_rows][256] uint8 (written), 16-byte aligned; scales [n_rows][2] fp32 (written),
 *   8-byte aligned. Device memory or mapped pinned host memory.
 * No workspace, no device-side errors (inputs are not indexed). n_rows = 0 is a no-op;
 * n_rows < 0 or above 2^34, NULL or misaligned pointers: QSA_ERR_INVALID_ARGUMENT. Non-finite
 * inputs are outside the contract. Use it to append the new token's rows to an FP8 cache. */
QSA_API qsa_status qsa_quantize_kv_fp8(const qsa_bf16 *x, int64_t n_rows, uint8_t *codes, float *scales,
                                       qsa_stream stream);

/* The inverse of qsa_quantize_kv_fp8 for computing on bf16 tiles: x[r][d] = the value
 * code_d x scales[r][d / 128] rounded once to bf16 (nearest, ties to even; magnitudes that
 * round past the largest bf16 become infinity; an E4M3 NaN code gives a NaN).
 *   codes [n_rows][256] uint8, 16-byte aligned; scales [n_rows][2] fp32, 8-byte aligned;
 *   x [n_rows][256] bf16 (written), 16-byte aligned. Device memory or mapped pinned host memory.
 * No workspace, no device-side errors. n_rows = 0 is a no-op; n_rows < 0 or above 2^34, NULL
 * or misaligned pointers: QSA_ERR_INVALID_ARGUMENT. */
QSA_API qsa_status qsa_dequantize_kv_fp8(const uint8_t *codes, const float *scales, int64_t n_rows, qsa_bf16 *x,
                                         qsa_stream stream);

/* a1-a5 fused over FP8 K/V rows — qsa_decode_step (bf16 indexer keys: `pooled`) or
 * qsa_decode_step_fp8 (FP8 indexer keys: `codes`, `scales`), with the selected tokens' K and
 * V read from FP8 rows as qsa_quantize_kv_fp8 writes them instead of bf16 rows. Give exactly
 * one key format (the other pointer(s) NULL), else QSA_ERR_INVALID_ARGUMENT.
 *   k_codes, v_codes [n_tokens_total][n_kv_heads][256] uint8, 16-byte aligned;
 *   k_scales, v_scales [n_tokens_total][n_kv_heads][2] fp32, 16-byte aligned.
 * Element d of a row has the value code_d x scale[d / 128]. The logit of query head h and
 * token t is scale_softmax x sum over the two groups of (scale_g x the fp32 sum of the
 * group's exact bf16 x E4M3 products); the output is sum_t softmax_t x (code x scale) in
 * fp32, rounded once to bf16. Selection, outputs, workspace (QSA_OP_DECODE_STEP), limits and
 * errors as qsa_decode_step; the rows (and scales) may live in mapped pinned host memory. */
QSA_API qsa_status qsa_decode_step_fp8kv(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, qsa_bf16 *pooled,
                                         uint8_t *codes, float *scales, int64_t n_pooled_total,
                                         const int32_t *blk_off, const qsa_bf16 *q_idx, const qsa_bf16 *q,
                                         const uint8_t *k_codes, const float *k_scales, const uint8_t *v_codes,
                                         const float *v_scales, int64_t n_tokens_total, const int32_t *tok_off,
                                         const int32_t *ctx_len, int32_t B, int64_t max_blocks, int32_t *blocks,
                                         int32_t *count, qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes,
                                         qsa_stream stream);

/* f1: a VRAM row cache in front of K/V that live in host memory ("125B MoE を 3090 3 枚で運用
 * する vLLM 最適化編", section 5: consecutive decode steps select largely the same rows, so rows
 * read over the host link are kept in unused device memory). A direct-mapped cache of n_slots
 * token rows; a slot holds one token's K and V rows of every KV head (n_kv_heads x 2 x 512 B)
 * with a tag (the token's index in the flat K/V arrays), the epoch of its last hit and the
 * epoch's winning claim. Layout inside the caller's buffer: rows, then int64 tags, uint32 hit
 * epochs, uint64 claims; its size is qsa_rowcache_bytes (0 for a bad configuration, more than
 * 2 KV heads, or n_slots outside [1, 2^31]). The caller owns the buffer (device memory,
 * 16-byte aligned) and keeps one per layer. */
QSA_API size_t qsa_rowcache_bytes(const qsa_config *cfg, int64_t n_slots);

/* Empty every slot of a row cache (tags -1, hit epochs and claims 0). Call it once before the
 * first step, and again whenever rows the cache may hold change in host memory other than by
 * appending new tokens (a sequence's cache reused for another request, blocks reassigned). */
QSA_API qsa_status qsa_rowcache_init(const qsa_config *cfg, void *cache, size_t cache_bytes, int64_t n_slots,
                                     qsa_stream stream);

/* a1-a5 fused with the row cache — qsa_decode_step, for K/V (and raw indexer keys) in mapped
 * pinned host memory (or device memory), with every selected row looked up in `cache` first.
 * Sequence s owns slots [s n_slots / B, (s + 1) n_slots / B); token t of it maps to slot
 * lo_s + t mod (its slot count). Per step (`epoch`: at least 1, larger than at every earlier
 * call with this cache):
 *   - a selected token whose slot's tag is the token's flat index is read from the cache and
 *     the slot is marked as hit in this epoch; any other selected token is read from k_cache /
 *     v_cache and claims its slot with an atomic max of (epoch << 32 | flat index);
 *   - after every CTA of the sequence has read its rows, a claim's winner writes the row and
 *     the tag, unless some token hit the slot in this epoch (the rows of each CTA's last two
 *     chunks of at most 32 tokens each are written, any earlier ones stay uncached this step).
 * The query's own (incomplete) block is always read from k_cache / v_cache and never cached:
 * the caller may still be writing it. Hits return exactly the bytes in host memory, so the
 * outputs equal qsa_decode_step's bit for bit. Cache errors: NULL or misaligned cache,
 * n_slots < B or above 2^31, epoch 0 -> QSA_ERR_INVALID_ARGUMENT; cache_bytes short ->
 * QSA_ERR_WORKSPACE_TOO_SMALL. Everything else (bf16 keys and K/V only) as qsa_decode_step. */
QSA_API qsa_status qsa_decode_step_rowcache(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, qsa_bf16 *pooled,
                                            int64_t n_pooled_total, const int32_t *blk_off, const qsa_bf16 *q_idx,
                                            const qsa_bf16 *q, const qsa_bf16 *k_cache, const qsa_bf16 *v_cache,
                                            int64_t n_tokens_total, const int32_t *tok_off, const int32_t *ctx_len,
                                            int32_t B, int64_t max_blocks, int32_t *blocks, int32_t *count,
                                            qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, void *cache,
                                            size_t cache_bytes, int64_t n_slots, uint32_t epoch, qsa_stream stream);

/* a1-a5 fused, with an L2 prefetch hint — qsa_decode_step (and qsa_decode_step_fp8) plus
 * the memory the caller's next call will read, typically the next layer's pooled keys (or
 * FP8 codes). Each CTA, once its own pooled-key stream is done, issues L2 prefetch hints for
 * its slice of [next_read, next_read + next_read_bytes), so the bytes the next layer-step
 * scans arrive in L2 while this step exchanges keys and partials (those phases leave HBM
 * idle). The next layer's keys do not depend on this step's output; nothing of the next
 * step is computed here. A hint only: results are bit-identical to qsa_decode_step's.
 *   next_read: 16-byte aligned, device memory or mapped pinned host memory, or NULL (no
 *   hint); next_read_bytes is rounded down to a multiple of 16 (below 16: no hint).
 * Everything else as qsa_decode_step / qsa_decode_step_fp8. A misaligned or unreadable
 * next_read is QSA_ERR_INVALID_ARGUMENT. */
QSA_API qsa_status qsa_decode_step_prefetch(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, qsa_bf16 *pooled,
                                            int64_t n_pooled_total, const int32_t *blk_off, const qsa_bf16 *q_idx,
                                            const qsa_bf16 *q, const qsa_bf16 *k_cache, const qsa_bf16 *v_cache,
                                            int64_t n_tokens_total, const int32_t *tok_off, const int32_t *ctx_len,
                                            int32_t B, int64_t max_blocks, int32_t *blocks, int32_t *count,
                                            qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes,
                                            const void *next_read, size_t next_read_bytes, qsa_stream stream);
QSA_API qsa_status qsa_decode_step_fp8_prefetch(const qsa_config *cfg, const qsa_bf16 *raw_idx_k, uint8_t *codes,
                                                float *scales, int64_t n_pooled_total, const int32_t *blk_off,
                                                const qsa_bf16 *q_idx, const qsa_bf16 *q, const qsa_bf16 *k_cache,
                                                const qsa_bf16 *v_cache, int64_t n_tokens_total,
                                                const int32_t *tok_off, const int32_t *ctx_len, int32_t B,
                                                int64_t max_blocks, int32_t *blocks, int32_t *count, qsa_bf16 *out,
                                                float *lse, void *ws, size_t ws_bytes, const void *next_read,
                                                size_t next_read_bytes, qsa_stream stream);

/* Allocation-free variant of qsa_sparse_decode (the pages have no counterpart; this
 * is a library convenience). Same arguments and result, but no workspace: the split
 * partials live in a 16 MiB static device array inside the library, for callers that
 * cannot allocate device memory at all (a plug-in inside a host application that owns
 * the whole device memory pool, a process whose device memory another allocator has
 * fully reserved, loops that must not risk an allocation's implicit synchronisation).
 *  - Limit: qsa_workspace_size(QSA_OP_SPARSE_DECODE, cfg, B, 0) must not exceed 16 MiB
 *    (B <= 30 at 16 query / 2 KV heads, B <= 61 at 8 / 2); larger batches return
 *    QSA_ERR_WORKSPACE_TOO_SMALL. Every host check (configuration, sizes, pointers, the
 *    stream's device) runs before anything is enqueued.
 *  - `stream` must belong to the current device (else QSA_ERR_INVALID_ARGUMENT): the
 *    array has one address per device.
 *  - The first call on a device resolves the array's device address
 *    (cudaGetSymbolAddress, with that device current) and caches it.
 *  - The array stays resident on every GPU that loads the library until exit.
 *  - Every call reuses the same array: calls that overlap on the GPU race. Each call
 *    clears the array's status block on `stream`; device-side bounds errors are not
 *    reported (the bad access is still skipped). It never calls cudaMalloc/cudaFree. */
QSA_API qsa_status qsa_sparse_decode_noalloc(const qsa_config *cfg, const qsa_bf16 *q, const qsa_bf16 *k_cache,
                                             const qsa_bf16 *v_cache, int64_t n_tokens_total,
                                             const int32_t *tok_off, const int32_t *ctx_len, int32_t B,
                                             const int32_t *blocks, const int32_t *count, qsa_bf16 *out,
                                             float *lse, qsa_stream stream);

/* f3 — Sparse MLA decode in its MQA form ("GLM-5.3 最適化 第2部：16基のH200上でのPCP、DCP、
 * およびHybrid HiSparse", footnote 1: each query reads 2,048 selected FP8 rows of 656 bytes;
 * QK runs over 576 dims, PV over 512; every row serves all heads). Row layout, 656 bytes:
 *   bytes 0..511   the 512-dim latent as E4M3 codes (dim d at byte d),
 *   bytes 512..527 four fp32 scales (scale g applies to latent dims 128g .. 128g+127),
 *   bytes 528..655 the 64 rotary dims as bf16.
 * With latent_j = code x scale and k_j = [latent_j, rope_j], query b's head h gives
 *   out[b][h] = sum_j softmax_j(scale_qk * q[b][h] . k_j) latent_j,  lse[b][h] = ln sum_j e^(...)
 * over j in rows[b][0 .. n_rows[b]) (token ids, any order, no repeats).
 *   q [B, n_heads, 576] bf16, 16-byte aligned; kv_rows [n_tokens, 656] uint8, 16-byte aligned;
 *   rows [B, max_rows] int32; n_rows [B] int32 (<= max_rows); out [B, n_heads, 512] bf16;
 *   lse [B, n_heads] fp32 or NULL; softmax_scale <= 0 selects 1/sqrt(576).
 * Tensor cores: tiles of 64 selected rows; latent values rounded once to bf16 for the MMA
 * (code x scale in fp32, then bf16), P rounded to bf16; fp32 accumulation; the tiles'
 * partials merged by log-sum-exp. n_heads 1..128 (MMA rows; else QSA_ERR_UNSUPPORTED).
 * Workspace: qsa_sparse_mla_workspace_size(n_heads, B, max_rows) bytes (status block + the
 * tiles' partials); device checks: 0 <= row id < n_tokens (a bad row is skipped and
 * QSA_ERR_DEVICE_BOUNDS recorded); n_rows[b] is clamped to [0, max_rows], a value above
 * max_rows also recording QSA_ERR_DEVICE_BOUNDS. A query with no rows gets out = 0 and
 * lse = -inf. */
QSA_API size_t qsa_sparse_mla_workspace_size(int32_t n_heads, int32_t B, int32_t max_rows);
QSA_API qsa_status qsa_sparse_mla_decode(const qsa_bf16 *q, int32_t n_heads, const uint8_t *kv_rows,
                                         int64_t n_tokens, const int32_t *rows, const int32_t *n_rows,
                                         int32_t max_rows, int32_t B, float softmax_scale, qsa_bf16 *out, float *lse,
                                         void *ws, size_t ws_bytes, qsa_stream stream);

/* ------------------------------------------------------------------ paged K/V cache
 * A cache cut into pages of page_size tokens, for layers that read their whole (or windowed)
 * history and for serving many requests from one pool. A pool plane is [n_pages][page_size][...]
 * (token-major inside a page, as the flat caches above); row r of a page table [n_rows][table_ld]
 * int32 lists the pages of one sequence in order: its token t is at
 *   slot = table[r * table_ld + t / page_size] * page_size + t % page_size,
 * and its K row of KV head h at k_cache + (slot * n_kv_heads + h) * head_dim ("3090x3で 314 万
 * コンテキスト", section "カーネルを書き換えずに済む": the same row address, with the slot in the
 * token's place). Entries behind a sequence's last page are not read; pages may be shared by
 * several rows. */
typedef struct {
    int32_t n_q_heads;   /* query head h reads KV head h / (n_q_heads / n_kv_heads); at most 16 per KV head */
    int32_t n_kv_heads;
    int32_t head_dim;    /* 64, 128 or 256 (FP8 rows: 128 or 256) */
    int32_t page_size;   /* tokens per page, >= 1 (no power of two needed) */
    int32_t window;      /* > 0: the new token sees the last `window` cached tokens only; 0: all */
    float softmax_scale; /* <= 0 selects 1/sqrt(head_dim) */
} qsa_paged_config;

/* Rotary positions. Pair i (0 <= i < rot_dim / 2) of a head turns by the angle p f_i:
 *   y[a] = amplitude (x[a] cos(p f_i) - x[b] sin(p f_i)),  y[b] = amplitude (x[b] cos(p f_i) + x[a] sin(p f_i))
 * with (a, b) = rot_begin + (i, i + rot_dim / 2) (halves) or rot_begin + (2i, 2i + 1) (interleaved);
 * other dims pass through. f_i = base^(-2i / rot_dim), rescaled for contexts longer than the trained
 * one by `scaling`:
 *   LINEAR    f_i / factor;
 *   NTK       the base becomes base x factor^(rot_dim / (rot_dim - 2));
 *   BY_PARTS  the interpolation by parts of YaRN (Peng et al. 2023, "YaRN: Efficient Context Window Extension of Large
 *             Language Models"): f_i (1 - g) + g f_i / factor with g = clamp((i - lo) / (hi - lo), 0, 1),
 *             lo = max(floor(c(beta_fast)), 0), hi = min(ceil(c(beta_slow)), rot_dim - 1) (hi - lo at least 0.001),
 *             c(b) = (rot_dim / 2) ln(original_len / (2 pi b)) / ln(base): pairs that turn more than beta_fast
 *             times over the trained length stay, those that turn less than beta_slow times are slowed. Where even the
 *             last pair turns more often than that (small bases, long trained lengths), hi lies past it and the
 *             ramp is cut off by the head's end;
 *             amplitude = 0.1 ln(factor) + 1 (factor > 1; else 1). The other scalings have amplitude 1. */
typedef enum {
    QSA_ROPE_NONE = 0,
    QSA_ROPE_LINEAR = 1,
    QSA_ROPE_NTK = 2,
    QSA_ROPE_BY_PARTS = 3
} qsa_rope_scaling;

typedef struct {
    int32_t head_dim;     /* multiple of 16, at most 1024 */
    int32_t rot_begin;    /* first turned dim: multiple of 8 */
    int32_t rot_dim;      /* turned dims: multiple of 16, 0 for none; rot_begin + rot_dim <= head_dim */
    int32_t interleaved;  /* pairs (2i, 2i+1) instead of (i, i + rot_dim/2) */
    int32_t scaling;      /* qsa_rope_scaling */
    int32_t original_len; /* BY_PARTS: trained context length */
    double base, factor;  /* base > 1; factor > 0 */
    double beta_fast, beta_slow; /* BY_PARTS: beta_fast > beta_slow > 0 */
} qsa_rope_config;

/* Host only: the table the rotary kernels read. phase[i] (rot_dim / 2 entries, HOST memory) is f_i / (2 pi)
 * modulo 1 as a 64-bit binary fraction of a turn, so position x phase modulo 2^64 is the angle exactly:
 * positions of millions lose nothing. *amplitude as above. Copy phase to the device once and keep it. A factor
 * that makes a frequency or the NTK base infinite or zero is QSA_ERR_INVALID_ARGUMENT. */
QSA_API qsa_status qsa_rope_table(const qsa_rope_config *rope, uint64_t *phase, float *amplitude);

/* Turn rows: out[n][h] = rotary(x[n][h], pos[n]) for n < N, h < n_heads, in fp32 with one rounding to bf16.
 * Negative positions turn backwards (the inverse, and the gradient, of position -p up to amplitude^2).
 *   x, out: rows of n_heads x head_dim contiguous bf16, x_ld / out_ld elements between rows (multiples of 8,
 *   at least n_heads head_dim); 16-byte aligned; out may be x (same ld), else they must not overlap;
 *   phase: the device copy of qsa_rope_table's, 16-byte aligned; pos [N] int32.
 * No workspace, no device-side errors. N = 0 is a no-op. */
QSA_API qsa_status qsa_rope(const qsa_rope_config *rope, const uint64_t *phase, float amplitude, const qsa_bf16 *x,
                            int64_t x_ld, const int32_t *pos, int32_t N, int32_t n_heads, qsa_bf16 *out,
                            int64_t out_ld, qsa_stream stream);

/* Bytes of a paged call's workspace for these heads (the same for every batch, length and page count; 0 on
 * unsupported geometry). Zero it once with qsa_workspace_init. */
QSA_API size_t qsa_paged_workspace_size(const qsa_paged_config *cfg);

/* Append new tokens to a paged cache: for n < N, token n belongs to row r = seq[n] (seq NULL: r = n) at
 * position p = pos[n]: q_out[n] = rotary(q[n], p), the K row at p becomes rotary(k[n], p) (each value rounded
 * once to bf16) and the V row v[n]. A token with r < 0 is padding: nothing of it is read or written.
 *   q [N] rows of n_q_heads x head_dim, q_ld elements apart (NULL: no queries); k, v likewise with n_kv_heads
 *   (q, k and v may be slices of one projection's rows); lds multiples of 8; 16-byte aligned;
 *   q_out rows q_out_ld apart (may be q with the same ld); rope->head_dim = cfg->head_dim.
 * No (row, position) twice in one call, and no page that another row reads at that position: which of two
 * writes stays is undefined. Device checks (the K/V write is skipped, QSA_ERR_DEVICE_BOUNDS recorded, q_out
 * still written): r < n_rows, 0 <= p < table_ld page_size, 0 <= page < n_pages. */
QSA_API qsa_status qsa_rope_append(const qsa_paged_config *cfg, const qsa_rope_config *rope, const uint64_t *phase,
                                   float amplitude, const qsa_bf16 *q, int64_t q_ld, const qsa_bf16 *k, int64_t k_ld,
                                   const qsa_bf16 *v, int64_t v_ld, const int32_t *seq, const int32_t *pos, int32_t N,
                                   qsa_bf16 *q_out, int64_t q_out_ld, qsa_bf16 *k_cache, qsa_bf16 *v_cache,
                                   int64_t n_pages, const int32_t *table, int64_t table_ld, int32_t n_rows, void *ws,
                                   size_t ws_bytes, qsa_stream stream);

/* qsa_rope_append into FP8 rows: the turned K row (in fp32, not rounded to bf16 first) and the V row are
 * quantised per 128 dims as qsa_quantize_kv_fp8 does (scale = max |x| / 448, E4M3(x / scale), scale 0 and
 * zero codes for zeros). A NaN gets a NaN code and counts as nothing in max |x|; a group with an infinite value has an
 * infinite scale, which makes NaN of it.
 *   codes [n_pages][page_size][n_kv_heads][head_dim] uint8, 16-byte aligned; scales [..][head_dim / 128] fp32,
 *   8-byte aligned. */
QSA_API qsa_status qsa_rope_append_fp8kv(const qsa_paged_config *cfg, const qsa_rope_config *rope,
                                         const uint64_t *phase, float amplitude, const qsa_bf16 *q, int64_t q_ld,
                                         const qsa_bf16 *k, int64_t k_ld, const qsa_bf16 *v, int64_t v_ld,
                                         const int32_t *seq, const int32_t *pos, int32_t N, qsa_bf16 *q_out,
                                         int64_t q_out_ld, uint8_t *k_codes, float *k_scales, uint8_t *v_codes,
                                         float *v_scales, int64_t n_pages, const int32_t *table, int64_t table_ld,
                                         int32_t n_rows, void *ws, size_t ws_bytes, qsa_stream stream);

/* Attention of one new token per sequence over its whole paged cache, split over the length and joined by
 * log-sum-exp (the dense companion of qsa_sparse_decode). Sequence s has n = seq_len[s] cached tokens, the new
 * one among them, and attends j in [max(0, n - window), n) (all n without a window):
 *   out[s][h] = sum_j softmax_j(scale q[s][h] . K[j]) V[j],   lse[s][h] = ln sum_j e^(scale q.K[j]).
 * A sequence with n = 0 gets out = 0 and lse = -inf. fp32 scores, softmax and sums; the weights enter the
 * second product as the sum of two bf16 values (2^-16 of each; an infinite V value of an attended token gives that
 * infinity). Pages that no attended token lies in are not read.
 *   q rows of n_q_heads x head_dim, q_ld elements apart (a multiple of 8), 16-byte aligned; k_cache, v_cache
 *   16-byte aligned, device memory or mapped pinned host memory; n_pages page_size < 2^31; seq_len [B];
 *   out [B][n_q_heads][head_dim] bf16, 16-byte aligned; lse [B][n_q_heads] fp32 or NULL.
 * Device checks: 0 <= n <= table_ld page_size (else the sequence counts as empty), 0 <= page < n_pages (its
 * tokens are then left out); QSA_ERR_DEVICE_BOUNDS is recorded. Results do not depend on timing: the split
 * depends on the lengths and the device alone. The first call on a device queries its occupancy and should
 * precede stream capture. */
QSA_API qsa_status qsa_paged_decode(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                    const qsa_bf16 *k_cache, const qsa_bf16 *v_cache, int64_t n_pages,
                                    const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                    qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, qsa_stream stream);

/* qsa_paged_decode over the FP8 rows qsa_rope_append_fp8kv writes (head_dim 128 or 256). Scores and softmax as there;
 * the codes enter both products exactly. q enters as f16 scaled by a power of two per head (exact down to 2^-17 of the
 * head's largest value, smaller ones off by at most 2^-25 of it), or (256 dims, at most 8 query heads per KV head) as
 * the sum of two scaled E4M3 values, which hold all of a bf16 value down to 2^-14 of the head's largest; smaller ones are
 * rounded by up to 2^-22 of that. Each weight x V scale is rounded once, by at most 2^-11 of it or 2^-40 of the largest of
 * its sequence (so what lies below 2^-40 of that is zero). Scales must not be negative; a V scale that is infinite or NaN
 * makes its 128 dims of its sequence's heads NaN, and nothing else; one below 2^-126 counts as zero. */
QSA_API qsa_status qsa_paged_decode_fp8kv(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                          const uint8_t *k_codes, const float *k_scales, const uint8_t *v_codes,
                                          const float *v_scales, int64_t n_pages, const int32_t *table,
                                          int64_t table_ld, const int32_t *seq_len, int32_t B, qsa_bf16 *out,
                                          float *lse, void *ws, size_t ws_bytes, qsa_stream stream);

/* Planes of a pool that move together: n_planes arrays [n_pages][page_bytes], plane_stride bytes apart (e.g.
 * the K caches of all layers). page_bytes a multiple of 4, plane_stride of page_bytes's alignment (16 where
 * page_bytes is a multiple of 16, else 4), bases aligned likewise; device memory or mapped pinned host memory. */
typedef struct {
    void *base;
    int64_t plane_stride;
    int64_t page_bytes;
    int32_t n_planes;
} qsa_page_planes;
#define QSA_MAX_PLANE_GROUPS 8

/* Workspace of the page calls for tables of at most n_rows rows and pools of at most n_pages pages. */
QSA_API size_t qsa_pages_workspace_size(int32_t n_rows, int64_t n_pages);

/* One step of a pool's bookkeeping: fork, extend, free and start sequences. Row i < n_out of the new table
 * continues row parent[i] of the old one (-1: starts empty) with room for add[i] >= 0 more tokens:
 *   seq_len_out[i] = seq_len[parent[i]] + add[i];
 *   full pages of the parent are shared; its partly filled last page stays with the first row that continues
 *   it if nothing else refers to it (ref 1), and every other row gets a page of its own with the used tokens
 *   copied in every plane (ceil(used page_bytes / page_size) bytes, rounded up to 16 or 4); then pages for the added tokens.
 * New pages are the lowest-numbered ones with ref = 0, taken in row order (a row's copied page first).
 * Old rows that nothing continues give their pages back. ref_out[p] = ref[p] - entries of the old table + entries of
 * the new table that name page p (other holders' references stay). Entries behind a row's last page are -1.
 * parent = row, add = 1 is a decode step's extension; a repeated parent is a fork; parent -1, add 0 frees.
 *   parent, add, seq_len_out [n_out]; seq_len [n_in]; table [n_in][ld], table_out [n_out][ld] (another array);
 *   ref, ref_out [n_pages] (another array); n_in, n_out <= 65536. planes: n_groups <= 8 groups (HOST
 *   array; 0 groups: bookkeeping alone).
 * A row that runs out of pages or of the table's ld, or names a parent outside [0, n_in), becomes empty
 * and QSA_ERR_DEVICE_BOUNDS is recorded with its index; what a row short of pages would have taken is not handed to
 * later rows. */
QSA_API qsa_status qsa_fork_pages(int32_t page_size, const int32_t *parent, const int32_t *add, int32_t n_out,
                                  const int32_t *table, const int32_t *seq_len, int32_t n_in, int64_t ld,
                                  const int32_t *ref, int64_t n_pages, int32_t *table_out, int32_t *seq_len_out,
                                  int32_t *ref_out, const qsa_page_planes *planes, int32_t n_groups, void *ws,
                                  size_t ws_bytes, qsa_stream stream);

/* Compact a pool: with n_live pages of ref > 0, every live page with id >= n_live moves (in ascending order) into the
 * free ids below n_live (ascending), in every plane; table_out and ref_out name the new places. The contents of
 * pages >= n_live are left as they were. table_out may be table; ref_out is another array than ref. A table entry inside its row's
 * length that names no live page is recorded (QSA_ERR_DEVICE_BOUNDS, the row) and becomes -1. */
QSA_API qsa_status qsa_compact_pages(int32_t page_size, const int32_t *table, const int32_t *seq_len, int32_t n_rows,
                                     int64_t ld, const int32_t *ref, int64_t n_pages, int32_t *table_out,
                                     int32_t *ref_out, const qsa_page_planes *planes, int32_t n_groups, void *ws,
                                     size_t ws_bytes, qsa_stream stream);

/* Copy pages: page dst[i] of every destination plane becomes page src[i] of the source plane, i < n; a pair with a
 * negative id is skipped, one out of range recorded (QSA_ERR_DEVICE_BOUNDS). dst_planes NULL: inside the same pool
 * (then no dst may be another pair's src or dst). Groups of dst_planes match planes' n_planes and page_bytes; planes may be
 * device or mapped pinned host memory, e.g. to move a sequence's pages to the host and back. */
QSA_API qsa_status qsa_copy_pages(const int32_t *src, const int32_t *dst, int32_t n, const qsa_page_planes *planes,
                                  int64_t n_pages, const qsa_page_planes *dst_planes, int64_t n_dst_pages,
                                  int32_t n_groups, void *ws, size_t ws_bytes, qsa_stream stream);

/* ------------------------------------------------- drafted tokens and eviction over a paged cache
 * Speculative decoding: qsa_rope_append_at stores a sequence's drafted tokens behind its cached ones,
 * qsa_tree_decode attends for all of them, qsa_accept_drafts keeps the accepted ones. A cache with a budget:
 * qsa_paged_decode_weights accumulates each token's attention weight and qsa_evict_tokens drops the lightest tokens.
 * There a token's place in its row (which fixes its page and slot) is no longer its position (which fixes its rotary
 * angle): a drafted token's position is its depth in the tree, and an evicted token's place is taken by a later one. */

/* qsa_rope_append for tokens whose place is not their position: token n turns to position pos[n] and is stored as token
 * place[n] of row seq[n]. positions (NULL: not wanted) [n_rows][positions_ld] int32: positions[r][place[n]] = pos[n], for
 * places below positions_ld. Everything else as qsa_rope_append, with place in pos's part in the device checks. */
QSA_API qsa_status qsa_rope_append_at(const qsa_paged_config *cfg, const qsa_rope_config *rope, const uint64_t *phase,
                                      float amplitude, const qsa_bf16 *q, int64_t q_ld, const qsa_bf16 *k, int64_t k_ld,
                                      const qsa_bf16 *v, int64_t v_ld, const int32_t *seq, const int32_t *pos,
                                      const int32_t *place, int32_t N, qsa_bf16 *q_out, int64_t q_out_ld,
                                      qsa_bf16 *k_cache, qsa_bf16 *v_cache, int64_t n_pages, const int32_t *table,
                                      int64_t table_ld, int32_t n_rows, int32_t *positions, int64_t positions_ld,
                                      void *ws, size_t ws_bytes, qsa_stream stream);
QSA_API qsa_status qsa_rope_append_at_fp8kv(const qsa_paged_config *cfg, const qsa_rope_config *rope,
                                            const uint64_t *phase, float amplitude, const qsa_bf16 *q, int64_t q_ld,
                                            const qsa_bf16 *k, int64_t k_ld, const qsa_bf16 *v, int64_t v_ld,
                                            const int32_t *seq, const int32_t *pos, const int32_t *place, int32_t N,
                                            qsa_bf16 *q_out, int64_t q_out_ld, uint8_t *k_codes, float *k_scales,
                                            uint8_t *v_codes, float *v_scales, int64_t n_pages, const int32_t *table,
                                            int64_t table_ld, int32_t n_rows, int32_t *positions, int64_t positions_ld,
                                            void *ws, size_t ws_bytes, qsa_stream stream);

#define QSA_MAX_DRAFT 128

/* Workspace of qsa_tree_decode for at most max_draft drafted tokens a sequence (the same for every batch, length and
 * page count; 0 on unsupported geometry). Zero it once with qsa_workspace_init. */
QSA_API size_t qsa_tree_workspace_size(const qsa_paged_config *cfg, int32_t max_draft);

/* Attention of every sequence's drafted tokens over its paged cache. Sequence s has the drafted tokens
 * i = draft_off[s] .. draft_off[s + 1] - 1 of the batch's list, T of them: the last T of its n = seq_len[s] cached
 * tokens, in the list's order. parent[i] is the place of token i's parent among the sequence's own T (below i's own
 * place), or -1 for a child of the cached tokens. Token i attends the n - T cached tokens before the drafts, its
 * ancestors and itself:
 *   out[i][h] = sum_j softmax_j(scale q[i][h] . K[j]) V[j],   lse[i][h] = ln sum_j e^(scale q.K[j]).
 * A chain (parent = place - 1) is the causal attention of several new tokens. With a window a token at depth d (1: no
 * drafted ancestor) has position n - T + d - 1 and attends positions above that - window; the cached tokens' positions
 * are their places.
 *   q [N] rows of n_q_heads x head_dim, q_ld elements apart (a multiple of 8), 16-byte aligned; draft_off [B + 1],
 *   ascending, within [0, N]; parent [N]; max_draft: the most drafted tokens of a sequence, 1 .. QSA_MAX_DRAFT (no more
 *   than there can be: the GPU is split among that many tokens' rows, so 4 drafts with max_draft 128 take 2 to 4.5 times as
 *   long as with 4);
 *   out [N][n_q_heads][head_dim] bf16, 16-byte aligned; lse [N][n_q_heads] fp32 or NULL; k_cache, v_cache 16-byte
 *   aligned device memory. Rows of out and lse that no sequence names stay as they were.
 * fp32 scores, softmax and sums; the weights enter the second product as bf16 (each rounded by at most 2^-8 of it, as out
 * itself is). V values that are not finite reach the tokens that attend them, and no others (as that value, or as NaN where
 * the weight is zero in that many bits).
 * Device checks (QSA_ERR_DEVICE_BOUNDS is recorded): a sequence whose offsets do not ascend within [0, N], or begin below an
 * earlier one's, attends nothing and its rows are not written; one with T > max_draft, T > n or n > table_ld page_size
 * attends nothing (out = 0, lse = -inf); a parent outside [-1, own place) counts as -1; a page outside [0, n_pages) has
 * its tokens left out. A token that attends nothing gets out = 0 and
 * lse = -inf. Results do not depend on timing: the split depends on the lengths, max_draft and the device alone. A wait inside
 * the kernel that makes no progress for 250 ms ends the call with QSA_ERR_DEVICE_TIMEOUT. The first call on a device queries
 * its occupancy and should precede stream capture. */
QSA_API qsa_status qsa_tree_decode(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                   const int32_t *draft_off, const int32_t *parent, int32_t N, int32_t max_draft,
                                   const qsa_bf16 *k_cache, const qsa_bf16 *v_cache, int64_t n_pages,
                                   const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                   qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, qsa_stream stream);

/* qsa_tree_decode over the FP8 rows qsa_rope_append_fp8kv writes (head_dim 128 or 256). The codes enter both products
 * exactly. q enters as the sum of two scaled E4M3 values, which hold all of a bf16 value down to 2^-10 of its head's largest;
 * smaller ones are rounded by up to 2^-17 of that. Each weight x V scale is rounded once, by at most 2^-11 of it or 2^-31 of
 * the largest weight times the largest V scale of the sequence. Scales must not be negative; a V scale that is infinite or
 * NaN makes its 128 dims NaN for the tokens that attend it, and nothing else; V scales outside 2^-120 .. 2^120 are not
 * told from those bounds. */
QSA_API qsa_status qsa_tree_decode_fp8kv(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                         const int32_t *draft_off, const int32_t *parent, int32_t N,
                                         int32_t max_draft, const uint8_t *k_codes, const float *k_scales,
                                         const uint8_t *v_codes, const float *v_scales, int64_t n_pages,
                                         const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                         qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, qsa_stream stream);

/* Workspace of qsa_paged_decode_weights for a batch of at most B sequences with at most n_tokens attended tokens
 * together (0 on unsupported geometry). Zero it once with qsa_workspace_init. */
QSA_API size_t qsa_paged_weights_workspace_size(const qsa_paged_config *cfg, int32_t B, int64_t n_tokens);

/* qsa_paged_decode that also accumulates what each cached token received:
 *   weights[s][j] += sum_h softmax_j(scale q[s][h] . K[j])   for the attended tokens j of sequence s,
 * in fp32, each head's weight from its final log-sum-exp and the heads summed in order. weights [B][weights_ld] fp32,
 * 4-byte aligned; entries of tokens that are not attended stay as they were. out and lse are qsa_paged_decode's, bit
 * for bit. Device checks beside those: tokens at or behind weights_ld, and those behind the workspace's n_tokens, add
 * nothing (QSA_ERR_DEVICE_BOUNDS). */
QSA_API qsa_status qsa_paged_decode_weights(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                            const qsa_bf16 *k_cache, const qsa_bf16 *v_cache, int64_t n_pages,
                                            const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                            qsa_bf16 *out, float *lse, float *weights, int64_t weights_ld, void *ws,
                                            size_t ws_bytes, qsa_stream stream);
QSA_API qsa_status qsa_paged_decode_weights_fp8kv(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                                  const uint8_t *k_codes, const float *k_scales,
                                                  const uint8_t *v_codes, const float *v_scales, int64_t n_pages,
                                                  const int32_t *table, int64_t table_ld, const int32_t *seq_len,
                                                  int32_t B, qsa_bf16 *out, float *lse, float *weights,
                                                  int64_t weights_ld, void *ws, size_t ws_bytes, qsa_stream stream);

/* Workspace of qsa_accept_drafts, qsa_accept_drafts_weights (max_tokens 0) and qsa_evict_tokens (max_tokens: its weights_ld) for at most n_rows
 * rows. Zero it once with qsa_workspace_init. */
QSA_API size_t qsa_keep_workspace_size(int32_t n_rows, int64_t max_tokens);

/* Keep the accepted drafted tokens. Row r's drafted tokens are the last T = draft_off[r + 1] - draft_off[r] of its
 * seq_len[r] tokens, with parents as in qsa_tree_decode. accepted[r] is the place of the last accepted one among them
 * (-1: none): it and its ancestors stay, oldest first, directly behind the cached tokens, in every plane; the rest is
 * dropped and pages that hold no token any more are given back:
 *   seq_len_out[r] = seq_len[r] - T + depth of accepted[r];  ref_out[p] = ref[p] - entries that named p and are dropped;
 *   table_out: the table with -1 behind each row's last page.
 * The pages of kept drafted tokens must be the row's own (qsa_fork_pages sees to that for tokens appended behind it).
 *   draft_off [n_rows + 1]; parent [N]; accepted, seq_len, seq_len_out [n_rows]; table, table_out [n_rows][ld]; ref, ref_out
 *   [n_pages] (each _out another array); n_rows <= 65536, n_pages page_size < 2^31; positions (NULL: none) [n_rows][positions_ld] int32, moved along in
 *   place; planes as in qsa_fork_pages, page_bytes a multiple of page_size x 4.
 * A row whose seq_len, draft_off, parents or accepted are out of range, or whose tokens would move into a page that other
 * references share (ref > 1), keeps all its tokens (QSA_ERR_DEVICE_BOUNDS, the row); a page out of range is left out. */
QSA_API qsa_status qsa_accept_drafts(int32_t page_size, const int32_t *draft_off, const int32_t *parent, int32_t N,
                                     const int32_t *accepted, const int32_t *table, const int32_t *seq_len,
                                     int32_t n_rows, int64_t ld, const int32_t *ref, int64_t n_pages, int32_t *table_out,
                                     int32_t *seq_len_out, int32_t *ref_out, int32_t *positions, int64_t positions_ld,
                                     const qsa_page_planes *planes, int32_t n_groups, void *ws, size_t ws_bytes,
                                     qsa_stream stream);

/* qsa_accept_drafts for rows that accumulate weights, with drafted tokens among those that were weighed: weights and
 * positions [n_rows][tokens_ld] move along with the accepted path in place, and become 0 and -1 from each row's new length to
 * its old one, so that a later token at a dropped one's place starts with nothing. A row that keeps all its tokens keeps
 * these too. weights fp32, both 4-byte aligned; everything else as in qsa_accept_drafts. */
QSA_API qsa_status qsa_accept_drafts_weights(int32_t page_size, const int32_t *draft_off, const int32_t *parent, int32_t N,
                                             const int32_t *accepted, float *weights, int32_t *positions, int64_t tokens_ld,
                                             const int32_t *table, const int32_t *seq_len, int32_t n_rows, int64_t ld,
                                             const int32_t *ref, int64_t n_pages, int32_t *table_out, int32_t *seq_len_out,
                                             int32_t *ref_out, const qsa_page_planes *planes, int32_t n_groups, void *ws,
                                             size_t ws_bytes, qsa_stream stream);

/* Cut rows down to their budget by accumulated weight. Row r of n = seq_len[r] tokens keeps all of them if n <=
 * budget[r] or budget[r] < 0. Otherwise it always keeps the tokens at positions below `first`, those at the last `recent`
 * positions (above the row's highest position - recent) and those in pages that other references share (ref > 1:
 * dropping them would free nothing), P tokens; of the others it keeps the heaviest, equal weights by lower place, until
 * K = max(budget[r], P) stay. Only kept tokens at places >= K move: in ascending order into the places below K that
 * dropped tokens held, ascending, in every plane, with their weights and positions. Pages that hold no token any more
 * are given back (ref_out, table_out as in qsa_accept_drafts). Rows are cut fastest where tokens_ld is at most 16,384: with
 * more room another kernel takes about three times as long for rows of 4,000 tokens.
 *   weights [n_rows][tokens_ld] fp32 (a NaN counts as the lightest, -0 as 0), positions [n_rows][tokens_ld] int32;
 *   weights_out, positions_out: other arrays of their shape, 0 and -1 behind a row's new length; budget [n_rows];
 *   first, recent >= 0; the rest as in qsa_accept_drafts.
 * A row with seq_len outside [0, ld page_size] or above tokens_ld keeps its table and length (QSA_ERR_DEVICE_BOUNDS, the
 * row); its weights_out and positions_out are copies. A page out of range is left out and recorded. */
QSA_API qsa_status qsa_evict_tokens(int32_t page_size, const int32_t *budget, int32_t first, int32_t recent,
                                    const float *weights, const int32_t *positions, int64_t tokens_ld,
                                    const int32_t *table, const int32_t *seq_len, int32_t n_rows, int64_t ld,
                                    const int32_t *ref, int64_t n_pages, float *weights_out, int32_t *positions_out,
                                    int32_t *table_out, int32_t *seq_len_out, int32_t *ref_out,
                                    const qsa_page_planes *planes, int32_t n_groups, void *ws, size_t ws_bytes,
                                    qsa_stream stream);

/* Static description of a status code. */
QSA_API const char *qsa_status_string(qsa_status s);

/* Detail of the last host-side error on the calling thread ("" if none). */
QSA_API const char *qsa_last_error(void);

/* Library version, e.g. "qsa-gb300 0.1.0 sm_103a". */
QSA_API const char *qsa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QSA_H */
