"""Device buffers and call sequences for one decode layer-step or one prefill chunk.

Only marshalling: torch allocates the buffers and the metadata tensors, and every
step of the path runs in libqsa.so through the ``qsa_*`` calls of :mod:`.binding`.
"""

from __future__ import annotations

import torch

from . import binding as qb

RATIO = 4


class DecodeBatch:
    """A ragged decode batch: sequence s has its query at p = ctx_len[s] and p + 1
    cached tokens at tok_off[s] .. tok_off[s+1]-1 of the flat K/V arrays."""

    def __init__(self, n_q_heads: int, n_kv_heads: int, ctx_len, device="cuda", softmax_scale: float = 0.0):
        self.cfg = qb.make_config(n_q_heads, n_kv_heads, softmax_scale=softmax_scale)
        self.ctx = [int(p) for p in ctx_len]
        self.B = len(self.ctx)
        self.device = device
        i32 = dict(dtype=torch.int32, device=device)
        tok_off, blk_off, nblk = [0], [0], []
        for p in self.ctx:
            tok_off.append(tok_off[-1] + p + 1)
            nblk.append((p + 1) // RATIO)          # complete blocks among the p+1 cached tokens
            blk_off.append(blk_off[-1] + nblk[-1])
        self.n_tokens = tok_off[-1]
        self.n_pooled = blk_off[-1]
        self.max_blocks = max(nblk) if nblk else 0
        self.ld = max(1, max((p // RATIO for p in self.ctx), default=1))
        self.tok_off = torch.tensor(tok_off, **i32)
        self.blk_off = torch.tensor(blk_off, **i32)
        self.ctx_len = torch.tensor(self.ctx, **i32)
        self.q_seq = torch.arange(self.B, **i32)
        self.blk_begin = torch.zeros(self.B, **i32)
        self.blk_end = torch.tensor(nblk, **i32)
        self.scores = torch.empty(self.B, self.ld, dtype=torch.float32, device=device)
        self.blocks = torch.empty(self.B, qb.BLOCK_TOPK, **i32)
        self.count = torch.empty(self.B, **i32)
        self.out = torch.empty(self.B, n_q_heads, 256, dtype=torch.bfloat16, device=device)
        self.lse = torch.empty(self.B, n_q_heads, dtype=torch.float32, device=device)
        sizes = [qb.workspace_size(qb.OP_POOL_KEYS, self.cfg, self.B, self.max_blocks),
                 qb.workspace_size(qb.OP_INDEX_SCORE, self.cfg, self.B, self.ld),
                 qb.workspace_size(qb.OP_TOPK_BLOCKS, self.cfg, self.B, self.ld),
                 qb.workspace_size(qb.OP_SPARSE_DECODE, self.cfg, self.B, self.ld)]
        self.ws = _workspace(max(sizes), device)
        self.step_ws = None
        if self.B <= 64:
            n = qb.workspace_size(qb.OP_DECODE_STEP, self.cfg, self.B, self.ld)
            if n:
                self.step_ws = _workspace(n, device)

    def new_pooled(self):
        return torch.empty(max(self.n_pooled, 1), 128, dtype=torch.bfloat16, device=self.device)

    def fused_step(self, raw_idx_k, pooled, q_idx, q, k_cache, v_cache, stream=None, next_read=None):
        """One decode layer-step in one launch (qsa_decode_step): re-pool the newest
        block, score, select, attend, merge. `next_read` (e.g. the next layer's pooled
        keys) is prefetched into L2 while the step exchanges keys and partials."""
        qb.qsa_decode_step(self.cfg, raw_idx_k, pooled, self.blk_off, q_idx, q, k_cache, v_cache, self.tok_off,
                           self.ctx_len, self.ld, self.blocks, self.count, self.out, self.lse, self.step_ws, stream,
                           next_read)

    def fused_step_fp8(self, raw_idx_k, codes, scales, q_idx, q, k_cache, v_cache, stream=None, next_read=None):
        """qsa_decode_step over FP8 indexer keys (qsa_decode_step_fp8)."""
        qb.qsa_decode_step_fp8(self.cfg, raw_idx_k, codes, scales, self.blk_off, q_idx, q, k_cache, v_cache,
                               self.tok_off, self.ctx_len, self.ld, self.blocks, self.count, self.out, self.lse,
                               self.step_ws, stream, next_read)

    def fused_step_fp8kv(self, raw_idx_k, keys, q_idx, q, kv8, stream=None):
        """The fused step over FP8 K/V rows (qsa_decode_step_fp8kv). `keys` is the bf16 pooled-key
        tensor or a (codes, scales) pair of FP8 keys; `kv8` is (k_codes, k_scales, v_codes,
        v_scales) as qsa_quantize_kv_fp8 writes them."""
        pooled, codes, scales = (keys, None, None) if torch.is_tensor(keys) else (None, *keys)
        qb.qsa_decode_step_fp8kv(self.cfg, raw_idx_k, pooled, codes, scales, self.blk_off, q_idx, q, *kv8,
                                 self.tok_off, self.ctx_len, self.ld, self.blocks, self.count, self.out, self.lse,
                                 self.step_ws, stream)

    def fused_step_rowcache(self, raw_idx_k, pooled, q_idx, q, k_cache, v_cache, cache, n_slots, epoch, stream=None):
        """qsa_decode_step with the VRAM row cache `cache` (binding.rowcache_new) in front of
        K/V in host memory; `epoch` grows by at least one per call with the same cache."""
        qb.qsa_decode_step_rowcache(self.cfg, raw_idx_k, pooled, self.blk_off, q_idx, q, k_cache, v_cache,
                                    self.tok_off, self.ctx_len, self.ld, self.blocks, self.count, self.out, self.lse,
                                    self.step_ws, cache, n_slots, epoch, stream)

    def fused_status(self, stream=None):
        return qb.qsa_read_device_status(self.step_ws, stream)

    def pool(self, raw_idx_k, pooled, stream=None):
        qb.qsa_pool_keys(self.cfg, raw_idx_k, self.tok_off, self.blk_off, self.blk_begin, self.blk_end,
                         self.max_blocks, pooled, self.ws, stream)

    def score(self, q_idx, pooled, stream=None):
        qb.qsa_index_score(self.cfg, q_idx, self.q_seq, self.ctx_len, pooled, self.blk_off, self.scores, self.ws,
                           stream)

    def topk(self, stream=None):
        qb.qsa_topk_blocks(self.cfg, self.scores, self.ctx_len, self.blocks, self.count, self.ws, stream)

    def attend(self, q, k_cache, v_cache, blocks=None, count=None, stream=None):
        qb.qsa_sparse_decode(self.cfg, q, k_cache, v_cache, self.tok_off, self.ctx_len,
                             self.blocks if blocks is None else blocks, self.count if count is None else count,
                             self.out, self.lse, self.ws, stream)

    def step(self, q_idx, q, k_cache, v_cache, pooled, stream=None):
        """One decode layer-step: score -> top-k -> sparse attention + LSE merge."""
        self.score(q_idx, pooled, stream)
        self.topk(stream)
        self.attend(q, k_cache, v_cache, stream=stream)

    def new_fp8_keys(self):
        """Buffers of the FP8 indexer keys: codes [n, 128] uint8 and scales [n] fp32, n = the
        pooled block count padded to a multiple of 4 (the fused step copies whole groups of 4 scales)."""
        n = max((self.n_pooled + 3) // 4 * 4, 4)
        return (torch.empty(n, 128, dtype=torch.uint8, device=self.device),
                torch.empty(n, dtype=torch.float32, device=self.device))

    def pool_fp8(self, raw_idx_k, codes, scales, stream=None):
        qb.qsa_pool_keys_fp8(self.cfg, raw_idx_k, self.tok_off, self.blk_off, self.blk_begin, self.blk_end,
                             self.max_blocks, codes, scales, self.ws, stream)

    def score_fp8(self, q_idx, codes, scales, stream=None):
        qb.qsa_index_score_fp8(self.cfg, q_idx, self.q_seq, self.ctx_len, codes, scales, self.blk_off, self.scores,
                               self.ws, stream)

    def step_fp8(self, q_idx, q, k_cache, v_cache, codes, scales, stream=None):
        """One decode layer-step with FP8 indexer keys: score -> top-k -> sparse attention."""
        self.score_fp8(q_idx, codes, scales, stream)
        self.topk(stream)
        self.attend(q, k_cache, v_cache, stream=stream)

    def device_status(self, stream=None):
        return qb.qsa_read_device_status(self.ws, stream)


class PrefillChunk:
    """A chunk of Nc queries at positions p0 .. p0+Nc-1 of one sequence whose cache
    holds p0 + Nc tokens (the chunk's K/V already appended)."""

    def __init__(self, n_q_heads: int, n_kv_heads: int, p0: int, n_chunk: int, interval_tokens: int = 8192,
                 device="cuda", softmax_scale: float = 0.0):
        self.cfg = qb.make_config(n_q_heads, n_kv_heads, softmax_scale=softmax_scale)
        self.p0, self.Nc, self.interval = int(p0), int(n_chunk), int(interval_tokens)
        self.device = device
        i32 = dict(dtype=torch.int32, device=device)
        self.n_tokens = self.p0 + self.Nc
        self.n_pooled = self.n_tokens // RATIO
        # score rows padded to 32 floats (128 bytes): aligned line writes and vector reads
        self.ld = max(1, (self.p0 + self.Nc - 1) // RATIO + 31) // 32 * 32
        self.tok_off = torch.tensor([0, self.n_tokens], **i32)
        self.blk_off = torch.zeros(2, **i32)
        self.q_seq = torch.zeros(self.Nc, **i32)
        self.q_pos = torch.arange(self.p0, self.p0 + self.Nc, **i32)
        self.scores = torch.empty(self.Nc, self.ld, dtype=torch.float32, device=device)
        self.blocks = torch.empty(self.Nc, qb.BLOCK_TOPK, **i32)
        self.count = torch.empty(self.Nc, **i32)
        self.out = torch.empty(self.Nc, n_q_heads, 256, dtype=torch.bfloat16, device=device)
        self.lse = torch.empty(self.Nc, n_q_heads, dtype=torch.float32, device=device)
        sizes = [qb.workspace_size(qb.OP_POOL_KEYS, self.cfg, 1, self.n_pooled),
                 qb.workspace_size(qb.OP_INDEX_SCORE, self.cfg, self.Nc, self.ld),
                 qb.workspace_size(qb.OP_TOPK_BLOCKS, self.cfg, self.Nc, self.ld),
                 qb.workspace_size(qb.OP_SPARSE_PREFILL_CHUNK, self.cfg, self.Nc, self.ld)]
        # scoring and top-k fused (no score matrix) for chunks of at least one 128-query tile
        self.fused_select = self.Nc >= 128 and self.n_pooled >= 256
        if self.fused_select:
            sizes.append(qb.workspace_size(qb.OP_PREFILL_SELECT, self.cfg, self.Nc, self.ld))
        self.ws = _workspace(max(sizes), device)

    def new_pooled(self):
        return torch.empty(max(self.n_pooled, 1), 128, dtype=torch.bfloat16, device=self.device)

    def pool(self, raw_idx_k, pooled, first_block: int = 0, stream=None):
        """Pool blocks [first_block, (p0+Nc)//4) (the whole history, or just the chunk's)."""
        i32 = dict(dtype=torch.int32, device=self.device)
        qb.qsa_pool_keys(self.cfg, raw_idx_k, self.tok_off, self.blk_off, torch.tensor([first_block], **i32),
                         torch.tensor([self.n_pooled], **i32), max(0, self.n_pooled - first_block), pooled, self.ws,
                         stream)

    def score(self, q_idx, pooled, stream=None, gemm=True):
        """All chunk queries share one history: with gemm the call passes no per-query
        sequence ids, which selects the tensor-core GEMM; otherwise one query at a time."""
        qb.qsa_index_score(self.cfg, q_idx, None if gemm else self.q_seq, self.q_pos, pooled, self.blk_off,
                           self.scores, self.ws, stream)

    def topk(self, stream=None):
        qb.qsa_topk_blocks(self.cfg, self.scores, self.q_pos, self.blocks, self.count, self.ws, stream)

    def select(self, q_idx, pooled, stream=None):
        """Scores and top-k in one call without the score matrix (qsa_prefill_select)."""
        qb.qsa_prefill_select(self.cfg, q_idx, self.q_pos, pooled, self.blk_off, self.scores, self.blocks, self.count,
                              self.ws, stream)

    def attend(self, q, k_cache, v_cache, blocks=None, count=None, stream=None):
        qb.qsa_sparse_prefill_chunk(self.cfg, q, self.p0, k_cache, v_cache,
                                    self.blocks if blocks is None else blocks,
                                    self.count if count is None else count, self.interval, self.out, self.lse,
                                    self.ws, stream)

    def attend_staged(self, q, k_cache, v_cache, stage, stream=None):
        """attend() with K/V (e.g. in pinned host memory) copied into the device arena `stage`
        first (qsa_sparse_prefill_chunk_staged)."""
        qb.qsa_sparse_prefill_chunk_staged(self.cfg, q, self.p0, k_cache, v_cache, self.blocks, self.count,
                                           self.interval, self.out, self.lse, self.ws, stage, stream)

    def attend_fp8kv(self, q, kv8, stage, stream=None):
        """attend() over FP8 K/V rows kv8 = (k_codes, k_scales, v_codes, v_scales), dequantised
        into the device arena `stage` first (qsa_sparse_prefill_chunk_fp8kv)."""
        qb.qsa_sparse_prefill_chunk_fp8kv(self.cfg, q, self.p0, kv8, self.blocks, self.count, self.interval,
                                          self.out, self.lse, self.ws, stage, stream)

    def run(self, q_idx, q, k_cache, v_cache, pooled, stream=None):
        """The chunk's path after pooling: score -> top-k (fused when the chunk has a full
        query tile) -> interval-walk attention."""
        if self.fused_select:
            self.select(q_idx, pooled, stream)
        else:
            self.score(q_idx, pooled, stream)
            self.topk(stream)
        self.attend(q, k_cache, v_cache, stream=stream)

    def device_status(self, stream=None):
        return qb.qsa_read_device_status(self.ws, stream)


def _workspace(nbytes: int, device):
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + nbytes]
    qb.qsa_workspace_init(ws)
    return ws


def _on_stream(stream):
    """The stream of a call (None, a torch stream or a cudaStream_t) as torch's current one."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream())


class PagedCache:
    """K/V of every layer in one pool of pages, and the sequences that share it: row r of `table` lists the
    pages of sequence r, `seq_len[r]` its tokens and `ref[p]` the rows that name page p.

    A decode step is ``extend`` (room for the new tokens of the rows in use), then per layer ``append`` and
    ``attend``; ``fork`` starts rows, lets them continue other rows (beams, shared prompts) or gives their pages
    back, and ``compact`` moves the live pages to the front of the pool. A row that finds no page left becomes empty,
    which ``status`` tells. Nothing else here synchronises. ``fork`` (``extend`` with it) and ``compact`` write
    beside what they read and then change over: a captured CUDA graph holds an even number of each."""

    def __init__(self, n_layers: int, n_pages: int, page_size: int, n_rows: int, max_pages: int, n_q_heads: int,
                 n_kv_heads: int, head_dim: int = 256, fp8: bool = False, softmax_scale: float = 0.0, window: int = 0,
                 device="cuda"):
        self.cfg = qb.make_paged_config(n_q_heads, n_kv_heads, head_dim, page_size, softmax_scale, window)
        self.fp8, self.device, self.n_rows = fp8, device, n_rows
        shape = (n_layers, n_pages, page_size, n_kv_heads)
        if fp8:
            codes = dict(dtype=torch.uint8, device=device)
            scales = dict(dtype=torch.float32, device=device)
            self.planes = [torch.zeros(*shape, head_dim, **codes), torch.zeros(*shape, head_dim // 128, **scales),
                           torch.zeros(*shape, head_dim, **codes), torch.zeros(*shape, head_dim // 128, **scales)]
        else:
            self.planes = [torch.zeros(*shape, head_dim, dtype=torch.bfloat16, device=device) for _ in range(2)]
        i32 = dict(dtype=torch.int32, device=device)
        # the page calls write new bookkeeping beside the old: two of each, in turn
        self._tables = [torch.full((n_rows, max_pages), -1, **i32) for _ in range(2)]
        self._lens = [torch.zeros(n_rows, **i32) for _ in range(2)]
        self._refs = [torch.zeros(n_pages, **i32) for _ in range(2)]
        self._now, self._ref_now = 0, 0
        self._rows = torch.arange(n_rows, **i32)
        self._one = torch.zeros(n_rows, **i32)        # extend's: 1 for each row that holds tokens
        self.ws = qb.paged_workspace(self.cfg, device)
        self.pages_ws = qb.pages_workspace(n_rows, n_pages, device)

    @property
    def table(self):
        return self._tables[self._now]

    @property
    def seq_len(self):
        return self._lens[self._now]

    @property
    def ref(self):
        return self._refs[self._ref_now]

    def fork(self, parent, add, stream=None):
        """Row i continues row parent[i] (-1: starts empty) with room for add[i] more tokens (qsa_fork_pages)."""
        new, new_ref = 1 - self._now, 1 - self._ref_now
        qb.qsa_fork_pages(self.cfg.page_size, parent, add, self.table, self.seq_len, self.ref, self._tables[new],
                          self._lens[new], self._refs[new_ref], self.planes, self.pages_ws, stream)
        self._now, self._ref_now = new, new_ref

    def extend(self, add=None, stream=None):
        """Room for add[i] more tokens in row i (None: one in each row that holds tokens, none in the empty ones)."""
        if add is None:
            with _on_stream(stream):
                add = torch.clamp(self.seq_len, 0, 1, out=self._one)
        self.fork(self._rows, add, stream)

    def compact(self, stream=None):
        new_ref = 1 - self._ref_now
        qb.qsa_compact_pages(self.cfg.page_size, self.table, self.seq_len, self.ref, self.table, self._refs[new_ref],
                             self.planes, self.pages_ws, stream)
        self._ref_now = new_ref

    def append(self, layer: int, rope, q, k, v, pos, seq=None, q_out=None, stream=None):
        """Store k (turned) and v at position pos[n] of row seq[n] (None: row n) of a layer; q turned into q_out."""
        planes = [p[layer] for p in self.planes]
        if self.fp8:
            qb.qsa_rope_append_fp8kv(self.cfg, rope, q, k, v, pos, seq, q_out, planes, self.table, self.ws, stream)
        else:
            qb.qsa_rope_append(self.cfg, rope, q, k, v, pos, seq, q_out, *planes, self.table, self.ws, stream)

    def attend(self, layer: int, q, out, lse=None, stream=None):
        """Attention of each row's newest token over the row's tokens of a layer."""
        planes = [p[layer] for p in self.planes]
        if self.fp8:
            qb.qsa_paged_decode_fp8kv(self.cfg, q, planes, self.table, self.seq_len, out, lse, self.ws, stream)
        else:
            qb.qsa_paged_decode(self.cfg, q, *planes, self.table, self.seq_len, out, lse, self.ws, stream)

    def status(self, stream=None):
        """(status, detail) of the attention and append calls, then of the page calls."""
        return qb.qsa_read_device_status(self.ws, stream), qb.qsa_read_device_status(self.pages_ws, stream)
