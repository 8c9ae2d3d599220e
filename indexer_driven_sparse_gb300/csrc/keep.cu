// Which cached tokens stay: qsa_accept_drafts[_weights] (the accepted path of a tree of drafted tokens) and qsa_evict_tokens
// (the heaviest tokens by accumulated weight). Both cut rows to a new length, move some of the kept tokens into earlier places in
// every plane, and give back the pages that empty.
#include "paged.cuh"

#include <algorithm>

namespace qsa {

namespace {

constexpr int kKeepThreads = 256;
constexpr int kSelectThreads = 512, kSelectCluster = 8;
constexpr int kSmallThreads = 1024, kSmallKeys = 16;  // rows of up to 16,384 places: one CTA, 16 keys in registers a thread
constexpr int kDigit = 11, kBins = 1 << kDigit;      // of the radix selection: 11, 11 and 10 bits of a key
constexpr uint32_t kAlways = 0xFFFFFFFFu;            // key of a token that is always kept

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct RowCut {
    int32_t len, moves;     // the new length (-1: the row is left as it is), tokens that move
};

struct KeepScratch {
    RowCut *cut;            // [n_rows]
    int2 *holes, *fillers;  // [n_rows][half]: (place, slot) of the places to fill, and of the tokens to move, the last first
    uint32_t *keys;         // [n_rows][tokens]
    int64_t half;
};

KeepScratch keep_scratch(char *w, int n_rows, int64_t tokens) {
    KeepScratch s;
    s.half = tokens / 2 + 1;                         // a moved token fills the place of a dropped one
    s.cut = reinterpret_cast<RowCut *>(w);
    w += up256(sizeof(RowCut) * (size_t)n_rows);
    s.holes = reinterpret_cast<int2 *>(w);
    w += up256(sizeof(int2) * (size_t)n_rows * s.half);
    s.fillers = reinterpret_cast<int2 *>(w);
    w += up256(sizeof(int2) * (size_t)n_rows * s.half);
    s.keys = reinterpret_cast<uint32_t *>(w);
    return s;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The word at p's address in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_word(const uint32_t *p, uint32_t rank) {
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return tokens / page_size + (tokens % page_size != 0);
}

// A place's slot, -1 where its page is out of range.
__device__ __forceinline__ int slot_of(const KeepArgs &a, const int32_t *row, int place) {
    const int e = a.page_shift >= 0 ? place >> a.page_shift : place / a.page_size;
    const int page = row[e];
    return (uint32_t)page < (uint32_t)a.n_pages ? page * a.page_size + (place - e * a.page_size) : -1;
}

// Row r's part of table_out, and the references of the pages it gives back, by threads first, first + step, ...
__device__ __forceinline__ void release(const KeepArgs &a, int r, int old_len, int new_len, int64_t first, int64_t step) {
    const int64_t kept = pages_of(new_len, a.page_size), held = pages_of(old_len, a.page_size);
    const int32_t *from = a.table + r * a.ld;
    int32_t *to = a.table_out + r * a.ld;
    for (int64_t j = first; j < a.ld; j += step) {
        const int e = from[j];
        if (j >= kept && j < held) {
            if ((uint32_t)e < (uint32_t)a.n_pages)
                atomicSub(a.ref_out + e, 1);
            else
                record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereKeep, r);
        }
        to[j] = j < kept ? e : -1;
    }
}

template <typename W>
__device__ __forceinline__ W *token_word(char *base, int64_t stride, int plane, int slot, int64_t bytes, int word) {
    return reinterpret_cast<W *>(base + plane * stride + slot * bytes) + word;
}

// ---------------------------------------------------------------------------- accepted drafts
__global__ void __launch_bounds__(kKeepThreads) copy_refs_kernel(const int32_t *ref, int32_t *ref_out, int n_pages) {
    let_next_begin();
    wait_for_previous();
    for (int64_t p = (int64_t)blockIdx.x * kKeepThreads + threadIdx.x; p < n_pages; p += (int64_t)gridDim.x * kKeepThreads)
        ref_out[p] = ref[p];
}

// The accepted path's words in one plane: token k of the path moves from place base + node[k] to base + k. node[k] >= k, ascending,
// so a thread that walks k upwards reads every place before it writes there; eight at a time, loads first.
template <typename W>
__device__ __forceinline__ void move_path(const PlaneGroup &g, int page_size, const int *from, const int *to, int n, int first,
                                          int step) {
    const int64_t bytes = g.page_bytes / page_size;
    const int words = (int)(bytes / (int64_t)sizeof(W));
    for (int64_t i = first; i < (int64_t)words * g.n_planes; i += step) {
        const int plane = (int)(i / words), w = (int)(i - (int64_t)plane * words);
        for (int k0 = 0; k0 < n; k0 += 8) {
            W v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k0 + u < n && from[k0 + u] >= 0) v[u] = *token_word<W>(g.src, g.src_stride, plane, from[k0 + u], bytes, w);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k0 + u < n && from[k0 + u] >= 0) *token_word<W>(g.src, g.src_stride, plane, to[k0 + u], bytes, w) = v[u];
        }
    }
}

// CTA (row, part): the row's accepted path, then its share of the planes' words; part 0 also does the bookkeeping.
__global__ void __launch_bounds__(kKeepThreads) accept_kernel(KeepArgs a, AcceptArgs d, PlaneGroups pg, int parts) {
    __shared__ int parent[QSA_MAX_DRAFT], node[QSA_MAX_DRAFT], from[QSA_MAX_DRAFT], to[QSA_MAX_DRAFT];
    __shared__ int found[2];                         // the path's length (-1: the row is left as it is), moves
    let_next_begin();
    wait_for_previous();
    const int r = blockIdx.x / parts, part = blockIdx.x % parts, tid = threadIdx.x;
    const int len = a.seq_len[r], off = d.draft_off[r], T = d.draft_off[r + 1] - off, last = d.accepted[r];
    const int32_t *row = a.table + r * a.ld;
    const bool ok = len >= 0 && len <= a.ld * a.page_size && off >= 0 && T >= 0 && T <= QSA_MAX_DRAFT && (int64_t)off + T <= d.N &&
                    T <= len && last >= -1 && last < T;
    const int mine = ok && tid < T ? d.parent[off + tid] : -1;
    if (ok && tid < T) parent[tid] = mine;
    const bool lost = __syncthreads_or(ok && tid < T && (mine < -1 || mine >= tid)) != 0;     // on the path or not
    if (tid == 0) {
        int n = ok && !lost ? 0 : -1;
        if (n == 0)
            for (int i = last; i >= 0; i = parent[i]) node[n++] = i;      // upwards; a parent is below its child, so this ends
        found[0] = n;
        found[1] = 0;
    }
    __syncthreads();
    const int base = len - T;
    if (tid < 32) {                                  // the moves, in order; a token already in place stays
        const int n = found[0];
        bool shared = false;                         // a move into a page that others read too
        for (int k0 = 0; k0 < n; k0 += 32) {
            const int k = k0 + tid, i = k < n ? node[n - 1 - k] : 0;
            const bool moves = k < n && i != k;
            const uint32_t all = __ballot_sync(0xffffffffu, moves);
            const int at = found[1] + __popc(all & ((1u << tid) - 1u));
            __syncwarp();
            if (moves) {
                const int s = slot_of(a, row, base + i), t = slot_of(a, row, base + k);
                if (part == 0 && (s < 0 || t < 0)) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereKeep, r);
                shared |= t >= 0 && a.ref[a.page_shift >= 0 ? t >> a.page_shift : t / a.page_size] > 1;
                from[at] = t < 0 ? -1 : s;
                to[at] = t;
            }
            if (tid == 0) found[1] += __popc(all);
            __syncwarp();
        }
        shared = __any_sync(0xffffffffu, shared);
        if (tid == 0 && shared) found[0] = -1;
        if (tid == 0 && part == 0 && found[0] < 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereKeep, r);
    }
    __syncthreads();
    const int n = found[0], new_len = n < 0 ? len : base + n;
    if (part == 0) {
        if (tid == 0) a.seq_len_out[r] = new_len;
        if (n < 0) {
            for (int64_t j = tid; j < a.ld; j += kKeepThreads) a.table_out[r * a.ld + j] = row[j];
        } else if (d.positions && tid < 32) {        // in batches of a warp, read before they are written
            int32_t *pos = d.positions + r * d.positions_ld;
            float *w = d.weights ? d.weights + r * d.positions_ld : nullptr;
            for (int k0 = 0; k0 < n; k0 += 32) {
                const int k = k0 + tid, src = k < n ? base + node[n - 1 - k] : 0;
                const bool some = k < n && src < d.positions_ld;
                const int v = some ? pos[src] : 0;
                const float x = some && w ? w[src] : 0.f;
                __syncwarp();
                if (some) {
                    pos[base + k] = v;
                    if (w) w[base + k] = x;
                }
                __syncwarp();
            }
            if (w)                                   // a later token at a dropped one's place starts with nothing
                for (int64_t j = new_len + tid; j < min((int64_t)len, d.positions_ld); j += 32) pos[j] = -1, w[j] = 0.f;
        }
    }
    if (n < 0) return;
    const int moves = found[1];
    if (moves > 0)
        for (int gi = 0; gi < pg.n; ++gi) {
            const int first = part * kKeepThreads + tid, step = parts * kKeepThreads;
            if (pg.g[gi].wide)
                move_path<uint4>(pg.g[gi], a.page_size, from, to, moves, first, step);
            else
                move_path<uint32_t>(pg.g[gi], a.page_size, from, to, moves, first, step);
        }
    if (part == 0) release(a, r, len, new_len, tid, kKeepThreads);
}

// ---------------------------------------------------------------------------- eviction
// fp32 weights as keys whose unsigned order is theirs; -0 as 0, a NaN below everything.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (isnan(w)) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the CTA of two counts; every thread gets both. sh: 2 words for each warp.
__device__ __forceinline__ uint2 block_sum2(uint32_t x, uint32_t y, uint32_t *sh) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[2 * warp] = x, sh[2 * warp + 1] = y;
    __syncthreads();
    uint2 t = make_uint2(0, 0);
#pragma unroll
    for (int w = 0; w < kSelectThreads / 32; ++w) t.x += sh[2 * w], t.y += sh[2 * w + 1];
    return t;
}

// Sums over the cluster of words x[0], x[1] of each CTA's shared memory; before: of the CTAs with a lower rank.
__device__ __forceinline__ uint2 cluster_sum2(const uint32_t *x, uint32_t rank, uint2 &before) {
    uint2 t = make_uint2(0, 0);
    before = t;
#pragma unroll
    for (uint32_t c = 0; c < kSelectCluster; ++c) {
        if (c == rank) before = t;
        t.x += cluster_word(x, c), t.y += cluster_word(x + 1, c);
    }
    return t;
}

// A cluster of CTAs settles one row: the keys of its tokens, the K-th largest by radix selection (11, 11 and 10 bits, each a
// pass over the keys and a cluster barrier), equal keys by place, then the list of holes and of tokens to move.
__global__ void __cluster_dims__(kSelectCluster, 1, 1) __launch_bounds__(kSelectThreads)
    evict_select_kernel(KeepArgs a, EvictArgs e, KeepScratch s) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t sums[2 * kSelectThreads / 32];
    __shared__ uint32_t mine[4];                     // this CTA's: highest position, protected; then larger, equal keys
    __shared__ uint32_t pick[2];                     // the chosen bin and the rank inside it
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int r = blockIdx.x / kSelectCluster;
    wait_for_previous();
    for (int64_t p = (int64_t)blockIdx.x * kSelectThreads + tid; p < a.n_pages; p += (int64_t)gridDim.x * kSelectThreads)
        a.ref_out[p] = a.ref[p];
    const int len = a.seq_len[r];
    const bool ok = len >= 0 && len <= a.ld * a.page_size && len <= e.tokens_ld;
    const int64_t row_at = r * e.tokens_ld;
    const float *w = e.weights + row_at;
    const int32_t *pos = e.positions + row_at;
    float *w_out = e.weights_out + row_at;
    int32_t *pos_out = e.positions_out + row_at;
    const int64_t all = rank * kSelectThreads + tid, all_step = kSelectCluster * kSelectThreads;
    if (!ok || e.budget[r] < 0 || e.budget[r] >= len) {      // nothing to drop
        for (int64_t j = all; j < e.tokens_ld; j += all_step) {
            const bool in = !ok || j < len;
            w_out[j] = in ? w[j] : 0.f;
            pos_out[j] = in ? pos[j] : -1;
        }
        if (all == 0) {
            if (!ok) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereKeep, r);
            s.cut[r] = {ok ? len : -1, 0};
            a.seq_len_out[r] = len;
        }
        return;                                      // the whole cluster
    }
    const int32_t *row = a.table + r * a.ld;
    uint32_t *keys = s.keys + row_at;
    // this CTA's places, unsigned: a step behind the last place of a row may pass 2^31
    const uint32_t share = ((uint32_t)len + kSelectCluster - 1) / kSelectCluster;
    const uint32_t lo = min(rank * share, (uint32_t)len), hi = min(lo + share, (uint32_t)len);

    int top = INT32_MIN;
    for (uint32_t j = lo + tid; j < hi; j += kSelectThreads) top = max(top, pos[j]);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) sums[warp] = (uint32_t)top;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kSelectThreads / 32; ++i) top = max(top, (int)sums[i]);
        mine[0] = (uint32_t)top;
    }
    cluster_sync();
#pragma unroll
    for (uint32_t c = 0; c < kSelectCluster; ++c) top = max(top, (int)cluster_word(mine, c));

    // ---- the keys, and how many tokens are always kept
    uint32_t always = 0, bad = 0;
    for (uint32_t j = lo + tid; j < hi; j += kSelectThreads) {
        const uint32_t entry = a.page_shift >= 0 ? j >> a.page_shift : j / (uint32_t)a.page_size;
        const int page = row[entry], p = pos[j];
        const bool real = (uint32_t)page < (uint32_t)a.n_pages;
        bad |= !real;
        const bool keep = p < e.first || (int64_t)p > (int64_t)top - e.recent || (real && a.ref[page] > 1);
        keys[j] = keep ? kAlways : key_of(w[j]);
        always += keep;
    }
    if (bad) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereKeep, r);
    const uint2 own = block_sum2(always, 0, sums);
    if (tid == 0) mine[1] = own.x;
    cluster_sync();
    uint32_t P = 0;
#pragma unroll
    for (uint32_t c = 0; c < kSelectCluster; ++c) P += cluster_word(mine + 1, c);
    const int K = max(e.budget[r], (int)P);          // P <= len, budget < len
    uint32_t need = K - P;                           // tokens to keep among the others

    // ---- the need-th largest key among the others
    uint32_t key = kAlways - (need == 0 ? 0u : 1u);  // no key below kAlways is kept, or
    if (need > 0) {
        uint32_t prefix = 0, known = 0;              // the key's upper bits
        for (int step = 0; step < 3; ++step) {
            const int bits = step == 2 ? 10 : kDigit, shift = step == 0 ? 21 : step == 1 ? 10 : 0;
            for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (uint32_t j = lo + tid; j < hi; j += kSelectThreads) {
                const uint32_t k = keys[j];
                if (k != kAlways && (k & known) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
            }
            cluster_sync();
            // bins from the highest down: a thread's four, scanned over the CTA
            constexpr int per = kBins / kSelectThreads;
            uint32_t n[per], run = 0;
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const int bin = kBins - 1 - (tid * per + i);
                n[i] = 0;
#pragma unroll
                for (uint32_t c = 0; c < kSelectCluster; ++c) n[i] += cluster_word(hist + bin, c);
                run += n[i];
            }
            uint32_t upto = run;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane == 31) sums[warp] = upto;
            __syncthreads();
            for (int i = 0; i < warp; ++i) upto += sums[i];
            uint32_t before = upto - run;
#pragma unroll
            for (int i = 0; i < per; ++i) {
                if (before < need && need <= before + n[i]) pick[0] = kBins - 1 - (tid * per + i), pick[1] = need - before;
                before += n[i];
            }
            __syncthreads();
            prefix |= pick[0] << shift;
            known |= ((1u << bits) - 1u) << shift;
            need = pick[1];
            cluster_sync();                          // before hist is cleared again
        }
        key = prefix;
    }

    // ---- keys above and equal, in this CTA and in those before it
    uint32_t above = 0, equal = 0;
    for (uint32_t j = lo + tid; j < hi; j += kSelectThreads) {
        const uint32_t k = keys[j];
        above += k > key || k == kAlways;
        equal += k == key && k != kAlways;
    }
    const uint2 sum = block_sum2(above, equal, sums);
    if (tid == 0) mine[2] = sum.x, mine[3] = sum.y;
    cluster_sync();
    uint2 passed;
    cluster_sum2(mine + 2, rank, passed);
    // tokens kept before place j: keys above + min(need, equal keys); a hole's number is j less those, the filler kept
    // as the x-th of all K has number K - 1 - x from the last
    for (uint32_t j0 = lo; j0 < hi; j0 += kSelectThreads) {
        const bool in = j0 + tid < hi;
        const int j = in ? (int)(j0 + tid) : 0;
        const uint32_t k = in ? keys[j] : 0u;
        const bool over = in && (k > key || k == kAlways), same = in && k == key && k != kAlways;
        const uint32_t overs = __ballot_sync(0xffffffffu, over), sames = __ballot_sync(0xffffffffu, same);
        __syncthreads();
        if (lane == 0) sums[2 * warp] = __popc(overs), sums[2 * warp + 1] = __popc(sames);
        __syncthreads();
        uint2 at = passed;
#pragma unroll
        for (int i = 0; i < kSelectThreads / 32; ++i) {
            if (i < warp) at.x += sums[2 * i], at.y += sums[2 * i + 1];
            passed.x += sums[2 * i], passed.y += sums[2 * i + 1];
        }
        at.x += __popc(overs & ((1u << lane) - 1u));
        at.y += __popc(sames & ((1u << lane) - 1u));
        if (in) {
            const int before = (int)(at.x + min(at.y, need));
            const bool kept = over || (same && at.y < need);
            const int64_t list = r * s.half;
            if (j < K && kept) w_out[j] = w[j], pos_out[j] = pos[j];
            if (j < K && !kept) s.holes[list + j - before] = make_int2(j, slot_of(a, row, j));
            if (j >= K) {
                w_out[j] = 0.f, pos_out[j] = -1;
                if (kept) s.fillers[list + K - 1 - before] = make_int2(j, slot_of(a, row, j));
            }
            if (j == K - 1) s.cut[r] = {K, K - before - (int)kept};
        }
    }
    for (int64_t j = len + all; j < e.tokens_ld; j += all_step) w_out[j] = 0.f, pos_out[j] = -1;
    if (all == 0) {
        a.seq_len_out[r] = K;
        if (K == 0) s.cut[r] = {0, 0};
    }
    cluster_sync();                                  // no CTA's shared memory goes while another reads it
}

// Rows of at most kSmallThreads kSmallKeys places: one CTA for a row, its keys in registers, so that each pass of the selection
// costs two barriers and no memory. Key i of thread x is that of place 1,024 i + x. 32 rows of 4,080 tokens: 20 us a call, the
// moves among them, with the cluster's kernel 86; 16 rows of 14,000: 81 and 132. The choice goes by the table's room, which the
// host knows, and the limit is what the registers hold: in tables of 32,768 or 131,072 places the same rows take the cluster's
// kernel (with the L2 flushed 105 to 107 us against 29, and 142 to 144 against 91 in tables of 16,384).
__global__ void __launch_bounds__(kSmallThreads) evict_small_kernel(KeepArgs a, EvictArgs e, KeepScratch s) {
    constexpr int W = kSmallThreads / 32;
    __shared__ uint32_t hist[kBins];
    __shared__ uint2 counts[kSmallKeys * W];         // keys above and equal of each warp's 32 places, then those before them
    __shared__ uint2 sums[W];
    __shared__ int tops[W];
    __shared__ uint32_t pick[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x;
    wait_for_previous();
    for (int64_t p = (int64_t)r * kSmallThreads + tid; p < a.n_pages; p += (int64_t)gridDim.x * kSmallThreads) a.ref_out[p] = a.ref[p];
    const int len = a.seq_len[r];
    const bool ok = len >= 0 && len <= a.ld * a.page_size && len <= e.tokens_ld;
    const int64_t row_at = r * e.tokens_ld;
    const float *w = e.weights + row_at;
    const int32_t *pos = e.positions + row_at;
    float *w_out = e.weights_out + row_at;
    int32_t *pos_out = e.positions_out + row_at;
    if (!ok || e.budget[r] < 0 || e.budget[r] >= len) {      // nothing to drop
        for (int64_t j = tid; j < e.tokens_ld; j += kSmallThreads) {
            const bool in = !ok || j < len;
            w_out[j] = in ? w[j] : 0.f;
            pos_out[j] = in ? pos[j] : -1;
        }
        if (tid == 0) {
            if (!ok) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereKeep, r);
            s.cut[r] = {ok ? len : -1, 0};
            a.seq_len_out[r] = len;
        }
        return;
    }
    const int32_t *row = a.table + r * a.ld;
    int p[kSmallKeys], top = INT32_MIN;
#pragma unroll
    for (int i = 0; i < kSmallKeys; ++i) {
        const int j = i * kSmallThreads + tid;
        p[i] = j < len ? pos[j] : INT32_MIN;
        top = max(top, p[i]);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) tops[warp] = top;
    uint32_t keys[kSmallKeys], shared = 0, bad = 0;  // shared: a bit for each key
#pragma unroll
    for (int i = 0; i < kSmallKeys; ++i) {
        const int j = i * kSmallThreads + tid;
        keys[i] = 0;
        if (j < len) {
            const int page = row[a.page_shift >= 0 ? j >> a.page_shift : j / a.page_size];
            const bool real = (uint32_t)page < (uint32_t)a.n_pages;
            bad |= !real;
            if (real && a.ref[page] > 1) shared |= 1u << i;
            keys[i] = key_of(w[j]);
        }
    }
    if (bad) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereKeep, r);
    for (int i = tid; i < kBins; i += kSmallThreads) hist[i] = 0;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, tops[lane]);
    uint32_t always = 0;
#pragma unroll
    for (int i = 0; i < kSmallKeys; ++i)
        if (i * kSmallThreads + tid < len && (p[i] < e.first || (int64_t)p[i] > (int64_t)top - e.recent || (shared >> i & 1u)))
            keys[i] = kAlways, ++always;
    always = __reduce_add_sync(0xffffffffu, always);
    if (lane == 0) sums[warp].x = always;
    __syncthreads();
    const uint32_t P = __reduce_add_sync(0xffffffffu, sums[lane].x);
    const int K = max(e.budget[r], (int)P);          // P <= len, budget < len
    uint32_t need = K - P, key = kAlways;            // tokens to keep among the others, the last one's key
    if (need > 0) {
        uint32_t prefix = 0, known = 0;              // the key's upper bits
#pragma unroll 1
        for (int step = 0; step < 3; ++step) {
            const int bits = step == 2 ? 10 : kDigit, shift = step == 0 ? 21 : step == 1 ? 10 : 0;
#pragma unroll
            for (int i = 0; i < kSmallKeys; ++i)
                if (i * kSmallThreads + tid < len && keys[i] != kAlways && (keys[i] & known) == prefix)
                    atomicAdd(&hist[(keys[i] >> shift) & ((1u << bits) - 1u)], 1u);
            __syncthreads();
            // bins from the highest down, two each thread
            const uint32_t n0 = hist[kBins - 1 - 2 * tid], n1 = hist[kBins - 2 - 2 * tid];
            uint32_t upto = n0 + n1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane == 31) sums[warp].y = upto;
            hist[kBins - 1 - 2 * tid] = hist[kBins - 2 - 2 * tid] = 0;      // its own, for the next pass
            __syncthreads();
            uint32_t before = upto - n0 - n1 + __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane].y : 0u);
            if (before < need && need <= before + n0) pick[0] = kBins - 1 - 2 * tid, pick[1] = need - before;
            before += n0;
            if (before < need && need <= before + n1) pick[0] = kBins - 2 - 2 * tid, pick[1] = need - before;
            __syncthreads();
            prefix |= pick[0] << shift;
            known |= ((1u << bits) - 1u) << shift;
            need = pick[1];
        }
        key = prefix;
    }
    // ---- keys above and equal before each warp's 32 places of each round
    uint32_t overs[kSmallKeys], sames[kSmallKeys];
#pragma unroll
    for (int i = 0; i < kSmallKeys; ++i) {
        const bool in = i * kSmallThreads + tid < len;
        overs[i] = __ballot_sync(0xffffffffu, in && (keys[i] > key || keys[i] == kAlways));
        sames[i] = __ballot_sync(0xffffffffu, in && keys[i] == key && keys[i] != kAlways);
        if (lane == 0) counts[i * W + warp] = make_uint2(__popc(overs[i]), __popc(sames[i]));
    }
    __syncthreads();
    uint2 mine = make_uint2(0, 0), run;
    if (tid < kSmallKeys * W) mine = counts[tid];
    run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, run.x, o), y = __shfl_up_sync(0xffffffffu, run.y, o);
        if (lane >= o) run.x += x, run.y += y;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    const uint2 part = lane < warp ? sums[lane] : make_uint2(0, 0);
    run.x += __reduce_add_sync(0xffffffffu, part.x) - mine.x;
    run.y += __reduce_add_sync(0xffffffffu, part.y) - mine.y;
    if (tid < kSmallKeys * W) counts[tid] = run;
    __syncthreads();
    const int64_t list = r * s.half;
#pragma unroll
    for (int i = 0; i < kSmallKeys; ++i) {
        const int j = i * kSmallThreads + tid;
        if (j >= len) break;
        const uint2 at = counts[i * W + warp];
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t equal = at.y + __popc(sames[i] & below);
        const int before = (int)(at.x + __popc(overs[i] & below) + min(equal, need));
        const bool kept = (overs[i] >> lane & 1u) || ((sames[i] >> lane & 1u) && equal < need);
        if (j < K && kept) w_out[j] = w[j], pos_out[j] = p[i];
        if (j < K && !kept) s.holes[list + j - before] = make_int2(j, slot_of(a, row, j));
        if (j >= K) {
            w_out[j] = 0.f, pos_out[j] = -1;
            if (kept) s.fillers[list + K - 1 - before] = make_int2(j, slot_of(a, row, j));
        }
        if (j == K - 1) s.cut[r] = {K, K - before - (int)kept};
    }
    for (int64_t j = len + tid; j < e.tokens_ld; j += kSmallThreads) w_out[j] = 0.f, pos_out[j] = -1;
    if (tid == 0) {
        a.seq_len_out[r] = K;
        if (K == 0) s.cut[r] = {0, 0};
    }
}

template <typename W>
__device__ __forceinline__ void move_tokens(const PlaneGroup &g, int page_size, const int2 *holes, const int2 *fillers, int n,
                                            int warp, int warps) {
    const int64_t bytes = g.page_bytes / page_size;
    const int words = (int)(bytes / (int64_t)sizeof(W)), lane = threadIdx.x & 31;
    int group = 32;                                  // lanes for a token
    while (group > 1 && group / 2 >= words) group /= 2;
    const int each = 32 / group, mine = lane / group, first = lane % group;
    // (plane, move) pairs, so that few moves in many planes are copied at once too
    const int64_t units = (int64_t)g.n_planes * n;
    for (int64_t u = (int64_t)warp * each + mine; u < units; u += (int64_t)warps * each) {
        const int plane = units >> 31 ? (int)(u / n) : (int)((uint32_t)u / (uint32_t)n), k = (int)(u - (int64_t)plane * n);
        const int to = holes[k].y, from = fillers[n - 1 - k].y;
        if (to < 0 || from < 0) continue;
        for (int w = first; w < words; w += group)
            *token_word<W>(g.src, g.src_stride, plane, to, bytes, w) = *token_word<W>(g.src, g.src_stride, plane, from, bytes, w);
    }
}

// CTA (row, part): the row's moves, which are independent of each other (tokens behind the new length into places before it).
__global__ void __launch_bounds__(kKeepThreads) evict_move_kernel(KeepArgs a, EvictArgs e, KeepScratch s, PlaneGroups pg, int parts) {
    let_next_begin();
    wait_for_previous();
    const int r = blockIdx.x / parts, part = blockIdx.x % parts, tid = threadIdx.x;
    const RowCut cut = s.cut[r];
    const int64_t first = (int64_t)part * kKeepThreads + tid, step = (int64_t)parts * kKeepThreads;
    if (cut.len < 0) {
        for (int64_t j = first; j < a.ld; j += step) a.table_out[r * a.ld + j] = a.table[r * a.ld + j];
        return;
    }
    const int2 *holes = s.holes + r * s.half, *fillers = s.fillers + r * s.half;
    const int warp = (part * kKeepThreads + tid) >> 5, warps = parts * (kKeepThreads / 32);
    for (int gi = 0; gi < pg.n; ++gi) {
        if (pg.g[gi].wide)
            move_tokens<uint4>(pg.g[gi], a.page_size, holes, fillers, cut.moves, warp, warps);
        else
            move_tokens<uint32_t>(pg.g[gi], a.page_size, holes, fillers, cut.moves, warp, warps);
    }
    for (int64_t k = first; k < cut.moves; k += step) {
        const int to = holes[k].x, from = fillers[cut.moves - 1 - k].x;
        e.weights_out[r * e.tokens_ld + to] = e.weights[r * e.tokens_ld + from];
        e.positions_out[r * e.tokens_ld + to] = e.positions[r * e.tokens_ld + from];
    }
    release(a, r, a.seq_len[r], cut.len, first, step);
}

// CTAs for each row of the moving kernels: eight for each of 152 SMs in all.
int parts_of(int n_rows) { return std::max(1, 152 * 8 / n_rows); }

}  // namespace

size_t keep_scratch_bytes(int n_rows, int64_t tokens) {
    const size_t half = (size_t)(tokens / 2 + 1);
    return up256(sizeof(RowCut) * (size_t)n_rows) + 2 * up256(sizeof(int2) * (size_t)n_rows * half) +
           sizeof(uint32_t) * (size_t)n_rows * (size_t)tokens;
}

cudaError_t launch_accept_drafts(const KeepArgs &a, const AcceptArgs &d, const PlaneGroups &p, cudaStream_t st) {
    const int ctas = (int)std::min<int64_t>(((int64_t)a.n_pages + kKeepThreads - 1) / kKeepThreads, 152 * 8);
    if (ctas > 0) {
        const cudaError_t e = launch_dependent(copy_refs_kernel, dim3(ctas), kKeepThreads, 0, st, a.ref, a.ref_out, a.n_pages);
        if (e != cudaSuccess || a.n_rows == 0) return e;
    }
    if (a.n_rows == 0) return cudaSuccess;
    // one thread for each word of a token in every plane, if the GPU has them
    int64_t words = 0;
    for (int i = 0; i < p.n; ++i)
        words = std::max(words, p.g[i].page_bytes / a.page_size / (p.g[i].wide ? 16 : 4) * p.g[i].n_planes);
    const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(parts_of(a.n_rows), (words + kKeepThreads - 1) / kKeepThreads));
    return launch_dependent(accept_kernel, dim3((unsigned)a.n_rows * parts), kKeepThreads, 0, st, a, d, p, parts);
}

cudaError_t launch_evict_tokens(const KeepArgs &a, const EvictArgs &e, const PlaneGroups &p, cudaStream_t st) {
    if (a.n_rows == 0) {
        const int ctas = (int)std::min<int64_t>(((int64_t)a.n_pages + kKeepThreads - 1) / kKeepThreads, 152 * 8);
        return ctas > 0 ? launch_dependent(copy_refs_kernel, dim3(ctas), kKeepThreads, 0, st, a.ref, a.ref_out, a.n_pages)
                        : cudaSuccess;
    }
    const KeepScratch s = keep_scratch(a.scratch, a.n_rows, e.tokens_ld);
    const cudaError_t err =
        e.tokens_ld <= kSmallThreads * kSmallKeys
            ? launch_dependent(evict_small_kernel, dim3((unsigned)a.n_rows), kSmallThreads, 0, st, a, e, s)
            : launch_dependent(evict_select_kernel, dim3((unsigned)a.n_rows * kSelectCluster), kSelectThreads, 0, st, a, e, s);
    if (err != cudaSuccess) return err;
    const int parts = parts_of(a.n_rows);
    return launch_dependent(evict_move_kernel, dim3((unsigned)a.n_rows * parts), kKeepThreads, 0, st, a, e, s, p, parts);
}

}  // namespace qsa
