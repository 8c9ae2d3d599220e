// Bookkeeping and copying of a paged cache's pages: fork / extend / free (qsa_fork_pages), compaction
// (qsa_compact_pages) and plain copies (qsa_copy_pages).
//
// The whole numbers are settled by one cluster of 8 CTAs: each thread counts the free (or live) pages of its run of
// ref, one scan numbers the runs inside a CTA, and one cluster barrier makes the CTAs' counts known; meanwhile CTA 0
// plans the rows of a fork. That kernel is a chain of dependent loads and is bound by their latency: it has one pass
// before the barrier and one after it. A second kernel, launched as its dependent, writes the tables and copies
// the pages with every SM: that part is bound by HBM.
//
// Pools and tables that one CTA can plan in its shared memory (kSmallPages, kSmallRows, kSmallEntries) take a single
// kernel instead: every CTA makes the whole plan for itself from L2, so none waits for another, and goes on to its
// share of the tables and copies. The plan's time grows with the pages and the table's entries, that of two kernels hardly; the
// limits are where they meet. One kernel against two, extending every row by a token (captured, 20 in a row):
//   pages 1,024: 5.4 and 8.1 us with 1,024 entries, 8.0 and 8.2 with 8,192, 10.8 and 8.1 with 16,384 (64 or 256 rows);
//   4,096: 6.2 and 8.2, 9.0 and 8.4, 13.4 and 8.5; 8,192: 7.3 and 8.6, 10.0 and 8.8, 14.5 and 9.0; 12,288 with 1,024: 8.8 and 8.4;
//   1,024 rows of 4 entries over 4,096 pages: 9.2 and 9.3. Compaction: 600 pages 2.9 and 4.5, 8,192 5.4 either way, 16,384 9.2 and 5.5.
#include "paged.cuh"

#include <algorithm>

namespace qsa {

namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 4096;       // one warp's share of a page copy at a time: eight 16-byte words a lane, in two goes
constexpr int kSharedRows = 4096;      // per-parent words kept in shared memory up to this many rows
constexpr int kSmallThreads = 512;
constexpr int kSmallPages = 8192;      // page ids in 16 bits
constexpr int kSmallRows = 1024;
constexpr int64_t kSmallEntries = 8192;    // table entries whose references one CTA counts
constexpr int kEntriesAhead = 12;      // ... this many of each thread's loaded before the plan, as many as there are registers for

struct RowCopy {                       // new page fresh[off] becomes page src's first `used` tokens
    int32_t src, off, used;
};

// Counts at the front of the scratch area.
struct PlanHead {
    int32_t per_cta[kCluster];         // free (fork) or live (compact) pages in each CTA's share
    int32_t n_pairs, n_live;
};
static_assert(sizeof(PlanHead) <= 256, "PlanHead fits its 256 bytes");

// Scratch: head, then arrays of int32 sized by rows and pages.
struct ForkScratch {
    PlanHead *head;
    int32_t *first, *children;         // [n_in] lowest row that continues it, how many do
    int32_t *off;                      // [n_out] first of its new pages in `fresh`, -1: row failed
    int32_t *keeps;                    // [n_out] keeps the parent's last page
    int32_t *fresh;                    // [n_pages] new pages in the order they are handed out
    RowCopy *pairs;                    // [n_out]
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Inclusive sum over the CTA's threads; *total gets the whole. `sh` holds 33 words.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *sh, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    if (warp == 0) {
        T w = lane < (int)(blockDim.x >> 5) ? sh[lane] : T(0);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        sh[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v += sh[warp - 1];
    *total = sh[(blockDim.x >> 5) - 1];
    __syncthreads();                    // sh may be used again
    return v;
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return tokens / page_size + (tokens % page_size != 0);
}

// A row's plan from its parent: -1 parent is an empty start.
struct RowPlan {
    int parent, base, total, full, used, pages;
    bool ok;
};

__device__ __forceinline__ RowPlan row_plan(const ForkArgs &a, int i) {
    RowPlan p;
    p.parent = a.parent[i];
    const int add = a.add[i];
    p.ok = p.parent >= -1 && p.parent < a.n_in && add >= 0;
    p.base = 0;
    if (p.ok && p.parent >= 0) {
        p.base = a.seq_len[p.parent];
        p.ok = p.base >= 0 && pages_of(p.base, a.page_size) <= a.ld;
    }
    const int64_t total = (int64_t)p.base + add;
    p.ok = p.ok && total <= INT32_MAX && pages_of((int)total, a.page_size) <= a.ld;
    if (!p.ok) p.parent = -1, p.base = 0;
    p.total = p.ok ? (int)total : 0;
    p.full = p.base / a.page_size;
    p.used = p.base % a.page_size;
    p.pages = pages_of(p.total, a.page_size);
    return p;
}

// f(p, ref[p]) for p in [lo, hi), eight loads at a time: f may store, and the compiler keeps loads behind stores.
template <typename F>
__device__ __forceinline__ void for_refs(const int32_t *ref, int lo, int hi, F f) {
    for (int p0 = lo; p0 < hi; p0 += 8) {
        int r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p0 + i < hi) r[i] = ref[p0 + i];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p0 + i < hi) f(p0 + i, r[i]);
    }
}

// A thread's run of page ids [lo, hi) in its CTA's share.
struct Run {
    int lo, hi;
};
__device__ __forceinline__ Run run_of_thread(int n_pages) {
    const int share = (n_pages + kCluster - 1) / kCluster, per = (share + kPlanThreads - 1) / kPlanThreads;
    const int end = min(n_pages, ((int)blockIdx.x + 1) * share);
    Run r;
    r.lo = min(end, (int)blockIdx.x * share + (int)threadIdx.x * per);
    r.hi = min(end, r.lo + per);
    return r;
}

// Before the barrier: every CTA numbers its free pages and copies ref; CTA 0 plans the rows (lowest row that
// continues each parent, pages each row needs, scanned over the rows). After it: the free pages that are handed out go
// to `fresh`; CTA 0, now knowing how many there are, strikes out the rows that find none and lists the copies.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    fork_plan_kernel(ForkArgs a, ForkScratch s) {
    __shared__ long long sh[33];
    __shared__ int first_sh[kSharedRows], children_sh[kSharedRows];
    const int cta = blockIdx.x, tid = threadIdx.x;
    let_next_begin();
    wait_for_previous();
    const Run run = run_of_thread(a.n_pages);
    int free_here = 0;
    for_refs(a.ref, run.lo, run.hi, [&](int p, int r) {
        free_here += r == 0;
        a.ref_out[p] = r;
    });
    long long total;
    int rank = (int)block_scan<long long>(free_here, sh, &total) - free_here;
    if (tid == 0) s.head->per_cta[cta] = (int)total;

    // CTA 0's rows: first and children live in shared memory, or in the workspace when there are many
    int *first = a.n_in <= kSharedRows ? first_sh : s.first;
    int *children = a.n_in <= kSharedRows ? children_sh : s.children;
    RowPlan plan{};                    // of row tid, the only one of this thread up to kPlanThreads rows
    long long need = 0;
    if (cta == 0) {
        for (int p = tid; p < a.n_in; p += kPlanThreads) {
            first[p] = INT32_MAX;
            children[p] = 0;
        }
        __syncthreads();
        for (int i = tid; i < a.n_out; i += kPlanThreads) {
            const RowPlan p = row_plan(a, i);
            if (i == tid) plan = p;
            if (!p.ok) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
            if (p.parent >= 0) atomicMin(first + p.parent, i);
        }
        __syncthreads();
        for (int i0 = 0; i0 < a.n_out; i0 += kPlanThreads) {
            const int i = i0 + tid;
            long long mine = 0;
            if (i < a.n_out) {
                const RowPlan p = i == tid ? plan : row_plan(a, i);
                int keep = 0;
                if (p.used > 0) {
                    const int last = a.table[(int64_t)p.parent * a.ld + p.full];
                    const bool named = last >= 0 && last < a.n_pages;
                    if (!named) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
                    keep = named && first[p.parent] == i && a.ref[last] == 1;
                }
                s.keeps[i] = keep;
                mine = p.pages - p.full - keep;
            }
            long long sum;
            const long long upto = need + block_scan<long long>(mine, sh, &sum);
            if (i < a.n_out) s.off[i] = (int)min(upto - mine, (long long)INT32_MAX);
            need += sum;
        }
    }
    cluster_sync();
    long long n_free = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
        const int n = s.head->per_cta[c];
        rank += c < cta ? n : 0;
        n_free += n;
    }
    // every free page has a place in the order; pages behind what is handed out are written and not read
    for_refs(a.ref, run.lo, run.hi, [&](int p, int r) {
        if (r == 0) s.fresh[rank++] = p;
    });
    if (cta != 0) return;
    int n_pairs = 0;
    for (int i0 = 0; i0 < a.n_out; i0 += kPlanThreads) {
        const int i = i0 + tid;
        bool copy = false;
        RowCopy c{};
        if (i < a.n_out) {
            const RowPlan p = i == tid ? plan : row_plan(a, i);
            const int keep = s.keeps[i], off = s.off[i], mine = p.pages - p.full - keep;
            const bool failed = mine > 0 && (long long)off + mine > n_free;
            if (failed) {
                record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
                s.off[i] = -1;
            } else if (p.parent >= 0) {
                atomicAdd(children + p.parent, 1);
            }
            a.seq_len_out[i] = failed ? 0 : p.total;
            if (!failed && p.used > 0 && !keep) {
                const int last = a.table[(int64_t)p.parent * a.ld + p.full];
                c = {last, off, p.used};
                copy = last >= 0 && last < a.n_pages;
            }
        }
        long long copies;
        const long long at = block_scan<long long>(copy, sh, &copies);
        if (copy) s.pairs[n_pairs + (int)at - 1] = c;
        n_pairs += (int)copies;
    }
    if (tid == 0) s.head->n_pairs = n_pairs;
    __syncthreads();
    if (a.n_in <= kSharedRows)
        for (int p = tid; p < a.n_in; p += kPlanThreads) {
            s.first[p] = first[p];
            s.children[p] = children[p];
        }
}

// ---------------------------------------------------------------------------- copies
// A warp's number with neighbours in different CTAs, so that a little work spreads over the SMs.
__device__ __forceinline__ int warp_spread() { return (int)(threadIdx.x >> 5) * gridDim.x + blockIdx.x; }

// Words of 16 or 4 bytes of one plane's page, [begin, end) bytes, by one warp.
template <typename W>
__device__ __forceinline__ void move_words(const char *src, char *dst, int64_t begin, int64_t end) {
    constexpr int U = 4, step = 32 * (int)sizeof(W);
    for (int64_t b = begin + (threadIdx.x & 31) * (int)sizeof(W); b < end; b += U * step) {
        W v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u * step < end) v[u] = *reinterpret_cast<const W *>(src + b + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u * step < end) *reinterpret_cast<W *>(dst + b + u * step) = v[u];
    }
}

// Every plane's pages of n pairs, a warp for each kMoveBytes; pair k by `pair`, which returns the used tokens
// (0: skip).
template <int Threads, typename Pair>
__device__ __forceinline__ void move_pages(const PlaneGroups &pg, int n, int page_size, Pair pair) {
    const int warps = gridDim.x * (Threads / 32);
    for (int gi = 0; gi < pg.n; ++gi) {
        const PlaneGroup &g = pg.g[gi];
        const int64_t parts = (g.page_bytes + kMoveBytes - 1) / kMoveBytes;
        const int64_t items = parts * g.n_planes * n;
        // a CTA's warps take neighbouring parts (2.1 GB of pages: 396 us, spread 417 us); fewer parts than warps are
        // spread, from the end that has no table rows
        const int warp = items < warps ? warps - 1 - warp_spread()
                                       : (int)((blockIdx.x * Threads + threadIdx.x) >> 5);
        for (int64_t w = warp; w < items; w += warps) {
            // the part is turned by the page: a warp that met the same part of every page would copy all of the partly
            // filled ones (low parts) or none
            int64_t rest, part;
            int plane, k;
            if ((items + 13) >> 32 == 0) {         // in 32 bits: a 64-bit division takes some 100 instructions
                const uint32_t p = (uint32_t)parts, r = (uint32_t)w / p;
                rest = r;
                part = ((uint32_t)w - r * p + r % 13u) % p;
                k = r / (uint32_t)g.n_planes;
                plane = r - k * g.n_planes;
            } else {
                rest = w / parts;
                part = (w - rest * parts + rest % 13) % parts;
                k = (int)(rest / g.n_planes);
                plane = (int)(rest % g.n_planes);
            }
            int src, dst;
            const int used = pair(k, src, dst);
            if (used == 0) continue;
            const int word = g.wide ? 16 : 4;
            int64_t bytes = ((int64_t)used * g.page_bytes + page_size - 1) / page_size;
            bytes = (bytes + word - 1) / word * word;
            const int64_t begin = part * kMoveBytes, end = min(begin + kMoveBytes, bytes);
            const char *from = g.src + plane * g.src_stride + src * g.page_bytes;
            char *to = g.dst + plane * g.dst_stride + dst * g.page_bytes;
            if (g.wide)
                move_words<uint4>(from, to, begin, end);
            else
                move_words<uint32_t>(from, to, begin, end);
        }
    }
}

// The new table's rows (a warp each), the references, then the copies.
__global__ void __launch_bounds__(kMoveThreads, 4) fork_move_kernel(ForkArgs a, ForkScratch s, PlaneGroups pg) {
    let_next_begin();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kMoveThreads / 32), warp = warp_spread();
    for (int i = warp; i < a.n_out; i += warps) {
        const RowPlan p = row_plan(a, i);
        const int off = s.off[i];
        const int kept = off < 0 ? 0 : p.full + s.keeps[i], pages = off < 0 ? 0 : p.pages;
        const int32_t *from = a.table + (int64_t)max(p.parent, 0) * a.ld;
        int32_t *to = a.table_out + (int64_t)i * a.ld;
        for (int64_t j = lane; j < a.ld; j += 32) {
            int e = -1;
            if (j < kept) {
                e = from[j];
            } else if (j < pages) {
                e = s.fresh[off + (int)j - kept];
                atomicAdd(a.ref_out + e, 1);
            }
            to[j] = e;
        }
    }
    // an old row's full pages: its own entry goes, each row that continues it adds one; its last, partly
    // filled page stays only with a row that keeps it
    const int skip = a.n_out % warps;              // on from where the new rows ended
    for (int p = warp >= skip ? warp - skip : warp - skip + warps; p < a.n_in; p += warps) {
        const int len = a.seq_len[p];
        if (len <= 0 || pages_of(len, a.page_size) > a.ld) continue;
        const int full = len / a.page_size, pages = pages_of(len, a.page_size), children = s.children[p];
        const int first = s.first[p];
        const int kept = first < a.n_out && s.off[first] >= 0 ? s.keeps[first] : 0;
        for (int j = lane; j < pages; j += 32) {
            const int delta = (j < full ? children : kept) - 1;
            const int e = a.table[(int64_t)p * a.ld + j];
            if (e < 0 || e >= a.n_pages)
                record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, p);
            else if (delta != 0)
                atomicAdd(a.ref_out + e, delta);
        }
    }
    move_pages<kMoveThreads>(pg, s.head->n_pairs, a.page_size, [&](int k, int &src, int &dst) {
        const RowCopy c = s.pairs[k];
        src = c.src;
        dst = s.fresh[c.off];
        return c.used;
    });
}

// ---------------------------------------------------------------------------- compaction
struct CompactScratch {
    PlanHead *head;
    int32_t *rank;                     // [n_pages] of a page that moves: its place among them from the last, -1: free
    int32_t *movers, *holes;           // [n_pages] from the last: mover i goes to hole i
};

// With L(p) live pages below p and n_live in all, a free page p < n_live is hole number p - L(p), and the page that
// moves into the last hole is the one with L(p) = n_live - 1: numbered from the last, mover p has place
// n_live - 1 - L(p). So one pass of live counts gives both lists; M = n_live - L(n_live) pages move, and hole number h
// has place M - 1 - h, which the second kernel, knowing M, resolves.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(CompactArgs a, CompactScratch s) {
    __shared__ long long sh[33];
    const int cta = blockIdx.x, tid = threadIdx.x;
    let_next_begin();
    wait_for_previous();
    const Run run = run_of_thread(a.n_pages);
    int live = 0;
    for_refs(a.ref, run.lo, run.hi, [&](int, int r) { live += r > 0; });
    long long total;
    int below = (int)block_scan<long long>(live, sh, &total) - live;
    if (tid == 0) s.head->per_cta[cta] = (int)total;
    cluster_sync();
    int n_live = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
        const int n = s.head->per_cta[c];
        below += c < cta ? n : 0;
        n_live += n;
    }
    for_refs(a.ref, run.lo, run.hi, [&](int p, int r) {
        if (p == n_live) s.head->n_pairs = n_live - below;
        if (r > 0) {
            if (p >= n_live) {
                s.rank[p] = n_live - 1 - below;
                s.movers[n_live - 1 - below] = p;
            } else {
                s.rank[p] = 0;
                a.ref_out[p] = r;
            }
            ++below;
        } else {
            s.rank[p] = -1;
            if (p < n_live) s.holes[p - below] = p;
        }
    });
    if (cta == 0 && tid == 0) {
        s.head->n_live = n_live;
        if (n_live == a.n_pages) s.head->n_pairs = 0;
    }
}

__global__ void __launch_bounds__(kMoveThreads, 4) compact_move_kernel(CompactArgs a, CompactScratch s, PlaneGroups pg) {
    let_next_begin();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kMoveThreads / 32), warp = warp_spread();
    const int n_live = s.head->n_live, moving = s.head->n_pairs;
    for (int i = warp; i < a.n_rows; i += warps) {
        int len = a.seq_len[i];
        if (len < 0 || pages_of(len, a.page_size) > a.ld) {
            if (lane == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
            len = 0;
        }
        const int pages = pages_of(len, a.page_size);
        for (int64_t j = lane; j < a.ld; j += 32) {
            int e = -1;
            if (j < pages) {
                e = a.table[(int64_t)i * a.ld + j];
                const int rank = e >= 0 && e < a.n_pages ? s.rank[e] : -1;
                if (rank < 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
                e = rank < 0 ? -1 : e < n_live ? e : s.holes[moving - 1 - rank];
            }
            a.table_out[(int64_t)i * a.ld + j] = e;
        }
    }
    // references: a page that moves takes its count along, the rest above n_live have none
    for (int p = blockIdx.x * kMoveThreads + threadIdx.x; p < a.n_pages; p += gridDim.x * kMoveThreads) {
        if (p < n_live) continue;
        const int rank = s.rank[p];
        if (rank >= 0) a.ref_out[s.holes[moving - 1 - rank]] = a.ref[p];
        a.ref_out[p] = 0;
    }
    move_pages<kMoveThreads>(pg, moving, 1, [&](int k, int &src, int &dst) {
        src = s.movers[k];
        dst = s.holes[moving - 1 - k];
        return 1;
    });
}

__global__ void __launch_bounds__(kMoveThreads, 4)
    copy_pages_kernel(const int32_t *src_ids, const int32_t *dst_ids, int n, PlaneGroups pg, int64_t n_src, int64_t n_dst,
                      WsHeader *hdr) {
    let_next_begin();
    wait_for_previous();
    move_pages<kMoveThreads>(pg, n, 1, [&](int k, int &src, int &dst) {
        src = src_ids[k];
        dst = dst_ids[k];
        if (src < 0 || dst < 0) return 0;
        if (src >= n_src || dst >= n_dst) {
            if ((threadIdx.x & 31) == 0) record_error(hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, k);
            return 0;
        }
        return 1;
    });
}

// ---------------------------------------------------------------------------- small pools: one kernel
// Shared memory of a CTA's plan.
struct SmallFork {
    int *len, *full;                       // [n_in] tokens, full pages (-1: an impossible length)
    int *last;                             // [n_in] the last, partly filled page (-1: none)
    int *first, *children;                 // [n_in] lowest row that continues it (later: whether one keeps the last page), how many do
    int *parent, *pages, *off;             // [n_out] parent -1: starts empty; pages in all; off kKeeps: keeps the parent's last page; -1: failed
    int *delta;                            // [n_pages] ref; later, in CTA 0, with the references that come and go
    uint16_t *pairs;                       // [n_out] rows that copy a page
    uint16_t *fresh;                       // [n_pages] free pages in order
};
constexpr int kKeeps = 1 << 30;
constexpr int kFewPages = 8;
constexpr int kSmallChunks = kSmallPages / kSmallThreads, kSmallWarps = kSmallThreads / 32;
static_assert(kSmallChunks <= 32 && kSmallChunks * kSmallWarps <= kSmallThreads, "a thread's pages fit a word, the counts a scan");

// Shared memory of the arrays above, in their order (and 16 bytes), and of compact_small_kernel's.
constexpr size_t small_fork_bytes(int n_in, int n_out, int n_pages) {
    return (size_t)n_in * 20 + (size_t)n_out * 12 + (size_t)n_pages * 4 + ((size_t)n_out + n_pages + 8) * 2;
}
constexpr size_t small_compact_bytes(int n_pages) { return ((size_t)n_pages * 2 + 8) * 2; }
constexpr size_t kSmallSmem = small_fork_bytes(kSmallRows, kSmallRows, kSmallPages);    // the most that a launch asks for
static_assert(small_compact_bytes(kSmallPages) <= kSmallSmem, "one limit serves both kernels");
static_assert(2 * (kSmallSmem + kSmallThreads * 4 + 33 * 12 + 1024) <= 228 * 1024, "two CTAs, with their static arrays, on an SM");

// test(ref[p]) for the pages p = tid, tid + kSmallThreads, ... as a word; counts[t] becomes the number of pages that
// pass before chunk t / kSmallWarps of kSmallThreads pages and warp t % kSmallWarps in it, *total all that pass.
// `also(p, r)` sees every page. Ahead: the thread's first ref is `ahead`. Ends with a barrier.
template <bool Ahead, typename Test, typename Also>
__device__ __forceinline__ uint32_t small_ranks(const int32_t *ref, int n_pages, int ahead, int *counts, int *sh, int *total,
                                                Test test, Also also) {
    const int tid = threadIdx.x, warp = tid >> 5, chunks = (n_pages + kSmallThreads - 1) / kSmallThreads;
    uint32_t mine = 0;
    for (int i0 = 0; i0 < chunks; i0 += 16) {
        int r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int p = (i0 + i) * kSmallThreads + tid;
            if (Ahead && i0 == 0 && i == 0)
                r[i] = ahead;
            else if (p < n_pages)
                r[i] = ref[p];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int p = (i0 + i) * kSmallThreads + tid;
            if (i0 + i >= chunks) break;
            const bool pass = p < n_pages && test(r[i]);
            const uint32_t m = __ballot_sync(0xffffffffu, pass);
            mine |= (uint32_t)pass << (i0 + i);
            if ((tid & 31) == 0) counts[(i0 + i) * kSmallWarps + warp] = __popc(m);
            if (p < n_pages) also(p, r[i]);
        }
    }
    __syncthreads();
    const int n = tid < chunks * kSmallWarps ? counts[tid] : 0;
    const int upto = block_scan<int>(n, sh, total);
    if (tid < chunks * kSmallWarps) counts[tid] = upto - n;
    __syncthreads();
    return mine;
}

// f(p, passes, passes before p) for the same pages.
template <typename F>
__device__ __forceinline__ void for_ranks(uint32_t mine, int n_pages, const int *counts, F f) {
    const int tid = threadIdx.x, warp = tid >> 5, chunks = (n_pages + kSmallThreads - 1) / kSmallThreads;
    const uint32_t lower = (1u << (tid & 31)) - 1u;
    for (int i = 0; i < chunks; ++i) {
        const bool pass = (mine >> i) & 1u;
        const uint32_t m = __ballot_sync(0xffffffffu, pass);
        const int p = i * kSmallThreads + tid;
        if (p < n_pages) f(p, pass, counts[i * kSmallWarps + warp] + __popc(m & lower));
    }
}

// CTA 0 also writes the references: ref and what rows give up or take, summed in shared memory.
__global__ void __launch_bounds__(kSmallThreads, 2) fork_small_kernel(ForkArgs a, PlaneGroups pg) {
    extern __shared__ __align__(16) int small_smem[];
    __shared__ int counts[kSmallThreads];
    __shared__ int sh[33];
    __shared__ long long sh64[33];
    let_next_begin();
    wait_for_previous();
    const int tid = threadIdx.x, lane = tid & 31;
    const int ps = a.page_size, shift = a.page_shift;
    auto over = [&](int tokens) { return shift >= 0 ? tokens >> shift : tokens / ps; };     // whole pages
    SmallFork s;
    s.len = small_smem;
    s.full = s.len + a.n_in;
    s.last = s.full + a.n_in;
    s.first = s.last + a.n_in;
    s.children = s.first + a.n_in;
    s.parent = s.children + a.n_in;
    s.pages = s.parent + a.n_out;
    s.off = s.pages + a.n_out;
    s.delta = s.off + a.n_out;
    s.pairs = reinterpret_cast<uint16_t *>(s.delta + a.n_pages);
    s.fresh = s.pairs + a.n_out;
    const int ahead = tid < a.n_pages ? a.ref[tid] : 0;    // before the rows' dependent loads
    // CTA 0's table entries come along with the first loads
    const int ld = (int)a.ld, entries = a.n_in * ld;
    int entry[kEntriesAhead];
    if (blockIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < kEntriesAhead; ++i) {
            const int x = tid + i * kSmallThreads;
            entry[i] = x < entries ? a.table[x] : -1;
        }
    }
    for (int i = tid; i < a.n_out; i += kSmallThreads) {
        s.parent[i] = a.parent[i];
        s.pages[i] = a.add[i];
    }
    for (int p = tid; p < a.n_in; p += kSmallThreads) {
        const int len = a.seq_len[p];
        int last = -1, full = len >= 0 ? over(len) : -1;
        if (full >= 0 && full + (len != full * ps) > ld) full = -1;
        if (full >= 0 && len != full * ps) {
            last = a.table[p * ld + full];
            if (last < 0 || last >= a.n_pages) last = -1;
        }
        s.len[p] = len;
        s.full[p] = full;
        s.last[p] = last;
        s.first[p] = INT32_MAX;
        s.children[p] = 0;
    }
    int n_free;
    const uint32_t is_free = small_ranks<true>(a.ref, a.n_pages, ahead, counts, sh, &n_free, [](int r) { return r == 0; },
                                         [&](int p, int r) { s.delta[p] = r; });
    for_ranks(is_free, a.n_pages, counts, [&](int p, bool free, int rank) {
        if (free) s.fresh[rank] = (uint16_t)p;
    });
    for (int i = tid; i < a.n_out; i += kSmallThreads) {
        const int parent = s.parent[i], add = s.pages[i];
        bool ok = parent >= -1 && parent < a.n_in && add >= 0 && (parent < 0 || s.full[parent] >= 0);
        const int base = ok && parent >= 0 ? s.len[parent] : 0;
        const int64_t total = (int64_t)base + add;
        ok = ok && total <= INT32_MAX;
        int pages = ok ? over((int)total) : 0;
        pages += ok && (int)total != pages * ps;
        ok = ok && pages <= ld;
        if (!ok && blockIdx.x == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
        s.parent[i] = ok ? parent : -1;
        s.pages[i] = ok ? pages : 0;
        if (blockIdx.x == gridDim.x - 1) a.seq_len_out[i] = ok ? (int)total : 0;    // a row that fails later is emptied there
        if (ok && parent >= 0) atomicMin(s.first + parent, i);
    }
    __syncthreads();
    // pages that each row needs and the copies, scanned together (copies above bit 48: at most kSmallRows)
    long long before = 0;
    for (int i0 = 0; i0 < a.n_out; i0 += kSmallThreads) {
        const int i = i0 + tid;
        long long mine = 0;
        int keep = 0;
        if (i < a.n_out) {
            const int parent = s.parent[i], full = parent >= 0 ? s.full[parent] : 0;
            long long copies = 0;
            if (parent >= 0 && s.len[parent] != full * ps) {
                const int last = s.last[parent];
                if (last < 0 && blockIdx.x == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
                keep = last >= 0 && s.delta[last] == 1 && s.first[parent] == i;
                copies = last >= 0 && !keep;
            }
            mine = s.pages[i] - full - keep + (copies << 48);
        }
        long long sum;
        const long long upto = before + block_scan<long long>(mine, sh64, &sum);
        constexpr long long kLow = (1ll << 48) - 1;
        if (i < a.n_out) {
            const int need = (int)(mine & kLow);
            const bool failed = need > 0 && (upto & kLow) > n_free;
            if (failed) {
                if (blockIdx.x == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
                s.off[i] = -1;
                if (blockIdx.x == gridDim.x - 1) a.seq_len_out[i] = 0;
            } else {
                s.off[i] = (need > 0 ? (int)((upto & kLow) - need) : 0) | (keep ? kKeeps : 0);
                if (s.parent[i] >= 0) atomicAdd(s.children + s.parent[i], 1);
            }
            if (mine >> 48) s.pairs[(int)(upto >> 48) - 1] = (uint16_t)i;
        }
        before += sum;
    }
    const int n_pairs = (int)(before >> 48);
    __syncthreads();
    const int warps = gridDim.x * kSmallWarps, warp = warp_spread();
    if (blockIdx.x == 0) {
        for (int p = tid; p < a.n_in; p += kSmallThreads) {
            const int first = s.first[p];
            s.first[p] = first < a.n_out && s.off[first] >= 0 && (s.off[first] & kKeeps) != 0;
        }
        __syncthreads();
        // table entry x = p ld + j, which is page e
        const int dp = kSmallThreads / max(ld, 1), dj = kSmallThreads - dp * ld;
        int p = tid / max(ld, 1), j = tid - p * ld;
        auto count = [&](int e) {
            const int full = s.full[p];
            if (full >= 0 && j < full + (s.len[p] != full * ps)) {
                const int delta = (j < full ? s.children[p] : s.first[p]) - 1;
                if (e < 0 || e >= a.n_pages)
                    record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, p);
                else if (delta != 0)
                    atomicAdd(s.delta + e, delta);
            }
            p += dp;
            j += dj;
            if (j >= ld) j -= ld, ++p;
        };
#pragma unroll
        for (int i = 0; i < kEntriesAhead; ++i)
            if (tid + i * kSmallThreads < entries) count(entry[i]);
#pragma unroll 4
        for (int x = tid + kEntriesAhead * kSmallThreads; x < entries; x += kSmallThreads) count(a.table[x]);
        // new pages were free: each is named once. A thread takes a row's first few, warps the rest of a row that starts
        // with many, as a prompt does: 1,000 pages 8.5 us, by one thread 29.8
        auto new_pages = [&](int i) {
            const int off = s.off[i], parent = s.parent[i];
            return off < 0 ? 0 : s.pages[i] - (parent >= 0 ? s.full[parent] : 0) - (off & kKeeps ? 1 : 0);
        };
        bool many = false;
        for (int i = tid; i < a.n_out; i += kSmallThreads) {
            const int mine = new_pages(i), off = s.off[i] & ~kKeeps;
            for (int k = 0; k < min(mine, kFewPages); ++k) atomicAdd(s.delta + s.fresh[off + k], 1);
            many |= mine > kFewPages;
        }
        if (__syncthreads_or(many)) {
            for (int i = tid >> 5; i < a.n_out; i += kSmallWarps) {
                const int mine = new_pages(i), off = s.off[i] & ~kKeeps;
                for (int k = kFewPages + lane; k < mine; k += 32) atomicAdd(s.delta + s.fresh[off + k], 1);
            }
            __syncthreads();
        }
        for (int x = tid; x < a.n_pages; x += kSmallThreads) a.ref_out[x] = s.delta[x];
    }
    for (int i = warp; i < a.n_out; i += warps) {
        const int off = s.off[i], parent = s.parent[i];
        const int kept = off < 0 || parent < 0 ? 0 : s.full[parent] + (off & kKeeps ? 1 : 0), pages = off < 0 ? 0 : s.pages[i];
        const int32_t *from = a.table + (int64_t)max(parent, 0) * a.ld;
        for (int64_t j = lane; j < a.ld; j += 32)
            a.table_out[(int64_t)i * a.ld + j] = j < kept ? from[j] : j < pages ? s.fresh[(off & ~kKeeps) + (int)j - kept] : -1;
    }
    move_pages<kSmallThreads>(pg, n_pairs, a.page_size, [&](int k, int &src, int &dst) {
        const int i = s.pairs[k], parent = s.parent[i], off = s.off[i];
        if (off < 0) return 0;                     // failed
        src = s.last[parent];
        dst = s.fresh[off];                        // a row that copies keeps nothing: no flag
        return s.len[parent] - s.full[parent] * ps;
    });
}

__global__ void __launch_bounds__(kSmallThreads, 2) compact_small_kernel(CompactArgs a, PlaneGroups pg) {
    extern __shared__ __align__(16) int small_smem[];
    __shared__ int counts[kSmallThreads];
    __shared__ int sh[33];
    __shared__ int moving_sh;
    let_next_begin();
    wait_for_previous();
    const int tid = threadIdx.x, lane = tid & 31;
    // [n_pages] a live page's new id, or a moving page's place from the last; [n_pages / 2] each
    uint16_t *const map = reinterpret_cast<uint16_t *>(small_smem), *const movers = map + a.n_pages,
                   *const holes = movers + (a.n_pages + 1) / 2;
    constexpr uint16_t kFree = 0xFFFF;
    int n_live;
    const uint32_t is_live = small_ranks<false>(a.ref, a.n_pages, 0, counts, sh, &n_live, [](int r) { return r > 0; }, [](int, int) {});
    if (tid == 0 && n_live == a.n_pages) moving_sh = 0;
    for_ranks(is_live, a.n_pages, counts, [&](int p, bool live, int below) {
        if (p == n_live) moving_sh = n_live - below;
        if (live) {
            map[p] = (uint16_t)(p < n_live ? p : n_live - 1 - below);
            if (p >= n_live) movers[n_live - 1 - below] = (uint16_t)p;
        } else {
            map[p] = kFree;
            if (p < n_live) holes[p - below] = (uint16_t)p;
        }
    });
    __syncthreads();
    const int moving = moving_sh;
    const int warps = gridDim.x * (kSmallThreads / 32), warp = warp_spread();
    for (int i = warp; i < a.n_rows; i += warps) {
        int len = a.seq_len[i];
        if (len < 0 || pages_of(len, a.page_size) > a.ld) {
            if (lane == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
            len = 0;
        }
        const int pages = pages_of(len, a.page_size);
        for (int64_t j = lane; j < a.ld; j += 32) {
            int e = -1;
            if (j < pages) {
                const int old = a.table[(int64_t)i * a.ld + j];
                const int to = old >= 0 && old < a.n_pages ? map[old] : kFree;
                if (to == kFree)
                    record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
                else
                    e = old < n_live ? to : holes[moving - 1 - to];
            }
            a.table_out[(int64_t)i * a.ld + j] = e;
        }
    }
    for (int p = blockIdx.x * kSmallThreads + tid; p < a.n_pages; p += gridDim.x * kSmallThreads) {
        if (p >= n_live) {
            const int to = map[p];
            if (to != kFree) a.ref_out[holes[moving - 1 - to]] = a.ref[p];
            a.ref_out[p] = 0;
        } else if (map[p] != kFree) {
            a.ref_out[p] = a.ref[p];
        }
    }
    move_pages<kSmallThreads>(pg, moving, 1, [&](int k, int &src, int &dst) {
        src = movers[k];
        dst = holes[moving - 1 - k];
        return 1;
    });
}

// CTAs of the small kernels: two for each of 152 SMs. The first call on a device raises the shared-memory limit.
template <typename K, typename A>
cudaError_t launch_small(K kern, const A &a, const PlaneGroups &p, size_t bytes, bool (&ready)[64], cudaStream_t st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmallSmem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    return launch_dependent(kern, dim3(152 * 2), kSmallThreads, bytes, st, a, p);
}

// CTAs of the copying kernels: four for each of 152 SMs.
constexpr int kMoveCtas = 152 * 4;

}  // namespace

size_t pages_scratch_bytes(int n_rows, int64_t n_pages) {
    const size_t rows = up256((size_t)n_rows * 4), pages = up256((size_t)n_pages * 4);
    return 256 + 4 * rows + up256((size_t)n_rows * sizeof(RowCopy)) + 3 * pages;
}

cudaError_t launch_fork_pages(const ForkArgs &a, const PlaneGroups &p, cudaStream_t st) {
    if (a.n_pages <= kSmallPages && a.n_in <= kSmallRows && a.n_out <= kSmallRows && a.n_in * a.ld <= kSmallEntries) {
        static bool ready[64];
        ForkArgs b = a;
        b.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
        return launch_small(fork_small_kernel, b, p, small_fork_bytes(a.n_in, a.n_out, a.n_pages), ready, st);
    }
    char *w = a.scratch;
    ForkScratch s;
    auto take = [&](size_t bytes) {
        char *at = w;
        w += up256(bytes);
        return at;
    };
    s.head = reinterpret_cast<PlanHead *>(take(256));
    s.first = reinterpret_cast<int32_t *>(take((size_t)a.n_in * 4));
    s.children = reinterpret_cast<int32_t *>(take((size_t)a.n_in * 4));
    s.off = reinterpret_cast<int32_t *>(take((size_t)a.n_out * 4));
    s.keeps = reinterpret_cast<int32_t *>(take((size_t)a.n_out * 4));
    s.pairs = reinterpret_cast<RowCopy *>(take((size_t)a.n_out * sizeof(RowCopy)));
    s.fresh = reinterpret_cast<int32_t *>(take((size_t)a.n_pages * 4));
    const cudaError_t e = launch_dependent(fork_plan_kernel, dim3(kCluster), kPlanThreads, 0, st, a, s);
    if (e != cudaSuccess) return e;
    return launch_dependent(fork_move_kernel, dim3(kMoveCtas), kMoveThreads, 0, st, a, s, p);
}

cudaError_t launch_compact_pages(const CompactArgs &a, const PlaneGroups &p, cudaStream_t st) {
    if (a.n_pages <= kSmallPages) {
        static bool ready[64];
        return launch_small(compact_small_kernel, a, p, small_compact_bytes(a.n_pages), ready, st);
    }
    char *w = a.scratch;
    CompactScratch s;
    s.head = reinterpret_cast<PlanHead *>(w);
    const size_t pages = up256((size_t)a.n_pages * 4);
    s.rank = reinterpret_cast<int32_t *>(w + 256);
    s.movers = reinterpret_cast<int32_t *>(w + 256 + pages);
    s.holes = reinterpret_cast<int32_t *>(w + 256 + 2 * pages);
    const cudaError_t e = launch_dependent(compact_plan_kernel, dim3(kCluster), kPlanThreads, 0, st, a, s);
    if (e != cudaSuccess) return e;
    return launch_dependent(compact_move_kernel, dim3(kMoveCtas), kMoveThreads, 0, st, a, s, p);
}

cudaError_t launch_copy_pages(const int32_t *src, const int32_t *dst, int n, const PlaneGroups &p, int64_t n_src,
                              int64_t n_dst, WsHeader *hdr, cudaStream_t st) {
    return launch_dependent(copy_pages_kernel, dim3(kMoveCtas), kMoveThreads, 0, st, src, dst, n, p, n_src, n_dst, hdr);
}

}  // namespace qsa
