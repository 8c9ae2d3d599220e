// Bookkeeping and copying of a paged cache's pages: fork / extend / free (qsa_fork_pages), compaction
// (qsa_compact_pages) and plain copies (qsa_copy_pages).
//
// The whole numbers are settled by one cluster of 8 CTAs (its hardware barrier joins the phases; the counts
// and lists between them live in the workspace), since every phase needs the one before it over all rows or
// pages: the lowest free pages are found by counting each CTA's share of ref first and numbering it after.
// A second kernel, launched as its programmatic dependent, writes the tables and copies the pages with every
// SM: that part is bound by HBM, the first by the latency of its dependent loads.
#include "paged.cuh"

#include <algorithm>

namespace qsa {

namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 16384;      // one CTA's share of a page copy at a time

struct RowCopy {                       // row `row`'s first new page becomes page src's first `used` tokens
    int32_t src, row, used;
};

// Counts at the front of the scratch area.
struct PlanHead {
    int32_t per_cta[kCluster];         // free (fork) or live (compact) pages in each CTA's share
    int32_t extra[kCluster];           // compact: moving pages in each share
    int32_t holes[kCluster];           // compact: free pages below n_live in each share
    int32_t n_pairs, n_live, need, pad;
};
static_assert(sizeof(PlanHead) <= 256, "PlanHead fits its 256 bytes");

// Scratch: head, then arrays of int32 sized by rows and pages.
struct ForkScratch {
    PlanHead *head;
    int32_t *first, *children;         // [n_in] lowest child row, rows that continue it
    int32_t *off;                      // [n_out] first of its new pages in `fresh`, -1: row is empty or failed
    int32_t *keeps;                    // [n_out] keeps the parent's last page
    int32_t *fresh;                    // [n_pages] new pages in the order they are handed out
    RowCopy *pairs;                   // [n_out]
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// Phases (cluster barriers between them):
//   1 count free pages per CTA share, copy ref, clear the per-parent words;
//   2 each row: lowest child of its parent;
//   3 CTA 0: pages each row needs, scanned over the rows -> off, pairs; rows that find no page fail;
//   4 every CTA: number its free pages -> fresh; children of each parent.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    fork_plan_kernel(ForkArgs a, ForkScratch s) {
    __shared__ long long sh[33];
    const int cta = blockIdx.x, tid = threadIdx.x;
    const int all = kCluster * kPlanThreads, me = cta * kPlanThreads + tid;
    launch_dependents();
    const int share = (a.n_pages + kCluster - 1) / kCluster;
    const int lo = min(a.n_pages, cta * share), hi = min(a.n_pages, lo + share);
    int free_here = 0;
    for (int p = lo + tid; p < hi; p += kPlanThreads) {
        const int r = a.ref[p];
        free_here += r == 0;
        a.ref_out[p] = r;
    }
    long long total;
    block_scan<long long>(free_here, sh, &total);
    if (tid == 0) s.head->per_cta[cta] = (int)total;
    for (int p = me; p < a.n_in; p += all) {
        s.first[p] = INT32_MAX;
        s.children[p] = 0;
    }
    cluster_sync();
    for (int i = me; i < a.n_out; i += all) {
        const RowPlan p = row_plan(a, i);
        if (!p.ok) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
        if (p.parent >= 0) atomicMin(s.first + p.parent, i);
    }
    cluster_sync();
    if (cta == 0) {
        long long n_free = 0;
#pragma unroll
        for (int c = 0; c < kCluster; ++c) n_free += s.head->per_cta[c];
        long long carry = 0;           // pages handed out in the low half, copies in the high half
        for (int i0 = 0; i0 < a.n_out; i0 += kPlanThreads) {
            const int i = i0 + tid;
            long long mine = 0;
            RowPlan p{};
            bool keep = false, copy = false;
            int last = -1;
            if (i < a.n_out) {
                p = row_plan(a, i);
                if (p.used > 0) {
                    last = a.table[(int64_t)p.parent * a.ld + p.full];
                    const bool named = last >= 0 && last < a.n_pages;
                    if (!named) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
                    keep = s.first[p.parent] == i && named && a.ref[last] == 1;
                    copy = !keep;
                    if (!named) last = -1;
                }
                mine = p.pages - p.full - (keep ? 1 : 0);
            }
            long long sum;
            const long long upto = carry + block_scan<long long>(mine, sh, &sum);
            const bool failed = mine > 0 && upto > n_free;
            carry += sum;
            if (failed) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
            if (i < a.n_out) {
                s.off[i] = failed ? -1 : (int)(upto - mine);
                s.keeps[i] = keep;
                a.seq_len_out[i] = failed ? 0 : p.total;
            }
            copy = copy && !failed && last >= 0;
            // the copies' list: rows in order
            long long copies;
            const long long rank = block_scan<long long>(copy, sh, &copies);
            const int before = i0 == 0 ? 0 : s.head->n_pairs;
            if (copy) s.pairs[before + (int)rank - 1] = {last, i, p.used};
            __syncthreads();
            if (tid == 0) s.head->n_pairs = before + (int)copies;
            __syncthreads();
        }
        if (tid == 0) {
            s.head->need = (int)min(carry, n_free);
            if (a.n_out == 0) s.head->n_pairs = 0;
        }
    }
    cluster_sync();
    for (int i = me; i < a.n_out; i += all)
        if (s.off[i] >= 0) {
            const int p = row_plan(a, i).parent;
            if (p >= 0) atomicAdd(s.children + p, 1);
        }
    const int need = s.head->need;
    int base = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) base += c < cta ? s.head->per_cta[c] : 0;
    for (int p0 = lo; p0 < hi && base < need; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const bool is_free = p < hi && a.ref[p] == 0;
        long long sum;
        const int rank = base + (int)block_scan<long long>(is_free, sh, &sum) - 1;
        if (is_free && rank < need) s.fresh[rank] = p;
        base += (int)sum;
    }
}

// ---------------------------------------------------------------------------- copies
// Words of 16 or 4 bytes of one plane's page, [begin, end) bytes, by the CTA's threads.
template <typename W>
__device__ __forceinline__ void move_words(const char *src, char *dst, int64_t begin, int64_t end) {
    constexpr int U = 4;
    const int64_t step = (int64_t)kMoveThreads * sizeof(W);
    for (int64_t b = begin + threadIdx.x * (int64_t)sizeof(W); b < end; b += U * step) {
        W v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u * step < end) v[u] = *reinterpret_cast<const W *>(src + b + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u * step < end) *reinterpret_cast<W *>(dst + b + u * step) = v[u];
    }
}

// Every plane's pages of n pairs; pair k by `pair`, which returns the used tokens (0: skip).
template <typename Pair>
__device__ __forceinline__ void move_pages(const PlaneGroups &pg, int n, int page_size, Pair pair) {
    for (int gi = 0; gi < pg.n; ++gi) {
        const PlaneGroup &g = pg.g[gi];
        const int64_t parts = (g.page_bytes + kMoveBytes - 1) / kMoveBytes;
        const int64_t items = parts * g.n_planes * n;
        for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
            const int64_t part = w % parts, rest = w / parts;
            const int plane = (int)(rest % g.n_planes), k = (int)(rest / g.n_planes);
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
__global__ void __launch_bounds__(kMoveThreads) fork_move_kernel(ForkArgs a, ForkScratch s, PlaneGroups pg) {
    wait_for_primary();
    const int lane = threadIdx.x & 31;
    const int warp = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5, warps = gridDim.x * (kMoveThreads / 32);
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
    for (int p = warp; p < a.n_in; p += warps) {
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
    move_pages(pg, s.head->n_pairs, a.page_size, [&](int k, int &src, int &dst) {
        const RowCopy c = s.pairs[k];
        src = c.src;
        dst = s.fresh[s.off[c.row]];
        return c.used;
    });
}

// ---------------------------------------------------------------------------- compaction
struct CompactScratch {
    PlanHead *head;
    int32_t *to;                       // [n_pages] new id of a live page, -1: free
    int32_t *movers, *holes;           // [n_pages] ascending
};

// Phases: 1 count live pages; 2 with n_live known, count the pages that move and the holes; 3 number them;
// 4 `to` and ref_out where pages move. (ref_out above n_live is cleared by the second kernel.)
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(CompactArgs a, CompactScratch s) {
    __shared__ long long sh[33];
    const int cta = blockIdx.x, tid = threadIdx.x;
    launch_dependents();
    const int share = (a.n_pages + kCluster - 1) / kCluster;
    const int lo = min(a.n_pages, cta * share), hi = min(a.n_pages, lo + share);
    long long total;
    int live = 0;
    for (int p = lo + tid; p < hi; p += kPlanThreads) live += a.ref[p] > 0;
    block_scan<long long>(live, sh, &total);
    if (tid == 0) s.head->per_cta[cta] = (int)total;
    cluster_sync();
    int n_live = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) n_live += s.head->per_cta[c];
    long long both = 0;                // movers in the high half, holes in the low half
    for (int p = lo + tid; p < hi; p += kPlanThreads) {
        const bool is_live = a.ref[p] > 0;
        both += ((long long)(is_live && p >= n_live) << 32) + (!is_live && p < n_live);
    }
    block_scan<long long>(both, sh, &total);
    if (tid == 0) {
        s.head->extra[cta] = (int)(total >> 32);
        s.head->holes[cta] = (int)(total & 0xffffffff);
    }
    cluster_sync();
    long long base = 0;
    int moving = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
        moving += s.head->extra[c];
        if (c < cta) base += ((long long)s.head->extra[c] << 32) + s.head->holes[c];
    }
    for (int p0 = lo; p0 < hi; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const bool is_live = p < hi && a.ref[p] > 0;
        const bool mover = is_live && p >= n_live, hole = p < hi && !is_live && p < n_live;
        const long long upto =
            base + block_scan<long long>(((long long)mover << 32) + (long long)hole, sh, &total);
        if (mover) s.movers[(int)(upto >> 32) - 1] = p;
        if (hole) s.holes[(int)(upto & 0xffffffff) - 1] = p;
        if (p < hi && !mover) {
            s.to[p] = is_live ? p : -1;
            if (is_live) a.ref_out[p] = a.ref[p];
        }
        base += total;
    }
    cluster_sync();
    const int all = kCluster * kPlanThreads, me = cta * kPlanThreads + tid;
    for (int k = me; k < moving; k += all) {
        s.to[s.movers[k]] = s.holes[k];
        a.ref_out[s.holes[k]] = a.ref[s.movers[k]];
    }
    if (cta == 0 && tid == 0) {
        s.head->n_pairs = moving;
        s.head->n_live = n_live;
    }
}

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(CompactArgs a, CompactScratch s, PlaneGroups pg) {
    wait_for_primary();
    const int lane = threadIdx.x & 31;
    const int warp = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5, warps = gridDim.x * (kMoveThreads / 32);
    const int n_live = s.head->n_live;
    for (int p = n_live + blockIdx.x * kMoveThreads + threadIdx.x; p < a.n_pages; p += gridDim.x * kMoveThreads)
        a.ref_out[p] = 0;
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
                e = e >= 0 && e < a.n_pages ? s.to[e] : -1;
                if (e < 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, i);
            }
            a.table_out[(int64_t)i * a.ld + j] = e;
        }
    }
    move_pages(pg, s.head->n_pairs, 1, [&](int k, int &src, int &dst) {
        src = s.movers[k];
        dst = s.holes[k];
        return 1;
    });
}

__global__ void __launch_bounds__(kMoveThreads)
    copy_pages_kernel(const int32_t *src_ids, const int32_t *dst_ids, int n, PlaneGroups pg, int64_t n_src, int64_t n_dst,
                      WsHeader *hdr) {
    move_pages(pg, n, 1, [&](int k, int &src, int &dst) {
        src = src_ids[k];
        dst = dst_ids[k];
        if (src < 0 || dst < 0) return 0;
        if (src >= n_src || dst >= n_dst) {
            if (threadIdx.x == 0) record_error(hdr, QSA_ERR_DEVICE_BOUNDS, kWherePages, k);
            return 0;
        }
        return 1;
    });
}

// CTAs of the copying kernels: four for each of 152 SMs.
constexpr int kMoveCtas = 152 * 4;

template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMoveCtas);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

size_t pages_scratch_bytes(int n_rows, int64_t n_pages) {
    const size_t rows = up256((size_t)n_rows * 4), pages = up256((size_t)n_pages * 4);
    return 256 + 4 * rows + up256((size_t)n_rows * sizeof(RowCopy)) + 3 * pages;
}

cudaError_t launch_fork_pages(const ForkArgs &a, const PlaneGroups &p, cudaStream_t st) {
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
    fork_plan_kernel<<<kCluster, kPlanThreads, 0, st>>>(a, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(fork_move_kernel, st, a, s, p);
}

cudaError_t launch_compact_pages(const CompactArgs &a, const PlaneGroups &p, cudaStream_t st) {
    char *w = a.scratch;
    CompactScratch s;
    s.head = reinterpret_cast<PlanHead *>(w);
    const size_t pages = up256((size_t)a.n_pages * 4);
    s.to = reinterpret_cast<int32_t *>(w + 256);
    s.movers = reinterpret_cast<int32_t *>(w + 256 + pages);
    s.holes = reinterpret_cast<int32_t *>(w + 256 + 2 * pages);
    compact_plan_kernel<<<kCluster, kPlanThreads, 0, st>>>(a, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(compact_move_kernel, st, a, s, p);
}

cudaError_t launch_copy_pages(const int32_t *src, const int32_t *dst, int n, const PlaneGroups &p, int64_t n_src,
                              int64_t n_dst, WsHeader *hdr, cudaStream_t st) {
    copy_pages_kernel<<<kMoveCtas, kMoveThreads, 0, st>>>(src, dst, n, p, n_src, n_dst, hdr);
    return cudaGetLastError();
}

}  // namespace qsa
