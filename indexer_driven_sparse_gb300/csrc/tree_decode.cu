// Attention of a tree of drafted tokens over a paged K/V cache (qsa_tree_decode, qsa_tree_decode_fp8kv):
//   out[i] = sum_j softmax_j(scale q[i] . K[j]) V[j] over the cached tokens before the drafts, i's ancestors and i.
//
// A sequence's T drafted tokens times the G query heads of a KV head are T G rows that share every K and V row: 4 T G flops
// per value read. 16 tokens with 8 heads each are the 128 rows of one tcgen05 tile; their 64 KB of K and V for 64 tokens of 256
// dims take an SM's share of HBM 2,900 cycles, the products 1,500: with one such M tile the rows' stream bounds the call, with
// two or more the products.
//
// Split: as in the decode of one token (paged_decode.cuh), the batch's tokens, cut into tiles of 64 of one sequence each, form one
// list, dealt to R ranges of equal length; CTA (range, KV head, M tile) walks its part. The M tiles of a range are neighbouring
// CTAs that read the same rows at the same time: from L2, all but one of them. A sequence that a range boundary cuts
// leaves partials (m, l, O), joined by tree_join_kernel; all others are written at once.
//
// Roles of a CTA's 20 warps (one CTA per SM), which meet at mbarriers only:
//   8 softmax warps  two threads a row, 32 of a tile's tokens each: running maximum and sum in base 2, O rescaled only when the
//                    maximum has grown by more than 2^8; weights go back to tensor memory over the scores they came from;
//   1 score warp     S = Q K^T (M 128, N 64) into the next of its buffers, queries (bf16 rows) from tensor memory;
//   1 output warp    O += P V (N 256), P from tensor memory. An instruction of N 64 takes as long as one of N 128 (61 cycles), so Q K^T
//                    runs at half the rate; 512 columns hold O, the queries and two buffers of 64 scores at 256 dims, not of 128;
//   1 index warp     page table -> slots, scales, up to 8 or 16 tiles ahead;
//   1 load warp      tiled TMA loads, a box for each run of a page; or all workers: cp.async of 16 bytes, row by row;
//   2 or 4 query warps  the rows' queries, the ancestors' bits, and the clean-up of V rows that not every row attends;
//   5 or 6 workers   cp.async loads; FP8 rows: V's codes -> f16 operands.
// K and V of a tile lie in shared memory as slots of 128-byte-swizzled blocks, a ring in the order in which the products take
// them: K0 K1 V0 K2 V1 ... The kernel is as short as it is for the instruction caches' sake: every role runs code of its own, and
// with the waits and walks inlined (256 KB of it) they waited for instructions three times as long as they issued them.
//
// A masked token's weight is zero, but zero times an infinite or undefined V value is not: V rows that no row attends (behind the
// sequence's end, before its window) become zeros, and values that are not finite in rows that only some attend (drafts, the
// window's edge) are taken out of the product and added at the end to the rows that attend them.
//
// bf16 rows: weights enter the second product as bf16 (2^-8 of each; the decode of one token adds a second bf16 value, which
// here would make half as many products again). FP8 rows: K's codes are multiplied as they are, q enters as the sum of two E4M3
// values scaled by a power of two per row (all of a bf16 value down to 2^-10 of the row's largest, smaller ones off by at most
// 2^-17 of that), K's scales multiply the fp32 sums of each 128 dims; V's codes become f16, exactly, and V's scales enter the weights:
// w = 2^(s - m) v_scale / u 2^6 with m the lazy maximum and u the power of two next to the largest V scale so far, one set for
// each 128 dims, below 2^15 and rounded to f16 (2^-11 of each, 2^-31 of the largest weight times the largest scale).
#include "paged_decode.cuh"
#include "qsa_tc.cuh"

#include <algorithm>

namespace qsa {

namespace {

constexpr int kRows = 128;                       // MMA M: rows of a CTA
constexpr int kTile = 64;                        // tokens of a tile
constexpr float kLazy = 8.f;                     // O is rescaled when a maximum has grown by more than 2^8
constexpr float kRaise = 6.f;                    // FP8 rows: weights up to 2^8, scales below 2, so below 2^15 in f16

// Tiled: rows come by TMA (pages of whole runs of tokens), else by cp.async.
template <int D_, bool F8_, bool Tiled_>
struct TreeCfg {
    static constexpr int D = D_;
    static constexpr bool tiled = Tiled_;
    static constexpr bool F8 = F8_;
    static constexpr int SG = F8 ? D / 128 : 1;                 // scales of a row, sets of weights
    static constexpr int slot = kTile * D * 2, code_slot = F8 ? kTile * D : 0;      // bytes: a tile's K or V
    // bf16 rows: one ring for K and V. FP8 rows: K's codes, V's codes, and V as f16 operands, each in a ring of its own.
    static constexpr int ring = F8 ? 2 : D == 64 ? 24 : 212992 / slot;
    static constexpr int k_ring = F8 ? (D == 256 ? 3 : 6) : 0, v_ring = F8 ? (D == 256 ? 2 : 6) : 0;
    static constexpr int ring_at = F8 ? kRows * D * 2 : 0, k_at = ring_at + ring * slot, v_at = k_at + k_ring * code_slot;
    static constexpr int smem = v_at + v_ring * code_slot + 1024;
    static_assert(smem + 17920 <= 227 * 1024, "shared memory of a CTA");
    // tensor memory columns: O, the queries (bf16 rows; with FP8 rows they are in shared memory), buffers of scores
    static constexpr uint32_t t_o = 0, t_q = F8 ? 0u : (uint32_t)D, t_s = D == 256 && !F8 ? 384 : 256, s_cols = SG * kTile;
    static constexpr int buffers = (512 - t_s) / s_cols;
    // tiles whose slots and scales are known: 4, 6, 8 and 16 of them took 270, 264, 254 and 251 us over 64 ragged sequences of FP8 rows
    static constexpr int metas = D == 128 ? 16 : 8;
    // 20 warps of 96 registers; the query warps' numbers modulo 4 are the four quarters of tensor memory's lanes
    static constexpr int softmax = 256, q_threads = F8 ? 64 : 128, workers = F8 ? 192 : 160;
    // FP8 rows: the converting warps 14 to 19 are two on schedulers 2 and 3; the index warp beside two of them slowed their softmax
    // warps by half
    static constexpr int s_warp = 8, o_warp = 9, index_warp = F8 ? 12 : 10, q_warp = F8 ? 10 : 11, load_warp = F8 ? 13 : 15;
    static constexpr int work_warp = F8 ? 14 : 15;
    static constexpr int threads = 640;
    static_assert(work_warp * 32 + workers == threads && t_o + D <= t_s && t_q + (F8 ? 0 : D / 2) <= t_s, "roles, columns");
};

// Two fp32 values an instruction, each rounded as alone.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

__device__ __forceinline__ float2 get2(const float *v, int k) { return make_float2(v[2 * k], v[2 * k + 1]); }
__device__ __forceinline__ void set2(float *v, int k, float2 x) { v[2 * k] = x.x, v[2 * k + 1] = x.y; }

// 16 consecutive fp32 columns of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

struct TreeMaps {
    CUtensorMap k, v;
};

// How rows get into shared memory: runs of `run` tokens by tiled TMA, or (0) by the worker warps.
struct TreePlan {
    int32_t ranges, m_tiles, run;
    int32_t page_shift;
    int32_t min_tiles;       // of a range
};

struct TreeScratch {
    int2 *meta;              // [ranges] (row, parts)
    float2 *ml;              // [2 ranges][Hkv m_tiles][128]
    float *o;                // [..][D]
};

struct TreeRow {
    int len, off, T, base, lo, t0, t1;    // tokens; drafts [off, off + T) in places [base, len); first attended place; tiles
    bool named;                           // its offsets are fine
};

// high: the largest offset of an earlier sequence (0 at first).
__device__ __forceinline__ TreeRow tree_row(const TreeArgs &a, int s, int &high) {
    TreeRow r;
    r.off = a.draft_off[s];
    const int end = a.draft_off[s + 1];
    r.named = r.off >= high && end >= r.off && end <= a.N;
    high = max(high, r.off);
    r.T = r.named ? end - r.off : 0;
    r.len = a.seq_len[s];
    r.t0 = r.t1 = 0;
    if (r.T > 0 && r.T <= a.max_draft && r.len >= r.T && r.len <= a.ld * a.page_size) {
        r.base = r.len - r.T;
        r.lo = a.window > 0 ? max(0, r.base + 1 - a.window) : 0;
        r.t0 = r.lo / kTile;
        r.t1 = r.len / kTile + (r.len % kTile != 0);
    }
    return r;
}

struct Seg {
    TreeRow r;
    int s, ta, tb;           // tiles [ta, tb) of sequence s
    int i0;                  // tiles of this CTA before them
    bool begins, ends;       // with the sequence
};

// The tiles [x, x1) of the list as segments of one sequence each; sequences without a row in this M tile are passed over.
struct Walk {
    long long x, x1;
    int s, skip, high, i = 0;
    __device__ __noinline__ bool next(const TreeArgs &a, int m_tile, Seg &g) {
        while (x < x1) {
            g.r = tree_row(a, s, high);
            const int n = g.r.t1 - g.r.t0;
            if (n == 0) {
                ++s;
                continue;
            }
            g.s = s++;
            g.ta = g.r.t0 + skip;
            g.tb = (int)min((long long)g.r.t1, g.ta + (x1 - x));
            g.begins = skip == 0;
            g.ends = g.tb == g.r.t1;
            x += g.tb - g.ta;
            skip = 0;
            if (m_tile * kRows >= g.r.T * a.G) continue;
            g.i0 = i;
            i += g.tb - g.ta;
            return true;
        }
        return false;
    }
};

// The order of a segment's n tiles in the ring, in slots of one tile's K or V: K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ int k_turn(int c) { return c == 0 ? 0 : 2 * c - 1; }
__device__ __forceinline__ int v_turn(int c, int n) { return c == n - 1 ? 2 * n - 1 : 2 * c + 2; }

// Whether some row may not attend some token of tile t.
__device__ __forceinline__ bool masked(const TreeArgs &a, const TreeRow &r, int t) {
    const int j0 = t * kTile;
    return j0 > r.base - kTile || (a.window > 0 && j0 < r.base + r.T - a.window);
}

// Whether every row attends token j of [r.lo, r.len). In a tile that is masked some tokens are for all rows nevertheless.
__device__ __forceinline__ bool for_all(const TreeArgs &a, const TreeRow &r, int j) {
    return j < r.base && (a.window == 0 || j >= r.base + r.T - a.window);
}

template <typename C>
struct TreeShared {
    uint64_t full[C::ring], empty[C::ring];
    uint64_t k_full[C::F8 ? C::k_ring : 1], k_empty[C::F8 ? C::k_ring : 1], v_full[C::F8 ? C::v_ring : 1], v_empty[C::F8 ? C::v_ring : 1];
    uint64_t s_full[C::buffers], p_full[C::buffers], pv_done[C::buffers], meta_full[C::metas], meta_empty[C::metas];
    uint64_t to_clean, clean, q_full, q_free, nodes_full, nodes_free, flags_full, o_free;
    uint32_t kin[QSA_MAX_DRAFT][QSA_MAX_DRAFT / 32];      // of each drafted token: itself and its ancestors inside the window
    int lo[QSA_MAX_DRAFT];                                // its first attended place
    uint32_t odd[2][QSA_MAX_DRAFT / 32];                  // tokens with values that are not finite: drafts, places from r.lo
    float q_scale[2][C::F8 ? kRows : 1];               // of every other segment
    int slots[C::metas][kTile];
    uint32_t real[C::metas][kTile / 32];                   // bit: the token's page exists
    float4 k_scales[C::metas][C::SG][C::F8 ? kTile / 4 : 1], v_scales[C::metas][C::SG][C::F8 ? kTile / 4 : 1];   // four tokens each
    float2 top[C::metas];                                 // powers of two at most 2 below the tile's largest V scales
    float tops[2][2][kRows];                              // of every other tile: the halves' maxima
    uint32_t tmem;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Operands in shared memory, both E4M3 (the descriptor's format bits are zero, as f16's are for kind::f16); 32 bytes of K.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0)
        : "memory");
}

// kind::f16 with f16 operands (tc_idesc is bf16's)
__host__ __device__ constexpr uint32_t f16_idesc(int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
                 "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Which of the eight bf16 values of v are not finite: all of them as zeros, and whether there was one.
__device__ __forceinline__ bool drop_odd(uint4 &v) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
    bool some = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u, some = true;
        if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu, some = true;
    }
    return some;
}

// Codes 0x7F and 0xFF of four E4M3 codes as zeros, and whether there was one.
__device__ __forceinline__ bool drop_nan_codes(uint32_t &w) {
    const uint32_t nan = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    w &= ~nan;
    return nan != 0;
}

// What a CTA's waits share: whether one of them has given up, how many tiles the index warp has named, and where to record. Not
// handed to each wait: two more arguments cost registers.
struct TreeWaits {
    uint32_t gave_up, tiles;
    WsHeader *hdr;
};
__shared__ volatile TreeWaits tree_waits;

// Wait for phase `parity` of an mbarrier: false if the CTA has given up, or if kWaitLimitNs pass without a further tile; that is
// recorded, and ends the CTA's other waits. (A wait for a segment's end may last longer while its tiles go by.) Each try may
// suspend the thread for kHintNs. Out of line: with the waits and the walks inlined the kernel had 256 KB of
// instructions, and its roles, each on a part of its own, waited for them more than for anything else.
constexpr uint32_t kHintNs = 1000000;
constexpr int kTries = 8;                        // between looks at the clock, which takes as long as many a wait
__device__ __forceinline__ bool try_turn(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kHintNs)
        : "memory");
    return done != 0;
}
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
    uint64_t since = 0;
    uint32_t seen = 0;
#pragma unroll 1
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < kTries; ++i)
            if (try_turn(bar, parity)) return true;
        if (tree_waits.gave_up) return false;
        const uint32_t now = tree_waits.tiles;
        if (since == 0 || now != seen) {
            seen = now, since = globaltimer_ns();
        } else if (globaltimer_ns() - since > kWaitLimitNs) {
            tree_waits.gave_up = 1;
            record_error(tree_waits.hdr, QSA_ERR_DEVICE_TIMEOUT, kWhereTree, blockIdx.x);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_turn(uint32_t bar, uint32_t parity) {
    return try_turn(bar, parity) || wait_long(bar, parity);
}
// Wait for what is on its way already, a copy or a product, before shared or tensor memory is given up: whether or not the CTA has
// given up, and for kWaitLimitNs at most.
__device__ __noinline__ void wait_landed(uint32_t bar, uint32_t parity) {
    if (!mbar_wait_bounded(bar, parity, kWaitLimitNs)) record_error(tree_waits.hdr, QSA_ERR_DEVICE_TIMEOUT, kWhereTree, blockIdx.x);
}
// A barrier of `threads` threads that also tells whether any of them came with `bad`. Warps that share a barrier leave together:
// one that left alone after a wait in vain would keep the others there for good.
__device__ __forceinline__ bool meet_any(int barrier, int threads, bool bad) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.aligned.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(bad ? 1u : 0u), "r"(barrier), "r"(threads)
        : "memory");
    return any != 0;
}

// Values that are not finite, of tokens that this row attends but not every row: added to its result (whole) or its partial.
template <int D, bool F8>
__device__ __noinline__ void add_odd(const TreeArgs &a, const Seg &g, const uint32_t (*odd)[QSA_MAX_DRAFT / 32], const uint32_t *kin,
                                     int lo, int kvh, int first, bool whole, uint16_t *dst, float *po) {
#pragma unroll 1
    for (int x = 0; x < 2 * QSA_MAX_DRAFT; ++x) {
        const int y = x % QSA_MAX_DRAFT, j = (x == y ? g.r.base : g.r.lo) + y;
        if (!(odd[x / QSA_MAX_DRAFT][y >> 5] >> (y & 31) & 1u)) continue;
        if (x == y ? !(kin[y >> 5] >> (y & 31) & 1u) : j < lo || j >= g.r.base) continue;
        const int page = a.table[g.s * a.ld + j / a.page_size];
        if ((uint32_t)page >= (uint32_t)a.n_pages) continue;
        const int64_t row = (((int64_t)page * a.page_size + j % a.page_size) * a.Hkv + kvh) * D;
#pragma unroll 1
        for (int d = first; d < first + D / 2; ++d) {
            const float z = F8 ? ((static_cast<const uint8_t *>(a.v)[row + d] & 0x7Fu) == 0x7Fu || !isfinite(a.v_scales[(row + d) / 128]) ? NAN : 0.f)
                               : bf16_bits_to_float(static_cast<const uint16_t *>(a.v)[row + d]);
            if (isfinite(z)) continue;
            if (whole)
                dst[d] = float_to_bf16_bits(bf16_bits_to_float(dst[d]) + z);
            else
                po[d] += z;
        }
    }
}

template <typename C>
__global__ void __launch_bounds__(C::threads, 1)
    tree_tile_kernel(TreeArgs a, TreePlan plan, TreeScratch ws, const __grid_constant__ TreeMaps maps) {
    constexpr int D = C::D, T = kTile, RING = C::ring, SG = C::SG, NB = C::buffers;
    constexpr bool F8 = C::F8;
    extern __shared__ uint8_t smem_raw[];
    __shared__ TreeShared<C> sh;
    __shared__ long long scan[C::threads / 32];
    __shared__ int start[3];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t q_at = smem_u32(sm), ring_at = q_at + C::ring_at;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int m_tile = blockIdx.x % plan.m_tiles, kvh = blockIdx.x / plan.m_tiles % a.Hkv, range = blockIdx.x / plan.m_tiles / a.Hkv;
    const bool speaks = kvh == 0 && m_tile == 0;          // records errors that all CTAs of a range see
    constexpr bool tiled = C::tiled;

    if (warp == C::s_warp) tmem_alloc(&sh.tmem, 512);
    {
        // the loads' arrivals: one with the bytes it expects, or every worker's
        const int load = tiled ? 1 : C::workers;
        if (warp == 0 && lane < RING) {
            mbar_init(smem_u32(&sh.full[lane]), F8 ? C::workers / 32 : load);
            mbar_init(smem_u32(&sh.empty[lane]), 1);
        }
        if constexpr (F8)
            if (warp == 1 && lane < C::k_ring + C::v_ring) {
                const bool k = lane < C::k_ring;
                mbar_init(smem_u32(k ? &sh.k_full[lane] : &sh.v_full[lane - C::k_ring]), load);
                mbar_init(smem_u32(k ? &sh.k_empty[lane] : &sh.v_empty[lane - C::k_ring]), k ? 1 : C::workers / 32);
            }
        if (warp == 2 && lane < NB) {
            mbar_init(smem_u32(&sh.s_full[lane]), 1);
            mbar_init(smem_u32(&sh.p_full[lane]), C::softmax / 32);
            mbar_init(smem_u32(&sh.pv_done[lane]), 1);
        }
        if (warp == 3 && lane < C::metas) {
            mbar_init(smem_u32(&sh.meta_full[lane]), 1);
            mbar_init(smem_u32(&sh.meta_empty[lane]), C::softmax / 32 + (tiled ? 1 : C::workers / 32));
        }
        if (tid == 128) {
            mbar_init(smem_u32(&sh.to_clean), 1);
            mbar_init(smem_u32(&sh.clean), C::q_threads);
            mbar_init(smem_u32(&sh.q_full), C::q_threads);
            mbar_init(smem_u32(&sh.q_free), 1);
            mbar_init(smem_u32(&sh.nodes_full), C::q_threads);
            mbar_init(smem_u32(&sh.nodes_free), C::softmax / 32);
            mbar_init(smem_u32(&sh.flags_full), C::q_threads);
            mbar_init(smem_u32(&sh.o_free), C::softmax / 32);
            tree_waits.gave_up = 0, tree_waits.tiles = 0, tree_waits.hdr = a.hdr;
        }
        fence_mbar_init();
        if (tiled && tid == 160) {
            tma_prefetch_desc(&maps.k);
            tma_prefetch_desc(&maps.v);
        }
    }
    wait_for_previous();

    // ---- this range's part of the list: tiles before each thread's run of sequences, then the place of the first tile.
    // Sequences that cannot be attended get their zeros here.
    Walk walk;
    {
        const int per = (a.B + C::threads - 1) / C::threads, s_lo = min(a.B, tid * per), s_hi = min(a.B, s_lo + per);
        int top = 0;                                      // the largest offset of the run
        for (int s = s_lo; s < s_hi; ++s) top = max(top, a.draft_off[s]);
        int upto_top = top;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto_top, o);
            if (lane >= o) upto_top = max(upto_top, v);
        }
        if (lane == 31) scan[warp] = upto_top;
        int high = __shfl_up_sync(0xffffffffu, upto_top, 1);
        if (lane == 0) high = 0;
        __syncthreads();
        for (int w = 0; w < warp; ++w) high = max(high, (int)scan[w]);
        const int high0 = high;
        long long mine = 0;
        for (int s = s_lo; s < s_hi; ++s) {
            const TreeRow r = tree_row(a, s, high);
            mine += r.t1 - r.t0;
            if (r.t1 > r.t0 || (r.named && r.T == 0)) continue;
            if (!speaks || s % plan.ranges != range) continue;
            record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereTree, s);
            for (int64_t i = (int64_t)r.off * a.Hq; r.named && i < (int64_t)(r.off + r.T) * a.Hq; ++i) {
                for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4 *>(a.out + i * D + d) = make_uint4(0, 0, 0, 0);
                if (a.lse) a.lse[i] = -INFINITY;
            }
        }
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        long long total = 0;
#pragma unroll 1
        for (int w = 0; w < C::threads / 32; ++w) {
            if (w < warp) upto += scan[w];
            total += scan[w];
        }
        const Ranges cut(total, (int)max(1ll, min((long long)plan.ranges, total / plan.min_tiles)));
        walk.x = walk.x1 = 0;
        if (range < cut.R) walk.x = cut.begin(range), walk.x1 = cut.begin(range + 1);
        if (walk.x < walk.x1 && upto - mine <= walk.x && walk.x < upto) {
            long long before = upto - mine;
            int at = high0;
            for (int s = s_lo;; ++s) {
                const int was = at;
                const TreeRow r = tree_row(a, s, at);
                if (walk.x < before + r.t1 - r.t0) {
                    start[0] = s, start[1] = (int)(walk.x - before), start[2] = was;
                    break;
                }
                before += r.t1 - r.t0;
            }
        }
        if (speaks && tid == 0) ws.meta[range] = make_int2(-1, 0);
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        walk.s = start[0], walk.skip = start[1], walk.high = start[2];
        if (walk.x >= walk.x1) walk.s = walk.skip = walk.high = 0;

        // the sequence that this range starts and leaves unfinished: how many ranges it spans
        if (speaks && tid == 0 && walk.x < walk.x1) {
            Walk w = walk;
            Seg g;
            while (w.next(a, 0, g))
                if (g.begins && !g.ends) {
                    const long long last = w.x - 1 + (g.r.t1 - g.tb);      // the list's number of its last tile
                    ws.meta[range] = make_int2(g.s, cut.of(last) - range + 1);
                }
        }
    }
    const uint32_t tmem = sh.tmem;

    // A role that waits in vain ends, and so do all others at their next wait.
    auto wait = [&](uint64_t *bar, uint32_t phase) -> bool { return wait_turn(smem_u32(bar), phase & 1u); };
    auto wait_warp = [&](uint64_t *bar, uint32_t phase) -> bool { return __all_sync(0xffffffffu, wait(bar, phase)); };

    Seg g{};
    if (warp == C::index_warp) {
        // ================================================================ slots of each tile; TMA loads
        constexpr int E = T / 32;                         // tokens of a lane: lane, 32 + lane
        int page[E], offset[E];
        bool ok = true;
        int pages_begin = 0, pages_end = 0;               // entries that g needs
        auto enter = [&]() { pages_end = (g.r.len - 1) / a.page_size, pages_begin = g.r.lo / a.page_size; };
        auto fetch = [&](int t) {                         // the page table's entries for tile t of g
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint32_t j = (uint32_t)t * T + e * 32 + lane;     // may pass 2^31
                const uint32_t entry = plan.page_shift >= 0 ? j >> plan.page_shift : j / (uint32_t)a.page_size;
                offset[e] = (int)(j - entry * a.page_size);
                const bool some = entry >= (uint32_t)pages_begin && entry <= (uint32_t)pages_end;
                page[e] = some ? a.table[g.s * a.ld + entry] : -2;
            }
        };
        Walk w = walk;
        int done = 0;
        bool more = w.next(a, m_tile, g);
        if (more) enter(), fetch(g.ta);
        while (more && ok) {
            const Seg now = g;
            const int n = now.tb - now.ta;
            float2 top = make_float2(0.f, 0.f);           // FP8: powers of two next to the largest V scales of the segment so far
            for (int c = 0; c < n && ok; ++c, ++done) {
                int slot[E];
                float4 scale[F8 ? E : 1];
                bool exists[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int j = (now.ta + c) * T + e * 32 + lane;
                    const bool in = (uint32_t)j >= (uint32_t)now.r.lo && (uint32_t)j < (uint32_t)now.r.len;
                    const bool fine = (uint32_t)page[e] < (uint32_t)a.n_pages;
                    if (in && !fine && speaks) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereTree, now.s);
                    slot[e] = fine ? page[e] * a.page_size + offset[e] : -1;
                    exists[e] = in && fine;
                    if (F8) {
                        scale[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (exists[e]) {
                            const int64_t at = ((int64_t)slot[e] * a.Hkv + kvh) * SG;
                            if (SG == 2) {
                                const float2 x = *reinterpret_cast<const float2 *>(a.k_scales + at);
                                const float2 y = *reinterpret_cast<const float2 *>(a.v_scales + at);
                                scale[e] = make_float4(x.x, x.y, y.x, y.y);
                            } else {
                                scale[e] = make_float4(a.k_scales[at], 0.f, a.v_scales[at], 0.f);
                            }
                        }
                    }
                }
                // the next tile's entries, on their way meanwhile
                const int t = now.ta + c;
                if (c + 1 < n) {
                    fetch(t + 1);
                } else {
                    more = w.next(a, m_tile, g);
                    if (more) enter(), fetch(g.ta);
                }
                const int m = done % C::metas;
                // the header's test knob: nothing comes after the third tile, and what waits for it waits in vain
                if ((done == 3 && a.hdr->debug == kDebugStallBarrier) ||
                    (done >= C::metas && !wait_warp(&sh.meta_empty[m], done / C::metas - 1))) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    sh.slots[m][e * 32 + lane] = exists[e] || tiled ? slot[e] : -1;       // a box may begin before the first token
                    const uint32_t bits = __ballot_sync(0xffffffffu, exists[e]);
                    if (lane == 0) sh.real[m][e] = bits;
                }
                if (F8) {
                    float z = 0.f, u = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        z = fmaxf(z, scale[e].z < INFINITY ? scale[e].z : 0.f);
                        u = fmaxf(u, scale[e].w < INFINITY ? scale[e].w : 0.f);
                    }
                    // scales are not negative: their order is that of their bits
                    z = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(z)));
                    if (SG == 2) u = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(u)));
                    auto power = [](float x) { return __uint_as_float(min(max(__float_as_uint(x) & 0x7F800000u, 7u << 23), 247u << 23)); };
                    top = make_float2(fmaxf(top.x, power(z)), fmaxf(top.y, power(u)));
                    auto inverse = [](float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); };
                    const float cx = inverse(top.x) * (float)(1 << (int)kRaise), cy = inverse(top.y) * (float)(1 << (int)kRaise);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float4 x = scale[e];              // infinite V scales become NaN; of tokens that not every row attends, at the end
                        if (!for_all(a, now.r, t * T + e * 32 + lane)) x.z = x.z < INFINITY ? x.z : 0.f, x.w = x.w < INFINITY ? x.w : 0.f;
                        float *ks = reinterpret_cast<float *>(sh.k_scales[m]), *vs = reinterpret_cast<float *>(sh.v_scales[m]);
                        const int tok = F8 ? e * 32 + lane : 0;
                        ks[tok] = x.x, vs[tok] = fmaf(x.z, 0.f, x.z) * cx;
                        if (SG == 2) ks[T + tok] = x.y, vs[T + tok] = fmaf(x.w, 0.f, x.w) * cy;
                    }
                    if (lane == 0) sh.top[m] = top;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.meta_full[m])), tree_waits.tiles = done + 1;
            }
        }
    } else if (warp >= C::load_warp) {
        // ================================================================ loads; codes -> f16
        const int wt = tid - C::work_warp * 32;
        constexpr int row_chunks = F8 ? D / 16 : D / 8;       // 16-byte chunks of a token's row
        const char *rows[2] = {static_cast<const char *>(a.k) + (int64_t)kvh * row_chunks * 16,
                               static_cast<const char *>(a.v) + (int64_t)kvh * row_chunks * 16};
        const int64_t pitch = (int64_t)a.Hkv * row_chunks * 16;
        // TMA: a box is a run of a page; a row that does not exist reads as zeros
        constexpr int blocks = row_chunks / 8;                // 128-byte blocks of a row
        const int rows_end = (int)min((int64_t)INT32_MAX, a.n_pages * a.page_size);
        const int boxes = tiled ? T / plan.run : 1, whole = boxes == 1 ? 1 : blocks, run = lane % boxes, block = lane / boxes;
        int asked[2] = {0, 0};                                // slots asked for, of each ring
        // a tile's K or V into the slot of turn q
        auto copy = [&](int is_v, int tile, int q) -> bool {
            const int m = tile % C::metas;
            if (!is_v && !wait_warp(&sh.meta_full[m], tile / C::metas)) return false;
            const int box = sh.slots[m][tiled ? run * plan.run : 0], y = box < 0 ? rows_end : box;
            // FP8 rows: rings of their own, by tiles; bf16 rows: one, by turns
            const int slots = F8 ? (is_v ? C::v_ring : C::k_ring) : RING, x = F8 ? tile : q, at = x % slots, turn = x / slots;
            uint64_t *full = F8 ? (is_v ? &sh.v_full[F8 ? at : 0] : &sh.k_full[F8 ? at : 0]) : &sh.full[F8 ? 0 : at];
            if (turn > 0 && !wait_warp(F8 ? (is_v ? &sh.v_empty[F8 ? at : 0] : &sh.k_empty[F8 ? at : 0]) : &sh.empty[F8 ? 0 : at], turn - 1))
                return false;
            const uint32_t dst = F8 ? q_at + (is_v ? C::v_at : C::k_at) + at * C::code_slot : ring_at + at * C::slot;
            if (tiled) {
                asked[F8 ? is_v : 0] = x + 1;
                if (lane == 0) mbar_arrive_expect_tx(smem_u32(full), F8 ? C::code_slot : C::slot);
                __syncwarp();
                if (block < whole)
                    tma_load_3d(dst + block * (T * 128) + run * plan.run * 128, is_v ? &maps.v : &maps.k, 0, y, kvh * blocks + block,
                                smem_u32(full));
            } else {
#pragma unroll
                for (int i = 0; i < (T * row_chunks + C::workers - 1) / C::workers; ++i) {
                    const int id = i * C::workers + wt, tok = id / row_chunks, gr = id % row_chunks;
                    if (tok >= T) break;
                    const int sl = sh.slots[m][tok];
                    cp_async16_zfill(dst + gr / 8 * (T * 128) + swz(tok, gr & 7), rows[is_v] + max(sl, 0) * pitch + gr * 16, sl >= 0);
                }
                cp_async_arrive(smem_u32(full));
            }
            if (is_v) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.meta_empty[m]));
            }
            return true;
        };
        // The copies' walk: turn cc of the segment's 2 n. 0: K0; 2i - 1: K of tile i; 2i + 2: V of tile i; 2n - 1: the last V.
        Walk wc = walk;
        Seg gc{};
        int cc = 0, nc = 0;
        const bool loads = tiled ? warp == C::load_warp : warp >= C::work_warp;
        bool more = loads && wc.next(a, m_tile, gc);
        if (more) nc = 2 * (gc.tb - gc.ta);
        auto turn_is_v = [](int c, int turns) { return c == turns - 1 || (c > 0 && (c & 1) == 0); };
        auto turn_tile = [&](int c, int turns) { return c == 0 ? 0 : c == turns - 1 ? turns / 2 - 1 : turn_is_v(c, turns) ? c / 2 - 1 : (c + 1) / 2; };
        auto ask = [&]() -> bool {
            if (!more) return true;
            if (!copy(turn_is_v(cc, nc), gc.i0 + turn_tile(cc, nc), 2 * gc.i0 + cc)) return false;
            if (++cc == nc) {
                more = wc.next(a, m_tile, gc);
                cc = 0;
                nc = more ? 2 * (gc.tb - gc.ta) : 0;
            }
            return true;
        };
        bool ok = true;
        if (!F8 || warp == C::load_warp) {
#pragma unroll 1
            while (ok && more) ok = ask();
            // no load may still be writing shared memory when the CTA ends
            for (int x = 0; x < (F8 ? 2 : 1); ++x) {
                const int slots = F8 ? (x ? C::v_ring : C::k_ring) : RING;
                for (int q = max(0, asked[x] - slots); q < asked[x]; ++q)
                    wait_landed(smem_u32(F8 ? (x ? &sh.v_full[F8 ? q % slots : 0] : &sh.k_full[F8 ? q % slots : 0]) : &sh.full[F8 ? 0 : q % slots]),
                                (uint32_t)(q / slots) & 1u);
            }
        } else if constexpr (F8) {
            // Without TMA the codes of a turn are asked for `ahead` turns before its V, if it is one, is converted: at most as many as
            // the rings hold, which a turn that is asked for may have to wait for, and fewer than 2 metas - 1, since a tile's K is
            // asked for when the softmax has left the tile `metas` before it, and with it when that tile's V has been converted.
            constexpr int ahead = D == 256 ? 2 : 6;
            static_assert(ahead < 2 * C::metas - 1, "turns");
            // a thread's chunks of 16 codes, the same in every slot: chunk `gr` of token `tok`, and where its two granules go. The
            // second half of a token's chunks goes in the other order, to other banks than the first half's.
            constexpr int N = (T * row_chunks + C::workers - 1) / C::workers;
            uint32_t src[N], dst[N][2];
            int toks[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int id = i * C::workers + wt, tok = id / row_chunks, gr = id % row_chunks, at = (gr & 3) * 2, swap = gr >> 2 & 1;
                toks[i] = tok < T ? tok : -1;
                src[i] = gr / 8 * (T * 128) + swz(tok & (T - 1), gr & 7);
                dst[i][0] = gr / 4 * (T * 128) + swz(tok & (T - 1), at + swap);
                dst[i][1] = gr / 4 * (T * 128) + swz(tok & (T - 1), at + 1 - swap);
            }
            const bool swap = wt % row_chunks >> 2 & 1;   // the same for every chunk: C::workers is a multiple of row_chunks
            static_assert(C::workers % row_chunks == 0, "a thread keeps its chunk");
            auto convert = [&](int i, int j0, const TreeRow &r, bool some) -> bool {       // tile i's V
                // rows that nothing attends become zeros, and NaN codes of rows that not every row attends
                const int edge = a.window > 0 ? r.base + r.T - a.window : 0;
                if (!wait_warp(&sh.v_full[i % C::v_ring], i / C::v_ring)) return false;
                if (i >= RING && !wait_warp(&sh.empty[i % RING], i / RING - 1)) return false;
                const uint8_t *from = sm + C::v_at + i % C::v_ring * C::code_slot;
                uint8_t *to = sm + C::ring_at + i % RING * C::slot;
                constexpr int H = 3;                      // chunks at a time
#pragma unroll
                for (int n0 = 0; n0 < N; n0 += H) {
                    uint4 v[H];
#pragma unroll
                    for (int n = 0; n < H; ++n)
                        if (n0 + n < N) v[n] = *reinterpret_cast<const uint4 *>(from + src[n0 + n]);
                    if (some)
#pragma unroll
                        for (int n = 0; n < H; ++n) {
                            if (n0 + n >= N) break;
                            const int j = j0 + toks[n0 + n];
                            if ((uint32_t)j >= (uint32_t)r.len || j < r.lo)
                                v[n] = make_uint4(0, 0, 0, 0);
                            else if (j >= r.base || j < edge)
                                drop_nan_codes(v[n].x), drop_nan_codes(v[n].y), drop_nan_codes(v[n].z), drop_nan_codes(v[n].w);
                        }
#pragma unroll
                    for (int n = 0; n < H; ++n) {
                        if (n0 + n >= N || toks[n0 + n] < 0) break;
                        const uint4 x = swap ? make_uint4(v[n].z, v[n].w, v[n].x, v[n].y) : v[n];
                        *reinterpret_cast<uint4 *>(to + dst[n0 + n][0]) =
                            make_uint4(e4m3_to_f16x2(x.x, 0), e4m3_to_f16x2(x.x, 1), e4m3_to_f16x2(x.y, 0), e4m3_to_f16x2(x.y, 1));
                        *reinterpret_cast<uint4 *>(to + dst[n0 + n][1]) =
                            make_uint4(e4m3_to_f16x2(x.z, 0), e4m3_to_f16x2(x.z, 1), e4m3_to_f16x2(x.w, 0), e4m3_to_f16x2(x.w, 1));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();                             // an arrival for each warp: 192 of them on one word take hundreds of cycles
                if (lane == 0) mbar_arrive(smem_u32(&sh.full[i % RING])), mbar_arrive(smem_u32(&sh.v_empty[i % C::v_ring]));
                return true;
            };
            Walk w = walk;
            for (int i = 0; i < ahead && ok; ++i) ok = ask();
            while (ok && w.next(a, m_tile, g)) {
                const int turns = 2 * (g.tb - g.ta);
                for (int c = 0; c < turns && ok; ++c) {
                    const int t = g.ta + turn_tile(c, turns);
                    ok = ask();
                    if (ok && turn_is_v(c, turns)) ok = convert(g.i0 + turn_tile(c, turns), t * T, g.r, masked(a, g.r, t));
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= C::q_warp) {
        // ================================================================ queries, ancestors, clean V rows
        const int qt = tid - C::q_warp * 32;
        Walk w = walk;
        bool bad = false;                                 // a wait in vain: up to the next barrier, where all of these warps leave
        int seg = 0, cleaned = 0;
        while (w.next(a, m_tile, g)) {
            const int n = g.tb - g.ta, rows = g.r.T * a.G - m_tile * kRows;     // this CTA's rows (maybe more than 128)
            bad = bad || (seg > 0 && !wait_warp(&sh.q_free, seg - 1));
            if (meet_any(2, C::q_threads, bad)) break;
            auto row_at = [&](int r) -> const uint16_t * {
                const int node = (m_tile * kRows + r) / a.G, h = (m_tile * kRows + r) % a.G;
                return a.q + (int64_t)(g.r.off + node) * a.q_ld + (kvh * a.G + h) * D;
            };
            if constexpr (!F8) {
                // a row each thread, into its lane of tensor memory (a warp reaches the lanes of its number modulo 4)
                const int r = 32 * (warp & 3) + lane;
                const uint32_t dst = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::t_q;
                const uint16_t *src = r < rows ? row_at(r) : nullptr;
#pragma unroll
                for (int c0 = 0; c0 < D / 2; c0 += 32) {          // 32 columns are 64 dims
                    uint32_t x[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (src) v = *reinterpret_cast<const uint4 *>(src + 2 * c0 + 8 * k);
                        x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
                    }
                    __syncwarp();
                    tmem_st32(dst + c0, x);
                }
                tc_fence_before();
            } else {
                // D / 16 lanes have a row, 16 values each, four rows on their way. Rows without a token keep the codes that are there,
                // which reach no other row.
                constexpr int each = C::q_threads / (D / 16), U = 4;
                static_assert(kRows % (U * each) == 0, "rows");
                const int gr = qt % (D / 16);
                for (int r = qt; r < kRows; r += C::q_threads)
                    if (r >= rows) sh.q_scale[seg & 1][r] = 0.f;
#pragma unroll 1
                for (int i = qt / (D / 16); i - qt / (D / 16) < min(rows, kRows); i += U * each) {
                    uint4 v[U][2];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool in = i + u * each < rows;
                        const uint4 *from = reinterpret_cast<const uint4 *>(row_at(in ? i + u * each : 0) + gr * 16);
                        v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
                        if (in) v[u][0] = from[0], v[u][1] = from[1];
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int r = i + u * each;
                        float f[2][8], top = 0.f;
                        unpack8(v[u][0], f[0]), unpack8(v[u][1], f[1]);
#pragma unroll
                        for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(f[k >> 3][k & 7]));
#pragma unroll
                        for (int o = D / 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        // the largest becomes 2^7 .. 2^8; an infinite one makes the row NaN, not E4M3's largest value
                        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -119), 126);
                        const float down = top == INFINITY ? NAN : __uint_as_float((uint32_t)(134 - e) << 23);
                        uint32_t part[2][4] = {};
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float x = f[k >> 2][2 * k & 7] * down, y = f[k >> 2][(2 * k & 7) + 1] * down;
                            const uint32_t c = e4m3x2_of(x, y), back = e4m3_to_f16x2(c, 0);
                            const float2 near = __half22float2(*reinterpret_cast<const __half2 *>(&back));
                            part[0][k >> 1] |= c << (16 * (k & 1));
                            part[1][k >> 1] |= e4m3x2_of(x - near.x, y - near.y) << (16 * (k & 1));
                        }
                        // first parts, then second ones; 128 dims are a block of 128 bytes
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(q_at + (z * SG + gr / 8) * (kRows * 128) + swz(r, gr & 7)),
                                         "r"(part[z][0]), "r"(part[z][1]), "r"(part[z][2]), "r"(part[z][3])
                                         : "memory");
                        if (gr == 0 && r < rows) sh.q_scale[seg & 1][r] = __uint_as_float((uint32_t)(120 + e) << 23);
                    }
                }
                fence_proxy_async_smem();
            }
            mbar_arrive(smem_u32(&sh.q_full));
            // ---- the drafted tokens' ancestors, once the last segment's are no longer needed
            if (meet_any(2, C::q_threads, seg > 0 && !wait_warp(&sh.nodes_free, seg - 1))) break;
            for (int i = qt; i < g.r.T; i += C::q_threads) {
                uint32_t kin[4] = {0u, 0u, 0u, 0u};
                int depth = 0;
                for (int j = i; j >= 0;) {                // parents lie below their children, so this ends
                    if (a.window == 0 || depth < a.window)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (j >> 5 == x) kin[x] |= 1u << (j & 31);
                    ++depth;
                    int p = a.parent[g.r.off + j];
                    if (p < -1 || p >= j) {
                        if (speaks) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereTree, g.s);
                        p = -1;
                    }
                    j = p;
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) sh.kin[i][x] = kin[x];
                sh.lo[i] = a.window > 0 ? max(0, g.r.base + depth - a.window) : 0;
            }
            if (qt < 8) sh.odd[qt >> 2][qt & 3] = 0u;
            mbar_arrive(smem_u32(&sh.nodes_full));
            asm volatile("bar.sync 2, %0;" ::"n"(C::q_threads) : "memory");        // the flags are cleared
            // ---- V rows that not every row attends
            const int edge = a.window > 0 ? g.r.base + g.r.T - a.window : 0;       // places below it: not for all
            auto flag = [&](int j) {
                const int x = j >= g.r.base ? j - g.r.base : j - g.r.lo, set = j >= g.r.base ? 0 : 1;
                if (x < QSA_MAX_DRAFT) atomicOr(&sh.odd[set][x >> 5], 1u << (x & 31));
            };
            for (int c = 0; c < n; ++c) {
                const int t = g.ta + c;
                if (!masked(a, g.r, t)) continue;
                if (!F8) {
                    // the output warp says when the rows are in: it meets every turn of its slots, and a wait tells only two from each other
                    bad = !wait_warp(&sh.to_clean, cleaned);
                    if (bad) break;
                    const int at = (2 * g.i0 + v_turn(c, n)) % RING;
                    for (int i = qt; i < T * (D / 8); i += C::q_threads) {
                        const int tok = i / (D / 8), gr = i % (D / 8), j = t * T + tok;
                        const bool out = (uint32_t)j >= (uint32_t)g.r.len || j < g.r.lo;
                        if (!out && j < g.r.base && j >= edge) continue;
                        uint4 *p = reinterpret_cast<uint4 *>(sm + C::ring_at + at * C::slot + gr / 8 * (T * 128) + swz(tok, gr & 7));
                        if (out) {
                            *p = make_uint4(0, 0, 0, 0);
                        } else {
                            uint4 v = *p;
                            if (drop_odd(v)) {
                                *p = v;
                                flag(j);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(smem_u32(&sh.clean));
                    ++cleaned;
                } else {
                    // the workers clean; the tokens to add at the end are found in the cache
                    for (int i = qt; i < T * (D / 16); i += C::q_threads) {
                        const int tok = i / (D / 16), gr = i % (D / 16), j = t * T + tok;
                        if ((uint32_t)j >= (uint32_t)g.r.len || j < g.r.lo || (j < g.r.base && j >= edge)) continue;
                        const int pg = a.table[g.s * a.ld + j / a.page_size];
                        if ((uint32_t)pg >= (uint32_t)a.n_pages) continue;
                        const int64_t row = ((int64_t)pg * a.page_size + j % a.page_size) * a.Hkv + kvh;
                        uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.v) + row * D + gr * 16);
                        if (drop_nan_codes(v.x) | drop_nan_codes(v.y) | drop_nan_codes(v.z) | drop_nan_codes(v.w) | !isfinite(a.v_scales[row * SG + gr / 8]))
                            flag(j);
                    }
                }
            }
            if (!bad) mbar_arrive(smem_u32(&sh.flags_full));
            ++seg;
        }
    } else if (warp == C::s_warp) {
        // ================================================================ scores
        // The warp stays together and one elected lane issues: addresses and descriptors are then the warp's, not a lane's, which
        // the instruction wants them to be.
        Walk w = walk;
        int seg = 0, i = 0;
        bool ok = true;
        for (; ok && w.next(a, m_tile, g); ++seg) {
            const int n = g.tb - g.ta;
            if (!wait_warp(&sh.q_full, seg)) break;
#pragma unroll 1
            for (int c = 0; c < n && ok; ++c, ++i) {
                // the buffer's last weights are used up
                if (i >= NB && !wait_warp(&sh.pv_done[i % NB], i / NB - 1)) {
                    ok = false;
                    break;
                }
                const uint32_t s_at = tmem + C::t_s + (i % NB) * C::s_cols;
                const int q = F8 ? i : 2 * g.i0 + k_turn(c), slots = F8 ? C::k_ring : RING, at = q % slots;
                uint64_t *full = F8 ? &sh.k_full[F8 ? at : 0] : &sh.full[F8 ? 0 : at];
                if (!wait_warp(full, q / slots)) {
                    ok = false;
                    break;
                }
                if (!tiled) fence_proxy_async_smem();                 // rows by cp.async; TMA needs none
                tc_fence_after();
                const uint64_t bd = tc_desc(F8 ? q_at + C::k_at + at * C::code_slot : ring_at + at * C::slot, 16, 1024), ad = tc_desc(q_at, 16, 1024);
                if (elect_one()) {
                    if constexpr (!F8) {
#pragma unroll
                        for (int z = 0; z < D / 16; ++z)              // 16 dims: 32 bytes on, or in the next block of 64
                            tc_mma_ta(s_at, tmem + C::t_q + z * 8, bd + (z >> 2) * (T * 128 / 16) + (z & 3) * 2, tc_idesc(kRows, T, 0), z > 0);
                        tc_commit(smem_u32(&sh.empty[at]));
                    } else {
                        // codes as they are; 32 dims: 32 bytes on; first and second parts of q into the same sums, for each 128 dims
#pragma unroll
                        for (int x = 0; x < SG; ++x)
#pragma unroll
                            for (int z = 0; z < 8; ++z)
                                mma_e4m3(s_at + x * T, ad + ((z >> 2) * SG + x) * (kRows * 128 / 16) + (z & 3) * 2,
                                         bd + x * (T * 128 / 16) + (z & 3) * 2, f16_idesc(T, 0), z > 0);
                        tc_commit(smem_u32(&sh.k_empty[at]));
                    }
                    tc_commit(smem_u32(&sh.s_full[i % NB]));
                    if (c + 1 == n) tc_commit(smem_u32(&sh.q_free));
                }
                __syncwarp();
            }
        }
        // the last commit covers every product issued: wait for it before tensor memory is freed
        if (i > 0 && lane == 0) wait_landed(smem_u32(&sh.s_full[(i - 1) % NB]), (uint32_t)((i - 1) / NB) & 1u);
    } else if (warp == C::o_warp) {
        // ================================================================ O (+)= P V
        Walk w = walk;
        int seg = 0, cleaned = 0, i = 0;
        bool ok = true;
        for (; ok && w.next(a, m_tile, g); ++seg) {
            const int n = g.tb - g.ta;
#pragma unroll 1
            for (int c = 0; c < n && ok; ++c, ++i) {
                const int q = F8 ? i : 2 * g.i0 + v_turn(c, n), at = q % RING;
                const bool part = !F8 && masked(a, g.r, g.ta + c);
                if (part) {
                    ok = wait_warp(&sh.full[at], q / RING);
                    if (lane == 0) mbar_arrive(smem_u32(&sh.to_clean));
                }
                if (!ok || !wait_warp(&sh.p_full[i % NB], i / NB) || (c == 0 && seg > 0 && !wait_warp(&sh.o_free, seg - 1)) ||
                    !wait_warp(part ? &sh.clean : &sh.full[at], part ? cleaned++ : q / RING)) {
                    ok = false;
                    break;
                }
                if (!F8 && !tiled) fence_proxy_async_smem();
                tc_fence_after();
                const uint32_t p_at = tmem + C::t_s + (i % NB) * C::s_cols;
                const uint64_t bd = tc_desc(ring_at + at * C::slot, T * 128, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int z = 0; z < T / 16; ++z)                  // 16 tokens are 2,048 bytes; each set of weights has its 128 dims
#pragma unroll
                        for (int x = 0; x < SG; ++x)
                            tc_mma_ta(tmem + C::t_o + x * 128, p_at + x * (T / 2) + z * 8, bd + z * 128 + x * (2 * T * 128 / 16),
                                      F8 ? f16_idesc(128, 1) : tc_idesc(kRows, D, 1), c > 0 || z > 0);
                    tc_commit(smem_u32(&sh.empty[at]));
                    tc_commit(smem_u32(&sh.pv_done[i % NB]));
                }
                __syncwarp();
            }
        }
        if (i > 0 && lane == 0) wait_landed(smem_u32(&sh.pv_done[(i - 1) % NB]), (uint32_t)((i - 1) / NB) & 1u);
    } else {
        // ================================================================ softmax
        // A row has two threads, each for half of a tile's tokens and half of O's columns, in warps that reach the same quarter of
        // the lanes; they exchange the maxima of a tile, and their sums at the end.
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const uint32_t t_row = tmem + ((uint32_t)(32 * quarter) << 16), t_o = t_row + C::t_o;
        auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(4 + quarter) : "memory"); };
        // They leave together: one that waits in vain comes to their next exchange all the same, and gives a NaN there that no
        // arithmetic gives. (A wait in vain carried in a register up to a barrier.red: FP8 rows of 256 dims 307 us, 292 so.)
        constexpr uint32_t gone = 0xFFC00001u;
        Walk w = walk;
        int seg = 0;
        int out = -1;                                     // the tile whose exchange it is; -2: the other has told
        for (; w.next(a, m_tile, g); ++seg) {
            const int n = g.tb - g.ta;
            const int node = (m_tile * kRows + row) / a.G, head = kvh * a.G + (m_tile * kRows + row) % a.G;
            const bool valid = node < g.r.T, some = __any_sync(0xffffffffu, valid);
            if (!wait_warp(&sh.nodes_full, seg)) {
                out = g.i0;
                break;
            }
            const int lo = sh.lo[min(node, g.r.T - 1)];
            // above zero: a masked token's -infinity times it stays one (queries of zeros have the scale 2^-126)
            const float scale = F8 ? fmaxf(a.scale_log2 * sh.q_scale[seg & 1][F8 ? row : 0], __uint_as_float(1u)) : a.scale_log2;
            float ref = -INFINITY, l = 0.f;               // the lazy maximum, and this thread's weights' sum relative to it
            float2 unit = make_float2(0.f, 0.f);          // FP8: O is in units of these over 2^kRaise
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
                const int i = g.i0 + c, t = g.ta + c, m = i % C::metas;
                if (!wait_warp(&sh.meta_full[m], i / C::metas)) {
                    out = i;
                    break;
                }
                // which of this half's tokens the row attends
                uint32_t see = sh.real[m][half];
                if (masked(a, g.r, t)) {
                    const int j = t * T + 32 * half, from = lo - j, to = g.r.base - j;
                    uint32_t v = to >= 32 ? ~0u : to > 0 ? (1u << to) - 1u : 0u;
                    if (from >= 32)
                        v = 0u;
                    else if (from > 0)
                        v &= ~0u << from;
                    const int o = -to;                    // place of bit 0 among the drafts
                    if (o > -32 && o < QSA_MAX_DRAFT && valid) {
                        if (o < 0) {
                            v |= sh.kin[node][0] << -o;
                        } else {
                            v |= sh.kin[node][o >> 5] >> (o & 31);
                            if ((o & 31) && (o >> 5) < QSA_MAX_DRAFT / 32 - 1) v |= sh.kin[node][(o >> 5) + 1] << (32 - (o & 31));
                        }
                    }
                    see &= v;
                }
                const bool all = __all_sync(0xffffffffu, see == ~0u || !valid);        // no token to mask in this warp
                if (!wait_warp(&sh.s_full[i % NB], i / NB)) {
                    out = i;
                    break;
                }
                tc_fence_after();
                const uint32_t t_s = t_row + C::t_s + (i % NB) * C::s_cols;
                float f = 1.f;
                const float2 was = unit;
                if (F8) unit = sh.top[m];
                if (some) {
                    float v[32];
                    tmem_ld32(t_s + 32 * half, v);
                    if constexpr (F8) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 s4 = sh.k_scales[m][0][half * 8 + k];
                            set2(v, 2 * k, mul2(get2(v, 2 * k), make_float2(s4.x, s4.y)));
                            set2(v, 2 * k + 1, mul2(get2(v, 2 * k + 1), make_float2(s4.z, s4.w)));
                        }
                        if constexpr (SG == 2) {
#pragma unroll
                            for (int k0 = 0; k0 < 8; k0 += 4) {       // all at once, registers spilled: 351 us, 307 so
                                float u[16];
                                tmem_ld16(t_s + 64 + 32 * half + 4 * k0, u);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float4 s4 = sh.k_scales[m][1][half * 8 + k0 + k];
                                    const int at = 2 * (k0 + k);
                                    set2(v, at, fma2(get2(u, 2 * k), make_float2(s4.x, s4.y), get2(v, at)));
                                    set2(v, at + 1, fma2(get2(u, 2 * k + 1), make_float2(s4.z, s4.w), get2(v, at + 1)));
                                }
                            }
                        }
                    }
                    if (!all)
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = (see >> k) & 1u ? v[k] : -INFINITY;
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 32; ++k) mx[k & 3] = fmaxf(mx[k & 3], v[k]);
                    const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                    sh.tops[i & 1][half][row] = mine;
                    meet();                               // both halves have read their scores, too
                    const float theirs = sh.tops[i & 1][half ^ 1][row];
                    if (__float_as_uint(theirs) == gone) {
                        out = -2;
                        break;
                    }
                    const float top = fmaxf(mine, theirs);
                    if (top > ref + kLazy) {
                        if (ref != -INFINITY) f = ex2(ref - top);
                        ref = top;
                    }
                    const float at = ref == -INFINITY ? 0.f : ref;
                    float2 ps[2] = {};
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 e = fma2(get2(v, k), make_float2(scale, scale), make_float2(-at, -at));
                        set2(v, k, make_float2(ex2(e.x), ex2(e.y)));
                        ps[k & 1] = add2(ps[k & 1], get2(v, k));
                    }
                    l = fmaf(l, f, (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y));
                    if constexpr (!F8) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) pk[k] = bf16x2(v[2 * k], v[2 * k + 1]);
                        tmem_st16(t_s + 16 * half, pk);   // over scores that have been read
                    } else {
#pragma unroll
                        for (int x = 0; x < SG; ++x) {
                            uint32_t pk[16];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float4 s4 = sh.v_scales[m][x][half * 8 + k];
                                const float2 w0 = mul2(get2(v, 2 * k), make_float2(s4.x, s4.y));
                                const float2 w1 = mul2(get2(v, 2 * k + 1), make_float2(s4.z, s4.w));
                                pk[2 * k] = f16x2(w0.x, w0.y), pk[2 * k + 1] = f16x2(w1.x, w1.y);
                            }
                            tmem_st16(t_s + 32 * x + 16 * half, pk);
                        }
                    }
                }
                const bool turned = F8 && (was.x != unit.x || was.y != unit.y);
                if (c > 0 && __any_sync(0xffffffffu, f != 1.f || turned)) {       // O follows, once the product before it is done
                    if (!wait_warp(&sh.pv_done[(i - 1) % NB], (i - 1) / NB)) {
                        out = i + 1;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                        float v[32];
                        const float by = !F8 ? f : c0 < 128 ? f * (was.x / unit.x) : f * (was.y / unit.y);
                        tmem_ld32(t_o + c0, v);
#pragma unroll
                        for (int k = 0; k < 16; ++k) set2(v, k, mul2(get2(v, k), make_float2(by, by)));
                        tmem_st32(t_o + c0, v);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[i % NB])), mbar_arrive(smem_u32(&sh.meta_empty[m]));
            }
            if (out != -1) break;
            // ---- the segment's end: out, or a partial
            const int i = g.i0 + n - 1;
            if (!wait_warp(&sh.pv_done[i % NB], i / NB) || !wait_warp(&sh.flags_full, seg)) {
                out = i + 1;
                break;
            }
            tc_fence_after();
            if (some) {
                sh.tops[(i & 1) ^ 1][half][row] = l;      // the sums, where the maxima two tiles back were
                meet();
                const float theirs = sh.tops[(i & 1) ^ 1][half ^ 1][row];
                if (__float_as_uint(theirs) == gone) break;
                l = half == 0 ? l + theirs : theirs + l;
                meet();
                const bool whole = g.begins && g.ends;
                const float by = l == 0.f ? 0.f : (whole ? 1.f / l : 1.f) * (F8 ? 1.f / (1 << (int)kRaise) : 1.f);
                // values that are not finite, of attended tokens that not every row attends
                bool strange = false;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    strange |= valid && ((sh.odd[0][x] & sh.kin[min(node, QSA_MAX_DRAFT - 1)][x]) | sh.odd[1][x]) != 0u;
                const int64_t at = (int64_t)(2 * range + (g.begins ? 1 : 0)) * a.Hkv * plan.m_tiles + kvh * plan.m_tiles + m_tile;
                float *po = ws.o + (at * kRows + row) * D;
                uint16_t *dst = a.out + ((int64_t)(g.r.off + min(node, g.r.T - 1)) * a.Hq + head) * D;
#pragma unroll 1
                for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                    float v[32];
                    const float times = !F8 ? by : by * (c0 < 128 ? unit.x : unit.y);
                    __syncwarp();
                    tmem_ld32(t_o + c0, v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = l == 0.f ? 0.f : v[k] * times;
                    if (valid && whole) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4 *>(dst + c0 + 8 * k) =
                                make_uint4(bf16x2(v[8 * k], v[8 * k + 1]), bf16x2(v[8 * k + 2], v[8 * k + 3]),
                                           bf16x2(v[8 * k + 4], v[8 * k + 5]), bf16x2(v[8 * k + 6], v[8 * k + 7]));
                    } else if (valid) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4 *>(po + c0 + 4 * k) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    }
                }
                if (strange) add_odd<D, F8>(a, g, sh.odd, sh.kin[node], lo, kvh, half * (D / 2), whole, dst, po);
                if (valid && half == 0) {
                    if (!whole)
                        ws.ml[at * kRows + row] = make_float2(ref, l);
                    else if (a.lse)
                        a.lse[(int64_t)(g.r.off + node) * a.Hq + head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.o_free)), mbar_arrive(smem_u32(&sh.nodes_free));
        }
        if (out >= 0) {                                   // segments without rows in this quarter have no exchange
            bool more = true;
            while (more && m_tile * kRows + 32 * quarter >= g.r.T * a.G) more = w.next(a, m_tile, g), out = g.i0;
            if (more) {
                sh.tops[out & 1][half][row] = __uint_as_float(gone);
                meet();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::s_warp) tmem_dealloc(tmem, 512);
}

// The partials of the sequences that a range starts and leaves unfinished, joined. A CTA takes every gridDim.y-th pair of rows
// of the y-th such range; D / 4 threads have a row, `Groups` of them every Groups-th partial, merged in order at the end. CTAs for
// single rows, 8,000 of them for 32 sequences of 16 drafted tokens, took longer to begin than to read their partials.
constexpr int kJoinThreads = 256;
template <int D, int Groups>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeArgs a, TreePlan plan, TreeScratch ws) {
    constexpr int cols = D / 4, Rows = kJoinThreads / cols / Groups, U = 4;
    static_assert(Rows >= 1, "a row");
    __shared__ float4 acc[Groups > 1 ? kJoinThreads : 1];
    __shared__ float2 pair[kJoinThreads / cols];
    __shared__ int4 job_sh;
    const int tid = threadIdx.x, col = tid % cols, group = tid / cols % Groups, sub = tid / cols / Groups;
    wait_for_previous();
    if (tid < 32) {
        if (tid == 0) job_sh.x = -1;
        __syncwarp();
        int n = 0;
        for (int r0 = 0; r0 < plan.ranges - 1; r0 += 32) {
            const int r = r0 + tid;
            const int2 meta = r < plan.ranges - 1 ? __ldcg(ws.meta + r) : make_int2(-1, 0);
            const uint32_t some = __ballot_sync(0xffffffffu, meta.x >= 0);
            if (meta.x >= 0 && n + __popc(some & ((1u << tid) - 1u)) == (int)blockIdx.x) job_sh = make_int4(r, meta.x, meta.y, 0);
            n += __popc(some);
        }
    }
    __syncthreads();
    const int4 job = job_sh;
    if (job.x < 0) return;
    const int off = a.draft_off[job.y], T = a.draft_off[job.y + 1] - off;
    // rows: (KV head, drafted token, query head of the KV head)
    const int per = T * a.G, rows = per * a.Hkv;
    const int64_t C = (int64_t)a.Hkv * plan.m_tiles;
    for (int id0 = blockIdx.y * Rows; id0 < rows; id0 += gridDim.y * Rows) {
        const int id = min(id0 + sub, rows - 1), kvh = id / per, r = id % per;
        const int64_t at = (int64_t)kvh * plan.m_tiles + r / kRows;
        float m = -INFINITY, l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = group; i0 < job.z; i0 += U * Groups) {
            float2 ml[U];
            float4 o[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * Groups;
                ml[u] = make_float2(-INFINITY, 0.f);
                o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < job.z) {
                    const int64_t p = (part_slot(job.x, i) * C + at) * kRows + r % kRows;
                    ml[u] = __ldcg(ws.ml + p);
                    o[u] = __ldcg(reinterpret_cast<const float4 *>(ws.o + p * D + 4 * col));
                }
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
            const float ref = top == -INFINITY ? 0.f : top, old = ex2(m - ref);
            m = top;
            l *= old;
            x.x *= old, x.y *= old, x.z *= old, x.w *= old;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = ex2(ml[u].x - ref);
                l = fmaf(w, ml[u].y, l);
                x.x = fmaf(w, o[u].x, x.x), x.y = fmaf(w, o[u].y, x.y);
                x.z = fmaf(w, o[u].z, x.z), x.w = fmaf(w, o[u].w, x.w);
            }
        }
        if (Groups > 1) {
            __syncthreads();                              // the row before has been merged
            acc[tid] = x;
            if (col == 0) pair[tid / cols] = make_float2(m, l);
            __syncthreads();
            if (group > 0) continue;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < Groups; ++i) top = fmaxf(top, pair[sub * Groups + i].x);
            const float ref = top == -INFINITY ? 0.f : top;
            l = 0.f, m = top;
            x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < Groups; ++i) {
                const float w = ex2(pair[sub * Groups + i].x - ref);
                const float4 v = acc[tid + i * cols];
                l = fmaf(w, pair[sub * Groups + i].y, l);
                x.x = fmaf(w, v.x, x.x), x.y = fmaf(w, v.y, x.y), x.z = fmaf(w, v.z, x.z), x.w = fmaf(w, v.w, x.w);
            }
        }
        if (id0 + sub >= rows) continue;
        const int64_t to = (int64_t)(off + r / a.G) * a.Hq + kvh * a.G + r % a.G;
        const float f = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<uint2 *>(a.out + to * D + 4 * col) = make_uint2(bf16x2(x.x * f, x.y * f), bf16x2(x.z * f, x.w * f));
        if (col == 0 && a.lse) a.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

constexpr int kMaxCtas = 160;

int m_tiles_of(int G, int max_draft) { return (max_draft * G + kRows - 1) / kRows; }

TreeScratch tree_scratch(char *w, int D, int Hkv, int m_tiles) {
    const size_t parts = 2 * (size_t)std::max(1, kMaxCtas / (Hkv * m_tiles)) * Hkv * m_tiles * kRows;
    TreeScratch s;
    s.meta = reinterpret_cast<int2 *>(w);
    s.ml = reinterpret_cast<float2 *>(w + kMaxCtas * sizeof(int2));
    s.o = reinterpret_cast<float *>(w + kMaxCtas * sizeof(int2) + parts * sizeof(float2));
    return s;
}

// SMs of the current device (cached per device; 0 on an error).
template <typename C>
int sms() {
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cached[dev] == 0) {
        int n = 0;
        if (cudaFuncSetAttribute(tree_tile_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        cached[dev] = std::min(n, kMaxCtas);
    }
    return cached[dev];
}

template <int D, bool F8, bool Tiled>
cudaError_t launch_as(const TreeArgs &a, int run, cudaStream_t st) {
    using C = TreeCfg<D, F8, Tiled>;
    const int ctas = sms<C>();
    if (ctas == 0) {
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    }
    TreePlan plan{};
    // The M tiles that max_draft may need: the host does not know the drafts that there are, and CTAs of M tiles without rows have
    // nothing to do. 4 drafts in each of 32 sequences of 32,768 tokens, 8 heads a KV head, 2 KV heads: 363 us with max_draft 4, 365
    // with 16, 416 with 32, 791 with 64, 1,635 with 128.
    plan.m_tiles = m_tiles_of(a.G, a.max_draft);
    plan.ranges = std::max(1, ctas / (a.Hkv * plan.m_tiles));
    // the least length of a part: one sequence of 4,096 tokens took 19.9, 19.2, 20.6 and 24.0 us with 1, 2, 4 and 8 tiles
    plan.min_tiles = 2;
    plan.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    TreeMaps maps;
    memset(&maps, 0, sizeof(maps));
    const int64_t rows = a.n_pages * a.page_size;
    if (Tiled) {
        plan.run = run;
        const uint64_t row = (uint64_t)a.Hkv * D * (F8 ? 1 : 2);
        const uint32_t blocks = run == kTile ? D * (F8 ? 1 : 2) / 128 : 1;
        if (!encode_tmap_rows(&maps.k, a.k, F8, rows, row / 128, row, run, blocks) ||
            !encode_tmap_rows(&maps.v, a.v, F8, rows, row / 128, row, run, blocks))
            return cudaErrorInvalidValue;
    }
    const TreeScratch ws = tree_scratch(a.scratch, D, a.Hkv, plan.m_tiles);
    const dim3 grid((unsigned)(plan.ranges * a.Hkv * plan.m_tiles));
    const cudaError_t e = launch_dependent(tree_tile_kernel<C>, grid, C::threads, C::smem, st, a, plan, ws, maps);
    if (e != cudaSuccess || plan.ranges == 1) return e;               // one range cuts no sequence
    // as many CTAs as fit at once; few rows have many partials each, and more threads for a row
    const int64_t jobs = std::min(plan.ranges - 1, a.B), most = (int64_t)a.max_draft * a.Hq;
    const int groups = kJoinThreads / (D / 4);
    const bool few = jobs * most <= 152 * 8;
    const int64_t each = few ? 1 : groups / 2;
    const dim3 join((unsigned)jobs, (unsigned)std::max<int64_t>(1, std::min((most + each - 1) / each, 152 * 8 / jobs)));
    return few ? launch_dependent(tree_join_kernel<D, kJoinThreads / (D / 4)>, join, kJoinThreads, 0, st, a, plan, ws)
               : launch_dependent(tree_join_kernel<D, 2>, join, kJoinThreads, 0, st, a, plan, ws);
}

template <int D, bool F8>
cudaError_t launch(const TreeArgs &a, cudaStream_t st) {
    // Tiled loads of runs of a page. 32 sequences of 4,096 to 32,768 tokens, 256 dims: bf16 rows in runs of 32 and 16 tokens 247 and 273 us,
    // by cp.async 273; FP8 rows, whose workers convert as well, in runs of 16, 8 and 4 tokens 279, 337 and 451, by cp.async 384 to 401.
    const int run = std::min(a.page_size & -a.page_size, kTile);
    return run >= (F8 ? 8 : 16) && a.n_pages > 0 ? launch_as<D, F8, true>(a, run, st) : launch_as<D, F8, false>(a, 0, st);
}

}  // namespace

size_t tree_scratch_bytes(int D, int Hq, int Hkv, int max_draft) {
    const int m_tiles = m_tiles_of(Hq / Hkv, max_draft);
    const size_t parts = 2 * (size_t)std::max(1, kMaxCtas / (Hkv * m_tiles)) * Hkv * m_tiles * kRows;
    return kMaxCtas * sizeof(int2) + (kMaxCtas / (Hkv * m_tiles) > 1 ? parts * (sizeof(float2) + D * sizeof(float)) : 0);
}

cudaError_t launch_tree_decode(const TreeArgs &a, int D, bool fp8, cudaStream_t st) {
    switch (D) {
        case 64: return fp8 ? cudaErrorInvalidValue : launch<64, false>(a, st);
        case 128: return fp8 ? launch<128, true>(a, st) : launch<128, false>(a, st);
        case 256: return fp8 ? launch<256, true>(a, st) : launch<256, false>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qsa
