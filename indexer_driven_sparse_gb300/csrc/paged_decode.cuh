// Attention of one new token over a paged K/V cache (qsa_paged_decode, qsa_paged_decode_fp8kv):
//   out = sum_j softmax_j(scale q . K[j]) V[j] over the sequence's cached tokens, with their log-sum-exp.
//
// What bounds it: every K and V row is read once (2 Hkv rows a token) and used by the G <= 16 query heads of
// its KV head: 4 G flop per value read, a fiftieth of what the tensor cores do per byte of HBM. So the
// kernel is a stream of rows, and the work goes into keeping enough of them in flight.
//
// Split: the batch's tokens, cut into tiles of 64 or 128 of one sequence each, form one list; it is dealt to R ranges of
// equal length (R Hkv CTAs fill the GPU once), so a ragged batch is balanced whatever its lengths. CTA
// (range, KV head) walks its tiles through a ring of shared-memory stages filled by 16-byte cp.async. A
// sequence that a range boundary cuts leaves partials (m, l, O), joined by paged_join_kernel; all others are
// written at once. The two KV heads of a range are neighbouring CTAs, so a token's rows are read together.
//
// A tile's products run on mma.sync m16n8k16: M is the G heads padded to 16, which a 128-row tcgen05 tile would
// fill to an eighth. D / 32 warps. For S = Q K^T a warp takes its share of the tile's tokens; the warps exchange their
// maxima, each turns its own scores into weights P (in shared memory), and for O += P V each takes 32 dims of V and
// all tokens. Every warp keeps the same running maximum; the sum of the weights stays with the warp that formed
// them until a segment ends.
//   bf16 rows: P = P_hi + P_lo, two bf16 values (2^-16 of each weight): one bf16 would add as much error
//     as the result's own rounding. P_hi is rounded toward zero and P_lo is at least 2^-126: neither is then zero, or of
//     another sign than the weight, and an infinite V value stays that infinity instead of becoming inf - inf or 0 x inf
//     (it is NaN only where its weight underflows, 2^-126 of the largest).
//   FP8 rows: E4M3 codes are exact in f16. Q enters as f16 scaled by a power of two per head (exact down to 2^-17 of the head's
//     largest, below that off by at most 2^-25 of it: beneath the fp32 sum's own rounding); or, with 8 head rows of 256 dims, as
//     the sum of two E4M3 values and K's codes as they are (m16n8k32): the second parts take the M rows that would be
//     empty. Two E4M3 values hold bf16's 8 significant bits; the second, at most 2^-4 of the first, is scaled by
//     another 2^5, so that its step is 2^-21 of the head's largest value (values below 2^-14 of that are rounded by up to
//     2^-22 of it: a score by 2^-22 max |q| sum |k|). The K scales multiply the fp32 sums of each 128 dims. V's scales
//     enter the weights, w = 2^(s + log2 v_scale - m + 15) with m the running maximum of s + log2 v_scale (so that the
//     largest is 2^15), one set of weights for each 128 dims, rounded to f16: 2^-11 of each down to 2^-29 of the largest,
//     well under the rows' own 2^-4, and 2^-40 of the largest below that, so that a million tokens that are light
//     beside one still count. The softmax's sum is taken without v_scale, relative to the first set's m.
#pragma once

#include "paged.cuh"
#include "qsa_ptx.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace qsa {

namespace {

constexpr int kFewJoins = 152;           // CTAs of the join up to which they have 512 threads, one for each SM
constexpr int kMaxRanges = 640;

template <int D_, int GT_, bool F8_>
struct PagedCfg {
    static constexpr int D = D_, GT = GT_;          // GT: head rows kept (8 or 16)
    static constexpr bool F8 = F8_;
    static constexpr int warps = D / 32;            // that multiply
    // that load; 0: those that multiply do. 16-byte cp.async keep the load/store unit busy for 1,100 of a 64 KB tile's 2,800
    // cycles, so warps of their own issue them beside the products; they meet the others once a tile. Against loads by
    // the multiplying warps, 32 sequences of 20,000 tokens in FP8 rows of 256 dims: 114 against 135 us (8 head rows), 122 and
    // 142 (16); bf16 rows of 256 dims: 192 and 194.5, 512 sequences of 200 tokens 48 and 51, one of 16,384 tokens 12.7 and 13.1,
    // but of 4,096 6.6 and 6.5; of 64 dims with 16 head rows 108 and 114. At 128 dims two or three CTAs on an SM do that for
    // each other: FP8 rows take 211 us without loading warps and 222 with (8 KV heads, 8 head rows), 114 either way with 16.
    static constexpr int loaders = D == 128 ? 0 : D == 256 ? 4 : 2;
    // Q as two E4M3 values, K's codes multiplied as they are: 114 against 121 us over FP8 rows of 256 dims. At 128 dims the
    // products are not what the kernel waits for (217 against 213 us), and with 16 head rows, where no M rows are free
    // for the second parts, there are not the registers.
    static constexpr bool split = F8 && D == 256 && GT == 8;
    static constexpr int threads = (warps + loaders) * 32;
    static constexpr int tile = F8 ? 128 : 64;      // tokens
    static constexpr int row = D * (F8 ? 1 : 2);    // bytes of a K or V row
    static constexpr int chunks = row / 16;         // 16-byte chunks of a row
    static constexpr int rows_per_copy = 32 / chunks;
    static constexpr int warp_tok = tile / warps;   // tokens a warp scores
    static constexpr int load_warps = loaders ? loaders : warps, load_tok = tile / load_warps;   // tokens a warp loads
    static constexpr int groups = F8 ? D / 128 : 1; // scales of a row (FP8), sets of weights
    static constexpr int k_bytes = tile * row, s_bytes = F8 ? tile * groups * 4 : 0, q_bytes = GT * D * 2;
    static constexpr int stage = 2 * k_bytes + 2 * s_bytes;
    static constexpr int stages = F8 && D == 128 ? 2 : 3;
    static constexpr int ctas = D == 256 ? 1 : D == 128 ? (F8 ? 3 : 2) : (GT == 8 ? 4 : 3);   // per SM
    static constexpr int p_pitch = tile * 2 + 16;   // bytes between two heads' weights: an odd number of 16-byte chunks
    static constexpr int p_sets = F8 ? groups : 2;  // FP8: one per V scale; bf16: high and low parts
    // log2 of what the largest weight x V scale of FP8 rows becomes: f16 reaches 2^16, so the weights below its normal range
    // (2^-14) lie under 2^-29 of the largest, and only those under 2^-40 are lost
    static constexpr float raise = F8 ? 15.f : 0.f, lower = F8 ? 0x1p-15f : 1.f;
    static constexpr int q_at = stages * stage, p_at = q_at + (stages - 1) * q_bytes, x_at = p_at + p_sets * GT * p_pitch;
    static constexpr int smem = x_at + groups * GT * warps * 4;
};

// Workspace behind the status block: meta [kMaxRanges] {row, parts}, (m, l) and O of the partials; range r has slot
// 2r for the sequence it continues and 2r + 1 for the one it starts and leaves unfinished.
struct PagedScratch {
    int2 *meta;
    float2 *ml;     // [2 R][Hq]
    float *o;       // [2 R][Hq][D]
};

constexpr int max_ctas(int D) { return D == 256 ? 160 : D == 128 ? 480 : 640; }

__host__ __device__ inline int ranges_for(int ctas, int Hkv) { return ctas / Hkv > 0 ? ctas / Hkv : 1; }

// total tiles cut into R ranges: range r begins at floor(total r / R). In 32 bits where they suffice, and without a
// division where every range is one tile: a 64-bit division takes a quarter of a microsecond of a kernel whose shortest
// calls take three.
struct Ranges {
    long long total, each;
    int R, rest;
    __device__ __forceinline__ Ranges(long long total_, int R_) : total(total_), R(R_) {
        each = total == R ? 1 : total >> 32 ? total / R : (uint32_t)total / (uint32_t)R;
        rest = (int)(total - each * R);
    }
    __device__ __forceinline__ long long begin(int r) const {
        return rest == 0 ? each * r : each * r + (uint32_t)(rest * r) / (uint32_t)R;
    }
    // The range that holds tile x: the last r with begin(r) <= x, so total r < (x + 1) R.
    __device__ __forceinline__ int of(long long x) const {
        if (total == R) return (int)x;
        const long long y = (x + 1) * R - 1;
        return y >> 32 ? (int)(y / total) : (int)((uint32_t)y / (uint32_t)total);
    }
};

struct Row {
    int len, lo, t0, t1;    // tokens, first attended token, tiles [t0, t1)
};

template <int T>
__device__ __forceinline__ Row row_of(const PagedArgs &a, int s) {
    Row r;
    r.len = a.seq_len[s];
    if (r.len < 0 || r.len > a.ld * a.page_size) r.len = 0;
    r.lo = a.window > 0 ? max(0, r.len - a.window) : 0;
    r.t0 = r.lo / T;
    r.t1 = r.len > 0 ? r.len / T + (r.len % T != 0) : r.t0;
    return r;
}

// A place in the tile list: tile t of row s.
template <int T>
struct Cursor {
    int s, t;
    Row r;
    __device__ __forceinline__ void at(const PagedArgs &a, int row, int skip) {
        s = row;
        r = row_of<T>(a, s);
        t = r.t0 + skip;
    }
    __device__ __forceinline__ bool next(const PagedArgs &a) {   // never called behind the list's last tile; true: a new row
        if (++t < r.t1) return false;
        do {
            ++s;
            r = row_of<T>(a, s);
        } while (r.t1 == r.t0);
        t = r.t0;
        return true;
    }
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small_zfill(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(real ? N : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16832_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 codes (the low or the high half of w) -> f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w, int half) {
    uint32_t r;
    const uint16_t c = (uint16_t)(half ? w >> 16 : w & 0xFFFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_toward_zero(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Partials in order: the first from range r's slot 2r + 1, the others from the slots 2r of the ranges behind it.
__device__ __forceinline__ int64_t part_slot(int range, int i) { return i == 0 ? 2 * (int64_t)range + 1 : 2 * ((int64_t)range + i); }

// (m, l, 4 dims of O) joined over the partials first, first + step, ... < n.
template <int D, int U>
__device__ __forceinline__ void join_parts(const PagedArgs &a, const PagedScratch &ws, int range, int n, int head, int col,
                                           int first, int step, float &m, float &l, float4 &x) {
    m = -INFINITY, l = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = first; i0 < n; i0 += U * step) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            ml[u] = make_float2(-INFINITY, 0.f);
            o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                const int64_t slot = part_slot(range, i) * a.Hq + head;
                ml[u] = __ldcg(ws.ml + slot);
                o[u] = __ldcg(reinterpret_cast<const float4 *>(ws.o + slot * D + 4 * col));
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
}

template <int D>
__device__ __forceinline__ void write_joined(const PagedArgs &a, int s, int head, int col, float m, float l, const float4 &x,
                                             float *all_lse2) {
    const float f = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2 *>(a.out + ((int64_t)s * a.Hq + head) * D + 4 * col) =
        make_uint2(bf16x2(x.x * f, x.y * f), bf16x2(x.z * f, x.w * f));
    if (col == 0 && (a.lse || all_lse2)) {
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        if (a.lse) a.lse[(int64_t)s * a.Hq + head] = lse2 * kLn2;
        if (all_lse2) all_lse2[(int64_t)s * a.Hq + head] = lse2;
    }
}

// What is left of a weight w >= 0 beside its high part: above zero unless w is zero.
__device__ __forceinline__ float low_part(float w, float high) { return fminf(fmaxf(w - high, 0x1p-126f), w); }

// The block's barrier, from more than one place in the code, and that of the multiplying warps.
__device__ __forceinline__ void sync_all() { asm volatile("bar.sync 0;" ::: "memory"); }
template <int Threads>
__device__ __forceinline__ void sync_some() {
    asm volatile("bar.sync 1, %0;" ::"n"(Threads) : "memory");
}

// FP8 rows: GT heads of D bf16 values in shared memory become, in place, D first parts and D second parts (bytes) of the
// values divided by scale[h], a power of two. A warp takes every W-th head.
template <int D, int GT, int W>
__device__ __forceinline__ void split_queries(uint32_t queries, int warp, int lane, float *scale) {
    static_assert(D == 256, "a lane has 8 dims");
    for (int h = warp; h < GT; h += W) {
        const uint32_t qrow = queries + h * D * 2, hx = h & 7;
        uint32_t x[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(qrow + ((lane ^ hx) << 4))
                     : "memory");
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xFFFF0000u))));
#pragma unroll
        for (int n = 16; n >= 1; n >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, n));
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -119), 126);
        // the largest becomes 2^7 .. 2^8; an infinite one makes the head NaN, not E4M3's largest value
        const float down = top == INFINITY ? NAN : __uint_as_float((uint32_t)(134 - e) << 23);
        uint32_t part[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            part[0][k] = part[1][k] = 0u;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const uint32_t y = x[2 * k + z];
                const float u = __uint_as_float(y << 16) * down, v = __uint_as_float(y & 0xFFFF0000u) * down;
                const uint32_t w = e4m3x2_of(u, v), back = e4m3_to_f16x2(w, 0);
                const float2 near = __half22float2(*reinterpret_cast<const __half2 *>(&back));
                part[0][k] |= w << (16 * z);
                part[1][k] |= e4m3x2_of((u - near.x) * 32.f, (v - near.y) * 32.f) << (16 * z);
            }
        }
        __syncwarp();
#pragma unroll
        for (int z = 0; z < 2; ++z)
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(qrow + (((z * D / 16 + (lane >> 1)) ^ hx) << 4) + (lane & 1) * 8),
                         "r"(part[z][0]), "r"(part[z][1])
                         : "memory");
        if (lane == 0) scale[h] = __uint_as_float((uint32_t)(120 + e) << 23);
    }
}

// dst + index x bytes, index >= 0
__device__ __forceinline__ const char *row_ptr(const char *base, int index, uint32_t bytes) {
    return base + (uint64_t)(uint32_t)index * bytes;
}

// Neither this kernel nor the join lets the next one begin early: join CTAs that wait beside it cost a call of 4,096
// tokens 0.7 us of 7.8, and a tile kernel whose CTAs find no room beside what still runs does not run in one wave, which
// its equal ranges are made for.
// Wt: the scores and each sequence's log-sum-exp are also kept, for the kernel that turns them into weights.
template <typename C, bool Wt>
__global__ void __launch_bounds__(C::threads, C::ctas) paged_tile_kernel(PagedArgs a, PagedScratch ws, int ranges, WeightArgs wt) {
    constexpr int D = C::D, GT = C::GT, W = C::warps, T = C::tile, TW = C::warp_tok, NS = C::stages, SG = C::groups;
    constexpr int LT = C::load_tok;
    constexpr bool F8 = C::F8;
    constexpr int HR = GT / 8;                     // head rows a lane holds: g and g + 8
    constexpr int NQ = TW / 8;                     // 8-token columns of the warp's scores
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long scan[W + C::loaders];
    __shared__ int start[2];
    __shared__ float head_scale[GT];               // split queries: Q is its parts' sum x head_scale
    __shared__ uint32_t real_tok[NS][C::load_warps];       // bit i: token i of the loading warp's share exists
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int range = blockIdx.x / a.Hkv, kvh = blockIdx.x % a.Hkv;
    const int Hkv = a.Hkv, G = a.G;
    wait_for_previous();

    // ---- this range's tiles: total over the batch, then the row and tile the range starts at. Up to 32 rows every warp
    // does that for itself, in 32 bits and without a barrier: 0.5 us of a call.
    long long x0 = 0, x1 = 0;
    Cursor<T> in, at;                              // the loads' place, and the products'
    int skip = 0;                                  // tiles of its first row that come before the range
    Ranges cut(1, 1);
    if (a.B <= 32) {                               // at most 2^30 tiles
        const Row r = row_of<T>(a, min(lane, a.B - 1));
        const uint32_t mine = lane < a.B ? r.t1 - r.t0 : 0;
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t total = __shfl_sync(0xffffffffu, upto, 31);
        cut = Ranges(total, (int)min((uint32_t)ranges, max(total, 1u)));
        if (range < cut.R) x0 = cut.begin(range), x1 = cut.begin(range + 1);
        const int s = min(__popc(__ballot_sync(0xffffffffu, upto <= (uint32_t)x0)), 31);
        skip = (int)((uint32_t)x0 - __shfl_sync(0xffffffffu, upto - mine, s));
        in.s = s;
        in.r = {__shfl_sync(0xffffffffu, r.len, s), __shfl_sync(0xffffffffu, r.lo, s), __shfl_sync(0xffffffffu, r.t0, s),
                __shfl_sync(0xffffffffu, r.t1, s)};
        in.t = in.r.t0 + skip;
    } else {
        const int per = (a.B + C::threads - 1) / C::threads, s_lo = min(a.B, tid * per), s_hi = min(a.B, s_lo + per);
        long long mine = 0;
        for (int s = s_lo; s < s_hi; ++s) {
            const Row r = row_of<T>(a, s);
            mine += r.t1 - r.t0;
        }
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        long long total = 0;
#pragma unroll
        for (int w = 0; w < W + C::loaders; ++w) {
            if (w < warp) upto += scan[w];
            total += scan[w];
        }
        cut = Ranges(total, (int)min((long long)ranges, max(total, 1ll)));
        if (range < cut.R) x0 = cut.begin(range), x1 = cut.begin(range + 1);
        if (x0 < x1 && upto - mine <= x0 && x0 < upto) {
            long long before = upto - mine;
            int s = s_lo;
            for (;; ++s) {
                const Row r = row_of<T>(a, s);
                if (x0 < before + r.t1 - r.t0) break;
                before += r.t1 - r.t0;
            }
            start[0] = s;
            start[1] = (int)(x0 - before);
        }
        __syncthreads();
        if (x0 < x1) {
            skip = start[1];
            in.at(a, start[0], skip);
        }
    }
    at = in;
    const long long n_tiles = x1 - x0;
    if (kvh == 0 && tid == 0) ws.meta[range] = make_int2(-1, 0);
    if (Wt && kvh == 0 && tid == 0 && range == cut.R - 1) *wt.n_tiles = (int)min(x1, (long long)INT32_MAX);

    for (int s = range; s < a.B; s += ranges) {    // rows without a token: zeros
        const Row r = row_of<T>(a, s);
        if (r.t1 > r.t0) continue;
        const int len = a.seq_len[s];
        if (len != 0 && kvh == 0 && tid == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePaged, s);
        uint16_t *o = a.out + ((int64_t)s * a.Hq + kvh * G) * D;
        for (int i = tid; i < G * D / 8; i += C::threads) reinterpret_cast<uint4 *>(o)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse && tid < G) a.lse[(int64_t)s * a.Hq + kvh * G + tid] = -INFINITY;
    }
    if (n_tiles == 0) return;
    const uint32_t base = smem_u32(smem);

    // ---- loads. Lane i < LT keeps token i of the loading warp's share: its page's place in the table and offset in the
    // page, stepped by a tile at a time, and the page id, fetched one tile ahead of the copies.
    const int lw = C::loaders ? warp - W : warp, lt = lw * 32 + lane;      // loading warp, thread among those that load
    const int chunk = lane % C::chunks;
    const uint32_t row_step = (uint32_t)Hkv * C::row;
    const char *k_rows = static_cast<const char *>(a.k) + kvh * C::row + chunk * 16;
    const char *v_rows = static_cast<const char *>(a.v) + kvh * C::row + chunk * 16;
    int entry, offset, page;
    bool wanted;
    auto fetch_page = [&](bool new_row) {
        const uint32_t tok = (uint32_t)in.t * T + lw * LT + lane;      // a tile may reach past 2^31
        if (new_row) {
            entry = a.page_shift >= 0 ? tok >> a.page_shift : tok / (uint32_t)a.page_size;
            offset = tok - (uint32_t)entry * a.page_size;
        } else {
            entry += a.tile_entries;
            offset += a.tile_rest;
            if (offset >= a.page_size) offset -= a.page_size, ++entry;
        }
        wanted = (LT == 32 || lane < LT) && tok >= (uint32_t)in.r.lo && tok < (uint32_t)in.r.len;
        page = wanted ? a.table[in.s * a.ld + entry] : -1;
    };
    auto issue = [&](int stage, int q_slot, bool first) {      // tile `in`
        const uint32_t st = base + stage * C::stage;
        const bool ok = (uint32_t)page < (uint32_t)a.n_pages;
        if (wanted && !ok && kvh == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePaged, in.s);
        const int slot = wanted && ok ? page * a.page_size + offset : -1;
        const uint32_t real = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) real_tok[stage][lw] = real;
#pragma unroll
        for (int i = 0; i < LT / C::rows_per_copy; ++i) {
            const int r = i * C::rows_per_copy + lane / C::chunks;
            const int sl = __shfl_sync(0xffffffffu, slot, r);
            const int t = lw * LT + r;
            const uint32_t to = st + t * C::row + ((chunk ^ (t & 7)) << 4);
            cp_async16_zfill(to, row_ptr(k_rows, max(sl, 0), row_step), sl >= 0);
            cp_async16_zfill(to + C::k_bytes, row_ptr(v_rows, max(sl, 0), row_step), sl >= 0);
        }
        if (F8 && (LT == 32 || lane < LT)) {
            constexpr int SB = SG * 4;
            const int64_t from = ((int64_t)max(slot, 0) * Hkv + kvh) * SG;
            const uint32_t to = st + 2 * C::k_bytes + (lw * LT + lane) * SB;
            cp_async_small_zfill<SB>(to, a.k_scales + from, slot >= 0);
            cp_async_small_zfill<SB>(to + C::s_bytes, a.v_scales + from, slot >= 0);
        }
        if (first) {                               // the row's queries, heads behind G as zeros
            const uint16_t *q = a.q + in.s * a.q_ld + (int64_t)kvh * G * D;
            const uint32_t to = base + C::q_at + q_slot * C::q_bytes;
            for (int i = lt; i < GT * D / 8; i += C::load_warps * 32) {
                const int h = i / (D / 8), ch = i % (D / 8);
                cp_async16_zfill(to + h * D * 2 + ((ch ^ (h & 7)) << 4), q + (h < G ? h * D + ch * 8 : 0), h < G);
            }
        }
    };
    // Queries wait in NS - 1 slots, one for each row in turn: a tile is issued once every warp has taken the queries
    // of the tile NS - 1 before it, so no slot in use is overwritten.
    long long issued = 0;
    int in_stage = 0, in_slot = 0;
    bool in_first = true;
    auto advance = [&]() {                         // issue the next tile (or an empty group) and step on
        if (issued < n_tiles) {
            issue(in_stage, in_slot, in_first);
            in_stage = in_stage + 1 == NS ? 0 : in_stage + 1;
            if (in_first) in_slot = in_slot + 1 == NS - 1 ? 0 : in_slot + 1;
            ++issued;
            if (issued < n_tiles) {
                in_first = in.next(a);
                fetch_page(in_first);
            }
        }
        cp_async_commit();
    };
    if (!C::loaders || warp >= W) {
        fetch_page(true);
#pragma unroll 1
        for (int i = 0; i < NS - 1; ++i) advance();
    }
    if (C::loaders && warp >= W) {                 // the barriers of the loop below, and the loads between them
        bool first = true;
        int stage = 0;
        for (long long i = 0; i < n_tiles; ++i) {
            cp_async_wait<NS - 2>();
            if (F8) {
                // infinite V scales become NaN, each by the lane that fetched it: a product with zero where the scales are
                // used costs 32 sequences of 20,000 tokens with 16 head rows 124.5 us instead of 122.4
                static_assert(!F8 || !C::loaders || LT == 32, "a lane for each token");
                float *v = reinterpret_cast<float *>(smem + stage * C::stage + 2 * C::k_bytes + C::s_bytes) + lt * SG;
#pragma unroll
                for (int gr = 0; gr < SG; ++gr)
                    if (v[gr] == INFINITY) v[gr] = NAN;
                stage = stage + 1 == NS ? 0 : stage + 1;
            }
            sync_all();
            if (first) sync_all();                 // tile i's queries, whose slot may be wanted now, are taken
            advance();
            first = at.t + 1 == at.r.t1;
            if (i + 1 < n_tiles) at.next(a);
        }
        return;
    }

    // ---- products
    auto sync_mul = []() {
        if (C::loaders)
            sync_some<W * 32>();
        else
            sync_all();
    };
    constexpr int KS = D / 16;
    uint32_t qf[KS][2 * HR];                       // Q operand: rows g (and g + 8), two k halves
    float q_scale[HR];                             // logit = score x q_scale (x K scale)
    float m[SG][HR], l[HR];                        // running maxima of the sets; this lane's own weights' sum
    float o[4][4];
    const int my_set = SG == 2 ? warp / 4 : 0;     // the weights this warp's dims use
    float *const maxima = reinterpret_cast<float *>(smem + C::x_at);    // [SG][GT][W]
    bool begins = skip == 0;                   // the segment starts its sequence
    bool first = true;
    int stage = 0, q_slot = 0;
    for (long long i = 0; i < n_tiles; ++i, stage = stage + 1 == NS ? 0 : stage + 1) {
        if (!C::loaders) cp_async_wait<NS - 2>();
        sync_all();                                // tile i is in; every warp has left tile i - 1
        const uint32_t st = base + stage * C::stage;
        if (first) {
            const uint32_t qa = base + C::q_at + q_slot * C::q_bytes;
            q_slot = q_slot + 1 == NS - 1 ? 0 : q_slot + 1;
            if (!F8) {
                if constexpr (GT == 16) {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const int h = (lane & 7) + ((lane >> 3) & 1) * 8, ch = 2 * k + (lane >> 4);
                        uint32_t r[4];
                        ldmatrix4(qa + h * D * 2 + ((ch ^ (h & 7)) << 4), r);
                        qf[k][0] = r[0], qf[k][1] = r[2];
                        qf[k][2] = r[1], qf[k][3] = r[3];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < KS; k += 2) {
                        const int h = lane & 7, ch = 2 * k + (lane >> 3);
                        uint32_t r[4];
                        ldmatrix4(qa + h * D * 2 + ((ch ^ h) << 4), r);
                        qf[k][0] = r[0], qf[k][1] = r[1];
                        qf[k + 1][0] = r[2], qf[k + 1][1] = r[3];
                    }
                }
#pragma unroll
                for (int h = 0; h < HR; ++h) q_scale[h] = a.scale_log2;
            } else if constexpr (C::split) {
                split_queries<D, GT, W>(qa, warp, lane, head_scale);
                sync_mul();
                // qf[k][0], [1]: first and second parts of dims 16k + 4c .. 4c + 3, as the codes of K lie
                q_scale[0] = a.scale_log2 * head_scale[g];
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int k = 0; k < KS; k += 4) {
                        uint32_t r[4];
                        ldmatrix4(qa + (lane & 7) * D * 2 + (((z * D / 16 + k + (lane >> 3)) ^ (lane & 7)) << 4), r);
#pragma unroll
                        for (int n = 0; n < 4; ++n) qf[k + n][z] = r[n];
                    }
            } else {
                // k index (2c, 2c+1 | 2c+8, 2c+9) of a step stands for dims 16k + 4c .. 4c + 3, as the codes of K lie
#pragma unroll
                for (int h = 0; h < HR; ++h) {
                    const uint32_t qrow = qa + (g + 8 * h) * D * 2;
                    float top = 0.f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t x, y;
                        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                                     : "=r"(x), "=r"(y)
                                     : "r"(qrow + (((2 * k + (c >> 1)) ^ g) << 4) + (c & 1) * 8));
                        qf[k][2 * h] = x, qf[k][2 * h + 1] = y;
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(x << 16)), fabsf(__uint_as_float(x & 0xFFFF0000u))),
                                               fmaxf(fabsf(__uint_as_float(y << 16)), fabsf(__uint_as_float(y & 0xFFFF0000u)))));
                    }
                    top = quad_max(top);
                    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                    q_scale[h] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t x = qf[k][2 * h + z];
                            qf[k][2 * h + z] = f16x2(__uint_as_float(x << 16) * down,
                                                     __uint_as_float(x & 0xFFFF0000u) * down);
                        }
                }
            }
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                l[h] = 0.f;
#pragma unroll
                for (int gr = 0; gr < SG; ++gr) m[gr][h] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][k] = 0.f;
            if (C::loaders) sync_all();
            first = false;
        }
        // S = Q K^T over this warp's tokens; s[nt]: tokens nt x 8 + 2c, + 1 for head rows g (and g + 8)
        float s[NQ][2 * HR];
        float lv[SG][NQ][2];                       // FP8: log2 of the tokens' V scales
        {
            // independent sums (FP8: of each 128 dims)
            constexpr int CH = C::split ? 1 : F8 ? (NQ <= 2 ? 2 : 1) : 4 / NQ > 0 ? 4 / NQ : 1;
            const uint32_t real = real_tok[stage][warp * TW / LT] >> (warp * TW % LT);
            constexpr int NB = C::split ? NQ : 1;  // columns of tokens whose sums are formed together
            float accs[NB][SG * CH][4];
#pragma unroll
            for (int nt = 0; nt < NQ; ++nt) {
                auto &acc = accs[nt % NB];
                if (nt == 0 || !C::split)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int x = 0; x < SG * CH; ++x) accs[n][x][0] = accs[n][x][1] = accs[n][x][2] = accs[n][x][3] = 0.f;
                const uint32_t krow = st + (warp * TW + nt * 8 + (lane & 7)) * C::row;
                if constexpr (C::split) {
                    constexpr int KG = C::chunks / 4 / SG;     // loads of 64 bytes of a row in 128 dims
#pragma unroll
                    for (int k = 0; k < (nt == 0 ? KG : 0); ++k) {
                        uint32_t b[NB][SG][4];
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int gr = 0; gr < SG; ++gr)
                                ldmatrix4(krow + n * 8 * C::row + (((4 * (k + gr * KG) + (lane >> 3)) ^ (lane & 7)) << 4), b[n][gr]);
#pragma unroll
                        for (int z = 0; z < 4; z += 2)
#pragma unroll
                            for (int gr = 0; gr < SG; ++gr)
#pragma unroll
                                for (int n = 0; n < NB; ++n) {
                                    const int step = 4 * (k + gr * KG) + z;
                                    mma16832_e4m3(accs[n][gr], qf[step][0], qf[step][1], qf[step + 1][0], qf[step + 1][1],
                                                  b[n][gr][z], b[n][gr][z + 1]);
                                }
                    }
                } else
#pragma unroll
                for (int k = 0; k < C::chunks / 4; ++k) {
                    uint32_t b[4];
                    ldmatrix4(krow + (((4 * k + (lane >> 3)) ^ (lane & 7)) << 4), b);
                    if (!F8) {
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t qa[4] = {qf[2 * k + z][0], HR == 2 ? qf[2 * k + z][2 * HR - 2] : 0u,
                                                    qf[2 * k + z][1], HR == 2 ? qf[2 * k + z][2 * HR - 1] : 0u};
                            mma16816<false>(acc[(2 * k + z) % CH], qa, b[2 * z], b[2 * z + 1]);
                        }
                    } else {
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int step = 4 * k + z;
                            const uint32_t qa[4] = {qf[step][0], HR == 2 ? qf[step][2 * HR - 2] : 0u, qf[step][1],
                                                    HR == 2 ? qf[step][2 * HR - 1] : 0u};
                            mma16816<true>(acc[(step / 8) * CH + step % CH], qa, e4m3_to_f16x2(b[z], 0),
                                           e4m3_to_f16x2(b[z], 1));
                        }
                    }
                }
                const int t = nt * 8 + 2 * c;      // this lane's two tokens of the warp's share
                float sc[2][SG];                   // K scales of the two tokens
                if (F8) {
                    const float *ks = reinterpret_cast<const float *>(smem + stage * C::stage + 2 * C::k_bytes) +
                                      (warp * TW + t) * SG;
                    const float *vs = ks + C::s_bytes / 4;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int gr = 0; gr < SG; ++gr) {
                            sc[x][gr] = ks[x * SG + gr];
                            // NaN stays NaN, and infinity becomes it (the loading warps see to that, or the product): as a
                            // maximum it would take every other token's weight to zero
                            const float v_scale = vs[x * SG + gr], e = lg2(v_scale);
                            lv[gr][nt][x] = C::loaders ? e : fmaf(v_scale, 0.f, e);
                        }
                }
#pragma unroll
                for (int x = 0; x < 2 * HR; ++x) {
                    float v = 0.f;
#pragma unroll
                    for (int gr = 0; gr < SG; ++gr) {
                        float sum = acc[gr * CH][x];
#pragma unroll
                        for (int y = 1; y < CH; ++y) sum += acc[gr * CH + y][x];
                        if (C::split) sum = fmaf(acc[gr * CH][(2 + x) & 3], 0.03125f, sum);     // the second parts' rows
                        v = F8 ? fmaf(sum, sc[x & 1][gr], v) : sum;
                    }
                    s[nt][x] = (real >> (t + (x & 1))) & 1 ? v * q_scale[x / 2] : -INFINITY;
                }
            }
        }
        if (Wt && x0 + i < wt.cap) {
            float *to = wt.scores + ((x0 + i) * a.Hq + kvh * G) * T + warp * TW + 2 * c;
#pragma unroll
            for (int h = 0; h < HR; ++h)
                if (g + 8 * h < G)
#pragma unroll
                    for (int nt = 0; nt < NQ; ++nt)
                        *reinterpret_cast<float2 *>(to + (g + 8 * h) * T + nt * 8) = make_float2(s[nt][2 * h], s[nt][2 * h + 1]);
            if (kvh == 0 && tid == 0) wt.tiles[x0 + i] = make_int2(at.s, at.t);
        }
        // the tile's maximum of every head: over this warp's tokens, then over the warps
#pragma unroll
        for (int gr = 0; gr < SG; ++gr)
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NQ; ++nt)
                    // a V scale below 2^-100, or that is not a number, counts as 2^-100 here: the maximum is finite
                    // whenever a score is
                    top = fmaxf(top, F8 ? fmaxf(s[nt][2 * h] + fmaxf(lv[gr][nt][0], -100.f),
                                                s[nt][2 * h + 1] + fmaxf(lv[gr][nt][1], -100.f))
                                        : fmaxf(s[nt][2 * h], s[nt][2 * h + 1]));
                top = quad_max(top);
                if (c == 0) maxima[(gr * GT + g + 8 * h) * W + warp] = top;
            }
        sync_mul();
        if (!C::loaders) advance();
        float alpha[HR];                           // of this warp's set
#pragma unroll
        for (int gr = 0; gr < SG; ++gr)
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                const float *x = maxima + (gr * GT + g + 8 * h) * W;
                float top = m[gr][h];
                if (W == 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(x);
                    top = fmaxf(top, fmaxf(v.x, v.y));
                } else {
#pragma unroll
                    for (int w = 0; w < W / 4; ++w) {
                        const float4 v = reinterpret_cast<const float4 *>(x)[w];
                        top = fmaxf(top, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
                    }
                }
                float ref = top == -INFINITY ? 0.f : top;
                const float al = ex2(m[gr][h] - ref);
                m[gr][h] = top;
                ref -= C::raise;
                if (gr == 0) l[h] *= al;
                if (SG == 1 || gr == my_set) alpha[h] = al;
                // weights of this warp's tokens
                unsigned char *p = smem + C::p_at + (g + 8 * h) * C::p_pitch + (warp * TW + 2 * c) * 2;
#pragma unroll
                for (int nt = 0; nt < NQ; ++nt) {
                    const float u = s[nt][2 * h] - ref, v = s[nt][2 * h + 1] - ref;
                    if (F8) {
                        if (gr == 0) l[h] = fmaf(ex2(u) + ex2(v), C::lower, l[h]);     // relative to m
                        *reinterpret_cast<uint32_t *>(p + gr * GT * C::p_pitch + nt * 16) =
                            f16x2(ex2(u + lv[gr][nt][0]), ex2(v + lv[gr][nt][1]));
                    } else {
                        const float e = ex2(u), f = ex2(v);
                        l[h] += e + f;
                        const uint32_t w = bf16x2_toward_zero(e, f);
                        *reinterpret_cast<uint32_t *>(p + nt * 16) = w;
                        *reinterpret_cast<uint32_t *>(p + GT * C::p_pitch + nt * 16) =
                            bf16x2(low_part(e, __uint_as_float(w << 16)), low_part(f, __uint_as_float(w & 0xFFFF0000u)));
                    }
                }
            }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            o[n][0] *= alpha[0], o[n][1] *= alpha[0];
            if (HR == 2) o[n][2] *= alpha[HR - 1], o[n][3] *= alpha[HR - 1];
        }
        sync_mul();
        // O += P V over this warp's 32 dims
        const uint32_t vt = st + C::k_bytes + ((lane & 7) + ((lane >> 3) & 1) * 8) * C::row;
        const uint32_t pt = base + C::p_at + (F8 ? my_set * GT * C::p_pitch : 0) +
                            (GT == 16 ? ((lane & 7) + ((lane >> 3) & 1) * 8) * C::p_pitch + (lane >> 4) * 16
                                      : (lane & 7) * C::p_pitch + (lane >> 3) * 16);
#pragma unroll
        for (int k0 = 0; k0 < T / 16; k0 += 2) {
            uint32_t pw[2][2][4];                  // [step][high, low]
#pragma unroll
            for (int z = 0; z < (F8 ? 1 : 2); ++z) {
                uint32_t r[4];
                if (GT == 16) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) ldmatrix4(pt + z * GT * C::p_pitch + (k0 + k) * 32, pw[k][z]);
                } else {
                    ldmatrix4(pt + z * GT * C::p_pitch + k0 * 32, r);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        pw[k][z][0] = r[2 * k], pw[k][z][2] = r[2 * k + 1];
                        pw[k][z][1] = pw[k][z][3] = 0u;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!F8) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t b[4];
                        ldmatrix4_trans(vt + 16 * (k0 + k) * C::row + (((4 * warp + 2 * j + (lane >> 4)) ^ (lane & 7)) << 4), b);
                        mma16816<false>(o[2 * j], pw[k][0], b[0], b[1]);
                        mma16816<false>(o[2 * j + 1], pw[k][0], b[2], b[3]);
                        mma16816<false>(o[2 * j], pw[k][1], b[0], b[1]);
                        mma16816<false>(o[2 * j + 1], pw[k][1], b[2], b[3]);
                    }
                } else {
                    // a 16-bit element of the transposed load is two codes, dims 2n and 2n + 1 of a chunk of 16
                    uint32_t b[4];
                    ldmatrix4_trans(vt + 16 * (k0 + k) * C::row + (((2 * warp + (lane >> 4)) ^ (lane & 7)) << 4), b);
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = __byte_perm(b[j], 0, 0x3120);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd)
                            mma16816<true>(o[2 * j + odd], pw[k][0], e4m3_to_f16x2(b[2 * j], odd),
                                           e4m3_to_f16x2(b[2 * j + 1], odd));
                }
            }
        }
        // the segment's end
        const bool ends = at.t + 1 == at.r.t1;
        if (ends || i + 1 == n_tiles) {
            const bool whole = begins && ends;
            const int slot = 2 * range + (begins ? 1 : 0);
            // the sums of every warp's weights, where the maxima were
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                l[h] = quad_sum(l[h]);
                if (c == 0) maxima[(g + 8 * h) * W + warp] = l[h];
            }
            sync_mul();
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                const int row = g + 8 * h;
                if (row >= G) continue;
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) sum += maxima[row * W + w];
                const int head = kvh * G + row;
                // bf16: O / sum, or (m, sum, O) as a partial. FP8: O 2^(m_set - 15 - log2 of the softmax's denominator), with
                // (that logarithm, 1) as the partial's pair: the sets' maxima may lie far apart
                const float lse2 = sum == 0.f ? -INFINITY : m[0][h] + log2f(sum);
                float f;
                if (F8)
                    f = sum == 0.f ? 0.f : ex2(m[SG == 2 ? 1 : 0][h] - C::raise - lse2);
                else
                    f = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                if (SG == 2 && my_set == 0) f = sum == 0.f ? 0.f : C::lower / sum;
                float *po = ws.o + ((int64_t)slot * a.Hq + head) * D + warp * 32;
                uint16_t *out = a.out + ((int64_t)at.s * a.Hq + head) * D + warp * 32;
#pragma unroll
                for (int j = 0; j < (F8 ? 2 : 4); ++j) {
                    if (!F8) {
                        const float x = o[j][2 * h] * f, y = o[j][2 * h + 1] * f;
                        if (whole)
                            *reinterpret_cast<uint32_t *>(out + 8 * j + 2 * c) = bf16x2(x, y);
                        else
                            *reinterpret_cast<float2 *>(po + 8 * j + 2 * c) = make_float2(x, y);
                    } else {
                        const float4 x = make_float4(o[2 * j][2 * h] * f, o[2 * j + 1][2 * h] * f, o[2 * j][2 * h + 1] * f,
                                                     o[2 * j + 1][2 * h + 1] * f);
                        if (whole)
                            *reinterpret_cast<uint2 *>(out + 16 * j + 4 * c) = make_uint2(bf16x2(x.x, x.y), bf16x2(x.z, x.w));
                        else
                            *reinterpret_cast<float4 *>(po + 16 * j + 4 * c) = x;
                    }
                }
                if (warp == 0 && c == 0) {
                    if (!whole)
                        ws.ml[(int64_t)slot * a.Hq + head] = F8 ? make_float2(lse2, 1.f) : make_float2(m[0][h], sum);
                    else if (a.lse)
                        a.lse[(int64_t)at.s * a.Hq + head] = lse2 * kLn2;
                    if (Wt && whole) wt.lse2[(int64_t)at.s * a.Hq + head] = lse2;
                }
            }
            if (begins && !ends && kvh == 0 && tid == 0) {
                // the sequence's last tile is number `end` of the list: how many ranges it spans
                const long long end = x0 + i + (at.r.t1 - 1 - at.t);
                ws.meta[range] = make_int2(at.s, cut.of(end) - range + 1);
            }
            begins = first = true;
        }
        if (i + 1 < n_tiles) at.next(a);
    }
}

// The partials of the sequences that a range starts and leaves unfinished, joined:
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i. CTA (y, head) takes the y-th such range (there are at most as many
// as sequences). Thread (row, 4 dims) takes every rows-th partial, its (m, l) and O loaded together and merged with a
// running maximum; then the rows of threads are merged in order. The time is that of two dependent loads.
template <int D, int Threads>
__global__ void __launch_bounds__(Threads) paged_join_kernel(PagedArgs a, PagedScratch ws, int ranges, float *all_lse2) {
    constexpr int cols = D / 4, rows = Threads / cols, U = D == 256 ? 8 : 4;
    __shared__ float4 acc[Threads];
    __shared__ float2 pair[rows];
    __shared__ int4 job_sh;                                                 // range, sequence, partials
    const int head = blockIdx.y, tid = threadIdx.x, col = tid % cols, row = tid / cols;
    wait_for_previous();
    if (tid < 32) {
        if (tid == 0) job_sh.x = -1;
        __syncwarp();
        int n = 0;
        for (int r0 = 0; r0 < ranges - 1; r0 += 32 * 8) {
            int2 meta[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = r0 + 32 * k + tid;
                meta[k] = r < ranges - 1 ? __ldcg(ws.meta + r) : make_int2(-1, 0);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t some = __ballot_sync(0xffffffffu, meta[k].x >= 0);
                if (meta[k].x >= 0 && n + __popc(some & ((1u << tid) - 1u)) == (int)blockIdx.x)
                    job_sh = make_int4(r0 + 32 * k + tid, meta[k].x, meta[k].y, 0);
                n += __popc(some);
            }
        }
    }
    __syncthreads();
    const int4 job = job_sh;
    if (job.x < 0) return;
    float m, l;
    float4 x;
    join_parts<D, U>(a, ws, job.x, job.z, head, col, row, rows, m, l, x);
    acc[tid] = x;
    if (col == 0) pair[row] = make_float2(m, l);
    __syncthreads();
    if (tid >= cols) return;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < rows; ++i) top = fmaxf(top, pair[i].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < rows; ++i) {
        const float w = ex2(pair[i].x - ref);
        const float4 v = acc[i * cols + tid];
        sum = fmaf(w, pair[i].y, sum);
        x.x = fmaf(w, v.x, x.x), x.y = fmaf(w, v.y, x.y), x.z = fmaf(w, v.z, x.z), x.w = fmaf(w, v.w, x.w);
    }
    write_joined<D>(a, job.y, head, col, top, sum, x, all_lse2);
}

// CTAs of one wave on the current device (cached per device; 0 on an error).
template <typename C, bool Wt>
int wave() {
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cached[dev] == 0) {
        int sms = 0, per_sm = 0;
        if (cudaFuncSetAttribute(paged_tile_kernel<C, Wt>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, paged_tile_kernel<C, Wt>, C::threads, C::smem) != cudaSuccess)
            return 0;
        cached[dev] = std::min(sms * per_sm, max_ctas(C::D));
    }
    return cached[dev];
}

PagedScratch scratch_of(char *w, int D, int Hq, int Hkv) {
    const size_t slots = 2 * (size_t)ranges_for(max_ctas(D), Hkv) * Hq;
    PagedScratch s;
    s.meta = reinterpret_cast<int2 *>(w);
    s.ml = reinterpret_cast<float2 *>(w + kMaxRanges * sizeof(int2));
    s.o = reinterpret_cast<float *>(w + kMaxRanges * sizeof(int2) + (slots * sizeof(float2) + 255) / 256 * 256);
    return s;
}

template <typename C, bool Wt>
cudaError_t launch(const PagedArgs &a, const WeightArgs &wt, cudaStream_t st) {
    const int ctas = wave<C, Wt>();
    if (ctas == 0) {
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    }
    const int ranges = ranges_for(ctas, a.Hkv);
    const PagedScratch ws = scratch_of(a.scratch, C::D, a.Hq, a.Hkv);
    PagedArgs b = a;
    b.tile_entries = C::tile / a.page_size;
    b.tile_rest = C::tile % a.page_size;
    b.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    const cudaError_t e = launch_dependent(paged_tile_kernel<C, Wt>, dim3(ranges * a.Hkv), C::threads, C::smem, st, b, ws, ranges, wt);
    if (e != cudaSuccess || ranges == 1) return e;      // one range cuts no sequence
    // few sequences have many partials each: more threads for them (one of 4,096 tokens 6.9 against 7.3 us; but 30 of 512
    // tokens 16.9 against 14.4)
    const dim3 grid(std::min(ranges - 1, a.B), a.Hq);
    return (int64_t)grid.x * grid.y <= kFewJoins ? launch_dependent(paged_join_kernel<C::D, 512>, grid, 512, 0, st, a, ws, ranges, wt.lse2)
                                                 : launch_dependent(paged_join_kernel<C::D, 256>, grid, 256, 0, st, a, ws, ranges, wt.lse2);
}

template <int D, bool F8, bool Wt>
cudaError_t launch_heads(const PagedArgs &a, const WeightArgs &wt, cudaStream_t st) {
    return a.G <= 8 ? launch<PagedCfg<D, 8, F8>, Wt>(a, wt, st) : launch<PagedCfg<D, 16, F8>, Wt>(a, wt, st);
}

template <bool Wt>
cudaError_t launch_dims(const PagedArgs &a, const WeightArgs &wt, int D, bool fp8, cudaStream_t st) {
    switch (D) {
        case 64: return fp8 ? cudaErrorInvalidValue : launch_heads<64, false, Wt>(a, wt, st);
        case 128: return fp8 ? launch_heads<128, true, Wt>(a, wt, st) : launch_heads<128, false, Wt>(a, wt, st);
        case 256: return fp8 ? launch_heads<256, true, Wt>(a, wt, st) : launch_heads<256, false, Wt>(a, wt, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

}  // namespace qsa
