// Rotary positions, alone (qsa_rope) and fused with appending K/V to a paged cache (qsa_rope_append).
//
// Pair i of a head at position p turns by the angle p f_i. f_i / (2 pi) modulo 1 is held as a 64-bit binary
// fraction of a turn, so the angle's fraction of a turn is (p x phase_i) mod 2^64: an integer product that is
// exact at every position (in fp32 the product of a position of millions and f_i is off by tenths of a
// radian). Its upper 32 bits give sin and cos.
//
// Both kernels stream: one thread owns 16 dims of a token's head (a "slot": 8 pairs, or 16 dims that pass through)
// for a run of heads, so the 8 sines and cosines are computed once and used for every head of the run. A slot's two
// 8-element vectors lie half a region apart, so neighbouring threads read and write neighbouring 16 bytes.
#include "paged.cuh"

#include <algorithm>

namespace qsa {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kBatch = 4;          // heads whose loads are in flight together
// K and V heads at a time. 4 took 95 registers a thread instead of 80: 4,096 tokens into FP8 rows 16.2 against 15.6 us;
// 1: 16.1.
constexpr int kKvBatch = 2;

struct Slot {
    int a, b;       // first dims of the slot's two 8-element vectors
    int fa, fb;     // first pairs of the slot's two groups of four, fa = -1: passes through
};

// The slots of a head: rot/16 turning ones first, then the dims that pass through in order.
__device__ __forceinline__ Slot slot_of(const RopeArgs &r, int s) {
    Slot t;
    const int turning = r.rot >> 4, half = r.rot >> 1;
    if (s < turning) {
        t.a = r.begin + 8 * s;
        t.b = t.a + half;
        t.fa = r.interleaved ? 4 * s : 8 * s;
        t.fb = r.interleaved ? 4 * s + (half >> 1) : 8 * s + 4;
    } else {
        const int e = 8 * (s - turning), f = e + ((r.D - r.rot) >> 1);
        t.fa = t.fb = -1;
        t.a = e < r.begin ? e : e + r.rot;
        t.b = f < r.begin ? f : f + r.rot;
    }
    return t;
}

// sin and cos of a 32-bit fraction of a turn. The nearest quarter turn comes off in integers, exactly; the rest
// x, at most pi/4, goes into the Taylor series of both (first omitted terms x^11/11! < 2e-9 and x^10/10! < 3e-8,
// both below fp32's own rounding of the results near 1).
__device__ __forceinline__ void sincos_turn(uint32_t turn, float &si, float &co) {
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(turn - (quarter << 30)) * 1.46291807926715968e-9f;   // 2 pi / 2^32
    const float z = x * x;
    float s = fmaf(z, 2.7557319224e-6f, -1.9841269841e-4f);
    s = fmaf(s, z, 8.3333333333e-3f);
    s = fmaf(s, z, -1.6666666667e-1f);
    s = fmaf(s * z, x, x);
    float c = fmaf(z, 2.4801587302e-5f, -1.3888888889e-3f);
    c = fmaf(c, z, 4.1666666667e-2f);
    c = fmaf(c, z, -0.5f);
    c = fmaf(c, z, 1.f);
    const float u = quarter & 1u ? c : s, v = quarter & 1u ? s : c;
    si = quarter & 2u ? -u : u;                             // quarters: (s, c), (c, -s), (-s, -c), (-c, s)
    co = (quarter + 1u) & 2u ? -v : v;
}

__device__ __forceinline__ void turns(const RopeArgs &r, const Slot &t, int pos, float (&co)[8], float (&si)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 f = __ldg(reinterpret_cast<const ulonglong2 *>(r.phase + (i < 2 ? t.fa : t.fb - 4) + 2 * i));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint64_t turn = (uint64_t)(int64_t)pos * (j ? f.y : f.x);
            sincos_turn((uint32_t)(turn >> 32), si[2 * i + j], co[2 * i + j]);
            si[2 * i + j] *= r.amplitude;
            co[2 * i + j] *= r.amplitude;
        }
    }
}

// Turn a slot's 16 values: pairs (x[i], x[8 + i]), or neighbours when interleaved.
__device__ __forceinline__ void turn16(float (&x)[16], const float (&co)[8], const float (&si)[8], bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[2 * i], w = x[2 * i + 1];
            x[2 * i] = u * co[i] - w * si[i];
            x[2 * i + 1] = w * co[i] + u * si[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[i], w = x[8 + i];
            x[i] = u * co[i] - w * si[i];
            x[8 + i] = w * co[i] + u * si[i];
        }
    }
}

__device__ __forceinline__ void unpack16(const uint4 &a, const uint4 &b, float (&x)[16]) {
    float f[8], g[8];
    unpack8(a, f);
    unpack8(b, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = f[i];
        x[8 + i] = g[i];
    }
}

__device__ __forceinline__ uint4 pack8(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A token's slot in heads [h0, h1), kBatch at a time: their loads are issued together, which the compiler cannot do
// by itself since dst may be src.
template <bool Inter>
__device__ __forceinline__ void turn_heads(const RopeArgs &r, const uint16_t *src, uint16_t *dst, int D, const Slot &sl, int pos,
                                           int h0, int h1) {
    uint4 va[kBatch], vb[kBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (h + i < h1) {
                va[i] = *reinterpret_cast<const uint4 *>(src + (int64_t)(h + i) * D + sl.a);
                vb[i] = *reinterpret_cast<const uint4 *>(src + (int64_t)(h + i) * D + sl.b);
            }
    };
    load(h0);
    float co[8], si[8];
    if (sl.fa >= 0) turns(r, sl, pos, co, si);
    for (int h = h0; h < h1; h += kBatch) {
        if (h > h0) load(h);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (h + i >= h1) break;
            if (sl.fa >= 0) {
                float x[16];
                unpack16(va[i], vb[i], x);
                turn16(x, co, si, Inter);
                va[i] = pack8(x);
                vb[i] = pack8(x + 8);
            }
            *reinterpret_cast<uint4 *>(dst + (int64_t)(h + i) * D + sl.a) = va[i];
            *reinterpret_cast<uint4 *>(dst + (int64_t)(h + i) * D + sl.b) = vb[i];
        }
    }
}

// Thread (token n, slot s) for heads [h0, h0 + run).
template <bool Inter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs r, RopeRows a, int run) {
    let_next_begin();
    wait_for_previous();
    const int S = r.D >> 4;
    const int64_t t = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    const int64_t n = t / S;
    if (n >= a.N) return;
    const Slot sl = slot_of(r, (int)(t - n * S));
    if (sl.fa < 0 && a.x == a.out) return;         // in place: nothing to do
    const int h0 = blockIdx.y * run;
    turn_heads<Inter>(r, a.x + n * a.x_ld, a.out + n * a.out_ld, r.D, sl, a.pos[n], h0, min(a.H, h0 + run));
}

// x / scale for inv = RN(1 / scale): the product by the reciprocal, corrected once by its remainder (Markstein 1990,
// "Computation of elementary functions on the IBM RISC System/6000 processor"). For scale = RN(amax / 448) of any bf16 amax
// and any bf16 x this is the correctly rounded quotient (tests/test_paged_abi.py goes through all 128 x 128 pairs of
// significands in exact arithmetic; powers of two do not matter in the range quantise16 uses it in); for a turned
// fp32 x it is at most one unit in the last place off.
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, scale, x), inv, q);
}

// Eight values of one 128-dim group (or of two groups, g0 != g1) quantised as quantize_kv_fp8_kernel does, but that a NaN
// keeps a NaN code in a group without other values too: the group's |max| over the row's S threads (a power of two <= 16 that starts at a multiple of S in the warp).
template <int S>
__device__ __forceinline__ void quantise16(const float (&x)[16], const Slot &sl, int s, uint8_t *codes, float *scales,
                                           int groups) {
    const unsigned mask = ((1u << S) - 1u) << ((threadIdx.x & 31) & ~(S - 1));
    const int ga = sl.a >> 7, gb = sl.b >> 7;
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ma = fmaxf(ma, fabsf(x[i]));
        mb = fmaxf(mb, fabsf(x[8 + i]));
    }
    float m0 = fmaxf(ga == 0 ? ma : 0.f, gb == 0 ? mb : 0.f), m1 = fmaxf(ga == 1 ? ma : 0.f, gb == 1 ? mb : 0.f);
#pragma unroll
    for (int o = S / 2; o >= 1; o >>= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(mask, m0, o, S));
        m1 = fmaxf(m1, __shfl_xor_sync(mask, m1, o, S));
    }
    const float s0 = __fdiv_rn(m0, kE4m3Max), s1 = __fdiv_rn(m1, kE4m3Max);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const float scale = (v ? gb : ga) ? s1 : s0;
        float y[8];
        if (scale > 0x1p-60f && scale < 0x1p60f) {             // no remainder below the normal range
            const float inv = __frcp_rn(scale);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = quotient(x[8 * v + i], scale, inv);
        } else if (scale > 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[8 * v + i], scale);
        } else {                                               // zeros, or NaN, which the maximum leaves out
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = isnan(x[8 * v + i]) ? x[8 * v + i] : 0.f;
        }
        const uint32_t w0 = e4m3x2_of(y[0], y[1]) | (e4m3x2_of(y[2], y[3]) << 16);
        const uint32_t w1 = e4m3x2_of(y[4], y[5]) | (e4m3x2_of(y[6], y[7]) << 16);
        *reinterpret_cast<uint2 *>(codes + (v ? sl.b : sl.a)) = make_uint2(w0, w1);
    }
    if (s == 0) {
        scales[0] = s0;
        if (groups == 2) scales[1] = s1;
    }
}

// Thread (token n, slot s) for a run of a token's heads, all of K and V (blockIdx.y < kv_slices) or all of q: k is
// turned into the cache, v copied into it, q turned into q_out. The K and V runs, which take longer, begin first. Runs of both
// kinds cost every head the choice between them: 4,096 tokens into FP8 rows 16.8 against 16.1 us. S = D / 16 threads of one warp
// carry a head.
template <int S, bool F8, bool Inter>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(RopeArgs r, AppendArgs a, int run, int kv_slices) {
    constexpr int D = S * 16;
    let_next_begin();
    wait_for_previous();
    const int64_t t = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    const int64_t n = t / S;
    const int s = (int)(t & (S - 1));
    if (n >= a.N) return;
    const int row = a.seq ? a.seq[n] : (int)n;
    if (row < 0) return;                                     // padding
    const int pos = a.pos[n];
    const Slot sl = slot_of(r, s);
    if ((int)blockIdx.y >= kv_slices) {
        const int h0 = ((int)blockIdx.y - kv_slices) * run, h1 = min(a.Hq, h0 + run);
        turn_heads<Inter>(r, a.q + n * a.q_ld, a.q_out + n * a.q_out_ld, D, sl, pos, h0, h1);
        return;
    }
    uint4 va[kKvBatch], vb[kKvBatch];
    float co[8], si[8];
    const Slot straight = {8 * s, D / 2 + 8 * s, -1, -1};
    const int h0 = blockIdx.y * run, h1 = min(2 * a.Hkv, h0 + run);
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kKvBatch; ++i) {
            const int hi = h + i;
            if (hi >= h1) break;
            const bool v = hi >= a.Hkv;
            const uint16_t *src = v ? a.v + n * a.v_ld + (hi - a.Hkv) * D : a.k + n * a.k_ld + hi * D;
            va[i] = *reinterpret_cast<const uint4 *>(src + (v ? straight.a : sl.a));
            vb[i] = *reinterpret_cast<const uint4 *>(src + (v ? straight.b : sl.b));
        }
    };
    load(h0);
    const int place = a.place ? a.place[n] : pos;
    bool ok = row < a.n_rows && place >= 0 && place / a.page_size < a.ld;
    int page = 0;
    if (ok) {
        page = a.table[(int64_t)row * a.ld + place / a.page_size];
        ok = page >= 0 && page < a.n_pages;
    }
    if (!ok) {                                                // its K and V are left out
        if (s == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereAppend, (int)n);
        return;
    }
    if (a.positions && s == 0 && h0 == 0 && place < a.positions_ld) a.positions[row * a.positions_ld + place] = pos;
    const int64_t slot = (int64_t)page * a.page_size + place % a.page_size;
    if (sl.fa >= 0 && h0 < a.Hkv) turns(r, sl, pos, co, si);
    for (int h = h0; h < h1; h += kKvBatch) {
        if (h > h0) load(h);
#pragma unroll
        for (int i = 0; i < kKvBatch; ++i) {
            const int hi = h + i;
            if (hi >= h1) break;
            const bool is_v = hi >= a.Hkv;
            const int g = hi - (is_v ? a.Hkv : 0);             // KV head
            const Slot at = is_v ? straight : sl;
            const bool turned = at.fa >= 0;
            float x[16];
            if (turned || F8) unpack16(va[i], vb[i], x);
            if (turned) turn16(x, co, si, Inter);
            const int64_t kv = (slot * a.Hkv + g) * D;
            if (F8) {
                quantise16<S>(x, at, s, (is_v ? a.v_codes : a.k_codes) + kv,
                              (is_v ? a.v_scales : a.k_scales) + (slot * a.Hkv + g) * (D / 128), D / 128);
            } else {
                if (turned) {
                    va[i] = pack8(x);
                    vb[i] = pack8(x + 8);
                }
                uint16_t *dst = (is_v ? a.v_cache : a.k_cache) + kv;
                *reinterpret_cast<uint4 *>(dst + at.a) = va[i];
                *reinterpret_cast<uint4 *>(dst + at.b) = vb[i];
            }
        }
    }
}

// Heads per thread: as long a run as keeps 1024 threads for each of 152 SMs, since a run shares its sines.
int run_of(int64_t threads_per_head, int heads) {
    const int64_t want = 152 * 1024;
    return (int)std::max<int64_t>(1, std::min<int64_t>(heads, threads_per_head * heads / want));
}

template <int S, bool F8>
cudaError_t append(const RopeArgs &r, const AppendArgs &a, cudaStream_t st) {
    const int q_heads = a.q ? a.Hq : 0, kv_heads = 2 * a.Hkv;
    const int64_t threads = (int64_t)a.N * S;
    const int run = run_of(threads, q_heads + kv_heads), kv_slices = (kv_heads + run - 1) / run;
    const dim3 grid((unsigned)((threads + kRopeThreads - 1) / kRopeThreads), kv_slices + (q_heads + run - 1) / run);
    return launch_dependent(r.interleaved ? rope_append_kernel<S, F8, true> : rope_append_kernel<S, F8, false>, grid, kRopeThreads,
                            0, st, r, a, run, kv_slices);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &r, const RopeRows &a, cudaStream_t st) {
    const int64_t threads = (int64_t)a.N * (r.D >> 4);
    const int run = run_of(threads, a.H);
    const dim3 grid((unsigned)((threads + kRopeThreads - 1) / kRopeThreads), (a.H + run - 1) / run);
    return launch_dependent(r.interleaved ? rope_kernel<true> : rope_kernel<false>, grid, kRopeThreads, 0, st, r, a, run);
}

cudaError_t launch_rope_append(const RopeArgs &r, const AppendArgs &a, cudaStream_t st) {
    const bool f8 = a.k_codes != nullptr;
    switch (r.D) {
        case 64: return f8 ? cudaErrorInvalidValue : append<4, false>(r, a, st);
        case 128: return f8 ? append<8, true>(r, a, st) : append<8, false>(r, a, st);
        case 256: return f8 ? append<16, true>(r, a, st) : append<16, false>(r, a, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qsa
