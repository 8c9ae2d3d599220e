// Attention of a tree of drafted tokens over a paged K/V cache (qsa_tree_decode, qsa_tree_decode_fp8kv).
#include "paged.cuh"

#include <algorithm>

namespace qsa {

namespace {

constexpr int kTreeThreads = 128;

// A warp for each (drafted token, query head).
template <int D, bool F8>
__global__ void __launch_bounds__(kTreeThreads) tree_kernel(TreeArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kTreeThreads / 32) + (threadIdx.x >> 5);
    wait_for_previous();
    const int i = (int)(item / a.Hq), h = (int)(item % a.Hq);
    if (i >= a.N) return;
    int s = -1, off = 0, T = 0, high = 0;            // high: the largest offset so far
    for (int b0 = 0; b0 < a.B && (s < 0 || item == 0); b0 += 32) {
        const int b = b0 + lane;
        const int lo = b < a.B ? a.draft_off[b] : 0, hi = b < a.B ? a.draft_off[b + 1] : 0;
        int top = max(high, lo);
        for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_up_sync(0xffffffffu, top, o));
        const bool fine = b < a.B && lo == top && hi >= lo && hi <= a.N;
        if (b < a.B && !fine && item == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereTree, b);
        const uint32_t in = __ballot_sync(0xffffffffu, fine && lo <= i && i < hi);
        if (in) {
            const int l = __ffs(in) - 1;
            s = b0 + l;
            off = __shfl_sync(0xffffffffu, lo, l);
            T = __shfl_sync(0xffffffffu, hi, l) - off;
        }
        high = __shfl_sync(0xffffffffu, top, 31);
    }
    if (s < 0) return;
    uint16_t *out = a.out + ((int64_t)i * a.Hq + h) * D;
    const int n = a.seq_len[s];
    const bool ok = T <= a.max_draft && n >= T && n <= a.ld * a.page_size;
    if (!ok && lane == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereTree, s);
    const int base = ok ? n - T : 0;
    uint32_t kin[4] = {0u, 0u, 0u, 0u};
    int depth = 0;
    if (ok)
        for (int j = i - off; j >= 0;) {
            ++depth;
            for (int w = 0; w < 4; ++w)
                if (j / 32 == w) kin[w] |= 1u << (j % 32);
            const int p = a.parent[off + j];
            if (p < -1 || p >= j) {
                if (lane == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereTree, s);
                break;
            }
            j = p;
        }
    const int own = base + depth - 1, lo = a.window > 0 ? max(0, own - a.window + 1) : 0;
    float q[E], o[E], m = -INFINITY, l = 0.f;
    const int kvh = h / a.G;
    for (int e = 0; e < E; ++e) {
        q[e] = bf16_bits_to_float(a.q[i * a.q_ld + h * D + lane * E + e]) * a.scale_log2;
        o[e] = 0.f;
    }
    int passed = 0;                                  // ancestors met
    for (int j = min(lo, base); j < (ok ? n : 0); ++j) {
        if (j >= base) {
            const int t = j - base;
            if (!(kin[t / 32] >> (t % 32) & 1u)) continue;
            ++passed;
            if (a.window > 0 && base + passed - 1 <= own - a.window) continue;
        } else if (j < lo) {
            continue;
        }
        const int page = a.table[s * a.ld + j / a.page_size];
        if ((uint32_t)page >= (uint32_t)a.n_pages) {
            if (lane == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereTree, s);
            continue;
        }
        const int64_t row = ((int64_t)page * a.page_size + j % a.page_size) * a.Hkv + kvh;
        float k[E], v[E];
        for (int e = 0; e < E; ++e) {
            const int64_t at = row * D + lane * E + e;
            if (F8) {
                const int g = (lane * E + e) / 128;
                const uint32_t c = static_cast<const uint8_t *>(a.k)[at] | static_cast<const uint8_t *>(a.v)[at] << 8;
                uint32_t f;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)c));
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&f));
                k[e] = x.x * a.k_scales[row * (D / 128) + g];
                v[e] = x.y * a.v_scales[row * (D / 128) + g];
            } else {
                k[e] = bf16_bits_to_float(static_cast<const uint16_t *>(a.k)[at]);
                v[e] = bf16_bits_to_float(static_cast<const uint16_t *>(a.v)[at]);
            }
        }
        float dot = 0.f;
        for (int e = 0; e < E; ++e) dot = fmaf(q[e], k[e], dot);
        for (int x = 16; x >= 1; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        const float top = fmaxf(m, dot), ref = top == -INFINITY ? 0.f : top;
        const float old = exp2f(m - ref), w = exp2f(dot - ref);
        m = top;
        l = l * old + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * old + w * v[e];
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < E; ++e) out[lane * E + e] = float_to_bf16_bits(o[e] * f);
    if (lane == 0 && a.lse) a.lse[(int64_t)i * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, bool F8>
cudaError_t launch(const TreeArgs &a, cudaStream_t st) {
    const int64_t items = (int64_t)a.N * a.Hq;
    const unsigned ctas = (unsigned)((items + kTreeThreads / 32 - 1) / (kTreeThreads / 32));
    return launch_dependent(tree_kernel<D, F8>, dim3(ctas), kTreeThreads, 0, st, a);
}

}  // namespace

size_t tree_scratch_bytes(int, int, int, int) { return 0; }

cudaError_t launch_tree_decode(const TreeArgs &a, int D, bool fp8, cudaStream_t st) {
    switch (D) {
        case 64: return fp8 ? cudaErrorInvalidValue : launch<64, false>(a, st);
        case 128: return fp8 ? launch<128, true>(a, st) : launch<128, false>(a, st);
        case 256: return fp8 ? launch<256, true>(a, st) : launch<256, false>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qsa
