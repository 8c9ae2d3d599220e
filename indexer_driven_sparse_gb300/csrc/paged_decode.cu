// Attention of one new token over a paged K/V cache (qsa_paged_decode, qsa_paged_decode_fp8kv):
//   out = sum_j softmax_j(scale q . K[j]) V[j] over the sequence's cached tokens, with their log-sum-exp.
// Plain form: one CTA per (sequence, query head) walks the tokens in chunks with a running maximum and sum.
#include "paged.cuh"

namespace qsa {

namespace {

constexpr int kPagedThreads = 256;
constexpr int kPagedChunk = 64;

template <int D, bool F8>
__global__ void __launch_bounds__(kPagedThreads) paged_plain_kernel(PagedArgs a) {
    const int s = blockIdx.y, h = blockIdx.x, g = h / a.G, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ float qs[D], w[kPagedChunk];
    __shared__ int64_t slots[kPagedChunk];
    int len = a.seq_len[s];
    if (len < 0 || len > a.ld * a.page_size) {
        if (tid == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePaged, s);
        len = 0;
    }
    const int lo = a.window > 0 ? max(0, len - a.window) : 0;
    if (tid < D) qs[tid] = bf16_bits_to_float(a.q[s * a.q_ld + h * D + tid]) * a.scale_log2;
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int c0 = lo; c0 < len; c0 += kPagedChunk) {
        const int n = min(kPagedChunk, len - c0);
        __syncthreads();
        if (tid < n) {
            const int t = c0 + tid, page = a.table[s * a.ld + t / a.page_size];
            const bool ok = page >= 0 && page < a.n_pages;
            if (!ok) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWherePaged, s);
            slots[tid] = ok ? (int64_t)page * a.page_size + t % a.page_size : -1;
        }
        __syncthreads();
        for (int i = warp; i < n; i += kPagedThreads / 32) {
            float x = 0.f;
            if (slots[i] >= 0) {
                const int64_t row = slots[i] * a.Hkv + g;
                for (int d = lane; d < D; d += 32) {
                    if (F8) {
                        float f[16];
                        const uint32_t c = static_cast<const uint8_t *>(a.k)[row * D + d];
                        e4m3x16_to_f32(make_uint4(c, 0, 0, 0), f);
                        x = fmaf(qs[d], f[0] * a.k_scales[row * (D / 128) + d / 128], x);
                    } else {
                        x = fmaf(qs[d], bf16_bits_to_float(static_cast<const uint16_t *>(a.k)[row * D + d]), x);
                    }
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) w[i] = slots[i] >= 0 ? x : -INFINITY;
        }
        __syncthreads();
        float mn = m;
        for (int i = 0; i < n; ++i) mn = fmaxf(mn, w[i]);
        const float ref = mn == -INFINITY ? 0.f : mn, alpha = exp2f(m - ref);
        l *= alpha;
        acc *= alpha;
        for (int i = 0; i < n; ++i) {
            const float p = exp2f(w[i] - ref);
            l += p;
            if (tid < D && slots[i] >= 0) {
                const int64_t row = slots[i] * a.Hkv + g;
                float v;
                if (F8) {
                    float f[16];
                    const uint32_t c = static_cast<const uint8_t *>(a.v)[row * D + tid];
                    e4m3x16_to_f32(make_uint4(c, 0, 0, 0), f);
                    v = f[0] * a.v_scales[row * (D / 128) + tid / 128];
                } else {
                    v = bf16_bits_to_float(static_cast<const uint16_t *>(a.v)[row * D + tid]);
                }
                acc = fmaf(p, v, acc);
            }
        }
        m = mn;
    }
    if (tid < D) a.out[((int64_t)s * a.Hq + h) * D + tid] = float_to_bf16_bits(l > 0.f ? acc / l : 0.f);
    if (tid == 0 && a.lse) a.lse[(int64_t)s * a.Hq + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int D, bool F8>
cudaError_t launch(const PagedArgs &a, cudaStream_t st) {
    paged_plain_kernel<D, F8><<<dim3(a.Hq, a.B), kPagedThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t paged_scratch_bytes(int, int, int) { return 0; }

cudaError_t launch_paged_decode(const PagedArgs &a, int D, bool fp8, cudaStream_t st) {
    switch (D) {
        case 64: return fp8 ? cudaErrorInvalidValue : launch<64, false>(a, st);
        case 128: return fp8 ? launch<128, true>(a, st) : launch<128, false>(a, st);
        case 256: return fp8 ? launch<256, true>(a, st) : launch<256, false>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qsa
