// Attention of one new token that accumulates what every cached token received (qsa_paged_decode_weights, _fp8kv):
//   weights[s][j] += sum_h 2^(score[s][h][j] - lse2[s][h]).
//
// A weight needs its head's final log-sum-exp, which is known only when all of the sequence has been read. Reading K again for
// it would cost half of the call's bytes once more; instead the tile kernel (paged_decode.cuh) keeps the fp32 scores, 4 Hq
// bytes a token beside the 4 Hkv D bytes of its bf16 rows (a 32nd of them with 16 query heads over 2 KV heads of 256 dims), and
// the kernel here turns them into weights, mostly out of L2.
#include "paged_decode.cuh"

namespace qsa {

namespace {

constexpr int kWeightThreads = 256;

// A warp for each tile of T tokens; a lane has T / 32 neighbouring tokens and sums their heads in order.
template <int T>
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(PagedArgs a, WeightArgs wt) {
    constexpr int E = T / 32, U = 8;
    const int lane = threadIdx.x & 31;
    wait_for_previous();
    const int64_t n = *wt.n_tiles, held = min(n, wt.cap);
    if (n > wt.cap && blockIdx.x == 0 && threadIdx.x == 0) record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereWeights, -1);
    const int64_t warps = (int64_t)gridDim.x * (kWeightThreads / 32);
    for (int64_t x = (int64_t)(threadIdx.x >> 5) * gridDim.x + blockIdx.x; x < held; x += warps) {
        const int2 place = wt.tiles[x];
        const int64_t j0 = (int64_t)place.y * T + lane * E;
        const float *score = wt.scores + x * a.Hq * T + lane * E;
        const float *lse2 = wt.lse2 + (int64_t)place.x * a.Hq;
        const int len = a.seq_len[place.x], lo = a.window > 0 ? max(0, len - a.window) : 0;
        float sum[E] = {};
        for (int h0 = 0; h0 < a.Hq; h0 += U) {
            float v[U][E], l[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = min(h0 + u, a.Hq - 1);
                l[u] = lse2[h];
                if constexpr (E == 2)
                    *reinterpret_cast<float2 *>(v[u]) = *reinterpret_cast<const float2 *>(score + h * T);
                else
                    *reinterpret_cast<float4 *>(v[u]) = *reinterpret_cast<const float4 *>(score + h * T);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h0 + u < a.Hq)
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[e] += v[u][e] == -INFINITY ? 0.f : ex2(v[u][e] - l[u]);
        }
        float *w = wt.weights + place.x * wt.weights_ld;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t j = j0 + e;
            if (j < lo || j >= len) continue;
            if (j < wt.weights_ld)
                w[j] += sum[e];
            else
                record_error(a.hdr, QSA_ERR_DEVICE_BOUNDS, kWhereWeights, place.x);
        }
    }
}

}  // namespace

int paged_tile_tokens(bool fp8) { return fp8 ? PagedCfg<128, 8, true>::tile : PagedCfg<128, 8, false>::tile; }

cudaError_t launch_paged_decode_weights(const PagedArgs &a, const WeightArgs &w, int D, bool fp8, cudaStream_t st) {
    const cudaError_t e = launch_dims<true>(a, w, D, fp8, st);
    if (e != cudaSuccess) return e;
    const int T = paged_tile_tokens(fp8);
    // a warp for each tile that the table has room for, up to eight CTAs for each of 152 SMs
    const int64_t room = (int64_t)a.B * (((int64_t)a.ld * a.page_size + T - 1) / T + 1);
    const unsigned ctas = (unsigned)std::max<int64_t>(1, std::min<int64_t>((room + kWeightThreads / 32 - 1) / (kWeightThreads / 32), 152 * 8));
    return fp8 ? launch_dependent(weights_kernel<PagedCfg<128, 8, true>::tile>, dim3(ctas), kWeightThreads, 0, st, a, w)
               : launch_dependent(weights_kernel<PagedCfg<128, 8, false>::tile>, dim3(ctas), kWeightThreads, 0, st, a, w);
}

}  // namespace qsa
