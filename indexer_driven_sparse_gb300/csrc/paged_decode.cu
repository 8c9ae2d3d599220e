// qsa_paged_decode and qsa_paged_decode_fp8kv: the kernels of paged_decode.cuh as they are.
#include "paged_decode.cuh"

namespace qsa {

size_t paged_scratch_bytes(int D, int Hq, int Hkv) {
    const size_t slots = 2 * (size_t)ranges_for(max_ctas(D), Hkv) * Hq;
    return kMaxRanges * sizeof(int2) + (slots * sizeof(float2) + 255) / 256 * 256 + slots * D * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedArgs &a, int D, bool fp8, cudaStream_t st) {
    return launch_dims<false>(a, WeightArgs{}, D, fp8, st);
}

}  // namespace qsa
