// Internal declarations of the paged-cache operators (rope.cu, paged_decode.cu, pages.cu, paged_api.cu).
#pragma once

#include "qsa_internal.cuh"

namespace qsa {

constexpr int kWhereAppend = 9, kWherePaged = 10, kWherePages = 11;

// Programmatic dependent launch: a kernel launched by launch_dependent may begin while the kernel before it on the
// stream ends; it waits for that one's memory before its first access. Every kernel here does that at its start, so
// each still follows all that came before it; the short streaming ones also let the next one begin at once. What such a
// kernel reads may thus be written while it already exists: ordinary loads only, since the read-only path (__ldg) is
// for memory that stays the same from the kernel's beginning. The rotary phases do.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct RopeArgs {
    const uint64_t *phase;    // turns per token as a 64-bit fraction, one per pair
    float amplitude;
    int32_t D, begin, rot, interleaved;
};

struct RopeRows {
    const uint16_t *x;
    uint16_t *out;
    int64_t x_ld, out_ld;     // elements between tokens
    const int32_t *pos;
    int32_t N, H;
};
cudaError_t launch_rope(const RopeArgs &r, const RopeRows &a, cudaStream_t st);

struct AppendArgs {
    const uint16_t *q, *k, *v;   // q may be nullptr
    int64_t q_ld, k_ld, v_ld;
    const int32_t *seq, *pos;    // seq may be nullptr: token n is row n
    int32_t N, Hq, Hkv;
    uint16_t *q_out;
    int64_t q_out_ld;
    uint16_t *k_cache, *v_cache; // bf16 rows (nullptr with FP8 rows)
    uint8_t *k_codes, *v_codes;  // FP8 rows
    float *k_scales, *v_scales;
    int64_t n_pages;
    const int32_t *table;
    int64_t ld;
    int32_t n_rows, page_size;
    WsHeader *hdr;
};
cudaError_t launch_rope_append(const RopeArgs &r, const AppendArgs &a, cudaStream_t st);

struct PagedArgs {
    const uint16_t *q;
    int64_t q_ld;
    const void *k, *v;                  // bf16 rows, or E4M3 codes
    const float *k_scales, *v_scales;   // nullptr with bf16 rows
    int64_t n_pages;
    const int32_t *table;
    int64_t ld;
    const int32_t *seq_len;
    int32_t B, Hq, Hkv, G, page_size, window;
    int32_t tile_entries, tile_rest;    // a tile's tokens / page_size and the remainder (set by the launcher)
    int32_t page_shift;                 // log2 of page_size, -1: no power of two (set by the launcher)
    float scale_log2;
    uint16_t *out;
    float *lse;
    WsHeader *hdr;
    char *scratch;                      // the workspace behind its status block
};
size_t paged_scratch_bytes(int D, int Hq, int Hkv);
cudaError_t launch_paged_decode(const PagedArgs &a, int D, bool fp8, cudaStream_t st);

struct PlaneGroup {
    char *src, *dst;
    int64_t src_stride, dst_stride, page_bytes;
    int32_t n_planes, wide;             // wide: 16-byte words, else 4-byte words
};
struct PlaneGroups {
    PlaneGroup g[QSA_MAX_PLANE_GROUPS];
    int32_t n;
};
struct ForkArgs {
    const int32_t *parent, *add, *table, *seq_len, *ref;
    int32_t *table_out, *seq_len_out, *ref_out;
    int32_t n_out, n_in, page_size, n_pages;
    int32_t page_shift;                 // log2 of page_size, -1: no power of two (set by the launcher)
    int64_t ld;
    WsHeader *hdr;
    char *scratch;
};
struct CompactArgs {
    const int32_t *table, *seq_len, *ref;
    int32_t *table_out, *ref_out;
    int32_t n_rows, page_size, n_pages;
    int64_t ld;
    WsHeader *hdr;
    char *scratch;
};
size_t pages_scratch_bytes(int n_rows, int64_t n_pages);
cudaError_t launch_fork_pages(const ForkArgs &a, const PlaneGroups &p, cudaStream_t st);
cudaError_t launch_compact_pages(const CompactArgs &a, const PlaneGroups &p, cudaStream_t st);
cudaError_t launch_copy_pages(const int32_t *src, const int32_t *dst, int n, const PlaneGroups &p, int64_t n_src,
                              int64_t n_dst, WsHeader *hdr, cudaStream_t st);

// Host checks shared with qsa_api.cu.
bool device_accessible(const void *p);
qsa_status host_ok();

}  // namespace qsa
