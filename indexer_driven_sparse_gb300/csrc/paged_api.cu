// extern "C" entry points of the paged-cache operators: host-side validation and launch on the caller's stream.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "paged.cuh"

using namespace qsa;

namespace {

qsa_status fail(qsa_status s, const char *call, const char *fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    return host_fail(s, call, text);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define QSA_TRY(expr)                \
    do {                             \
        const qsa_status _s = (expr); \
        if (_s != QSA_OK) return _s; \
    } while (0)

#define QSA_NEED(call, cond, ...)                                              \
    do {                                                                       \
        if (!(cond)) return fail(QSA_ERR_INVALID_ARGUMENT, call, __VA_ARGS__); \
    } while (0)

qsa_status launched(cudaError_t e, const char *call) {
    if (e != cudaSuccess) return fail(QSA_ERR_CUDA, call, "launch: %s", cudaGetErrorString(e));
    return host_ok();
}

qsa_status check_rope(const char *call, const qsa_rope_config *r) {
    QSA_NEED(call, r != nullptr, "rope is NULL");
    if (r->head_dim < 16 || r->head_dim > 1024 || r->head_dim % 16 != 0)
        return fail(QSA_ERR_UNSUPPORTED, call, "rope head_dim %d (a multiple of 16 up to 1024)", r->head_dim);
    if (r->rot_dim < 0 || r->rot_dim % 16 != 0 || r->rot_begin < 0 || r->rot_begin % 8 != 0)
        return fail(QSA_ERR_UNSUPPORTED, call, "rot_dim %d (a multiple of 16) at rot_begin %d (a multiple of 8)",
                    r->rot_dim, r->rot_begin);
    QSA_NEED(call, (int64_t)r->rot_begin + r->rot_dim <= r->head_dim, "rot_begin %d + rot_dim %d exceed head_dim %d",
             r->rot_begin, r->rot_dim, r->head_dim);
    return QSA_OK;
}

qsa_status check_paged(const char *call, const qsa_paged_config *c, bool fp8) {
    QSA_NEED(call, c != nullptr, "config is NULL");
    if (c->head_dim != 256 && c->head_dim != 128 && (c->head_dim != 64 || fp8))
        return fail(QSA_ERR_UNSUPPORTED, call, "head_dim %d (64, 128 or 256; FP8 rows 128 or 256)", c->head_dim);
    QSA_NEED(call, c->n_kv_heads >= 1 && c->n_q_heads >= 1, "head counts must be positive (%d, %d)", c->n_q_heads,
             c->n_kv_heads);
    if (c->n_q_heads % c->n_kv_heads != 0 || c->n_q_heads / c->n_kv_heads > 16)
        return fail(QSA_ERR_UNSUPPORTED, call, "%d query heads over %d KV heads (a multiple, at most 16 each)",
                    c->n_q_heads, c->n_kv_heads);
    if (c->n_q_heads > 4096) return fail(QSA_ERR_UNSUPPORTED, call, "n_q_heads %d (at most 4096)", c->n_q_heads);
    QSA_NEED(call, c->page_size >= 1, "page_size %d must be positive", c->page_size);
    QSA_NEED(call, c->window >= 0, "window %d must not be negative", c->window);
    QSA_NEED(call, c->softmax_scale <= 0.f || isfinite(c->softmax_scale), "softmax_scale must be finite");
    return QSA_OK;
}

qsa_status check_workspace(const char *call, const void *ws, size_t bytes, size_t need) {
    QSA_NEED(call, ws != nullptr, "workspace is NULL");
    QSA_NEED(call, aligned(ws, 256), "workspace must be 256-byte aligned");
    if (bytes < need)
        return fail(QSA_ERR_WORKSPACE_TOO_SMALL, call, "workspace %zu bytes < %zu needed", bytes, need);
    return QSA_OK;
}

size_t paged_ws(const qsa_paged_config *c) {
    return kWsHeaderBytes + paged_scratch_bytes(c->head_dim, c->n_q_heads, c->n_kv_heads);
}

// A pool's size and a page table over it.
qsa_status check_table(const char *call, const qsa_paged_config *c, int64_t n_pages, int64_t ld) {
    QSA_NEED(call, n_pages >= 0 && ld >= 0, "negative size");
    if (n_pages > INT32_MAX / c->page_size)
        return fail(QSA_ERR_UNSUPPORTED, call, "n_pages %lld x page_size %d exceed 2^31 - 1 tokens", (long long)n_pages,
                    c->page_size);
    QSA_NEED(call, ld <= INT32_MAX, "table_ld too large");
    return QSA_OK;
}

RopeArgs rope_args(const qsa_rope_config *r, const uint64_t *phase, float amplitude) {
    RopeArgs a{};
    a.phase = phase;
    a.amplitude = amplitude;
    a.D = r->head_dim;
    a.begin = r->rot_begin;
    a.rot = r->rot_dim;
    a.interleaved = r->interleaved != 0;
    return a;
}

qsa_status check_rows(const char *call, const char *name, const void *p, int64_t ld, int64_t width) {
    QSA_NEED(call, p != nullptr, "%s is NULL", name);
    QSA_NEED(call, aligned(p, 16), "%s must be 16-byte aligned", name);
    QSA_NEED(call, ld >= width && ld % 8 == 0, "%s: %lld elements between rows (a multiple of 8, at least %lld)", name,
             (long long)ld, (long long)width);
    return QSA_OK;
}

}  // namespace

extern "C" {

QSA_API qsa_status qsa_rope_table(const qsa_rope_config *rope, uint64_t *phase, float *amplitude) {
    const char *call = "qsa_rope_table";
    QSA_TRY(check_rope(call, rope));
    QSA_NEED(call, amplitude != nullptr && (phase != nullptr || rope->rot_dim == 0), "phase and amplitude must be non-NULL");
    QSA_NEED(call, isfinite(rope->base) && rope->base > 1.0, "base must be finite and above 1");
    const int scaling = rope->scaling, half = rope->rot_dim / 2;
    QSA_NEED(call, scaling >= QSA_ROPE_NONE && scaling <= QSA_ROPE_BY_PARTS, "scaling %d unknown", scaling);
    QSA_NEED(call, scaling == QSA_ROPE_NONE || (isfinite(rope->factor) && rope->factor > 0.0),
             "factor must be finite and positive");
    double base = rope->base, lo = 0.0, hi = 0.0;
    *amplitude = 1.f;
    if (scaling == QSA_ROPE_NTK && rope->rot_dim > 2)
        base *= pow(rope->factor, rope->rot_dim / (rope->rot_dim - 2.0));
    QSA_NEED(call, isfinite(base) && base > 0.0, "factor %g takes the base out of range", rope->factor);
    if (scaling == QSA_ROPE_BY_PARTS) {
        QSA_NEED(call, rope->original_len > 0, "original_len must be positive");
        QSA_NEED(call, isfinite(rope->beta_fast) && rope->beta_slow > 0.0 && rope->beta_fast > rope->beta_slow,
                 "beta_fast must be above beta_slow, and both positive");
        auto at = [&](double beta) { return half * log(rope->original_len / (beta * 2.0 * M_PI)) / log(base); };
        lo = std::max(floor(at(rope->beta_fast)), 0.0);
        hi = std::min(ceil(at(rope->beta_slow)), rope->rot_dim - 1.0);    // in dims, not pairs: the ramp may end past the last pair
        if (rope->factor > 1.0) *amplitude = (float)(0.1 * log(rope->factor) + 1.0);
    }
    for (int i = 0; i < half; ++i) {
        double f = pow(base, -2.0 * i / rope->rot_dim);
        if (scaling == QSA_ROPE_LINEAR) f /= rope->factor;
        if (scaling == QSA_ROPE_BY_PARTS) {
            const double g = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
            f = f * (1.0 - g) + f / rope->factor * g;
        }
        QSA_NEED(call, isfinite(f), "factor %g makes pair %d's frequency infinite", rope->factor, i);
        const double turn = f / (2.0 * M_PI);
        phase[i] = (uint64_t)ldexp(turn - floor(turn), 64);   // below 2^64: the fraction is at most 1 - 2^-53
    }
    return host_ok();
}

QSA_API qsa_status qsa_rope(const qsa_rope_config *rope, const uint64_t *phase, float amplitude, const qsa_bf16 *x,
                            int64_t x_ld, const int32_t *pos, int32_t N, int32_t n_heads, qsa_bf16 *out,
                            int64_t out_ld, qsa_stream stream) {
    const char *call = "qsa_rope";
    QSA_TRY(check_rope(call, rope));
    QSA_NEED(call, N >= 0 && n_heads >= 0, "negative size");
    if (n_heads > 65535) return fail(QSA_ERR_UNSUPPORTED, call, "n_heads %d (at most 65535)", n_heads);
    if (N == 0 || n_heads == 0) return host_ok();
    const int64_t width = (int64_t)n_heads * rope->head_dim;
    QSA_TRY(check_rows(call, "x", x, x_ld, width));
    QSA_TRY(check_rows(call, "out", out, out_ld, width));
    QSA_NEED(call, x != out || x_ld == out_ld, "in place needs out_ld = x_ld");
    QSA_NEED(call, pos != nullptr && (phase != nullptr || rope->rot_dim == 0), "NULL tensor pointer");
    QSA_NEED(call, aligned(pos, 4) && aligned(phase, 16), "pos must be 4-byte and phase 16-byte aligned");
    const RopeRows rows{x, out, x_ld, out_ld, pos, N, n_heads};
    return launched(launch_rope(rope_args(rope, phase, amplitude), rows, static_cast<cudaStream_t>(stream)), call);
}

QSA_API size_t qsa_paged_workspace_size(const qsa_paged_config *cfg) {
    return check_paged("qsa_paged_workspace_size", cfg, false) == QSA_OK ? paged_ws(cfg) : 0;
}

}  // extern "C"

namespace {

// qsa_rope_append into bf16 or FP8 rows; the caller has set a's cache pointers.
qsa_status rope_append(const char *call, const qsa_paged_config *cfg, const qsa_rope_config *rope, const uint64_t *phase,
                       float amplitude, AppendArgs a, void *ws, size_t ws_bytes, qsa_stream stream, bool fp8) {
    QSA_TRY(check_paged(call, cfg, fp8));
    QSA_TRY(check_rope(call, rope));
    QSA_NEED(call, rope->head_dim == cfg->head_dim, "rope head_dim %d, cache head_dim %d", rope->head_dim, cfg->head_dim);
    QSA_NEED(call, a.N >= 0 && a.n_rows >= 0, "negative size");
    QSA_TRY(check_table(call, cfg, a.n_pages, a.ld));
    QSA_TRY(check_workspace(call, ws, ws_bytes, kWsHeaderBytes));
    if (a.N == 0) return host_ok();
    a.Hq = cfg->n_q_heads;
    a.Hkv = cfg->n_kv_heads;
    a.page_size = cfg->page_size;
    a.hdr = static_cast<WsHeader *>(ws);
    const int64_t q_width = (int64_t)a.Hq * cfg->head_dim, kv_width = (int64_t)a.Hkv * cfg->head_dim;
    if (a.q != nullptr) {
        QSA_TRY(check_rows(call, "q", a.q, a.q_ld, q_width));
        QSA_TRY(check_rows(call, "q_out", a.q_out, a.q_out_ld, q_width));
        QSA_NEED(call, a.q != a.q_out || a.q_ld == a.q_out_ld, "in place needs q_out_ld = q_ld");
    }
    QSA_TRY(check_rows(call, "k", a.k, a.k_ld, kv_width));
    QSA_TRY(check_rows(call, "v", a.v, a.v_ld, kv_width));
    QSA_NEED(call, a.pos && a.table && (phase != nullptr || rope->rot_dim == 0), "NULL tensor pointer");
    QSA_NEED(call, aligned(phase, 16), "phase must be 16-byte aligned");
    QSA_NEED(call, aligned(a.pos, 4) && aligned(a.seq, 4) && aligned(a.table, 4), "pos, seq and table must be 4-byte aligned");
    QSA_NEED(call, aligned(a.place, 4) && aligned(a.positions, 4), "place and positions must be 4-byte aligned");
    QSA_NEED(call, a.positions == nullptr || a.positions_ld >= 0, "positions_ld must not be negative");
    if (fp8) {
        QSA_NEED(call, a.k_codes && a.v_codes && a.k_scales && a.v_scales, "NULL tensor pointer");
        QSA_NEED(call, aligned(a.k_codes, 16) && aligned(a.v_codes, 16) && aligned(a.k_scales, 8) && aligned(a.v_scales, 8),
                 "codes must be 16-byte and scales 8-byte aligned");
    } else {
        QSA_NEED(call, a.k_cache && a.v_cache, "NULL tensor pointer");
        QSA_NEED(call, aligned(a.k_cache, 16) && aligned(a.v_cache, 16), "k_cache and v_cache must be 16-byte aligned");
    }
    QSA_NEED(call, fp8 ? device_accessible(a.k_codes) && device_accessible(a.v_codes) && device_accessible(a.k_scales) &&
                             device_accessible(a.v_scales)
                       : device_accessible(a.k_cache) && device_accessible(a.v_cache),
             "the K/V rows (and their scales) must be device memory or mapped pinned host memory");
    return launched(launch_rope_append(rope_args(rope, phase, amplitude), a, static_cast<cudaStream_t>(stream)), call);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// What qsa_paged_decode_weights keeps behind qsa_paged_decode's workspace: the batch's log-sum-exps and tile count, then for
// each tile its row and the scores of its tokens.
size_t weights_fixed(const qsa_paged_config *c, int32_t B) {
    return up256(paged_ws(c)) + 256 + up256((size_t)B * c->n_q_heads * sizeof(float));
}
size_t weights_per_tile(const qsa_paged_config *c, bool fp8) {
    return sizeof(int2) + (size_t)paged_tile_tokens(fp8) * c->n_q_heads * sizeof(float);
}

// weights: w.weights is set (the rest of w is filled in here).
qsa_status paged_decode(const char *call, const qsa_paged_config *cfg, PagedArgs a, void *ws, size_t ws_bytes,
                        qsa_stream stream, bool fp8, WeightArgs w = WeightArgs{}, bool weights = false) {
    QSA_TRY(check_paged(call, cfg, fp8));
    QSA_NEED(call, a.B >= 0 && a.B <= 65535, "B = %d out of range [0, 65535]", a.B);
    QSA_TRY(check_table(call, cfg, a.n_pages, a.ld));
    QSA_TRY(check_workspace(call, ws, ws_bytes, weights ? weights_fixed(cfg, a.B) : paged_ws(cfg)));
    QSA_NEED(call, !weights || w.weights_ld >= 0, "weights_ld must not be negative");
    if (a.B == 0) return host_ok();
    QSA_NEED(call, !weights || w.weights != nullptr, "weights is NULL");
    QSA_NEED(call, aligned(w.weights, 4), "weights must be 4-byte aligned");
    QSA_TRY(check_rows(call, "q", a.q, a.q_ld, (int64_t)cfg->n_q_heads * cfg->head_dim));
    QSA_NEED(call, a.k && a.v && a.table && a.seq_len && a.out && (!fp8 || (a.k_scales && a.v_scales)),
             "NULL tensor pointer");
    QSA_NEED(call, aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.out, 16),
             "the K/V rows and out must be 16-byte aligned");
    QSA_NEED(call, !fp8 || (aligned(a.k_scales, 8) && aligned(a.v_scales, 8)), "scales must be 8-byte aligned");
    QSA_NEED(call, aligned(a.table, 4) && aligned(a.seq_len, 4) && aligned(a.lse, 4),
             "table, seq_len and lse must be 4-byte aligned");
    QSA_NEED(call, device_accessible(a.k) && device_accessible(a.v) &&
                 (!fp8 || (device_accessible(a.k_scales) && device_accessible(a.v_scales))),
             "the K/V rows (and their scales) must be device memory or mapped pinned host memory");
    a.Hq = cfg->n_q_heads;
    a.Hkv = cfg->n_kv_heads;
    a.G = a.Hq / a.Hkv;
    a.page_size = cfg->page_size;
    a.window = cfg->window;
    a.scale_log2 = (cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.0f / sqrtf((float)cfg->head_dim)) * kLog2e;
    a.hdr = static_cast<WsHeader *>(ws);
    a.scratch = static_cast<char *>(ws) + kWsHeaderBytes;
    if (weights) {
        char *at = static_cast<char *>(ws) + up256(paged_ws(cfg));
        w.n_tiles = reinterpret_cast<int32_t *>(at);
        w.lse2 = reinterpret_cast<float *>(at + 256);
        at = static_cast<char *>(ws) + weights_fixed(cfg, a.B);
        // the scores first: 16-byte vectors
        w.cap = (int64_t)((ws_bytes - weights_fixed(cfg, a.B)) / weights_per_tile(cfg, fp8));
        w.scores = reinterpret_cast<float *>(at);
        w.tiles = reinterpret_cast<int2 *>(at + (size_t)w.cap * (weights_per_tile(cfg, fp8) - sizeof(int2)));
        return launched(launch_paged_decode_weights(a, w, cfg->head_dim, fp8, static_cast<cudaStream_t>(stream)), call);
    }
    return launched(launch_paged_decode(a, cfg->head_dim, fp8, static_cast<cudaStream_t>(stream)), call);
}

qsa_status check_drafts(const char *call, int32_t max_draft) {
    if (max_draft < 1 || max_draft > QSA_MAX_DRAFT)
        return fail(QSA_ERR_UNSUPPORTED, call, "max_draft %d (1 to %d)", max_draft, QSA_MAX_DRAFT);
    return QSA_OK;
}

size_t tree_ws(const qsa_paged_config *c, int32_t max_draft) {
    return kWsHeaderBytes + tree_scratch_bytes(c->head_dim, c->n_q_heads, c->n_kv_heads, max_draft);
}

qsa_status tree_decode(const char *call, const qsa_paged_config *cfg, TreeArgs a, void *ws, size_t ws_bytes,
                       qsa_stream stream, bool fp8) {
    QSA_TRY(check_paged(call, cfg, fp8));
    QSA_TRY(check_drafts(call, a.max_draft));
    QSA_NEED(call, a.B >= 0 && a.B <= 65535, "B = %d out of range [0, 65535]", a.B);
    QSA_NEED(call, a.N >= 0, "N must not be negative");
    QSA_TRY(check_table(call, cfg, a.n_pages, a.ld));
    QSA_TRY(check_workspace(call, ws, ws_bytes, tree_ws(cfg, a.max_draft)));
    if (a.B == 0 || a.N == 0) return host_ok();
    QSA_TRY(check_rows(call, "q", a.q, a.q_ld, (int64_t)cfg->n_q_heads * cfg->head_dim));
    QSA_NEED(call, a.draft_off && a.parent && a.k && a.v && a.table && a.seq_len && a.out &&
                       (!fp8 || (a.k_scales && a.v_scales)),
             "NULL tensor pointer");
    QSA_NEED(call, aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.out, 16),
             "the K/V rows and out must be 16-byte aligned");
    QSA_NEED(call, !fp8 || (aligned(a.k_scales, 8) && aligned(a.v_scales, 8)), "scales must be 8-byte aligned");
    QSA_NEED(call, aligned(a.table, 4) && aligned(a.seq_len, 4) && aligned(a.lse, 4) && aligned(a.draft_off, 4) &&
                 aligned(a.parent, 4),
             "table, seq_len, draft_off, parent and lse must be 4-byte aligned");
    QSA_NEED(call, device_resident(a.k) && device_resident(a.v) &&
                 (!fp8 || (device_resident(a.k_scales) && device_resident(a.v_scales))),
             "the K/V rows (and their scales) must be device memory");
    a.Hq = cfg->n_q_heads;
    a.Hkv = cfg->n_kv_heads;
    a.G = a.Hq / a.Hkv;
    a.page_size = cfg->page_size;
    a.window = cfg->window;
    a.scale_log2 = (cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.0f / sqrtf((float)cfg->head_dim)) * kLog2e;
    a.hdr = static_cast<WsHeader *>(ws);
    a.scratch = static_cast<char *>(ws) + kWsHeaderBytes;
    return launched(launch_tree_decode(a, cfg->head_dim, fp8, static_cast<cudaStream_t>(stream)), call);
}

constexpr int kMaxPageRows = 65536;

qsa_status plane_groups(const char *call, const qsa_page_planes *from, const qsa_page_planes *to, int32_t n,
                        PlaneGroups *out) {
    QSA_NEED(call, n >= 0 && n <= QSA_MAX_PLANE_GROUPS, "n_groups = %d out of range [0, %d]", n, QSA_MAX_PLANE_GROUPS);
    QSA_NEED(call, n == 0 || from != nullptr, "planes is NULL");
    memset(out, 0, sizeof(*out));
    out->n = n;
    for (int i = 0; i < n; ++i) {
        const qsa_page_planes &s = from[i], &d = to ? to[i] : from[i];
        QSA_NEED(call, s.n_planes >= 0 && s.page_bytes >= 0, "planes[%d]: negative size", i);
        QSA_NEED(call, s.n_planes == d.n_planes && s.page_bytes == d.page_bytes, "planes[%d]: source and destination differ",
                 i);
        QSA_NEED(call, s.base && d.base, "planes[%d]: base is NULL", i);
        const size_t word = s.page_bytes % 16 == 0 ? 16 : 4;
        QSA_NEED(call, s.page_bytes % 4 == 0, "planes[%d]: page_bytes %lld must be a multiple of 4", i,
                 (long long)s.page_bytes);
        QSA_NEED(call, aligned(s.base, word) && aligned(d.base, word) && s.plane_stride % (int64_t)word == 0 &&
                     d.plane_stride % (int64_t)word == 0,
                 "planes[%d]: base and plane_stride must be %zu-byte aligned", i, word);
        PlaneGroup &g = out->g[i];
        g.src = static_cast<char *>(s.base);
        g.dst = static_cast<char *>(d.base);
        g.src_stride = s.plane_stride;
        g.dst_stride = d.plane_stride;
        g.page_bytes = s.page_bytes;
        g.n_planes = s.n_planes;
        g.wide = word == 16;
    }
    return QSA_OK;
}

qsa_status check_planes_memory(const char *call, const PlaneGroups &p) {
    for (int i = 0; i < p.n; ++i)
        QSA_NEED(call, device_accessible(p.g[i].src) && (p.g[i].src == p.g[i].dst || device_accessible(p.g[i].dst)),
                 "planes[%d] must be device memory or mapped pinned host memory", i);
    return QSA_OK;
}

qsa_status check_pool(const char *call, int32_t page_size, int64_t n_pages, int64_t ld) {
    QSA_NEED(call, page_size >= 1, "page_size %d must be positive", page_size);
    QSA_NEED(call, n_pages >= 0 && ld >= 0, "negative size");
    if (n_pages > (1 << 30)) return fail(QSA_ERR_UNSUPPORTED, call, "n_pages %lld (at most 2^30)", (long long)n_pages);
    QSA_NEED(call, ld <= INT32_MAX, "ld too large");
    return QSA_OK;
}

// The arguments that qsa_accept_drafts and qsa_evict_tokens share; the caller has set a's arrays.
qsa_status keep_args(const char *call, int32_t page_size, int32_t n_rows, int64_t ld, int64_t n_pages, int64_t max_tokens,
                     const qsa_page_planes *planes, int32_t n_groups, void *ws, size_t ws_bytes, KeepArgs *a,
                     PlaneGroups *groups) {
    QSA_TRY(check_pool(call, page_size, n_pages, ld));
    if (n_pages > INT32_MAX / page_size)
        return fail(QSA_ERR_UNSUPPORTED, call, "n_pages %lld x page_size %d exceed 2^31 - 1 tokens", (long long)n_pages, page_size);
    QSA_NEED(call, n_rows >= 0 && n_rows <= kMaxPageRows, "n_rows = %d out of range [0, %d]", n_rows, kMaxPageRows);
    QSA_TRY(plane_groups(call, planes, nullptr, n_groups, groups));
    for (int i = 0; i < groups->n; ++i) {
        PlaneGroup &g = groups->g[i];
        QSA_NEED(call, g.page_bytes % (4 * (int64_t)page_size) == 0,
                 "planes[%d]: page_bytes %lld must be a multiple of 4 bytes for each of %d tokens", i, (long long)g.page_bytes,
                 page_size);
        g.wide = g.wide && g.page_bytes / page_size % 16 == 0;      // a token's words
    }
    QSA_TRY(check_workspace(call, ws, ws_bytes, kWsHeaderBytes + keep_scratch_bytes(n_rows, max_tokens)));
    QSA_NEED(call, n_rows == 0 || (a->seq_len && a->seq_len_out && (ld == 0 || (a->table && a->table_out))), "NULL tensor pointer");
    QSA_NEED(call, n_pages == 0 || (a->ref && a->ref_out), "NULL tensor pointer");
    QSA_NEED(call, a->table == nullptr || a->table_out != a->table, "table_out must be another array than table");
    QSA_NEED(call, a->seq_len == nullptr || a->seq_len_out != a->seq_len, "seq_len_out must be another array than seq_len");
    QSA_NEED(call, a->ref == nullptr || a->ref_out != a->ref, "ref_out must be another array than ref");
    for (const void *p : {static_cast<const void *>(a->table), static_cast<const void *>(a->seq_len),
                          static_cast<const void *>(a->ref), static_cast<const void *>(a->table_out),
                          static_cast<const void *>(a->seq_len_out), static_cast<const void *>(a->ref_out)})
        QSA_NEED(call, aligned(p, 4), "the int32 arrays must be 4-byte aligned");
    a->n_rows = n_rows, a->page_size = page_size, a->n_pages = (int32_t)n_pages, a->ld = ld;
    a->page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1;
    a->hdr = static_cast<WsHeader *>(ws);
    a->scratch = static_cast<char *>(ws) + kWsHeaderBytes;
    return QSA_OK;
}

// qsa_accept_drafts[_weights]; the caller has set a's and d's arrays.
qsa_status accept_drafts(const char *call, int32_t page_size, KeepArgs a, const AcceptArgs &d, int32_t n_rows, int64_t ld,
                         int64_t n_pages, const qsa_page_planes *planes, int32_t n_groups, void *ws, size_t ws_bytes,
                         qsa_stream stream) {
    PlaneGroups groups;
    QSA_TRY(keep_args(call, page_size, n_rows, ld, n_pages, 0, planes, n_groups, ws, ws_bytes, &a, &groups));
    QSA_NEED(call, d.N >= 0 && d.positions_ld >= 0, "negative size");
    QSA_NEED(call, n_rows == 0 || (d.draft_off && d.accepted && (d.parent || d.N == 0)), "NULL tensor pointer");
    QSA_NEED(call, aligned(d.draft_off, 4) && aligned(d.parent, 4) && aligned(d.accepted, 4) && aligned(d.positions, 4) &&
                 aligned(d.weights, 4),
             "the arrays must be 4-byte aligned");
    if (n_rows == 0 && n_pages == 0) return host_ok();
    QSA_TRY(check_planes_memory(call, groups));
    return launched(launch_accept_drafts(a, d, groups, static_cast<cudaStream_t>(stream)), call);
}

}  // namespace

extern "C" {

QSA_API qsa_status qsa_rope_append(const qsa_paged_config *cfg, const qsa_rope_config *rope, const uint64_t *phase,
                                   float amplitude, const qsa_bf16 *q, int64_t q_ld, const qsa_bf16 *k, int64_t k_ld,
                                   const qsa_bf16 *v, int64_t v_ld, const int32_t *seq, const int32_t *pos, int32_t N,
                                   qsa_bf16 *q_out, int64_t q_out_ld, qsa_bf16 *k_cache, qsa_bf16 *v_cache,
                                   int64_t n_pages, const int32_t *table, int64_t table_ld, int32_t n_rows, void *ws,
                                   size_t ws_bytes, qsa_stream stream) {
    AppendArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.v = v, a.v_ld = v_ld;
    a.seq = seq, a.pos = pos, a.N = N, a.q_out = q_out, a.q_out_ld = q_out_ld;
    a.k_cache = k_cache, a.v_cache = v_cache;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.n_rows = n_rows;
    return rope_append("qsa_rope_append", cfg, rope, phase, amplitude, a, ws, ws_bytes, stream, false);
}

QSA_API qsa_status qsa_rope_append_fp8kv(const qsa_paged_config *cfg, const qsa_rope_config *rope,
                                         const uint64_t *phase, float amplitude, const qsa_bf16 *q, int64_t q_ld,
                                         const qsa_bf16 *k, int64_t k_ld, const qsa_bf16 *v, int64_t v_ld,
                                         const int32_t *seq, const int32_t *pos, int32_t N, qsa_bf16 *q_out,
                                         int64_t q_out_ld, uint8_t *k_codes, float *k_scales, uint8_t *v_codes,
                                         float *v_scales, int64_t n_pages, const int32_t *table, int64_t table_ld,
                                         int32_t n_rows, void *ws, size_t ws_bytes, qsa_stream stream) {
    AppendArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.v = v, a.v_ld = v_ld;
    a.seq = seq, a.pos = pos, a.N = N, a.q_out = q_out, a.q_out_ld = q_out_ld;
    a.k_codes = k_codes, a.k_scales = k_scales, a.v_codes = v_codes, a.v_scales = v_scales;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.n_rows = n_rows;
    return rope_append("qsa_rope_append_fp8kv", cfg, rope, phase, amplitude, a, ws, ws_bytes, stream, true);
}

QSA_API qsa_status qsa_rope_append_at(const qsa_paged_config *cfg, const qsa_rope_config *rope, const uint64_t *phase,
                                      float amplitude, const qsa_bf16 *q, int64_t q_ld, const qsa_bf16 *k, int64_t k_ld,
                                      const qsa_bf16 *v, int64_t v_ld, const int32_t *seq, const int32_t *pos,
                                      const int32_t *place, int32_t N, qsa_bf16 *q_out, int64_t q_out_ld,
                                      qsa_bf16 *k_cache, qsa_bf16 *v_cache, int64_t n_pages, const int32_t *table,
                                      int64_t table_ld, int32_t n_rows, int32_t *positions, int64_t positions_ld,
                                      void *ws, size_t ws_bytes, qsa_stream stream) {
    const char *call = "qsa_rope_append_at";
    QSA_NEED(call, place != nullptr || N <= 0, "place is NULL");
    AppendArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.v = v, a.v_ld = v_ld;
    a.seq = seq, a.pos = pos, a.place = place, a.N = N, a.q_out = q_out, a.q_out_ld = q_out_ld;
    a.k_cache = k_cache, a.v_cache = v_cache;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.n_rows = n_rows;
    a.positions = positions, a.positions_ld = positions_ld;
    return rope_append(call, cfg, rope, phase, amplitude, a, ws, ws_bytes, stream, false);
}

QSA_API qsa_status qsa_rope_append_at_fp8kv(const qsa_paged_config *cfg, const qsa_rope_config *rope,
                                            const uint64_t *phase, float amplitude, const qsa_bf16 *q, int64_t q_ld,
                                            const qsa_bf16 *k, int64_t k_ld, const qsa_bf16 *v, int64_t v_ld,
                                            const int32_t *seq, const int32_t *pos, const int32_t *place, int32_t N,
                                            qsa_bf16 *q_out, int64_t q_out_ld, uint8_t *k_codes, float *k_scales,
                                            uint8_t *v_codes, float *v_scales, int64_t n_pages, const int32_t *table,
                                            int64_t table_ld, int32_t n_rows, int32_t *positions, int64_t positions_ld,
                                            void *ws, size_t ws_bytes, qsa_stream stream) {
    const char *call = "qsa_rope_append_at_fp8kv";
    QSA_NEED(call, place != nullptr || N <= 0, "place is NULL");
    AppendArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.v = v, a.v_ld = v_ld;
    a.seq = seq, a.pos = pos, a.place = place, a.N = N, a.q_out = q_out, a.q_out_ld = q_out_ld;
    a.k_codes = k_codes, a.k_scales = k_scales, a.v_codes = v_codes, a.v_scales = v_scales;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.n_rows = n_rows;
    a.positions = positions, a.positions_ld = positions_ld;
    return rope_append(call, cfg, rope, phase, amplitude, a, ws, ws_bytes, stream, true);
}

QSA_API qsa_status qsa_paged_decode(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                    const qsa_bf16 *k_cache, const qsa_bf16 *v_cache, int64_t n_pages,
                                    const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                    qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, qsa_stream stream) {
    PagedArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k_cache, a.v = v_cache;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.seq_len = seq_len, a.B = B;
    a.out = out, a.lse = lse;
    return paged_decode("qsa_paged_decode", cfg, a, ws, ws_bytes, stream, false);
}

QSA_API qsa_status qsa_paged_decode_fp8kv(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                          const uint8_t *k_codes, const float *k_scales, const uint8_t *v_codes,
                                          const float *v_scales, int64_t n_pages, const int32_t *table,
                                          int64_t table_ld, const int32_t *seq_len, int32_t B, qsa_bf16 *out,
                                          float *lse, void *ws, size_t ws_bytes, qsa_stream stream) {
    PagedArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k_codes, a.v = v_codes, a.k_scales = k_scales, a.v_scales = v_scales;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.seq_len = seq_len, a.B = B;
    a.out = out, a.lse = lse;
    return paged_decode("qsa_paged_decode_fp8kv", cfg, a, ws, ws_bytes, stream, true);
}

QSA_API size_t qsa_paged_weights_workspace_size(const qsa_paged_config *cfg, int32_t B, int64_t n_tokens) {
    const char *call = "qsa_paged_weights_workspace_size";
    if (check_paged(call, cfg, false) != QSA_OK || B < 0 || B > 65535 || n_tokens < 0) return 0;
    // a sequence's first and last tile may each hold tokens that are not attended
    const auto bytes = [&](bool fp8) {
        const int64_t T = paged_tile_tokens(fp8);
        return weights_fixed(cfg, B) + (size_t)(n_tokens / T + 2 * (int64_t)B) * weights_per_tile(cfg, fp8);
    };
    return std::max(bytes(false), bytes(true));
}

QSA_API qsa_status qsa_paged_decode_weights(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                            const qsa_bf16 *k_cache, const qsa_bf16 *v_cache, int64_t n_pages,
                                            const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                            qsa_bf16 *out, float *lse, float *weights, int64_t weights_ld, void *ws,
                                            size_t ws_bytes, qsa_stream stream) {
    PagedArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k_cache, a.v = v_cache;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.seq_len = seq_len, a.B = B;
    a.out = out, a.lse = lse;
    WeightArgs w{};
    w.weights = weights, w.weights_ld = weights_ld;
    return paged_decode("qsa_paged_decode_weights", cfg, a, ws, ws_bytes, stream, false, w, true);
}

QSA_API qsa_status qsa_paged_decode_weights_fp8kv(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                                  const uint8_t *k_codes, const float *k_scales,
                                                  const uint8_t *v_codes, const float *v_scales, int64_t n_pages,
                                                  const int32_t *table, int64_t table_ld, const int32_t *seq_len,
                                                  int32_t B, qsa_bf16 *out, float *lse, float *weights,
                                                  int64_t weights_ld, void *ws, size_t ws_bytes, qsa_stream stream) {
    PagedArgs a{};
    a.q = q, a.q_ld = q_ld, a.k = k_codes, a.v = v_codes, a.k_scales = k_scales, a.v_scales = v_scales;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.seq_len = seq_len, a.B = B;
    a.out = out, a.lse = lse;
    WeightArgs w{};
    w.weights = weights, w.weights_ld = weights_ld;
    return paged_decode("qsa_paged_decode_weights_fp8kv", cfg, a, ws, ws_bytes, stream, true, w, true);
}

QSA_API size_t qsa_tree_workspace_size(const qsa_paged_config *cfg, int32_t max_draft) {
    const char *call = "qsa_tree_workspace_size";
    return check_paged(call, cfg, false) == QSA_OK && check_drafts(call, max_draft) == QSA_OK ? tree_ws(cfg, max_draft) : 0;
}

QSA_API qsa_status qsa_tree_decode(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                   const int32_t *draft_off, const int32_t *parent, int32_t N, int32_t max_draft,
                                   const qsa_bf16 *k_cache, const qsa_bf16 *v_cache, int64_t n_pages,
                                   const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                   qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, qsa_stream stream) {
    TreeArgs a{};
    a.q = q, a.q_ld = q_ld, a.draft_off = draft_off, a.parent = parent, a.N = N, a.max_draft = max_draft;
    a.k = k_cache, a.v = v_cache, a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.seq_len = seq_len, a.B = B;
    a.out = out, a.lse = lse;
    return tree_decode("qsa_tree_decode", cfg, a, ws, ws_bytes, stream, false);
}

QSA_API qsa_status qsa_tree_decode_fp8kv(const qsa_paged_config *cfg, const qsa_bf16 *q, int64_t q_ld,
                                         const int32_t *draft_off, const int32_t *parent, int32_t N,
                                         int32_t max_draft, const uint8_t *k_codes, const float *k_scales,
                                         const uint8_t *v_codes, const float *v_scales, int64_t n_pages,
                                         const int32_t *table, int64_t table_ld, const int32_t *seq_len, int32_t B,
                                         qsa_bf16 *out, float *lse, void *ws, size_t ws_bytes, qsa_stream stream) {
    TreeArgs a{};
    a.q = q, a.q_ld = q_ld, a.draft_off = draft_off, a.parent = parent, a.N = N, a.max_draft = max_draft;
    a.k = k_codes, a.v = v_codes, a.k_scales = k_scales, a.v_scales = v_scales;
    a.n_pages = n_pages, a.table = table, a.ld = table_ld, a.seq_len = seq_len, a.B = B;
    a.out = out, a.lse = lse;
    return tree_decode("qsa_tree_decode_fp8kv", cfg, a, ws, ws_bytes, stream, true);
}

QSA_API size_t qsa_pages_workspace_size(int32_t n_rows, int64_t n_pages) {
    if (n_rows < 0 || n_rows > kMaxPageRows || n_pages < 0 || n_pages > (1 << 30)) return 0;
    return kWsHeaderBytes + pages_scratch_bytes(n_rows, n_pages);
}

QSA_API qsa_status qsa_fork_pages(int32_t page_size, const int32_t *parent, const int32_t *add, int32_t n_out,
                                  const int32_t *table, const int32_t *seq_len, int32_t n_in, int64_t ld,
                                  const int32_t *ref, int64_t n_pages, int32_t *table_out, int32_t *seq_len_out,
                                  int32_t *ref_out, const qsa_page_planes *planes, int32_t n_groups, void *ws,
                                  size_t ws_bytes, qsa_stream stream) {
    const char *call = "qsa_fork_pages";
    QSA_TRY(check_pool(call, page_size, n_pages, ld));
    QSA_NEED(call, n_out >= 0 && n_out <= kMaxPageRows && n_in >= 0 && n_in <= kMaxPageRows,
             "n_in = %d, n_out = %d out of range [0, %d]", n_in, n_out, kMaxPageRows);
    ForkArgs a{};
    PlaneGroups groups;
    QSA_TRY(plane_groups(call, planes, nullptr, n_groups, &groups));
    QSA_TRY(check_workspace(call, ws, ws_bytes, qsa_pages_workspace_size(std::max(n_in, n_out), n_pages)));
    QSA_NEED(call, n_out == 0 || (parent && add && seq_len_out), "NULL tensor pointer");
    QSA_NEED(call, n_in == 0 || (seq_len && (table || ld == 0)), "NULL tensor pointer");
    QSA_NEED(call, n_out == 0 || ld == 0 || table_out, "NULL tensor pointer");
    QSA_NEED(call, n_pages == 0 || (ref && ref_out), "NULL tensor pointer");
    QSA_NEED(call, table == nullptr || table_out != table, "table_out must be another array than table");
    QSA_NEED(call, seq_len == nullptr || seq_len_out != seq_len, "seq_len_out must be another array than seq_len");
    QSA_NEED(call, ref == nullptr || ref_out != ref, "ref_out must be another array than ref");
    for (const void *p : {static_cast<const void *>(parent), static_cast<const void *>(add), static_cast<const void *>(table),
                          static_cast<const void *>(seq_len), static_cast<const void *>(ref),
                          static_cast<const void *>(table_out), static_cast<const void *>(seq_len_out),
                          static_cast<const void *>(ref_out)})
        QSA_NEED(call, aligned(p, 4), "the int32 arrays must be 4-byte aligned");
    if (n_out == 0 && n_in == 0 && n_pages == 0) return host_ok();
    QSA_TRY(check_planes_memory(call, groups));
    a.parent = parent, a.add = add, a.table = table, a.seq_len = seq_len, a.ref = ref;
    a.table_out = table_out, a.seq_len_out = seq_len_out, a.ref_out = ref_out;
    a.n_out = n_out, a.n_in = n_in, a.page_size = page_size, a.n_pages = (int32_t)n_pages, a.ld = ld;
    a.hdr = static_cast<WsHeader *>(ws);
    a.scratch = static_cast<char *>(ws) + kWsHeaderBytes;
    return launched(launch_fork_pages(a, groups, static_cast<cudaStream_t>(stream)), call);
}

QSA_API qsa_status qsa_compact_pages(int32_t page_size, const int32_t *table, const int32_t *seq_len, int32_t n_rows,
                                     int64_t ld, const int32_t *ref, int64_t n_pages, int32_t *table_out,
                                     int32_t *ref_out, const qsa_page_planes *planes, int32_t n_groups, void *ws,
                                     size_t ws_bytes, qsa_stream stream) {
    const char *call = "qsa_compact_pages";
    QSA_TRY(check_pool(call, page_size, n_pages, ld));
    QSA_NEED(call, n_rows >= 0 && n_rows <= kMaxPageRows, "n_rows = %d out of range [0, %d]", n_rows, kMaxPageRows);
    CompactArgs a{};
    PlaneGroups groups;
    QSA_TRY(plane_groups(call, planes, nullptr, n_groups, &groups));
    QSA_TRY(check_workspace(call, ws, ws_bytes, qsa_pages_workspace_size(n_rows, n_pages)));
    if (n_pages == 0 && n_rows == 0) return host_ok();
    QSA_NEED(call, n_rows == 0 || (seq_len && ((table && table_out) || ld == 0)), "NULL tensor pointer");
    QSA_NEED(call, n_pages == 0 || (ref && ref_out), "NULL tensor pointer");
    QSA_NEED(call, ref == nullptr || ref_out != ref, "ref_out must be another array than ref");
    for (const void *p : {static_cast<const void *>(table), static_cast<const void *>(seq_len), static_cast<const void *>(ref),
                          static_cast<const void *>(table_out), static_cast<const void *>(ref_out)})
        QSA_NEED(call, aligned(p, 4), "the int32 arrays must be 4-byte aligned");
    QSA_TRY(check_planes_memory(call, groups));
    a.table = table, a.seq_len = seq_len, a.ref = ref, a.table_out = table_out, a.ref_out = ref_out;
    a.n_rows = n_rows, a.page_size = page_size, a.n_pages = (int32_t)n_pages, a.ld = ld;
    a.hdr = static_cast<WsHeader *>(ws);
    a.scratch = static_cast<char *>(ws) + kWsHeaderBytes;
    return launched(launch_compact_pages(a, groups, static_cast<cudaStream_t>(stream)), call);
}

QSA_API size_t qsa_keep_workspace_size(int32_t n_rows, int64_t max_tokens) {
    if (n_rows < 0 || n_rows > kMaxPageRows || max_tokens < 0 || max_tokens > INT32_MAX) return 0;
    return kWsHeaderBytes + keep_scratch_bytes(n_rows, max_tokens);
}

QSA_API qsa_status qsa_accept_drafts(int32_t page_size, const int32_t *draft_off, const int32_t *parent, int32_t N,
                                     const int32_t *accepted, const int32_t *table, const int32_t *seq_len,
                                     int32_t n_rows, int64_t ld, const int32_t *ref, int64_t n_pages, int32_t *table_out,
                                     int32_t *seq_len_out, int32_t *ref_out, int32_t *positions, int64_t positions_ld,
                                     const qsa_page_planes *planes, int32_t n_groups, void *ws, size_t ws_bytes,
                                     qsa_stream stream) {
    AcceptArgs d{};
    d.draft_off = draft_off, d.parent = parent, d.accepted = accepted, d.N = N;
    d.positions = positions, d.positions_ld = positions_ld;
    KeepArgs a{};
    a.table = table, a.seq_len = seq_len, a.ref = ref;
    a.table_out = table_out, a.seq_len_out = seq_len_out, a.ref_out = ref_out;
    return accept_drafts("qsa_accept_drafts", page_size, a, d, n_rows, ld, n_pages, planes, n_groups, ws, ws_bytes, stream);
}

QSA_API qsa_status qsa_accept_drafts_weights(int32_t page_size, const int32_t *draft_off, const int32_t *parent, int32_t N,
                                             const int32_t *accepted, float *weights, int32_t *positions, int64_t tokens_ld,
                                             const int32_t *table, const int32_t *seq_len, int32_t n_rows, int64_t ld,
                                             const int32_t *ref, int64_t n_pages, int32_t *table_out, int32_t *seq_len_out,
                                             int32_t *ref_out, const qsa_page_planes *planes, int32_t n_groups, void *ws,
                                             size_t ws_bytes, qsa_stream stream) {
    const char *call = "qsa_accept_drafts_weights";
    QSA_NEED(call, n_rows <= 0 || tokens_ld == 0 || (weights && positions), "weights and positions must be non-NULL");
    AcceptArgs d{};
    d.draft_off = draft_off, d.parent = parent, d.accepted = accepted, d.N = N;
    d.positions = positions, d.positions_ld = tokens_ld, d.weights = weights;
    KeepArgs a{};
    a.table = table, a.seq_len = seq_len, a.ref = ref;
    a.table_out = table_out, a.seq_len_out = seq_len_out, a.ref_out = ref_out;
    return accept_drafts(call, page_size, a, d, n_rows, ld, n_pages, planes, n_groups, ws, ws_bytes, stream);
}

QSA_API qsa_status qsa_evict_tokens(int32_t page_size, const int32_t *budget, int32_t first, int32_t recent,
                                    const float *weights, const int32_t *positions, int64_t tokens_ld,
                                    const int32_t *table, const int32_t *seq_len, int32_t n_rows, int64_t ld,
                                    const int32_t *ref, int64_t n_pages, float *weights_out, int32_t *positions_out,
                                    int32_t *table_out, int32_t *seq_len_out, int32_t *ref_out,
                                    const qsa_page_planes *planes, int32_t n_groups, void *ws, size_t ws_bytes,
                                    qsa_stream stream) {
    const char *call = "qsa_evict_tokens";
    KeepArgs a{};
    PlaneGroups groups;
    a.table = table, a.seq_len = seq_len, a.ref = ref;
    a.table_out = table_out, a.seq_len_out = seq_len_out, a.ref_out = ref_out;
    QSA_NEED(call, first >= 0 && recent >= 0, "first %d and recent %d must not be negative", first, recent);
    QSA_NEED(call, tokens_ld >= 0 && tokens_ld <= INT32_MAX, "tokens_ld %lld out of range [0, 2^31 - 1]", (long long)tokens_ld);
    QSA_TRY(keep_args(call, page_size, n_rows, ld, n_pages, tokens_ld, planes, n_groups, ws, ws_bytes, &a, &groups));
    QSA_NEED(call, n_rows == 0 || (budget && (tokens_ld == 0 || (weights && positions && weights_out && positions_out))),
             "NULL tensor pointer");
    QSA_NEED(call, tokens_ld == 0 || n_rows == 0 || (weights != weights_out && positions != positions_out),
             "weights_out and positions_out must be other arrays than weights and positions");
    QSA_NEED(call, aligned(budget, 4) && aligned(weights, 4) && aligned(positions, 4) && aligned(weights_out, 4) &&
                 aligned(positions_out, 4),
             "the arrays must be 4-byte aligned");
    if (n_rows == 0 && n_pages == 0) return host_ok();
    QSA_TRY(check_planes_memory(call, groups));
    EvictArgs e{};
    e.budget = budget, e.first = first, e.recent = recent, e.weights = weights, e.positions = positions;
    e.weights_out = weights_out, e.positions_out = positions_out, e.tokens_ld = tokens_ld;
    return launched(launch_evict_tokens(a, e, groups, static_cast<cudaStream_t>(stream)), call);
}

QSA_API qsa_status qsa_copy_pages(const int32_t *src, const int32_t *dst, int32_t n, const qsa_page_planes *planes,
                                  int64_t n_pages, const qsa_page_planes *dst_planes, int64_t n_dst_pages,
                                  int32_t n_groups, void *ws, size_t ws_bytes, qsa_stream stream) {
    const char *call = "qsa_copy_pages";
    QSA_NEED(call, n >= 0 && n_pages >= 0 && n_dst_pages >= 0, "negative size");
    PlaneGroups groups;
    QSA_TRY(plane_groups(call, planes, dst_planes, n_groups, &groups));
    QSA_TRY(check_workspace(call, ws, ws_bytes, kWsHeaderBytes));
    if (n == 0 || n_groups == 0) return host_ok();
    QSA_NEED(call, src && dst, "NULL tensor pointer");
    QSA_NEED(call, aligned(src, 4) && aligned(dst, 4), "src and dst must be 4-byte aligned");
    QSA_TRY(check_planes_memory(call, groups));
    return launched(launch_copy_pages(src, dst, n, groups, n_pages, dst_planes ? n_dst_pages : n_pages,
                                      static_cast<WsHeader *>(ws), static_cast<cudaStream_t>(stream)), call);
}

}  // extern "C"
