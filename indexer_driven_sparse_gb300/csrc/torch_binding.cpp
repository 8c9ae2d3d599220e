// Python marshalling of the paged-cache calls, which run once per layer and token: every tensor is checked and its
// address taken in C++, where the same checks cost a Python binding more than the launch (a decode step's append: 12 us
// a call through ctypes, 3.5 us here). Only marshalling: each function calls the C entry point of its name
// with device pointers and returns its status; wrong tensors raise TypeError or ValueError before that.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>

#include "qsa.h"

namespace {

struct Raised : std::exception {};    // a Python error is set

[[noreturn]] void raise(PyObject *type, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw Raised();
}

using at::Tensor;

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

const Tensor &of_type(PyObject *o, const char *name, at::ScalarType type) {
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, "%s must be torch.%s, got torch.%s", name, c10::toString(type), c10::toString(t.scalar_type()));
    return t;
}

void shaped(const Tensor &t, const char *name, at::IntArrayRef want) {
    if (t.sizes() == want) return;
    std::string a, b;
    for (int64_t n : want) a += (a.empty() ? "" : ", ") + std::to_string(n);
    for (int64_t n : t.sizes()) b += (b.empty() ? "" : ", ") + std::to_string(n);
    raise(PyExc_ValueError, "%s must be [%s], got [%s]", name, a.c_str(), b.c_str());
}

// The stream of a call: the caller's, or the current one of the current device, on which every tensor must be.
struct Call {
    int device = -1;
    int current() {
        if (device < 0) device = c10::cuda::current_device();
        return device;
    }
    void on(const Tensor &t, const char *name, bool or_host = false) {
        const c10::Device d = t.device();
        if (d.is_cpu() && or_host) return;
        if (d.is_cuda() && d.index() == current()) return;
        raise(PyExc_ValueError, "%s is on %s, not on the current CUDA device", name, d.str().c_str());
    }
    void *stream(PyObject *o) {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(current())).stream();
        void *p = PyLong_AsVoidPtr(o);
        if (p == nullptr && PyErr_Occurred()) throw Raised();
        return p;
    }
    // A contiguous tensor's address.
    template <typename T = void>
    T *at(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, bool or_host = false) {
        const Tensor &t = of_type(o, name, type);
        shaped(t, name, shape);
        return address<T>(t, name, or_host);
    }
    template <typename T = void>
    T *address(const Tensor &t, const char *name, bool or_host = false) {
        if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
        on(t, name, or_host);
        return static_cast<T *>(t.data_ptr());
    }
    // bf16 [n, heads, dim] with contiguous heads: the address and the elements between rows.
    qsa_bf16 *rows(PyObject *o, const char *name, int64_t n, int64_t heads, int64_t dim, int64_t &ld) {
        const Tensor &t = of_type(o, name, at::kBFloat16);
        shaped(t, name, {n, heads, dim});
        if ((t.stride(2) != 1 && dim > 1) || (t.stride(1) != dim && heads > 1))
            raise(PyExc_ValueError, "the heads of %s must be contiguous", name);
        on(t, name);
        ld = n > 1 ? t.stride(0) : heads * dim;
        return static_cast<qsa_bf16 *>(t.data_ptr());
    }
};

template <typename T>
T config(PyObject *o, const char *name) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Raised();
    T v{};
    const bool fits = b.len == static_cast<Py_ssize_t>(sizeof(T));
    if (fits) memcpy(&v, b.buf, sizeof(T));
    PyBuffer_Release(&b);
    if (!fits) raise(PyExc_TypeError, "%s is not a %s", Py_TYPE(o)->tp_name, name);
    return v;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}

int32_t whole(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (v != static_cast<int32_t>(v)) raise(PyExc_ValueError, "%ld does not fit 32 bits", v);
    return static_cast<int32_t>(v);
}

struct Workspace {
    void *p;
    size_t bytes;
};
Workspace workspace(Call &c, PyObject *o) {
    const Tensor &t = of_type(o, "ws", at::kByte);
    return {c.address(t, "ws"), static_cast<size_t>(t.numel())};
}

const Tensor &matrix(PyObject *o, const char *name) {
    const Tensor &t = of_type(o, name, at::kInt);
    if (t.dim() != 2) raise(PyExc_ValueError, "%s must have two dimensions", name);
    return t;
}

int32_t length(const Tensor &t, const char *name) {
    if (t.dim() < 1 || t.size(0) > INT32_MAX) raise(PyExc_ValueError, "%s: %lld dimensions", name, (long long)t.dim());
    return static_cast<int32_t>(t.size(0));
}

// rope(cfg, phase, amplitude, x, pos, out, stream)
qsa_status rope(PyObject *const *a) {
    Call c;
    const auto cfg = config<qsa_rope_config>(a[0], "qsa_rope_config");
    const Tensor &x = of_type(a[3], "x", at::kBFloat16);
    if (x.dim() != 3) raise(PyExc_ValueError, "x must be [N, heads, head_dim]");
    const int64_t n = length(x, "x"), heads = x.size(1);
    if (heads > INT32_MAX) raise(PyExc_ValueError, "x has too many heads");
    int64_t x_ld, out_ld;
    const auto *xp = c.rows(a[3], "x", n, heads, cfg.head_dim, x_ld);
    auto *out = c.rows(a[5], "out", n, heads, cfg.head_dim, out_ld);
    const auto *pos = c.at<int32_t>(a[4], "pos", at::kInt, {n});
    const auto *phase = c.address<uint64_t>(of_type(a[1], "phase", at::kLong), "phase");
    return qsa_rope(&cfg, phase, static_cast<float>(number(a[2])), xp, x_ld, pos, static_cast<int32_t>(n),
                    static_cast<int32_t>(heads), out, out_ld, c.stream(a[6]));
}

struct Planes {
    qsa_bf16 *k, *v;
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int64_t n_pages;
};

// kv: (k_cache, v_cache), or (k_codes, k_scales, v_codes, v_scales)
Planes planes(Call &c, const qsa_paged_config &cfg, PyObject *kv, bool fp8) {
    Planes p{};
    PyObject *fast = PySequence_Fast(kv, "the cache must be a sequence of tensors");
    if (fast == nullptr) throw Raised();
    struct Release {
        PyObject *o;
        ~Release() { Py_DECREF(o); }
    } release{fast};
    if (PySequence_Fast_GET_SIZE(fast) != (fp8 ? 4 : 2)) raise(PyExc_ValueError, "a cache has %d tensors", fp8 ? 4 : 2);
    PyObject **o = PySequence_Fast_ITEMS(fast);
    p.n_pages = length(of_type(o[0], fp8 ? "k_codes" : "k_cache", fp8 ? at::kByte : at::kBFloat16), "the cache");
    const int64_t rows[4] = {p.n_pages, cfg.page_size, cfg.n_kv_heads, cfg.head_dim};
    const int64_t groups[4] = {p.n_pages, cfg.page_size, cfg.n_kv_heads, cfg.head_dim / 128};
    if (fp8) {
        p.k_codes = c.at<uint8_t>(o[0], "k_codes", at::kByte, rows, true);
        p.k_scales = c.at<float>(o[1], "k_scales", at::kFloat, groups, true);
        p.v_codes = c.at<uint8_t>(o[2], "v_codes", at::kByte, rows, true);
        p.v_scales = c.at<float>(o[3], "v_scales", at::kFloat, groups, true);
    } else {
        p.k = c.at<qsa_bf16>(o[0], "k_cache", at::kBFloat16, rows, true);
        p.v = c.at<qsa_bf16>(o[1], "v_cache", at::kBFloat16, rows, true);
    }
    return p;
}

// rope_append[_fp8kv](cfg, rope_cfg, phase, amplitude, q, k, v, pos, seq, q_out, kv, table, ws, stream)
template <bool F8>
qsa_status rope_append(PyObject *const *a) {
    Call c;
    const auto cfg = config<qsa_paged_config>(a[0], "qsa_paged_config");
    const auto rope = config<qsa_rope_config>(a[1], "qsa_rope_config");
    const int64_t n = length(tensor(a[5], "k"), "k");
    const int64_t D = cfg.head_dim, Hq = cfg.n_q_heads, Hkv = cfg.n_kv_heads;
    int64_t q_ld = 0, q_out_ld = 0, k_ld, v_ld;
    const qsa_bf16 *q = nullptr;
    qsa_bf16 *q_out = nullptr;
    if (a[4] != Py_None) {
        q = c.rows(a[4], "q", n, Hq, D, q_ld);
        q_out = c.rows(a[9], "q_out", n, Hq, D, q_out_ld);
    }
    const qsa_bf16 *k = c.rows(a[5], "k", n, Hkv, D, k_ld), *v = c.rows(a[6], "v", n, Hkv, D, v_ld);
    const auto *pos = c.at<int32_t>(a[7], "pos", at::kInt, {n});
    const auto *seq = a[8] == Py_None ? nullptr : c.at<int32_t>(a[8], "seq", at::kInt, {n});
    const Planes p = planes(c, cfg, a[10], F8);
    const Tensor &table = matrix(a[11], "table");
    const auto *entries = c.address<int32_t>(table, "table");
    const auto *phase = c.address<uint64_t>(of_type(a[2], "phase", at::kLong), "phase");
    const Workspace ws = workspace(c, a[12]);
    const float amplitude = static_cast<float>(number(a[3]));
    const auto N = static_cast<int32_t>(n), rows = length(table, "table");
    void *st = c.stream(a[13]);
    if (F8)
        return qsa_rope_append_fp8kv(&cfg, &rope, phase, amplitude, q, q_ld, k, k_ld, v, v_ld, seq, pos, N, q_out, q_out_ld,
                                     p.k_codes, p.k_scales, p.v_codes, p.v_scales, p.n_pages, entries, table.size(1), rows,
                                     ws.p, ws.bytes, st);
    return qsa_rope_append(&cfg, &rope, phase, amplitude, q, q_ld, k, k_ld, v, v_ld, seq, pos, N, q_out, q_out_ld, p.k, p.v,
                           p.n_pages, entries, table.size(1), rows, ws.p, ws.bytes, st);
}

// paged_decode[_fp8kv](cfg, q, kv, table, seq_len, out, lse, ws, stream)
template <bool F8>
qsa_status paged_decode(PyObject *const *a) {
    Call c;
    const auto cfg = config<qsa_paged_config>(a[0], "qsa_paged_config");
    const Tensor &table = matrix(a[3], "table");
    const int32_t B = length(table, "table");
    int64_t q_ld;
    const auto *q = c.rows(a[1], "q", B, cfg.n_q_heads, cfg.head_dim, q_ld);
    const auto *seq_len = c.at<int32_t>(a[4], "seq_len", at::kInt, {B});
    auto *out = c.at<qsa_bf16>(a[5], "out", at::kBFloat16, {B, cfg.n_q_heads, cfg.head_dim});
    auto *lse = a[6] == Py_None ? nullptr : c.at<float>(a[6], "lse", at::kFloat, {B, cfg.n_q_heads});
    const auto *entries = c.address<int32_t>(table, "table");
    const Planes p = planes(c, cfg, a[2], F8);
    const Workspace ws = workspace(c, a[7]);
    void *st = c.stream(a[8]);
    if (F8)
        return qsa_paged_decode_fp8kv(&cfg, q, q_ld, p.k_codes, p.k_scales, p.v_codes, p.v_scales, p.n_pages, entries,
                                      table.size(1), seq_len, B, out, lse, ws.p, ws.bytes, st);
    return qsa_paged_decode(&cfg, q, q_ld, p.k, p.v, p.n_pages, entries, table.size(1), seq_len, B, out, lse, ws.p, ws.bytes,
                            st);
}

// A list of pool tensors [n_planes, n_pages, ...] with contiguous planes.
struct Groups {
    qsa_page_planes g[QSA_MAX_PLANE_GROUPS];
    int32_t n;
};
Groups groups(Call &c, PyObject *list, int64_t n_pages) {
    Groups out{};
    PyObject *fast = PySequence_Fast(list, "planes must be a sequence of tensors");
    if (fast == nullptr) throw Raised();
    struct Release {
        PyObject *o;
        ~Release() { Py_DECREF(o); }
    } release{fast};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    if (n > QSA_MAX_PLANE_GROUPS) raise(PyExc_ValueError, "%zd plane groups (at most %d)", n, QSA_MAX_PLANE_GROUPS);
    out.n = static_cast<int32_t>(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Tensor &t = tensor(PySequence_Fast_GET_ITEM(fast, i), "a plane");
        if (t.dim() < 2 || t.size(1) != n_pages || t.size(0) > INT32_MAX)
            raise(PyExc_ValueError, "a plane group must be [n_planes, %lld, ...]", (long long)n_pages);
        int64_t inner = 1;
        bool whole_planes = true;
        for (int64_t d = t.dim() - 1; d >= 1; --d) {
            whole_planes = whole_planes && (t.size(d) == 1 || t.stride(d) == inner);
            inner *= t.size(d);
        }
        if (!whole_planes) raise(PyExc_ValueError, "the planes of a group must be contiguous");
        c.on(t, "a plane group", true);
        const int64_t size = static_cast<int64_t>(t.element_size());
        out.g[i].base = t.data_ptr();
        out.g[i].plane_stride = t.size(0) > 1 ? t.stride(0) * size : 0;
        out.g[i].page_bytes = n_pages > 0 ? inner / n_pages * size : 0;
        out.g[i].n_planes = static_cast<int32_t>(t.size(0));
    }
    return out;
}

// fork_pages(page_size, parent, add, table, seq_len, ref, table_out, seq_len_out, ref_out, planes, ws, stream)
qsa_status fork_pages(PyObject *const *a) {
    Call c;
    const Tensor &table = matrix(a[3], "table");
    const int32_t n_out = length(tensor(a[1], "parent"), "parent"), n_in = length(table, "table");
    const int64_t ld = table.size(1), n_pages = length(tensor(a[5], "ref"), "ref");
    const auto *parent = c.at<int32_t>(a[1], "parent", at::kInt, {n_out});
    const auto *add = c.at<int32_t>(a[2], "add", at::kInt, {n_out});
    const auto *entries = c.address<int32_t>(table, "table");
    const auto *seq_len = c.at<int32_t>(a[4], "seq_len", at::kInt, {n_in});
    const auto *ref = c.at<int32_t>(a[5], "ref", at::kInt, {n_pages});
    auto *table_out = c.at<int32_t>(a[6], "table_out", at::kInt, {n_out, ld});
    auto *len_out = c.at<int32_t>(a[7], "seq_len_out", at::kInt, {n_out});
    auto *ref_out = c.at<int32_t>(a[8], "ref_out", at::kInt, {n_pages});
    const Groups g = groups(c, a[9], n_pages);
    const Workspace ws = workspace(c, a[10]);
    return qsa_fork_pages(whole(a[0]), parent, add, n_out, entries, seq_len, n_in, ld, ref, n_pages, table_out, len_out,
                          ref_out, g.g, g.n, ws.p, ws.bytes, c.stream(a[11]));
}

// compact_pages(page_size, table, seq_len, ref, table_out, ref_out, planes, ws, stream)
qsa_status compact_pages(PyObject *const *a) {
    Call c;
    const Tensor &table = matrix(a[1], "table");
    const int32_t rows = length(table, "table");
    const int64_t ld = table.size(1), n_pages = length(tensor(a[3], "ref"), "ref");
    const auto *entries = c.address<int32_t>(table, "table");
    const auto *seq_len = c.at<int32_t>(a[2], "seq_len", at::kInt, {rows});
    const auto *ref = c.at<int32_t>(a[3], "ref", at::kInt, {n_pages});
    auto *table_out = c.at<int32_t>(a[4], "table_out", at::kInt, {rows, ld});
    auto *ref_out = c.at<int32_t>(a[5], "ref_out", at::kInt, {n_pages});
    const Groups g = groups(c, a[6], n_pages);
    const Workspace ws = workspace(c, a[7]);
    return qsa_compact_pages(whole(a[0]), entries, seq_len, rows, ld, ref, n_pages, table_out, ref_out, g.g, g.n, ws.p,
                             ws.bytes, c.stream(a[8]));
}

// copy_pages(src, dst, planes, ws, dst_planes, stream)
qsa_status copy_pages(PyObject *const *a) {
    Call c;
    const int32_t n = length(tensor(a[0], "src"), "src");
    const auto *src = c.at<int32_t>(a[0], "src", at::kInt, {n});
    const auto *dst = c.at<int32_t>(a[1], "dst", at::kInt, {n});
    auto pages_of = [](PyObject *list) -> int64_t {
        if (!PySequence_Check(list) || PySequence_Size(list) < 1) return 0;
        PyObject *first = PySequence_GetItem(list, 0);
        if (first == nullptr) throw Raised();
        const bool ok = THPVariable_Check(first) && THPVariable_Unpack(first).dim() >= 2;
        const int64_t pages = ok ? THPVariable_Unpack(first).size(1) : 0;
        Py_DECREF(first);
        return pages;
    };
    const int64_t n_pages = pages_of(a[2]), n_dst = a[4] == Py_None ? n_pages : pages_of(a[4]);
    const Groups g = groups(c, a[2], n_pages);
    Groups to{};
    if (a[4] != Py_None) {
        to = groups(c, a[4], n_dst);
        if (to.n != g.n) raise(PyExc_ValueError, "dst_planes must match planes");
    }
    const Workspace ws = workspace(c, a[3]);
    return qsa_copy_pages(src, dst, n, g.g, n_pages, a[4] == Py_None ? nullptr : to.g, n_dst, g.n, ws.p, ws.bytes,
                          c.stream(a[5]));
}

template <qsa_status (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define QSA_METHOD(name, f, n) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    QSA_METHOD("rope", rope, 7),
    QSA_METHOD("rope_append", rope_append<false>, 14),
    QSA_METHOD("rope_append_fp8kv", rope_append<true>, 14),
    QSA_METHOD("paged_decode", paged_decode<false>, 9),
    QSA_METHOD("paged_decode_fp8kv", paged_decode<true>, 9),
    QSA_METHOD("fork_pages", fork_pages, 12),
    QSA_METHOD("compact_pages", compact_pages, 9),
    QSA_METHOD("copy_pages", copy_pages, 6),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "qsa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qsa_torch() { return PyModule_Create(&module); }
