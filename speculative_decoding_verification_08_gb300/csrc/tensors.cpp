// tensors.cpp -- torch tensors to the C calls of the target pass: argument
// checks, outputs, and one call each of sv_append_kv, sv_append_kv_normed,
// sv_read_kv, sv_paged_attention, sv_paged_attention_scaled and sv_warp_sample.
//
// These calls take a few microseconds on the GPU when they are small, and
// reading some sixty tensor attributes from Python takes three times as long
// (one token appended: 18.7 us of host time from Python, of which the C call is
// 3.9).  Nothing is computed here, and there is no path without the library:
// its entry points are handed over by bind().  Each call runs with its tensors'
// device as the current one.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <c10/util/Exception.h>

#include <cmath>
#include <limits>
#include <sstream>
#include <string>
#include <tuple>

#include "specverify.h"

namespace {

decltype(&sv_append_kv) g_append = nullptr;
decltype(&sv_paged_attention) g_attend = nullptr;
decltype(&sv_warp_sample) g_warp = nullptr;
decltype(&sv_append_kv_normed) g_append_normed = nullptr;
decltype(&sv_read_kv) g_read = nullptr;
decltype(&sv_paged_attention_scaled) g_attend8 = nullptr;
decltype(&sv_paged_attention_scratch_size) g_scratch = nullptr;
PyObject *g_error = nullptr;  // the exception class
PyObject *g_check = nullptr;  // check(code, name) raises

struct Refused {
    std::string text;
};
struct Raised {};  // a Python exception is set

template <class... A>
[[noreturn]] void refuse(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    throw Refused{s.str()};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(name, " must be a torch tensor");
    return THPVariable_Unpack(o);
}

int32_t int32(int64_t x, const char *name) {
    if (x < std::numeric_limits<int32_t>::min() || x > std::numeric_limits<int32_t>::max())
        refuse(name, ": ", x, " is too large");
    return (int32_t)x;
}

int64_t integer(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    return x;
}

void *pointer(PyObject *o) {
    const unsigned long long x = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw Raised{};
    return reinterpret_cast<void *>((uintptr_t)x);
}

sv_stream_t stream(PyObject *o) { return static_cast<sv_stream_t>(pointer(o)); }

void check(int rc, const char *what) {
    if (rc == SV_OK) return;
    PyObject *r = PyObject_CallFunction(g_check, "is", rc, what);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(g_error, "%s: code %d", what, rc);
    throw Raised{};
}

// A contiguous vector of n elements on the device.
void *vector(PyObject *o, at::ScalarType type, int64_t n, int64_t dev, const char *name) {
    const at::Tensor &x = tensor(o, name);
    if (x.scalar_type() != type || x.get_device() != dev || x.numel() != n || !x.is_contiguous())
        refuse(name, ": expected ", n, " contiguous ", type, " on cuda:", dev, ", got ", x.sizes(), " ",
               x.scalar_type(), " on ", x.device());
    return x.data_ptr();
}

void *vector_or_null(PyObject *o, at::ScalarType type, int64_t n, int64_t dev, const char *name) {
    return o == Py_None ? nullptr : vector(o, type, n, dev, name);
}

// The stride of axis i; that of an axis of length one, which means nothing, as one
// that every call takes.
int64_t stride_of(const at::Tensor &x, int i) { return x.size(i) == 1 ? 0 : x.stride(i); }

int32_t code_of(at::ScalarType type) { return type == at::kBFloat16 ? SV_BF16 : SV_F16; }

struct Paged {
    sv_paged_cache c;
    sv_cache_scales s;
    at::ScalarType type;  // of the tokens
    int64_t dev;
    bool eight = false;   // a cache of 8-bit values, with scales

    Paged(PyObject *ko, PyObject *vo, PyObject *pages_o, PyObject *start_o, PyObject *len_o, int64_t N,
          at::ScalarType tokens = at::ScalarType::Undefined, PyObject *ks = Py_None, PyObject *vs = Py_None) {
        const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
        dev = k.get_device();
        type = k.scalar_type();
        if (dev < 0 || v.get_device() != dev) refuse("k_cache and v_cache must be CUDA tensors on one device");
        eight = ks != Py_None || vs != Py_None;
        if (eight) {
            if (ks == Py_None || vs == Py_None) refuse("k_scale and v_scale come together");
            if (type != at::kFloat8_e4m3fn) refuse("k_cache with scales must be torch.float8_e4m3fn, got ", type);
        } else if (type != at::kBFloat16 && type != at::kHalf) {
            refuse("k_cache must be torch.bfloat16 or torch.float16 (torch.float8_e4m3fn with k_scale and v_scale), got ",
                   type);
        }
        if (k.dim() != 4 || v.scalar_type() != type || v.sizes() != k.sizes())
            refuse("k_cache and v_cache must be [pages][page_size][kv_heads][head_dim] of one type");
        if (k.stride(3) != 1 || v.stride(3) != 1) refuse("the caches' head dimension must be contiguous");
        const at::Tensor &len = tensor(len_o, "kv_len"), &pages = tensor(pages_o, "pages");
        const int64_t B = len.numel();
        for (const auto &[o, n, name] : {std::tuple{len_o, B, "kv_len"}, std::tuple{start_o, B + 1, "q_start"}})
            if (tensor(o, name).dim() != 1) refuse(name, ": expected a vector of ", n);
        if (pages.scalar_type() != at::kInt || pages.get_device() != dev)
            refuse("pages must be torch.int32 on cuda:", dev, ", got ", pages.scalar_type(), " on ", pages.device());
        if (pages.dim() != 2 || pages.size(0) != B || (pages.size(1) > 1 && pages.stride(1) != 1))
            refuse("pages: expected [", B, "][max_pages] rows, got ", pages.sizes());
        c.k = k.data_ptr();
        c.v = v.data_ptr();
        for (int i = 0; i < 3; ++i) {
            c.k_stride[i] = stride_of(k, i);
            c.v_stride[i] = stride_of(v, i);
        }
        c.num_pages = int32(k.size(0), "pages");
        c.page_size = int32(k.size(1), "page_size");
        c.kv_heads = int32(k.size(2), "kv_heads");
        c.head_dim = int32(k.size(3), "head_dim");
        c.dtype = eight ? SV_E4M3 : code_of(type);
        if (eight) {
            s.k = scales(ks, k, s.k_stride, "k_scale");
            s.v = scales(vs, v, s.v_stride, "v_scale");
            type = tokens;
            if (type != at::kBFloat16 && type != at::kHalf)
                refuse("tokens must be torch.bfloat16 or torch.float16, got ", type);
        }
        c.B = int32(B, "sequences");
        c.tokens = int32(N, "tokens");
        c.max_pages = int32(pages.size(1), "max_pages");
        c.pages = static_cast<const int32_t *>(pages.data_ptr());
        c.pages_stride = B > 1 ? pages.stride(0) : pages.size(1);
        c.q_start = static_cast<const int32_t *>(vector(start_o, at::kInt, B + 1, dev, "q_start"));
        c.kv_len = static_cast<const int32_t *>(vector(len_o, at::kInt, B, dev, "kv_len"));
    }

    uint8_t *scales(PyObject *o, const at::Tensor &cache, int64_t *stride, const char *name) const {
        const at::Tensor &x = tensor(o, name);
        if (x.scalar_type() != at::kFloat8_e8m0fnu || x.get_device() != dev || x.dim() != 3 ||
            x.sizes() != cache.sizes().slice(0, 3))
            refuse(name, ": expected ", cache.sizes().slice(0, 3), " torch.float8_e8m0fnu on cuda:", dev, ", got ",
                   x.sizes(), " ", x.scalar_type(), " on ", x.device());
        for (int i = 0; i < 3; ++i) stride[i] = stride_of(x, i);
        return static_cast<uint8_t *>(x.data_ptr());
    }

    const sv_cache_scales *scales_or_null() const { return eight ? &s : nullptr; }
};

// A token array [N][heads][D] of the cache's type and device.
struct Heads {
    void *p = nullptr;
    int64_t st[2] = {0, 0};

    Heads() = default;
    Heads(const at::Tensor &x, const Paged &P, int64_t heads, const char *name) {
        if (x.scalar_type() != P.type || x.get_device() != P.dev)
            refuse(name, " must be ", P.type, " on cuda:", P.dev, ", got ", x.scalar_type(), " on ", x.device());
        if (x.dim() != 3 || x.size(0) != P.c.tokens || x.size(1) != heads || x.size(2) != P.c.head_dim)
            refuse(name, ": expected [", P.c.tokens, "][", heads, "][", P.c.head_dim, "], got ", x.sizes());
        if (x.stride(2) != 1 && x.size(2) > 1) refuse(name, ": the head dimension must be contiguous");
        p = x.data_ptr();
        st[0] = stride_of(x, 0);
        st[1] = stride_of(x, 1);
    }
};

int64_t rows_of(const at::Tensor &x, const char *name) {
    if (x.dim() != 3) refuse(name, ": expected [tokens][heads][head_dim], got ", x.sizes());
    return x.size(0);
}

// k, v, k_cache, v_cache, pages, q_start, kv_len, inv_freq, q, q_out,
// positions, interleaved, workspace, its bytes, stream
PyObject *append_kv(PyObject *const *a) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int64_t N = rows_of(k, "k");
    const Paged P(a[2], a[3], a[4], a[5], a[6], N);
    const c10::DeviceGuard here(tensor(a[2], "k_cache").device());
    const Heads hk(k, P, P.c.kv_heads, "k"), hv(v, P, P.c.kv_heads, "v");
    const double *freq = nullptr;
    int64_t rot = 0;
    if (a[7] != Py_None) {
        const at::Tensor &f = tensor(a[7], "inv_freq");
        if (f.dim() != 1) refuse("inv_freq must be a contiguous float64 vector on cuda:", P.dev);
        freq = static_cast<const double *>(vector(a[7], at::kDouble, f.numel(), P.dev, "inv_freq"));
        rot = 2 * f.numel();
    }
    Heads hq, ho;
    int64_t heads = 0;
    at::Tensor made;
    if (a[8] != Py_None) {
        const at::Tensor &q = tensor(a[8], "q");
        rows_of(q, "q");
        heads = q.size(1);
        hq = Heads(q, P, heads, "q");
        if (a[9] == Py_None) made = at::empty_like(q);
        ho = Heads(a[9] == Py_None ? made : tensor(a[9], "q_out"), P, heads, "q_out");
    } else if (a[9] != Py_None) {
        refuse("q_out without q");
    }
    const int32_t *positions = static_cast<const int32_t *>(vector_or_null(a[10], at::kInt, N, P.dev, "positions"));
    const int turn = PyObject_IsTrue(a[11]);
    if (turn < 0) throw Raised{};
    check(g_append(&P.c, hk.p, hk.st, hv.p, hv.st, hq.p, hq.st, ho.p, ho.st, int32(heads, "q heads"), freq,
                   int32(rot, "inv_freq"), turn, positions, pointer(a[12]), (size_t)integer(a[13]), stream(a[14])),
          "sv_append_kv");
    if (made.defined()) return THPVariable_Wrap(made);
    return Py_NewRef(a[9]);
}

// q, k_cache, v_cache, pages, q_start, kv_len, scale, window, out, workspace,
// its bytes, stream
PyObject *paged_attention(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q");
    const int64_t N = rows_of(q, "q"), heads = q.size(1);
    const Paged P(a[1], a[2], a[3], a[4], a[5], N);
    const c10::DeviceGuard here(tensor(a[1], "k_cache").device());
    const Heads hq(q, P, heads, "q");
    at::Tensor made;
    if (a[8] == Py_None) made = at::empty_like(q);
    const Heads ho(a[8] == Py_None ? made : tensor(a[8], "out"), P, heads, "out");
    double scale = 1.0 / std::sqrt((double)P.c.head_dim);
    if (a[6] != Py_None) {
        scale = PyFloat_AsDouble(a[6]);
        if (PyErr_Occurred()) throw Raised{};
    }
    check(g_attend(&P.c, hq.p, hq.st, ho.p, ho.st, int32(heads, "q heads"), (float)scale,
                   int32(integer(a[7]), "window"), pointer(a[9]), (size_t)integer(a[10]), stream(a[11])),
          "sv_paged_attention");
    if (made.defined()) return THPVariable_Wrap(made);
    return Py_NewRef(a[8]);
}

// k, v, k_cache, v_cache, pages, q_start, kv_len, inv_freq, q, q_out,
// positions, interleaved, q_norm, k_norm, eps, k_scale, v_scale, workspace, its
// bytes, stream
PyObject *append_kv_normed(PyObject *const *a) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int64_t N = rows_of(k, "k");
    const Paged P(a[2], a[3], a[4], a[5], a[6], N, k.scalar_type(), a[15], a[16]);
    const c10::DeviceGuard here(tensor(a[2], "k_cache").device());
    const Heads hk(k, P, P.c.kv_heads, "k"), hv(v, P, P.c.kv_heads, "v");
    const double *freq = nullptr;
    int64_t rot = 0;
    if (a[7] != Py_None) {
        const at::Tensor &f = tensor(a[7], "inv_freq");
        if (f.dim() != 1) refuse("inv_freq must be a contiguous float64 vector on cuda:", P.dev);
        freq = static_cast<const double *>(vector(a[7], at::kDouble, f.numel(), P.dev, "inv_freq"));
        rot = 2 * f.numel();
    }
    Heads hq, ho;
    int64_t heads = 0;
    at::Tensor made;
    if (a[8] != Py_None) {
        const at::Tensor &q = tensor(a[8], "q");
        rows_of(q, "q");
        heads = q.size(1);
        hq = Heads(q, P, heads, "q");
        if (a[9] == Py_None) made = at::empty_like(q);
        ho = Heads(a[9] == Py_None ? made : tensor(a[9], "q_out"), P, heads, "q_out");
    } else if (a[9] != Py_None) {
        refuse("q_out without q");
    } else if (a[12] != Py_None) {
        refuse("q_norm without q");
    }
    const int32_t *positions = static_cast<const int32_t *>(vector_or_null(a[10], at::kInt, N, P.dev, "positions"));
    const int turn = PyObject_IsTrue(a[11]);
    if (turn < 0) throw Raised{};
    at::ScalarType norm = at::kFloat;
    for (int i : {12, 13})
        if (a[i] != Py_None) norm = tensor(a[i], i == 12 ? "q_norm" : "k_norm").scalar_type();
    if (norm != at::kFloat && norm != P.type) refuse("norms must be torch.float32 or ", P.type, ", got ", norm);
    const void *qn = vector_or_null(a[12], norm, P.c.head_dim, P.dev, "q_norm");
    const void *kn = vector_or_null(a[13], norm, P.c.head_dim, P.dev, "k_norm");
    const double eps = PyFloat_AsDouble(a[14]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    check(g_append_normed(&P.c, P.scales_or_null(), code_of(P.type), hk.p, hk.st, hv.p, hv.st, hq.p, hq.st, ho.p,
                          ho.st, int32(heads, "q heads"), qn, kn, norm == at::kFloat ? SV_F32 : code_of(norm),
                          (float)eps, freq, int32(rot, "inv_freq"), turn, positions, pointer(a[17]),
                          (size_t)integer(a[18]), stream(a[19])),
          "sv_append_kv_normed");
    if (made.defined()) return THPVariable_Wrap(made);
    return Py_NewRef(a[9]);
}

// k_cache, v_cache, pages, q_start, kv_len, rows (-1: the outputs'), type (SV_BF16,
// SV_F16 or 0: the cache's), k_scale, v_scale, k_out, v_out, workspace, its bytes,
// stream
PyObject *read_kv(PyObject *const *a) {
    const at::Tensor &cache = tensor(a[0], "k_cache");
    int64_t N = integer(a[5]);
    for (int i : {9, 10})
        if (a[i] != Py_None) {
            const int64_t rows = rows_of(tensor(a[i], "k_out and v_out"), "k_out and v_out");
            if (N >= 0 && N != rows) refuse("expected ", N, " rows in k_out and v_out, got ", rows);
            N = rows;
        }
    if (N < 0) refuse("rows: how many there are is needed without k_out and v_out");
    const int64_t code = integer(a[6]);
    const at::ScalarType type = code == SV_BF16 ? at::kBFloat16 : code == SV_F16 ? at::kHalf : cache.scalar_type();
    const Paged P(a[0], a[1], a[2], a[3], a[4], N, type, a[7], a[8]);
    if (P.type != type) refuse("a cache of ", P.type, " is read as such, not as ", type);
    const c10::DeviceGuard here(cache.device());
    at::Tensor k, v;
    const auto options = cache.options().dtype(type);
    if (a[9] == Py_None) k = at::empty({N, P.c.kv_heads, P.c.head_dim}, options);
    if (a[10] == Py_None) v = at::empty({N, P.c.kv_heads, P.c.head_dim}, options);
    const Heads hk(k.defined() ? k : tensor(a[9], "k_out"), P, P.c.kv_heads, "k_out");
    const Heads hv(v.defined() ? v : tensor(a[10], "v_out"), P, P.c.kv_heads, "v_out");
    check(g_read(&P.c, P.scales_or_null(), code_of(type), hk.p, hk.st, hv.p, hv.st, pointer(a[11]),
                 (size_t)integer(a[12]), stream(a[13])),
          "sv_read_kv");
    PyObject *ko = k.defined() ? THPVariable_Wrap(k) : Py_NewRef(a[9]);
    PyObject *vo = v.defined() ? THPVariable_Wrap(v) : Py_NewRef(a[10]);
    PyObject *both = ko && vo ? PyTuple_Pack(2, ko, vo) : nullptr;
    Py_XDECREF(ko);
    Py_XDECREF(vo);
    return both;
}

// q, k_cache, v_cache, pages, q_start, kv_len, scale, window, out, k_scale,
// v_scale, workspace, its bytes, stream
PyObject *paged_attention_scaled(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q");
    const int64_t N = rows_of(q, "q"), heads = q.size(1);
    const Paged P(a[1], a[2], a[3], a[4], a[5], N, q.scalar_type(), a[9], a[10]);
    const c10::DeviceGuard here(tensor(a[1], "k_cache").device());
    const Heads hq(q, P, heads, "q");
    at::Tensor made, scratch;
    if (a[8] == Py_None) made = at::empty_like(q);
    const Heads ho(a[8] == Py_None ? made : tensor(a[8], "out"), P, heads, "out");
    double scale = 1.0 / std::sqrt((double)P.c.head_dim);
    if (a[6] != Py_None) {
        scale = PyFloat_AsDouble(a[6]);
        if (PyErr_Occurred()) throw Raised{};
    }
    const int32_t window = int32(integer(a[7]), "window"), q_heads = int32(heads, "q heads");
    // (from the current stream's pool, as the outputs)
    size_t bytes = g_scratch(&P.c, q_heads);
    if (bytes) {
        try {
            scratch = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
        } catch (const c10::OutOfMemoryError &) {
            bytes = 0;  // (what it is for is faster, not needed)
        }
    }
    check(g_attend8(&P.c, P.scales_or_null(), code_of(P.type), hq.p, hq.st, ho.p, ho.st, q_heads, (float)scale, window,
                    bytes ? scratch.data_ptr() : nullptr, bytes, pointer(a[11]), (size_t)integer(a[12]),
                    stream(a[13])),
          "sv_paged_attention_scaled");
    if (made.defined()) return THPVariable_Wrap(made);
    return Py_NewRef(a[8]);
}

// z, u, temperature, top_k, top_p, min_p, probs, probs_out, token_out,
// workspace, its bytes, stream
PyObject *warp_sample(PyObject *const *a) {
    const at::Tensor &given = tensor(a[0], "z");
    const int64_t dev = given.get_device();
    if (dev < 0) refuse("z must be a CUDA tensor");
    const c10::DeviceGuard here(given.device());
    const at::ScalarType type = given.scalar_type();
    if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
        refuse("z must be torch.float32, torch.bfloat16 or torch.float16, got ", type);
    if (given.dim() < 1) refuse("z: expected [..., V]");
    const int64_t V = given.size(-1);
    at::Tensor flat;
    if (given.dim() > 2) {
        try {
            flat = given.view({-1, V});
        } catch (const c10::Error &) {
            refuse("z: rows of all leading axes must be evenly strided, got ", given.sizes(), " with strides ",
                   given.strides());
        }
    }
    const at::Tensor &z = given.dim() > 2 ? flat : given;
    const int64_t R = z.dim() == 2 ? z.size(0) : 1, row = R > 1 ? z.stride(0) : V;
    if (z.stride(-1) != 1 && V > 1) refuse("z: the vocabulary dimension must be contiguous");
    const double *u = static_cast<const double *>(vector_or_null(a[1], at::kDouble, R, dev, "u"));
    const float *temperature = static_cast<const float *>(vector_or_null(a[2], at::kFloat, R, dev, "temperature"));
    const int32_t *top_k = static_cast<const int32_t *>(vector_or_null(a[3], at::kInt, R, dev, "top_k"));
    const float *top_p = static_cast<const float *>(vector_or_null(a[4], at::kFloat, R, dev, "top_p"));
    const float *min_p = static_cast<const float *>(vector_or_null(a[5], at::kFloat, R, dev, "min_p"));
    const bool draw = a[1] != Py_None;
    const int asked = PyObject_IsTrue(a[6]);
    if (asked < 0) throw Raised{};
    const bool want = asked || a[7] != Py_None;
    at::Tensor token, probs;
    int32_t *tp = nullptr;
    float *pp = nullptr;
    if (draw) {
        if (a[8] == Py_None) {
            token = at::empty(given.sizes().slice(0, given.dim() - 1), given.options().dtype(at::kInt));
            tp = static_cast<int32_t *>(token.data_ptr());
        } else {
            tp = static_cast<int32_t *>(vector(a[8], at::kInt, R, dev, "token_out"));
        }
    } else if (a[8] != Py_None) {
        refuse("token_out without u");
    }
    if (want) {
        if (a[7] == Py_None) {
            probs = at::empty(given.sizes(), given.options().dtype(at::kFloat));
            pp = static_cast<float *>(probs.data_ptr());
        } else {
            const at::Tensor &x = tensor(a[7], "probs_out");
            if (x.scalar_type() != at::kFloat || x.get_device() != dev || x.sizes() != given.sizes() ||
                !x.is_contiguous())
                refuse("probs_out: expected ", given.sizes(), " contiguous float32 on cuda:", dev);
            pp = static_cast<float *>(x.data_ptr());
            // (a row's draw reads its logits after its probabilities are written)
            const char *z0 = static_cast<const char *>(z.data_ptr()), *p0 = reinterpret_cast<const char *>(pp);
            if (R > 0 && p0 < z0 + ((R - 1) * row + V) * (int64_t)z.element_size() && z0 < p0 + 4 * R * V)
                refuse("probs_out must not overlap z");
        }
    }
    if (!draw && !want && R > 0) refuse("nothing to compute: give u, or ask for probs");
    check(g_warp(z.data_ptr(), row, type == at::kFloat ? SV_F32 : type == at::kBFloat16 ? SV_BF16 : SV_F16,
                 int32(R, "rows"), V, temperature, top_k, top_p, min_p, u, tp, pp, V, pointer(a[9]),
                 (size_t)integer(a[10]), stream(a[11])),
          "sv_warp_sample");
    PyObject *t = token.defined() ? THPVariable_Wrap(token) : Py_NewRef(a[8]);
    PyObject *p = probs.defined() ? THPVariable_Wrap(probs) : Py_NewRef(a[7]);
    PyObject *both = t && p ? PyTuple_Pack(2, t, p) : nullptr;
    Py_XDECREF(t);
    Py_XDECREF(p);
    return both;
}

// No C++ exception leaves a call.
template <PyObject *(*F)(PyObject *const *), int kArgs>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        if (n != kArgs) refuse("expected ", kArgs, " arguments, got ", n);
        if (!g_warp || !g_attend8) refuse("the library is not loaded");
        return F(a);
    } catch (const Refused &e) {
        PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.text.c_str());
        return nullptr;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <int kCount>
bool addresses(PyObject *const *a, void *(&f)[kCount]) {
    for (int i = 0; i < kCount; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return false;
    }
    return true;
}

// bind(sv_append_kv, sv_paged_attention, sv_warp_sample, error class, check)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes three addresses, an exception class and a function");
        return nullptr;
    }
    void *f[3];
    if (!addresses(a, f)) return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(f[0]);
    g_attend = reinterpret_cast<decltype(g_attend)>(f[1]);
    g_warp = reinterpret_cast<decltype(g_warp)>(f[2]);
    Py_XSETREF(g_error, Py_NewRef(a[3]));
    Py_XSETREF(g_check, Py_NewRef(a[4]));
    Py_RETURN_NONE;
}

// bind8(sv_append_kv_normed, sv_read_kv, sv_paged_attention_scaled,
// sv_paged_attention_scratch_size)
PyObject *bind8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind8 takes four addresses");
        return nullptr;
    }
    void *f[4];
    if (!addresses(a, f)) return nullptr;
    g_append_normed = reinterpret_cast<decltype(g_append_normed)>(f[0]);
    g_read = reinterpret_cast<decltype(g_read)>(f[1]);
    g_attend8 = reinterpret_cast<decltype(g_attend8)>(f[2]);
    g_scratch = reinterpret_cast<decltype(g_scratch)>(f[3]);
    Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"bind8", fast(bind8), METH_FASTCALL, nullptr},
                         {"append_kv", fast(entry<append_kv, 15>), METH_FASTCALL, nullptr},
                         {"append_kv_normed", fast(entry<append_kv_normed, 20>), METH_FASTCALL, nullptr},
                         {"read_kv", fast(entry<read_kv, 14>), METH_FASTCALL, nullptr},
                         {"paged_attention", fast(entry<paged_attention, 12>), METH_FASTCALL, nullptr},
                         {"paged_attention_scaled", fast(entry<paged_attention_scaled, 14>), METH_FASTCALL, nullptr},
                         {"warp_sample", fast(entry<warp_sample, 12>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
