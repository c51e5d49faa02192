// Argument checks of the calls that a step makes in every layer (mla_rope,
// mla_cache_append, mla_decode_fp8_page), for the Python binding. The kernels behind
// them take two to five microseconds, and asking ten tensors for their types,
// sizes, strides and addresses through Python takes three times that, so it is
// done here: a call in 17 us became one in 5.
//
// Each function takes the library's entry point (its address, or a callable that
// gets the arguments instead), the stream (None: PyTorch's current one), a device
// that stands in for the current one (None as a rule) and the call's arguments. It
// returns the library's status, a text where an argument is refused, or None where
// one is not a tensor of the current device (the binding then says which).
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>
#include <tuple>
#include <utility>

#include "mla.h"

namespace {

using at::Tensor;

struct Refused {
    std::string why;
};
struct NotThere {};
struct Raised {};  // a Python error is set

void need(bool ok, const char* why) {
    if (!ok) throw Refused{why};
}

int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
int small(PyObject* o, const char* what) {
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(what) + " " + std::to_string(v)};
    return static_cast<int>(v);
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}

// Where a call runs: the current device, if `first` is on one.
struct Place {
    int64_t dev;
    void* stream;
};
Place place(PyObject* stream, PyObject* dev, PyObject* first) {
    Place p{};
    if (dev != Py_None) {
        p.dev = whole(dev);
    } else {
        if (!THPVariable_Check(first) || !THPVariable_Unpack(first).is_cuda()) throw NotThere{};
        p.dev = c10::cuda::current_device();
    }
    if (stream == Py_None) {
        if (dev == Py_None) p.stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(p.dev)).stream();
    } else if (PyLong_Check(stream)) {
        p.stream = PyLong_AsVoidPtr(stream);
    } else {
        PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) throw Raised{};
        p.stream = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
    }
    if (PyErr_Occurred()) throw Raised{};
    return p;
}

const Tensor& tensor(PyObject* o, int64_t dev) {
    if (!THPVariable_Check(o)) throw NotThere{};
    const Tensor& t = THPVariable_Unpack(o);
    if (t.get_device() != dev || t.layout() != at::kStrided) throw NotThere{};
    return t;
}
const Tensor* maybe(PyObject* o, int64_t dev) { return o == Py_None ? nullptr : &tensor(o, dev); }

bool plain(const Tensor& t, at::ScalarType type) { return t.scalar_type() == type && t.is_contiguous(); }
template <class T>
const T* in(const Tensor& t) {
    return static_cast<const T*>(t.const_data_ptr());
}
template <class T>
const T* in(const Tensor* t) {
    return t ? in<T>(*t) : nullptr;
}
void* out(const Tensor& t) { return t.mutable_data_ptr(); }
void* out(const Tensor* t) { return t ? out(*t) : nullptr; }

std::string num(int64_t v) { return std::to_string(v); }

int32_t* status_word(const Tensor* t) {
    if (!t) return nullptr;
    need(t->scalar_type() == at::kInt && t->numel() >= 1, "status must be an int32 tensor");
    return static_cast<int32_t*>(out(*t));
}

struct Table {
    const int32_t* at;
    int64_t stride, cols;
};
Table table_of(const Tensor& t, int64_t B) {
    need(t.scalar_type() == at::kInt && t.dim() == 2 && t.stride(1) == 1,
         "block_table must be a 2-D int32 tensor with contiguous rows");
    const int64_t rows = t.size(0), cols = t.size(1);
    if (rows < B) throw Refused{"block_table has " + num(rows) + " rows for " + num(B) + " requests"};
    const int64_t stride = rows > 1 ? t.stride(0) : cols;  // (one row: its stride says nothing)
    need(stride >= cols, "block_table's rows overlap");
    return {in<int32_t>(t), stride, cols};
}

PyObject* py(int64_t v) { return PyLong_FromLongLong(v); }
PyObject* py(int v) { return PyLong_FromLong(v); }
PyObject* py(size_t v) { return PyLong_FromSize_t(v); }
PyObject* py(float v) { return PyFloat_FromDouble(v); }
PyObject* py(const void* v) {
    if (v) return PyLong_FromVoidPtr(const_cast<void*>(v));
    Py_RETURN_NONE;
}

// The entry point `call` with these arguments.
template <class... A, class... B>
PyObject* enter(PyObject* call, int (*)(A...), B... b) {
    static_assert(sizeof...(A) == sizeof...(B), "arguments");
    if (PyLong_Check(call)) {
        auto fn = reinterpret_cast<int (*)(A...)>(PyLong_AsVoidPtr(call));
        if (!fn) throw Raised{};
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = fn(static_cast<A>(b)...);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(st);
    }
    PyObject* args = PyTuple_New(sizeof...(B));
    if (!args) throw Raised{};
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(args, i++, py(static_cast<A>(b))), ...);
    PyObject* r = PyObject_CallObject(call, args);
    Py_DECREF(args);
    if (!r) throw Raised{};
    return r;
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused& e) {
        return PyUnicode_FromString(e.why.c_str());
    } catch (const NotThere&) {
        Py_RETURN_NONE;
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// entry, stream, device, x, positions, steps, out, interleaved, mscale
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const Place at = place(a[1], a[2], a[3]);
        const int64_t dev = at.dev;
        const Tensor &x = tensor(a[3], dev), &pos = tensor(a[4], dev), &steps = tensor(a[5], dev), &y = tensor(a[6], dev);
        need(x.dim() == 3, "x must be [T, H, R]");
        const int64_t T = x.size(0), H = x.size(1), R = x.size(2);
        const bool f32 = x.scalar_type() == at::kFloat;
        need(f32 || x.scalar_type() == at::kBFloat16, "x must be bf16 or fp32");
        need(y.sizes() == x.sizes() && y.scalar_type() == x.scalar_type(), "out must be a tensor of x's shape and type");
        if (R < 2 || R % 2) throw Refused{num(R) + " values a head: an even number is rotated"};
        need(x.stride(2) == 1 && y.stride(2) == 1, "x and out must have contiguous last dimensions");
        if (!plain(pos, at::kInt) || pos.dim() != 1 || pos.size(0) != T)
            throw Refused{"positions must be contiguous int32 [" + num(T) + "]"};
        if (!plain(steps, at::kLong) || steps.dim() != 1 || steps.size(0) != R / 2)
            throw Refused{"steps must be contiguous int64 [" + num(R / 2) + "]"};
        need(H <= INT32_MAX && R <= INT32_MAX, "x must be [T, H, R]");
        return enter(a[0], &mla_rope, x.const_data_ptr(), x.stride(0), x.stride(1), in<int32_t>(pos), in<int64_t>(steps), T,
                     static_cast<int>(H), static_cast<int>(R), f32 ? 1 : 0, small(a[7], "interleaved") ? 1 : 0, real(a[8]), out(y),
                     y.stride(0), y.stride(1), at.stream);
    });
}

// entry, stream, device, latent, k_pe, cu_new_lens, seq_lens, block_table, page_size, cache,
// cache_kind, steps, positions, interleaved, mscale, norm_weight, eps, scales, rows, lat_dim, status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 21, [&] {
        const Place at = place(a[1], a[2], a[3]);
        const int64_t dev = at.dev;
        const Tensor &lat = tensor(a[3], dev), &pe = tensor(a[4], dev), &cu = tensor(a[5], dev), &sl = tensor(a[6], dev),
                     &bt = tensor(a[7], dev), &cache = tensor(a[9], dev);
        const Tensor *steps = maybe(a[11], dev), *pos = maybe(a[12], dev), *norm = maybe(a[15], dev), *scales = maybe(a[17], dev),
                     *rows = maybe(a[18], dev), *status = maybe(a[20], dev);
        const int page = small(a[8], "page_size"), kind = small(a[10], "cache kind"), D = small(a[19], "lat_dim");
        int64_t rb = 0;
        if (kind == MLA_CACHE_BF16_576) {
            if (D <= 0) throw Refused{"lat_dim " + num(D)};
            rb = 2 * (static_cast<int64_t>(D) + 64);
        } else if (kind == MLA_CACHE_FP8_DS_MLA_656 || kind == MLA_CACHE_FP8_PAGE_576) {
            need(D == 512, "rows of this cache kind have lat_dim 512");
            rb = kind == MLA_CACHE_FP8_PAGE_576 ? 576 : 656;
        } else {
            throw Refused{"unknown cache kind " + num(kind)};
        }
        if (lat.scalar_type() != at::kBFloat16 || lat.dim() != 2 || lat.size(1) != D || lat.stride(1) != 1)
            throw Refused{"latent must be bf16 [total, " + num(D) + "] with contiguous rows"};
        const int64_t total = lat.size(0);
        if (pe.scalar_type() != at::kBFloat16 || pe.dim() != 2 || pe.size(0) != total || pe.size(1) != 64 || pe.stride(1) != 1)
            throw Refused{"k_pe must be bf16 [" + num(total) + ", 64] with contiguous rows"};
        if (page < 1) throw Refused{"page_size " + num(page)};
        need(cache.is_contiguous(), "cache must be contiguous");
        need(plain(sl, at::kInt), "seq_lens must be contiguous int32");
        const int64_t B = sl.numel();
        need(B <= INT32_MAX, "seq_lens must be contiguous int32");
        if (!plain(cu, at::kInt) || cu.numel() != B + 1)
            throw Refused{"cu_new_lens must be contiguous int32 with " + num(B + 1) + " entries"};
        const Table tb = table_of(bt, B);
        if (steps) need(plain(*steps, at::kLong) && steps->dim() == 1 && steps->size(0) == 32, "steps must be contiguous int64 [32]");
        if (pos && (!plain(*pos, at::kInt) || pos->dim() != 1 || pos->size(0) != total))
            throw Refused{"positions must be contiguous int32 [" + num(total) + "]"};
        if (norm && (!plain(*norm, at::kBFloat16) || norm->dim() != 1 || norm->size(0) != D))
            throw Refused{"norm_weight must be contiguous bf16 [" + num(D) + "]"};
        const int64_t slots = static_cast<int64_t>(cache.nbytes()) / rb;
        if (kind == MLA_CACHE_FP8_PAGE_576) {
            if (!scales || !plain(*scales, at::kFloat) || scales->numel() < slots / page)
                throw Refused{"scales must be contiguous fp32 of at least " + num(slots / page) + " values"};
        } else {
            need(!scales, "scales belong to rows of MLA_CACHE_FP8_PAGE_576 alone");
        }
        if (rows && (rows->scalar_type() != at::kBFloat16 || rows->dim() != 2 || rows->size(0) < total ||
                     rows->size(1) < D + 64 || rows->stride(1) != 1))
            throw Refused{"rows must be bf16 [>= " + num(total) + ", >= " + num(D + 64) + "] with contiguous rows"};
        int32_t* st = status_word(status);
        const bool one = total <= 1;  // (the stride of a dimension of one entry says nothing)
        return enter(a[0], &mla_cache_append, lat.const_data_ptr(), one ? D : lat.stride(0), pe.const_data_ptr(),
                     one ? 64 : pe.stride(0), in<int32_t>(cu), in<int32_t>(sl), tb.at, tb.stride, tb.cols, static_cast<int>(B),
                     total, page, in<int32_t>(pos), in<int64_t>(steps), small(a[13], "interleaved") ? 1 : 0, real(a[14]),
                     norm ? norm->const_data_ptr() : nullptr, real(a[16]), out(cache), kind, D, slots,
                     static_cast<float*>(out(scales)), out(rows), rows ? (one ? D + 64 : rows->stride(0)) : 0, st,
                     at.stream);
    });
}

// entry, stream, device, q_lat, q_pe, cache, scales, page_size, block_table, seq_lens, q_len, scale, out, lse,
// workspace, cu_q_lens, num_ctas
PyObject* decode_page(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&] {
        const Place at = place(a[1], a[2], a[3]);
        const int64_t dev = at.dev;
        const Tensor &ql = tensor(a[3], dev), &qp = tensor(a[4], dev), &cache = tensor(a[5], dev), &scales = tensor(a[6], dev),
                     &bt = tensor(a[8], dev), &sl = tensor(a[9], dev), &o = tensor(a[12], dev), &lse = tensor(a[13], dev),
                     &ws = tensor(a[14], dev);
        const Tensor* cu = maybe(a[15], dev);
        const int page = small(a[7], "page_size"), q_len = small(a[10], "q_len"), ctas = small(a[16], "num_ctas");
        need(ql.dim() == 3 && ql.size(2) == 512 && qp.dim() == 3 && qp.size(0) == ql.size(0) && qp.size(1) == ql.size(1) &&
                 qp.size(2) == 64,
             "q_lat must be [tokens, Hq, 512] and q_pe [tokens, Hq, 64]");
        const int64_t tokens = ql.size(0), Hq = ql.size(1), B = sl.numel();
        need(plain(ql, at::kBFloat16) && plain(qp, at::kBFloat16), "q_lat and q_pe must be contiguous bf16");
        need(plain(sl, at::kInt) && B <= INT32_MAX, "seq_lens must be contiguous int32");
        if (!cu) {
            if (tokens != B * q_len)
                throw Refused{"q_lat holds " + num(tokens) + " tokens, " + num(B) + " requests of " + num(q_len) + " expected"};
        } else if (!plain(*cu, at::kInt) || cu->numel() != B + 1) {
            throw Refused{"cu_q_lens must be contiguous int32 with " + num(B + 1) + " entries"};
        }
        const bool f32 = o.scalar_type() == at::kFloat;
        if ((!f32 && o.scalar_type() != at::kBFloat16) || o.sizes() != ql.sizes() || !o.is_contiguous())
            throw Refused{"out must be a contiguous bf16 or fp32 [" + num(tokens) + ", " + num(Hq) + ", 512] tensor"};
        if (!plain(lse, at::kFloat) || lse.dim() != 2 || lse.size(0) != tokens || lse.size(1) != Hq)
            throw Refused{"lse must be a contiguous fp32 [" + num(tokens) + ", " + num(Hq) + "] tensor"};
        need(cache.is_contiguous() && ws.is_contiguous(), "cache and workspace must be contiguous");
        if (page < 1) throw Refused{"page_size " + num(page)};
        const int64_t slots = static_cast<int64_t>(cache.nbytes()) / 576;
        if (!plain(scales, at::kFloat) || scales.numel() < slots / page)
            throw Refused{"scales must be contiguous fp32 of at least " + num(slots / page) + " values"};
        const Table tb = table_of(bt, B);
        need(Hq <= INT32_MAX, "q_lat must be [tokens, Hq, 512]");
        return enter(a[0], &mla_decode_fp8_page, ql.const_data_ptr(), qp.const_data_ptr(), tokens, cache.const_data_ptr(),
                     in<float>(scales), slots, page, tb.at, tb.stride, tb.cols, in<int32_t>(sl), in<int32_t>(cu),
                     static_cast<int>(B), q_len, static_cast<int>(Hq), real(a[11]), out(o),
                     static_cast<int>(f32 ? MLA_OUT_F32 : MLA_OUT_BF16), static_cast<float*>(out(lse)), out(ws), ws.nbytes(), ctas,
                     at.stream);
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"rope", fast<rope>(), METH_FASTCALL, "checks and calls mla_rope"},
                         {"append", fast<append>(), METH_FASTCALL, "checks and calls mla_cache_append"},
                         {"decode_page", fast<decode_page>(), METH_FASTCALL, "checks and calls mla_decode_fp8_page"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_bind", "Argument checks of the binding.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_bind(void) { return PyModule_Create(&module); }
