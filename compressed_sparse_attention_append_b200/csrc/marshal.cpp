// marshal.cpp -- the argument marshalling of layer.py for its plain calls, as a CPython module.
//
// A decode step makes many small calls, and checking five tensors and filling a ctypes call takes 3 to 5 us
// of host time, as long as the kernels run. Each function here makes the checks of its namesake in
// layer.py (type, device, shape, strides) on the tensors and calls the C entry point (bound by address);
// it returns the status, or None for anything it does not take: then layer.py makes the call, or names what is
// wrong with it. Nothing is kept between calls. Host time a call with its launch, here and through ctypes:
// csa2_norm_rope 3.2 and 8.1 us, csa2_fp8_quantize with csa2_fp8_gemm 6.3 and 13.0, csa2_paged_append with
// csa2_paged_gather 7.1 and 15.2.
#include <Python.h>

#include <climits>
#include <cstdint>
#include <cstring>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/csa2_layer.h"

namespace {

decltype(&csa2_rope) f_rope;
decltype(&csa2_norm_rope) f_norm_rope;
decltype(&csa2_fp8_quantize) f_quantize;
decltype(&csa2_fp8_gemm) f_gemm;
decltype(&csa2_paged_append) f_append;
decltype(&csa2_paged_gather) f_gather;
decltype(&csa2_paged_attend) f_attend;

using c10::ScalarType;

// layer.py's _rope_on
struct RopeOn {
    csa2_rope_spec spec;
    int dev;
};

// The checks of one call; the first that fails leaves `ok` false.
struct Call {
    bool ok = true;
    int dev = -1;

    const at::Tensor* tensor(PyObject* o) {
        if (!ok || !THPVariable_CheckExact(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    void need(bool x) { ok = ok && x; }
    // the device of the call: the current one, which has to be that of its first tensor
    void device(const at::Tensor* t) {
        need(t && t->is_cuda());
        if (ok) dev = c10::cuda::current_device();
    }
    bool shaped(const at::Tensor& t, std::initializer_list<int64_t> shape) {
        if (t.dim() != (int64_t)shape.size()) return false;
        int i = 0;
        for (int64_t n : shape)
            if (t.size(i++) != n) return false;
        return true;
    }
    // a tensor whose strides travel with it
    void* strided(const at::Tensor* t, ScalarType type, std::initializer_list<int64_t> shape) {
        need(t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && shaped(*t, shape));
        return ok ? t->data_ptr() : nullptr;
    }
    void* dense(PyObject* o, ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = tensor(o);
        need(t && t->is_contiguous());
        return strided(t, type, shape);
    }
    void* dense_or_none(PyObject* o, ScalarType type, std::initializer_list<int64_t> shape) {
        return o == Py_None ? nullptr : dense(o, type, shape);
    }
    // E4M3 values, also as bytes
    void* e4m3(PyObject* o, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = tensor(o);
        need(t && t->is_contiguous());
        const bool bytes = ok && t->scalar_type() == ScalarType::Byte;
        return strided(t, bytes ? ScalarType::Byte : ScalarType::Float8_e4m3fn, shape);
    }
    int64_t integer(PyObject* o, int64_t lo, int64_t hi) {
        if (!ok || !PyLong_CheckExact(o)) {
            ok = false;
            return 0;
        }
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(o, &over);
        need(!over && v >= lo && v <= hi);
        return v;
    }
    int small(PyObject* o) { return (int)integer(o, INT_MIN, INT_MAX); }
    void* address(PyObject* o) { return o == Py_None ? nullptr : reinterpret_cast<void*>(integer(o, 0, LLONG_MAX)); }
    double real(PyObject* o) {
        if (!ok || !PyFloat_CheckExact(o)) {
            ok = false;
            return 0.0;
        }
        return PyFloat_AS_DOUBLE(o);
    }
    // None, or the address of a rotation, which has to be of the call's device
    const csa2_rope_spec* rope(PyObject* o) {
        const auto* r = static_cast<const RopeOn*>(address(o));
        need(!r || (ok && r->dev == dev));
        return ok && r ? &r->spec : nullptr;
    }
    // None: the current stream; else a handle
    void* stream(PyObject* o) {
        if (o != Py_None) return address(o);
        return ok ? c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream() : nullptr;
    }
    // a cache's address, device and sequences, of which the call has `batch`
    const csa2_paged_cache* cache(PyObject* at, PyObject* on, PyObject* batch_all, PyObject* batch, int* b) {
        const int d = small(on);
        need(d >= 0);
        if (ok) dev = c10::cuda::current_device();
        need(dev == d);
        *b = small(batch);
        need(*b <= small(batch_all));
        return static_cast<const csa2_paged_cache*>(address(at));
    }
};

int type_code(ScalarType t) { return t == ScalarType::BFloat16 ? CSA2_BF16 : t == ScalarType::Float ? CSA2_F32 : -1; }

// Makes the call if the checks have passed, with the interpreter free for other threads meanwhile.
template <typename F>
PyObject* finish(const Call& c, F&& f) {
    if (!c.ok) Py_RETURN_NONE;
    long s;
    Py_BEGIN_ALLOW_THREADS;
    s = (long)f();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(s);
}

// x and out [tokens, heads, d], dense along d
void heads(Call& c, csa2_heads* h, PyObject* px, PyObject* pout, PyObject* pw, ScalarType type, int64_t tokens, int64_t d) {
    const at::Tensor *x = c.tensor(px), *out = c.tensor(pout);
    c.need(x && out && x->dim() == 3 && out->dim() == 3);
    if (!c.ok) return;
    const int64_t n = x->size(1);
    c.need(x->stride(2) == 1 && out->stride(2) == 1 && n <= INT_MAX);
    memset(h, 0, sizeof *h);
    h->x = c.strided(x, type, {tokens, n, d});
    h->out = c.strided(out, type, {tokens, n, d});
    h->x_token = x->stride(0), h->x_head = x->stride(1);
    h->out_token = out->stride(0), h->out_head = out->stride(1);
    h->weight = c.dense_or_none(pw, type, {d});
    h->heads = (int)n;
}

// (rope, pos, x, out, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) Py_RETURN_NONE;
    try {
        Call c;
        const at::Tensor* x = c.tensor(a[2]);
        c.device(x);
        c.need(c.ok && x->dim() == 3 && x->size(2) <= INT_MAX && type_code(x->scalar_type()) >= 0);
        if (!c.ok) Py_RETURN_NONE;
        const int64_t t = x->size(0), d = x->size(2);
        csa2_heads h;
        heads(c, &h, a[2], a[3], Py_None, x->scalar_type(), t, d);
        const auto* spec = c.rope(a[0]);
        const auto* pos = static_cast<const int64_t*>(c.dense_or_none(a[1], ScalarType::Long, {t}));
        const int type = type_code(x->scalar_type());
        void* s = c.stream(a[4]);
        return finish(c, [&] { return f_rope(spec, type, t, (int)d, pos, &h, s); });
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (rope, pos, eps, q, wq, q_out, k, wk, k_out, stream)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 10) Py_RETURN_NONE;
    try {
        Call c;
        const at::Tensor* q = c.tensor(a[3]);
        c.device(q);
        c.need(c.ok && q->dim() == 3 && q->size(2) <= INT_MAX && type_code(q->scalar_type()) >= 0);
        if (!c.ok) Py_RETURN_NONE;
        const int64_t t = q->size(0), d = q->size(2);
        csa2_heads hq, hk;
        heads(c, &hq, a[3], a[5], a[4], q->scalar_type(), t, d);
        const bool keys = a[6] != Py_None;
        if (keys) heads(c, &hk, a[6], a[8], a[7], q->scalar_type(), t, d);
        const auto* spec = c.rope(a[0]);
        const auto* pos = static_cast<const int64_t*>(c.dense_or_none(a[1], ScalarType::Long, {t}));
        const int type = type_code(q->scalar_type());
        const float eps = (float)c.real(a[2]);
        void* s = c.stream(a[9]);
        return finish(c, [&] { return f_norm_rope(spec, type, t, (int)d, pos, eps, &hq, keys ? &hk : nullptr, s); });
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (x, data, scale, stream)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) Py_RETURN_NONE;
    try {
        Call c;
        const at::Tensor* x = c.tensor(a[0]);
        c.device(x);
        c.need(c.ok && x->dim() == 2 && x->size(1) <= INT_MAX && (x->stride(1) == 1 || x->size(1) == 1));
        if (!c.ok) Py_RETURN_NONE;
        const int64_t rows = x->size(0), k = x->size(1);
        const auto* src = static_cast<const uint16_t*>(c.strided(x, ScalarType::BFloat16, {rows, k}));
        auto* data = static_cast<uint8_t*>(c.e4m3(a[1], {rows, k}));
        auto* scale = static_cast<float*>(c.dense(a[2], ScalarType::Float, {(k + 127) / 128, rows}));
        const int64_t stride = x->stride(0);
        void* s = c.stream(a[3]);
        return finish(c, [&] { return f_quantize(rows, (int)k, src, stride, data, scale, s); });
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (x, xs, w, ws, out, status address, status bytes, stream)
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 8) Py_RETURN_NONE;
    try {
        Call c;
        const at::Tensor *x = c.tensor(a[0]), *w = c.tensor(a[2]), *out = c.tensor(a[4]);
        c.device(x);
        c.need(c.ok && x->dim() == 2 && w->dim() == 2 && out->dim() == 2 && x->size(1) <= INT_MAX);
        if (!c.ok) Py_RETURN_NONE;
        const int64_t m = x->size(0), k = x->size(1), rows = w->size(0), nb = (k + 127) / 128;
        const int type = type_code(out->scalar_type());
        c.need(type >= 0 && (out->stride(1) == 1 || rows == 1));
        const auto* xq = static_cast<const uint8_t*>(c.e4m3(a[0], {m, k}));
        const auto* xs = static_cast<const float*>(c.dense(a[1], ScalarType::Float, {nb, m}));
        const auto* wq = static_cast<const uint8_t*>(c.e4m3(a[2], {rows, k}));
        const auto* ws = static_cast<const float*>(c.dense(a[3], ScalarType::Float, {(rows + 127) / 128, nb}));
        void* to = c.strided(out, out->scalar_type(), {m, rows});
        const int64_t stride = m > 1 ? out->stride(0) : rows;  // (a single row's means nothing; overlapping rows are refused)
        void* st = c.address(a[5]);
        const size_t bytes = (size_t)c.integer(a[6], 0, LLONG_MAX);
        void* s = c.stream(a[7]);
        return finish(c, [&] { return f_gemm(m, rows, (int)k, xq, xs, wq, ws, type, to, stride, st, bytes, s); });
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// x [batch, t, channels] bf16, dense rows, with its weight and rotation; false: there is none
bool row(Call& c, csa2_append_row* r, PyObject* px, PyObject* pw, PyObject* spec, int64_t batch, int64_t t, int64_t channels) {
    if (px == Py_None) return false;
    const at::Tensor* x = c.tensor(px);
    c.need(x && x->dim() == 3 && x->stride(2) == 1);
    if (!c.ok) return false;
    memset(r, 0, sizeof *r);
    r->x = static_cast<const uint16_t*>(c.strided(x, ScalarType::BFloat16, {batch, t, channels}));
    r->x_batch = x->stride(0), r->x_token = x->stride(1);
    r->weight = static_cast<const uint16_t*>(c.dense_or_none(pw, ScalarType::BFloat16, {channels}));
    r->rope = c.rope(spec);
    return true;
}

// (cache, its device, its sequences, batch, t, pos, length, rpos, eps, latent, weight, rope, idx_k, weight, rope,
//  swa, weight, rope, status address, status bytes, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 21) Py_RETURN_NONE;
    try {
        Call c;
        int b = 0;
        const csa2_paged_cache* cache = c.cache(a[0], a[1], a[2], a[3], &b);
        const int t = c.small(a[4]);
        const auto* pos = static_cast<const int64_t*>(c.dense_or_none(a[5], ScalarType::Long, {b}));
        const auto* length = static_cast<const int32_t*>(c.dense_or_none(a[6], ScalarType::Int, {b}));
        const auto* rpos = static_cast<const int64_t*>(c.dense_or_none(a[7], ScalarType::Long, {b, t}));
        const float eps = (float)c.real(a[8]);
        csa2_append_row r[3];
        bool on[3];
        for (int i = 0; i < 3; ++i) on[i] = row(c, &r[i], a[9 + 3 * i], a[10 + 3 * i], a[11 + 3 * i], b, t, i == 1 ? 128 : 512);
        void* st = c.address(a[18]);
        const size_t bytes = (size_t)c.integer(a[19], 0, LLONG_MAX);
        void* s = c.stream(a[20]);
        return finish(c, [&] {
            return f_append(cache, b, t, pos, length, rpos, eps, on[0] ? &r[0] : nullptr, on[1] ? &r[1] : nullptr,
                            on[2] ? &r[2] : nullptr, st, bytes, s);
        });
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (cache, its device, its sequences, batch, idx, latent, key, status address, status bytes, stream)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 10) Py_RETURN_NONE;
    try {
        Call c;
        int b = 0;
        const csa2_paged_cache* cache = c.cache(a[0], a[1], a[2], a[3], &b);
        const at::Tensor* idx = c.tensor(a[4]);
        c.need(idx && idx->dim() == 2 && idx->size(1) <= INT_MAX);
        if (!c.ok) Py_RETURN_NONE;
        const int64_t e = idx->size(1);
        const auto* at = static_cast<const int32_t*>(c.dense(a[4], ScalarType::Int, {b, e}));
        auto* latent = static_cast<uint16_t*>(c.dense_or_none(a[5], ScalarType::BFloat16, {b, e, 512}));
        auto* key = static_cast<uint16_t*>(c.dense_or_none(a[6], ScalarType::BFloat16, {b, e, 128}));
        void* st = c.address(a[7]);
        const size_t bytes = (size_t)c.integer(a[8], 0, LLONG_MAX);
        void* s = c.stream(a[9]);
        return finish(c, [&] { return f_gather(cache, b, (int)e, at, latent, key, st, bytes, s); });
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (cache, its device, its sequences, batch, tq, qpos, q, idx, k, swa_begin, win, ratio, sm_scale, out, out_f32, lse,
//  status address, status bytes, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 19) Py_RETURN_NONE;
    try {
        Call c;
        int b = 0;
        const csa2_paged_cache* cache = c.cache(a[0], a[1], a[2], a[3], &b);
        const int tq = c.small(a[4]), k = c.small(a[8]), win = c.small(a[10]), ratio = c.small(a[11]);
        const int64_t rows = (int64_t)b * tq;
        const auto* qpos = static_cast<const int64_t*>(c.dense_or_none(a[5], ScalarType::Long, {rows}));
        const auto* q = static_cast<const uint16_t*>(c.dense_or_none(a[6], ScalarType::BFloat16, {rows, 64, 512}));
        const auto* idx = static_cast<const int32_t*>(c.dense_or_none(a[7], ScalarType::Int, {rows, k}));
        const auto* begin = static_cast<const int64_t*>(c.dense_or_none(a[9], ScalarType::Long, {b}));
        const float scale = (float)c.real(a[12]);
        auto* out = static_cast<uint16_t*>(c.dense_or_none(a[13], ScalarType::BFloat16, {rows, 64, 512}));
        auto* out_f32 = static_cast<float*>(c.dense_or_none(a[14], ScalarType::Float, {rows, 64, 512}));
        auto* lse = static_cast<float*>(c.dense_or_none(a[15], ScalarType::Float, {rows, 64}));
        void* st = c.address(a[16]);
        const size_t bytes = (size_t)c.integer(a[17], 0, LLONG_MAX);
        void* s = c.stream(a[18]);
        return finish(c, [&] {
            return f_attend(cache, b, tq, qpos, q, idx, k, begin, win, ratio, scale, out, out_f32, lse, st, bytes, s);
        });
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// The entry points' addresses, in the order above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[7];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "expected seven addresses");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "expected an address");
            return nullptr;
        }
    }
    f_rope = reinterpret_cast<decltype(f_rope)>(p[0]);
    f_norm_rope = reinterpret_cast<decltype(f_norm_rope)>(p[1]);
    f_quantize = reinterpret_cast<decltype(f_quantize)>(p[2]);
    f_gemm = reinterpret_cast<decltype(f_gemm)>(p[3]);
    f_append = reinterpret_cast<decltype(f_append)>(p[4]);
    f_gather = reinterpret_cast<decltype(f_gather)>(p[5]);
    f_attend = reinterpret_cast<decltype(f_attend)>(p[6]);
    Py_RETURN_NONE;
}

#define FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(bind), FN(rope), FN(norm_rope), FN(quantize), FN(gemm), FN(append), FN(gather), FN(attend),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
