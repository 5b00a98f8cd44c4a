// Native front end of the 8-bit floating point and key-value cache calls for torch
// tensors: argument checks, outputs that were not given, and the C call, in one step.
//
// A decode step's kernels take 2 to 6 us each; the same checks and allocations in
// Python took 5 to 12 us a call of the host (Neoverse V2) on top of the launch, here
// they take 0.3 to 1.5.  Nothing is computed here, and nothing is kept from one call to
// the next.  Python sees the
// functions through api.py, which documents them and turns a `stream` argument into
// the current stream (outputs are allocated, and kernels launched, there).
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "qgemv.h"

namespace {

using at::Tensor;
using c10::IntArrayRef;
using c10::ScalarType;

PyObject *qg_error = nullptr;  // _lib.QGError

// The entry points of the library that _lib has loaded (bind); this module is linked to none.
struct Library {
    decltype(&::quantize_act_e4m3) quantize_act_e4m3;
    decltype(&::rmsnorm_add_quantize_e4m3) rmsnorm_add_quantize_e4m3;
    decltype(&::qgemm_e4m3) qgemm_e4m3;
    decltype(&::qg_ffn_up_e4m3) qg_ffn_up_e4m3;
    decltype(&::qg_ffn_e4m3) qg_ffn_e4m3;
    decltype(&::qg_status_str) qg_status_str;
};
Library lib = {};

// The same for the key-value cache (bind_kv).
struct KvLibrary {
    decltype(&::qg_kv_write) qg_kv_write;
    decltype(&::qg_kv_read) qg_kv_read;
    decltype(&::qg_attn_decode) qg_attn_decode;
};
KvLibrary kv_lib = {};

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject *kind, const std::string &what)
{
    PyErr_SetString(kind, what.c_str());
    throw Refused();
}

std::string text(IntArrayRef shape)
{
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

const Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

const Tensor *optional(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

// The device the kernels are launched on: the tensor's, which has to be the current one.
int device_of(const Tensor &t, const char *name)
{
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be on a CUDA device (there is no CPU path)");
    const int dev = t.get_device(), now = c10::cuda::current_device();
    if (dev != now)
        refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(dev) +
                                     ", the current device is cuda:" + std::to_string(now));
    return dev;
}

void need(const Tensor &t, const char *name, ScalarType type, IntArrayRef shape, int dev)
{
    if (t.is_cuda() && t.scalar_type() == type && t.get_device() == dev && t.sizes() == shape && t.is_contiguous()) return;
    const std::string n = name;
    if (!t.is_cuda()) refuse(PyExc_ValueError, n + " must be on a CUDA device (there is no CPU path)");
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, n + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (!t.is_contiguous()) refuse(PyExc_ValueError, n + " must be contiguous");
    if (t.sizes() != shape) refuse(PyExc_ValueError, n + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    refuse(PyExc_ValueError, n + " must be on cuda:" + std::to_string(dev));
}

int stream_type(ScalarType t, const char *name)
{
    if (t == ScalarType::Float) return QG_F32;
    if (t == ScalarType::BFloat16) return QG_BF16;
    refuse(PyExc_TypeError, std::string(name) + " must be torch.float32 or torch.bfloat16, got " + c10::toString(t));
}

constexpr ScalarType E4M3 = ScalarType::Float8_e4m3fn;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// The output given, checked, or a new one.
Tensor output(PyObject *given, const char *name, ScalarType type, IntArrayRef shape, int dev)
{
    if (const Tensor *t = optional(given, name)) {
        need(*t, name, type, shape, dev);
        return *t;
    }
    return at::detail::empty_cuda(shape, type, c10::Device(c10::DeviceType::CUDA, static_cast<c10::DeviceIndex>(dev)),
                                  std::nullopt);
}

struct Rows {
    int64_t rows, k;
};
Rows rows_of(const Tensor &t, const char *name)
{
    if (t.dim() == 1) return {1, t.size(0)};
    if (t.dim() == 2) return {t.size(0), t.size(1)};
    refuse(PyExc_ValueError, std::string(name) + " must have shape [rows, k] or [k], got " + text(t.sizes()));
}

template <typename T>
T *at_(const Tensor &t)
{
    return static_cast<T *>(t.data_ptr());
}

qg_stream_t stream_on(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

void done(const char *fn, qg_status st)
{
    if (st == QG_OK) return;
    if (PyObject *e = PyObject_CallFunction(qg_error, "sis", fn, static_cast<int>(st), lib.qg_status_str(st))) {
        PyErr_SetObject(qg_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}

PyObject *give(const Tensor &t) { return THPVariable_Wrap(t); }

PyObject *give(PyObject *a, PyObject *b, PyObject *c = nullptr)
{
    PyObject *r = a && b ? c ? PyTuple_Pack(3, a, b, c) : PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    Py_XDECREF(c);
    return r;
}

// No C++ exception leaves the module: torch's own (a failed allocation, a CUDA error) become
// the Python exceptions that torch itself raises for them.
template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&f)
{
    if (!qg_error) {
        PyErr_SetString(PyExc_RuntimeError, "no library is bound");
        return nullptr;
    }
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &) {
        return nullptr;
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

// (x, q, d) -> (q, d)
PyObject *quantize_act(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 3, [&] {
        const Tensor &x = tensor(a[0], "x");
        const int dev = device_of(x, "x"), kind = stream_type(x.scalar_type(), "x");
        const Rows r = rows_of(x, "x");
        need(x, "x", x.scalar_type(), x.sizes(), dev);
        const Tensor q = output(a[1], "q", E4M3, {r.rows, r.k}, dev);
        const Tensor d = output(a[2], "d", ScalarType::Float, {r.rows, blocks(r.k)}, dev);
        done("quantize_act_e4m3", lib.quantize_act_e4m3(x.data_ptr(), kind, r.rows, r.k, at_<uint8_t>(q), at_<float>(d),
                                                        stream_on(dev)));
        return give(give(q), give(d));
    });
}

// (x, gamma, residual, eps, s, q, d) -> (q, d, s)
PyObject *rmsnorm_add_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        const Tensor &x = tensor(a[0], "x");
        const int dev = device_of(x, "x"), kind = stream_type(x.scalar_type(), "x");
        const Rows r = rows_of(x, "x");
        need(x, "x", x.scalar_type(), x.sizes(), dev);
        const Tensor &gamma = tensor(a[1], "gamma");
        need(gamma, "gamma", x.scalar_type(), {r.k}, dev);
        const Tensor *residual = optional(a[2], "residual");
        const double eps = PyFloat_AsDouble(a[3]);
        if (eps == -1.0 && PyErr_Occurred()) throw Refused();
        Tensor s = x;
        if (residual) {
            need(*residual, "residual", x.scalar_type(), x.sizes(), dev);
            s = output(a[4], "s", x.scalar_type(), x.sizes(), dev);
        } else if (a[4] != Py_None && a[4] != a[0]) {
            refuse(PyExc_ValueError, "s is written only with a residual");
        }
        const Tensor q = output(a[5], "q", E4M3, {r.rows, r.k}, dev);
        const Tensor d = output(a[6], "d", ScalarType::Float, {r.rows, blocks(r.k)}, dev);
        done("rmsnorm_add_quantize_e4m3",
             lib.rmsnorm_add_quantize_e4m3(x.data_ptr(), residual ? residual->data_ptr() : nullptr, gamma.data_ptr(),
                                           kind, r.rows, r.k, static_cast<float>(eps), s.data_ptr(), at_<uint8_t>(q),
                                           at_<float>(d), stream_on(dev)));
        return give(give(q), give(d), give(s));
    });
}

struct Operands {
    int64_t n_rows, k, m;
};

// A weight (`scale_rows` rows of scales) and the activations that it meets.
Operands operands(const Tensor &codes, const Tensor &scales, bool stacked, const Tensor &xq, const Tensor &xd, int dev)
{
    if (codes.dim() != 2) refuse(PyExc_ValueError, "w.codes must have shape [n_rows, k], got " + text(codes.sizes()));
    const int64_t n = codes.size(0), k = codes.size(1), kb = blocks(k);
    if (stacked && n % 32)
        refuse(PyExc_ValueError,
               "a stacked gate|up weight has 2 ffn rows, ffn a multiple of 16: got " + std::to_string(n));
    need(codes, "w.codes", E4M3, codes.sizes(), dev);
    need(scales, "w.scales", ScalarType::Float, {stacked ? 2 * blocks(n / 2) : blocks(n), kb}, dev);
    int64_t m = 1;
    if (xq.dim() == 1 && xd.dim() == 1) {
        need(xq, "xq", E4M3, {k}, dev);
        need(xd, "xd", ScalarType::Float, {kb}, dev);
    } else {
        m = xq.dim() > 0 ? xq.size(0) : 0;
        need(xq, "xq", E4M3, {m, k}, dev);
        need(xd, "xd", ScalarType::Float, {m, kb}, dev);
    }
    return {n, k, m};
}

// (codes, scales, xq, xd, epilogue, residual, y, out type: 0 f32, 1 bf16, None) -> y
PyObject *qgemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const Tensor &codes = tensor(a[0], "w.codes"), &scales = tensor(a[1], "w.scales");
        const Tensor &xq = tensor(a[2], "xq"), &xd = tensor(a[3], "xd");
        const int dev = device_of(xq, "xq");
        const Operands o = operands(codes, scales, false, xq, xd, dev);
        const long epi = PyLong_AsLong(a[4]);
        if (epi == -1 && PyErr_Occurred()) throw Refused();
        const Tensor *residual = optional(a[5], "residual"), *y_in = optional(a[6], "y");
        if (epi == QG_EPI_RESIDUAL_ADD && !residual) refuse(PyExc_ValueError, "the residual epilogue needs a residual");
        if (epi != QG_EPI_RESIDUAL_ADD && residual) refuse(PyExc_ValueError, "a residual goes with epilogue='residual'");
        ScalarType type = y_in ? y_in->scalar_type() : residual ? residual->scalar_type() : ScalarType::Float;
        if (a[7] != Py_None) type = PyLong_AsLong(a[7]) == QG_BF16 ? ScalarType::BFloat16 : ScalarType::Float;
        const int kind = stream_type(type, "y");
        const Tensor y = output(a[6], "y", type, {o.m, o.n_rows}, dev);
        if (residual) need(*residual, "residual", type, {o.m, o.n_rows}, dev);
        done("qgemm_e4m3", lib.qgemm_e4m3(at_<uint8_t>(codes), at_<float>(scales), o.n_rows, o.k, at_<uint8_t>(xq),
                                          at_<float>(xd), o.m, static_cast<int>(epi),
                                          residual ? residual->data_ptr() : nullptr, y.data_ptr(), kind,
                                          stream_on(dev)));
        return give(y);
    });
}

// (codes, scales, xq, xd, hq, hd) -> (hq, hd)
PyObject *ffn_up(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        const Tensor &codes = tensor(a[0], "w.codes"), &scales = tensor(a[1], "w.scales");
        const Tensor &xq = tensor(a[2], "xq"), &xd = tensor(a[3], "xd");
        const int dev = device_of(xq, "xq");
        const Operands o = operands(codes, scales, true, xq, xd, dev);
        const int64_t ffn = o.n_rows / 2;
        const Tensor hq = output(a[4], "hq", E4M3, {o.m, ffn}, dev);
        const Tensor hd = output(a[5], "hd", ScalarType::Float, {o.m, blocks(ffn)}, dev);
        done("qg_ffn_up_e4m3",
             lib.qg_ffn_up_e4m3(at_<uint8_t>(codes), at_<float>(scales), ffn, o.k, at_<uint8_t>(xq), at_<float>(xd), o.m,
                                at_<uint8_t>(hq), at_<float>(hd), stream_on(dev)));
        return give(give(hq), give(hd));
    });
}

// (x, residual, gamma, gate_up codes, scales, down codes, scales, eps, xq, xd, hq, hd, y) -> y
PyObject *ffn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const Tensor &x = tensor(a[0], "x");
        const int dev = device_of(x, "x"), kind = stream_type(x.scalar_type(), "x");
        const Rows r = rows_of(x, "x");
        const ScalarType type = x.scalar_type();
        need(x, "x", type, x.sizes(), dev);
        const Tensor *residual = optional(a[1], "residual");
        if (residual) need(*residual, "residual", type, x.sizes(), dev);
        const Tensor &gamma = tensor(a[2], "layer.gamma");
        const Tensor &gu = tensor(a[3], "layer.gate_up.codes"), &gud = tensor(a[4], "layer.gate_up.scales");
        const Tensor &dn = tensor(a[5], "layer.down.codes"), &dnd = tensor(a[6], "layer.down.scales");
        if (dn.dim() != 2)
            refuse(PyExc_ValueError, "layer.down.codes must have shape [hidden, ffn], got " + text(dn.sizes()));
        const int64_t f = dn.size(1), hb = blocks(r.k), fb = blocks(f);
        need(gamma, "layer.gamma", type, {r.k}, dev);
        need(gu, "layer.gate_up.codes", E4M3, {2 * f, r.k}, dev);
        need(gud, "layer.gate_up.scales", ScalarType::Float, {2 * fb, hb}, dev);
        need(dn, "layer.down.codes", E4M3, {r.k, f}, dev);
        need(dnd, "layer.down.scales", ScalarType::Float, {hb, fb}, dev);
        const double eps = PyFloat_AsDouble(a[7]);
        if (eps == -1.0 && PyErr_Occurred()) throw Refused();
        const Tensor xq = output(a[8], "buf.xq", E4M3, {r.rows, r.k}, dev);
        const Tensor xd = output(a[9], "buf.xd", ScalarType::Float, {r.rows, hb}, dev);
        const Tensor hq = output(a[10], "buf.hq", E4M3, {r.rows, f}, dev);
        const Tensor hd = output(a[11], "buf.hd", ScalarType::Float, {r.rows, fb}, dev);
        const Tensor y = output(a[12], "y", type, x.sizes(), dev);
        done("qg_ffn_e4m3",
             lib.qg_ffn_e4m3(x.data_ptr(), residual ? residual->data_ptr() : nullptr, gamma.data_ptr(), kind, r.rows,
                             r.k, f, static_cast<float>(eps), at_<uint8_t>(gu), at_<float>(gud), at_<uint8_t>(dn),
                             at_<float>(dnd), at_<uint8_t>(xq), at_<float>(xd), at_<uint8_t>(hq), at_<float>(hd),
                             y.data_ptr(), stream_on(dev)));
        return give(y);
    });
}

// ---- key-value cache --------------------------------------------------------

// The four planes of a cache (k codes, k scales, v codes, v scales), checked, as the library takes them.
qg_kv_cache cache_of(PyObject *const *a, int dev)
{
    if (!kv_lib.qg_kv_write) refuse(PyExc_RuntimeError, "no library is bound");
    const Tensor &kq = tensor(a[0], "cache.k"), &kd = tensor(a[1], "cache.k_scales");
    const Tensor &vq = tensor(a[2], "cache.v"), &vd = tensor(a[3], "cache.v_scales");
    if (kq.dim() != 4)
        refuse(PyExc_ValueError, "cache.k must have shape [n_pages, heads, page_size, head_dim], got " + text(kq.sizes()));
    const ScalarType t = kq.scalar_type();
    if (t != ScalarType::Char && t != E4M3)
        refuse(PyExc_TypeError, std::string("cache.k must be torch.int8 (Q8_0) or torch.float8_e4m3fn, got ") + c10::toString(t));
    const bool e4m3 = t == E4M3;
    const int64_t pages = kq.size(0), heads = kq.size(1), page = kq.size(2), dim = kq.size(3);
    const int64_t nb = e4m3 ? blocks(dim) : dim / 32, most = INT32_MAX;
    const ScalarType st = e4m3 ? ScalarType::Float : ScalarType::Half;
    need(kq, "cache.k", t, kq.sizes(), dev);
    need(vq, "cache.v", t, kq.sizes(), dev);
    need(kd, "cache.k_scales", st, {pages, heads, page, nb}, dev);
    need(vd, "cache.v_scales", st, {pages, heads, page, nb}, dev);
    if (heads > most || page > most || dim > most) refuse(PyExc_ValueError, "cache.k has a side beyond 2^31");
    return {kq.data_ptr(), kd.data_ptr(), vq.data_ptr(), vd.data_ptr(), pages, static_cast<int32_t>(page),
            static_cast<int32_t>(heads), static_cast<int32_t>(dim), e4m3 ? QG_KV_E4M3 : QG_KV_Q8_0};
}

// [rows, heads, dim] with contiguous rows of dim values; the strides of its other sides.
struct Strided {
    int64_t row, head;
};
Strided strided(const Tensor &t, const char *name, ScalarType type, IntArrayRef shape, int dev)
{
    const std::string n = name;
    if (!t.is_cuda()) refuse(PyExc_ValueError, n + " must be on a CUDA device (there is no CPU path)");
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, n + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape) refuse(PyExc_ValueError, n + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    if (t.get_device() != dev) refuse(PyExc_ValueError, n + " must be on cuda:" + std::to_string(dev));
    if (t.size(2) > 1 && t.stride(2) != 1) refuse(PyExc_ValueError, n + " must have contiguous rows of head_dim values");
    return {t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

// (k codes, k scales, v codes, v scales, k, v, slots) -> None
PyObject *kv_write(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&]() -> PyObject * {
        const Tensor &k = tensor(a[4], "k"), &v = tensor(a[5], "v"), &slots = tensor(a[6], "slots");
        const int dev = device_of(k, "k"), kind = stream_type(k.scalar_type(), "k");
        const qg_kv_cache c = cache_of(a, dev);
        if (k.dim() != 3) refuse(PyExc_ValueError, "k must have shape [rows, heads, head_dim], got " + text(k.sizes()));
        const int64_t rows = k.size(0), shape[] = {rows, c.heads, c.head_dim};
        const Strided ks = strided(k, "k", k.scalar_type(), shape, dev), vs = strided(v, "v", k.scalar_type(), shape, dev);
        need(slots, "slots", ScalarType::Long, {rows}, dev);
        done("qg_kv_write", kv_lib.qg_kv_write(&c, k.data_ptr(), ks.row, ks.head, v.data_ptr(), vs.row, vs.head, kind,
                                               at_<int64_t>(slots), rows, stream_on(dev)));
        Py_RETURN_NONE;
    });
}

// (k codes, k scales, v codes, v scales, slots, out type: 0 f32, 1 bf16, None, k, v) -> (k, v)
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const Tensor &slots = tensor(a[4], "slots"), *k_in = optional(a[6], "k");
        const int dev = device_of(slots, "slots");
        const qg_kv_cache c = cache_of(a, dev);
        if (slots.dim() != 1) refuse(PyExc_ValueError, "slots must have shape [rows], got " + text(slots.sizes()));
        const int64_t rows = slots.size(0), shape[] = {rows, c.heads, c.head_dim};
        need(slots, "slots", ScalarType::Long, {rows}, dev);
        ScalarType type = k_in ? k_in->scalar_type() : ScalarType::Float;
        if (a[5] != Py_None) type = PyLong_AsLong(a[5]) == QG_BF16 ? ScalarType::BFloat16 : ScalarType::Float;
        const int kind = stream_type(type, "k");
        const Tensor k = output(a[6], "k", type, shape, dev), v = output(a[7], "v", type, shape, dev);
        done("qg_kv_read", kv_lib.qg_kv_read(&c, at_<int64_t>(slots), rows, k.data_ptr(), v.data_ptr(), kind, stream_on(dev)));
        return give(give(k), give(v));
    });
}

// (k codes, k scales, v codes, v scales, q, pages, lengths, scale or None, window, out, out type: 0 f32, 1 bf16, None,
//  lse or None, work) -> out
PyObject *attn_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const Tensor &q = tensor(a[4], "q"), &pages = tensor(a[5], "pages"), &lengths = tensor(a[6], "lengths");
        const Tensor *out_in = optional(a[9], "out"), *lse = optional(a[11], "lse"), &work = tensor(a[12], "work.buf");
        const int dev = device_of(q, "q"), kind = stream_type(q.scalar_type(), "q");
        const qg_kv_cache c = cache_of(a, dev);
        if (q.dim() != 3 || q.size(2) != c.head_dim)
            refuse(PyExc_ValueError, "q must have shape [batch, q_heads, " + std::to_string(c.head_dim) + "], got " + text(q.sizes()));
        if (c.heads == 0 || q.size(1) == 0 || q.size(1) % c.heads)
            refuse(PyExc_ValueError, "q's heads must be a multiple of the cache's " + std::to_string(c.heads) + ", got " +
                                         std::to_string(q.size(1)));
        const int64_t batch = q.size(0), heads = q.size(1);
        const Strided qs = strided(q, "q", q.scalar_type(), q.sizes(), dev);
        if (pages.dim() != 2 || pages.size(0) != batch)
            refuse(PyExc_ValueError, "pages must have shape [" + std::to_string(batch) + ", max_pages], got " + text(pages.sizes()));
        need(pages, "pages", ScalarType::Int, pages.sizes(), dev);
        need(lengths, "lengths", ScalarType::Int, {batch}, dev);
        double scale = 1.0 / std::sqrt(static_cast<double>(c.head_dim));
        if (a[7] != Py_None) scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) throw Refused();
        const long long window = PyLong_AsLongLong(a[8]);
        if (window == -1 && PyErr_Occurred()) throw Refused();
        ScalarType type = out_in ? out_in->scalar_type() : q.scalar_type();
        if (a[10] != Py_None) type = PyLong_AsLong(a[10]) == QG_BF16 ? ScalarType::BFloat16 : ScalarType::Float;
        const int out_kind = stream_type(type, "out");
        const Tensor out = output(a[9], "out", type, q.sizes(), dev);
        if (lse) need(*lse, "lse", ScalarType::Float, {batch, heads}, dev);
        need(work, "work.buf", ScalarType::Byte, {work.numel()}, dev);
        done("qg_attn_decode",
             kv_lib.qg_attn_decode(&c, q.data_ptr(), qs.row, qs.head, kind, batch, heads, at_<int32_t>(pages), pages.size(1),
                                   at_<int32_t>(lengths), static_cast<float>(scale), window, out.data_ptr(), out_kind,
                                   lse ? at_<float>(*lse) : nullptr, work.data_ptr(), work.numel(), stream_on(dev)));
        return give(out);
    });
}

// The entry point whose address is a[i].
template <typename F>
bool entry(PyObject *const *a, int i, F &f)
{
    void *p = PyLong_AsVoidPtr(a[i]);
    if (!p && !PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
    f = reinterpret_cast<F>(p);
    return p != nullptr;
}

// (the error class, then the entry points' addresses in Library's order)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 7) {
        PyErr_Format(PyExc_TypeError, "expected 7 arguments, got %zd", n);
        return nullptr;
    }
    Library l;
    if (!entry(a, 1, l.quantize_act_e4m3) || !entry(a, 2, l.rmsnorm_add_quantize_e4m3) || !entry(a, 3, l.qgemm_e4m3) ||
        !entry(a, 4, l.qg_ffn_up_e4m3) || !entry(a, 5, l.qg_ffn_e4m3) || !entry(a, 6, l.qg_status_str))
        return nullptr;
    lib = l;
    Py_INCREF(a[0]);
    Py_XDECREF(qg_error);
    qg_error = a[0];
    Py_RETURN_NONE;
}

// (the error class, then the entry points' addresses in KvLibrary's order, then qg_status_str's)
PyObject *bind_kv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_Format(PyExc_TypeError, "expected 5 arguments, got %zd", n);
        return nullptr;
    }
    KvLibrary l;
    decltype(lib.qg_status_str) str;
    if (!entry(a, 1, l.qg_kv_write) || !entry(a, 2, l.qg_kv_read) || !entry(a, 3, l.qg_attn_decode) || !entry(a, 4, str))
        return nullptr;
    kv_lib = l;
    lib.qg_status_str = str;
    Py_INCREF(a[0]);
    Py_XDECREF(qg_error);
    qg_error = a[0];
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(bind)},
                         {"bind_kv", FAST(bind_kv)},
                         {"quantize_act", FAST(quantize_act)},
                         {"rmsnorm_add_quantize", FAST(rmsnorm_add_quantize)},
                         {"qgemm", FAST(qgemm)},
                         {"ffn_up", FAST(ffn_up)},
                         {"ffn", FAST(ffn)},
                         {"kv_write", FAST(kv_write)},
                         {"kv_read", FAST(kv_read)},
                         {"attn_decode", FAST(attn_decode)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qg_torch() { return PyModule_Create(&module); }
