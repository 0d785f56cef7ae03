// Host path of the FP8 and pooled calls for Python: checks a call's tensors and hands their pointers to the C entry
// points (include/gdn.h) on the current stream. A decode step makes these calls once per layer, and checking a dozen
// tensors and marshalling thirty arguments from Python takes two to three times as long as their kernels do.
//
// Every function either does the whole call and returns its result, or returns None having done nothing: an argument
// that is not plainly right (type, dtype, device, layout, size), another device than the current one, a status
// other than GDN_OK. The Python binding then goes its own way, which names what is wrong. So all that can fail (outputs,
// their views, the objects of the result) is made before the entry point is called, and nothing after: a call that the
// binding makes again would advance states in place twice. No exception leaves a function, no tensor is kept.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdn.h"

namespace {

// The entry points of the library that the Python binding has loaded.
struct Entries {
    decltype(&fp8_gemm) gemm;
    decltype(&fp8_quantize_act) quantize_act;
    decltype(&fp8_quantize_weight) quantize_weight;
    decltype(&gdn_gated_rmsnorm_silu_fp8) tail;
    decltype(&gdn_decode_step_pooled) decode;
    decltype(&gdn_decode_step_pooled_gated_fp8) decode_fp8;
    decltype(&gdn_short_conv1d_silu_decode_pooled) conv;
} lib = {};

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kF8 = at::kFloat8_e4m3fn;

struct No {};   // the call is not for this path

const at::Tensor &tensor(PyObject *o) {
    if (!THPVariable_Check(o)) throw No{};
    return THPVariable_Unpack(o);
}
void need(bool ok) {
    if (!ok) throw No{};
}
// A tensor of dtype `t` on CUDA device `dev`.
const at::Tensor &on(const at::Tensor &x, int dev, at::ScalarType t) {
    need(x.is_cuda() && x.get_device() == dev && x.scalar_type() == t && x.layout() == at::kStrided);
    return x;
}
// ... contiguous and with at least n elements.
const at::Tensor &whole(const at::Tensor &x, int dev, at::ScalarType t, int64_t n) {
    on(x, dev, t);
    need(x.is_contiguous() && x.numel() >= n);
    return x;
}
int current_device_of(const at::Tensor &x) {
    need(x.is_cuda());
    const int dev = x.get_device();
    need(dev == c10::cuda::current_device());
    return dev;
}
gdn_dtype io_type(const at::Tensor &x) {
    need(x.scalar_type() == kBf16 || x.scalar_type() == kF32);
    return x.scalar_type() == kBf16 ? GDN_BF16 : GDN_F32;
}
int32_t i32(int64_t v) {
    need(v >= 0 && v <= INT32_MAX);
    return (int32_t)v;
}
gdn_stream_t stream() { return reinterpret_cast<gdn_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }
template <typename T>
T *ptr(const at::Tensor &x) {
    return reinterpret_cast<T *>(x.data_ptr());
}
// An output: the given tensor, or a new one.
at::Tensor out(PyObject *o, int dev, at::ScalarType t, at::IntArrayRef shape, bool zero = false) {
    int64_t n = 1;
    for (int64_t d : shape) n *= d;
    if (o != Py_None) return whole(tensor(o), dev, t, n);
    const auto opt = at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)dev);
    return zero ? at::zeros(shape, opt) : at::empty(shape, opt);
}
// Row stride of a 2-D tensor with unit column stride.
int64_t row_stride(const at::Tensor &x) {
    need(x.dim() == 2 && (x.size(1) <= 1 || x.stride(1) == 1));
    return x.size(0) > 1 ? x.stride(0) : std::max<int64_t>(x.size(1), 1);
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw No{};
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    need(v >= 0);
    return v != 0;
}
// A new reference (the call is not for this path where there is none), given up with the call that fails.
class Ref {
    PyObject *p_;

public:
    explicit Ref(PyObject *p) : p_(p) { need(p != nullptr); }
    Ref(Ref &&r) noexcept : p_(r.p_) { r.p_ = nullptr; }
    Ref(const Ref &) = delete;
    ~Ref() { Py_XDECREF(p_); }
    PyObject *get() const { return p_; }
    PyObject *release() {
        PyObject *p = p_;
        p_ = nullptr;
        return p;
    }
};
// The result of a call whose entry point answered `s`.
PyObject *done(gdn_status s, Ref &&result) {
    need(s == GDN_OK);
    return result.release();
}
Ref give(PyObject *given, const at::Tensor &x) {
    if (given == Py_None) return Ref(THPVariable_Wrap(x));
    Py_INCREF(given);
    return Ref(given);
}
Ref pair(const Ref &a, const Ref &b) { return Ref(PyTuple_Pack(2, a.get(), b.get())); }

template <typename F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (...) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// fp8_gemm(aq, as, bq, bs, y or None, new y in fp32)
PyObject *py_gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 6 && lib.gemm);
        const at::Tensor &aq = tensor(a[0]), &bq = tensor(a[2]);
        const int dev = current_device_of(aq);
        need(aq.dim() == 2 && bq.dim() == 2 && bq.size(1) == aq.size(1));
        const int32_t M = i32(aq.size(0)), N = i32(bq.size(0)), K = i32(aq.size(1));
        const int64_t kb = ((int64_t)K + 127) / 128;
        whole(aq, dev, kF8, 0);
        whole(bq, dev, kF8, 0);
        const at::Tensor &as = whole(tensor(a[1]), dev, kF32, M * kb);
        const at::Tensor &bs = whole(tensor(a[3]), dev, kF32, ((int64_t)N + 127) / 128 * kb);
        at::ScalarType t = truth(a[5]) ? kF32 : kBf16;
        if (a[4] != Py_None) {
            t = tensor(a[4]).scalar_type();
            need(t == kBf16 || t == kF32);
        }
        const at::Tensor y = out(a[4], dev, t, {M, N});
        Ref r = give(a[4], y);
        return done(lib.gemm(ptr<uint8_t>(aq), ptr<float>(as), ptr<uint8_t>(bq), ptr<float>(bs), M, N, K,
                             t == kBf16 ? GDN_BF16 : GDN_F32, y.data_ptr(), stream()), std::move(r));
    });
}

// fp8_quantize(x, xq or None, xs or None, weight)
PyObject *py_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 4 && lib.quantize_act);
        const at::Tensor &x = tensor(a[0]);
        const int dev = current_device_of(x);
        const gdn_dtype t = io_type(x);
        const int64_t ldx = row_stride(x);
        const int32_t M = i32(x.size(0)), K = i32(x.size(1));
        const bool weight = truth(a[3]);
        const int64_t kb = ((int64_t)K + 127) / 128, rows = weight ? ((int64_t)M + 127) / 128 : M;
        const at::Tensor xq = out(a[1], dev, kF8, {M, K}), xs = out(a[2], dev, kF32, {rows, kb});
        Ref r = pair(give(a[1], xq), give(a[2], xs));
        return done((weight ? lib.quantize_weight : lib.quantize_act)(x.data_ptr(), ldx, t, M, K, ptr<uint8_t>(xq), ptr<float>(xs),
                                                                      stream()), std::move(r));
    });
}

// gdn_gated_rmsnorm_silu_fp8(o, z, weight, eps, xq or None, xs or None)
PyObject *py_tail(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 6 && lib.tail);
        const at::Tensor &o = tensor(a[0]);
        const int dev = current_device_of(o);
        const gdn_dtype t = io_type(o);
        need(o.dim() == 3);
        const int32_t M = i32(o.size(0)), Hv = i32(o.size(1)), D = i32(o.size(2));
        const int64_t K = (int64_t)Hv * D, kb = (K + 127) / 128;
        whole(o, dev, o.scalar_type(), 0);
        const at::Tensor &z = whole(tensor(a[1]), dev, o.scalar_type(), M * K), &w = whole(tensor(a[2]), dev, kF32, D);
        const double eps = number(a[3]);
        const at::Tensor xq = out(a[4], dev, kF8, {M, K}), xs = out(a[5], dev, kF32, {M, kb});
        Ref r = pair(give(a[4], xq), give(a[5], xs));
        return done(lib.tail(o.data_ptr(), z.data_ptr(), ptr<float>(w), (float)eps, M, Hv, D, t, ptr<uint8_t>(xq), ptr<float>(xs),
                             stream()), std::move(r));
    });
}

// gdn_decode_step_pooled(q, k, v, a, b, A_log, dt_bias, state_pool, slots, scale, qk_l2norm, o or None, new o in fp32), or
// ..._gated_fp8(q, k, v, a, b, A_log, dt_bias, state_pool, slots, scale, qk_l2norm, o or None, z, norm_weight, eps, xq or None,
// xs or None)
PyObject *py_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need((n == 13 || n == 17) && lib.decode);
        const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &ga = tensor(a[3]), &gb = tensor(a[4]);
        const at::Tensor &pool = tensor(a[7]);
        const int dev = current_device_of(q);
        need(q.dim() == 3 && k.sizes() == q.sizes() && v.dim() == 3 && v.size(0) == q.size(0) && v.size(2) == q.size(2));
        const int32_t B = i32(q.size(0)), Hk = i32(q.size(1)), D = i32(q.size(2)), Hv = i32(v.size(1));
        need(pool.dim() == 4 && pool.size(1) == Hv && pool.size(2) == D && pool.size(3) == D);
        whole(q, dev, kBf16, 0);
        whole(k, dev, kBf16, 0);
        whole(v, dev, kBf16, 0);
        const gdn_dtype gt = io_type(ga);
        need(ga.dim() == 2 && ga.size(0) == B && ga.size(1) == Hv && gb.sizes() == ga.sizes());
        on(ga, dev, ga.scalar_type());
        on(gb, dev, ga.scalar_type());
        const int64_t ldg = row_stride(ga);
        need(row_stride(gb) == ldg);
        const at::Tensor &A_log = whole(tensor(a[5]), dev, kF32, Hv), &dt_bias = whole(tensor(a[6]), dev, kF32, Hv);
        whole(pool, dev, kF32, 0);
        const at::Tensor &slots = whole(tensor(a[8]), dev, at::kInt, B);
        const double scale = number(a[9]);
        const int l2 = truth(a[10]) ? 1 : 0;
        if (n == 13) {
            at::ScalarType t = truth(a[12]) ? kF32 : kBf16;
            if (a[11] != Py_None) {
                t = tensor(a[11]).scalar_type();
                need(t == kBf16 || t == kF32);
            }
            const at::Tensor o = out(a[11], dev, t, {B, Hv, D}, true);
            Ref r = give(a[11], o);
            return done(lib.decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), ga.data_ptr(), gb.data_ptr(), ldg, gt, ptr<float>(A_log),
                                   ptr<float>(dt_bias), B, Hk, Hv, D, D, (float)scale, l2, GDN_BF16, ptr<float>(pool),
                                   i32(pool.size(0)), ptr<int32_t>(slots), o.data_ptr(), t == kBf16 ? GDN_BF16 : GDN_F32, stream()),
                        std::move(r));
        }
        const at::Tensor &z = on(tensor(a[12]), dev, kBf16), &w = whole(tensor(a[13]), dev, kF32, 128);
        need(z.sizes() == v.sizes() && z.stride(2) == 1 && (Hv <= 1 || z.stride(1) == D));
        const double eps = number(a[14]);
        void *o = a[11] == Py_None ? nullptr : whole(tensor(a[11]), dev, kBf16, v.numel()).data_ptr();
        const at::Tensor xq = out(a[15], dev, kF8, {B, (int64_t)Hv * D}, true), xs = out(a[16], dev, kF32, {B, Hv}, true);
        const Ref r0 = give(a[15], xq), r1 = give(a[16], xs);
        Ref r(PyTuple_Pack(3, r0.get(), r1.get(), a[11]));
        return done(lib.decode_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), ga.data_ptr(), gb.data_ptr(), ldg, gt, ptr<float>(A_log),
                                   ptr<float>(dt_bias), B, Hk, Hv, D, D, (float)scale, l2, GDN_BF16, ptr<float>(pool),
                                   i32(pool.size(0)), ptr<int32_t>(slots), z.data_ptr(), B > 1 ? z.stride(0) : (int64_t)Hv * D,
                                   ptr<float>(w), (float)eps, ptr<uint8_t>(xq), ptr<float>(xs), o, stream()),
                    std::move(r));
    });
}

// gdn_short_conv1d_silu_decode_pooled(x, weight, conv_pool, slots, plane widths or None, y or None): y or the planes' views
PyObject *py_conv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 6 && lib.conv);
        const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]), &pool = tensor(a[2]);
        const int dev = current_device_of(x);
        on(x, dev, kBf16);
        need(x.dim() == 2 && w.dim() == 2 && pool.dim() == 3 && (x.size(1) <= 1 || x.stride(1) == 1));
        const int32_t B = i32(x.size(0)), C = i32(x.size(1)), K = i32(w.size(1));
        need(w.size(0) == C && pool.size(1) == K - 1 && pool.size(2) == C);
        whole(w, dev, kF32, 0);
        whole(pool, dev, kBf16, 0);
        const at::Tensor &slots = whole(tensor(a[3]), dev, at::kInt, B);
        int32_t widths[4] = {0, 0, 0, 0}, parts = 0;
        int64_t sum = 0;
        if (a[4] != Py_None) {
            need(PyTuple_Check(a[4]) || PyList_Check(a[4]));
            need(PySequence_Fast_GET_SIZE(a[4]) >= 1 && PySequence_Fast_GET_SIZE(a[4]) <= 4);
            for (; parts < PySequence_Fast_GET_SIZE(a[4]); ++parts) {
                const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(a[4], parts));
                need(!PyErr_Occurred());
                widths[parts] = i32(v);
                sum += v;
            }
            need(sum == C);
        }
        const at::Tensor y = out(a[5], dev, kBf16, {B, C}, true);
        auto result = [&]() -> Ref {
            if (!parts && y.dim() == 2 && y.size(0) == B && y.size(1) == C) return give(a[5], y);
            const at::Tensor flat = y.view({-1});
            if (!parts) return Ref(THPVariable_Wrap(flat.narrow(0, 0, (int64_t)B * C).view({B, C})));
            Ref list(PyList_New(parts));
            int64_t at = 0;
            for (int32_t p = 0; p < parts; ++p) {
                Ref view(THPVariable_Wrap(flat.narrow(0, at, (int64_t)B * widths[p]).view({B, widths[p]})));
                PyList_SET_ITEM(list.get(), p, view.release());
                at += (int64_t)B * widths[p];
            }
            return list;
        };
        Ref r = result();
        return done(lib.conv(x.data_ptr(), B > 1 ? x.stride(0) : C, ptr<float>(w), B, C, K, pool.data_ptr(), i32(pool.size(0)),
                             ptr<int32_t>(slots), y.data_ptr(), parts ? widths : nullptr, parts, stream()),
                    std::move(r));
    });
}

// bind(addresses of fp8_gemm, fp8_quantize_act, fp8_quantize_weight, gdn_gated_rmsnorm_silu_fp8, gdn_decode_step_pooled,
// gdn_decode_step_pooled_gated_fp8, gdn_short_conv1d_silu_decode_pooled)
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
        return nullptr;
    }
    void *p[7];
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    lib.gemm = reinterpret_cast<decltype(lib.gemm)>(p[0]);
    lib.quantize_act = reinterpret_cast<decltype(lib.quantize_act)>(p[1]);
    lib.quantize_weight = reinterpret_cast<decltype(lib.quantize_weight)>(p[2]);
    lib.tail = reinterpret_cast<decltype(lib.tail)>(p[3]);
    lib.decode = reinterpret_cast<decltype(lib.decode)>(p[4]);
    lib.decode_fp8 = reinterpret_cast<decltype(lib.decode_fp8)>(p[5]);
    lib.conv = reinterpret_cast<decltype(lib.conv)>(p[6]);
    Py_RETURN_NONE;
}

#define ENTRY(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("bind", py_bind),
                         ENTRY("fp8_gemm", py_gemm),
                         ENTRY("fp8_quantize", py_quantize),
                         ENTRY("tail", py_tail),
                         ENTRY("decode", py_decode),
                         ENTRY("conv", py_conv),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#ifndef GDN_HOST_KEY   // what this file was built from and for (build.py)
#define GDN_HOST_KEY ""
#endif

PyMODINIT_FUNC PyInit__gdn_host() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "KEY", GDN_HOST_KEY) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
