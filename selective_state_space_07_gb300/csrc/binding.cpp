// The short way from Python to the C entry points of the language-model
// operators: each function here takes tensors as the Python binding gets them,
// and if every one is as it should be (CUDA, one device, the types, shapes,
// strides and alignment that the call wants, the current stream) allocates the
// outputs, makes the call and returns them. Anything else, and any error code,
// returns None: the Python binding then does the whole of it again, with its
// checks and messages. So nothing is decided here, and nothing kept.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <string>

#include "../../include/embedding.h"
#include "../../include/glr.h"
#include "../../include/layernorm.h"
#include "../../include/w4.h"

namespace {

// The library's entry points, as the Python binding loaded them.
struct Entries {
    decltype(&ssm_glr_fwd) glr_fwd;
    decltype(&ssm_glr_bwd) glr_bwd;
    decltype(&ssm_glr_step) glr_step;
    decltype(&ssm_glr_workspace_bytes) glr_workspace_bytes;
    decltype(&ssm_layernorm_fwd) layernorm_fwd;
    decltype(&ssm_layernorm_bwd) layernorm_bwd;
    decltype(&ssm_layernorm_workspace_bytes) layernorm_workspace_bytes;
    decltype(&ssm_embed_fwd) embed_fwd;
    decltype(&ssm_embed_bwd) embed_bwd;
    decltype(&ssm_embed_workspace_bytes) embed_workspace_bytes;
    decltype(&ssm_w4_matvec) w4_matvec;
    decltype(&ssm_w4_workspace_bytes) w4_workspace_bytes;
} lib;

constexpr int kSavedEvery = 32;  // tokens between the recurrence's saved states

// One call's arguments; `good` falls when one is not as the call wants it.
struct Call {
    bool good = true;
    c10::Device device{c10::DeviceType::CPU};
    cudaStream_t stream = nullptr;

    // The argument that the device and stream are taken from.
    const at::Tensor* lead(PyObject* o, int64_t dims) {
        if (!THPVariable_CheckExact(o)) return fail();
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || (dims >= 0 && t.dim() != dims) || t.layout() != c10::kStrided) return fail();
        device = t.device();
        if (device.index() != c10::cuda::current_device()) return fail();
        stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        return &t;
    }
    const at::Tensor* fail() {
        good = false;
        return nullptr;
    }
    static int io(const at::Tensor& t) {
        return t.scalar_type() == at::kBFloat16 ? (int)SSM_BF16 : t.scalar_type() == at::kFloat ? (int)SSM_F32 : -1;
    }
    bool is(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
        return t.scalar_type() == type && t.device() == device && t.sizes() == shape;
    }
    // Address of a dense tensor (None: null where that may be).
    template <typename T = void> T* dense(PyObject* o, at::ScalarType type, at::IntArrayRef shape, unsigned align, bool optional = false) {
        if (!good || (optional && o == Py_None)) return nullptr;
        if (!THPVariable_CheckExact(o)) return (T*)fail();
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!is(t, type, shape) || !t.is_contiguous()) return (T*)fail();
        void* p = t.data_ptr();
        if ((uintptr_t)p & (align - 1)) return (T*)fail();
        return static_cast<T*>(p);
    }
    // Address and row stride (0: dense) of rows [*, N] that are evenly spaced, both on 16 bytes.
    const void* rows(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int64_t& stride) {
        stride = 0;
        if (!good) return nullptr;
        if (!THPVariable_CheckExact(o)) return fail();
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!is(t, type, shape)) return fail();
        const int64_t n = t.dim();
        if (!t.is_contiguous()) {
            if (t.numel() == 0 || t.stride(n - 1) != 1) return fail();
            stride = t.stride(n - 2);
            if (stride < t.size(n - 1) || stride * (int64_t)t.element_size() % 16) return fail();
            for (int64_t i = n - 3; i >= 0; --i)
                if (t.stride(i) != t.stride(i + 1) * t.size(i + 1)) return fail();
        }
        void* p = t.data_ptr();
        if ((uintptr_t)p & 15) return fail();
        return p;
    }
    // A switch, as Python takes it: any object that counts as true.
    bool flag(PyObject* o) {
        const int v = o == Py_True ? 1 : o == Py_False ? 0 : PyObject_IsTrue(o);
        if (v < 0) good = false;  // (it has no truth: the long way raises what it raised)
        return v > 0;
    }
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) {
        return at::detail::empty_cuda(shape, type, device, std::nullopt);
    }
    // An output: the one given, checked, or a new one.
    template <typename T = void> T* out(PyObject* o, at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, unsigned align) {
        if (!good) return nullptr;
        if (o == Py_None) {
            t = make(shape, type);
            return static_cast<T*>(t.data_ptr());
        }
        T* p = dense<T>(o, type, shape, align);
        if (good) t = THPVariable_Unpack(o);
        return p;
    }
};

double number(PyObject* o) { return PyFloat_AsDouble(o); }  // (-1 with an error set if it is none: the caller looks)

// The buffer of the caller's workspace, on the call's device; None: none.
struct Space {
    void* at;
    size_t bytes;
};
Space space(Call& call, PyObject* o) {
    if (!call.good || o == Py_None) return {nullptr, 0};
    if (!THPVariable_CheckExact(o)) return call.fail(), Space{nullptr, 0};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != at::kByte || t.device() != call.device || t.dim() != 1 || !t.is_contiguous()) return call.fail(), Space{nullptr, 0};
    return {t.data_ptr(), (size_t)t.numel()};
}
// ... of which the status word is wanted only.
void* status(Call& call, PyObject* o) {
    const Space w = space(call, o);
    if (w.at && w.bytes < 256) call.fail();
    return w.at;
}

PyObject* none() {
    PyErr_Clear();
    Py_RETURN_NONE;
}
PyObject* give(std::initializer_list<const at::Tensor*> tensors) {
    PyObject* t = PyTuple_New((Py_ssize_t)tensors.size());
    Py_ssize_t i = 0;
    for (const at::Tensor* v : tensors) {
        PyObject* o = v && v->defined() ? THPVariable_Wrap(*v) : Py_NewRef(Py_None);
        PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

#define BINDING(name, count)                                                     \
    PyObject* name##_body(PyObject* const* a);                                   \
    PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {                \
        if (n != count) return none();                                           \
        try {                                                                    \
            return name##_body(a);                                               \
        } catch (const std::exception&) { /* out of memory, for one: said by the long way */ \
            return none();                                                       \
        }                                                                        \
    }                                                                            \
    PyObject* name##_body(PyObject* const* a)

// state, x, rgate, igate, lam, c, y or None, workspace or None
BINDING(glr_step, 8) {
    Call call;
    const at::Tensor* x = call.lead(a[1], 2);
    const double c = number(a[5]);
    if (!x || PyErr_Occurred()) return none();
    const auto type = x->scalar_type();
    const auto shape = x->sizes();
    ssm_glr_step_args s{};
    s.io_dtype = Call::io(*x);
    if (s.io_dtype < 0) return none();
    s.B = shape[0], s.D = shape[1], s.c = (float)c;
    s.x_t = call.rows(a[1], type, shape, s.x_stride);
    s.rgate_t = call.rows(a[2], type, shape, s.r_stride);
    s.igate_t = call.rows(a[3], type, shape, s.i_stride);
    s.lam = call.dense<float>(a[4], at::kFloat, {s.D}, 16);
    s.state = call.dense<float>(a[0], at::kFloat, shape, 16);
    at::Tensor y;
    s.y_t = call.out(a[6], y, type, shape, 16);
    s.workspace = status(call, a[7]);
    if (!call.good || PyErr_Occurred() || lib.glr_step(&s, call.stream)) return none();
    return THPVariable_Wrap(y);
}

bool glr_inputs(Call& call, PyObject* const* a, ssm_glr_args& s, const at::Tensor*& x) {
    x = call.lead(a[0], 3);
    const double c = number(a[4]);
    if (!x || PyErr_Occurred()) return false;
    const auto shape = x->sizes();
    s.io_dtype = Call::io(*x);
    if (s.io_dtype < 0) return false;
    s.B = shape[0], s.L = shape[1], s.D = shape[2], s.c = (float)c;
    s.x = call.rows(a[0], x->scalar_type(), shape, s.x_stride);
    s.rgate = call.rows(a[1], x->scalar_type(), shape, s.r_stride);
    s.igate = call.rows(a[2], x->scalar_type(), shape, s.i_stride);
    s.lam = call.dense<float>(a[3], at::kFloat, {s.D}, 16);
    return call.good;
}
// The caller's workspace, or scratch for this call.
bool glr_space(Call& call, PyObject* o, ssm_glr_args& s, at::Tensor& scratch) {
    const Space w = space(call, o);
    if (!call.good) return false;
    const size_t need = lib.glr_workspace_bytes(s.B, s.L, s.D);
    s.workspace = w.at, s.workspace_bytes = w.bytes;
    if (!w.at) {
        scratch = call.make({(int64_t)need}, at::kByte);
        s.workspace = scratch.data_ptr(), s.workspace_bytes = need;
    }
    return !PyErr_Occurred() && s.workspace_bytes >= need;
}

// x, rgate, igate, lam, c, h0, y, h_last, ckpt (each or None), want h_last, want ckpt, workspace or None
BINDING(glr_fwd, 12) {
    Call call;
    ssm_glr_args s{};
    const at::Tensor* x;
    if (!glr_inputs(call, a, s, x)) return none();
    at::Tensor y, last, ckpt, scratch;
    s.h0 = call.dense<float>(a[5], at::kFloat, {s.B, s.D}, 16, true);
    s.y = call.out(a[6], y, x->scalar_type(), x->sizes(), 16);
    if (a[7] != Py_None || call.flag(a[9])) s.h_last = call.out<float>(a[7], last, at::kFloat, {s.B, s.D}, 16);
    if (a[8] != Py_None) return none();  // (a buffer of the caller's may have any shape)
    if (call.flag(a[10])) s.ckpt = call.out<float>(Py_None, ckpt, at::kFloat, {s.B, (s.L + kSavedEvery - 1) / kSavedEvery, s.D}, 16);
    if (!call.good || !glr_space(call, a[11], s, scratch) || lib.glr_fwd(&s, call.stream)) return none();
    return give({&y, &last, &ckpt});
}

// x, rgate, igate, lam, c, dy, ckpt, dh_last or None, want dh0, workspace or None
BINDING(glr_bwd, 10) {
    Call call;
    ssm_glr_bwd_args s{};
    const at::Tensor* x;
    if (!glr_inputs(call, a, s.f, x)) return none();
    const ssm_glr_args& f = s.f;
    const auto type = x->scalar_type();
    const auto shape = x->sizes();
    s.dy = call.dense(a[5], type, shape, 16);
    s.f.ckpt = call.dense<float>(a[6], at::kFloat, {f.B, (f.L + kSavedEvery - 1) / kSavedEvery, f.D}, 16);
    s.dh_last = call.dense<float>(a[7], at::kFloat, {f.B, f.D}, 16, true);
    if (!call.good) return none();
    at::Tensor dx, dr, di, dlam, dh0, scratch;
    s.dx = call.out(Py_None, dx, type, shape, 16);
    s.drgate = call.out(Py_None, dr, type, shape, 16);
    s.digate = call.out(Py_None, di, type, shape, 16);
    s.dlam = call.out<float>(Py_None, dlam, at::kFloat, {f.D}, 16);
    if (call.flag(a[8])) s.dh0 = call.out<float>(Py_None, dh0, at::kFloat, {f.B, f.D}, 16);
    if (!call.good || !glr_space(call, a[9], s.f, scratch) || lib.glr_bwd(&s, call.stream)) return none();
    return give({&dx, &dr, &di, &dlam, &dh0});
}

bool norm_inputs(Call& call, PyObject* const* a, ssm_layernorm_args& s, const at::Tensor*& x) {
    x = call.lead(a[0], -1);
    if (!x || x->dim() < 1 || !x->is_contiguous()) return false;  // (slices go the long way)
    s.io_dtype = Call::io(*x);
    if (s.io_dtype < 0) return false;
    s.D = x->size(-1);
    s.rows = s.D ? x->numel() / s.D : 0;
    if (!s.D) return false;
    s.x = x->data_ptr();
    return true;
}

// x, weight, bias, eps, y or None, want statistics, workspace or None
BINDING(layer_norm_fwd, 7) {
    Call call;
    ssm_layernorm_args s{};
    const at::Tensor* x;
    if (!norm_inputs(call, a, s, x)) return none();
    s.eps = (float)number(a[3]);
    s.w = call.dense<float>(a[1], at::kFloat, {s.D}, 4, true);
    s.b = call.dense<float>(a[2], at::kFloat, {s.D}, 4, true);
    at::Tensor y, mean, rstd;
    const auto lead = x->sizes().slice(0, x->dim() - 1);
    s.y = call.out(a[4], y, x->scalar_type(), x->sizes(), 1);
    if (call.flag(a[5])) {
        s.mean = call.out<float>(Py_None, mean, at::kFloat, lead, 4);
        s.rstd = call.out<float>(Py_None, rstd, at::kFloat, lead, 4);
    }
    s.status = status(call, a[6]);
    if (!call.good || PyErr_Occurred() || lib.layernorm_fwd(&s, call.stream)) return none();
    return give({&y, &mean, &rstd});
}

// x, dy, mean, rstd, weight or None, dx or None, want dweight, want dbias, workspace or None
BINDING(layer_norm_bwd, 9) {
    Call call;
    ssm_layernorm_bwd_args s{};
    const at::Tensor* x;
    if (!norm_inputs(call, a, s.f, x)) return none();
    const auto lead = x->sizes().slice(0, x->dim() - 1);
    s.dy = call.dense(a[1], x->scalar_type(), x->sizes(), 1);
    s.f.mean = call.dense<float>(a[2], at::kFloat, lead, 4);
    s.f.rstd = call.dense<float>(a[3], at::kFloat, lead, 4);
    s.f.w = call.dense<float>(a[4], at::kFloat, {s.f.D}, 4, true);
    at::Tensor dx, dw, db, scratch;
    s.dx = call.out(a[5], dx, x->scalar_type(), x->sizes(), 1);
    if (call.flag(a[6])) s.dw = call.out<float>(Py_None, dw, at::kFloat, {s.f.D}, 4);
    if (call.flag(a[7])) s.db = call.out<float>(Py_None, db, at::kFloat, {s.f.D}, 4);
    s.f.status = status(call, a[8]);
    if (!call.good) return none();
    if (s.dw || s.db) {
        s.workspace_bytes = lib.layernorm_workspace_bytes(s.f.rows, s.f.D);
        if (s.workspace_bytes) {
            scratch = call.make({(int64_t)s.workspace_bytes}, at::kByte);
            s.workspace = scratch.data_ptr();
        }
    }
    if (PyErr_Occurred() || lib.layernorm_bwd(&s, call.stream)) return none();
    return give({&dx, &dw, &db});
}

const at::Tensor* ids_of(Call& call, PyObject* o, int32_t& ids64) {
    const at::Tensor* t = call.lead(o, -1);
    if (!t || !t->is_contiguous()) return nullptr;
    ids64 = t->scalar_type() == at::kLong;
    return ids64 || t->scalar_type() == at::kInt ? t : nullptr;
}

// ids, weight, scale, out or None, workspace or None
BINDING(embed_fwd, 5) {
    Call call;
    ssm_embed_args s{};
    const at::Tensor* ids = ids_of(call, a[0], s.ids64);
    if (!ids || !THPVariable_CheckExact(a[1])) return none();
    const at::Tensor& W = THPVariable_Unpack(a[1]);
    s.io_dtype = Call::io(W);
    if (s.io_dtype < 0 || W.dim() != 2 || W.device() != call.device || !W.is_contiguous()) return none();
    s.tokens = ids->numel(), s.V = W.size(0), s.D = W.size(1), s.scale = (float)number(a[2]);
    s.ids = ids->data_ptr(), s.W = W.data_ptr();
    c10::SmallVector<int64_t, 6> shape(ids->sizes().begin(), ids->sizes().end());
    shape.push_back(s.D);
    at::Tensor out;
    s.out = call.out(a[3], out, W.scalar_type(), shape, 1);
    s.status = status(call, a[4]);
    if (!call.good || PyErr_Occurred() || lib.embed_fwd(&s, call.stream)) return none();
    return THPVariable_Wrap(out);
}

// ids, dy, V, scale, padding id (-1: none), dweight or None, workspace or None
BINDING(embed_bwd, 7) {
    Call call;
    ssm_embed_bwd_args s{};
    const at::Tensor* ids = ids_of(call, a[0], s.ids64);
    if (!ids || !THPVariable_CheckExact(a[1])) return none();
    const at::Tensor& dy = THPVariable_Unpack(a[1]);
    s.io_dtype = Call::io(dy);
    if (s.io_dtype < 0 || dy.dim() < 1) return none();
    s.V = PyLong_AsLongLong(a[2]), s.scale = (float)number(a[3]), s.padding_id = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred() || s.V < 0 || s.padding_id < -1 || s.padding_id >= s.V) return none();
    s.tokens = ids->numel(), s.D = dy.size(-1);
    s.ids = ids->data_ptr();
    c10::SmallVector<int64_t, 6> shape(ids->sizes().begin(), ids->sizes().end());
    shape.push_back(s.D);
    s.dy = call.dense(a[1], dy.scalar_type(), shape, 1);
    at::Tensor dw, scratch;
    s.dW = call.out<float>(a[5], dw, at::kFloat, {s.V, s.D}, 4);
    s.status = status(call, a[6]);
    if (!call.good) return none();
    s.workspace_bytes = lib.embed_workspace_bytes(s.tokens, s.V, s.D);
    if (s.workspace_bytes) {
        scratch = call.make({(int64_t)s.workspace_bytes}, at::kByte);
        s.workspace = scratch.data_ptr();
    }
    if (PyErr_Occurred() || lib.embed_bwd(&s, call.stream)) return none();
    return THPVariable_Wrap(dw);
}

// x, qweight, scales, bias or None, out or None, out is fp32, workspace or None
BINDING(w4_matvec, 7) {
    Call call;
    ssm_w4_args s{};
    const at::Tensor* x = call.lead(a[0], -1);
    if (!x || x->dim() < 1 || !THPVariable_CheckExact(a[1]) || !THPVariable_CheckExact(a[2])) return none();
    const at::Tensor &q = THPVariable_Unpack(a[1]), &scales = THPVariable_Unpack(a[2]);
    if (q.dim() != 2 || scales.dim() != 2 || scales.size(1) == 0) return none();
    s.K = x->size(-1), s.N = q.size(0);
    s.group = (int32_t)(s.K / scales.size(1));
    if (s.K == 0 || (int64_t)s.group * scales.size(1) != s.K) return none();
    s.M = x->numel() / s.K;
    s.x = call.rows(a[0], at::kBFloat16, x->sizes(), s.x_stride);
    s.q = call.dense(a[1], at::kByte, {s.N, s.K / 2}, 16);
    s.s = call.dense(a[2], at::kBFloat16, {s.N, scales.size(1)}, 2);
    s.bias = call.dense<float>(a[3], at::kFloat, {s.N}, 4, true);
    const auto type = a[5] == Py_True ? at::kFloat : at::kBFloat16;
    s.y_dtype = a[5] == Py_True ? SSM_F32 : SSM_BF16;
    c10::SmallVector<int64_t, 6> shape(x->sizes().begin(), x->sizes().end() - 1);
    shape.push_back(s.N);
    at::Tensor y, scratch;
    s.y = call.out(a[4], y, type, shape, type == at::kFloat ? 4 : 2);
    const Space w = space(call, a[6]);
    if (!call.good || PyErr_Occurred()) return none();
    const size_t need = lib.w4_workspace_bytes(s.M, s.N, s.K);
    s.workspace = w.at, s.workspace_bytes = w.bytes;
    if (!w.at) {
        s.workspace_bytes = need;
        if (need > 256) {  // (256 bytes hold only the status, which nobody asked for)
            scratch = call.make({(int64_t)need}, at::kByte);
            s.workspace = scratch.data_ptr();
        }
    }
    if (lib.w4_matvec(&s, call.stream)) return none();
    return THPVariable_Wrap(y);
}

// Takes the entry points' addresses, in the order of Entries.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != (Py_ssize_t)(sizeof(Entries) / sizeof(void*))) {
        PyErr_SetString(PyExc_ValueError, "bind: another number of entry points");
        return nullptr;
    }
    void* at[sizeof(Entries) / sizeof(void*)];
    for (Py_ssize_t i = 0; i < n; ++i) at[i] = reinterpret_cast<void*>(PyLong_AsUnsignedLongLong(a[i]));
    if (PyErr_Occurred()) return nullptr;
    std::memcpy(&lib, at, sizeof lib);
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),           METHOD(glr_step),  METHOD(glr_fwd),   METHOD(glr_bwd),   METHOD(layer_norm_fwd),
                         METHOD(layer_norm_bwd), METHOD(embed_fwd), METHOD(embed_bwd), METHOD(w4_matvec), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
