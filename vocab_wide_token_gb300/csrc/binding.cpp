// binding.cpp -- argument marshalling of the sampling, filtered-statistics and
// gradient-clipping entry points, as a CPython module over torch's tensors.
//
// The same marshalling as in pstat.py costs 12 to 20 us of a call there, as much
// as the kernels of a decode step take, and 0.35 us per tensor of a gradient
// list.  Each function here takes the well-formed call only: it checks the
// arguments, allocates the outputs and the workspace, and calls the library.
// Whatever it does not take (a wrong type or shape, another device than the
// current one, an argument that the library refuses) it answers with None, having
// launched nothing, and pstat.py's own path then serves or refuses the call; so
// the rules and the messages are written once, there.  A failed launch is
// answered with its status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <optional>
#include <vector>

#include "pstat.h"

namespace {

// Addresses in the library that pstat.py loaded.
struct Library {
    decltype(&pstat_filter_workspace_size) filter_workspace_size;
    decltype(&pstat_sample) sample;
    decltype(&pstat_filtered_forward) filtered_forward;
    decltype(&pstat_filtered_backward) filtered_backward;
    decltype(&pstat_grad_workspace_size) grad_workspace_size;
    decltype(&pstat_grad_norm) grad_norm;
    decltype(&pstat_clip_grad_norm) clip_grad_norm;
} lib = {};

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Logits {
    const at::Tensor* t;
    int64_t T, V, ld;
    pstat_dtype dt;
    int device;
};
bool take_logits(PyObject* o, Logits& l) {
    l.t = tensor(o);
    if (!l.t || !l.t->defined() || !l.t->is_cuda() || l.t->dim() != 2 || l.t->stride(1) != 1) return false;
    if (l.t->scalar_type() == at::kBFloat16)
        l.dt = PSTAT_BF16;
    else if (l.t->scalar_type() == at::kFloat)
        l.dt = PSTAT_F32;
    else
        return false;
    l.T = l.t->size(0);
    l.V = l.t->size(1);
    l.ld = l.T > 1 ? l.t->stride(0) : l.V;
    l.device = l.t->get_device();
    return l.device == c10::cuda::current_device();
}

// A contiguous [T] (or [T, width]) tensor on the device.
bool take(PyObject* o, at::ScalarType type, int64_t T, int64_t width, int device, const void** p) {
    const at::Tensor* t = tensor(o);
    if (!t || !t->defined() || !t->is_cuda() || t->get_device() != device || t->scalar_type() != type ||
        t->dim() != (width ? 2 : 1) || t->size(0) != T || (width && t->size(1) != width) ||
        !t->is_contiguous())
        return false;
    *p = t->const_data_ptr();
    return true;
}
bool take_or_none(PyObject* o, at::ScalarType type, int64_t T, int device, const void** p) {
    *p = nullptr;
    return o == Py_None || take(o, type, T, 0, device, p);
}
bool take_flag(PyObject* o, int device, int** p) {
    *p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor* t = tensor(o);
    if (!t || !t->defined() || !t->is_cuda() || t->get_device() != device ||
        t->scalar_type() != at::kInt || t->numel() < 1 || !t->is_contiguous())
        return false;
    *p = t->mutable_data_ptr<int>();
    return true;
}
// A setting: a number, or a row array.
bool take_real(PyObject* o, int64_t T, int device, float* one, const float** many) {
    if (PyFloat_Check(o) || PyLong_Check(o)) {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
        *one = (float)v;
        return true;
    }
    return take(o, at::kFloat, T, 0, device, reinterpret_cast<const void**>(many));
}
bool take_filters(PyObject* const* a, int64_t T, int device, pstat_filters& f) {
    f = {1.f, 1.f, 0.f, 0, nullptr, nullptr, nullptr, nullptr};
    if (!take_real(a[0], T, device, &f.temperature, &f.temperatures)) return false;
    if (PyLong_Check(a[1])) {
        int over = 0;
        const long long k = PyLong_AsLongLongAndOverflow(a[1], &over);
        if (over) return false;
        f.top_k = k;
    } else if (!take(a[1], at::kInt, T, 0, device, reinterpret_cast<const void**>(&f.top_ks))) {
        return false;
    }
    return take_real(a[2], T, device, &f.top_p, &f.top_ps) && take_real(a[3], T, device, &f.min_p, &f.min_ps);
}
bool take_index(PyObject* o, int64_t* v) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    *v = PyLong_AsLongLongAndOverflow(o, &over);
    return !over;
}

// Straight to the allocator: through torch's dispatcher an output takes 0.5 us more.
at::Tensor empty(const at::Tensor& like, at::IntArrayRef size, at::ScalarType type) {
    return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}
pstat_stream_t stream_of(int device) {
    return reinterpret_cast<pstat_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
}
constexpr int kThrown = 1;  // no status of the library is positive

// Runs `work`, which returns a status of the library, without the interpreter lock.
template <typename F>
int run(F work) {
    int rc = kThrown;
    Py_BEGIN_ALLOW_THREADS;
    try {
        rc = work();
    } catch (const std::exception&) {  // out of memory, say: pstat.py meets it again
    }
    Py_END_ALLOW_THREADS;
    return rc;
}
PyObject* refuse(int rc) {
    if (rc == PSTAT_ERR_CUDA) return PyLong_FromLong(rc);
    Py_RETURN_NONE;
}
// torch's accessors throw on tensors without storage, sparse ones and the like;
// nothing may leave a C entry as an exception.
using Entry = PyObject* (*)(PyObject* const*, Py_ssize_t);
template <Entry entry>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        return entry(a, n);
    } catch (const std::exception&) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}
PyObject* pack(std::vector<at::Tensor>& v) {
    PyObject* t = PyTuple_New((Py_ssize_t)v.size());
    if (!t) return nullptr;
    for (size_t i = 0; i < v.size(); ++i) {
        PyObject* o = THPVariable_Wrap(std::move(v[i]));
        if (!o) {
            Py_DECREF(t);
            return nullptr;
        }
        PyTuple_SET_ITEM(t, (Py_ssize_t)i, o);
    }
    return t;
}

// sample(logits, uniform, temperature, top_k, top_p, min_p, dev_error)
PyObject* sample(PyObject* const* a, Py_ssize_t n) {
    Logits l;
    pstat_filters f;
    const void* u;
    int* err;
    if (n != 7 || !take_logits(a[0], l) || !take(a[1], at::kFloat, l.T, 0, l.device, &u) ||
        !take_filters(a + 2, l.T, l.device, f) || !take_flag(a[6], l.device, &err))
        Py_RETURN_NONE;
    std::vector<at::Tensor> out(2);
    const int rc = run([&] {
        size_t bytes = 0;
        const int fit = lib.filter_workspace_size(l.T, l.V, l.dt, &bytes);
        if (fit != PSTAT_OK) return fit;
        out[0] = empty(*l.t, {l.T}, at::kLong);
        out[1] = empty(*l.t, {l.T}, at::kFloat);
        at::Tensor ws = empty(*l.t, {(int64_t)bytes}, at::kByte);
        return lib.sample(l.t->const_data_ptr(), l.dt, l.T, l.V, l.ld, static_cast<const float*>(u), &f,
                          out[0].mutable_data_ptr<int64_t>(), out[1].mutable_data_ptr<float>(),
                          ws.mutable_data_ptr(), bytes, err, stream_of(l.device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    return pack(out);
}

// filtered_forward(logits, labels, temperature, top_k, top_p, min_p, ignore_index, dev_error)
PyObject* filtered_forward(PyObject* const* a, Py_ssize_t n) {
    Logits l;
    pstat_filters f;
    const void* y;
    int64_t ignore;
    int* err;
    if (n != 8 || !take_logits(a[0], l) || !take_or_none(a[1], at::kLong, l.T, l.device, &y) ||
        !take_filters(a + 2, l.T, l.device, f) || !take_index(a[6], &ignore) ||
        !take_flag(a[7], l.device, &err))
        Py_RETURN_NONE;
    std::vector<at::Tensor> out(5);
    const int rc = run([&] {
        size_t bytes = 0;
        const int fit = lib.filter_workspace_size(l.T, l.V, l.dt, &bytes);
        if (fit != PSTAT_OK) return fit;
        out[0] = empty(*l.t, {l.T}, at::kFloat);
        out[1] = empty(*l.t, {l.T}, at::kFloat);
        out[2] = empty(*l.t, {l.T, 2}, at::kFloat);
        out[3] = empty(*l.t, {l.T}, at::kFloat);
        out[4] = empty(*l.t, {l.T}, at::kLong);
        at::Tensor ws = empty(*l.t, {(int64_t)bytes}, at::kByte);
        return lib.filtered_forward(
            l.t->const_data_ptr(), l.dt, l.T, l.V, l.ld, static_cast<const int64_t*>(y), ignore, &f,
            out[0].mutable_data_ptr<float>(), out[1].mutable_data_ptr<float>(),
            out[2].mutable_data_ptr<float>(), out[3].mutable_data_ptr<float>(),
            out[4].mutable_data_ptr<int64_t>(), ws.mutable_data_ptr(), bytes, err, stream_of(l.device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    return pack(out);
}

// filtered_backward(logits, labels, weights, rowstats, cut_logit, cut_index, temperature,
//                   ignore_index, dev_error): a gradient of the logits' type
PyObject* filtered_backward(PyObject* const* a, Py_ssize_t n) {
    Logits l;
    const void *y, *w, *rs, *tau, *index;
    float t = 1.f;
    const float* ts = nullptr;
    int64_t ignore;
    int* err;
    if (n != 9 || !take_logits(a[0], l) || !take_or_none(a[1], at::kLong, l.T, l.device, &y) ||
        !take_or_none(a[2], at::kFloat, l.T, l.device, &w) ||
        !take(a[3], at::kFloat, l.T, 2, l.device, &rs) || !take(a[4], at::kFloat, l.T, 0, l.device, &tau) ||
        !take(a[5], at::kLong, l.T, 0, l.device, &index) || !take_real(a[6], l.T, l.device, &t, &ts) ||
        !take_index(a[7], &ignore) || !take_flag(a[8], l.device, &err))
        Py_RETURN_NONE;
    at::Tensor out;
    const int rc = run([&] {
        out = empty(*l.t, {l.T, l.V}, l.t->scalar_type());
        return lib.filtered_backward(
            l.t->const_data_ptr(), l.dt, l.T, l.V, l.ld, static_cast<const int64_t*>(y), ignore,
            static_cast<const float*>(w), static_cast<const float*>(rs), static_cast<const float*>(tau),
            static_cast<const int64_t*>(index), t, ts, out.mutable_data_ptr(), l.dt, l.V, err,
            stream_of(l.device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    return THPVariable_Wrap(std::move(out));
}

// The tensors of a tuple, and where each is written (itself, or `outs`).  No list is
// taken: the call goes on without the interpreter lock, and another thread could
// empty a list meanwhile and free what the launch uses.  A tuple keeps its tensors.
bool take_tuple(PyObject* list, PyObject* outs, bool writes, std::vector<pstat_tensor>& v,
                const at::Tensor** first) {
    if (!PyTuple_Check(list)) return false;
    const Py_ssize_t n = PyTuple_GET_SIZE(list);
    const bool apart = outs != Py_None;
    if (n == 0 || (apart && (!PyTuple_Check(outs) || PyTuple_GET_SIZE(outs) != n))) return false;
    v.resize((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor* x = tensor(PyTuple_GET_ITEM(list, i));
        const at::Tensor* o = apart ? tensor(PyTuple_GET_ITEM(outs, i)) : x;
        if (!x || !o || !x->defined() || !o->defined() || !x->is_cuda() || !x->is_contiguous()) return false;
        if (i == 0) *first = x;
        const at::ScalarType type = x->scalar_type();
        if ((type != at::kBFloat16 && type != at::kFloat) || x->get_device() != (*first)->get_device())
            return false;
        if (o != x && (!o->is_cuda() || o->get_device() != x->get_device() || o->scalar_type() != type ||
                       !o->is_contiguous() || o->sizes() != x->sizes()))
            return false;
        v[(size_t)i] = {x->const_data_ptr(), writes ? o->mutable_data_ptr() : nullptr, x->numel(),
                        type == at::kBFloat16 ? PSTAT_BF16 : PSTAT_F32};
    }
    return (*first)->get_device() == c10::cuda::current_device();
}

// grad_norm(tensors, dev_error) and clip_grad_norm(tensors, max_norm, out, dev_error): the norm
PyObject* norm_of(PyObject* list, PyObject* outs, PyObject* flag, bool clip, float max_norm) {
    std::vector<pstat_tensor> v;
    const at::Tensor* first = nullptr;
    int* err;
    if (!take_tuple(list, outs, clip, v, &first)) Py_RETURN_NONE;
    const at::Tensor& like = *first;
    const int device = like.get_device();
    if (!take_flag(flag, device, &err)) Py_RETURN_NONE;
    at::Tensor norm;
    const int rc = run([&] {
        size_t bytes = 0;
        const int fit = lib.grad_workspace_size(v.data(), (int64_t)v.size(), &bytes);
        if (fit != PSTAT_OK) return fit;
        norm = empty(like, {}, at::kFloat);
        at::Tensor ws = empty(like, {(int64_t)bytes}, at::kByte);
        return clip ? lib.clip_grad_norm(v.data(), (int64_t)v.size(), max_norm, norm.mutable_data_ptr<float>(),
                                         ws.mutable_data_ptr(), bytes, err, stream_of(device))
                    : lib.grad_norm(v.data(), (int64_t)v.size(), norm.mutable_data_ptr<float>(),
                                    ws.mutable_data_ptr(), bytes, err, stream_of(device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    if (clip) {  // an in-place change, for autograd to notice (inference tensors have no count)
        PyObject* written = outs == Py_None ? list : outs;
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(written); ++i) {
            const at::Tensor* x = tensor(PyTuple_GET_ITEM(written, i));
            if (!x->is_inference()) x->unsafeGetTensorImpl()->bump_version();
        }
    }
    return THPVariable_Wrap(std::move(norm));
}
PyObject* grad_norm(PyObject* const* a, Py_ssize_t n) {
    if (n != 2) Py_RETURN_NONE;
    return norm_of(a[0], Py_None, a[1], false, 0.f);
}
PyObject* clip_grad_norm(PyObject* const* a, Py_ssize_t n) {
    if (n != 4 || !(PyFloat_Check(a[1]) || PyLong_Check(a[1]))) Py_RETURN_NONE;
    const double limit = PyFloat_AsDouble(a[1]);
    if (limit == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return norm_of(a[0], a[2], a[3], true, (float)limit);
}

// bind(addresses): the library's functions, in the order of Library.
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
    void* p[7];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "seven addresses expected");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
            return nullptr;
        }
    }
    lib.filter_workspace_size = reinterpret_cast<decltype(lib.filter_workspace_size)>(p[0]);
    lib.sample = reinterpret_cast<decltype(lib.sample)>(p[1]);
    lib.filtered_forward = reinterpret_cast<decltype(lib.filtered_forward)>(p[2]);
    lib.filtered_backward = reinterpret_cast<decltype(lib.filtered_backward)>(p[3]);
    lib.grad_workspace_size = reinterpret_cast<decltype(lib.grad_workspace_size)>(p[4]);
    lib.grad_norm = reinterpret_cast<decltype(lib.grad_norm)>(p[5]);
    lib.clip_grad_norm = reinterpret_cast<decltype(lib.clip_grad_norm)>(p[6]);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),      FAST(sample),         FAST(filtered_forward), FAST(filtered_backward),
                         FAST(grad_norm), FAST(clip_grad_norm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module_def); }
