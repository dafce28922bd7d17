// binding.cpp -- argument marshalling of the sampling, filtered-statistics,
// gradient-clipping, optimiser, 8-bit head and beam search entry points, as a CPython
// module over torch's tensors.
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
    decltype(&pstat_adamw_step) adamw_step;
    decltype(&pstat_adamw_moments) adamw_moments;
    decltype(&pstat_fp8_quantize) fp8_quantize;
    decltype(&pstat_fp8_logits) fp8_logits;
    decltype(&pstat_beam_workspace_size) beam_workspace_size;
    decltype(&pstat_beam_select) beam_select;
    decltype(&pstat_beam_reorder) beam_reorder;
    decltype(&pstat_beam_gather) beam_gather;
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

// ---- the optimiser's step ------------------------------------------------------------

// An in-place change, for autograd to notice (inference tensors have no count).
void count_written(PyObject* tuple) {
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tuple); ++i) {
        const at::Tensor* x = tensor(PyTuple_GET_ITEM(tuple, i));
        if (!x->is_inference()) x->unsafeGetTensorImpl()->bump_version();
    }
}
bool take_number(PyObject* o, double* v) {
    if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
    *v = PyFloat_AsDouble(o);
    if (*v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}
// A contiguous tensor on `device`, of one of two types.
const at::Tensor* take_one(PyObject* o, int device, at::ScalarType a, at::ScalarType b) {
    const at::Tensor* t = tensor(o);
    if (!t || !t->defined() || !t->is_cuda() || t->get_device() != device || !t->is_contiguous() ||
        (t->scalar_type() != a && t->scalar_type() != b))
        return nullptr;
    return t;
}
int dtype_of(const at::Tensor* t) { return t->scalar_type() == at::kBFloat16 ? PSTAT_BF16 : PSTAT_F32; }
constexpr int64_t kAdamwBlock = 128;
int64_t codes_of(int64_t n) { return n + (n + kAdamwBlock - 1) / kAdamwBlock; }
// Tuples of one length, not empty.
bool take_tuples(PyObject* const* a, int count, Py_ssize_t* n) {
    for (int i = 0; i < count; ++i)
        if (!PyTuple_Check(a[i]) || PyTuple_GET_SIZE(a[i]) != PyTuple_GET_SIZE(a[0])) return false;
    *n = PyTuple_GET_SIZE(a[0]);
    return *n > 0;
}

// adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr, beta1, beta2, eps, weight_decay, norm,
//            max_norm, seed, dev_error): True.  Step, lr and seed as numbers.
PyObject* adamw_step(PyObject* const* a, Py_ssize_t argc) {
    Py_ssize_t n;
    if (argc != 14 || !take_tuples(a, 4, &n)) Py_RETURN_NONE;
    const int device = c10::cuda::current_device();
    pstat_adamw_options o = {};
    double max_norm = 0.0;
    int64_t seed = 0;
    int* err;
    if (!take_index(a[4], &o.step) || !take_number(a[5], &o.lr) || !take_number(a[6], &o.beta1) ||
        !take_number(a[7], &o.beta2) || !take_number(a[8], &o.eps) || !take_number(a[9], &o.weight_decay) ||
        !take_flag(a[13], device, &err) || (a[10] == Py_None) != (a[11] == Py_None))
        Py_RETURN_NONE;
    if (a[10] != Py_None) {
        const at::Tensor* norm = take_one(a[10], device, at::kFloat, at::kFloat);
        if (!norm || norm->dim() != 0 || !take_number(a[11], &max_norm)) Py_RETURN_NONE;
        o.norm = norm->const_data_ptr<float>();
        o.max_norm = (float)max_norm;
    }
    if (a[12] != Py_None) {
        if (!take_index(a[12], &seed)) Py_RETURN_NONE;
        o.seed = (uint64_t)seed;
        o.random = 1;
    }
    std::vector<pstat_adamw_tensor> v((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor* p = take_one(PyTuple_GET_ITEM(a[0], i), device, at::kBFloat16, at::kFloat);
        const at::Tensor* g = take_one(PyTuple_GET_ITEM(a[1], i), device, at::kBFloat16, at::kFloat);
        const at::Tensor* m = take_one(PyTuple_GET_ITEM(a[2], i), device, at::kFloat, at::kByte);
        const at::Tensor* s = take_one(PyTuple_GET_ITEM(a[3], i), device, at::kFloat, at::kByte);
        if (!p || !g || !m || !s || g->sizes() != p->sizes() || m->scalar_type() != s->scalar_type()) Py_RETURN_NONE;
        const bool small = m->scalar_type() == at::kByte;
        const int64_t size = p->numel(), want = small ? codes_of(size) : size;
        if (m->numel() != want || s->numel() != want) Py_RETURN_NONE;
        v[(size_t)i] = {p->mutable_data_ptr(), g->const_data_ptr(), m->mutable_data_ptr(), s->mutable_data_ptr(),
                        size, dtype_of(p), dtype_of(g), small ? 8 : 32, 0};
    }
    const int rc = run([&] { return lib.adamw_step(v.data(), (int64_t)n, &o, err, stream_of(device)); });
    if (rc != PSTAT_OK) return refuse(rc);
    count_written(a[0]);
    count_written(a[2]);
    count_written(a[3]);
    Py_RETURN_TRUE;
}

// adamw_moments(exp_avgs, exp_avg_sqs, params, out_avgs, out_avg_sqs): True.
PyObject* adamw_moments(PyObject* const* a, Py_ssize_t argc) {
    Py_ssize_t n;
    if (argc != 5 || !take_tuples(a, 5, &n)) Py_RETURN_NONE;
    const int device = c10::cuda::current_device();
    std::vector<pstat_adamw_moment> v((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor* p = tensor(PyTuple_GET_ITEM(a[2], i));
        const at::Tensor* m = take_one(PyTuple_GET_ITEM(a[0], i), device, at::kByte, at::kByte);
        const at::Tensor* s = take_one(PyTuple_GET_ITEM(a[1], i), device, at::kByte, at::kByte);
        const at::Tensor* om = take_one(PyTuple_GET_ITEM(a[3], i), device, at::kFloat, at::kFloat);
        const at::Tensor* os = take_one(PyTuple_GET_ITEM(a[4], i), device, at::kFloat, at::kFloat);
        if (!p || !p->defined() || !m || !s || !om || !os || om->sizes() != p->sizes() || os->sizes() != p->sizes() ||
            m->numel() != codes_of(p->numel()) || s->numel() != codes_of(p->numel()))
            Py_RETURN_NONE;
        v[(size_t)i] = {m->const_data_ptr(), s->const_data_ptr(), om->mutable_data_ptr<float>(),
                        os->mutable_data_ptr<float>(), p->numel()};
    }
    const int rc = run([&] { return lib.adamw_moments(v.data(), (int64_t)n, stream_of(device)); });
    if (rc != PSTAT_OK) return refuse(rc);
    count_written(a[3]);
    count_written(a[4]);
    Py_RETURN_TRUE;
}

// ---- the head in 8 bits ----------------------------------------------------------------

constexpr int64_t kFp8Block = 128;
int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// fp8_quantize(x, rows, dev_error): (codes, scales)
PyObject* fp8_quantize(PyObject* const* a, Py_ssize_t argc) {
    Logits l;
    int64_t rows;
    int* err;
    if (argc != 3 || !take_logits(a[0], l) || !take_index(a[1], &rows) || (rows != 1 && rows != kFp8Block) ||
        !take_flag(a[2], l.device, &err))
        Py_RETURN_NONE;
    std::vector<at::Tensor> out(2);
    const int rc = run([&] {
        const int64_t r = (l.T + rows - 1) / rows, c = blocks_of(l.V);
        out[0] = empty(*l.t, {l.T, l.V}, at::kFloat8_e4m3fn);
        out[1] = rows != 1 ? empty(*l.t, {r, c}, at::kFloat) : empty(*l.t, {c, r}, at::kFloat).t();
        return lib.fp8_quantize(l.t->const_data_ptr(), l.dt, l.T, l.V, l.ld, (int)rows, out[0].mutable_data_ptr(),
                                out[1].mutable_data_ptr<float>(), out[1].stride(0), out[1].stride(1), err,
                                stream_of(l.device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    return pack(out);
}

// fp8_logits(q, q_scale, W, W_scale, bf16, dev_error): logits
PyObject* fp8_logits(PyObject* const* a, Py_ssize_t argc) {
    if (argc != 6 || !PyBool_Check(a[4])) Py_RETURN_NONE;
    const int device = c10::cuda::current_device();
    const at::Tensor* q = take_one(a[0], device, at::kFloat8_e4m3fn, at::kFloat8_e4m3fn);
    const at::Tensor* W = take_one(a[2], device, at::kFloat8_e4m3fn, at::kFloat8_e4m3fn);
    const at::Tensor* Ws = take_one(a[3], device, at::kFloat, at::kFloat);
    const at::Tensor* qs = tensor(a[1]);
    int* err;
    if (!q || !W || !Ws || !qs || !qs->defined() || !qs->is_cuda() || qs->get_device() != device ||
        qs->scalar_type() != at::kFloat || q->dim() != 2 || W->dim() != 2 || qs->dim() != 2 || Ws->dim() != 2 ||
        !take_flag(a[5], device, &err))
        Py_RETURN_NONE;
    const int64_t T = q->size(0), K = q->size(1), V = W->size(0), c = blocks_of(K);
    if (W->size(1) != K || qs->size(0) != T || qs->size(1) != c || Ws->size(0) != blocks_of(V) || Ws->size(1) != c)
        Py_RETURN_NONE;
    const bool bf16 = a[4] == Py_True;
    at::Tensor out;
    const int rc = run([&] {
        out = empty(*q, {T, V}, bf16 ? at::kBFloat16 : at::kFloat);
        return lib.fp8_logits(q->const_data_ptr(), qs->const_data_ptr<float>(), qs->stride(0), qs->stride(1),
                              W->const_data_ptr(), Ws->const_data_ptr<float>(), T, V, K, out.mutable_data_ptr(),
                              bf16 ? PSTAT_BF16 : PSTAT_F32, V, err, stream_of(device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    return THPVariable_Wrap(std::move(out));
}

// ---- beam search ------------------------------------------------------------------------

// beam_select(logits, scores, n, dev_error): (score, parent, token)
PyObject* beam_select(PyObject* const* a, Py_ssize_t argc) {
    Logits l;
    int64_t n;
    int* err;
    if (argc != 4 || !take_logits(a[0], l) || !take_index(a[2], &n) || n < 1 || n > PSTAT_BEAM_MAX_N ||
        !take_flag(a[3], l.device, &err))
        Py_RETURN_NONE;
    const at::Tensor* scores = take_one(a[1], l.device, at::kFloat, at::kFloat);
    if (!scores || scores->dim() != 2 || scores->numel() != l.T) Py_RETURN_NONE;
    const int64_t B = scores->size(0), beams = scores->size(1);
    std::vector<at::Tensor> out(3);
    const int rc = run([&] {
        size_t bytes = 0;
        const int fit = lib.beam_workspace_size(B, beams, l.V, l.dt, &bytes);
        if (fit != PSTAT_OK) return fit;
        out[0] = empty(*l.t, {B, n}, at::kFloat);
        out[1] = empty(*l.t, {B, n}, at::kLong);
        out[2] = empty(*l.t, {B, n}, at::kLong);
        at::Tensor ws = empty(*l.t, {(int64_t)bytes}, at::kByte);
        return lib.beam_select(l.t->const_data_ptr(), l.dt, B, beams, l.V, l.ld, scores->const_data_ptr<float>(), n,
                               out[0].mutable_data_ptr<float>(), out[1].mutable_data_ptr<int64_t>(),
                               out[2].mutable_data_ptr<int64_t>(), ws.mutable_data_ptr(), bytes, err,
                               stream_of(l.device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    return pack(out);
}

// A row of `x` and of `o` as evenly spaced runs; false where it takes more than one set.
bool take_runs(const at::Tensor& x, const at::Tensor& o, pstat_beam_state* s) {
    const int64_t size = (int64_t)x.element_size();
    int64_t d = x.dim() - 1, run_size = 1;
    for (; d > 0; --d) {
        if (x.size(d) == 1) continue;
        if (x.stride(d) != run_size || o.stride(d) != run_size) break;
        run_size *= x.size(d);
    }
    int64_t segments = 1, sx = run_size, so = run_size;
    bool any = false;
    for (; d > 0; --d) {
        if (x.size(d) == 1) continue;
        if (!any) {
            segments = x.size(d);
            sx = x.stride(d);
            so = o.stride(d);
            any = true;
        } else if (x.stride(d) == segments * sx && o.stride(d) == segments * so) {
            segments *= x.size(d);
        } else {
            return false;
        }
    }
    *s = {x.const_data_ptr(), const_cast<void*>(o.const_data_ptr()), x.stride(0) * size, o.stride(0) * size, segments,
          sx * size, so * size, run_size * size};
    return true;
}

// beam_reorder(states, parents, outs or None, dev_error): True, or the new tensors
PyObject* beam_reorder(PyObject* const* a, Py_ssize_t argc) {
    if (argc != 4 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) == 0) Py_RETURN_NONE;
    const bool given = a[2] != Py_None;
    const Py_ssize_t n = PyTuple_GET_SIZE(a[0]);
    if (given && (!PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) != n)) Py_RETURN_NONE;
    const int device = c10::cuda::current_device();
    const at::Tensor* parents = take_one(a[1], device, at::kLong, at::kLong);
    int* err;
    if (!parents || parents->dim() != 2 || parents->size(0) == 0 || !take_flag(a[3], device, &err)) Py_RETURN_NONE;
    const int64_t B = parents->size(0), out_beams = parents->size(1);
    std::vector<at::Tensor> made(given ? 0 : (size_t)n);
    std::vector<const at::Tensor*> xs((size_t)n), os((size_t)n);
    int64_t rows = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor* x = tensor(PyTuple_GET_ITEM(a[0], i));
        const at::Tensor* o = given ? tensor(PyTuple_GET_ITEM(a[2], i)) : nullptr;
        if (!x || !x->defined() || !x->is_cuda() || x->layout() != at::kStrided || x->get_device() != device ||
            x->dim() < 1 || x->is_conj() || x->is_neg() || x->numel() == 0 || (i > 0 && x->size(0) != rows))
            Py_RETURN_NONE;
        rows = x->size(0);
        if (given) {
            if (!o || !o->defined() || !o->is_cuda() || o->layout() != at::kStrided || o->get_device() != device ||
                o->scalar_type() != x->scalar_type() || o->dim() != x->dim() || o->size(0) != B * out_beams ||
                o->sizes().slice(1) != x->sizes().slice(1) || o->is_conj() || o->is_neg())
                Py_RETURN_NONE;
            os[(size_t)i] = o;
        }
        xs[(size_t)i] = x;
    }
    if (rows % B) Py_RETURN_NONE;
    bool taken = true;
    const int rc = run([&] {
        std::vector<pstat_beam_state> v((size_t)n);
        for (size_t i = 0; i < (size_t)n; ++i) {
            if (!given) {
                std::vector<int64_t> shape(xs[i]->sizes().begin(), xs[i]->sizes().end());
                shape[0] = B * out_beams;
                made[i] = empty(*xs[i], shape, xs[i]->scalar_type());
                os[i] = &made[i];
            }
            taken = taken && take_runs(*xs[i], *os[i], &v[i]);
        }
        if (!taken) return (int)PSTAT_OK;
        return (given ? lib.beam_reorder : lib.beam_gather)(v.data(), (int64_t)n, parents->const_data_ptr<int64_t>(),
                                                            B, rows / B, out_beams, err, stream_of(device));
    });
    if (rc != PSTAT_OK) return refuse(rc);
    if (!taken) Py_RETURN_NONE;
    if (!given) return pack(made);
    count_written(a[2]);
    Py_RETURN_TRUE;
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

// bind_gather(address): the last one.
PyObject* bind_gather(PyObject* const* a, Py_ssize_t n) {
    void* p = n == 1 ? PyLong_AsVoidPtr(a[0]) : nullptr;
    if (!p) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "one address expected, not null");
        return nullptr;
    }
    lib.beam_gather = reinterpret_cast<decltype(lib.beam_gather)>(p);
    Py_RETURN_NONE;
}

// bind_more(addresses): those from adamw_step to beam_reorder.
PyObject* bind_more(PyObject* const* a, Py_ssize_t n) {
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
    lib.adamw_step = reinterpret_cast<decltype(lib.adamw_step)>(p[0]);
    lib.adamw_moments = reinterpret_cast<decltype(lib.adamw_moments)>(p[1]);
    lib.fp8_quantize = reinterpret_cast<decltype(lib.fp8_quantize)>(p[2]);
    lib.fp8_logits = reinterpret_cast<decltype(lib.fp8_logits)>(p[3]);
    lib.beam_workspace_size = reinterpret_cast<decltype(lib.beam_workspace_size)>(p[4]);
    lib.beam_select = reinterpret_cast<decltype(lib.beam_select)>(p[5]);
    lib.beam_reorder = reinterpret_cast<decltype(lib.beam_reorder)>(p[6]);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),      FAST(sample),         FAST(filtered_forward), FAST(filtered_backward),
                         FAST(grad_norm), FAST(clip_grad_norm), FAST(bind_more),    FAST(bind_gather),
                         FAST(adamw_step), FAST(adamw_moments), FAST(fp8_quantize), FAST(fp8_logits),
                         FAST(beam_select), FAST(beam_reorder), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module_def); }
