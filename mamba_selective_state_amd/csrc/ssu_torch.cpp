// The layer operators' Python functions in C++: torch tensors to the C ABI's
// descriptors, outputs and workspaces allocated, statuses to exceptions. It holds no
// arithmetic. A decode step's norms and small products take a few microseconds on
// the GPU; the same marshalling in Python took 10 to 15 us a call, this 4 to 5.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/DeviceGuard.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "../../include/ssu.h"

namespace {

PyObject *g_error_type = nullptr;  // SsuError

// Carries a Python exception that is already set.
struct PythonError {};

[[noreturn]] void raise(PyObject *type, const std::string &msg) {
    PyErr_SetString(type, msg.c_str());
    throw PythonError();
}

void check(ssu_status_t st, const char *what) {
    if (st == SSU_OK)
        return;
    raise(st == SSU_ERR_VALUE             ? PyExc_ValueError
          : st == SSU_ERR_NOT_IMPLEMENTED ? PyExc_NotImplementedError
                                          : (g_error_type ? g_error_type : PyExc_RuntimeError),
          std::string(what) + ": " + ssu_last_error());
}

int dtype_code(at::ScalarType t) {
    switch (t) {
    case at::kFloat: return SSU_F32;
    case at::kHalf: return SSU_F16;
    case at::kBFloat16: return SSU_BF16;
    case at::kInt: return SSU_I32;
    case at::kLong: return SSU_I64;
    case at::kByte: return SSU_U8;
    default: raise(PyExc_ValueError, std::string("unsupported dtype ") + c10::toString(t));
    }
}

// A tensor argument, or null for None.
const at::Tensor *tensor(PyObject *o) {
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        raise(PyExc_TypeError, std::string("expected a torch.Tensor, got ") + Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}
const at::Tensor &required(PyObject *o, const char *name) {
    const at::Tensor *t = tensor(o);
    if (!t)
        raise(PyExc_TypeError, std::string(name) + " is required");
    return *t;
}

void describe_base(const at::Tensor &t, const at::Device &dev, ssu_tensor_t *d) {
    if (!t.is_cuda() || t.device() != dev)
        raise(PyExc_ValueError, "every tensor must live on the first one's GPU");
    d->data = t.data_ptr() ? t.data_ptr() : reinterpret_cast<void *>(16);  // empty, not absent
    d->dtype = dtype_code(t.scalar_type());
}

void describe(const at::Tensor &t, const at::Device &dev, ssu_tensor_t *d) {
    describe_base(t, dev, d);
    if (t.dim() > 4)
        raise(PyExc_ValueError, "tensors have at most 4 dimensions");
    d->ndim = static_cast<int32_t>(t.dim());
    for (int64_t i = 0; i < t.dim(); i++)
        d->size[i] = t.size(i), d->stride[i] = t.stride(i);
}

// [..., k] as [rows, k] without a copy.
void describe_rows(const at::Tensor &t, const at::Device &dev, const char *name, ssu_tensor_t *d) {
    describe_base(t, dev, d);
    const int64_t n = t.dim();
    if (n == 0)
        raise(PyExc_ValueError, std::string(name) + " must have at least one dimension");
    d->ndim = 2;
    d->size[0] = 1;
    d->size[1] = t.size(n - 1);
    d->stride[0] = d->size[1];
    d->stride[1] = t.stride(n - 1);
    bool first = true;
    for (int64_t i = n - 2; i >= 0; i--) {
        const int64_t size = t.size(i);
        if (size != 1) {
            if (first)
                d->stride[0] = t.stride(i);
            else if (t.stride(i) != d->stride[0] * d->size[0] && d->size[0] != 0 && size != 0)
                raise(PyExc_ValueError, std::string(name) + ": its leading dimensions must collapse to rows of one stride");
            first = false;
        }
        d->size[0] *= size;
    }
}

// Shape of `t` with its last dimension replaced.
std::vector<int64_t> shape_with(const at::Tensor &t, int64_t last) {
    std::vector<int64_t> s(t.sizes().begin(), t.sizes().end());
    if (s.empty())
        raise(PyExc_ValueError, "tensors must have at least one dimension");
    s.back() = last;
    return s;
}
int64_t last_size(const at::Tensor &t) { return t.dim() ? t.size(t.dim() - 1) : 0; }

at::Tensor make(const at::Tensor &like, at::IntArrayRef shape, at::ScalarType dtype) {
    return at::empty(shape, like.options().dtype(dtype));
}

// Whether what is enqueued on the stream now goes into a graph.
bool capturing(uintptr_t stream) {
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(reinterpret_cast<hipStream_t>(stream), &status) != hipSuccess)
        (void)hipGetLastError();  // the launch reports what is wrong with the stream
    return status != hipStreamCaptureStatusNone;
}

// Scratch memory of one call, from torch's allocator and on the call's stream: given back when the call
// has been enqueued, it is handed out again only behind the call's kernels. While a graph is
// captured it is the graph's own memory, which stays with the graph.
at::Tensor scratch(const at::Tensor &like, int64_t bytes) {
    return bytes > 0 ? at::empty({bytes}, like.options().dtype(at::kByte)) : at::Tensor();
}

// The workspaces of token_logprobs, whose first bytes are zero between calls: one per device and
// stream, on which calls are ordered, grown to what a call needs. No graph uses them: a graph would
// go on writing to one that has been replaced, or while another graph that was captured on the same stream runs.
struct Workspace {
    int8_t device;
    uintptr_t stream;
    at::Tensor memory;
};
// never destroyed: the interpreter may end after torch's allocator
std::vector<Workspace> &workspaces = *new std::vector<Workspace>();

at::Tensor logprob_workspace(const at::Tensor &like, uintptr_t stream, int64_t bytes) {
    if (bytes == 0)
        return at::Tensor();
    if (capturing(stream)) {  // the call's own, zeroed by every replay
        at::Tensor own = scratch(like, bytes);
        own.narrow(0, 0, SSU_LOGPROB_ZEROED_BYTES).zero_();
        return own;
    }
    Workspace *w = nullptr;
    for (Workspace &c : workspaces)
        if (c.device == like.get_device() && c.stream == stream)
            w = &c;
    if (!w) {
        workspaces.push_back({static_cast<int8_t>(like.get_device()), stream, at::Tensor()});
        w = &workspaces.back();
    }
    if (!w->memory.defined() || w->memory.numel() < bytes)
        w->memory = at::zeros({bytes}, like.options().dtype(at::kByte));
    return w->memory;
}

int64_t as_int(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw PythonError();
    return v;
}
double as_double(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw PythonError();
    return v;
}
uintptr_t as_stream(PyObject *o) {
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (v == static_cast<unsigned long long>(-1) && PyErr_Occurred())
        throw PythonError();
    return static_cast<uintptr_t>(v);
}

// torch.OutOfMemoryError, by which callers tell it from other errors.
void set_out_of_memory(const char *what) {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type)
        PyErr_SetString(type, what);  // otherwise the import's own error stands
    Py_XDECREF(type);
    Py_XDECREF(torch);
}

// No C++ exception leaves the module.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F &&f) {
    try {
        if (n != want)
            raise(PyExc_TypeError, "wrong number of arguments");
        return f();
    } catch (const PythonError &) {
    } catch (const c10::OutOfMemoryError &e) {
        set_out_of_memory(e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *none() { return Py_NewRef(Py_None); }
// a given output itself, or a made one
PyObject *given(PyObject *o, const at::Tensor &t) { return o != Py_None ? Py_NewRef(o) : t.defined() ? wrap(t) : none(); }

// (x, weight, residual, gate, groups, eps, format, out, out_scales, residual_out, stream)
// -> (out, out_scales or None, residual_out or None)
PyObject *add_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const at::Tensor &x = required(a[0], "x"), &weight = required(a[1], "weight");
        const at::Tensor *residual = tensor(a[2]), *gate = tensor(a[3]);
        const int format = static_cast<int>(as_int(a[6]));
        const at::Tensor *out = tensor(a[7]), *scales = tensor(a[8]), *residual_out = tensor(a[9]);
        const at::Device dev = x.device();
        const c10::DeviceGuard guard(dev);  // the default stream's handle is the current GPU's
        ssu_norm_args_t args = {};
        describe_rows(x, dev, "x", &args.x);
        describe(weight, dev, &args.weight);
        at::Tensor made_out, made_scales, made_residual;
        const int64_t dim = last_size(x);
        if (!out) {
            made_out = format == SSU_FORMAT_SAME ? make(x, x.sizes(), x.scalar_type())
                                                 : make(x, shape_with(x, format == SSU_FORMAT_MXFP4 ? dim / 2 : dim), at::kByte);
            out = &made_out;
        }
        describe_rows(*out, dev, "out", &args.out);
        if (!scales && format != SSU_FORMAT_SAME) {
            made_scales = make(x, shape_with(x, dim / 32), at::kByte);
            scales = &made_scales;
        }
        if (scales)
            describe_rows(*scales, dev, "out_scales", &args.out_scales);
        if (residual) {
            describe_rows(*residual, dev, "residual", &args.residual);
            if (!residual_out) {
                made_residual = make(x, residual->sizes(), residual->scalar_type());
                residual_out = &made_residual;
            }
        }
        if (residual_out)
            describe_rows(*residual_out, dev, "residual_out", &args.residual_out);
        if (gate)
            describe_rows(*gate, dev, "gate", &args.gate);
        args.groups = as_int(a[4]);
        args.eps = static_cast<float>(as_double(a[5]));
        args.out_format = format;
        check(ssu_add_rms_norm(&args, reinterpret_cast<void *>(as_stream(a[10]))), "ssu_add_rms_norm");
        PyObject *r = PyTuple_New(3);
        if (!r)
            throw PythonError();
        PyTuple_SET_ITEM(r, 0, given(a[7], made_out));
        PyTuple_SET_ITEM(r, 1, given(a[8], made_scales));
        PyTuple_SET_ITEM(r, 2, given(a[9], made_residual));
        return r;
    });
}

// (x, x_scale, weight, weight_scale, bias, format, out, like, stream) -> out; `like`: a tensor
// of the dtype that a made output takes, or None for bf16
PyObject *mx_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const at::Tensor &x = required(a[0], "x"), &w = required(a[2], "weight"), &ws = required(a[3], "weight_scale");
        const at::Tensor *x_scale = tensor(a[1]), *bias = tensor(a[4]), *out = tensor(a[6]);
        const at::Device dev = x.device();
        const c10::DeviceGuard guard(dev);  // the default stream's handle is the current GPU's
        ssu_mx_linear_args_t args = {};
        describe_rows(x, dev, "x", &args.x);
        describe(w, dev, &args.w);
        describe(ws, dev, &args.w_scale);
        if (x_scale)
            describe_rows(*x_scale, dev, "x_scale", &args.x_scale);
        if (bias)
            describe(*bias, dev, &args.bias);
        args.x_format = static_cast<int32_t>(as_int(a[5]));
        at::Tensor made;
        if (!out) {
            const at::Tensor *like = tensor(a[7]);
            made = make(x, shape_with(x, w.dim() ? w.size(0) : 0), like ? like->scalar_type() : at::kBFloat16);
            out = &made;
        }
        describe_rows(*out, dev, "out", &args.out);
        const uintptr_t stream = as_stream(a[8]);
        const at::Tensor ws_mem = scratch(x, ssu_mx_linear_workspace_bytes(&args));
        check(ssu_mx_linear(&args, ws_mem.defined() ? ws_mem.data_ptr() : nullptr, ws_mem.defined() ? ws_mem.numel() : 0,
                            reinterpret_cast<void *>(stream)),
              "ssu_mx_linear");
        return given(a[6], made);
    });
}

// (logits, tokens, mask, temperature, top, stream) -> (logprob, entropy, rank, top_tokens, top_logprobs)
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor &logits = required(a[0], "logits"), &tokens = required(a[1], "tokens");
        const at::Tensor *mask = tensor(a[2]), *temperature = tensor(a[3]);
        const int64_t top = as_int(a[4]);
        const at::Device dev = logits.device();
        const c10::DeviceGuard guard(dev);
        if (top < 0)
            raise(PyExc_ValueError, "top must not be negative");
        ssu_logprob_args_t args = {};
        describe(logits, dev, &args.logits);
        describe(tokens, dev, &args.tokens);
        const int64_t rows = tokens.dim() ? tokens.size(0) : 0;
        if (mask) {
            describe(*mask, dev, &args.mask);
            if (args.mask.ndim == 2 && args.mask.size[0] == 1 && rows != 1)  // one mask for all rows
                args.mask.size[0] = rows, args.mask.stride[0] = 0;
        }
        if (temperature)
            describe(*temperature, dev, &args.temperature);
        at::Tensor made[5] = {make(logits, {rows}, at::kFloat), make(logits, {rows}, at::kFloat), make(logits, {rows}, at::kInt)};
        ssu_tensor_t *at[5] = {&args.logprob, &args.entropy, &args.rank, &args.top_tokens, &args.top_logprobs};
        if (top) {
            made[3] = make(logits, {rows, top}, at::kInt);
            made[4] = make(logits, {rows, top}, at::kFloat);
        }
        for (int i = 0; i < (top ? 5 : 3); i++)
            describe(made[i], dev, at[i]);
        const uintptr_t stream = as_stream(a[5]);
        const at::Tensor ws = logprob_workspace(logits, stream, ssu_token_logprobs_workspace_bytes(&args));
        check(ssu_token_logprobs(&args, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0,
                                 reinterpret_cast<void *>(stream)),
              "ssu_token_logprobs");
        PyObject *r = PyTuple_New(5);
        if (!r)
            throw PythonError();
        for (int i = 0; i < 5; i++)
            PyTuple_SET_ITEM(r, i, made[i].defined() ? wrap(made[i]) : none());
        return r;
    });
}

PyObject *set_error_type(PyObject *, PyObject *type) {
    Py_XDECREF(g_error_type);
    g_error_type = Py_NewRef(type);
    return none();
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"add_rms_norm", fast<add_rms_norm>(), METH_FASTCALL, nullptr},
    {"mx_linear", fast<mx_linear>(), METH_FASTCALL, nullptr},
    {"token_logprobs", fast<token_logprobs>(), METH_FASTCALL, nullptr},
    {"set_error_type", set_error_type, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ssu_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__ssu_torch(void) { return PyModule_Create(&module); }
