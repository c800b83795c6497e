// binding.cpp -- the Python calls of layer norm, embeddings and AdamW over torch tensors:
// checks, outputs and workspaces from torch's allocator, then the C ABI (migemm.h).
//
// The same in Python, through ctypes, took 10 us for a layer norm with its statistics, 17
// for its backward pass and 1.1 to 2 us for each tensor of an AdamW step, most of it in
// reading tensors' attributes, beside kernels of 3 to 7 us.
//
// Functions take their arguments in order (the package's functions give them names and
// defaults) and end with the stream's handle and whether the workspace is to be returned
// as well, for a stream that torch's allocator does not know of.  They return a tuple of
// tensors, or the call's status where it is not MIGEMM_OK; a refused argument raises
// ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <sstream>
#include <string>
#include <vector>

#include "migemm.h"

namespace {

struct Refused {
    std::string what;
};
template <typename... P> [[noreturn]] void refuse(const P&... p) {
    std::ostringstream s;
    (s << ... << p);
    throw Refused{s.str()};
}
struct PythonError {};  // one is set

const char* name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kChar: return "torch.int8";
        case at::kInt: return "torch.int32";
        default: return c10::toString(t);
    }
}

int code_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return MIGEMM_F32;
        case at::kHalf: return MIGEMM_F16;
        case at::kBFloat16: return MIGEMM_BF16;
        case at::kChar: return MIGEMM_I8;
        case at::kInt: return MIGEMM_I32;
        default:
            refuse("unsupported dtype ", name_of(t.scalar_type()),
                   "; expected float32, float16, bfloat16, int8 (operands) or int32 (output of an "
                   "int8 product)");
    }
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor (got ", Py_TYPE(o)->tp_name, ")");
    return THPVariable_Unpack(o);
}
// None: no tensor.
const at::Tensor* optional(const char* name, PyObject* o) {
    return o == Py_None ? nullptr : &tensor(name, o);
}

void check_device(const char* name, const at::Tensor& t, at::Device device) {
    if (!t.is_cuda()) refuse(name, " must be on the GPU (got ", t.device().str(), ")");
    if (t.device() != device)
        refuse(name, " is on ", t.device().str(), ", the operands on ", device.str());
}

// The leading dimension of a matrix with unit column stride.
int64_t leading(const at::Tensor& t) {
    if (t.dim() != 2) refuse("operands must be 2-D");
    if (t.size(1) > 1 && t.stride(1) != 1)
        refuse("operands must have unit stride along rows (row-major)");
    if (t.size(0) <= 1) return std::max<int64_t>(1, t.size(1));
    if (t.stride(0) == 0 && t.size(1) > 0)
        refuse("rows that share memory (stride 0) are not supported; copy them with contiguous()");
    return std::max<int64_t>(1, t.stride(0));
}

const void* pointer(const at::Tensor& t) { return t.numel() ? t.const_data_ptr() : nullptr; }
// (of a tensor that may not be defined, too)
void* writable(const at::Tensor& t) {
    return t.defined() && t.numel() ? t.mutable_data_ptr() : nullptr;
}

void check_vector(const char* name, const at::Tensor& t, at::Device device, at::ScalarType kind,
                  int64_t size) {
    check_device(name, t, device);
    if (t.scalar_type() != kind || t.dim() != 1 || t.size(0) != size || !t.is_contiguous())
        refuse(name, " must be a contiguous ", name_of(kind), " vector of ", size, " (got ",
               name_of(t.scalar_type()), ", ", t.sizes(), ", strides ", t.strides(), ")");
}

// The code of a second type: like's own, or float32.
int second_code(const char* name, at::ScalarType kind, const at::Tensor& like) {
    const int code = code_of(like);
    if (kind == like.scalar_type()) return code;
    if (kind != at::kFloat)
        refuse(name, " must be ", name_of(like.scalar_type()), " or torch.float32 (got ",
               name_of(kind), ")");
    return MIGEMM_F32;
}

// The matrix a result is written to: `given`, checked, or a new one of like's dtype and device.
at::Tensor matrix(const char* name, const at::Tensor* given, const at::Tensor& like, int64_t rows,
                  int64_t cols, at::ScalarType kind) {
    if (!given) return at::empty({rows, cols}, like.options().dtype(kind));
    check_device(name, *given, like.device());
    if (given->scalar_type() != kind || given->dim() != 2 || given->size(0) != rows ||
        given->size(1) != cols)
        refuse(name, " must be ", name_of(kind), ", ", rows, " x ", cols);
    return *given;
}

at::Tensor workspace(int64_t bytes, const at::Tensor& like) {
    return bytes ? at::empty({bytes}, like.options().dtype(at::kByte)) : at::Tensor();
}

bool truth(PyObject* o) {
    const int b = PyObject_IsTrue(o);
    if (b < 0) throw PythonError{};
    return b != 0;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}
int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
void* stream_of(PyObject* o) {
    void* const p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return p;
}

PyObject* status(int st) { return PyLong_FromLong(st); }

// A tuple of tensors; one that is not defined becomes None.
PyObject* tuple(std::initializer_list<at::Tensor> list, bool with_last) {
    const Py_ssize_t n = static_cast<Py_ssize_t>(list.size()) - (with_last ? 0 : 1);
    PyObject* const out = PyTuple_New(n);
    if (!out) throw PythonError{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : list) {
        if (i == n) break;
        PyObject* item = Py_None;
        if (t.defined())
            item = THPVariable_Wrap(t);
        else
            Py_INCREF(item);
        if (!item) {
            Py_DECREF(out);
            throw PythonError{};
        }
        PyTuple_SET_ITEM(out, i++, item);
    }
    return out;
}

// x, weight, bias, eps, out, stats, stream, with workspace -> y, mean, rstd
PyObject* layer_norm(PyObject* const* a) {
    const at::Tensor& x = tensor("x", a[0]);
    const at::Tensor *const weight = optional("weight", a[1]), *const bias = optional("bias", a[2]);
    const at::Device device = x.device();
    check_device("x", x, device);
    const int64_t ldx = leading(x), T = x.size(0), D = x.size(1);
    const at::ScalarType kind = (weight ? *weight : bias ? *bias : x).scalar_type();
    const int wd = second_code("weight and bias", kind, x);
    if (weight) check_vector("weight", *weight, device, kind, D);
    if (bias) check_vector("bias", *bias, device, kind, D);
    const c10::DeviceGuard guard(device);
    const at::Tensor y = matrix("out", optional("out", a[4]), x, T, D, x.scalar_type());
    at::Tensor mean, rstd;
    if (truth(a[5])) {
        mean = at::empty({T}, x.options().dtype(at::kFloat));
        rstd = at::empty({T}, x.options().dtype(at::kFloat));
    }
    const int st = migemm_layer_norm_forward(
        T, D, code_of(x), pointer(x), ldx, wd, weight ? pointer(*weight) : nullptr,
        bias ? pointer(*bias) : nullptr, static_cast<float>(number(a[3])), writable(y), leading(y),
        static_cast<float*>(writable(mean)), static_cast<float*>(writable(rstd)), stream_of(a[6]));
    return st == MIGEMM_OK ? tuple({y, mean, rstd, {}}, false) : status(st);
}

// dy, x, weight, mean, rstd, dx, dw, db, need dx, need dw, need db, stream, with workspace
// -> dx, dw, db
PyObject* layer_norm_backward(PyObject* const* a) {
    const at::Tensor &dy = tensor("dy", a[0]), &x = tensor("x", a[1]);
    const at::Tensor* const weight = optional("weight", a[2]);
    const at::Tensor &mean = tensor("mean", a[3]), &rstd = tensor("rstd", a[4]);
    const at::Tensor *const dx_in = optional("dx", a[5]), *const dw_in = optional("dw", a[6]),
                     *const db_in = optional("db", a[7]);
    const at::Device device = x.device();
    check_device("x", x, device);
    check_device("dy", dy, device);
    const int64_t ldx = leading(x), lddy = leading(dy), T = x.size(0), D = x.size(1);
    if (dy.scalar_type() != x.scalar_type() || dy.sizes() != x.sizes())
        refuse("dy must have x's shape and dtype");
    const at::ScalarType kind = (weight ? *weight : x).scalar_type();
    const int wd = second_code("weight", kind, x);
    if (weight) check_vector("weight", *weight, device, kind, D);
    check_vector("mean", mean, device, at::kFloat, T);
    check_vector("rstd", rstd, device, at::kFloat, T);
    if (!weight && dw_in) refuse("dw needs a weight");
    const c10::DeviceGuard guard(device);
    at::Tensor dx, dw, db;
    if (dx_in || truth(a[8])) dx = matrix("dx", dx_in, x, T, D, x.scalar_type());
    auto vector = [&](const char* name, const at::Tensor* given, bool wanted) {
        if (given) check_vector(name, *given, device, kind, D);
        return given ? *given : wanted ? at::empty({D}, x.options().dtype(kind)) : at::Tensor();
    };
    dw = vector("dw", dw_in, weight && truth(a[9]));
    db = vector("db", db_in, truth(a[10]));
    int64_t bytes = 0;
    int st = migemm_layer_norm_workspace_size(T, D, dw.defined() || db.defined(), &bytes);
    if (st != MIGEMM_OK) return status(st);
    const at::Tensor ws = workspace(bytes, x);
    st = migemm_layer_norm_backward(
        T, D, code_of(x), pointer(dy), lddy, pointer(x), ldx, wd,
        weight ? pointer(*weight) : nullptr, static_cast<const float*>(pointer(mean)),
        static_cast<const float*>(pointer(rstd)), writable(dx), dx.defined() ? leading(dx) : D,
        writable(dw), writable(db), writable(ws), bytes, stream_of(a[11]));
    return st == MIGEMM_OK ? tuple({dx, dw, db, ws}, truth(a[12])) : status(st);
}

// w, index, scale, ignore_index, out, stream, with workspace -> y
PyObject* embedding(PyObject* const* a) {
    const at::Tensor &w = tensor("w", a[0]), &index = tensor("index", a[1]);
    check_device("w", w, w.device());
    const int64_t ldw = leading(w), T = index.numel(), V = w.size(0), D = w.size(1);
    check_vector("index", index, w.device(), at::kLong, T);
    const c10::DeviceGuard guard(w.device());
    const int dt = code_of(w);
    const at::Tensor y = matrix("out", optional("out", a[4]), w, T, D, w.scalar_type());
    const int st = migemm_embedding_forward(
        T, V, D, dt, pointer(w), ldw, static_cast<const int64_t*>(pointer(index)), whole(a[3]),
        static_cast<float>(number(a[2])), writable(y), leading(y), stream_of(a[5]));
    return st == MIGEMM_OK ? tuple({y, {}}, false) : status(st);
}

// dy, index, vocab, scale, ignore_index, dw, accumulate, out_dtype, stream, with workspace
// -> dw
PyObject* embedding_backward(PyObject* const* a) {
    const at::Tensor &dy = tensor("dy", a[0]), &index = tensor("index", a[1]);
    const at::Tensor* const given = optional("dw", a[5]);
    check_device("dy", dy, dy.device());
    const int64_t lddy = leading(dy), T = dy.size(0), D = dy.size(1), V = whole(a[2]);
    check_vector("index", index, dy.device(), at::kLong, T);
    const bool accumulate = truth(a[6]);
    if (accumulate && !given) refuse("accumulate needs an existing dw");
    at::ScalarType kind = (given ? *given : dy).scalar_type();
    if (a[7] != Py_None) {
        if (!THPDtype_Check(a[7])) refuse("out_dtype must be a torch dtype");
        const at::ScalarType wanted = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
        if (given && wanted != kind) refuse("dw must have out_dtype, if given");
        kind = wanted;
    }
    const int wd = second_code("dw", kind, dy);
    const c10::DeviceGuard guard(dy.device());
    int64_t bytes = 0;
    int st = migemm_embedding_workspace_size(T, V, D, &bytes);
    if (st != MIGEMM_OK) return status(st);
    const at::Tensor dw = matrix("dw", given, dy, V, D, kind);
    const at::Tensor ws = workspace(bytes, dy);
    st = migemm_embedding_backward(
        T, V, D, code_of(dy), pointer(dy), lddy, static_cast<const int64_t*>(pointer(index)),
        whole(a[4]), static_cast<float>(number(a[3])), accumulate, wd, writable(dw), leading(dw),
        writable(ws), bytes, stream_of(a[8]));
    return st == MIGEMM_OK ? tuple({dw, ws}, truth(a[9])) : status(st);
}

// The items of a list or tuple.
struct Items {
    PyObject* held;
    Py_ssize_t count;
    PyObject** at;
    Items(PyObject* o, const char* what) : held(PySequence_Fast(o, what)) {
        if (!held) throw PythonError{};
        count = PySequence_Fast_GET_SIZE(held);
        at = PySequence_Fast_ITEMS(held);
    }
    Items(const Items&) = delete;
    ~Items() { Py_DECREF(held); }
};

// One element on the GPU, and its address.
const void* number_on_device(const char* name, PyObject* o, at::Device device,
                             at::ScalarType kind) {
    const at::Tensor& t = tensor(name, o);
    check_device(name, t, device);
    if (t.scalar_type() != kind || t.numel() != 1)
        refuse(name, " must be a number or one ", name_of(kind), " on the GPU (got ",
               name_of(t.scalar_type()), ", ", t.sizes(), ")");
    return t.const_data_ptr();
}

// params, grads, states, step, lr, beta1, beta2, eps, weight_decay, grad_scale, stream,
// with workspace
PyObject* adamw(PyObject* const* a) {
    const Items params(a[0], "params must be a list"), grads(a[1], "grads must be a list"),
        states(a[2], "states must be a list");
    const Py_ssize_t n = params.count;
    if (grads.count != n || states.count != n)
        refuse(n, " parameters, ", grads.count, " gradients and ", states.count, " states");
    if (n == 0) return status(MIGEMM_OK);
    const at::Tensor &p0 = tensor("params", params.at[0]), &g0 = tensor("grads", grads.at[0]);
    const at::Device device = p0.device();
    check_device("params", p0, device);
    const at::ScalarType pd = p0.scalar_type(), gd = g0.scalar_type();
    const int pcode = code_of(p0), gcode = second_code("gradients", gd, p0);
    std::vector<migemm_adamw_tensor> list(static_cast<size_t>(n));
    at::ScalarType sd = at::kFloat;
    bool eight = false, master = false;
    auto take = [&](PyObject* o, at::ScalarType kind, int64_t size) {
        const at::Tensor& t = tensor("a tensor of the step", o);
        if (t.scalar_type() != kind || t.numel() != size || t.device() != device ||
            !t.is_contiguous())
            refuse("a tensor of the step must be contiguous, ", name_of(kind), ", of ", size,
                   " elements on ", device.str(), " (got ", name_of(t.scalar_type()), ", ",
                   t.numel(), " on ", t.device().str(), ", strides ", t.strides(), ")");
        return writable(t);
    };
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Items s(states.at[i], "a state must be an AdamState");
        if (s.count != 5) refuse("a state must be an AdamState");
        if (i == 0) {
            sd = tensor("avg", s.at[0]).scalar_type();
            eight = sd != at::kFloat;
            master = s.at[4] != Py_None;
            if (eight && sd != at::kFloat8_e4m3fn && sd != at::kByte)
                refuse("states must be float32, float8_e4m3fn or uint8 (got ", name_of(sd), ")");
            if (master && pd == at::kFloat) refuse("float32 parameters take no master copy");
        }
        if ((s.at[2] != Py_None) != eight || (s.at[3] != Py_None) != eight ||
            (s.at[4] != Py_None) != master)
            refuse("states must all be of 32 or all of 8 bits, with a master copy in all or in "
                   "none");
        const int64_t size = tensor("params", params.at[i]).numel(), blocks = (size + 255) / 256;
        migemm_adamw_tensor& t = list[static_cast<size_t>(i)];
        t.count = size;
        t.param = take(params.at[i], pd, size);
        t.grad = take(grads.at[i], gd, size);
        t.avg = take(s.at[0], sd, size);
        t.sq = take(s.at[1], sd, size);
        t.avg_scales = eight ? static_cast<float*>(take(s.at[2], at::kFloat, blocks)) : nullptr;
        t.sq_scales = eight ? static_cast<float*>(take(s.at[3], at::kFloat, blocks)) : nullptr;
        t.master = master ? static_cast<float*>(take(s.at[4], at::kFloat, size)) : nullptr;
    }
    migemm_adamw_options o{};
    if (THPVariable_Check(a[3]))
        o.step_device =
            static_cast<const int64_t*>(number_on_device("step", a[3], device, at::kLong));
    else
        o.step = whole(a[3]);
    if (THPVariable_Check(a[4]))
        o.lr_device = static_cast<const float*>(number_on_device("lr", a[4], device, at::kFloat));
    else
        o.lr = number(a[4]);
    o.beta1 = number(a[5]);
    o.beta2 = number(a[6]);
    o.eps = number(a[7]);
    o.weight_decay = number(a[8]);
    if (a[9] != Py_None)
        o.grad_scale =
            static_cast<const float*>(number_on_device("grad_scale", a[9], device, at::kFloat));
    const c10::DeviceGuard guard(device);
    return status(migemm_adamw(n, list.data(), pcode, gcode, eight ? 8 : 32, &o, stream_of(a[10])));
}

// Runs a function on `count` arguments; what it throws becomes a Python exception.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t COUNT>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t count) {
    if (count != COUNT) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", COUNT, count);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (const PythonError&) {
    } catch (...) {  // torch's own, its allocator's among them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t COUNT>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(call<F, COUNT>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<layer_norm, 8>("layer_norm"),
                         method<layer_norm_backward, 13>("layer_norm_backward"),
                         method<embedding, 7>("embedding"),
                         method<embedding_backward, 10>("embedding_backward"),
                         method<adamw, 12>("adamw"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
