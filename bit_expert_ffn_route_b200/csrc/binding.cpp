// binding.cpp — the Python side of include/moe_ops.h as an extension module
// (bit_expert_ffn_route_b200._ops): marshalling only, as in moe.py, in native code
// because these calls take 3 us in the library and are made once or more per layer
// and step.  Called back to back, one token's norm takes 3.4 us; it took 6.3 us with
// ctypes and the checks alone in native code, 8.8 us with both in Python.
//
// Every function takes torch tensors on one CUDA device, checks type, shape and
// contiguity (ValueError), makes that device current, and calls the library on
// `stream` or the device's current stream.  A status other than MOE_OK is raised as
// moe.MoeError.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <initializer_list>
#include <string>

#include "moe_ops.h"

namespace {

using at::ScalarType;
using Shape = std::initializer_list<int64_t>;

struct Raised {};                               // a Python error is set

[[noreturn]] void refuse(PyObject* type, const std::string& why) {
    PyErr_SetString(type, why.c_str());
    throw Raised();
}

constexpr int kMaxArgs = 20;

// A function's parameters in order; the first `required` have no default.
struct Signature {
    const char* name;
    int required, n;
    const char* params[kMaxArgs];
    PyObject* interned[kMaxArgs] = {};
};

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}
std::string type_text(ScalarType t) { return std::string("torch.") + torch::getTHPDtype(t)->name; }

class Call {
public:
    Call(Signature& sig, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) : sig_(sig) {
        if (nargs > sig.n) refuse(PyExc_TypeError, said() + "takes at most " + std::to_string(sig.n) + " arguments");
        for (Py_ssize_t i = 0; i < nargs; ++i) v_[i] = args[i];
        const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t j = 0; j < nkw; ++j) {
            const int i = index(PyTuple_GET_ITEM(kwnames, j));
            if (v_[i]) refuse(PyExc_TypeError, said() + "got two values for " + sig.params[i]);
            v_[i] = args[nargs + j];
        }
        for (int i = 0; i < sig.n; ++i) {
            if (!v_[i] && i < sig.required) refuse(PyExc_TypeError, said() + "needs " + sig.params[i]);
            if (!v_[i]) v_[i] = Py_None;
        }
    }
    bool given(int i) const { return v_[i] != Py_None; }
    const at::Tensor& tensor(int i) const {
        if (!THPVariable_Check(v_[i])) refuse(PyExc_ValueError, std::string(sig_.params[i]) + " must be a tensor");
        return THPVariable_Unpack(v_[i]);
    }
    // A dimension of a 2-dimensional tensor, as the library's int.
    int dim(int i, int d) const {
        const at::Tensor& t = tensor(i);
        if (t.dim() != 2) refuse(PyExc_ValueError, std::string(sig_.params[i]) + " must have two dimensions, not " + shape_text(t.sizes()));
        if (t.size(d) > INT_MAX) refuse(PyExc_ValueError, std::string(sig_.params[i]) + " is too large");
        return (int)t.size(d);
    }
    int dtype(int i) const {
        switch (tensor(i).scalar_type()) {
            case ScalarType::BFloat16: return MOE_BF16;
            case ScalarType::Half: return MOE_F16;
            case ScalarType::Float: return MOE_F32;
            default: refuse(PyExc_ValueError, std::string(sig_.params[i]) + " must be bfloat16, float16 or float32, not " +
                                                  type_text(tensor(i).scalar_type()));
        }
    }
    // The address of a contiguous tensor of this type and shape on the call's device; null for None.
    template <typename P = void>
    P* at(int i, ScalarType type, Shape shape) const {
        if (!given(i)) return nullptr;
        if (!THPVariable_Check(v_[i])) refuse(PyExc_ValueError, std::string(sig_.params[i]) + " must be a tensor or None");
        const at::Tensor& t = THPVariable_Unpack(v_[i]);
        if (t.scalar_type() != type || t.get_device() != device_ || t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous())
            refuse(PyExc_ValueError, std::string(sig_.params[i]) + " must be a contiguous " + type_text(type) + " tensor of shape " +
                                         shape_text(at::IntArrayRef(shape)) + " on device " + std::to_string(device_) + ", not " +
                                         type_text(t.scalar_type()) + " " + shape_text(t.sizes()) + " on " + t.device().str() +
                                         (t.is_contiguous() ? "" : ", strided"));
        return static_cast<P*>(t.data_ptr());
    }
    // A byte buffer of any shape.
    void* bytes(int i, size_t* n) const {
        const at::Tensor& t = tensor(i);
        *n = (size_t)t.numel();
        if (t.scalar_type() != ScalarType::Byte || t.get_device() != device_ || !t.is_contiguous())
            refuse(PyExc_ValueError, std::string(sig_.params[i]) + " must be a contiguous torch.uint8 tensor on device " + std::to_string(device_));
        return t.data_ptr();
    }
    int integer(int i) const {
        const long n = PyLong_AsLong(v_[i]);
        if (n == -1 && PyErr_Occurred()) throw Raised();
        if (n > INT_MAX || n < INT_MIN) refuse(PyExc_ValueError, std::string(sig_.params[i]) + " is out of range");
        return (int)n;
    }
    float real(int i, double otherwise) const {
        if (!given(i)) return (float)otherwise;
        const double x = PyFloat_AsDouble(v_[i]);
        if (x == -1.0 && PyErr_Occurred()) throw Raised();
        return (float)x;
    }
    int gate_mode(int i) const {
        if (!given(i)) return MOE_GATE_NONE;
        if (PyUnicode_Check(v_[i])) {
            if (PyUnicode_CompareWithASCIIString(v_[i], "channel") == 0) return MOE_GATE_CHANNEL;
            if (PyUnicode_CompareWithASCIIString(v_[i], "token") == 0) return MOE_GATE_TOKEN;
            if (PyUnicode_CompareWithASCIIString(v_[i], "none") == 0) return MOE_GATE_NONE;
        }
        refuse(PyExc_ValueError, std::string(sig_.params[i]) + " must be 'none', 'channel' or 'token'");
    }
    // The call's device is this tensor's.
    void on(int i) { device_ = (int)tensor(i).get_device(); }
    // fn(stream) on the device, with the last parameter's stream or the current one.
    template <typename Fn>
    PyObject* run(Fn&& fn) const {
        if (device_ < 0) refuse(PyExc_ValueError, said() + "takes CUDA tensors");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device_);
        cudaStream_t s;
        if (given(sig_.n - 1)) {
            PyObject* stream = v_[sig_.n - 1];
            if (number(stream, "device_index") != device_)
                refuse(PyExc_ValueError, said() + "the stream is not on the tensors' device " + std::to_string(device_));
            s = reinterpret_cast<cudaStream_t>((uintptr_t)number(stream, "cuda_stream"));
        } else {
            s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_).stream();
        }
        moe_status st;
        Py_BEGIN_ALLOW_THREADS;
        st = fn(reinterpret_cast<moe_stream_t>(s));
        Py_END_ALLOW_THREADS;
        if (st != MOE_OK) failed(st);
        Py_RETURN_NONE;
    }

private:
    std::string said() const { return std::string(sig_.name) + ": "; }
    int index(PyObject* name) const {
        for (int i = 0; i < sig_.n; ++i)
            if (sig_.interned[i] == name) return i;
        for (int i = 0; i < sig_.n; ++i)
            if (PyUnicode_Compare(sig_.interned[i], name) == 0) return i;
        PyErr_Format(PyExc_TypeError, "%s: no parameter %R", sig_.name, name);
        throw Raised();
    }
    static long long number(PyObject* o, const char* attr) {
        PyObject* v = PyObject_GetAttrString(o, attr);
        if (!v) throw Raised();
        const long long n = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (n == -1 && PyErr_Occurred()) throw Raised();
        return n;
    }
    [[noreturn]] void failed(moe_status st) const {
        PyObject* m = PyImport_ImportModule("bit_expert_ffn_route_b200.moe");
        PyObject* type = m ? PyObject_GetAttrString(m, "MoeError") : nullptr;
        PyObject* e = type ? PyObject_CallFunction(type, "si", sig_.name, (int)st) : nullptr;
        if (e) PyErr_SetObject(type, e);
        Py_XDECREF(e);
        Py_XDECREF(type);
        Py_XDECREF(m);
        throw Raised();
    }

    const Signature& sig_;
    PyObject* v_[kMaxArgs] = {};
    int device_ = -1;
};

constexpr ScalarType I32 = ScalarType::Int, F32 = ScalarType::Float, B16 = ScalarType::BFloat16;

// ---------------------------------------------------------------- the calls
Signature kPermute{"moe_permute", 5, 10, {"ids", "E", "offsets", "pair_row", "row_pair", "x", "rows", "slot_table", "n_slots", "stream"}};
PyObject* permute(Call& a) {
    const int T = a.dim(0, 0), k = a.dim(0, 1), E = a.integer(1);
    a.on(0);
    int D = 1, dtype = MOE_BF16;
    ScalarType type = B16;
    if (a.given(5)) {
        dtype = a.dtype(5);
        D = a.dim(5, 1);
        type = a.tensor(5).scalar_type();
    }
    if (a.given(5) != a.given(6)) refuse(PyExc_ValueError, "moe_permute: x and rows come together");
    if (a.given(7) && !a.given(8)) refuse(PyExc_ValueError, "moe_permute: slot_table comes with the pool's n_slots");
    const int n_slots = a.given(8) ? a.integer(8) : 0;
    auto *ids = a.at<int32_t>(0, I32, {T, k}), *table = a.at<int32_t>(7, I32, {E}), *offsets = a.at<int32_t>(2, I32, {(int64_t)E + 1});
    auto *pair_row = a.at<int32_t>(3, I32, {T, k}), *row_pair = a.at<int32_t>(4, I32, {(int64_t)T * k});
    void *x = a.at(5, type, {T, D}), *rows = a.at(6, type, {(int64_t)T * k, D});
    return a.run([&](moe_stream_t s) {
        return moe_permute(ids, T, k, E, table, n_slots, x, D, dtype, rows, offsets, pair_row, row_pair, s);
    });
}

Signature kPermuteBackward{"moe_permute_backward", 3, 4, {"drows", "pair_row", "dx", "stream"}};
PyObject* permute_backward(Call& a) {
    const int T = a.dim(1, 0), k = a.dim(1, 1), n = a.dim(0, 0), D = a.dim(0, 1), dtype = a.dtype(0);
    a.on(0);
    const ScalarType type = a.tensor(0).scalar_type();
    void *drows = a.at(0, type, {n, D}), *dx = a.at(2, type, {T, D});
    auto* pair_row = a.at<int32_t>(1, I32, {T, k});
    return a.run([&](moe_stream_t s) { return moe_permute_backward(drows, n, pair_row, T, k, D, dtype, dx, s); });
}

Signature kUnpermute{"moe_unpermute", 3, 5, {"rows", "pair_row", "out", "weights", "stream"}};
PyObject* unpermute(Call& a) {
    const int T = a.dim(1, 0), k = a.dim(1, 1), n = a.dim(0, 0), D = a.dim(0, 1), dtype = a.dtype(0), out_dtype = a.dtype(2);
    a.on(0);
    void *rows = a.at(0, a.tensor(0).scalar_type(), {n, D}), *out = a.at(2, a.tensor(2).scalar_type(), {T, D});
    auto* pair_row = a.at<int32_t>(1, I32, {T, k});
    auto* weights = a.at<float>(3, F32, {T, k});
    return a.run([&](moe_stream_t s) { return moe_unpermute(rows, n, pair_row, weights, T, k, D, dtype, out, out_dtype, s); });
}

Signature kUnpermuteBackward{"moe_unpermute_backward", 2, 7, {"dout", "pair_row", "drows", "rows", "weights", "dweights", "stream"}};
PyObject* unpermute_backward(Call& a) {
    if (!a.given(2) && !a.given(3))
        refuse(PyExc_ValueError, "moe_unpermute_backward writes drows, dweights (from rows), or both");
    const int like = a.given(2) ? 2 : 3, T = a.dim(1, 0), k = a.dim(1, 1), n = a.dim(like, 0), D = a.dim(like, 1);
    const int dtype = a.dtype(like), out_dtype = a.dtype(0);
    a.on(0);
    const ScalarType type = a.tensor(like).scalar_type();
    void *dout = a.at(0, a.tensor(0).scalar_type(), {T, D}), *drows = a.at(2, type, {n, D}), *rows = a.at(3, type, {n, D});
    auto* pair_row = a.at<int32_t>(1, I32, {T, k});
    auto *weights = a.at<float>(4, F32, {T, k}), *dweights = a.at<float>(5, F32, {T, k});
    return a.run([&](moe_stream_t s) {
        return moe_unpermute_backward(dout, out_dtype, rows, n, pair_row, weights, T, k, D, dtype, drows, dweights, s);
    });
}

Signature kRouteBackward{"moe_route_backward", 9, 14, {"dgates", "gates", "ids", "x", "Wr", "offsets", "row_pair", "dlogits", "ws", "dx", "dx_add", "dWr", "dbias", "stream"}};
PyObject* route_backward(Call& a) {
    const int T = a.dim(2, 0), k = a.dim(2, 1), E = a.dim(4, 0), D = a.dim(4, 1);
    a.on(2);
    size_t n;
    void* ws = a.bytes(8, &n);
    auto *dgates = a.at<float>(0, F32, {T, k}), *gates = a.at<float>(1, F32, {T, k}), *dlogits = a.at<float>(7, F32, {T, k});
    auto *ids = a.at<int32_t>(2, I32, {T, k}), *offsets = a.at<int32_t>(5, I32, {(int64_t)E + 1}), *row_pair = a.at<int32_t>(6, I32, {(int64_t)T * k});
    auto *x = a.at<uint16_t>(3, B16, {T, D}), *Wr = a.at<uint16_t>(4, B16, {E, D});
    auto *dx = a.at<uint16_t>(9, B16, {T, D}), *dx_add = a.at<uint16_t>(10, B16, {T, D});
    auto *dWr = a.at<float>(11, F32, {E, D}), *dbias = a.at<float>(12, F32, {E});
    return a.run([&](moe_stream_t s) {
        return moe_route_backward(dgates, gates, ids, x, Wr, offsets, row_pair, T, D, E, k, dx_add, dlogits, dx, dWr, dbias, ws, n, s);
    });
}

Signature kBlockNorm{"moe_block_norm", 1, 13, {"y", "x_out", "residual", "alpha", "gate", "gate_mode", "w_post", "w_next", "normed", "rstd_post", "rstd_next", "eps", "stream"}};
PyObject* block_norm(Call& a) {
    const int T = a.dim(0, 0), D = a.dim(0, 1), dtype = a.dtype(0), mode = a.gate_mode(5);
    a.on(0);
    const ScalarType type = a.tensor(0).scalar_type();
    const float alpha = a.real(3, 1.0), eps = a.real(11, 1e-6);
    void *y = a.at(0, type, {T, D}), *x_out = a.at(1, type, {T, D}), *residual = a.at(2, type, {T, D}), *normed = a.at(8, type, {T, D});
    auto *gate = a.at<float>(4, F32, {mode == MOE_GATE_TOKEN ? T : D}), *w_post = a.at<float>(6, F32, {D}), *w_next = a.at<float>(7, F32, {D});
    auto *rstd_post = a.at<float>(9, F32, {T}), *rstd_next = a.at<float>(10, F32, {T});
    return a.run([&](moe_stream_t s) {
        return moe_block_norm(y, residual, gate, mode, alpha, w_post, w_next, eps, T, D, dtype, x_out, normed, rstd_post, rstd_next, s);
    });
}

Signature kBlockNormBackward{"moe_block_norm_backward", 6, 18, {"dx_out", "dnormed", "x_out", "y", "dy", "ws", "dresidual", "alpha", "gate", "gate_mode", "dgate", "w_post", "dw_post", "rstd_post", "w_next", "dw_next", "rstd_next", "stream"}};
PyObject* block_norm_backward(Call& a) {
    const int T = a.dim(4, 0), D = a.dim(4, 1), dtype = a.dtype(4), mode = a.gate_mode(9);
    a.on(4);
    const ScalarType type = a.tensor(4).scalar_type();
    const float alpha = a.real(7, 1.0);
    const int64_t gates = mode == MOE_GATE_TOKEN ? T : D;
    size_t n;
    void* ws = a.bytes(5, &n);
    void *dx_out = a.at(0, type, {T, D}), *dnormed = a.at(1, type, {T, D}), *x_out = a.at(2, type, {T, D}), *y = a.at(3, type, {T, D});
    void *dy = a.at(4, type, {T, D}), *dresidual = a.at(6, type, {T, D});
    auto *gate = a.at<float>(8, F32, {gates}), *dgate = a.at<float>(10, F32, {gates});
    auto *w_post = a.at<float>(11, F32, {D}), *dw_post = a.at<float>(12, F32, {D}), *rstd_post = a.at<float>(13, F32, {T});
    auto *w_next = a.at<float>(14, F32, {D}), *dw_next = a.at<float>(15, F32, {D}), *rstd_next = a.at<float>(16, F32, {T});
    return a.run([&](moe_stream_t s) {
        return moe_block_norm_backward(dx_out, dnormed, x_out, y, gate, mode, alpha, w_post, rstd_post, w_next, rstd_next, T, D,
                                       dtype, dy, dresidual, dgate, dw_post, dw_next, ws, n, s);
    });
}

// No C++ exception passes into the interpreter.
template <Signature* SIG, PyObject* (*FN)(Call&)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    try {
        Call a(*SIG, args, nargs, kwnames);
        return FN(a);
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <Signature* SIG, PyObject* (*FN)(Call&)>
PyMethodDef method(const char* doc) {
    return {SIG->name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<SIG, FN>)), METH_FASTCALL | METH_KEYWORDS, doc};
}

PyMethodDef methods[] = {
    method<&kPermute, permute>(
        "moe_permute(ids, E, offsets, pair_row, row_pair, x=None, rows=None, slot_table=None, n_slots=None, stream=None)\n\n"
        "Tokens sorted by expert: rows[i] = x[row_pair[i] // k], grouped by expert (all pairs, or with slot_table the\n"
        "missed ones, given n_slots as well).  Without x and rows only the plan (offsets, pair_row, row_pair) is made."),
    method<&kPermuteBackward, permute_backward>(
        "moe_permute_backward(drows, pair_row, dx, stream=None)\n\ndx[t] = the sum of drows over token t's rows."),
    method<&kUnpermute, unpermute>(
        "moe_unpermute(rows, pair_row, out, weights=None, stream=None)\n\n"
        "out[t] = the sum of weights[t, r] * rows[pair_row[t, r]]; out of rows' type or float32 (a miss_partial)."),
    method<&kUnpermuteBackward, unpermute_backward>(
        "moe_unpermute_backward(dout, pair_row, drows=None, rows=None, weights=None, dweights=None, stream=None)\n\n"
        "drows[pair_row[t, r]] = weights[t, r] * dout[t] and dweights[t, r] = <dout[t], rows[pair_row[t, r]]>."),
    method<&kRouteBackward, route_backward>(
        "moe_route_backward(dgates, gates, ids, x, Wr, offsets, row_pair, dlogits, ws, dx=None, dx_add=None, dWr=None,\n"
        "                   dbias=None, stream=None)\n\n"
        "Gradient of moe_route_topk's gates; offsets and row_pair are moe_permute's of the same ids (no slot_table)."),
    method<&kBlockNorm, block_norm>(
        "moe_block_norm(y, x_out=None, residual=None, alpha=1.0, gate=None, gate_mode=None, w_post=None, w_next=None,\n"
        "               normed=None, rstd_post=None, rstd_next=None, eps=1e-6, stream=None)\n\n"
        "x_out = alpha * residual + gate * norm(y) * w_post (y itself without w_post); normed = norm(x_out) * w_next.\n"
        "gate_mode: 'channel' (gate [D]) or 'token' (gate [T])."),
    method<&kBlockNormBackward, block_norm_backward>(
        "moe_block_norm_backward(dx_out, dnormed, x_out, y, dy, ws, dresidual=None, alpha=1.0, gate=None, gate_mode=None,\n"
        "                        dgate=None, w_post=None, dw_post=None, rstd_post=None, w_next=None, dw_next=None,\n"
        "                        rstd_next=None, stream=None)\n\n"
        "Gradients of moe_block_norm; the arguments left None there stay None here, as do gradients not wanted."),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", "The calls of moe_ops.h on torch tensors.", -1, methods};

}  // namespace

// The module reads tensors through functions that the compiler put into it, and its own objects lie as this
// Python's headers say: with another torch or Python it refuses to load.  Only calls of Python's stable ABI here.
static bool built_for_this_process() {
    const std::string python = std::to_string(PY_MAJOR_VERSION) + "." + std::to_string(PY_MINOR_VERSION) + ".";
    if (std::string(Py_GetVersion()).compare(0, python.size(), python) != 0) {
        PyErr_Format(PyExc_ImportError, "_ops.so was built for Python %s, not %s", PY_VERSION, Py_GetVersion());
        return false;
    }
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
    PyObject* text = version ? PyObject_Str(version) : nullptr;
    const int differs = text ? PyUnicode_CompareWithASCIIString(text, MOE_TORCH_VERSION) : 1;
    if (text && differs) PyErr_Format(PyExc_ImportError, "_ops.so was built for torch %s, not %U", MOE_TORCH_VERSION, text);
    Py_XDECREF(text);
    Py_XDECREF(version);
    Py_XDECREF(torch);
    return !differs;
}

PyMODINIT_FUNC PyInit__ops() {
    if (!built_for_this_process()) return nullptr;
    for (Signature* s : {&kPermute, &kPermuteBackward, &kUnpermute, &kUnpermuteBackward, &kRouteBackward, &kBlockNorm, &kBlockNormBackward})
        for (int i = 0; i < s->n; ++i)
            if (!(s->interned[i] = PyUnicode_InternFromString(s->params[i]))) return nullptr;
    return PyModule_Create(&module);
}
