// The layer operators on torch tensors, as a CPython extension over the C ABI
// of sgemm_gb300_layers.h and sgemm_gb300_block.h: checks the tensors, reads their pointers and
// strides, allocates outputs and scratch memory with torch's allocator on the
// current stream, and calls the entry point through an address that the
// package hands over from the library it loaded (bind).  A decoding step makes
// several of these calls for each of its short kernels; the same steps in
// Python took 12 to 20 us a call, these take 3 to 5, the launch included.
// Nothing here computes.  layers.py documents the calls.
#include <cstdint>
#include <stdexcept>
#include <string>
#include <vector>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sgemm_gb300_block.h"
#include "sgemm_gb300_layers.h"

namespace {

decltype(&sgemm_linear) f_linear;
decltype(&sgemm_linear_workspace_size) f_linear_ws;
decltype(&sgemm_linear_backward) f_linear_backward;
decltype(&sgemm_linear_backward_workspace_size) f_linear_backward_ws;
decltype(&sgemm_add_rmsnorm) f_add_rmsnorm;
decltype(&sgemm_add_rmsnorm_backward) f_add_rmsnorm_backward;
decltype(&sgemm_add_rmsnorm_backward_workspace_size) f_add_rmsnorm_backward_ws;
decltype(&sgemm_quantize_rows) f_quantize_rows;
decltype(&sgemm_gated_linear) f_gated_linear;
decltype(&sgemm_gated_linear_workspace_size) f_gated_linear_ws;
decltype(&sgemm_gated_linear_backward) f_gated_linear_backward;
decltype(&sgemm_gated_linear_backward_workspace_size) f_gated_linear_backward_ws;
decltype(&sgemm_add_layernorm) f_add_layernorm;
decltype(&sgemm_add_layernorm_backward) f_add_layernorm_backward;
decltype(&sgemm_add_layernorm_backward_workspace_size) f_add_layernorm_backward_ws;
decltype(&sgemm_clip_grad_norm) f_clip_grad_norm;
decltype(&sgemm_clip_grad_norm_workspace_size) f_clip_grad_norm_ws;
PyObject *py_raise;   // called with a nonzero status; raises
PyObject *py_out_of_memory;   // torch.OutOfMemoryError

// An exception of the C++ side that names the Python type to raise.
struct Refusal {
    PyObject *type;
    std::string what;
};
[[noreturn]] void type_error(const std::string &s) { throw Refusal{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string &s) { throw Refusal{PyExc_ValueError, s}; }
struct Raised {};   // a Python error is set

void check_status(int st) {
    if (st == SGEMM_OK) return;
    PyObject *r = PyObject_CallFunction(py_raise, "i", st);
    Py_XDECREF(r);
    throw Raised{};
}

using at::ScalarType;

int type_code(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return SGEMM_F32;
        case ScalarType::BFloat16: return SGEMM_BF16;
        case ScalarType::Half: return SGEMM_F16;
        case ScalarType::Float8_e4m3fn: return SGEMM_E4M3;
        default: return -1;
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

bool present(PyObject *o) { return o != nullptr && o != Py_None; }

int operand_type(const at::Tensor &t, const char *name, bool e4m3) {
    const int c = type_code(t.scalar_type());
    if (c < 0 || (c == SGEMM_E4M3 && !e4m3))
        type_error(std::string(name) + " has an unsupported type " + c10::toString(t.scalar_type()));
    return c;
}

// The device of a call's first tensor made current for the call, if another one is
// (a guard for every call, which asks three times which one is, took 0.2 us).
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    explicit OnDevice(c10::Device d) {
        if (c10::cuda::current_device() != d.index()) guard.set_device(d);
    }
};

// Every tensor of a call is on the device of its first one, `like`.
void same_device(const at::Tensor &t, const at::Tensor &like, const char *name) {
    if (t.device() != like.device())
        value_error(std::string(name) + " is on " + t.device().str() + ", the call's first tensor on " +
                    like.device().str());
}

// Pointer and leading dimension of a 2-D CUDA tensor with contiguous rows.
struct Mat {
    void *p = nullptr;
    int64_t ld = 0;
};
Mat matrix(const at::Tensor &t, const char *name, const at::Tensor &like, ScalarType type,
           int64_t rows = -1, int64_t cols = -1) {
    if (!t.is_cuda() || t.dim() != 2 || t.scalar_type() != type)
        type_error(std::string(name) + " must be a 2-D CUDA tensor of " + c10::toString(type));
    same_device(t, like, name);
    const int64_t r = t.size(0), c = t.size(1);
    if (rows >= 0 && (r != rows || c != cols))
        value_error(std::string(name) + " has shape (" + std::to_string(r) + ", " +
                    std::to_string(c) + "), expected (" + std::to_string(rows) + ", " +
                    std::to_string(cols) + ")");
    const int64_t sr = t.stride(0), sc = t.stride(1);
    if ((c > 1 && sc != 1) || (r > 1 && sr < c))
        value_error(std::string(name) + " must have contiguous rows that do not overlap");
    const int64_t ld = r > 1 ? sr : c;
    return {t.data_ptr(), ld > 1 ? ld : 1};
}
Mat optional_matrix(PyObject *o, const char *name, const at::Tensor &like, ScalarType type,
                    int64_t rows, int64_t cols) {
    return present(o) ? matrix(tensor(o, name), name, like, type, rows, cols) : Mat{};
}

// Pointer of a contiguous vector of n elements.
void *vector(PyObject *o, const char *name, const at::Tensor &like, ScalarType type, int64_t n) {
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda() || t.scalar_type() != type || t.dim() != 1 || t.size(0) != n ||
        (n > 1 && t.stride(0) != 1))
        value_error(std::string(name) + " must be a contiguous " + c10::toString(type) +
                    " CUDA tensor of " + std::to_string(n) + " elements");
    same_device(t, like, name);
    return t.data_ptr();
}
void *optional_vector(PyObject *o, const char *name, const at::Tensor &like, ScalarType type,
                      int64_t n) {
    return present(o) ? vector(o, name, like, type, n) : nullptr;
}

// An (N, K) weight stored by rows (trans 1) or as the transposed view of a
// K x N matrix (trans 0).
struct Weight {
    void *p;
    int64_t n, ld;
    int trans;
};
Weight weight(const at::Tensor &w, const at::Tensor &like, int64_t k, ScalarType type) {
    if (!w.is_cuda() || w.dim() != 2 || w.scalar_type() != type)
        type_error(std::string("weight must be a 2-D CUDA tensor of ") + c10::toString(type));
    same_device(w, like, "weight");
    const int64_t n = w.size(0), sr = w.stride(0), sc = w.stride(1);
    if (w.size(1) != k)
        value_error("weight has " + std::to_string(w.size(1)) + " input features, expected " +
                    std::to_string(k));
    const int64_t one = 1;
    if ((sc == 1 || k <= 1) && (n <= 1 || sr >= k))
        return {w.data_ptr(), n, std::max(n > 1 ? sr : k, one), 1};
    if ((sr == 1 || n <= 1) && (k <= 1 || sc >= n))
        return {w.data_ptr(), n, std::max(k > 1 ? sc : n, one), 0};
    value_error("weight must have one unit stride");
}

// The gated layer's two weights, both stored by rows (trans 1) or both as transposed views.
struct WeightPair {
    void *g, *u;
    int64_t n, ldg, ldu;
    int trans;
};
WeightPair weight_pair(const at::Tensor &g, const at::Tensor &u, const at::Tensor &like, int64_t k,
                       ScalarType type) {
    for (const at::Tensor *w : {&g, &u}) {
        const char *name = w == &g ? "w_gate" : "w_up";
        if (!w->is_cuda() || w->dim() != 2 || w->scalar_type() != type)
            type_error(std::string(name) + " must be a 2-D CUDA tensor of " + c10::toString(type));
        same_device(*w, like, name);
        if (w->size(1) != k)
            value_error(std::string(name) + " has " + std::to_string(w->size(1)) +
                        " input features, expected " + std::to_string(k));
    }
    const int64_t n = g.size(0);
    if (u.size(0) != n)
        value_error("w_gate has " + std::to_string(n) + " output features, w_up " +
                    std::to_string(u.size(0)));
    // the leading dimension where w is stored in that order, else 0
    auto ld = [&](const at::Tensor &w, int trans) -> int64_t {
        const int64_t rows = trans ? n : k, cols = trans ? k : n;
        const int64_t sr = w.stride(trans ? 0 : 1), sc = w.stride(trans ? 1 : 0);
        if ((cols > 1 && sc != 1) || (rows > 1 && sr < cols)) return 0;
        return std::max<int64_t>(rows > 1 ? sr : cols, 1);
    };
    for (int trans : {1, 0})
        if (ld(g, trans) > 0 && ld(u, trans) > 0)
            return {g.data_ptr(), u.data_ptr(), n, ld(g, trans), ld(u, trans), trans};
    value_error("w_gate and w_up must each have one unit stride, both the same one");
}

// torch's CUDA allocation without its dispatcher (at::empty takes about twice
// as long).
at::Tensor fresh(const at::Tensor &like, at::IntArrayRef size, ScalarType type) {
    return at::detail::empty_cuda(size, type, like.device(), c10::nullopt);
}

// Contiguous tensor of `size` from element `offset` of a fresh one on: outputs of a few values each
// share one allocation (an allocation takes 0.6 us, this 0.2).
at::Tensor part(const at::Tensor &of, int64_t offset, at::IntArrayRef size) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(),
                                                            of.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(offset);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(size);
    return t;
}

// Scratch memory: the caller's where it is large enough, else torch's.
struct Scratch {
    at::Tensor own;
    void *p = nullptr;
    uint64_t bytes = 0;
    Scratch(PyObject *given, uint64_t need, const at::Tensor &like) {
        if (need == 0) return;
        if (present(given)) {
            const at::Tensor &t = tensor(given, "workspace");
            if (!t.is_cuda() || t.scalar_type() != ScalarType::Byte || !t.is_contiguous())
                type_error("workspace must be a contiguous uint8 CUDA tensor");
            same_device(t, like, "workspace");
            if ((uint64_t)t.numel() >= need && reinterpret_cast<uintptr_t>(t.data_ptr()) % 256 == 0) {
                p = t.data_ptr();
                bytes = (uint64_t)t.numel();
                return;
            }
        }
        own = fresh(like, {(int64_t)need}, ScalarType::Byte);
        p = own.data_ptr();
        bytes = need;
    }
};

void *current_stream(const at::Tensor &t) {
    return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}

PyObject *none() {
    Py_INCREF(Py_None);
    return Py_None;
}

bool flag(PyObject *o) {
    if (o == Py_True || o == Py_False) return o == Py_True;
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};   // an object without a truth value
    return v == 1;
}

// Runs `body`, turning C++ exceptions into Python ones.
template <class F>
PyObject *guarded(F body) {
    try {
        at::AutoDispatchBelowADInplaceOrView no_autograd;
        if (py_raise == nullptr) throw Refusal{PyExc_RuntimeError, "bind() has not been called"};
        return body();
    } catch (const Refusal &r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const Raised &) {
    } catch (const c10::OutOfMemoryError &e) {   // the type that torch's own calls raise
        PyErr_SetString(py_out_of_memory, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

bool arity(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return false;
}

// x, weight, bias, activation (int), residual, x_scale, w_scale, half
// (whether an e4m3 product gives float16), save_preact, out, workspace
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const int type = operand_type(x, "x", true);
        const Mat X = matrix(x, "x", x, x.scalar_type());
        const OnDevice device(x.device());
        const int64_t m = x.size(0), k = x.size(1);
        const Weight W = weight(tensor(a[1], "weight"), x, k, x.scalar_type());
        ScalarType out_type = x.scalar_type();
        if (type == SGEMM_E4M3) {
            out_type = flag(a[7]) ? ScalarType::Half : ScalarType::BFloat16;
            if (!present(a[5]) || !present(a[6]))
                value_error("float8_e4m3fn operands need x_scale and w_scale");
            if (!W.trans) value_error("a float8_e4m3fn weight must be stored by rows");
        } else if (present(a[5]) || present(a[6])) {
            value_error("scales go with float8_e4m3fn operands only");
        }
        const int act = (int)PyLong_AsLong(a[3]);
        at::Tensor y, z;
        Mat Y, Z;
        if (present(a[9])) {
            Y = matrix(tensor(a[9], "out"), "out", x, out_type, m, W.n);
        } else {
            y = fresh(x, {m, W.n}, out_type);
            Y = {y.data_ptr(), std::max<int64_t>(W.n, 1)};
        }
        const bool save = flag(a[8]);
        if (save) {
            z = fresh(x, {m, W.n}, out_type);
            Z = {z.data_ptr(), std::max<int64_t>(W.n, 1)};
        }
        const Mat R = optional_matrix(a[4], "residual", x, out_type, m, W.n);
        void *xs = optional_vector(a[5], "x_scale", x, ScalarType::Float, m);
        void *ws = optional_vector(a[6], "w_scale", x, ScalarType::Float, W.n);
        void *bias = optional_vector(a[2], "bias", x, out_type, W.n);
        const Scratch s(a[10], f_linear_ws(type, m, W.n, k, X.p, X.ld, W.p, W.ld, W.trans), x);
        check_status(f_linear(type, m, W.n, k, X.p, X.ld, (const float *)xs, W.p, W.ld, W.trans,
                              (const float *)ws, bias, act, R.p, R.ld, type_code(out_type), Y.p,
                              Y.ld, Z.p, Z.ld, s.p, s.bytes, current_stream(x)));
        PyObject *py;
        if (present(a[9])) {
            // written in place: autograd then sees that what it saved has changed
            const at::Tensor &out = tensor(a[9], "out");
            if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
            py = a[9];
            Py_INCREF(py);
        } else {
            py = THPVariable_Wrap(std::move(y));
        }
        return save ? Py_BuildValue("(NN)", py, THPVariable_Wrap(std::move(z))) : py;
    });
}

// dy, x, weight, preact, activation (int), need_dx, need_dw, need_db, workspace
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 9)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x");
        const ScalarType t = dy.scalar_type();
        const int type = operand_type(dy, "dy", false);
        const Mat G = matrix(dy, "dy", dy, t), X = matrix(x, "x", dy, t);
        const OnDevice device(dy.device());
        const int64_t m = dy.size(0), n = dy.size(1), k = x.size(1);
        if (x.size(0) != m)
            value_error("x has " + std::to_string(x.size(0)) + " rows, dy " + std::to_string(m));
        const Weight W = weight(tensor(a[2], "weight"), dy, k, t);
        if (W.n != n)
            value_error("weight has " + std::to_string(W.n) + " output features, dy " +
                        std::to_string(n));
        const int act = (int)PyLong_AsLong(a[4]);
        if (act != SGEMM_ACT_NONE && !present(a[3]))
            value_error("this activation's gradient needs preact");
        const Mat Z =
            act != SGEMM_ACT_NONE ? optional_matrix(a[3], "preact", dy, t, m, n) : Mat{};
        at::Tensor dx, dw, db;
        if (flag(a[5])) dx = fresh(dy, {m, k}, t);
        if (flag(a[6])) dw = W.trans ? fresh(dy, {n, k}, t) : fresh(dy, {k, n}, t);
        if (flag(a[7])) db = fresh(dy, {n}, t);
        auto ptr = [](const at::Tensor &v) { return v.defined() ? v.data_ptr() : nullptr; };
        const Scratch s(a[8], f_linear_backward_ws(type, m, n, k, G.p, G.ld, act, X.p, X.ld, W.p,
                                                   W.ld, W.trans), dy);
        check_status(f_linear_backward(type, m, n, k, G.p, G.ld, Z.p, Z.ld, act, X.p, X.ld, W.p,
                                       W.ld, W.trans, ptr(dx), std::max<int64_t>(k, 1), ptr(dw),
                                       std::max<int64_t>(W.trans ? k : n, 1), ptr(db), s.p, s.bytes,
                                       current_stream(dy)));
        if (dw.defined() && !W.trans) dw = dw.t();
        auto wrap = [](at::Tensor &v) {
            return v.defined() ? THPVariable_Wrap(std::move(v)) : none();
        };
        return Py_BuildValue("(NNN)", wrap(dx), wrap(dw), wrap(db));
    });
}

// x, weight, residual, eps, quantize
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 5)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const ScalarType t = x.scalar_type();
        const int type = operand_type(x, "x", false);
        const Mat X = matrix(x, "x", x, t);
        const OnDevice device(x.device());
        const int64_t rows = x.size(0), d = x.size(1), ld = std::max<int64_t>(d, 1);
        void *w = vector(a[1], "weight", x, t, d);
        const Mat R = optional_matrix(a[2], "residual", x, t, rows, d);
        const double eps = PyFloat_AsDouble(a[3]);
        if (PyErr_Occurred()) throw Raised{};
        const bool quantize = flag(a[4]);
        at::Tensor s, scale;
        if (R.p != nullptr || present(a[2])) s = fresh(x, {rows, d}, t);
        at::Tensor y = fresh(x, {rows, d}, quantize ? ScalarType::Float8_e4m3fn : t);
        at::Tensor rstd = fresh(x, {rows}, ScalarType::Float);
        if (quantize) scale = fresh(x, {rows}, ScalarType::Float);
        check_status(f_add_rmsnorm(type, rows, d, X.p, X.ld, R.p, R.ld, w, (float)eps,
                                   s.defined() ? s.data_ptr() : nullptr, ld, y.data_ptr(), ld,
                                   quantize ? (float *)scale.data_ptr() : nullptr,
                                   (float *)rstd.data_ptr(), current_stream(x)));
        PyObject *ps;
        if (s.defined()) {
            ps = THPVariable_Wrap(std::move(s));
        } else {
            ps = a[0];
            Py_INCREF(ps);
        }
        PyObject *py = THPVariable_Wrap(std::move(y)), *pr = THPVariable_Wrap(std::move(rstd));
        if (quantize)
            return Py_BuildValue("(NNNN)", py, THPVariable_Wrap(std::move(scale)), ps, pr);
        return Py_BuildValue("(NNN)", py, ps, pr);
    });
}

// dy, s, rstd, weight, ds, need_dweight, workspace
PyObject *add_rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 7)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dy = tensor(a[0], "dy");
        const ScalarType t = dy.scalar_type();
        const int type = operand_type(dy, "dy", false);
        const Mat G = matrix(dy, "dy", dy, t);
        const OnDevice device(dy.device());
        const int64_t rows = dy.size(0), d = dy.size(1);
        const Mat S = matrix(tensor(a[1], "s"), "s", dy, t, rows, d);
        const Mat D = optional_matrix(a[4], "ds", dy, t, rows, d);
        void *rstd = vector(a[2], "rstd", dy, ScalarType::Float, rows);
        void *w = vector(a[3], "weight", dy, t, d);
        const bool need = flag(a[5]);
        at::Tensor dx = fresh(dy, {rows, d}, t), dw;
        if (need) dw = fresh(dy, {d}, t);
        const Scratch s(a[6], need ? f_add_rmsnorm_backward_ws(type, rows, d) : 0, dy);
        check_status(f_add_rmsnorm_backward(type, rows, d, G.p, G.ld, S.p, S.ld, (const float *)rstd,
                                            w, D.p, D.ld, dx.data_ptr(), std::max<int64_t>(d, 1),
                                            need ? dw.data_ptr() : nullptr, s.p, s.bytes,
                                            current_stream(dy)));
        return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(dx)),
                             need ? THPVariable_Wrap(std::move(dw)) : none());
    });
}

// x
PyObject *quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 1)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const int type = operand_type(x, "x", false);
        const Mat X = matrix(x, "x", x, x.scalar_type());
        const OnDevice device(x.device());
        const int64_t rows = x.size(0), d = x.size(1);
        at::Tensor q = fresh(x, {rows, d}, ScalarType::Float8_e4m3fn);
        at::Tensor scale = fresh(x, {rows}, ScalarType::Float);
        check_status(f_quantize_rows(type, rows, d, X.p, X.ld, q.data_ptr(),
                                     std::max<int64_t>(d, 1), (float *)scale.data_ptr(),
                                     current_stream(x)));
        return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(q)),
                             THPVariable_Wrap(std::move(scale)));
    });
}

// x, w_gate, w_up, b_gate, b_up, activation (int), x_scale, gate_scale, up_scale, half (whether
// an e4m3 product gives float16), save_preact, out, workspace
PyObject *gated_linear(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 13)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const int type = operand_type(x, "x", true);
        const Mat X = matrix(x, "x", x, x.scalar_type());
        const OnDevice device(x.device());
        const int64_t m = x.size(0), k = x.size(1);
        const WeightPair W = weight_pair(tensor(a[1], "w_gate"), tensor(a[2], "w_up"), x, k,
                                         x.scalar_type());
        const int64_t n = W.n;
        ScalarType out_type = x.scalar_type();
        if (type == SGEMM_E4M3) {
            out_type = flag(a[9]) ? ScalarType::Half : ScalarType::BFloat16;
            if (!present(a[6]) || !present(a[7]) || !present(a[8]))
                value_error("float8_e4m3fn operands need x_scale, gate_scale and up_scale");
            if (!W.trans) value_error("float8_e4m3fn weights must be stored by rows");
        } else if (present(a[6]) || present(a[7]) || present(a[8])) {
            value_error("scales go with float8_e4m3fn operands only");
        }
        const int act = (int)PyLong_AsLong(a[5]);
        const int64_t ld = std::max<int64_t>(n, 1);
        at::Tensor h, zg, zu;
        Mat H, Zg, Zu;
        if (present(a[11])) {
            H = matrix(tensor(a[11], "out"), "out", x, out_type, m, n);
        } else {
            h = fresh(x, {m, n}, out_type);
            H = {h.data_ptr(), ld};
        }
        const bool save = flag(a[10]);
        if (save) {
            zg = fresh(x, {m, n}, out_type);
            zu = fresh(x, {m, n}, out_type);
            Zg = {zg.data_ptr(), ld};
            Zu = {zu.data_ptr(), ld};
        }
        void *xs = optional_vector(a[6], "x_scale", x, ScalarType::Float, m);
        void *gs = optional_vector(a[7], "gate_scale", x, ScalarType::Float, n);
        void *us = optional_vector(a[8], "up_scale", x, ScalarType::Float, n);
        void *bg = optional_vector(a[3], "b_gate", x, out_type, n);
        void *bu = optional_vector(a[4], "b_up", x, out_type, n);
        const Scratch s(a[12], f_gated_linear_ws(type, m, n, k, X.p, X.ld, W.g, W.ldg, W.u, W.ldu,
                                                 W.trans), x);
        check_status(f_gated_linear(type, m, n, k, X.p, X.ld, (const float *)xs, W.g, W.ldg,
                                    (const float *)gs, W.u, W.ldu, (const float *)us, W.trans, bg,
                                    bu, act, type_code(out_type), H.p, H.ld, Zg.p, Zg.ld, Zu.p,
                                    Zu.ld, s.p, s.bytes, current_stream(x)));
        PyObject *ph;
        if (present(a[11])) {
            // written in place: autograd then sees that what it saved has changed
            const at::Tensor &out = tensor(a[11], "out");
            if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
            ph = a[11];
            Py_INCREF(ph);
        } else {
            ph = THPVariable_Wrap(std::move(h));
        }
        return save ? Py_BuildValue("(NNN)", ph, THPVariable_Wrap(std::move(zg)),
                                    THPVariable_Wrap(std::move(zu)))
                    : ph;
    });
}

// dh, x, w_gate, w_up, z_gate, z_up, activation (int), need_dx, need_dw, need_db, workspace
PyObject *gated_linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dh = tensor(a[0], "dh"), &x = tensor(a[1], "x");
        const ScalarType t = dh.scalar_type();
        const int type = operand_type(dh, "dh", false);
        const Mat G = matrix(dh, "dh", dh, t), X = matrix(x, "x", dh, t);
        const OnDevice device(dh.device());
        const int64_t m = dh.size(0), n = dh.size(1), k = x.size(1);
        if (x.size(0) != m)
            value_error("x has " + std::to_string(x.size(0)) + " rows, dh " + std::to_string(m));
        const WeightPair W = weight_pair(tensor(a[2], "w_gate"), tensor(a[3], "w_up"), dh, k, t);
        if (W.n != n)
            value_error("the weights have " + std::to_string(W.n) + " output features, dh " +
                        std::to_string(n));
        const Mat Zg = matrix(tensor(a[4], "z_gate"), "z_gate", dh, t, m, n);
        const Mat Zu = matrix(tensor(a[5], "z_up"), "z_up", dh, t, m, n);
        const int act = (int)PyLong_AsLong(a[6]);
        at::Tensor dx, dg, du, bg, bu;
        auto like_weight = [&] { return W.trans ? fresh(dh, {n, k}, t) : fresh(dh, {k, n}, t); };
        if (flag(a[7])) dx = fresh(dh, {m, k}, t);
        if (flag(a[8])) {
            dg = like_weight();
            du = like_weight();
        }
        if (flag(a[9])) {
            const at::Tensor both = fresh(dh, {2 * n}, t);
            bg = part(both, 0, {n});
            bu = part(both, n, {n});
        }
        auto ptr = [](const at::Tensor &v) { return v.defined() ? v.data_ptr() : nullptr; };
        const int64_t ldw = std::max<int64_t>(W.trans ? k : n, 1);
        const Scratch s(a[10], f_gated_linear_backward_ws(type, m, n, k, X.p, X.ld, W.g, W.ldg, W.u,
                                                          W.ldu, W.trans), dh);
        check_status(f_gated_linear_backward(
            type, m, n, k, G.p, G.ld, Zg.p, Zg.ld, Zu.p, Zu.ld, act, X.p, X.ld, W.g, W.ldg, W.u,
            W.ldu, W.trans, ptr(dx), std::max<int64_t>(k, 1), ptr(dg), ldw, ptr(du), ldw, ptr(bg),
            ptr(bu), s.p, s.bytes, current_stream(dh)));
        if (dg.defined() && !W.trans) {
            dg = dg.t();
            du = du.t();
        }
        auto wrap = [](at::Tensor &v) {
            return v.defined() ? THPVariable_Wrap(std::move(v)) : none();
        };
        return Py_BuildValue("(NNNNN)", wrap(dx), wrap(dg), wrap(du), wrap(bg), wrap(bu));
    });
}

// x, weight, bias, residual, eps, quantize
PyObject *add_layernorm(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 6)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const ScalarType t = x.scalar_type();
        const int type = operand_type(x, "x", false);
        const Mat X = matrix(x, "x", x, t);
        const OnDevice device(x.device());
        const int64_t rows = x.size(0), d = x.size(1), ld = std::max<int64_t>(d, 1);
        void *w = vector(a[1], "weight", x, t, d);
        void *b = optional_vector(a[2], "bias", x, t, d);
        const Mat R = optional_matrix(a[3], "residual", x, t, rows, d);
        const double eps = PyFloat_AsDouble(a[4]);
        if (PyErr_Occurred()) throw Raised{};
        const bool quantize = flag(a[5]);
        at::Tensor s, scale;
        if (present(a[3])) s = fresh(x, {rows, d}, t);
        at::Tensor y = fresh(x, {rows, d}, quantize ? ScalarType::Float8_e4m3fn : t);
        const at::Tensor few = fresh(x, {(quantize ? 3 : 2) * rows}, ScalarType::Float);
        at::Tensor mean = part(few, 0, {rows}), rstd = part(few, rows, {rows});
        if (quantize) scale = part(few, 2 * rows, {rows});
        check_status(f_add_layernorm(type, rows, d, X.p, X.ld, R.p, R.ld, w, b, (float)eps,
                                     s.defined() ? s.data_ptr() : nullptr, ld, y.data_ptr(), ld,
                                     quantize ? (float *)scale.data_ptr() : nullptr,
                                     (float *)mean.data_ptr(), (float *)rstd.data_ptr(),
                                     current_stream(x)));
        PyObject *ps;
        if (s.defined()) {
            ps = THPVariable_Wrap(std::move(s));
        } else {
            ps = a[0];
            Py_INCREF(ps);
        }
        PyObject *py = THPVariable_Wrap(std::move(y)), *pm = THPVariable_Wrap(std::move(mean));
        PyObject *pr = THPVariable_Wrap(std::move(rstd));
        if (quantize)
            return Py_BuildValue("(NNNNN)", py, THPVariable_Wrap(std::move(scale)), ps, pm, pr);
        return Py_BuildValue("(NNNN)", py, ps, pm, pr);
    });
}

// dy, s, mean, rstd, weight, ds, need_dweight, need_dbias, workspace
PyObject *add_layernorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 9)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dy = tensor(a[0], "dy");
        const ScalarType t = dy.scalar_type();
        const int type = operand_type(dy, "dy", false);
        const Mat G = matrix(dy, "dy", dy, t);
        const OnDevice device(dy.device());
        const int64_t rows = dy.size(0), d = dy.size(1);
        const Mat S = matrix(tensor(a[1], "s"), "s", dy, t, rows, d);
        const Mat D = optional_matrix(a[5], "ds", dy, t, rows, d);
        void *mean = vector(a[2], "mean", dy, ScalarType::Float, rows);
        void *rstd = vector(a[3], "rstd", dy, ScalarType::Float, rows);
        void *w = vector(a[4], "weight", dy, t, d);
        const bool need_w = flag(a[6]), need_b = flag(a[7]);
        at::Tensor dx = fresh(dy, {rows, d}, t), dw, db;
        if (need_w && need_b) {
            const at::Tensor both = fresh(dy, {2 * d}, t);
            dw = part(both, 0, {d});
            db = part(both, d, {d});
        } else if (need_w || need_b) {
            (need_w ? dw : db) = fresh(dy, {d}, t);
        }
        const Scratch s(a[8], need_w || need_b ? f_add_layernorm_backward_ws(type, rows, d) : 0, dy);
        check_status(f_add_layernorm_backward(
            type, rows, d, G.p, G.ld, S.p, S.ld, (const float *)mean, (const float *)rstd, w, D.p,
            D.ld, dx.data_ptr(), std::max<int64_t>(d, 1), need_w ? dw.data_ptr() : nullptr,
            need_b ? db.data_ptr() : nullptr, s.p, s.bytes, current_stream(dy)));
        return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(dx)),
                             need_w ? THPVariable_Wrap(std::move(dw)) : none(),
                             need_b ? THPVariable_Wrap(std::move(db)) : none());
    });
}

// The items of a Python list or tuple (of any sequence, as a list of its items).
struct Items {
    PyObject *seq;
    Items(PyObject *o, const char *name) : seq(PySequence_Fast(o, "")) {
        if (seq == nullptr) {
            PyErr_Clear();
            type_error(std::string(name) + " must be a sequence of tensors");
        }
    }
    Items(const Items &) = delete;
    ~Items() { Py_DECREF(seq); }
    int64_t size() const { return PySequence_Fast_GET_SIZE(seq); }
    PyObject *operator[](int64_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// tensors, scale (whether they are scaled), max_norm, eps, out, workspace
PyObject *clip_grad_norm(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 6)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Items list(a[0], "tensors");
        const int64_t count = list.size();
        if (count == 0) value_error("tensors is empty: it names no device for the norm");
        const bool scale = flag(a[1]), apart = scale && present(a[4]);
        const double max_norm = PyFloat_AsDouble(a[2]), eps = PyFloat_AsDouble(a[3]);
        if (PyErr_Occurred()) throw Raised{};
        const Items results(apart ? a[4] : a[0], "out");
        if (results.size() != count)
            value_error("out has " + std::to_string(results.size()) + " tensors, expected " +
                        std::to_string(count));
        std::vector<int> types(count);
        std::vector<int64_t> sizes(count);
        std::vector<const void *> x(count);
        std::vector<void *> y(count);
        const at::Tensor &like = tensor(list[0], "a tensor of the list");
        for (int64_t i = 0; i < count; ++i) {
            const at::Tensor &t = tensor(list[i], "a tensor of the list");
            types[i] = operand_type(t, "a tensor of the list", false);
            if (!t.is_cuda()) type_error("the tensors must be CUDA tensors");
            same_device(t, like, "a tensor of the list");
            if (!t.is_non_overlapping_and_dense())
                value_error("tensor " + std::to_string(i) + " has gaps between its elements, or shares them");
            sizes[i] = t.numel();
            x[i] = t.data_ptr();
            if (!scale) continue;
            const at::Tensor &o = tensor(results[i], "a tensor of out");
            bool alike = o.scalar_type() == t.scalar_type() && o.is_cuda() && o.sizes() == t.sizes();
            for (int64_t d = 0; alike && d < t.dim(); ++d)
                alike = t.size(d) <= 1 || o.stride(d) == t.stride(d);
            if (!alike)
                value_error("out's tensor " + std::to_string(i) +
                            " must have the type, shape and strides of the list's");
            same_device(o, like, "a tensor of out");
            y[i] = o.data_ptr();
        }
        const OnDevice device(like.device());
        at::Tensor norm = fresh(like, {}, ScalarType::Float);
        const Scratch s(a[5], f_clip_grad_norm_ws(count, types.data(), sizes.data()), like);
        check_status(f_clip_grad_norm(count, types.data(), sizes.data(), x.data(),
                                      scale ? y.data() : nullptr, (float)max_norm, (float)eps,
                                      (float *)norm.data_ptr(), s.p, s.bytes, current_stream(like)));
        for (int64_t i = 0; scale && i < count; ++i) {
            const at::Tensor &o = tensor(results[i], "a tensor of out");
            if (!o.is_inference()) o.unsafeGetTensorImpl()->bump_version();
        }
        return THPVariable_Wrap(std::move(norm));
    });
}

// t, like: what every entry asks of its tensors' devices
PyObject *check_device(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 2)) return nullptr;
    return guarded([&]() -> PyObject * {
        same_device(tensor(a[0], "t"), tensor(a[1], "like"), "t");
        return none();
    });
}

// bind({name: address}, raise, out_of_memory): the loaded library's entry points,
// what to call with a nonzero status, and the type to raise when torch's allocator
// has no memory left.
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *table, *raise, *out_of_memory;
    if (!PyArg_ParseTuple(args, "O!OO", &PyDict_Type, &table, &raise, &out_of_memory))
        return nullptr;
#define BIND(name, f)                                                                           \
    do {                                                                                       \
        PyObject *v = PyDict_GetItemString(table, #name);                                      \
        if (v == nullptr) {                                                                    \
            PyErr_SetString(PyExc_KeyError, #name);                                            \
            return nullptr;                                                                    \
        }                                                                                      \
        const unsigned long long p = PyLong_AsUnsignedLongLong(v);                             \
        if (PyErr_Occurred()) return nullptr;                                                  \
        f = reinterpret_cast<decltype(f)>(static_cast<uintptr_t>(p));                          \
    } while (0)
    BIND(sgemm_linear, f_linear);
    BIND(sgemm_linear_workspace_size, f_linear_ws);
    BIND(sgemm_linear_backward, f_linear_backward);
    BIND(sgemm_linear_backward_workspace_size, f_linear_backward_ws);
    BIND(sgemm_add_rmsnorm, f_add_rmsnorm);
    BIND(sgemm_add_rmsnorm_backward, f_add_rmsnorm_backward);
    BIND(sgemm_add_rmsnorm_backward_workspace_size, f_add_rmsnorm_backward_ws);
    BIND(sgemm_quantize_rows, f_quantize_rows);
    BIND(sgemm_gated_linear, f_gated_linear);
    BIND(sgemm_gated_linear_workspace_size, f_gated_linear_ws);
    BIND(sgemm_gated_linear_backward, f_gated_linear_backward);
    BIND(sgemm_gated_linear_backward_workspace_size, f_gated_linear_backward_ws);
    BIND(sgemm_add_layernorm, f_add_layernorm);
    BIND(sgemm_add_layernorm_backward, f_add_layernorm_backward);
    BIND(sgemm_add_layernorm_backward_workspace_size, f_add_layernorm_backward_ws);
    BIND(sgemm_clip_grad_norm, f_clip_grad_norm);
    BIND(sgemm_clip_grad_norm_workspace_size, f_clip_grad_norm_ws);
#undef BIND
    Py_INCREF(raise);
    Py_INCREF(out_of_memory);
    py_raise = raise;
    py_out_of_memory = out_of_memory;
    return none();
}

#define ENTRY(name)                                                                             \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    ENTRY(linear),
    ENTRY(linear_backward),
    ENTRY(add_rmsnorm),
    ENTRY(add_rmsnorm_backward),
    ENTRY(quantize_rows),
    ENTRY(gated_linear),
    ENTRY(gated_linear_backward),
    ENTRY(add_layernorm),
    ENTRY(add_layernorm_backward),
    ENTRY(clip_grad_norm),
    ENTRY(check_device),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers", "The layer operators on torch tensors", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers(void) { return PyModule_Create(&module); }
