// bsf8_torch.cpp -- the decode operators' calls from torch tensors, as a CPython extension.
//
// The ctypes binding spends more time on a call's arguments (up to thirty, some twenty tensors)
// than the GPU does on a decode step's operators.  This module checks and marshals them in C++: one
// positional call per operator, outputs from torch's allocator, the current stream, then the C
// ABI.  A call that the library refuses returns its status as an int; what is wrong with a tensor
// itself raises ValueError or TypeError.  decode.py holds the signatures and the documentation.
// Host time a call, here and by ctypes: append and read together 8.3 and 42 us, read 4.6 and 19, attention
// 7.2, verification 5.1.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <string>

#include "bsf8.h"

namespace {

struct Refused {
    PyObject *type;
    std::string what;
};

std::string shape_text(const int64_t *s, int n) {
    std::string t = "(";
    for (int i = 0; i < n; ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (n == 1 ? ",)" : ")");
}

const char *type_text(at::ScalarType t) {
    switch (t) {
        case at::kByte: return "torch.uint8";
        case at::kInt: return "torch.int32";
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        default: return c10::toString(t);
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
    return THPVariable_Unpack(o);
}

// One call's device: that of its first tensor, current until the call returns (the library launches on
// the current device and reads its status word there).
struct Call {
    int dev = -1;
    c10::cuda::OptionalCUDAGuard guard;

    void cuda(const at::Tensor &t, const char *name) {
        if (!t.is_cuda())
            throw Refused{PyExc_ValueError, std::string(name) + " must be a CUDA tensor (libbsf8 has no CPU path)"};
        const int d = t.get_device();
        if (dev < 0) {
            dev = d;
            guard.set_index((c10::DeviceIndex)d);
        }
        if (d != dev)
            throw Refused{PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(d) + ", the call on cuda:" +
                                                std::to_string(dev)};
    }
    void type(const at::Tensor &t, at::ScalarType want, const char *name) {
        if (t.scalar_type() != want)
            throw Refused{PyExc_TypeError,
                          std::string(name) + " must be " + type_text(want) + ", got " + type_text(t.scalar_type())};
    }
    // A contiguous tensor of this type and shape.
    template <int N>
    void *whole(const at::Tensor &t, at::ScalarType want, const int64_t (&shape)[N], const char *name) {
        bool same = t.dim() == N;
        for (int i = 0; same && i < N; ++i) same = t.size(i) == shape[i];
        if (!same)
            throw Refused{PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape, N) + ", got " +
                                                shape_text(t.sizes().data(), (int)t.dim())};
        cuda(t, name);
        type(t, want, name);
        if (!t.is_contiguous()) throw Refused{PyExc_ValueError, std::string(name) + " must be contiguous"};
        return t.data_ptr();
    }
    template <int N>
    void *whole(PyObject *o, at::ScalarType want, const int64_t (&shape)[N], const char *name) {
        return whole(tensor(o, name), want, shape, name);
    }
    template <int N>
    void *maybe(PyObject *o, at::ScalarType want, const int64_t (&shape)[N], const char *name) {
        return o == Py_None ? nullptr : whole(o, want, shape, name);
    }
    template <int N>
    at::Tensor fresh(at::ScalarType type, const int64_t (&shape)[N]) {
        // past the dispatcher: half the host time
        return at::Tensor(at::detail::empty_cuda(c10::IntArrayRef(shape, N), type, c10::Device(c10::kCUDA, dev), std::nullopt));
    }
    // The output the caller gave, checked, or a new one.
    template <int N>
    at::Tensor output(PyObject *o, at::ScalarType type, const int64_t (&shape)[N], const char *name) {
        if (o == Py_None) return fresh(type, shape);
        const at::Tensor &t = tensor(o, name);
        whole(t, type, shape, name);
        return t;
    }
    bsf8_stream_t stream() const {
        return reinterpret_cast<bsf8_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    }
};

// Arguments 0 .. 3: k8, kexp, v8, vexp.
bsf8_kv_cache cache_of(Call &c, PyObject *const *a) {
    const at::Tensor &k8 = tensor(a[0], "k8"), &ke = tensor(a[1], "kexp"), &v8 = tensor(a[2], "v8"),
                     &ve = tensor(a[3], "vexp");
    if (k8.dim() != 4) throw Refused{PyExc_ValueError, "k8 must be [pages, heads, page_size, dim]"};
    const int64_t code[4] = {k8.size(0), k8.size(1), k8.size(2), k8.size(3)};
    const int64_t byte[4] = {code[0], code[1], code[2], code[3] / 32};
    bsf8_kv_cache s;
    // shapes before devices, so that a wrong shape is named wherever the tensors are
    auto shape = [](const at::Tensor &t, const int64_t (&want)[4], const char *name) {
        bool same = t.dim() == 4;
        for (int i = 0; same && i < 4; ++i) same = t.size(i) == want[i];
        if (!same)
            throw Refused{PyExc_ValueError, std::string(name) + " must have shape " + shape_text(want, 4) + ", got " +
                                                shape_text(t.sizes().data(), (int)t.dim())};
    };
    shape(ke, byte, "kexp");
    shape(v8, code, "v8");
    shape(ve, byte, "vexp");
    s.k8 = static_cast<uint8_t *>(c.whole(k8, at::kByte, code, "k8"));
    s.kexp = static_cast<uint8_t *>(c.whole(ke, at::kByte, byte, "kexp"));
    s.v8 = static_cast<uint8_t *>(c.whole(v8, at::kByte, code, "v8"));
    s.vexp = static_cast<uint8_t *>(c.whole(ve, at::kByte, byte, "vexp"));
    for (const int64_t n : code)
        if (n > 0x7FFFFFFF) throw Refused{PyExc_ValueError, "the cache's sizes must fit 31 bits"};
    s.pages = (int)code[0];
    s.heads = (int)code[1];
    s.page_size = (int)code[2];
    s.dim = (int)code[3];
    return s;
}

struct Table {
    const int32_t *at;
    int requests, pages;
};

Table table_of(Call &c, PyObject *o) {
    const at::Tensor &t = tensor(o, "table");
    if (t.dim() != 2) throw Refused{PyExc_ValueError, "table must be [requests, table_pages]"};
    const int64_t shape[2] = {t.size(0), t.size(1)};
    return Table{static_cast<const int32_t *>(c.whole(t, at::kInt, shape, "table")), (int)shape[0], (int)shape[1]};
}

// [N, heads, dim] bf16 rows whose heads lie one after another.
struct Rows {
    const void *at;
    int64_t n, heads, ld;
};

Rows rows_of(Call &c, PyObject *o, const char *name, int64_t heads, int64_t dim) {
    const at::Tensor &t = tensor(o, name);
    c.cuda(t, name);
    c.type(t, at::kBFloat16, name);
    if (t.dim() != 3 || (heads >= 0 && t.size(1) != heads) || t.size(2) != dim)
        throw Refused{PyExc_ValueError, std::string(name) + " must be [N, " +
                                            (heads >= 0 ? std::to_string(heads) : std::string("Hq")) + ", " +
                                            std::to_string(dim) + "], got " +
                                            shape_text(t.sizes().data(), (int)t.dim())};
    const int64_t n = t.size(0), h = t.size(1);
    if (t.numel() && (t.stride(2) != 1 || (h > 1 && t.stride(1) != dim)))
        throw Refused{PyExc_ValueError, std::string(name) + "'s heads must lie one after another (strides (*, " +
                                            std::to_string(dim) + ", 1))"};
    return Rows{t.data_ptr(), n, h, n > 1 ? t.stride(0) : h * dim};
}

int small(int64_t n, const char *name) {
    if (n > 0x7FFFFFFF) throw Refused{PyExc_ValueError, std::string(name) + " must fit 31 bits"};
    return (int)n;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{nullptr, ""};
    return v != 0;
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &r) {
        if (r.type) PyErr_SetString(r.type, r.what.c_str());
    } catch (...) {  // torch's own (out of memory and the like) as its Python errors
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// k8 kexp v8 vexp | q k v table req slot pos cos_sin q_norm k_norm eps interleaved out
PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 17, [&]() -> PyObject * {
        Call c;
        const bsf8_kv_cache s = cache_of(c, a);
        const Rows k = rows_of(c, a[5], "k", s.heads, s.dim), v = rows_of(c, a[6], "v", s.heads, s.dim);
        if (v.n != k.n) throw Refused{PyExc_ValueError, "k and v must have the same tokens"};
        Rows q{nullptr, k.n, 0, 0};
        at::Tensor out;
        if (a[4] != Py_None) {
            q = rows_of(c, a[4], "q", -1, s.dim);
            if (q.n != k.n) throw Refused{PyExc_ValueError, "q must have the tokens of k"};
            const int64_t shape[3] = {q.n, q.heads, s.dim};
            out = c.output(a[16], at::kBFloat16, shape, "out");
        }
        const Table t = table_of(c, a[7]);
        const int64_t tokens[1] = {k.n}, dim[1] = {s.dim};
        const auto *req = static_cast<const int32_t *>(c.whole(a[8], at::kInt, tokens, "req"));
        const auto *slot = static_cast<const int32_t *>(c.whole(a[9], at::kInt, tokens, "slot"));
        const int32_t *pos = nullptr;
        const float *cs = nullptr;
        int positions = 0, rot = 0;
        if (a[11] != Py_None) {
            const at::Tensor &x = tensor(a[11], "cos_sin");
            if (x.dim() != 2) throw Refused{PyExc_ValueError, "cos_sin must be [positions, rot]"};
            if (a[10] == Py_None) throw Refused{PyExc_ValueError, "a rotation needs pos"};
            const int64_t shape[2] = {x.size(0), x.size(1)};
            cs = static_cast<const float *>(c.whole(x, at::kFloat, shape, "cos_sin"));
            pos = static_cast<const int32_t *>(c.whole(a[10], at::kInt, tokens, "pos"));
            positions = small(shape[0], "cos_sin");
            rot = small(shape[1], "cos_sin");
        }
        const void *qn = c.maybe(a[12], at::kBFloat16, dim, "q_norm"), *kn = c.maybe(a[13], at::kBFloat16, dim, "k_norm");
        const int status = bsf8_qkv_append(q.at, k.at, v.at, q.ld, k.ld, v.ld, out.defined() ? out.data_ptr() : nullptr, &s,
                                           t.at, t.requests, t.pages, req, slot, pos, cs, positions, rot,
                                           truth(a[15]), qn, kn, (float)number(a[14]), small(k.n, "the tokens"),
                                           small(q.heads, "Hq"), c.stream());
        if (status) return PyLong_FromLong(status);
        if (!out.defined()) Py_RETURN_NONE;
        if (a[16] != Py_None) return Py_NewRef(a[16]);
        return THPVariable_Wrap(std::move(out));
    });
}

// k8 kexp v8 vexp | table req slot k_out v_out
PyObject *py_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        Call c;
        const bsf8_kv_cache s = cache_of(c, a);
        const Table t = table_of(c, a[4]);
        const at::Tensor &req = tensor(a[5], "req");
        const int64_t tokens[1] = {req.dim() == 1 ? req.size(0) : -1}, shape[3] = {tokens[0], s.heads, s.dim};
        const auto *rp = static_cast<const int32_t *>(c.whole(req, at::kInt, tokens, "req"));
        const auto *sp = static_cast<const int32_t *>(c.whole(a[6], at::kInt, tokens, "slot"));
        at::Tensor k = c.output(a[7], at::kBFloat16, shape, "k_out"), v = c.output(a[8], at::kBFloat16, shape, "v_out");
        const int status = bsf8_kv_read(&s, t.at, t.requests, t.pages, rp, sp, k.data_ptr(), v.data_ptr(),
                                        small(tokens[0], "the tokens"), c.stream());
        if (status) return PyLong_FromLong(status);
        PyObject *ko = a[7] != Py_None ? Py_NewRef(a[7]) : THPVariable_Wrap(std::move(k));
        PyObject *vo = a[8] != Py_None ? Py_NewRef(a[8]) : THPVariable_Wrap(std::move(v));
        PyObject *r = ko && vo ? PyTuple_Pack(2, ko, vo) : nullptr;
        Py_XDECREF(ko);
        Py_XDECREF(vo);
        return r;
    });
}

// k8 kexp v8 vexp | q table ctx nodes mask scale max_len out lse workspace
PyObject *py_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        Call c;
        const bsf8_kv_cache s = cache_of(c, a);
        const at::Tensor &q = tensor(a[4], "q");
        c.cuda(q, "q");
        c.type(q, at::kBFloat16, "q");
        if (q.dim() != 4 || q.size(3) != s.dim)
            throw Refused{PyExc_ValueError, "q must be [B, T, Hq, " + std::to_string(s.dim) + "]"};
        const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2);
        const int64_t ldq = T > 1 ? q.stride(1) : B > 1 ? q.stride(0) : Hq * s.dim;
        if (q.stride(3) != 1 || (Hq > 1 && q.stride(2) != s.dim) || (B > 1 && q.stride(0) != T * ldq))
            throw Refused{PyExc_ValueError, "q must have strides (T * ld, ld, " + std::to_string(s.dim) + ", 1)"};
        const Table t = table_of(c, a[5]);
        if (t.requests != B) throw Refused{PyExc_ValueError, "table must have a row for each request"};
        const int64_t per[1] = {B}, words[3] = {B, T, (T + 31) / 32}, rows[3] = {B, T, Hq}, shape[4] = {B, T, Hq, s.dim};
        const auto *ctx = static_cast<const int32_t *>(c.whole(a[6], at::kInt, per, "ctx"));
        const auto *nodes = static_cast<const int32_t *>(c.maybe(a[7], at::kInt, per, "nodes"));
        const auto *mask = static_cast<const int32_t *>(c.maybe(a[8], at::kInt, words, "mask"));
        auto *lse = static_cast<float *>(c.maybe(a[12], at::kFloat, rows, "lse"));
        at::Tensor out = c.output(a[11], at::kBFloat16, shape, "out"), ws;
        const int b = small(B, "B"), tt = small(T, "T"), hq = small(Hq, "Hq");
        const size_t need = bsf8_tree_attention_workspace_bytes(b, tt, hq, s.heads, s.dim);
        size_t have = 0;
        if (need) {
            if (a[13] == Py_None) {
                const int64_t bytes[1] = {(int64_t)need};
                ws = c.fresh(at::kByte, bytes);
            } else {
                ws = tensor(a[13], "workspace");
                const int64_t bytes[1] = {ws.numel()};
                c.whole(ws, at::kByte, bytes, "workspace");
            }
            have = (size_t)ws.numel();
        }
        long max_len = 0;
        if (a[10] == Py_None) {
            max_len = std::min((long)t.pages * s.page_size, (long)BSF8_MAX_LEN);
        } else {
            max_len = PyLong_AsLong(a[10]);
            if (max_len == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
        }
        if (max_len > 0x7FFFFFFF || max_len < -1) throw Refused{PyExc_ValueError, "max_len must fit 31 bits"};
        const double scale = a[9] == Py_None ? 1.0 / std::sqrt((double)s.dim) : number(a[9]);
        const int status =
            bsf8_tree_attention(q.data_ptr(), ldq, &s, t.at, t.pages, ctx, nodes, mask, (float)scale, (int)max_len,
                                out.data_ptr(), lse, b, tt, hq, need ? ws.data_ptr() : nullptr, have, c.stream());
        if (status) return PyLong_FromLong(status);
        return a[11] != Py_None ? Py_NewRef(a[11]) : THPVariable_Wrap(std::move(out));
    });
}

// p tokens parent u q nodes
PyObject *py_verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject * {
        Call c;
        const at::Tensor &p = tensor(a[0], "p");
        if (p.dim() != 3) throw Refused{PyExc_ValueError, "p must be [B, T, V]"};
        const int64_t B = p.size(0), T = p.size(1), V = p.size(2);
        const int64_t ld = T > 1 ? p.stride(1) : B > 1 ? p.stride(0) : V;
        auto probabilities = [&](const at::Tensor &t, const char *name) -> const float * {
            c.cuda(t, name);
            c.type(t, at::kFloat, name);
            if (t.dim() != 3 || t.size(0) != B || t.size(1) != T || t.size(2) != V || (V > 1 && t.stride(2) != 1) ||
                (T > 1 && t.stride(1) != ld) || (B > 1 && t.stride(0) != T * ld))
                throw Refused{PyExc_ValueError, std::string(name) + " must be [B, T, V] with strides (T * ld, ld, 1), p's "
                                                                    "and q's ld the same"};
            return static_cast<const float *>(t.data_ptr());
        };
        const float *pp = probabilities(p, "p"), *qp = a[4] == Py_None ? nullptr : probabilities(tensor(a[4], "q"), "q");
        const int64_t each[2] = {B, T}, per[1] = {B};
        const auto *tok = static_cast<const int32_t *>(c.whole(a[1], at::kInt, each, "tokens"));
        const auto *par = static_cast<const int32_t *>(c.whole(a[2], at::kInt, each, "parent"));
        const auto *u = static_cast<const float *>(c.whole(a[3], at::kFloat, each, "u"));
        const auto *nodes = static_cast<const int32_t *>(c.maybe(a[5], at::kInt, per, "nodes"));
        at::Tensor path = c.fresh(at::kInt, each), count = c.fresh(at::kInt, per), token = c.fresh(at::kInt, per);
        const int status = bsf8_verify_tree(pp, qp, ld, tok, par, u, nodes, static_cast<int32_t *>(path.data_ptr()),
                                            static_cast<int32_t *>(count.data_ptr()),
                                            static_cast<int32_t *>(token.data_ptr()), small(B, "B"), small(T, "T"),
                                            small(V, "V"), c.stream());
        if (status) return PyLong_FromLong(status);
        PyObject *o[3] = {THPVariable_Wrap(std::move(path)), THPVariable_Wrap(std::move(count)),
                          THPVariable_Wrap(std::move(token))};
        PyObject *r = o[0] && o[1] && o[2] ? PyTuple_Pack(3, o[0], o[1], o[2]) : nullptr;
        for (PyObject *x : o) Py_XDECREF(x);
        return r;
    });
}

// k8 kexp v8 vexp | table ctx path count
PyObject *py_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        Call c;
        const bsf8_kv_cache s = cache_of(c, a);
        const Table t = table_of(c, a[4]);
        const at::Tensor &path = tensor(a[6], "path");
        if (path.dim() != 2) throw Refused{PyExc_ValueError, "path must be [B, T]"};
        const int64_t B = path.size(0), T = path.size(1);
        if (t.requests != B) throw Refused{PyExc_ValueError, "table must have a row for each request"};
        const int64_t each[2] = {B, T}, per[1] = {B};
        const auto *ctx = static_cast<const int32_t *>(c.whole(a[5], at::kInt, per, "ctx"));
        const auto *pp = static_cast<const int32_t *>(c.whole(path, at::kInt, each, "path"));
        const auto *count = static_cast<const int32_t *>(c.whole(a[7], at::kInt, per, "count"));
        const int status = bsf8_kv_commit(&s, t.at, t.pages, ctx, pp, count, small(B, "B"), small(T, "T"), c.stream());
        if (status) return PyLong_FromLong(status);
        Py_RETURN_NONE;
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<py_append>("qkv_append"), method<py_read>("kv_read"),
                         method<py_attention>("tree_attention"), method<py_verify>("verify_tree"),
                         method<py_commit>("kv_commit"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bsf8_torch", "Calls of libbsf8's decode operators from torch tensors.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bsf8_torch(void) { return PyModule_Create(&module); }
