// rog_binding.cpp -- the quick way through the Python binding's argument
// marshalling, for the vocabulary-side operators and the head's products: a CPython module that reads
// tensors' addresses, types and shapes directly and calls the C interface
// (include/rog.h).  Every function returns True if the call was enqueued and
// False if anything about it is out of the ordinary -- an argument that the
// library would refuse, a workspace that has to be made or grown, a stream
// that is being captured -- and has then enqueued nothing: rog.py takes the
// call from there, and raises what is to be raised.  It keeps no tensor, and
// allocates but the head's products' workspaces.  (Through ctypes alone these calls take 4 to 6
// microseconds of Python beside 3 to 4 of launching.)
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <mutex>
#include <unordered_map>

#include "rog.h"

namespace {

// Set once by bind(): the library's entry points and torch's callables.
struct Bound {
    decltype(&rog_logprob_ex) logprob = nullptr;
    decltype(&rog_logprob_grad) grad = nullptr;
    decltype(&rog_policy_loss) loss = nullptr;
    decltype(&rog_linear_logprob) linear_logprob = nullptr;
    decltype(&rog_linear_logprob_grad) linear_grad = nullptr;
    decltype(&rog_quantize_i8) quantize = nullptr;
    decltype(&rog_linear_i8) linear_i8 = nullptr;
    decltype(&rog_linear_logprob_plan) linear_logprob_plan = nullptr;
    decltype(&rog_linear_logprob_grad_plan) linear_grad_plan = nullptr;
    int max_peers = 0;
    PyObject *current_device = nullptr, *raw_stream = nullptr, *capturing = nullptr;
} bound;

// The streams' own workspaces, as rog.py keeps them (it never frees one).
struct Workspace {
    void *address;
    size_t bytes;
};
struct StreamKey {
    int device;
    uint64_t stream;
    bool operator==(const StreamKey &o) const { return device == o.device && stream == o.stream; }
};
struct StreamHash {
    size_t operator()(const StreamKey &k) const { return std::hash<uint64_t>()(k.stream * 31 + uint64_t(k.device)); }
};
std::unordered_map<StreamKey, Workspace, StreamHash> workspaces;
std::mutex workspaces_lock;

long call_long(PyObject *f, PyObject *arg, bool *ok) {
    PyObject *r = arg ? PyObject_CallOneArg(f, arg) : PyObject_CallNoArgs(f);
    const long v = r ? PyLong_AsLong(r) : -1;
    Py_XDECREF(r);
    if (PyErr_Occurred()) *ok = false;
    return v;
}

// The stream to launch on, where the tensors' device is the current one.
struct Where {
    bool ok = true;
    uint64_t stream = 0;
    Workspace ws{nullptr, 0};
    Where(int device, bool may_need_workspace) {
        ok = device >= 0 && call_long(bound.current_device, nullptr, &ok) == device && ok;
        if (!ok) return;
        PyObject *d = PyLong_FromLong(device);
        stream = uint64_t(call_long(bound.raw_stream, d, &ok));
        Py_DECREF(d);
        if (!ok || !may_need_workspace) return;
        {
            std::lock_guard<std::mutex> hold(workspaces_lock);
            const auto it = workspaces.find(StreamKey{device, stream});
            if (it != workspaces.end()) ws = it->second;
        }
        // a captured call gets a workspace of its own (rog.py)
        if (ws.bytes) ok = call_long(bound.capturing, nullptr, &ok) == 0 && ok;
    }
    hipStream_t hip() const { return reinterpret_cast<hipStream_t>(stream); }
};

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const at::Tensor &t, int device) { return t.is_cuda() && t.get_device() == device; }

// The address of a contiguous vector of n elements; NULL for None.
template <typename P>
bool vector(PyObject *o, int64_t n, at::ScalarType type, int device, P **p) {
    *p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o);
    if (!t || t->scalar_type() != type || !on(*t, device) || t->numel() != n || !t->is_contiguous()) return false;
    *p = static_cast<P *>(t->data_ptr());
    return true;
}

bool dtype_of(at::ScalarType t, rog_dtype *d) {
    switch (t) {
    case at::kFloat: *d = ROG_DTYPE_F32; return true;
    case at::kBFloat16: *d = ROG_DTYPE_BF16; return true;
    case at::kHalf: *d = ROG_DTYPE_F16; return true;
    default: return false;
    }
}

// W logits matrices (a list or tuple).
struct Shards {
    rog_logit_shard s[64];
    int W = 0, device = -1;
    int64_t rows = 0;
    at::ScalarType type = at::kFloat;
    rog_dtype dtype = ROG_DTYPE_F32;
    bool read(PyObject *list) {
        if (!PyList_Check(list) && !PyTuple_Check(list)) return false;
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
        if (n < 1 || n > 64 || n > bound.max_peers) return false;
        W = int(n);
        for (int i = 0; i < W; ++i) {
            const at::Tensor *t = tensor(PySequence_Fast_GET_ITEM(list, i));
            if (!t || t->dim() != 2) return false;
            if (i == 0) {
                rows = t->size(0);
                type = t->scalar_type();
                if (!t->is_cuda() || !dtype_of(type, &dtype)) return false;
                device = t->get_device();
            }
            if (t->size(0) != rows || t->scalar_type() != type || !on(*t, device) || (t->size(1) > 1 && t->stride(1) != 1)) return false;
            s[i] = rog_logit_shard{t->data_ptr(), t->stride(0), t->size(1)};
        }
        return true;
    }
};

// A matrix that is contiguous within its rows; rows or columns of -1: any.
struct Matrix {
    void *p;
    int64_t stride, rows, columns;
    at::ScalarType type;
    int device;
    bool read(PyObject *o) {
        const at::Tensor *t = tensor(o);
        if (!t || t->dim() != 2 || !t->is_cuda() || (t->size(1) > 1 && t->stride(1) != 1)) return false;
        *this = Matrix{t->data_ptr(), t->stride(0), t->size(0), t->size(1), t->scalar_type(), t->get_device()};
        return true;
    }
    bool is(int64_t r, int64_t c, at::ScalarType want, int d) const { return rows == r && columns == c && type == want && device == d; }
};

// The items of a list or tuple of between 1 and 64, and no more than the library takes.
bool items(PyObject *list, Py_ssize_t *n) {
    if (!PyList_Check(list) && !PyTuple_Check(list)) return false;
    *n = PySequence_Fast_GET_SIZE(list);
    return *n >= 1 && *n <= 64 && *n <= bound.max_peers;
}

// Hidden states and the head's W weight matrices (a list or tuple).
struct Head {
    Matrix h;
    rog_weight_shard s[64];
    Py_ssize_t W = 0;
    rog_dtype dtype = ROG_DTYPE_BF16;
    bool read(PyObject *hidden, PyObject *list) {
        if (!h.read(hidden) || !items(list, &W)) return false;
        if (h.type != at::kChar && (!dtype_of(h.type, &dtype) || dtype == ROG_DTYPE_F32)) return false;
        for (Py_ssize_t i = 0; i < W; ++i) {
            Matrix m;
            if (!m.read(PySequence_Fast_GET_ITEM(list, i)) || !m.is(m.rows, h.columns, h.type, h.device)) return false;
            s[i] = rog_weight_shard{m.p, m.stride, m.rows};
        }
        return true;
    }
    // W matrices to write, of the weights' shapes, or [rows][width] of `type`.
    bool outputs(PyObject *list, bool weights, at::ScalarType type, rog_grad_shard *g) const {
        Py_ssize_t n;
        if (!items(list, &n) || n != W) return false;
        for (Py_ssize_t i = 0; i < W; ++i) {
            Matrix m;
            if (!m.read(PySequence_Fast_GET_ITEM(list, i)) ||
                !m.is(weights ? s[i].width : h.rows, weights ? h.columns : s[i].width, type, h.device))
                return false;
            g[i] = rog_grad_shard{m.p, m.stride};
        }
        return true;
    }
};

// A workspace of one call's own, made on the current stream by torch's allocator:
// the head's products hand data from launch to launch through it, and another
// thread's call on the same stream may come between two of them.  It goes back when
// the call has enqueued them all, for what is enqueued on this stream behind them.
struct Scratch {
    at::Tensor t;
    Scratch(int device, size_t bytes) {
        if (bytes) t = at::empty({int64_t(bytes)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, c10::DeviceIndex(device)));
    }
    void *address() const { return t.defined() ? t.data_ptr() : nullptr; }
};

bool number(PyObject *o, float *f) {
    const double v = PyFloat_AsDouble(o);
    *f = float(v);
    return !(v == -1.0 && PyErr_Occurred());
}

template <typename F>
bool launched(F call) {
    rog_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    return st == ROG_OK;
}

// Runs body() and turns its answer into True or False; errors on the way (a
// tensor without storage, a callable that raised) are False too.
template <typename F>
PyObject *answer(F body) {
    bool ok = false;
    try {
        ok = bound.logprob && body();
    } catch (...) {
        ok = false;
    }
    if (PyErr_Occurred()) {
        PyErr_Clear();
        ok = false;
    }
    return PyBool_FromLong(ok);
}

// logprob(shards, tokens, top_k, temperature, out, form)
PyObject *py_logprob(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return answer([&] {
        Shards sh;
        float temperature;
        rog_logprob_out out;
        const int64_t *tokens;
        if (n != 6 || !sh.read(a[0]) || !PyLong_Check(a[2]) || !PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 5 ||
            !PyLong_Check(a[5]) || !number(a[3], &temperature))
            return false;
        const long top_k = PyLong_AsLong(a[2]), form = PyLong_AsLong(a[5]);
        if (top_k < 0 || top_k > 1024) return false;
        PyObject *const *o = &PyTuple_GET_ITEM(a[4], 0);
        const int64_t rows = sh.rows, tops = rows * top_k;
        if (!vector(a[1], rows, at::kLong, sh.device, &tokens) || !vector(o[0], rows, at::kFloat, sh.device, &out.logp) ||
            !vector(o[1], rows, at::kFloat, sh.device, &out.entropy) || !vector(o[2], rows, at::kFloat, sh.device, &out.lse) ||
            !vector(o[3], tops, at::kFloat, sh.device, &out.top_logp) || !vector(o[4], tops, at::kLong, sh.device, &out.top_ids) ||
            (top_k == 0 && (o[3] != Py_None || o[4] != Py_None)))
            return false;
        const Where at(sh.device, true);
        return at.ok && launched([&] {
            return bound.logprob(sh.s, sh.W, size_t(rows), sh.dtype, temperature, tokens, int(top_k), &out, at.ws.address,
                                 at.ws.bytes, at.hip(), rog_logprob_form(form));
        });
    });
}

// grad(shards, tokens, lse, entropy, g_logp, g_entropy, temperature, out)
PyObject *py_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return answer([&] {
        Shards sh;
        rog_grad_shard g[64];
        float temperature;
        const int64_t *tokens;
        const float *v[4];
        if (n != 8 || !sh.read(a[0]) || !number(a[6], &temperature) || a[1] == Py_None) return false;
        if ((!PyList_Check(a[7]) && !PyTuple_Check(a[7])) || PySequence_Fast_GET_SIZE(a[7]) != sh.W) return false;
        for (int i = 0; i < sh.W; ++i) {
            const at::Tensor *t = tensor(PySequence_Fast_GET_ITEM(a[7], i));
            if (!t || t->dim() != 2 || t->size(0) != sh.rows || t->size(1) != sh.s[i].width || t->scalar_type() != sh.type ||
                !on(*t, sh.device) || (t->size(1) > 1 && t->stride(1) != 1))
                return false;
            g[i] = rog_grad_shard{t->data_ptr(), t->stride(0)};
        }
        if (!vector(a[1], sh.rows, at::kLong, sh.device, &tokens)) return false;
        for (int i = 0; i < 4; ++i)
            if ((i < 3 && a[2 + i] == Py_None) || !vector(a[2 + i], sh.rows, at::kFloat, sh.device, &v[i])) return false;
        const Where at(sh.device, false);
        return at.ok && launched([&] {
            return bound.grad(sh.s, g, sh.W, size_t(sh.rows), sh.dtype, temperature, tokens, v[0], v[1], v[2], v[3], at.hip());
        });
    });
}

// loss(logp, old_logp, advantage, weight, ref_logp, entropy, clip_low, clip_high, kl_coef, entropy_coef, grad_scale, out)
PyObject *py_loss(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return answer([&] {
        if (n != 12 || !PyTuple_Check(a[11]) || PyTuple_GET_SIZE(a[11]) != 3) return false;
        const at::Tensor *first = tensor(a[0]);
        if (!first || !first->is_cuda() || a[1] == Py_None || a[2] == Py_None) return false;
        const int device = first->get_device();
        const int64_t count = first->numel();
        const float *in[6];
        float k[5];
        rog_policy_out out;
        for (int i = 0; i < 6; ++i)
            if (!vector(a[i], count, at::kFloat, device, &in[i])) return false;
        for (int i = 0; i < 5; ++i)
            if (!number(a[6 + i], &k[i])) return false;
        PyObject *const *o = &PyTuple_GET_ITEM(a[11], 0);
        if (o[0] == Py_None || !vector(o[0], 4, at::kFloat, device, &out.stats) || !vector(o[1], count, at::kFloat, device, &out.g_logp) ||
            !vector(o[2], count, at::kFloat, device, &out.g_entropy))
            return false;
        const rog_policy_in ins{in[0], in[1], in[2], in[3], in[4], in[5]};
        const rog_policy_params params{k[0], k[1], k[2], k[3], k[4]};
        const Where at(device, true);
        return at.ok && launched([&] { return bound.loss(&ins, size_t(count), &params, &out, at.ws.address, at.ws.bytes, at.hip()); });
    });
}

// linear_logprob(hidden, weights, tokens, temperature, out)
PyObject *py_linear_logprob(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return answer([&] {
        Head head;
        float temperature;
        rog_logprob_out out{};
        const int64_t *tokens;
        if (n != 5 || !head.read(a[0], a[1]) || head.h.type == at::kChar || !number(a[3], &temperature) || !PyTuple_Check(a[4]) ||
            PyTuple_GET_SIZE(a[4]) != 5)
            return false;
        PyObject *const *o = &PyTuple_GET_ITEM(a[4], 0);
        const int64_t rows = head.h.rows;
        const int device = head.h.device;
        if (!vector(a[2], rows, at::kLong, device, &tokens) || !vector(o[0], rows, at::kFloat, device, &out.logp) ||
            !vector(o[1], rows, at::kFloat, device, &out.entropy) || !vector(o[2], rows, at::kFloat, device, &out.lse) ||
            o[3] != Py_None || o[4] != Py_None)
            return false;
        const Where at(device, false);
        rog_linear_plan_info need;
        if (!at.ok || bound.linear_logprob_plan(head.s, int(head.W), size_t(rows), head.h.columns, head.dtype, tokens != nullptr, &need) != ROG_OK)
            return false;
        const Scratch ws(device, need.workspace_bytes);
        return launched([&] {
            return bound.linear_logprob(head.h.p, head.h.stride, size_t(rows), head.h.columns, head.s, int(head.W), head.dtype, temperature,
                                        tokens, &out, ws.address(), need.workspace_bytes, at.hip());
        });
    });
}

// linear_grad(hidden, weights, tokens, lse, entropy, g_logp, g_entropy, temperature, d_hidden, d_weights)
PyObject *py_linear_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return answer([&] {
        Head head;
        Matrix d;
        rog_grad_shard g[64];
        float temperature;
        const int64_t *tokens;
        const float *v[4];
        // without rows the library enqueues nothing: rog.py fills the weights' gradients
        if (n != 10 || !head.read(a[0], a[1]) || head.h.type == at::kChar || !number(a[7], &temperature) || a[2] == Py_None || head.h.rows == 0)
            return false;
        if (!d.read(a[8]) || !d.is(head.h.rows, head.h.columns, head.h.type, head.h.device) || !head.outputs(a[9], true, head.h.type, g))
            return false;
        if (!vector(a[2], head.h.rows, at::kLong, head.h.device, &tokens)) return false;
        for (int i = 0; i < 4; ++i)
            if ((i < 3 && a[3 + i] == Py_None) || !vector(a[3 + i], head.h.rows, at::kFloat, head.h.device, &v[i])) return false;
        const Where at(head.h.device, false);
        rog_linear_plan_info need;
        if (!at.ok || bound.linear_grad_plan(head.s, int(head.W), size_t(head.h.rows), head.h.columns, head.dtype, &need) != ROG_OK) return false;
        const Scratch ws(head.h.device, need.workspace_bytes);
        return launched([&] {
            return bound.linear_grad(head.h.p, head.h.stride, size_t(head.h.rows), head.h.columns, head.s, int(head.W), head.dtype,
                                     temperature, tokens, v[0], v[1], v[2], v[3], d.p, d.stride, g, ws.address(), need.workspace_bytes, at.hip());
        });
    });
}

// quantize(x, q, scale)
PyObject *py_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return answer([&] {
        Matrix x, q;
        rog_dtype dtype;
        float *scale;
        if (n != 3 || !x.read(a[0]) || !q.read(a[1]) || !dtype_of(x.type, &dtype) || !q.is(x.rows, x.columns, at::kChar, x.device) ||
            a[2] == Py_None || !vector(a[2], x.rows, at::kFloat, x.device, &scale))
            return false;
        const Where at(x.device, false);
        return at.ok && launched([&] {
            return bound.quantize(x.p, x.stride, size_t(x.rows), x.columns, dtype, static_cast<int8_t *>(q.p), q.stride, scale, at.hip());
        });
    });
}

// linear_i8(q, scale, weights, weight_scales, out)
PyObject *py_linear_i8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return answer([&] {
        Head head;
        rog_i8_shard s[64];
        rog_grad_shard out[64];
        rog_dtype dtype;
        const float *scale;
        Py_ssize_t scales;
        Matrix first;
        if (n != 5 || !head.read(a[0], a[2]) || head.h.type != at::kChar || a[1] == Py_None ||
            !vector(a[1], head.h.rows, at::kFloat, head.h.device, &scale) || !items(a[3], &scales) || scales != head.W)
            return false;
        for (Py_ssize_t i = 0; i < head.W; ++i) {
            PyObject *const r = PySequence_Fast_GET_ITEM(a[3], i);
            const float *p;
            if (r == Py_None || !vector(r, head.s[i].width, at::kFloat, head.h.device, &p)) return false;
            s[i] = rog_i8_shard{static_cast<const int8_t *>(head.s[i].weight), head.s[i].row_stride, head.s[i].width, p};
        }
        Py_ssize_t outs;
        if (!items(a[4], &outs) || !first.read(PySequence_Fast_GET_ITEM(a[4], 0)) || !dtype_of(first.type, &dtype) ||
            !head.outputs(a[4], false, first.type, out))
            return false;
        const Where at(head.h.device, false);
        return at.ok && launched([&] {
            return bound.linear_i8(static_cast<const int8_t *>(head.h.p), head.h.stride, scale, size_t(head.h.rows), head.h.columns, s,
                                   int(head.W), dtype, out, at.hip());
        });
    });
}

// workspace(device, stream, address, bytes): a stream's own workspace, made or grown
PyObject *py_workspace(PyObject *, PyObject *args) {
    int device;
    unsigned long long stream, address, bytes;
    if (!PyArg_ParseTuple(args, "iKKK", &device, &stream, &address, &bytes)) return nullptr;
    std::lock_guard<std::mutex> hold(workspaces_lock);
    workspaces[StreamKey{device, stream}] = Workspace{reinterpret_cast<void *>(address), size_t(bytes)};
    Py_RETURN_NONE;
}

// bind(entry points, max_peers, current_device, raw_stream, is_capturing): the entry
// points' addresses, in the order of `Bound`, and torch's callables
PyObject *py_bind(PyObject *, PyObject *args) {
    PyObject *entries, *device, *stream, *capturing;
    int max_peers;
    if (!PyArg_ParseTuple(args, "O!iOOO", &PyTuple_Type, &entries, &max_peers, &device, &stream, &capturing)) return nullptr;
    unsigned long long e[9];
    if (PyTuple_GET_SIZE(entries) != 9) {
        PyErr_SetString(PyExc_ValueError, "nine entry points");
        return nullptr;
    }
    for (int i = 0; i < 9; ++i) {
        e[i] = PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(entries, i));
        if (PyErr_Occurred()) return nullptr;
    }
    Py_INCREF(device);
    Py_INCREF(stream);
    Py_INCREF(capturing);
    bound.logprob = reinterpret_cast<decltype(bound.logprob)>(e[0]);
    bound.grad = reinterpret_cast<decltype(bound.grad)>(e[1]);
    bound.loss = reinterpret_cast<decltype(bound.loss)>(e[2]);
    bound.linear_logprob = reinterpret_cast<decltype(bound.linear_logprob)>(e[3]);
    bound.linear_grad = reinterpret_cast<decltype(bound.linear_grad)>(e[4]);
    bound.quantize = reinterpret_cast<decltype(bound.quantize)>(e[5]);
    bound.linear_i8 = reinterpret_cast<decltype(bound.linear_i8)>(e[6]);
    bound.linear_logprob_plan = reinterpret_cast<decltype(bound.linear_logprob_plan)>(e[7]);
    bound.linear_grad_plan = reinterpret_cast<decltype(bound.linear_grad_plan)>(e[8]);
    bound.max_peers = max_peers;
    bound.current_device = device;
    bound.raw_stream = stream;
    bound.capturing = capturing;
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fn(F *f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"logprob", fn(&py_logprob), METH_FASTCALL, nullptr},
                         {"grad", fn(&py_grad), METH_FASTCALL, nullptr},
                         {"loss", fn(&py_loss), METH_FASTCALL, nullptr},
                         {"linear_logprob", fn(&py_linear_logprob), METH_FASTCALL, nullptr},
                         {"linear_grad", fn(&py_linear_grad), METH_FASTCALL, nullptr},
                         {"quantize", fn(&py_quantize), METH_FASTCALL, nullptr},
                         {"linear_i8", fn(&py_linear_i8), METH_FASTCALL, nullptr},
                         {"workspace", py_workspace, METH_VARARGS, nullptr},
                         {"bind", py_bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rog_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rog_binding(void) { return PyModule_Create(&module); }
