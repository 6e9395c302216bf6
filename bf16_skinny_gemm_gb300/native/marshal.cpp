// The short way from torch tensors to the decode operators' C calls.
//
// A call for one token runs for 2 to 4 us on the GPU; reading a dozen tensors' attributes from
// Python takes longer than that.  This module does what decode.py does for a well-formed call
// with all its buffers given: the same checks, the same argument structure, the same C call.
// Whatever is not as it should be is left to decode.py (the functions return -1), whose checks
// say what is wrong; nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "sgemm_decode.h"

namespace {

using Fast = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);

sgemm_status_t (*g_norm)(const sgemm_add_rmsnorm_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_append)(const sgemm_latent_append_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_attention)(const sgemm_latent_attention_t *, sgemm_stream_t) = nullptr;

// The device that is current in this call, which all of its tensors have to be on: the library
// launches there.
struct Device {
    c10::DeviceIndex at = -1;
    bool has(const at::Tensor &t) {
        const c10::Device d = t.device();
        if (!d.is_cuda()) return false;
        if (at < 0) at = c10::cuda::current_device();
        return d.index() == at;
    }
};

// A dense tensor on that device, of this type and rank, whose last dimension has unit stride.
struct View {
    Device &here;
    void *p = nullptr;
    const int64_t *n = nullptr, *s = nullptr;  // sizes, strides

    explicit View(Device &d) : here(d) {}
    bool of(PyObject *o, at::ScalarType type, int rank) {
        if (!THPVariable_Check(o)) return false;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided || t.scalar_type() != type || t.dim() != rank || !here.has(t)) return false;
        n = t.sizes().data();
        s = t.strides().data();
        p = t.data_ptr();
        return s[rank - 1] == 1;
    }
    bool of(PyObject *o, at::ScalarType type, int64_t a) { return of(o, type, 1) && n[0] == a; }
    bool of(PyObject *o, at::ScalarType type, int64_t a, int64_t b) { return of(o, type, 2) && n[0] == a && n[1] == b; }
    bool of(PyObject *o, at::ScalarType type, int64_t a, int64_t b, int64_t c) {
        return of(o, type, 3) && n[0] == a && n[1] == b && n[2] == c;
    }
    template <class T>
    T *as() const {
        return static_cast<T *>(p);
    }
};

bool stream_of(PyObject *o, const Device &here, sgemm_stream_t *out) {
    if (o == Py_None) {
        *out = c10::cuda::getCurrentCUDAStream(here.at).stream();
        return true;
    }
    if (!PyLong_Check(o)) return false;
    *out = reinterpret_cast<sgemm_stream_t>(PyLong_AsVoidPtr(o));
    return !PyErr_Occurred();
}

bool int_of(PyObject *o, long long lo, long long hi, long long *out) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    *out = PyLong_AsLongLongAndOverflow(o, &over);
    return !over && *out >= lo && *out <= hi;
}

bool float_of(PyObject *o, float *out) {
    if (!PyFloat_Check(o)) return false;
    *out = static_cast<float>(PyFloat_AS_DOUBLE(o));
    return true;
}

// The call itself, without the interpreter's lock, as through ctypes: a launch waits where the
// stream's queue is full, and what it waits for may need another thread of this program.
template <class Args>
PyObject *launched(sgemm_status_t (*call)(const Args *, sgemm_stream_t), const Args &args, sgemm_stream_t stream) {
    sgemm_status_t status;
    Py_BEGIN_ALLOW_THREADS;
    status = call(&args, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

PyObject *left() { return PyLong_FromLong(-1); }

constexpr long long kMaxInt = 0x7fffffffLL;
const at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI64 = at::kLong, kI32 = at::kInt;

// (x, weight, residual, eps, form, y, scales, residual_out, flags, stream)
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10 || !g_norm) return left();
    sgemm_add_rmsnorm_t g;
    std::memset(&g, 0, sizeof(g));
    Device here;
    View x(here), v(here);
    long long form = 0, flags = 0;
    sgemm_stream_t stream;
    if (!x.of(a[0], kBf16, 2) || x.n[0] < 1 || x.n[1] > kMaxInt || !int_of(a[4], 0, 2, &form) ||
        !int_of(a[8], 0, kMaxInt, &flags) || !float_of(a[3], &g.eps) || !stream_of(a[9], here, &stream))
        return left();
    const int64_t T = x.n[0], D = x.n[1];
    auto ld = [&](const View &w, int64_t width) { return T > 1 ? w.s[0] : width; };
    g.x = x.as<sgemm_bf16_t>();
    g.ldx = ld(x, D);
    if (!v.of(a[1], kBf16, D)) return left();
    g.weight = v.as<sgemm_bf16_t>();
    g.ldr = g.ldro = D;
    if (a[2] != Py_None) {
        if (a[7] == Py_None || !v.of(a[2], kBf16, T, D)) return left();
        g.residual = v.as<sgemm_bf16_t>();
        g.ldr = ld(v, D);
    }
    if (a[7] != Py_None) {
        if (!v.of(a[7], kBf16, T, D)) return left();
        g.residual_out = v.as<sgemm_bf16_t>();
        g.ldro = ld(v, D);
    }
    if (!v.of(a[5], form == SGEMM_NORM_BF16 ? kBf16 : at::kFloat8_e4m3fn, T, D)) return left();
    g.y = v.p;
    g.ldy = ld(v, D);
    if (form != SGEMM_NORM_BF16) {
        const int64_t groups = form == SGEMM_NORM_E4M3_GROUP128 ? (D + 127) / 128 : 1;
        if (!v.of(a[6], kF32, T, groups)) return left();
        g.scales = v.as<float>();
        g.lds = ld(v, groups);
    }
    g.T = T;
    g.D = static_cast<int>(D);
    g.form = static_cast<int>(form);
    g.flags = static_cast<unsigned>(flags);
    return launched(g_norm, g, stream);
}

// (kv, cache, slots, positions, cos_sin, weight, eps, q, q_out, interleaved, flags, stream)
PyObject *latent_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12 || !g_append) return left();
    sgemm_latent_append_t g;
    std::memset(&g, 0, sizeof(g));
    Device here;
    View kv(here), cache(here), cs(here), v(here);
    long long flags = 0;
    sgemm_stream_t stream;
    if (!kv.of(a[0], kBf16, 2) || !cache.of(a[1], kBf16, 3) || !cs.of(a[4], kF32, 2) || !float_of(a[6], &g.eps) ||
        !int_of(a[10], 0, kMaxInt, &flags) || !stream_of(a[11], here, &stream))
        return left();
    const int64_t T = kv.n[0], W = kv.n[1], E = cs.n[1], R = W - E;
    if (T < 1 || R < 1 || W > kMaxInt || cache.n[2] != W || cache.n[1] > kMaxInt) return left();
    g.T = T;
    g.R = static_cast<int>(R);
    g.E = static_cast<int>(E);
    g.kv = kv.as<sgemm_bf16_t>();
    g.ldkv = T > 1 ? kv.s[0] : W;
    g.cache = cache.as<sgemm_bf16_t>();
    g.pages = cache.n[0];
    g.page_size = static_cast<int>(cache.n[1]);
    g.row_stride = cache.n[1] > 1 ? cache.s[1] : W;
    g.page_stride = cache.n[0] > 1 ? cache.s[0] : g.page_size * g.row_stride;
    g.cos_sin = cs.as<float>();
    g.max_position = cs.n[0];
    g.ldcs = cs.n[0] > 1 ? cs.s[0] : E;
    if (!v.of(a[2], kI64, T)) return left();
    g.slots = v.as<long long>();
    if (!v.of(a[3], kI64, T)) return left();
    g.positions = v.as<long long>();
    if (a[5] != Py_None) {
        if (!v.of(a[5], kBf16, R)) return left();
        g.weight = v.as<sgemm_bf16_t>();
    }
    if (a[7] != Py_None) {
        View o(here);
        if (!v.of(a[7], kBf16, 3) || v.n[0] != T || v.n[1] < 1 || v.n[1] > kMaxInt || v.n[2] != E ||
            !o.of(a[8], kBf16, T, v.n[1], E))
            return left();
        g.H = static_cast<int>(v.n[1]);
        g.q = v.as<sgemm_bf16_t>();
        g.q_token = v.s[0];
        g.q_head = v.s[1];
        g.q_out = o.as<sgemm_bf16_t>();
        g.qo_token = o.s[0];
        g.qo_head = o.s[1];
    } else if (a[8] != Py_None) {
        return left();
    }
    g.interleaved = PyObject_IsTrue(a[9]);
    if (g.interleaved < 0) return nullptr;
    g.flags = static_cast<unsigned>(flags);
    return launched(g_append, g, stream);
}

// (q, cache, block_table, seq_lens, rank, scale, cu_q, max_q, out, lse, workspace, flags, stream)
PyObject *latent_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13 || !g_attention) return left();
    sgemm_latent_attention_t g;
    std::memset(&g, 0, sizeof(g));
    Device here;
    View q(here), cache(here), table(here), v(here);
    long long rank = 0, max_q = 0, flags = 0;
    sgemm_stream_t stream;
    if (!q.of(a[0], kBf16, 3) || !cache.of(a[1], kBf16, 3) || !table.of(a[2], kI32, 2) || !int_of(a[4], 1, kMaxInt, &rank) ||
        !float_of(a[5], &g.scale) || !int_of(a[7], 1, kMaxInt, &max_q) || !int_of(a[11], 0, kMaxInt, &flags) ||
        !stream_of(a[12], here, &stream))
        return left();
    const int64_t total = q.n[0], H = q.n[1], W = q.n[2], B = table.n[0];
    if (total < 1 || B < 1 || H > kMaxInt || B > kMaxInt || table.n[1] > kMaxInt || cache.n[1] > kMaxInt || cache.n[2] != W ||
        rank >= W || W > kMaxInt)
        return left();
    g.q = q.as<sgemm_bf16_t>();
    g.q_token = q.s[0];
    g.q_head = q.s[1];
    g.total_q = total;
    g.H = static_cast<int>(H);
    g.R = static_cast<int>(rank);
    g.E = static_cast<int>(W - rank);
    g.cache = cache.as<sgemm_bf16_t>();
    g.pages = cache.n[0];
    g.page_size = static_cast<int>(cache.n[1]);
    g.row_stride = cache.n[1] > 1 ? cache.s[1] : W;
    g.page_stride = cache.n[0] > 1 ? cache.s[0] : g.page_size * g.row_stride;
    g.block_table = table.as<int>();
    g.B = static_cast<int>(B);
    g.table_width = static_cast<int>(table.n[1]);
    g.ldt = B > 1 ? table.s[0] : table.n[1];
    if (!v.of(a[3], kI32, B)) return left();
    g.seq_lens = v.as<int>();
    g.max_q = static_cast<int>(max_q);
    if (a[6] != Py_None) {
        if (!v.of(a[6], kI32, B + 1)) return left();
        g.cu_q = v.as<int>();
    } else if (total != B * max_q) {
        return left();
    }
    if (!v.of(a[8], kBf16, total, H, rank)) return left();
    g.out = v.as<sgemm_bf16_t>();
    g.out_token = v.s[0];
    g.out_head = v.s[1];
    if (a[9] != Py_None) {
        if (!v.of(a[9], kF32, total, H)) return left();
        g.lse = v.as<float>();
        g.lse_token = v.s[0];
    }
    if (!THPVariable_Check(a[10])) return left();
    const at::Tensor &w = THPVariable_Unpack(a[10]);
    if (!here.has(w) || !w.is_contiguous()) return left();
    g.workspace = w.data_ptr();
    g.workspace_bytes = static_cast<long long>(w.nbytes());
    g.flags = static_cast<unsigned>(flags);
    return launched(g_attention, g, stream);
}

// The addresses of the library's functions.
PyObject *bind(PyObject *, PyObject *args) {
    unsigned long long a, b, c;
    if (!PyArg_ParseTuple(args, "KKK", &a, &b, &c)) return nullptr;
    g_norm = reinterpret_cast<decltype(g_norm)>(a);
    g_append = reinterpret_cast<decltype(g_append)>(b);
    g_attention = reinterpret_cast<decltype(g_attention)>(c);
    Py_RETURN_NONE;
}

template <Fast F>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const std::exception &e) {  // a tensor without storage, a stream that cannot be had
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <Fast F>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>));
}

PyMethodDef kMethods[] = {{"bind", &bind, METH_VARARGS, "Set the addresses of the library's functions."},
                          {"add_rmsnorm", fast<&add_rmsnorm>(), METH_FASTCALL, "A status, or -1."},
                          {"latent_append", fast<&latent_append>(), METH_FASTCALL, "A status, or -1."},
                          {"latent_attention", fast<&latent_attention>(), METH_FASTCALL, "A status, or -1."},
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&kModule); }
