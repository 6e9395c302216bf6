// The short way from torch tensors to the decode operators' C calls.
//
// A call for one token runs for 2 to 4 us on the GPU; reading a dozen tensors' attributes from
// Python takes longer than that.  This module does what decode.py does for a well-formed call
// with all its buffers given: the same checks, the same argument structure, the same C call.
// Whatever is not as it should be is left to decode.py (the functions return -1), whose checks
// say what is wrong; nothing is computed here.  The same for the operators of sgemm_layers.h and layers.py.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "sgemm_layers.h"

namespace {

using Fast = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);

sgemm_status_t (*g_norm)(const sgemm_add_rmsnorm_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_append)(const sgemm_latent_append_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_attention)(const sgemm_latent_attention_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_route)(const sgemm_moe_route_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_experts)(const sgemm_moe_experts_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_tree)(const sgemm_latent_attention_t *, const long long *, long long, int, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_step)(const sgemm_linear_step_t *, sgemm_stream_t) = nullptr;
sgemm_status_t (*g_linear)(const sgemm_linear_attention_t *, sgemm_stream_t) = nullptr;

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

// The arguments of attention: (q, cache, block_table, seq_lens, rank, scale, cu_q, max_q, out, lse, workspace,
// flags, stream).  False: left to the checks.
bool attention_of(PyObject *const *a, Device &here, sgemm_latent_attention_t &g, sgemm_stream_t &stream) {
    std::memset(&g, 0, sizeof(g));
    View q(here), cache(here), table(here), v(here);
    long long rank = 0, max_q = 0, flags = 0;
    if (!q.of(a[0], kBf16, 3) || !cache.of(a[1], kBf16, 3) || !table.of(a[2], kI32, 2) || !int_of(a[4], 1, kMaxInt, &rank) ||
        !float_of(a[5], &g.scale) || !int_of(a[7], 1, kMaxInt, &max_q) || !int_of(a[11], 0, kMaxInt, &flags) ||
        !stream_of(a[12], here, &stream))
        return false;
    const int64_t total = q.n[0], H = q.n[1], W = q.n[2], B = table.n[0];
    if (total < 1 || B < 1 || H > kMaxInt || B > kMaxInt || table.n[1] > kMaxInt || cache.n[1] > kMaxInt || cache.n[2] != W ||
        rank >= W || W > kMaxInt)
        return false;
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
    if (!v.of(a[3], kI32, B)) return false;
    g.seq_lens = v.as<int>();
    g.max_q = static_cast<int>(max_q);
    if (a[6] != Py_None) {
        if (!v.of(a[6], kI32, B + 1)) return false;
        g.cu_q = v.as<int>();
    } else if (total != B * max_q) {
        return false;
    }
    if (!v.of(a[8], kBf16, total, H, rank)) return false;
    g.out = v.as<sgemm_bf16_t>();
    g.out_token = v.s[0];
    g.out_head = v.s[1];
    if (a[9] != Py_None) {
        if (!v.of(a[9], kF32, total, H)) return false;
        g.lse = v.as<float>();
        g.lse_token = v.s[0];
    }
    if (!THPVariable_Check(a[10])) return false;
    const at::Tensor &w = THPVariable_Unpack(a[10]);
    if (!here.has(w) || !w.is_contiguous()) return false;
    g.workspace = w.data_ptr();
    g.workspace_bytes = static_cast<long long>(w.nbytes());
    g.flags = static_cast<unsigned>(flags);
    return true;
}

PyObject *latent_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    sgemm_latent_attention_t g;
    Device here;
    sgemm_stream_t stream;
    if (n != 13 || !g_attention || !attention_of(a, here, g, stream)) return left();
    return launched(g_attention, g, stream);
}

// The same, then tree.
PyObject *latent_tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    sgemm_latent_attention_t g;
    Device here;
    sgemm_stream_t stream;
    if (n != 14 || !g_tree || !attention_of(a, here, g, stream)) return left();
    View v(here);
    if (!v.of(a[13], kI64, 2) || v.n[0] != g.total_q || v.n[1] > kMaxInt) return left();
    const long long ld = g.total_q > 1 ? v.s[0] : v.n[1];
    sgemm_status_t status;
    Py_BEGIN_ALLOW_THREADS;
    status = g_tree(&g, v.as<long long>(), ld, static_cast<int>(v.n[1]), stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

// A contiguous tensor of scratch.
bool scratch_of(PyObject *o, Device &here, void **p, long long *bytes) {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor &w = THPVariable_Unpack(o);
    if (!here.has(w) || !w.is_contiguous()) return false;
    *p = w.data_ptr();
    *bytes = static_cast<long long>(w.nbytes());
    return true;
}

// (x, w, k, bias, scoring, renormalize, scale, ids, weights, flags, stream)
PyObject *moe_route(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 11 || !g_route) return left();
    sgemm_moe_route_t g;
    std::memset(&g, 0, sizeof(g));
    Device here;
    View x(here), w(here), v(here);
    long long k = 0, scoring = 0, flags = 0;
    sgemm_stream_t stream;
    if (!x.of(a[0], kBf16, 2) || x.n[0] < 1 || x.n[1] > kMaxInt || !w.of(a[1], kBf16, 2) || w.n[1] != x.n[1] || w.n[0] < 1 ||
        w.n[0] > kMaxInt || !int_of(a[2], 1, kMaxInt, &k) || !int_of(a[4], 0, 1, &scoring) || !float_of(a[6], &g.scale) ||
        !int_of(a[9], 0, kMaxInt, &flags) || !stream_of(a[10], here, &stream))
        return left();
    const int64_t T = x.n[0], D = x.n[1], E = w.n[0], wide = (D + 7) / 8 * 8;
    g.x = x.as<sgemm_bf16_t>();
    g.ldx = T > 1 ? x.s[0] : wide;
    g.w = w.as<sgemm_bf16_t>();
    g.ldw = E > 1 ? w.s[0] : wide;
    if (a[3] != Py_None) {
        if (!v.of(a[3], kF32, E)) return left();
        g.bias = v.as<float>();
    }
    if (!v.of(a[7], kI32, T, k)) return left();
    g.ids = v.as<int>();
    g.ldi = T > 1 ? v.s[0] : k;
    if (!v.of(a[8], kF32, T, k)) return left();
    g.weights = v.as<float>();
    g.ldwt = T > 1 ? v.s[0] : k;
    g.T = T;
    g.D = static_cast<int>(D);
    g.E = static_cast<int>(E);
    g.k = static_cast<int>(k);
    g.scoring = static_cast<int>(scoring);
    g.renormalize = PyObject_IsTrue(a[5]);
    if (g.renormalize < 0) return nullptr;
    g.flags = static_cast<unsigned>(flags);
    return launched(g_route, g, stream);
}

// (x, w_gate_up, w_down, ids, weights, y, workspace, flags, stream)
PyObject *moe_experts(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9 || !g_experts) return left();
    sgemm_moe_experts_t g;
    std::memset(&g, 0, sizeof(g));
    Device here;
    View x(here), gu(here), dn(here), v(here);
    long long flags = 0;
    sgemm_stream_t stream;
    if (!x.of(a[0], kBf16, 2) || x.n[0] < 1 || x.n[0] > kMaxInt || x.n[1] > kMaxInt || !gu.of(a[1], kBf16, 3) || gu.n[0] < 1 ||
        gu.n[0] > kMaxInt || gu.n[1] < 2 || gu.n[1] % 2 || gu.n[1] > kMaxInt || gu.n[2] != x.n[1] ||
        !dn.of(a[2], kBf16, gu.n[0], x.n[1], gu.n[1] / 2) || !v.of(a[3], kI32, 2) || v.n[0] != x.n[0] || v.n[1] > kMaxInt ||
        !int_of(a[7], 0, kMaxInt, &flags) || !stream_of(a[8], here, &stream))
        return left();
    const int64_t T = x.n[0], D = x.n[1], E = gu.n[0], F = gu.n[1] / 2, k = v.n[1];
    g.x = x.as<sgemm_bf16_t>();
    g.ldx = T > 1 ? x.s[0] : (D + 7) / 8 * 8;
    g.w_gate_up = gu.as<sgemm_bf16_t>();
    g.gu_row = gu.s[1];
    g.gu_expert = E > 1 ? gu.s[0] : 2 * F * gu.s[1];
    g.w_down = dn.as<sgemm_bf16_t>();
    g.dn_row = dn.s[1];
    g.dn_expert = E > 1 ? dn.s[0] : D * dn.s[1];
    g.ids = v.as<int>();
    g.ldi = T > 1 ? v.s[0] : k;
    if (!v.of(a[4], kF32, T, k)) return left();
    g.weights = v.as<float>();
    g.ldwt = T > 1 ? v.s[0] : k;
    if (!v.of(a[5], kBf16, T, D)) return left();
    g.y = v.as<sgemm_bf16_t>();
    g.ldy = T > 1 ? v.s[0] : D;
    if (!scratch_of(a[6], here, &g.workspace, &g.workspace_bytes)) return left();
    g.T = static_cast<int>(T);
    g.D = static_cast<int>(D);
    g.F = static_cast<int>(F);
    g.E = static_cast<int>(E);
    g.k = static_cast<int>(k);
    g.flags = static_cast<unsigned>(flags);
    return launched(g_experts, g, stream);
}

// What both forms of linear attention have: q, k, v, g, state, and out.
template <class Args>
bool linear_of(PyObject *const *a, PyObject *o, Device &here, Args &g, int64_t *tokens) {
    View q(here), v(here), s(here), w(here);
    if (!q.of(a[0], kBf16, 3) || !v.of(a[2], kBf16, 3) || !s.of(a[4], kF32, 4)) return false;
    const int64_t N = q.n[0], Hk = q.n[1], Dk = q.n[2], Hv = v.n[1], Dv = v.n[2];
    if (N < 1 || v.n[0] != N || Hk < 1 || Hk > kMaxInt || Hv < 1 || Hv > kMaxInt || Dk > kMaxInt || Dv > kMaxInt || s.n[1] != Hv ||
        s.n[2] != Dk || s.n[3] != Dv || s.s[2] != Dv)
        return false;
    auto tok = [&](const View &x) { return N > 1 ? x.s[0] : 0; };
    g.q = q.template as<sgemm_bf16_t>();
    g.q_token = tok(q);
    g.q_head = Hk > 1 ? q.s[1] : 0;
    g.v = v.template as<sgemm_bf16_t>();
    g.v_token = tok(v);
    g.v_head = Hv > 1 ? v.s[1] : 0;
    g.state = s.template as<float>();
    g.s_slot = s.n[0] > 1 ? s.s[0] : 0;
    g.s_head = Hv > 1 ? s.s[1] : 0;
    g.pool = s.n[0];
    if (!w.of(a[1], kBf16, N, Hk, Dk)) return false;
    g.k = w.template as<sgemm_bf16_t>();
    g.k_token = tok(w);
    g.k_head = Hk > 1 ? w.s[1] : 0;
    if (!THPVariable_Check(a[3])) return false;
    const at::Tensor &d = THPVariable_Unpack(a[3]);
    if (d.layout() != at::kStrided || d.scalar_type() != kF32 || d.dim() != 2 || d.size(0) != N || d.size(1) != Hv || !here.has(d)) return false;
    g.g = static_cast<const float *>(d.data_ptr());
    g.g_token = N > 1 ? d.stride(0) : 0;
    g.g_head = Hv > 1 ? d.stride(1) : 0;
    if (!w.of(o, kBf16, N, Hv, Dv)) return false;
    g.out = w.template as<sgemm_bf16_t>();
    g.o_token = tok(w);
    g.o_head = Hv > 1 ? w.s[1] : 0;
    g.Hk = static_cast<int>(Hk);
    g.Hv = static_cast<int>(Hv);
    g.Dk = static_cast<int>(Dk);
    g.Dv = static_cast<int>(Dv);
    *tokens = N;
    return true;
}

// (q, k, v, g, state, slots, scale, out, flags, stream)
PyObject *linear_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10 || !g_step) return left();
    sgemm_linear_step_t g;
    std::memset(&g, 0, sizeof(g));
    Device here;
    View v(here);
    long long flags = 0;
    int64_t B = 0;
    sgemm_stream_t stream;
    if (!linear_of(a, a[7], here, g, &B) || !v.of(a[5], kI64, B) || !float_of(a[6], &g.scale) ||
        !int_of(a[8], 0, kMaxInt, &flags) || !stream_of(a[9], here, &stream))
        return left();
    g.slots = v.as<long long>();
    g.B = B;
    g.flags = static_cast<unsigned>(flags);
    return launched(g_step, g, stream);
}

// (q, k, v, g, state, slots, cu, scale, fresh, out, workspace, flags, stream)
PyObject *linear_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13 || !g_linear) return left();
    sgemm_linear_attention_t g;
    std::memset(&g, 0, sizeof(g));
    Device here;
    View v(here);
    long long flags = 0;
    int64_t N = 0;
    sgemm_stream_t stream;
    if (!linear_of(a, a[9], here, g, &N) || !v.of(a[5], kI64, 1) || v.n[0] < 1 || !float_of(a[7], &g.scale) ||
        !int_of(a[11], 0, kMaxInt, &flags) || !stream_of(a[12], here, &stream))
        return left();
    const int64_t B = v.n[0];
    g.N = N;
    g.B = B;
    g.slots = v.as<long long>();
    if (!v.of(a[6], kI32, B + 1)) return left();
    g.cu = v.as<int>();
    if (a[8] != Py_None) {
        if (!v.of(a[8], kI32, B)) return left();
        g.fresh = v.as<int>();
    }
    if (!scratch_of(a[10], here, &g.workspace, &g.workspace_bytes)) return left();
    g.flags = static_cast<unsigned>(flags);
    return launched(g_linear, g, stream);
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

// Those of the operators of sgemm_layers.h.
PyObject *bind_layers(PyObject *, PyObject *args) {
    unsigned long long a, b, c, d, e;
    if (!PyArg_ParseTuple(args, "KKKKK", &a, &b, &c, &d, &e)) return nullptr;
    g_route = reinterpret_cast<decltype(g_route)>(a);
    g_experts = reinterpret_cast<decltype(g_experts)>(b);
    g_tree = reinterpret_cast<decltype(g_tree)>(c);
    g_step = reinterpret_cast<decltype(g_step)>(d);
    g_linear = reinterpret_cast<decltype(g_linear)>(e);
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
                          {"bind_layers", &bind_layers, METH_VARARGS, "The same for the layers' operators."},
                          {"moe_route", fast<&moe_route>(), METH_FASTCALL, "A status, or -1."},
                          {"moe_experts", fast<&moe_experts>(), METH_FASTCALL, "A status, or -1."},
                          {"latent_tree_attention", fast<&latent_tree_attention>(), METH_FASTCALL, "A status, or -1."},
                          {"linear_step", fast<&linear_step>(), METH_FASTCALL, "A status, or -1."},
                          {"linear_attention", fast<&linear_attention>(), METH_FASTCALL, "A status, or -1."},
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&kModule); }
