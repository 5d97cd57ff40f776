// Argument marshalling of the operators around the gated delta rule: torch tensors in, a call of libkda's C ABI, torch
// tensors out.  It checks the tensors, allocates the results and passes addresses and the device's current stream;
// everything that is computed is computed by libkda, which knows nothing of torch.
//
// These calls take a few microseconds on the GPU, and so do their arguments to check: in Python a decode step's 13
// arguments cost 8 us a call, here under 2.  The entry points come from the loaded library by address (bind), so that
// the bounds-checked build runs through the same code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "kda.h"

namespace {

struct Entry {
    decltype(&kda_qk_norm_fwd) qk_norm_fwd;
    decltype(&kda_qk_norm_bwd_workspace_size) qk_norm_bwd_workspace_size;
    decltype(&kda_qk_norm_bwd) qk_norm_bwd;
    decltype(&kda_gdn_decode_step) gdn_decode_step;
    decltype(&kda_gdn_chunk_bwd_workspace_size) gdn_chunk_bwd_workspace_size;
    decltype(&kda_gdn_chunk_bwd) gdn_chunk_bwd;
    decltype(&kda_quant_fp8) quant_fp8;
    decltype(&kda_norm_gate_fp8) norm_gate_fp8;
    decltype(&kda_out_proj_fp8) out_proj_fp8;
} F;
bool g_bound = false;
PyObject *g_loader = nullptr;  // loads the library and calls bind()

// A Python exception to raise, or (with no type) one that is already set.
struct Refusal {
    PyObject *type;
    std::string text;
};
[[noreturn]] void refuse(PyObject *type, const std::string &text) { throw Refusal{type, text}; }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}
std::string type_text(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}

using Shape = c10::SmallVector<int64_t, 5>;

// The call's first tensor: on a CUDA device.
const at::Tensor &first(PyObject *o, const char *name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}
kda_dtype_t dtype_code(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kFloat) return KDA_F32;
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    refuse(PyExc_TypeError, std::string(name) + ": unsupported dtype " + type_text(t.scalar_type()) + " (float32 or bfloat16)");
}

const at::Tensor &on(PyObject *o, const char *name, int device) {
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).get_device() != device)
        refuse(PyExc_ValueError, std::string(name) + " must be a tensor on cuda:" + std::to_string(device));
    return THPVariable_Unpack(o);
}
void check_type(const at::Tensor &t, const char *name, at::ScalarType dt) {
    if (t.scalar_type() != dt)
        refuse(PyExc_TypeError, std::string(name) + " must be " + type_text(dt) + " (got " + type_text(t.scalar_type()) + ")");
}
// The address of a tensor of the call (NULL for None), which must be as described.
void *need(PyObject *o, const char *name, int device, at::ScalarType dt, at::IntArrayRef shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = on(o, name, device);
    check_type(t, name, dt);
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + " (got " + shape_text(t.sizes()) + ")");
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void *required(PyObject *o, const char *name, int device, at::ScalarType dt, at::IntArrayRef shape) {
    if (o == Py_None) refuse(PyExc_ValueError, std::string(name) + " must be a tensor on cuda:" + std::to_string(device));
    return need(o, name, device, dt, shape);
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refusal{nullptr, ""};
    return v;
}
long integer(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refusal{nullptr, ""};
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refusal{nullptr, ""};
    return v != 0;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType dt, int device) {
    return at::empty(shape, at::TensorOptions().dtype(dt).device(at::kCUDA, (c10::DeviceIndex)device));
}

// Runs a call of the library with the device current and the interpreter released.
template <typename Fn>
kda_status_t call(int device, Fn &&fn) {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    kda_status_t s;
    Py_BEGIN_ALLOW_THREADS
    s = fn();
    Py_END_ALLOW_THREADS
    return s;
}
void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// The workspace of a call: the given tensor, or one allocated for the size the query answers.
template <typename Args, typename Query>
kda_status_t workspace(Args &a, Query query, PyObject *given, int device, at::Tensor &ws) {
    size_t n = 0;
    const kda_status_t s = call(device, [&] { return query(&a, &n); });
    if (s != KDA_OK || n == 0) return s;
    if (given == Py_None) {
        ws = make({(int64_t)n}, at::kByte, device);
    } else {
        ws = on(given, "workspace", device);
        check_type(ws, "workspace", at::kByte);
        if (!ws.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
    }
    a.workspace = ws.data_ptr();
    a.workspace_bytes = (size_t)ws.numel();
    return KDA_OK;
}

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = r ? wrap(t) : nullptr;
        if (!o) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Every function answers its results, or the library's status as an int.
using Body = PyObject *(*)(PyObject *const *);
template <int N, Body body>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments (got %zd)", N, n);
        return nullptr;
    }
    try {
        if (!g_bound) {
            PyObject *r = g_loader ? PyObject_CallNoArgs(g_loader) : nullptr;
            if (!r) {
                if (!PyErr_Occurred()) PyErr_SetString(PyExc_ImportError, "the library is not loaded");
                return nullptr;
            }
            Py_DECREF(r);
        }
        return body(args);
    } catch (const Refusal &e) {
        if (e.type) PyErr_SetString(e.type, e.text.c_str());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// ---------------------------------------------------------------- norms of queries and keys
struct Rows {  // (B, S, H, D) of a (B, S, H, D) or (S, H, D) tensor and its token strides
    int64_t B, S, H, D, b, s;
};
Rows rows_of(const at::Tensor &t, const char *name) {
    const auto n = t.sizes(), st = t.strides();
    const size_t d = n.size();
    if (d != 3 && d != 4)
        refuse(PyExc_ValueError, std::string(name) + " must have shape (B, S, H, D) or (S, H, D) (got " + shape_text(n) + ")");
    Rows r{d == 4 ? n[0] : 1, n[d - 3], n[d - 2], n[d - 1], d == 4 ? st[0] : 0, st[d - 3]};
    if ((r.D > 1 && st[d - 1] != 1) || (r.H > 1 && st[d - 2] != r.D))
        refuse(PyExc_ValueError, std::string(name) + ": the heads and channels of a token must be contiguous");
    if (r.B <= 1) r.b = 0;  // (the stride of a dimension of one says nothing)
    if (r.S <= 1) r.s = 0;
    return r;
}

// a[0 .. 8]: q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved
kda_qk_norm_args qk_args(PyObject *const *a, int &device) {
    const at::Tensor &q = first(a[0], "q");
    device = q.get_device();
    const at::Tensor &k = on(a[1], "k", device);
    kda_qk_norm_args r = {};
    r.dtype = dtype_code(q, "q");
    check_type(k, "k", q.scalar_type());
    const Rows x = rows_of(q, "q"), y = rows_of(k, "k");
    if (x.B != y.B || x.S != y.S || x.D != y.D || q.dim() != k.dim())
        refuse(PyExc_ValueError, "k's shape " + shape_text(k.sizes()) + " does not go with q's " + shape_text(q.sizes()));
    if (x.H > INT32_MAX || y.H > INT32_MAX || x.D > INT32_MAX) refuse(PyExc_ValueError, "more than 2^31 - 1 heads or channels");
    r.B = x.B;
    r.S = x.S;
    r.H_q = (int32_t)x.H;
    r.H_k = (int32_t)y.H;
    r.D = (int32_t)x.D;
    r.q = q.data_ptr();
    r.k = k.data_ptr();
    r.q_stride_b = x.b;
    r.q_stride_s = x.s;
    r.k_stride_b = y.b;
    r.k_stride_s = y.s;
    r.norm = (kda_norm_t)integer(a[2]);
    r.eps = (float)number(a[3]);
    r.q_weight = (const float *)need(a[4], "q_weight", device, at::kFloat, {x.D});
    r.k_weight = (const float *)need(a[5], "k_weight", device, at::kFloat, {x.D});
    if ((a[6] == Py_None) != (a[7] == Py_None)) refuse(PyExc_ValueError, "positions and inv_freq go together");
    if (a[7] != Py_None) {
        r.positions = (const int64_t *)need(a[6], "positions", device, at::kLong, q.sizes().slice(0, q.dim() - 2));
        const int64_t n = on(a[7], "inv_freq", device).numel();
        r.inv_freq = (const float *)need(a[7], "inv_freq", device, at::kFloat, {n});
        if (n > INT32_MAX / 2) refuse(PyExc_ValueError, "inv_freq is too long");
        r.rot_dim = (int32_t)(2 * n);
    }
    r.interleaved = truth(a[8]);
    r.stream = stream_of(device);
    return r;
}

PyObject *qk_norm(PyObject *const *a) {  // .. , out_q, out_k
    int device = 0;
    kda_qk_norm_args r = qk_args(a, device);
    const at::Tensor &q = THPVariable_Unpack(a[0]), &k = THPVariable_Unpack(a[1]);
    at::Tensor oq, ok;
    if (a[9] == Py_None) {
        oq = make(q.sizes(), q.scalar_type(), device);
        r.q_out = oq.data_ptr();
    } else {
        r.q_out = need(a[9], "out_q", device, q.scalar_type(), q.sizes());
        oq = THPVariable_Unpack(a[9]);
    }
    if (a[10] == Py_None) {
        ok = make(k.sizes(), q.scalar_type(), device);
        r.k_out = ok.data_ptr();
    } else {
        r.k_out = need(a[10], "out_k", device, q.scalar_type(), k.sizes());
        ok = THPVariable_Unpack(a[10]);
    }
    const kda_status_t s = call(device, [&] { return F.qk_norm_fwd(&r); });
    return s == KDA_OK ? tuple_of({oq, ok}) : PyLong_FromLong(s);
}

PyObject *qk_norm_bwd(PyObject *const *a) {  // .. , dq_out, dk_out, workspace
    int device = 0;
    kda_qk_norm_bwd_args r = {};
    r.fwd = qk_args(a, device);
    const at::Tensor &q = THPVariable_Unpack(a[0]), &k = THPVariable_Unpack(a[1]);
    const at::Tensor &g = on(a[9], "dq_out", device);
    if (g.scalar_type() != at::kFloat && g.scalar_type() != q.scalar_type())
        refuse(PyExc_TypeError, "dq_out must be torch.float32 or " + type_text(q.scalar_type()) + " (got " +
                                    type_text(g.scalar_type()) + ")");
    r.grad_dtype = g.scalar_type() == at::kFloat ? KDA_F32 : KDA_BF16;
    r.dq_out = need(a[9], "dq_out", device, g.scalar_type(), q.sizes());
    r.dk_out = required(a[10], "dk_out", device, g.scalar_type(), k.sizes());
    const at::Tensor dq = make(q.sizes(), q.scalar_type(), device), dk = make(k.sizes(), q.scalar_type(), device);
    at::Tensor dqw, dkw, ws;
    r.dq = dq.data_ptr();
    r.dk = dk.data_ptr();
    if (r.fwd.q_weight) r.dq_weight = (float *)(dqw = make({r.fwd.D}, at::kFloat, device)).data_ptr();
    if (r.fwd.k_weight) r.dk_weight = (float *)(dkw = make({r.fwd.D}, at::kFloat, device)).data_ptr();
    kda_status_t s = workspace(r, F.qk_norm_bwd_workspace_size, a[11], device, ws);
    if (s == KDA_OK) s = call(device, [&] { return F.qk_norm_bwd(&r); });
    return s == KDA_OK ? tuple_of({dq, dk, dqw, dkw}) : PyLong_FromLong(s);
}

// ---------------------------------------------------------------- the gated delta rule
// Sizes that the library takes as 32 bits.
int32_t i32(int64_t v, const char *name) {
    if (v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " exceeds 2^31 - 1");
    return (int32_t)v;
}
// beta: the lead shape, or that and a last dimension of one.
void *beta_of(PyObject *o, int device, at::ScalarType dt, const Shape &lead) {
    if (THPVariable_Check(o) && THPVariable_Unpack(o).dim() == (int64_t)lead.size() + 1) {
        Shape wide(lead);
        wide.push_back(1);
        return required(o, "beta", device, dt, wide);
    }
    return required(o, "beta", device, dt, lead);
}
int64_t last_dim(PyObject *o, const char *name, int device) {
    const at::Tensor &t = on(o, name, device);
    if (t.dim() < 1) refuse(PyExc_ValueError, std::string(name) + " must have at least one dimension");
    return t.size(-1);
}

// q, k, v, beta, state, z, log_decay, g_min, gate_logits, eps, slots, out, dev_status
PyObject *gdn_decode_step(PyObject *const *a) {
    const at::Tensor &q = first(a[0], "q");
    const int device = q.get_device();
    kda_gdn_decode_args r = {};
    r.dtype = dtype_code(q, "q");
    const at::ScalarType dt = q.scalar_type();
    const int64_t d = q.dim();
    if (d != 3 && d != 4)
        refuse(PyExc_ValueError, "q must have shape (B, H, D_k) or (B, T, H, D_k) (got " + shape_text(q.sizes()) + ")");
    if (!q.is_contiguous()) refuse(PyExc_ValueError, "q must be contiguous");
    const Shape tok(q.sizes().begin(), q.sizes().end() - 1);
    Shape val(tok);
    val.push_back(last_dim(a[2], "v", device));
    r.B = q.size(0);
    r.T = d == 4 ? i32(q.size(1), "T") : 1;
    r.H = i32(q.size(d - 2), "H");
    r.D_k = i32(q.size(d - 1), "D_k");
    r.D_v = i32(val.back(), "D_v");
    r.q = q.data_ptr();
    r.k = required(a[1], "k", device, dt, q.sizes());
    r.v = required(a[2], "v", device, dt, val);
    r.beta = beta_of(a[3], device, dt, tok);
    const at::Tensor &state = on(a[4], "state", device);
    r.num_slots = state.dim() == 4 ? state.size(0) : 0;
    r.state = (float *)need(a[4], "state", device, at::kFloat, {r.num_slots, r.H, r.D_k, r.D_v});
    r.z = need(a[5], "z", device, dt, tok);
    r.log_decay = (const float *)need(a[6], "log_decay", device, at::kFloat, tok);
    r.g_min = (float)number(a[7]);
    r.gate_logits = need(a[8], "gate_logits", device, dt, val);
    r.eps = (float)number(a[9]);
    r.slots = (const int32_t *)need(a[10], "slots", device, at::kInt, {r.B});
    at::Tensor out;
    if (a[11] == Py_None) {
        out = make(val, dt, device);
        r.o = out.data_ptr();
    } else {
        r.o = need(a[11], "out", device, dt, val);
        out = THPVariable_Unpack(a[11]);
    }
    if (a[12] != Py_None) {
        const at::Tensor &st = on(a[12], "dev_status", device);
        r.dev_status = (int32_t *)need(a[12], "dev_status", device, at::kInt, st.sizes());
        if (st.numel() < 1) refuse(PyExc_ValueError, "dev_status is empty");
    }
    r.stream = stream_of(device);
    const kda_status_t s = call(device, [&] { return F.gdn_decode_step(&r); });
    return s == KDA_OK ? wrap(out) : PyLong_FromLong(s);
}

// q, k, v, beta, d_o, z, log_decay, g_min, initial_state, d_final_state, want_d_initial_state, workspace
PyObject *gdn_chunk_bwd(PyObject *const *a) {
    const at::Tensor &q = first(a[0], "q");
    const int device = q.get_device();
    kda_recurrent_bwd_args r = {};
    r.dtype = dtype_code(q, "q");
    const at::ScalarType dt = q.scalar_type();
    if (q.dim() != 4) refuse(PyExc_ValueError, "q must have shape (B, S, H, D_k) (got " + shape_text(q.sizes()) + ")");
    if (!q.is_contiguous()) refuse(PyExc_ValueError, "q must be contiguous");
    const Shape tok(q.sizes().begin(), q.sizes().end() - 1);
    Shape val(tok);
    val.push_back(last_dim(a[2], "v", device));
    const Shape st{tok[0], tok[2], q.size(3), val[3]};
    r.B = tok[0];
    r.S = tok[1];
    r.H = i32(tok[2], "H");
    r.D_k = i32(q.size(3), "D_k");
    r.D_v = i32(val[3], "D_v");
    r.q = q.data_ptr();
    r.k = required(a[1], "k", device, dt, q.sizes());
    r.v = required(a[2], "v", device, dt, val);
    r.beta = beta_of(a[3], device, dt, tok);
    r.d_o = required(a[4], "d_o", device, dt, val);
    r.z = need(a[5], "z", device, dt, tok);
    r.log_decay = (const float *)need(a[6], "log_decay", device, at::kFloat, tok);
    r.g_min = (float)number(a[7]);
    r.initial_state = (const float *)need(a[8], "initial_state", device, at::kFloat, st);
    r.d_final_state = (const float *)need(a[9], "d_final_state", device, at::kFloat, st);
    const at::Tensor dq = make(q.sizes(), at::kFloat, device), dk = make(q.sizes(), at::kFloat, device);
    const at::Tensor dv = make(val, at::kFloat, device), db = make(tok, at::kFloat, device), dz = make(tok, at::kFloat, device);
    at::Tensor ds, ws;
    r.dq = (float *)dq.data_ptr();
    r.dk = (float *)dk.data_ptr();
    r.dv = (float *)dv.data_ptr();
    r.dbeta = (float *)db.data_ptr();
    r.dz = (float *)dz.data_ptr();
    if (truth(a[10])) r.d_initial_state = (float *)(ds = make(st, at::kFloat, device)).data_ptr();
    r.stream = stream_of(device);
    kda_status_t s = workspace(r, F.gdn_chunk_bwd_workspace_size, a[11], device, ws);
    if (s == KDA_OK) s = call(device, [&] { return F.gdn_chunk_bwd(&r); });
    return s == KDA_OK ? tuple_of({dq, dk, dv, db, dz, ds}) : PyLong_FromLong(s);
}

// ---------------------------------------------------------------- the output path in e4m3
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

PyObject *quant_fp8(PyObject *const *a) {  // x, block_rows
    // the scales are sized by what the library gets: 32 bits, which 2^32 + 1 would leave as 1
    const long wide = integer(a[1]);
    const int32_t rows_per = (int32_t)wide;
    if (rows_per != wide) refuse(PyExc_ValueError, "block_rows must be 1 or 128 (got " + std::to_string(wide) + ")");
    const at::Tensor &x = first(a[0], "x");
    const int device = x.get_device();
    const kda_dtype_t code = dtype_code(x, "x");
    if (x.dim() < 1 || (rows_per != 1 && x.dim() != 2))
        refuse(PyExc_ValueError, x.dim() < 1 ? "x must have at least one dimension" : "blocks of several rows need a matrix");
    const void *px = need(a[0], "x", device, x.scalar_type(), x.sizes());
    const int64_t K = x.size(-1), n = K ? x.numel() / K : 0;
    Shape shape(x.sizes().begin(), x.sizes().end());
    shape.back() = blocks128(K);
    if (rows_per > 1) shape[0] = (n + rows_per - 1) / rows_per;
    const at::Tensor x8 = make(x.sizes(), at::kFloat8_e4m3fn, device), sc = make(shape, at::kFloat, device);
    void *st = stream_of(device);
    const kda_status_t s = call(device, [&] {
        return F.quant_fp8(px, code, n, K, rows_per, x8.data_ptr(), (float *)sc.data_ptr(), st);
    });
    return s == KDA_OK ? tuple_of({x8, sc}) : PyLong_FromLong(s);
}

PyObject *norm_gate_fp8(PyObject *const *a) {  // o, gate_logits, eps
    const at::Tensor &o = first(a[0], "o");
    const int device = o.get_device();
    const kda_dtype_t code = dtype_code(o, "o");
    if (o.dim() < 2) refuse(PyExc_ValueError, "o must have shape (..., H, D_v)");
    const void *po = need(a[0], "o", device, o.scalar_type(), o.sizes());
    const void *pg = required(a[1], "gate_logits", device, o.scalar_type(), o.sizes());
    const float eps = (float)number(a[2]);
    const int32_t H = i32(o.size(-2), "H"), Dv = i32(o.size(-1), "D_v");
    const int64_t K = (int64_t)H * Dv, n = K ? o.numel() / K : 0;
    Shape shape(o.sizes().begin(), o.sizes().end() - 1);
    shape.back() = K;
    const at::Tensor x8 = make(shape, at::kFloat8_e4m3fn, device);
    shape.back() = blocks128(K);
    const at::Tensor sc = make(shape, at::kFloat, device);
    void *st = stream_of(device);
    const kda_status_t s = call(device, [&] {
        return F.norm_gate_fp8(po, pg, n, H, Dv, eps, code, x8.data_ptr(), (float *)sc.data_ptr(), st);
    });
    return s == KDA_OK ? tuple_of({x8, sc}) : PyLong_FromLong(s);
}

PyObject *out_proj_fp8(PyObject *const *a) {  // x8, x_scale, W8, W_scale, out dtype code, out
    const at::Tensor &x = first(a[0], "x8");
    const int device = x.get_device();
    const at::Tensor &w = on(a[2], "W8", device);
    if (w.dim() != 2 || x.dim() < 1) refuse(PyExc_ValueError, "W8 must have shape (D_model, K), x8 (..., K)");
    const int64_t M = w.size(0), K = w.size(1), kb = blocks128(K), n = K ? x.numel() / K : 0;
    Shape shape(x.sizes().begin(), x.sizes().end());
    shape.back() = K;
    const void *px = need(a[0], "x8", device, at::kFloat8_e4m3fn, shape);
    shape.back() = kb;
    const float *ps = (const float *)required(a[1], "x_scale", device, at::kFloat, shape);
    const void *pw = need(a[2], "W8", device, at::kFloat8_e4m3fn, {M, K});
    const float *pv = (const float *)required(a[3], "W_scale", device, at::kFloat, {blocks128(M), kb});
    const kda_dtype_t code = (kda_dtype_t)integer(a[4]);
    const at::ScalarType dt = code == KDA_F32 ? at::kFloat : at::kBFloat16;
    shape.back() = M;
    at::Tensor y;
    void *py;
    if (a[5] == Py_None) {
        y = make(shape, dt, device);
        py = y.data_ptr();
    } else {
        py = need(a[5], "out", device, dt, shape);
        y = THPVariable_Unpack(a[5]);
    }
    const int32_t k32 = i32(K, "K"), m32 = i32(M, "D_model");
    void *st = stream_of(device);
    const kda_status_t s = call(device, [&] { return F.out_proj_fp8(px, ps, pw, pv, n, k32, m32, py, code, st); });
    return s == KDA_OK ? wrap(y) : PyLong_FromLong(s);
}

// ---------------------------------------------------------------- module
// bind({name: address}): the entry points of the loaded library.  loader(callable): what loads it and calls bind.
PyObject *bind(PyObject *, PyObject *table) {
    bool ok = true;
    auto get = [&](const char *name, auto &fn) {
        PyObject *v = PyDict_Check(table) ? PyDict_GetItemString(table, name) : nullptr;
        void *p = v ? PyLong_AsVoidPtr(v) : nullptr;
        if (!p) ok = false;
        fn = reinterpret_cast<std::decay_t<decltype(fn)>>(p);
    };
    get("kda_qk_norm_fwd", F.qk_norm_fwd);
    get("kda_qk_norm_bwd_workspace_size", F.qk_norm_bwd_workspace_size);
    get("kda_qk_norm_bwd", F.qk_norm_bwd);
    get("kda_gdn_decode_step", F.gdn_decode_step);
    get("kda_gdn_chunk_bwd_workspace_size", F.gdn_chunk_bwd_workspace_size);
    get("kda_gdn_chunk_bwd", F.gdn_chunk_bwd);
    get("kda_quant_fp8", F.quant_fp8);
    get("kda_norm_gate_fp8", F.norm_gate_fp8);
    get("kda_out_proj_fp8", F.out_proj_fp8);
    if (!ok) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: an entry point is missing");
        return nullptr;
    }
    g_bound = true;
    Py_RETURN_NONE;
}
PyObject *loader(PyObject *, PyObject *fn) {
    Py_INCREF(fn);
    Py_XDECREF(g_loader);
    g_loader = fn;
    Py_RETURN_NONE;
}

#define KDA_FAST(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<n, name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    {"loader", loader, METH_O, nullptr},
    KDA_FAST(qk_norm, 11),
    KDA_FAST(qk_norm_bwd, 12),
    KDA_FAST(gdn_decode_step, 13),
    KDA_FAST(gdn_chunk_bwd, 12),
    KDA_FAST(quant_fp8, 2),
    KDA_FAST(norm_gate_fp8, 3),
    KDA_FAST(out_proj_fp8, 6),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Marshalling of libkda's layer operators.", -1, methods,
                      nullptr,               nullptr,    nullptr,                                    nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
