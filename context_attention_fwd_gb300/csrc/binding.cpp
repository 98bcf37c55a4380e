// binding.cpp -- Python marshalling of the calls that a decoding loop makes.
//
// The work of these entry points on a few new tokens takes some microseconds
// on the GPU; describing four tensors and allocating two results from Python
// took sixteen on the host (rotating one token's q and k: 15.6 us a call
// through ctypes, 6.0 through this module, 3 of them on the GPU).  This
// module does that part natively: it checks
// the torch tensors, fills the descriptors of include/ctx_attn.h, allocates
// results that were not given, and calls the C ABI on the current stream.  It
// computes nothing.  Every function returns its results, or the library's
// status code (an int) when the library refused the call; what is wrong with
// a tensor itself is a ValueError.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string.h>

#include <sstream>
#include <string>

#include "../../include/ctx_attn.h"

namespace {

using at::Tensor;

struct Refused {  // becomes a ValueError
    std::string text;
};
template <typename... A>
[[noreturn]] void refuse(const A&... parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw Refused{s.str()};
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, ": expected a tensor");
    return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

// ctx_tensor_t of a logical [B,S,H,D] tensor of this type and device.
ctx_tensor_t describe(const Tensor& t, const char* name, at::ScalarType type, c10::Device dev) {
    if (t.dim() != 4) refuse(name, ": expected a logical [B,S,H,D] tensor, got ", t.dim(), " dims");
    if (t.scalar_type() != type) refuse(name, ": dtype must be ", type, ", got ", t.scalar_type());
    if (t.device() != dev || !dev.is_cuda()) refuse(name, ": on ", t.device(), "; every tensor must be on one CUDA device");
    if (t.stride(3) != 1) refuse(name, ": the D dimension must be contiguous");
    return ctx_tensor_t{t.data_ptr(), t.size(0), t.size(1), t.size(2), t.size(3), t.stride(0), t.stride(1), t.stride(2)};
}

// Allocations go past torch's dispatcher, which has nothing to decide here.
Tensor empty(at::IntArrayRef size, at::ScalarType type, c10::Device dev) {
    return Tensor(at::detail::empty_cuda(size, type, dev, std::nullopt));
}

// A result: the tensor given, or a new one of `like`'s type, shape and storage order.
Tensor result(PyObject* o, const char* name, const Tensor& like, ctx_tensor_t* d) {
    Tensor t;
    if (given(o)) {
        t = tensor(o, name);
    } else {
        const int64_t B = like.size(0), S = like.size(1), H = like.size(2), D = like.size(3);
        const bool bshd = like.stride(0) >= like.stride(1);
        t = Tensor(at::detail::empty_strided_cuda({B, S, H, D}, {bshd ? S * H * D : H * D, bshd ? H * D : B * H * D, D, 1},
                                                  like.scalar_type(), like.device()));
    }
    *d = describe(t, name, like.scalar_type(), like.device());
    return t;
}

Tensor lse_result(PyObject* o, int64_t B, int64_t H, int64_t S, c10::Device dev) {
    if (!given(o)) return empty({B, H, S}, at::kFloat, dev);
    const Tensor& t = tensor(o, "lse");
    if (t.scalar_type() != at::kFloat || t.dim() != 3 || t.size(0) != B || t.size(1) != H || t.size(2) != S ||
        !t.is_contiguous() || t.device() != dev)
        refuse("lse: expected a contiguous float32 tensor of shape (", B, ", ", H, ", ", S, ") on ", dev, ", got ",
               t.scalar_type(), " ", t.sizes(), " on ", t.device());
    return t;
}

struct Scratch {
    Tensor t;
    void* p = nullptr;
    size_t bytes = 0;
};
Scratch scratch(PyObject* o, size_t need, c10::Device dev) {
    Scratch s;
    if (given(o)) {
        s.t = tensor(o, "workspace");
        if (s.t.device() != dev || !s.t.is_contiguous())
            refuse("workspace: expected a contiguous tensor on ", dev, ", got one on ", s.t.device());
        s.bytes = s.t.nbytes();
    } else if (need) {
        s.t = empty({(int64_t)need}, at::kByte, dev);
        s.bytes = need;
    }
    if (s.t.defined()) s.p = s.t.data_ptr();
    return s;
}

ctx_stream_t stream_of(c10::Device dev) {
    return reinterpret_cast<ctx_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

int as_int(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v < INT32_MIN || v > INT32_MAX) refuse(name, ": ", v, " does not fit 32 bits");
    return (int)v;
}
double as_double(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

int row_type(const Tensor& t, const char* name) {
    if (t.dim() != 4) refuse(name, ": expected a logical [B,S,H,D] tensor, got ", t.dim(), " dims");
    switch (t.scalar_type()) {
        case at::kBFloat16: return CTX_DTYPE_BF16;
        case at::kHalf: return CTX_DTYPE_FP16;
        case at::kFloat: return CTX_DTYPE_FP32;
        default: refuse(name, ": dtype must be bfloat16, float16 or float32, got ", t.scalar_type());
    }
}

// ctx_rope_t of a call from its table (the structure without positions, as
// bytes, and the tensor it points into); false without a table.
bool rope_of(PyObject* head, PyObject* turns, PyObject* positions, PyObject* offset, int64_t B, int64_t S,
             c10::Device dev, ctx_rope_t* r) {
    if (!given(head)) {
        if (given(positions)) refuse("positions given without a table");
        return false;
    }
    const Tensor& t = tensor(turns, "table");
    if (t.device() != dev) refuse("table: on ", t.device(), ", the tensors are on ", dev);
    if (!PyBytes_Check(head) || PyBytes_GET_SIZE(head) != (Py_ssize_t)sizeof(ctx_rope_t)) refuse("table: not a RopeTable");
    memcpy(r, PyBytes_AS_STRING(head), sizeof(ctx_rope_t));
    r->turns = static_cast<const uint64_t*>(t.data_ptr());
    if (!given(positions)) {
        if (r->n_axes > 1) refuse("a table with several position axes needs positions");
        r->offset = PyLong_AsLongLong(offset);
        if (r->offset == -1 && PyErr_Occurred()) throw python_error();
        return true;
    }
    const Tensor& p = tensor(positions, "positions");
    if (p.scalar_type() != at::kLong || p.device() != dev)
        refuse("positions: expected int64 on ", dev, ", got ", p.scalar_type(), " on ", p.device());
    int64_t dims = p.dim();
    if (r->n_axes > 1) {
        if (dims < 2 || p.size(dims - 1) != r->n_axes)
            refuse("positions: expected [S, ", r->n_axes, "] or [B, S, ", r->n_axes, "], got ", p.sizes());
        r->pos_stride_axis = p.stride(--dims);
    }
    if (dims == 1 && p.size(0) == S) {
        r->pos_stride_s = p.stride(0);
    } else if (dims == 2 && (p.size(0) == 1 || p.size(0) == B) && p.size(1) == S) {
        r->pos_stride_b = p.size(0) == 1 ? 0 : p.stride(0);
        r->pos_stride_s = p.stride(1);
    } else {
        refuse("positions: ", p.sizes(), " does not fit ", B, " sequences of ", S, " tokens");
    }
    r->positions = static_cast<const int64_t*>(p.data_ptr());
    return true;
}

struct Weights {
    const void* w[2] = {nullptr, nullptr};
    int type = CTX_DTYPE_FP32;
};
Weights weights_of(PyObject* wq, PyObject* wk, int64_t D, c10::Device dev) {
    Weights r;
    PyObject* o[2] = {wq, wk};
    const char* names[2] = {"wq", "wk"};
    int type = -1;
    for (int i = 0; i < 2; ++i) {
        if (!given(o[i])) continue;
        const Tensor& t = tensor(o[i], names[i]);
        const int ty = t.scalar_type() == at::kFloat ? CTX_DTYPE_FP32
                       : t.scalar_type() == at::kHalf ? CTX_DTYPE_FP16
                       : t.scalar_type() == at::kBFloat16 ? CTX_DTYPE_BF16 : -1;
        if (t.dim() != 1 || t.size(0) != D || !t.is_contiguous() || t.device() != dev || ty < 0)
            refuse(names[i], ": expected a contiguous [", D, "] tensor on ", dev, ", got ", t.scalar_type(), " ", t.sizes());
        if (type >= 0 && ty != type) refuse(names[i], ": both weights must have one dtype");
        type = ty;
        r.w[i] = t.data_ptr();
    }
    if (type >= 0) r.type = type;
    return r;
}

PyObject* pack(std::initializer_list<Tensor> ts) {  // undefined tensors become None
    PyObject* tuple = PyTuple_New(ts.size());
    if (!tuple) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o = t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None);
        if (!o) {
            Py_DECREF(tuple);
            throw python_error();
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}
// The library's answer: its status code, or the results.
PyObject* answer(int rc, std::initializer_list<Tensor> ts) { return rc ? PyLong_FromLong(rc) : pack(ts); }

// backward, head, turns, a, b, positions, offset, a_out, b_out
PyObject* rotate(PyObject* const* a) {
    const bool back = as_int(a[0], "backward") != 0;
    const char *na = back ? "dq_out" : "q", *nb = back ? "dk_out" : "k", *noa = back ? "dq" : "q_out",
               *nob = back ? "dk" : "k_out";
    const Tensor& x = tensor(a[3], na);
    const int type = row_type(x, na);
    const c10::Device dev = x.device();
    if (!given(a[1])) refuse("table: a RopeTable is required");
    ctx_tensor_t dx = describe(x, na, x.scalar_type(), dev), dy, ox, oy;
    const bool both = given(a[4]);
    if (both) dy = describe(tensor(a[4], nb), nb, x.scalar_type(), dev);
    ctx_rope_t rope;
    rope_of(a[1], a[2], a[5], a[6], x.size(0), x.size(1), dev, &rope);
    const c10::cuda::CUDAGuard guard(dev);
    Tensor rx = result(a[7], noa, x, &ox), ry;
    if (both) ry = result(a[8], nob, tensor(a[4], nb), &oy);
    else if (given(a[8])) refuse(nob, ": given without ", nb);
    int rc;
    const ctx_stream_t s = stream_of(dev);
    Py_BEGIN_ALLOW_THREADS
    rc = (back ? ctx_rope_bwd : ctx_rope_fwd)(&dx, both ? &dy : nullptr, &rope, (ctx_dtype_t)type, CTX_LAYOUT_BSHD, &ox,
                                              both ? &oy : nullptr, s);
    Py_END_ALLOW_THREADS
    return answer(rc, {rx, ry});
}

// head, turns, q, k, wq, wk, positions, offset, eps, q_out, k_out
PyObject* norm_fwd(PyObject* const* a) {
    const Tensor& q = tensor(a[2], "q");
    const int type = row_type(q, "q");
    const c10::Device dev = q.device();
    ctx_tensor_t dq = describe(q, "q", q.scalar_type(), dev), dk, oq, ok;
    const bool both = given(a[3]);
    if (both) dk = describe(tensor(a[3], "k"), "k", q.scalar_type(), dev);
    const Weights w = weights_of(a[4], a[5], q.size(3), dev);
    ctx_rope_t rope;
    const bool turn = rope_of(a[0], a[1], a[6], a[7], q.size(0), q.size(1), dev, &rope);
    const float eps = (float)as_double(a[8]);
    const c10::cuda::CUDAGuard guard(dev);
    Tensor rq = result(a[9], "q_out", q, &oq), rk;
    if (both) rk = result(a[10], "k_out", tensor(a[3], "k"), &ok);
    else if (given(a[10])) refuse("k_out: given without k");
    int rc;
    const ctx_stream_t s = stream_of(dev);
    Py_BEGIN_ALLOW_THREADS
    rc = ctx_qk_norm_rope_fwd(&dq, both ? &dk : nullptr, w.w[0], w.w[1], (ctx_dtype_t)w.type, eps, turn ? &rope : nullptr,
                              (ctx_dtype_t)type, CTX_LAYOUT_BSHD, &oq, both ? &ok : nullptr, s);
    Py_END_ALLOW_THREADS
    return answer(rc, {rq, rk});
}

Tensor weight_grad(PyObject* o, const char* name, PyObject* w, int64_t D, c10::Device dev) {
    if (!given(o)) return given(w) ? empty({D}, at::kFloat, dev) : Tensor();
    const Tensor& t = tensor(o, name);
    if (!given(w) || t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != D || !t.is_contiguous() || t.device() != dev)
        refuse(name, ": expected a contiguous float32 [", D, "] tensor on ", dev, ", beside its weight");
    return t;
}

// head, turns, dq_out, dk_out, q, k, wq, wk, positions, offset, eps, dq, dk, dwq, dwk, workspace
PyObject* norm_bwd(PyObject* const* a) {
    const bool both = given(a[5]);
    if (both != given(a[3])) refuse("k and dk_out go together");
    const Tensor& q = tensor(a[4], "q");
    const int type = row_type(q, "q");
    const c10::Device dev = q.device();
    const int64_t D = q.size(3);
    ctx_tensor_t dq = describe(q, "q", q.scalar_type(), dev), dk, gq, gk, oq, ok;
    gq = describe(tensor(a[2], "dq_out"), "dq_out", q.scalar_type(), dev);
    if (both) {
        dk = describe(tensor(a[5], "k"), "k", q.scalar_type(), dev);
        gk = describe(tensor(a[3], "dk_out"), "dk_out", q.scalar_type(), dev);
    }
    const Weights w = weights_of(a[6], a[7], D, dev);
    ctx_rope_t rope;
    const bool turn = rope_of(a[0], a[1], a[8], a[9], q.size(0), q.size(1), dev, &rope);
    const float eps = (float)as_double(a[10]);
    const c10::cuda::CUDAGuard guard(dev);
    Tensor rq = result(a[11], "dq", q, &oq), rk;
    if (both) rk = result(a[12], "dk", tensor(a[5], "k"), &ok);
    else if (given(a[12])) refuse("dk: given without k");
    const Tensor wq = weight_grad(a[13], "dwq", a[6], D, dev), wk = weight_grad(a[14], "dwk", a[7], D, dev);
    const bool sums = wq.defined() || wk.defined();
    const Scratch ws = scratch(a[15], sums ? ctx_qk_norm_rope_workspace_size((int)D) : 0, dev);
    int rc;
    const ctx_stream_t s = stream_of(dev);
    float* pq = wq.defined() ? static_cast<float*>(wq.data_ptr()) : nullptr;
    float* pk = wk.defined() ? static_cast<float*>(wk.data_ptr()) : nullptr;
    Py_BEGIN_ALLOW_THREADS
    rc = ctx_qk_norm_rope_bwd(&gq, both ? &gk : nullptr, &dq, both ? &dk : nullptr, w.w[0], w.w[1], (ctx_dtype_t)w.type,
                              eps, turn ? &rope : nullptr, (ctx_dtype_t)type, CTX_LAYOUT_BSHD, &oq, both ? &ok : nullptr,
                              pq, pk, ws.p, ws.bytes, s);
    Py_END_ALLOW_THREADS
    return answer(rc, {rq, rk, wq, wk});
}

const int* offsets_of(PyObject* o) {  // bytes of P + 1 ints, or None
    return given(o) ? reinterpret_cast<const int*>(PyBytes_AS_STRING(o)) : nullptr;
}

// q, k, v, P, offsets, causal, left, right, sinks, scale, out, lse
PyObject* window_fwd(PyObject* const* a) {
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const c10::Device dev = q.device();
    const ctx_tensor_t dq = describe(q, "q", at::kBFloat16, dev), dk = describe(k, "k", at::kBFloat16, dev),
                       dv = describe(v, "v", at::kBFloat16, dev);
    const int P = as_int(a[3], "P"), causal = as_int(a[5], "causal"), left = as_int(a[6], "window"),
              right = as_int(a[7], "window"), sinks = as_int(a[8], "sinks");
    const float scale = (float)as_double(a[9]);
    const c10::cuda::CUDAGuard guard(dev);
    ctx_tensor_t od;
    const Tensor out = result(a[10], "out", q, &od), lse = lse_result(a[11], q.size(0), q.size(2), q.size(1), dev);
    int rc;
    const ctx_stream_t s = stream_of(dev);
    Py_BEGIN_ALLOW_THREADS
    rc = ctx_attn_window_fwd(&dq, &dk, &dv, P, offsets_of(a[4]), CTX_LAYOUT_BSHD, causal, left, right, sinks, scale, &od,
                             static_cast<float*>(lse.data_ptr()), s);
    Py_END_ALLOW_THREADS
    return answer(rc, {out, lse});
}

// q, k, v, out, lse, dout, P, offsets, causal, left, right, sinks, scale, dq, dk, dv, workspace
PyObject* window_bwd(PyObject* const* a) {
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const c10::Device dev = q.device();
    const ctx_tensor_t tq = describe(q, "q", at::kBFloat16, dev), tk = describe(k, "k", at::kBFloat16, dev),
                       tv = describe(tensor(a[2], "v"), "v", at::kBFloat16, dev),
                       to = describe(tensor(a[3], "out"), "out", at::kBFloat16, dev),
                       tg = describe(tensor(a[5], "dout"), "dout", at::kBFloat16, dev);
    if (!given(a[4])) refuse("lse: expected the forward's");
    const Tensor lse = lse_result(a[4], q.size(0), q.size(2), q.size(1), dev);
    const int P = as_int(a[6], "P"), causal = as_int(a[8], "causal"), left = as_int(a[9], "window"),
              right = as_int(a[10], "window"), sinks = as_int(a[11], "sinks");
    const float scale = (float)as_double(a[12]);
    const c10::cuda::CUDAGuard guard(dev);
    ctx_tensor_t oq, ok, ov;
    const Tensor dq = result(a[13], "dq", q, &oq), dk = result(a[14], "dk", k, &ok), dv = result(a[15], "dv", k, &ov);
    auto dim = [](int64_t n) { return n > INT32_MAX ? 0 : (int)n; };  // 0: refused by the library
    const Scratch ws = scratch(a[16], ctx_attn_window_workspace_size(dim(q.size(0)), dim(q.size(1)), dim(q.size(2)),
                                                                     dim(k.size(2)), dim(q.size(3)), P, causal, left, right,
                                                                     sinks), dev);
    int rc;
    const ctx_stream_t s = stream_of(dev);
    Py_BEGIN_ALLOW_THREADS
    rc = ctx_attn_window_bwd(&tq, &tk, &tv, &to, static_cast<const float*>(lse.data_ptr()), &tg, P, offsets_of(a[7]),
                             CTX_LAYOUT_BSHD, causal, left, right, sinks, scale, &oq, &ok, &ov, ws.p, ws.bytes, s);
    Py_END_ALLOW_THREADS
    return answer(rc, {dq, dk, dv});
}

// q, k, v, lengths, left, sinks, scale, out, lse, workspace
PyObject* decode(PyObject* const* a) {
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const c10::Device dev = q.device();
    const ctx_tensor_t dq = describe(q, "q", at::kBFloat16, dev), dk = describe(k, "k", at::kBFloat16, dev),
                       dv = describe(v, "v", at::kBFloat16, dev);
    const int* lengths = nullptr;
    if (given(a[3])) {
        const Tensor& n = tensor(a[3], "lengths");
        if (n.scalar_type() != at::kInt || n.dim() != 1 || n.size(0) != q.size(0) || !n.is_contiguous() || n.device() != dev)
            refuse("lengths: expected a contiguous int32 tensor of shape (", q.size(0), ",) on ", dev, ", got ",
                   n.scalar_type(), " ", n.sizes(), " on ", n.device());
        lengths = static_cast<const int*>(n.data_ptr());
    }
    const int left = as_int(a[4], "window"), sinks = as_int(a[5], "sinks");
    const float scale = (float)as_double(a[6]);
    const c10::cuda::CUDAGuard guard(dev);
    ctx_tensor_t od;
    const Tensor out = result(a[7], "out", q, &od), lse = lse_result(a[8], q.size(0), q.size(2), q.size(1), dev);
    auto dim = [](int64_t n) { return n > INT32_MAX ? 0 : (int)n; };  // 0: refused by the library
    const Scratch ws = scratch(a[9], ctx_attn_decode_workspace_size(dim(q.size(0)), dim(q.size(1)), dim(q.size(2)),
                                                                    dim(k.size(2)), dim(q.size(3)), dim(k.size(1)), left,
                                                                    sinks), dev);
    int rc;
    const ctx_stream_t s = stream_of(dev);
    Py_BEGIN_ALLOW_THREADS
    rc = ctx_attn_decode(&dq, &dk, &dv, lengths, CTX_LAYOUT_BSHD, left, sinks, scale, &od,
                         static_cast<float*>(lse.data_ptr()), ws.p, ws.bytes, s);
    Py_END_ALLOW_THREADS
    return answer(rc, {out, lse});
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return kCall(args);
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define CTX_METHOD(name, args) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<name, args>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {CTX_METHOD(rotate, 9),      CTX_METHOD(norm_fwd, 11),  CTX_METHOD(norm_bwd, 16),
                          CTX_METHOD(window_fwd, 12), CTX_METHOD(window_bwd, 17), CTX_METHOD(decode, 10),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
