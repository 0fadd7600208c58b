// The Python side of csa2_linear_fp4, csa2_norm_rope and csa2_dense_attn: argument checks and marshalling
// from PyTorch tensors to the C ABI.  These calls run for a few microseconds on the GPU, so what a call costs
// on the host counts: done here, a call takes a third of the time that checking in Python and ctypes take.
// The module knows the library's functions by the addresses that bind() is given, so that it calls the
// same library that the rest of the binding has loaded.
//
// Every function checks types, shapes and strides (ValueError), and returns either its outputs or, where the
// library refuses or fails, its status as an int.
#include <Python.h>

#include <ATen/MemoryOverlap.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/csa2.h"

namespace {

decltype(&csa2_linear_fp4) f_linear = nullptr;
decltype(&csa2_norm_rope) f_rope = nullptr;
decltype(&csa2_dense_attn) f_dense = nullptr;
decltype(&csa2_workspace_size) f_ws = nullptr;

struct Bad {                                     // a refused argument
    const char* what;
};
void need(bool ok, const char* what) {
    if (!ok) throw Bad{what};
}
const at::Tensor& tensor(PyObject* o, const char* what) {
    need(THPVariable_Check(o), what);
    return THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_none(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

// every given tensor on the current device (the last check: it is the one that needs a GPU)
template <typename... T>
void on_device(const T*... t) {
    const auto one = [](const at::Tensor* v) { return v == nullptr || v->is_cuda(); };
    need((one(t) && ...), "tensors on the GPU");
    const auto here = c10::cuda::current_device();
    const auto same = [&](const at::Tensor* v) { return v == nullptr || v->get_device() == here; };
    need((same(t) && ...), "tensors on the current device");
}

const at::Tensor* ws_or_none(PyObject* o) {
    const at::Tensor* t = tensor_or_none(o, "ws: a tensor");
    need(t == nullptr || t->is_contiguous(), "ws: contiguous");
    return t;
}
// an output's rows lie apart (several blocks would write one row)
void rows_apart(const at::Tensor& t) {
    need(at::has_internal_overlap(t) != at::MemOverlap::Yes, "an output's rows: apart from each other");
}

int type_of(const at::Tensor& t, const char* what) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return CSA2_BF16;
        case at::kHalf: return CSA2_F16;
        case at::kFloat: return CSA2_F32;
        default: throw Bad{what};
    }
}
at::ScalarType dtype_or(PyObject* o, at::ScalarType other) {
    if (o == Py_None) return other;
    need(THPDtype_Check(o), "out_dtype: a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad{nullptr};
    return v;
}
int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad{nullptr};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Bad{nullptr};
    return v != 0;
}
// the given cudaStream_t, or PyTorch's current one
cudaStream_t stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Bad{nullptr};
    return reinterpret_cast<cudaStream_t>(p);
}

// The workspace of one call: the given tensor, or scratch from PyTorch's allocator for the stream that the
// call runs on (a tensor would belong to the current stream, and be given to other work there while this
// stream still uses it).  Freed as soon as the call is enqueued, it goes to later work of that stream alone.
struct Workspace {
    void* p = nullptr;
    size_t n = 0;
    bool own = false;
    void given(const at::Tensor& t) { p = t.data_ptr(), n = (size_t)t.nbytes(); }     // (contiguous: all of it is there)
    void scratch(size_t bytes, cudaStream_t st) {
        if (bytes == 0) return;
        p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, st);
        n = bytes, own = true;
    }
    ~Workspace() {
        if (own) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
};

PyObject* out_of(const at::Tensor* given, PyObject* o, const at::Tensor& made) {
    if (given == nullptr) return THPVariable_Wrap(made);
    Py_INCREF(o);
    return o;
}

// linear_fp4(x, codes, scales, alpha, out, out_dtype, ws, stream)
PyObject* linear(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x: a tensor"), &codes = tensor(a[1], "codes: a tensor"),
                     &scales = tensor(a[2], "scales: a tensor");
    const int64_t nd = x.dim();
    need((nd == 2 || nd == 3) && codes.dim() == nd && scales.dim() == nd,
         "x, codes and scales: [T, n_in] with a matrix, or [T, G, n_in] with one per group");
    const int64_t T = x.size(0), G = nd == 3 ? x.size(1) : 1, n_in = x.size(nd - 1), n_out = codes.size(nd - 2);
    need(n_in % 16 == 0 && codes.size(nd - 1) * 2 == n_in && scales.size(nd - 1) * 16 == n_in && scales.size(nd - 2) == n_out &&
             (nd == 2 || (codes.size(0) == G && scales.size(0) == G)),
         "codes [.., n_out, n_in/2] and scales [.., n_out, n_in/16] of x [.., n_in], n_in a multiple of 16");
    need(codes.scalar_type() == at::kByte && scales.scalar_type() == at::kByte && codes.is_contiguous() && scales.is_contiguous(),
         "codes and scales: contiguous uint8");
    const int x_type = type_of(x, "x: bf16, fp16 or fp32");
    const at::Tensor* given = tensor_or_none(a[4], "out: a tensor");
    at::Tensor made;
    if (given == nullptr) {
        const at::ScalarType t = dtype_or(a[5], x.scalar_type());
        made = nd == 3 ? at::empty({T, G, n_out}, x.options().dtype(t)) : at::empty({T, n_out}, x.options().dtype(t));
    } else {
        need(given->dim() == nd && given->size(0) == T && (nd == 2 || given->size(1) == G) && given->size(nd - 1) == n_out &&
                 (a[5] == Py_None || given->scalar_type() == dtype_or(a[5], at::kFloat)),
             "out [.., n_out] with the leading sizes of x");
    }
    const at::Tensor& y = given ? *given : made;
    const int y_type = type_of(y, "out: bf16, fp16 or fp32");
    need((x.stride(nd - 1) == 1 || n_in == 0) && (n_out <= 1 || y.stride(nd - 1) == 1), "rows of x and out: contiguous");
    need(T <= INT32_MAX && G <= INT32_MAX && n_in <= INT32_MAX && n_out <= INT32_MAX, "sizes of 31 bits");
    const double alpha = number(a[3]);
    rows_apart(y);
    const at::Tensor* given_ws = ws_or_none(a[6]);
    on_device(&x, &codes, &scales, &y, given_ws);
    const cudaStream_t st = stream_of(a[7]);
    Workspace ws;
    if (given_ws != nullptr)
        ws.given(*given_ws);
    else
        ws.scratch(f_ws(CSA2_OP_LINEAR_FP4, (int32_t)T, (int32_t)G, x_type, 0, n_in), st);
    const int status = f_linear(x.data_ptr(), x_type, x.stride(0), nd == 3 ? x.stride(1) : 0, (int32_t)T, (int32_t)G,
                                (int32_t)n_in, (int32_t)n_out, (const uint8_t*)codes.data_ptr(),
                                (const uint8_t*)scales.data_ptr(), (float)alpha, y.data_ptr(), y_type, y.stride(0),
                                nd == 3 ? y.stride(1) : 0, ws.p, ws.n, st);
    return status ? PyLong_FromLong(status) : out_of(given, a[4], made);
}

csa2_head_rows rows_of(const at::Tensor& x, const at::Tensor& y, const at::Tensor* w, int64_t T, int64_t d) {
    need(x.dim() == 3 && x.size(0) == T && x.size(2) == d && y.sizes() == x.sizes(), "a head set and its output: [T, heads, d]");
    need(x.stride(2) == 1 && y.stride(2) == 1, "rows of a head set and its output: contiguous");
    rows_apart(y);
    need(x.size(1) <= INT32_MAX, "sizes of 31 bits");
    need(w == nullptr || (w->scalar_type() == at::kFloat && w->dim() == 1 && w->size(0) == d && w->is_contiguous()),
         "weights: contiguous fp32 [d]");
    return csa2_head_rows{x.data_ptr(), y.data_ptr(), w ? (const float*)w->data_ptr() : nullptr, x.stride(0), x.stride(1),
                          y.stride(0), y.stride(1), (int32_t)x.size(1)};
}

// norm_rope(q, pos, inv_freq, q_weight, k, k_weight, eps, norm, halves, inverse, q_out, k_out, out_dtype, stream)
PyObject* rope(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0], "q: a tensor");
    need(q.dim() == 3, "q: [T, heads, d]");
    const int64_t T = q.size(0), d = q.size(2);
    const at::Tensor *pos = tensor_or_none(a[1], "pos: a tensor"), *freq = tensor_or_none(a[2], "inv_freq: a tensor"),
                     *qw = tensor_or_none(a[3], "q_weight: a tensor"), *k = tensor_or_none(a[4], "k: a tensor"),
                     *kw = tensor_or_none(a[5], "k_weight: a tensor"), *qg = tensor_or_none(a[10], "q_out: a tensor"),
                     *kg = tensor_or_none(a[11], "k_out: a tensor");
    int64_t d_rot = 0;
    if (freq != nullptr) {
        d_rot = 2 * freq->numel();
        need(freq->scalar_type() == at::kFloat && freq->is_contiguous() && pos != nullptr && pos->scalar_type() == at::kLong &&
                 pos->dim() == 1 && pos->size(0) == T && pos->is_contiguous(),
             "inv_freq: contiguous fp32; pos: contiguous int64 [T]");
    }
    at::Tensor qm, km;
    if (qg == nullptr) qm = at::empty(q.sizes(), q.options().dtype(dtype_or(a[12], q.scalar_type())));
    const at::Tensor& qo = qg ? *qg : qm;
    const int x_type = type_of(q, "q: bf16, fp16 or fp32"), y_type = type_of(qo, "q_out: bf16, fp16 or fp32");
    need(a[12] == Py_None || qo.scalar_type() == dtype_or(a[12], at::kFloat), "q_out: of out_dtype");
    need(T <= INT32_MAX && d <= INT32_MAX && d_rot <= INT32_MAX, "sizes of 31 bits");
    const csa2_head_rows rq = rows_of(q, qo, qw, T, d);
    csa2_head_rows rk{};
    if (k != nullptr) {
        if (kg == nullptr) km = at::empty(k->sizes(), k->options().dtype(qo.scalar_type()));
        const at::Tensor& ko = kg ? *kg : km;
        need(k->scalar_type() == q.scalar_type() && ko.scalar_type() == qo.scalar_type(), "k has the type of q, k_out that of q_out");
        rk = rows_of(*k, ko, kw, T, d);
    }
    const int flags = (truth(a[8]) ? CSA2_ROPE_HALVES : 0) | (truth(a[9]) ? CSA2_ROPE_INVERSE : 0) |
                      (truth(a[7]) ? 0 : CSA2_ROPE_NO_NORM);
    const double eps = number(a[6]);
    on_device(&q, pos, freq, qw, k, kw, &qo, k ? (kg ? kg : &km) : nullptr);
    const int status = f_rope(&rq, k ? &rk : nullptr, x_type, y_type, (int32_t)T, (int32_t)d, (int32_t)d_rot,
                              d_rot ? (const int64_t*)pos->data_ptr() : nullptr, d_rot ? (const float*)freq->data_ptr() : nullptr,
                              (float)eps, flags, stream_of(a[13]));
    if (status) return PyLong_FromLong(status);
    PyObject* first = out_of(qg, a[10], qm);
    PyObject* second = k ? out_of(kg, a[11], km) : (Py_INCREF(Py_None), Py_None);
    PyObject* both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
}

// dense_attn(lat_codes, lat_scales, ratio, q, q_pos, swa, swa_pos0, scale, out, out_dtype, lse, want_lse, ws, stream)
PyObject* dense(PyObject* const* a) {
    const at::Tensor &codes = tensor(a[0], "lat_codes: a tensor"), &scales = tensor(a[1], "lat_scales: a tensor"),
                     &q = tensor(a[3], "q: a tensor"), &pos = tensor(a[4], "q_pos: a tensor");
    need(codes.scalar_type() == at::kByte && scales.scalar_type() == at::kByte && codes.dim() == 3 && scales.dim() == 3 &&
             codes.size(2) == 256 && scales.size(2) == 32 && codes.size(0) == scales.size(0) && codes.size(1) == scales.size(1) &&
             codes.is_contiguous() && scales.is_contiguous(),
         "the cache's latent planes: contiguous uint8 [batch, capacity, 256] and [batch, capacity, 32]");
    const int64_t B = codes.size(0), cap = codes.size(1);
    need(q.scalar_type() == at::kBFloat16 && q.dim() == 4 && q.size(0) == B && q.size(3) == 512 && q.is_contiguous(),
         "q: contiguous bf16 [batch, n_q, heads, 512]");
    const int64_t Q = q.size(1), H = q.size(2);
    need(pos.scalar_type() == at::kLong && pos.dim() == 2 && pos.size(0) == B && pos.size(1) == Q && pos.is_contiguous(),
         "q_pos: contiguous int64 [batch, n_q]");
    const at::Tensor *swa = tensor_or_none(a[5], "swa: a tensor"), *pos0 = tensor_or_none(a[6], "swa_pos0: a tensor"),
                     *given = tensor_or_none(a[8], "out: a tensor"), *lse_given = tensor_or_none(a[10], "lse: a tensor");
    need(swa == nullptr || (swa->scalar_type() == at::kBFloat16 && swa->dim() == 3 && swa->size(0) == B && swa->size(2) == 512 &&
                            swa->size(1) <= INT32_MAX && swa->is_contiguous()),
         "swa: contiguous bf16 [batch, swa_len, 512]");
    need(pos0 == nullptr || (pos0->scalar_type() == at::kLong && pos0->dim() == 1 && pos0->size(0) == B && pos0->is_contiguous()),
         "swa_pos0: contiguous int64 [batch]");
    need(B <= INT32_MAX && cap <= INT32_MAX && Q <= INT32_MAX && H <= INT32_MAX, "sizes of 31 bits");
    at::Tensor made, lse_made;
    if (given == nullptr) made = at::empty(q.sizes(), q.options().dtype(dtype_or(a[9], at::kBFloat16)));
    const at::Tensor& o = given ? *given : made;
    const int o_type = type_of(o, "out: bf16, fp16 or fp32");
    need(o.sizes() == q.sizes() && o.is_contiguous(), "out: contiguous, the shape of q");
    if (lse_given == nullptr && truth(a[11])) lse_made = at::empty({B, Q, H}, q.options().dtype(at::kFloat));
    const at::Tensor* lse = lse_given ? lse_given : lse_made.defined() ? &lse_made : nullptr;
    need(lse == nullptr || (lse->scalar_type() == at::kFloat && lse->dim() == 3 && lse->size(0) == B && lse->size(1) == Q &&
                            lse->size(2) == H && lse->is_contiguous()),
         "lse: contiguous fp32 [batch, n_q, heads]");
    const double scale = number(a[7]);
    const csa2_cache cache{(uint8_t*)codes.data_ptr(), (uint8_t*)scales.data_ptr(), nullptr, nullptr, (int32_t)B, (int32_t)cap,
                           512, 128, (int32_t)whole(a[2])};
    const at::Tensor* given_ws = ws_or_none(a[12]);
    on_device(&codes, &scales, &q, &pos, swa, pos0, &o, lse, given_ws);
    const cudaStream_t st = stream_of(a[13]);
    Workspace ws;
    if (given_ws != nullptr)
        ws.given(*given_ws);
    else
        ws.scratch(f_ws(CSA2_OP_DENSE_ATTN, (int32_t)B, (int32_t)Q, (int32_t)H, 0, cap), st);
    const int status = f_dense(&cache, (const uint16_t*)q.data_ptr(), (int32_t)Q, (int32_t)H, (const int64_t*)pos.data_ptr(),
                               swa ? (const uint16_t*)swa->data_ptr() : nullptr,
                               pos0 ? (const int64_t*)pos0->data_ptr() : nullptr, swa ? (int32_t)swa->size(1) : 0, (float)scale,
                               o.data_ptr(), o_type, lse ? (float*)lse->data_ptr() : nullptr, ws.p, ws.n, st);
    if (status) return PyLong_FromLong(status);
    PyObject* first = out_of(given, a[8], made);
    PyObject* second = lse ? out_of(lse_given, a[10], lse_made) : (Py_INCREF(Py_None), Py_None);
    PyObject* both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
}

// nothing thrown leaves a C entry
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        if (f_ws == nullptr) throw Bad{"the library is not loaded"};
        return F(a);
    } catch (const Bad& e) {
        if (e.what != nullptr) PyErr_SetString(PyExc_ValueError, e.what);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// bind(linear, norm_rope, dense_attn, workspace_size): the library's functions, as addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "four addresses");
        return nullptr;
    }
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    f_linear = reinterpret_cast<decltype(f_linear)>(p[0]);
    f_rope = reinterpret_cast<decltype(f_rope)>(p[1]);
    f_dense = reinterpret_cast<decltype(f_dense)>(p[2]);
    f_ws = reinterpret_cast<decltype(f_ws)>(p[3]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
    {"linear_fp4", (PyCFunction)(void*)(entry<linear, 8>), METH_FASTCALL, nullptr},
    {"norm_rope", (PyCFunction)(void*)(entry<rope, 14>), METH_FASTCALL, nullptr},
    {"dense_attn", (PyCFunction)(void*)(entry<dense, 14>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
