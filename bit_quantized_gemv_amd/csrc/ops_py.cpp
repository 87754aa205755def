// ops_py.cpp -- the torch binding of the operators beside qmv (ops.py calls it).
//
// Compiled, because the small calls are bound by the host: checks, outputs,
// scratch memory and the call took 14 us in Python beside 7 us for two launches,
// and take 2 us here.  Checks and marshalling only: every step runs in the HIP
// kernels of libqmv.so.  Outputs and scratch memory come from torch's allocator
// on the inputs' device and its current stream; scratch memory goes back to it
// when the launches are enqueued, and is reused in that stream's order.
#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <vector>

#include "qmv_ops.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;     // QmvError(status, where)

// ---- Python arguments -----------------------------------------------------

const Tensor& tensor(PyObject* o, const char* name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

const Tensor* optional_tensor(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject* o, const char* name)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_TYPE(false, name, " must be an integer");
    }
    return v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();        // it raised
    return v != 0;
}

// ---- checks ---------------------------------------------------------------

std::string dtype_name(ScalarType t)
{
    switch (t) {
        case at::kFloat: return "float32";
        case at::kHalf: return "float16";
        case at::kBFloat16: return "bfloat16";
        case at::kInt: return "int32";
        case at::kUInt32: return "uint32";
        case at::kLong: return "int64";
        case at::kDouble: return "float64";
        default: return c10::toString(t);
    }
}

void need_dtype(const Tensor& t, const char* name, ScalarType a)
{
    TORCH_CHECK_TYPE(t.scalar_type() == a, name, " must be ", dtype_name(a), ", got ", dtype_name(t.scalar_type()));
}

void need_dtype(const Tensor& t, const char* name, ScalarType a, ScalarType b)
{
    TORCH_CHECK_TYPE(t.scalar_type() == a || t.scalar_type() == b, name, " must be ", dtype_name(a), " or ", dtype_name(b),
                     ", got ", dtype_name(t.scalar_type()));
}

void need_shape(const Tensor& t, const char* name, at::IntArrayRef shape)
{
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
}

int dt_of(ScalarType t) { return t == at::kFloat ? QMV_DT_F32 : t == at::kHalf ? QMV_DT_F16 : QMV_DT_BF16; }
int dt_of(const Tensor& t) { return dt_of(t.scalar_type()); }

// Inputs must lie on one GPU; all but rows of logits and probabilities are whole.
struct Device {
    c10::Device dev{c10::DeviceType::CPU};
    bool any = false;
    void add(const Tensor& t, const char* name)
    {
        TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA (HIP) tensor");
        if (!any) dev = t.device();
        any = true;
        TORCH_CHECK_VALUE(t.device() == dev, name, " is on ", t.device(), ", the other inputs on ", dev);
    }
    void whole(const Tensor& t, const char* name)
    {
        add(t, name);
        TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    }
};

void need_format(int64_t bits, int64_t gs)
{
    TORCH_CHECK_VALUE(bits == 2 || bits == 4, "bits must be 2 or 4, got ", bits);
    TORCH_CHECK_VALUE(gs == 64 || gs == 128, "group_size must be 64 or 128, got ", gs);
}

// A quantized matrix: packed codes, scales and biases whose leading sizes are `lead`.
void need_matrix(const Tensor& w, const Tensor& s, const Tensor& b, at::IntArrayRef lead, int64_t K, int64_t bits, int64_t gs,
                 const std::string& name)
{
    TORCH_CHECK_VALUE(K >= gs && K % gs == 0, name, ": ", K, " columns are not a multiple of group_size = ", gs);
    need_dtype(w, name.c_str(), at::kInt, at::kUInt32);
    const std::string sn = name + " scales", bn = name + " biases";
    need_dtype(s, sn.c_str(), at::kBFloat16, at::kHalf);
    TORCH_CHECK_TYPE(b.scalar_type() == s.scalar_type(), name, ": scales and biases must share a dtype");
    c10::SmallVector<int64_t, 4> shape(lead.begin(), lead.end());
    shape.push_back(K * bits / 32);
    need_shape(w, name.c_str(), shape);
    shape.back() = K / gs;
    need_shape(s, sn.c_str(), shape);
    need_shape(b, bn.c_str(), shape);
}

// ---- outputs and the call -------------------------------------------------

Tensor fresh(at::IntArrayRef shape, ScalarType t, c10::Device dev)
{
    return at::detail::empty_cuda(shape, t, dev, std::nullopt);
}

Tensor output(PyObject* out, PyObject* dtype, at::IntArrayRef shape, c10::Device dev)
{
    if (out == Py_None) {
        ScalarType t = at::kBFloat16;
        if (dtype != Py_None) {
            TORCH_CHECK_TYPE(THPDtype_Check(dtype), "out_dtype must be a torch dtype");
            t = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
        }
        TORCH_CHECK_TYPE(t == at::kBFloat16 || t == at::kFloat, "out must be bfloat16 or float32, got ", dtype_name(t));
        return fresh(shape, t, dev);
    }
    Tensor y = tensor(out, "out");
    TORCH_CHECK_VALUE(y.device() == dev && y.is_contiguous() && y.sizes() == shape, "out must be a contiguous ", shape,
                      " tensor on the inputs' device");
    need_dtype(y, "out", at::kBFloat16, at::kFloat);
    return y;
}

// Sizes outside the limits are the C ABI's to refuse, by name: what has no memory then, an
// empty tensor or scratch memory of no size, is not passed as a missing pointer.  It is not read.
alignas(256) char g_nothing[256];

struct Scratch {
    c10::DataPtr at;
    long long size;
    explicit Scratch(long long n) : size(n)
    {
        if (n > 0) at = c10::hip::HIPCachingAllocator::get()->allocate((size_t)n);
    }
    void* get() const { return at ? at.get() : g_nothing; }
};

const void* data(const Tensor& t) { return t.numel() > 0 ? t.const_data_ptr() : g_nothing; }
void* data_out(Tensor& t) { return t.numel() > 0 ? t.mutable_data_ptr() : g_nothing; }

void* stream_of(c10::Device dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }

void check_status(int status, const char* where)
{
    if (status == QMV_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

const float* floats(const Tensor* t) { return t ? static_cast<const float*>(data(*t)) : nullptr; }
const float* floats(const Tensor& t) { return floats(&t); }
const int32_t* ints(const Tensor& t) { return static_cast<const int32_t*>(data(t)); }
const uint32_t* words(const Tensor& t) { return static_cast<const uint32_t*>(data(t)); }
int size32(int64_t v, const char* name)
{
    TORCH_CHECK_VALUE(v <= INT32_MAX, name, " = ", v, " is too large");
    return (int)v;
}

PyObject* wrap(Tensor&& t) { return THPVariable_Wrap(std::move(t)); }

PyObject* wrap(std::initializer_list<Tensor> ts)
{
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

void need_args(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// w, scales, biases, x, lora_a, lora_b, ids, scaling, bits, group_size, out, out_dtype
PyObject* affine_lora(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 12);
    const Tensor &w = tensor(a[0], "w"), &s = tensor(a[1], "scales"), &b = tensor(a[2], "biases"), &x = tensor(a[3], "x");
    const Tensor &la = tensor(a[4], "lora_a"), &lb = tensor(a[5], "lora_b"), &ids = tensor(a[6], "ids");
    const Tensor* scaling = optional_tensor(a[7], "scaling");
    const int64_t bits = integer(a[8], "bits"), gs = integer(a[9], "group_size");
    const bool one = x.dim() == 1;
    TORCH_CHECK_VALUE((one || x.dim() == 2) && w.dim() == 2 && la.dim() == 3,
                      "x must be [M][K] (or [K]), w [N][K*bits/32] and lora_a [L][R][K]");
    const int64_t M = one ? 1 : x.size(0), K = x.size(-1), N = w.size(0), L = la.size(0), R = la.size(1);
    need_dtype(x, "x", at::kBFloat16, at::kFloat);
    need_format(bits, gs);
    need_matrix(w, s, b, {N}, K, bits, gs, "w");
    need_dtype(la, "lora_a", at::kBFloat16, at::kHalf);
    TORCH_CHECK_TYPE(lb.scalar_type() == la.scalar_type(), "lora_a and lora_b must share a dtype");
    need_shape(la, "lora_a", {L, R, K});
    need_shape(lb, "lora_b", {L, N, R});
    need_dtype(ids, "ids", at::kInt);
    need_shape(ids, "ids", {M});
    if (scaling) {
        need_dtype(*scaling, "scaling", at::kFloat);
        need_shape(*scaling, "scaling", {L});
    }
    Device d;
    d.whole(w, "w");
    d.whole(s, "scales");
    d.whole(b, "biases");
    d.whole(x, "x");
    d.whole(la, "lora_a");
    d.whole(lb, "lora_b");
    d.whole(ids, "ids");
    if (scaling) d.whole(*scaling, "scaling");
    const c10::DeviceGuard guard(d.dev);
    Tensor y = one && a[10] == Py_None ? output(a[10], a[11], {N}, d.dev) : output(a[10], a[11], {M, N}, d.dev);
    if (M > 0) {
        const int m = size32(M, "M"), k = size32(K, "K"), r = size32(R, "the rank");
        Scratch ws(qmv_affine_lora_workspace(m, k, r));
        check_status(qmv_affine_lora(words(w), data(s), data(b), data(x), data_out(y),
                                     data(la), data(lb), ints(ids), floats(scaling), ws.get(), ws.size, m,
                                     size32(N, "N"), k, (int)bits, (int)gs, size32(L, "the adapters"), r, dt_of(x), dt_of(s),
                                     dt_of(y), dt_of(la), stream_of(d.dev)),
                     "qmv_affine_lora");
    }
    return wrap(one && y.dim() == 2 ? y.select(0, 0) : std::move(y));
    END_HANDLE_TH_ERRORS
}

void need_tokens(const Tensor& x)
{
    TORCH_CHECK_VALUE(x.dim() == 2, "x must be [T][D]");
    need_dtype(x, "x", at::kBFloat16, at::kFloat);
}

int64_t need_router(const Tensor& x, const Tensor& router, int64_t k)
{
    need_dtype(router, "router", at::kBFloat16, at::kFloat);
    TORCH_CHECK_VALUE(router.dim() == 2 && router.size(1) == x.size(1), "router must be [E][", x.size(1), "], got ", router.sizes());
    const int64_t E = router.size(0);
    TORCH_CHECK_VALUE(k >= 1 && k <= E, "top_k must be in [1, ", E, "], got ", k);
    return E;
}

struct Experts {
    const Tensor *w13, *s13, *b13, *w2, *s2, *b2;
    int64_t E, F;
    // the six tensors at a; E: as many as the router has, or -1
    Experts(PyObject* const* a, int64_t E_, int64_t D, int64_t bits, int64_t gs)
        : w13(&tensor(a[0], "gate_up")), s13(&tensor(a[1], "gate_up scales")), b13(&tensor(a[2], "gate_up biases")),
          w2(&tensor(a[3], "down")), s2(&tensor(a[4], "down scales")), b2(&tensor(a[5], "down biases"))
    {
        TORCH_CHECK_VALUE(w13->dim() == 3 && w13->size(1) % 2 == 0, "the gate and up codes must be [E][2F][D*bits/32]");
        E = E_ < 0 ? w13->size(0) : E_;
        F = w13->size(1) / 2;
        need_format(bits, gs);
        need_matrix(*w13, *s13, *b13, {E, 2 * F}, D, bits, gs, "gate_up");
        need_matrix(*w2, *s2, *b2, {E, D}, F, bits, gs, "down");
        TORCH_CHECK_TYPE(s2->scalar_type() == s13->scalar_type(), "the two products' scales must share a dtype");
    }
    void place(Device& d) const
    {
        d.whole(*w13, "gate_up");
        d.whole(*s13, "gate_up scales");
        d.whole(*b13, "gate_up biases");
        d.whole(*w2, "down");
        d.whole(*s2, "down scales");
        d.whole(*b2, "down biases");
    }
};

// x, router, top_k, renormalize
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 4);
    const Tensor &x = tensor(a[0], "x"), &router = tensor(a[1], "router");
    const int64_t k = integer(a[2], "top_k");
    const bool renorm = truth(a[3]);
    need_tokens(x);
    const int64_t T = x.size(0), D = x.size(1), E = need_router(x, router, k);
    Device d;
    d.whole(x, "x");
    d.whole(router, "router");
    const c10::DeviceGuard guard(d.dev);
    Tensor weights = fresh({T, k}, at::kFloat, d.dev), ids = fresh({T, k}, at::kInt, d.dev);
    if (T > 0) {
        const int t = size32(T, "T"), dd = size32(D, "D"), e = size32(E, "E");
        Scratch ws(qmv_route_workspace(t, dd, e));
        check_status(qmv_route(data(x), data(router), static_cast<float*>(data_out(weights)),
                               static_cast<int32_t*>(data_out(ids)), ws.get(), ws.size, t, dd, e, (int)k,
                               renorm, dt_of(x), dt_of(router), stream_of(d.dev)),
                     "qmv_route");
    }
    return wrap({weights, ids});
    END_HANDLE_TH_ERRORS
}

// x, weights, ids, six expert tensors, bits, group_size, out, out_dtype
PyObject* experts(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 13);
    const Tensor &x = tensor(a[0], "x"), &weights = tensor(a[1], "weights"), &ids = tensor(a[2], "ids");
    const int64_t bits = integer(a[9], "bits"), gs = integer(a[10], "group_size");
    need_tokens(x);
    const int64_t T = x.size(0), D = x.size(1);
    const Experts ex(a + 3, -1, D, bits, gs);
    need_dtype(weights, "weights", at::kFloat);
    need_dtype(ids, "ids", at::kInt);
    TORCH_CHECK_VALUE(ids.dim() == 2, "ids must be [T][k]");
    const int64_t k = ids.size(1);
    need_shape(ids, "ids", {T, k});
    need_shape(weights, "weights", {T, k});
    Device d;
    d.whole(x, "x");
    d.whole(weights, "weights");
    d.whole(ids, "ids");
    ex.place(d);
    const c10::DeviceGuard guard(d.dev);
    Tensor y = output(a[11], a[12], {T, D}, d.dev);
    if (T > 0) {
        const int t = size32(T, "T"), dd = size32(D, "D"), f = size32(ex.F, "F"), kk = size32(k, "top_k");
        Scratch ws(qmv_experts_workspace(t, dd, f, kk));
        check_status(qmv_experts(data(x), floats(weights), ints(ids), words(*ex.w13), data(*ex.s13),
                                 data(*ex.b13), words(*ex.w2), data(*ex.s2), data(*ex.b2),
                                 data_out(y), ws.get(), ws.size, t, dd, f, size32(ex.E, "E"), kk, (int)bits, (int)gs,
                                 dt_of(x), dt_of(*ex.s13), dt_of(y), stream_of(d.dev)),
                     "qmv_experts");
    }
    return wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// x, router, six expert tensors, top_k, renormalize, bits, group_size, out, out_dtype
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 14);
    const Tensor &x = tensor(a[0], "x"), &router = tensor(a[1], "router");
    const int64_t k = integer(a[8], "top_k"), bits = integer(a[10], "bits"), gs = integer(a[11], "group_size");
    const bool renorm = truth(a[9]);
    need_tokens(x);
    const int64_t T = x.size(0), D = x.size(1), E = need_router(x, router, k);
    const Experts ex(a + 2, E, D, bits, gs);
    Device d;
    d.whole(x, "x");
    d.whole(router, "router");
    ex.place(d);
    const c10::DeviceGuard guard(d.dev);
    Tensor y = output(a[12], a[13], {T, D}, d.dev);
    Tensor weights = fresh({T, k}, at::kFloat, d.dev), ids = fresh({T, k}, at::kInt, d.dev);
    if (T > 0) {
        const int t = size32(T, "T"), dd = size32(D, "D"), f = size32(ex.F, "F"), e = size32(E, "E");
        Scratch ws(qmv_moe_workspace(t, dd, f, e, (int)k));
        check_status(qmv_moe(data(x), data(router), words(*ex.w13), data(*ex.s13),
                             data(*ex.b13), words(*ex.w2), data(*ex.s2), data(*ex.b2),
                             data_out(y), static_cast<float*>(data_out(weights)),
                             static_cast<int32_t*>(data_out(ids)), ws.get(), ws.size, t, dd, f, e, (int)k,
                             renorm, (int)bits, (int)gs, dt_of(x), dt_of(router), dt_of(*ex.s13), dt_of(y),
                             stream_of(d.dev)),
                     "qmv_moe");
    }
    return wrap({y, weights, ids});
    END_HANDLE_TH_ERRORS
}

// logits, draft, uniforms, draft_probs, temperature, lengths
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 6);
    const Tensor &logits = tensor(a[0], "logits"), &draft = tensor(a[1], "draft"), &u = tensor(a[2], "uniforms");
    const Tensor *q = optional_tensor(a[3], "draft_probs"), *temp = optional_tensor(a[4], "temperature");
    const Tensor* len = optional_tensor(a[5], "lengths");
    TORCH_CHECK_VALUE(logits.dim() == 3 && logits.size(1) >= 1, "logits must be [B][S+1][V]");
    const int64_t B = logits.size(0), S1 = logits.size(1), S = S1 - 1, V = logits.size(2);
    need_dtype(logits, "logits", at::kBFloat16, at::kFloat);
    need_dtype(draft, "draft", at::kInt);
    need_shape(draft, "draft", {B, S});
    need_dtype(u, "uniforms", at::kFloat);
    need_shape(u, "uniforms", {B, S1});
    if (q) {
        need_dtype(*q, "draft_probs", at::kBFloat16, at::kFloat);
        need_shape(*q, "draft_probs", {B, S, V});
    }
    if (temp) {
        need_dtype(*temp, "temperature", at::kFloat);
        need_shape(*temp, "temperature", {B});
    }
    if (len) {
        need_dtype(*len, "lengths", at::kInt);
        need_shape(*len, "lengths", {B});
    }
    Device d;
    d.add(logits, "logits");
    TORCH_CHECK_VALUE(V <= 1 || logits.stride(2) == 1, "logits: the values of a row must be contiguous");
    if (q) {
        d.add(*q, "draft_probs");
        TORCH_CHECK_VALUE(V <= 1 || q->stride(2) == 1, "draft_probs: the values of a row must be contiguous");
    }
    d.whole(draft, "draft");
    d.whole(u, "uniforms");
    if (temp) d.whole(*temp, "temperature");
    if (len) d.whole(*len, "lengths");
    const c10::DeviceGuard guard(d.dev);
    Tensor tokens = fresh({B, S1}, at::kInt, d.dev), accepted = fresh({B}, at::kInt, d.dev);
    if (B > 0) {
        if (S == 0) q = nullptr;
        const int b = size32(B, "B"), s = size32(S, "S"), v = size32(V, "V");
        Scratch ws(qmv_verify_workspace(b, s, v));
        check_status(qmv_verify(data(logits), ints(draft), floats(u), q ? data(*q) : nullptr, floats(temp),
                                len ? ints(*len) : nullptr, static_cast<int32_t*>(data_out(tokens)),
                                static_cast<int32_t*>(data_out(accepted)), ws.get(), ws.size, b, s, v,
                                logits.stride(0), logits.stride(1), q ? q->stride(0) : 0, q ? q->stride(1) : 0, dt_of(logits),
                                q ? dt_of(*q) : QMV_DT_F32, stream_of(d.dev)),
                     "qmv_verify");
    }
    return wrap({tokens, accepted});
    END_HANDLE_TH_ERRORS
}

// the exception type that a status other than QMV_OK raises
PyObject* set_error(PyObject*, PyObject* type)
{
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<affine_lora>("affine_lora"), method<route>("route"), method<experts>("experts"),
                           method<moe>("moe"), method<verify>("verify"), {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "qmv_ops_py", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qmv_ops_py() { return PyModule_Create(&g_module); }
