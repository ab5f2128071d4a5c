// wq_torch.cpp -- the binding of the prompt-side calls as a CPython extension.
//
// A call of these operators at decode sizes is a few microseconds of kernel,
// so what the host does around the launch is what a user waits for: the same
// checks, output allocations and ctypes marshalling in Python took 11 to 16
// microseconds a call, this file's 3 to 5.5 (B200 host, calls back to back).
// It marshals arguments only: types, shapes, strides and devices are checked
// here, everything else by the C entry points of libwq (include/wq.h), whose
// status codes go back through the `raise_status` callable.
//
// Every function takes its arguments by position, outputs, workspace and
// stream handle as None when they are not given (then: new tensors, a new
// workspace, the current stream of the inputs' device, which is made current
// for the call).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "../../include/wq.h"

namespace {

PyObject *raise_status = nullptr;  // callable: status code -> raises

struct Refused {};  // the Python error is set

[[noreturn]] void refuse(PyObject *type, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw Refused();
}

void check(int rc)
{
    if (rc == WQ_OK) return;
    PyObject *r = PyObject_CallFunction(raise_status, "i", rc);
    if (r) {
        Py_DECREF(r);
        PyErr_SetString(PyExc_RuntimeError, "libwq call failed");
    }
    throw Refused();
}

const at::Tensor &cuda(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        refuse(PyExc_TypeError, "%s must be a CUDA tensor (libwq has no CPU path)", name);
    return THPVariable_Unpack(o);
}

void on_device(const at::Tensor &t, const char *name, const at::Tensor &like)
{
    if (t.get_device() != like.get_device())
        refuse(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d", name, (int)t.get_device(), (int)like.get_device());
}

// A contiguous tensor of this type and shape on like's device.
void *dense(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Tensor &like)
{
    const at::Tensor &t = cuda(o, name);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s", name, c10::toString(type));
    if (t.sizes() != shape) refuse(PyExc_ValueError, "%s has the wrong shape", name);
    on_device(t, name, like);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

// An output: the given tensor, checked, or a new one.  `ref` receives a new reference to its Python object.
void *output(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Tensor &like, PyObject **ref)
{
    if (o == Py_None) {
        at::Tensor t = at::detail::empty_cuda(shape, type, like.device(), std::nullopt);  // at::empty without its dispatch
        void *p = t.data_ptr();
        *ref = THPVariable_Wrap(std::move(t));
        if (!*ref) throw Refused();
        return p;
    }
    void *p = dense(o, name, type, shape, like);
    Py_INCREF(o);
    *ref = o;
    return p;
}

struct Heads {
    uint16_t *p;
    int64_t ld, tokens, heads, dim;
};

// bf16 [tokens][heads][D] whose rows hold their heads one after another, any row distance.
Heads heads(PyObject *o, const char *name, const at::Tensor *like = nullptr, const Heads *same = nullptr, int64_t n = -1)
{
    const at::Tensor &t = cuda(o, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3)
        refuse(PyExc_TypeError, "%s must be a 3-D bfloat16 tensor [tokens][heads][D]", name);
    if (like) on_device(t, name, *like);
    const int64_t M = t.size(0), H = t.size(1), D = t.size(2);
    if (same && (M != same->tokens || D != same->dim || (n >= 0 && H != n)))
        refuse(PyExc_ValueError, "%s does not have the tokens, heads or head size of the other tensors", name);
    if ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D))
        refuse(PyExc_ValueError, "%s must hold each token's heads one after another (strides D and 1)", name);
    return {static_cast<uint16_t *>(t.data_ptr()), M > 1 ? t.stride(0) : H * D, M, H, D};
}

Heads heads_output(PyObject *o, const char *name, const at::Tensor &like, const Heads &same, int64_t n, PyObject **ref)
{
    if (o == Py_None) {
        void *p = output(o, name, at::kBFloat16, {same.tokens, n, same.dim}, like, ref);
        return {static_cast<uint16_t *>(p), n * same.dim, same.tokens, n, same.dim};
    }
    const Heads h = heads(o, name, &like, &same, n);
    Py_INCREF(o);
    *ref = o;
    return h;
}

// Makes the tensors' device current and gives the stream to launch on; a given one also becomes current, so that
// what the call allocates and clears belongs to it.
struct Launch {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard given;
    void *stream;
    Launch(const at::Tensor &t, PyObject *handle)
    {
        const auto dev = t.get_device();
        if (handle == Py_None) {
            if (c10::cuda::current_device() != dev) device.set_index(dev);
            stream = c10::cuda::getCurrentCUDAStream(dev).stream();
            return;
        }
        stream = PyLong_AsVoidPtr(handle);
        if (!stream && PyErr_Occurred()) throw Refused();
        given.reset_stream(stream ? c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), dev)
                                  : c10::cuda::getDefaultCUDAStream(dev));
    }
};

// References that a call holds until it returns them (dropped when it fails).
struct Refs {
    PyObject *o[2] = {nullptr, nullptr};
    ~Refs()
    {
        Py_XDECREF(o[0]);
        Py_XDECREF(o[1]);
    }
    PyObject *take(int i)
    {
        PyObject *p = o[i];
        o[i] = nullptr;
        return p;
    }
    PyObject *pair()
    {
        PyObject *t = PyTuple_Pack(2, o[0], o[1]);
        return t;
    }
};

void arity(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want) refuse(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
}

// x, q, scales, stream -> (q, scales)
PyObject *quantize_int8_tokens(PyObject *const *a, Py_ssize_t n)
{
    arity(n, 4);
    const at::Tensor &x = cuda(a[0], "x");
    if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
        refuse(PyExc_ValueError, "x must be a 2-D tensor with unit stride along K");
    const auto type = x.scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) refuse(PyExc_TypeError, "input must be float32 or bfloat16");
    const int64_t M = x.size(0), K = x.size(1);
    Launch l(x, a[3]);
    Refs r;
    void *q = output(a[1], "q", at::kChar, {M, K}, x, &r.o[0]);
    void *s = output(a[2], "scales", at::kFloat, {M}, x, &r.o[1]);
    check(wq_quantize_int8_tokens(x.data_ptr(), type == at::kFloat ? WQ_F32 : WQ_BF16, M, K, M > 1 ? x.stride(0) : K,
                                  static_cast<int8_t *>(q), static_cast<float *>(s), l.stream));
    return r.pair();
}

// xq, xscales, qweight, scales, y, workspace, stream -> y
PyObject *gemm_w8a8_int8(PyObject *const *a, Py_ssize_t n)
{
    arity(n, 7);
    const at::Tensor &xq = cuda(a[0], "xq"), &w = cuda(a[2], "qweight");
    if (xq.scalar_type() != at::kChar || w.scalar_type() != at::kChar || xq.dim() != 2 || w.dim() != 2)
        refuse(PyExc_TypeError, "xq and qweight must be 2-D int8 tensors");
    if (!xq.is_contiguous()) refuse(PyExc_ValueError, "xq must be contiguous");
    const int64_t M = xq.size(0), K = xq.size(1), N = w.size(0);
    const void *xs = dense(a[1], "xscales", at::kFloat, {M}, xq);
    dense(a[2], "qweight", at::kChar, {N, K}, xq);
    const at::Tensor &s = cuda(a[3], "scales");
    const void *ws = s.dim() == 2 ? dense(a[3], "scales", at::kBFloat16, {N, 1}, xq) : dense(a[3], "scales", at::kBFloat16, {N}, xq);
    Launch l(xq, a[6]);
    Refs r;
    void *y = output(a[4], "y", at::kBFloat16, {M, N}, xq, &r.o[0]);
    at::Tensor space;
    if (a[5] == Py_None) {
        space = at::zeros({(int64_t)wq_gemm_w8a8_int8_workspace_bytes(M, N, K)}, xq.options().dtype(at::kByte));
    } else {
        space = cuda(a[5], "workspace");
        on_device(space, "workspace", xq);
        if (!space.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
    }
    check(wq_gemm_w8a8_int8(static_cast<const int8_t *>(xq.data_ptr()), static_cast<const float *>(xs), M, N, K,
                            static_cast<const int8_t *>(w.data_ptr()), static_cast<const uint16_t *>(ws),
                            static_cast<uint16_t *>(y), space.data_ptr(), space.nbytes(), l.stream));
    return r.take(0);
}

// q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream -> (q_out, k_out)
PyObject *qk_norm_rope(PyObject *const *a, Py_ssize_t n)
{
    arity(n, 11);
    const at::Tensor &qt = cuda(a[0], "q");
    const Heads q = heads(a[0], "q"), k = heads(a[1], "k", &qt, &q);
    const at::Tensor &f = cuda(a[3], "inv_freq");
    if (f.dim() != 1) refuse(PyExc_ValueError, "inv_freq must be a 1-D tensor");
    const int64_t half = f.numel();
    const void *pos = dense(a[2], "positions", at::kInt, {q.tokens}, qt), *freq = dense(a[3], "inv_freq", at::kFloat, {half}, qt);
    const void *qw = a[4] == Py_None ? nullptr : dense(a[4], "q_weight", at::kBFloat16, {q.dim}, qt);
    const void *kw = a[5] == Py_None ? nullptr : dense(a[5], "k_weight", at::kBFloat16, {q.dim}, qt);
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused();
    const int interleaved = PyObject_IsTrue(a[7]);
    if (interleaved < 0) throw Refused();
    Launch l(qt, a[10]);
    Refs r;
    const Heads qo = heads_output(a[8], "q_out", qt, q, q.heads, &r.o[0]), ko = heads_output(a[9], "k_out", qt, k, k.heads, &r.o[1]);
    check(wq_qk_norm_rope(q.p, q.ld, k.p, k.ld, static_cast<const uint16_t *>(qw), static_cast<const uint16_t *>(kw), (float)eps,
                          static_cast<const int32_t *>(pos), static_cast<const float *>(freq), 2 * half, interleaved, q.tokens,
                          q.heads, k.heads, q.dim, qo.p, qo.ld, ko.p, ko.ld, l.stream));
    return r.pair();
}

// What both stores check: k, v, slots and the shape of the codes.
struct Store {
    const at::Tensor &like;
    Heads k, v;
    const int64_t *slots;
    int64_t B, T;
    Store(PyObject *const *a, PyObject *codes)
        : like(cuda(a[0], "k")), k(heads(a[0], "k")), v(heads(a[1], "v", &like, &k, k.heads)),
          slots(static_cast<const int64_t *>(dense(a[2], "slots", at::kLong, {k.tokens}, like)))
    {
        const at::Tensor &c = cuda(codes, "k_codes");
        if (c.dim() != 4 || c.size(2) != k.heads) refuse(PyExc_ValueError, "the codes must be [B][T][H][...] with k's heads");
        B = c.size(0);
        T = c.size(1);
    }
    uint8_t *codes(PyObject *o, const char *name, int64_t width) const
    {
        return static_cast<uint8_t *>(dense(o, name, at::kByte, {B, T, k.heads, width}, like));
    }
    uint16_t *params(PyObject *o, const char *name) const
    {
        return static_cast<uint16_t *>(dense(o, name, at::kBFloat16, {B, T, k.heads}, like));
    }
    float *scale(PyObject *o, const char *name) const { return static_cast<float *>(dense(o, name, at::kFloat, {1}, like)); }
};

// k, v, slots, k_codes, k_scales, k_zeros, v_codes, v_scales, v_zeros, stream
PyObject *kv_store_int4(PyObject *const *a, Py_ssize_t n)
{
    arity(n, 10);
    const Store s(a, a[3]);
    uint8_t *kc = s.codes(a[3], "k_codes", s.k.dim / 2), *vc = s.codes(a[6], "v_codes", s.k.dim / 2);
    uint16_t *ks = s.params(a[4], "k_scales"), *kz = s.params(a[5], "k_zeros");
    uint16_t *vs = s.params(a[7], "v_scales"), *vz = s.params(a[8], "v_zeros");
    Launch l(s.like, a[9]);
    check(wq_kv_store_int4(s.k.p, s.k.ld, s.v.p, s.v.ld, s.slots, s.k.tokens, s.B * s.T, s.k.heads, s.k.dim, kc, ks, kz, vc, vs,
                           vz, l.stream));
    Py_RETURN_NONE;
}

// k, v, slots, k_codes, k_scale, v_codes, v_scale, stream
PyObject *kv_store_fp8(PyObject *const *a, Py_ssize_t n)
{
    arity(n, 8);
    const Store s(a, a[3]);
    uint8_t *kc = s.codes(a[3], "k_codes", s.k.dim), *vc = s.codes(a[5], "v_codes", s.k.dim);
    const float *ks = s.scale(a[4], "k_scale"), *vs = s.scale(a[6], "v_scale");
    Launch l(s.like, a[7]);
    check(wq_kv_store_fp8(s.k.p, s.k.ld, s.v.p, s.v.ld, s.slots, s.k.tokens, s.B * s.T, s.k.heads, s.k.dim, kc, ks, vc, vs, l.stream));
    Py_RETURN_NONE;
}

// q, k, v, starts, o, stream -> o
PyObject *prompt_attention(PyObject *const *a, Py_ssize_t n)
{
    arity(n, 6);
    const at::Tensor &qt = cuda(a[0], "q");
    const Heads q = heads(a[0], "q"), k = heads(a[1], "k", &qt, &q), v = heads(a[2], "v", &qt, &k, k.heads);
    const at::Tensor &st = cuda(a[3], "starts");
    if (st.dim() != 1 || st.numel() < 2) refuse(PyExc_ValueError, "starts must be a 1-D tensor of at least two values");
    const int64_t B = st.numel() - 1;
    const void *starts = dense(a[3], "starts", at::kInt, {B + 1}, qt);
    Launch l(qt, a[5]);
    Refs r;
    const Heads o = heads_output(a[4], "o", qt, q, q.heads, &r.o[0]);
    check(wq_prompt_attention(q.p, q.ld, k.p, k.ld, v.p, v.ld, static_cast<const int32_t *>(starts), B, q.tokens, q.heads, k.heads,
                              q.dim, o.p, o.ld, l.stream));
    return r.take(0);
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_raise_status(PyObject *, PyObject *f)
{
    Py_INCREF(f);
    Py_XSETREF(raise_status, f);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<quantize_int8_tokens>("quantize_int8_tokens"),
    method<gemm_w8a8_int8>("gemm_w8a8_int8"),
    method<qk_norm_rope>("qk_norm_rope"),
    method<kv_store_int4>("kv_store_int4"),
    method<kv_store_fp8>("kv_store_fp8"),
    method<prompt_attention>("prompt_attention"),
    {"set_raise_status", set_raise_status, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_wq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wq_torch(void) { return PyModule_Create(&module); }
