// torch-facing marshalling of the single-token calls (module _decode, used by binding.py): shapes,
// strides and pointers of the tensors, the checks the C ABI cannot make (types, layouts, devices), the
// output and workspace allocations and the current stream. These calls take a few microseconds on
// the GPU, and the same steps in Python take longer than that (16 us for the norm + rotation).
// Host code only; all arithmetic is behind the C ABI of libw4a4.so.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <c10/hip/HIPStream.h>

#include "w4a4.h"

namespace {

PyObject *error_class = nullptr;  // binding.W4A4Error, set once by init()

void want(bool cond, const char *what)
{
    if (!cond) TORCH_CHECK_VALUE(false, what);
}

// ---- argument access ----------------------------------------------------------------------------

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) TORCH_CHECK_TYPE(false, name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// undefined for None
at::Tensor optional(PyObject *o, const char *name) { return o == Py_None ? at::Tensor() : tensor(o, name); }

int64_t integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v != (int)v) TORCH_CHECK_VALUE(false, name, " = ", v, " does not fit 32 bits");
    return v;
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

int size(int64_t n, const char *name)
{
    if (n != (int)n) TORCH_CHECK_VALUE(false, name, " of ", n, " does not fit 32 bits");
    return (int)n;
}

int code_of(const at::Tensor &t, const char *name, bool f32)
{
    switch (t.scalar_type()) {
    case at::kHalf: return W4A4_F16;
    case at::kBFloat16: return W4A4_BF16;
    case at::kFloat:
        if (f32) return W4A4_F32;
        [[fallthrough]];
    default: TORCH_CHECK_TYPE(false, name, ": unsupported dtype ", t.scalar_type());
    }
}

// row stride, the row's length where there is only one row
int64_t ld(const at::Tensor &t, int64_t row) { return t.size(0) > 1 ? t.stride(0) : row; }

// The device all of a call's tensors are on, made current for the call, and its current stream.
class Place {
  public:
    explicit Place(const at::Tensor &first) : dev_(first.device())
    {
        if (!first.is_cuda()) TORCH_CHECK_VALUE(false, "expected GPU tensors, got one on ", dev_);
        c10::impl::VirtualGuardImpl impl(dev_.type());
        if (impl.getDevice() != dev_) guard_.reset_device(dev_);
        stream_ = c10::hip::getCurrentHIPStream(dev_.index()).stream();
    }
    void same(const at::Tensor &t) const
    {
        if (t.defined() && t.device() != dev_)
            TORCH_CHECK_VALUE(false, "tensors on different devices: ", dev_, " and ", t.device());
    }
    hipStream_t stream() const { return stream_; }

  private:
    c10::Device dev_;
    c10::OptionalDeviceGuard guard_;
    hipStream_t stream_;
};

void check(int rc)
{
    if (rc == W4A4_OK) return;
    PyObject *e = error_class ? PyObject_CallFunction(error_class, "is", rc, w4a4_last_error()) : nullptr;
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, w4a4_last_error());
    }
    throw python_error();
}

void arity(Py_ssize_t n, Py_ssize_t wanted)
{
    if (n != wanted) TORCH_CHECK_TYPE(false, wanted, " arguments expected, got ", n);
}

void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// ---- gemv(X, wt, w_scale, Y, epilogue, residual) -------------------------------------------------

PyObject *gemv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 6);
    const at::Tensor &X = tensor(a[0], "X"), &wt = tensor(a[1], "wt"), &ws = tensor(a[2], "w_scale");
    at::Tensor Y = optional(a[3], "Y"), res = optional(a[5], "residual");
    const int epilogue = (int)integer(a[4], "epilogue"), dt = code_of(X, "X", true);
    const auto ydt = dt == W4A4_BF16 ? at::kBFloat16 : at::kHalf;
    want(X.dim() == 2 && ws.dim() == 2, "X and w_scale must be 2-D");
    const int64_t M = X.size(0), K = X.size(1), groups = ws.size(0), N = ws.size(1);
    want(X.stride(1) == 1, "X must have unit column stride");
    if (groups <= 0 || K % groups) TORCH_CHECK_VALUE(false, "K = ", K, " does not hold ", groups, " groups");
    want(ws.scalar_type() == at::kHalf && ws.is_contiguous(), "w_scale must be contiguous fp16");
    want(wt.scalar_type() == at::kByte && wt.is_contiguous() &&
             (size_t)wt.numel() == w4a4_w4g_operand_bytes(size(N, "N"), size(K, "K")),
         "wt does not hold [N, K] weights");
    auto like_y = [&](const at::Tensor &t, const char *name) {
        if (t.scalar_type() != ydt || t.dim() != 2 || t.size(0) != M || t.size(1) != N || t.stride(1) != 1)
            TORCH_CHECK_VALUE(false, name, " must be ", ydt, " [M, N] with unit column stride");
    };
    if (Y.defined()) like_y(Y, "Y");
    if (res.defined()) like_y(res, "residual");
    const Place at_(X);
    if (!Y.defined()) Y = at::empty({M, N}, X.options().dtype(ydt));
    at_.same(wt), at_.same(ws), at_.same(Y), at_.same(res);
    check(w4a4_gemv_w4g(X.data_ptr(), dt, size(M, "M"), (int)K, ld(X, K), (const uint8_t *)wt.data_ptr(),
                        (const uint16_t *)ws.data_ptr(), (int)(K / groups), (int)N, (uint16_t *)Y.data_ptr(),
                        ld(Y, N), epilogue, (const uint16_t *)ptr(res), res.defined() ? ld(res, N) : 0,
                        at_.stream()));
    return THPVariable_Wrap(std::move(Y));
    END_HANDLE_TH_ERRORS
}

// ---- rows of heads and the paged cache -----------------------------------------------------------

struct Heads {
    int code;
    int64_t rows, heads, D;
    int64_t width() const { return heads * D; }
};

// [rows, heads, D] with adjacent heads
Heads heads_of(const at::Tensor &t, const char *name)
{
    if (t.dim() != 3 || t.stride(2) != 1 || (t.stride(1) != t.size(2) && t.size(1) != 1))
        TORCH_CHECK_VALUE(false, name, " must be [rows, heads, head_dim] with adjacent heads");
    return {code_of(t, name, false), t.size(0), t.size(1), t.size(2)};
}

void same_heads(const at::Tensor &t, const char *name, const Heads &h)
{
    const Heads o = heads_of(t, name);
    if (o.code != h.code || o.rows != h.rows || o.heads != h.heads || o.D != h.D)
        TORCH_CHECK_VALUE(false, name, " must be [", h.rows, ", ", h.heads, ", ", h.D, "] of the queries' dtype");
}

struct Cache {
    int pages, page;
    int64_t stride;
};

// [pages, kv_heads, page_size, D], dense inside a page
Cache cache_of(const at::Tensor &k, const at::Tensor &v, const at::Tensor &q, int64_t kv_heads, int64_t D)
{
    if (k.dim() != 4 || k.size(1) != kv_heads || k.size(3) != D || k.scalar_type() != q.scalar_type() ||
        v.scalar_type() != q.scalar_type())
        TORCH_CHECK_VALUE(false, "cache must be ", q.scalar_type(), " [pages, ", kv_heads, ", page_size, ", D, "]");
    want(v.sizes() == k.sizes() && v.strides() == k.strides(), "k_cache and v_cache must be laid out alike");
    const int64_t page = k.size(2);
    want(k.stride(3) == 1 && k.stride(2) == D && (k.stride(1) == page * D || kv_heads == 1),
         "a cache page must be dense");
    return {size(k.size(0), "pages"), size(page, "page_size"), ld(k, kv_heads * page * D)};
}

void dense(const at::Tensor &t, at::ScalarType dt, int64_t n, const char *name)
{
    if (t.scalar_type() != dt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        TORCH_CHECK_VALUE(false, name, " must be contiguous ", dt, " [", n, "]");
}

// ---- norm_rope(q, k, v, q_weight, k_weight, inv_freq, positions, eps, interleaved, q_out, k_out,
//                k_cache, v_cache, slots) ----------------------------------------------------------

PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 14);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const at::Tensor v = optional(a[2], "v"), qw = optional(a[3], "q_weight"), kw = optional(a[4], "k_weight"),
                     freq = optional(a[5], "inv_freq"), pos = optional(a[6], "positions"),
                     ko = optional(a[10], "k_out"), kc = optional(a[11], "k_cache"),
                     vc = optional(a[12], "v_cache"), slots = optional(a[13], "slots");
    at::Tensor qo = optional(a[9], "q_out");
    const double eps = real(a[7]);
    const int interleaved = PyObject_IsTrue(a[8]);
    if (interleaved < 0) throw python_error();

    const Heads hq = heads_of(q, "q");
    Heads hk = heads_of(k, "k");
    if (hk.code != hq.code || hk.rows != hq.rows || hk.D != hq.D)
        TORCH_CHECK_VALUE(false, "k must be [", hq.rows, ", kv_heads, ", hq.D, "] of the queries' dtype");
    if (qo.defined()) same_heads(qo, "q_out", hq);
    if (ko.defined()) same_heads(ko, "k_out", hk);
    if (qw.defined()) dense(qw, at::kFloat, hq.D, "q_weight");
    if (kw.defined()) dense(kw, at::kFloat, hq.D, "k_weight");
    int64_t rot = 0;
    if (freq.defined()) {
        rot = 2 * freq.numel();
        dense(freq, at::kDouble, freq.numel(), "inv_freq");
        want(pos.defined(), "positions are required");
        dense(pos, at::kLong, hq.rows, "positions");
    }
    Cache c{0, 0, 0};
    const bool cached = kc.defined() || vc.defined();
    if (cached) {
        want(kc.defined() && vc.defined() && v.defined() && slots.defined(),
             "v, k_cache, v_cache and slots are required");
        same_heads(v, "v", hk);
        c = cache_of(kc, vc, q, hk.heads, hq.D);
        dense(slots, at::kLong, hq.rows, "slots");
    }
    const Place at_(q);
    if (!qo.defined()) qo = at::empty({hq.rows, hq.heads, hq.D}, q.options());
    at_.same(k), at_.same(qw), at_.same(kw), at_.same(freq), at_.same(qo), at_.same(ko);
    if (freq.defined()) at_.same(pos);
    if (cached) at_.same(v), at_.same(kc), at_.same(vc), at_.same(slots);
    check(w4a4_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), cached ? v.data_ptr() : nullptr, hq.code, size(hq.rows, "rows"),
        size(hq.heads, "heads"), size(hk.heads, "kv_heads"), size(hq.D, "head_dim"), ld(q, hq.width()),
        ld(k, hk.width()), cached ? ld(v, hk.width()) : 0, (const float *)ptr(qw), (const float *)ptr(kw),
        (float)eps, (const double *)ptr(freq), size(rot, "rot_dim"), interleaved,
        freq.defined() ? (const int64_t *)ptr(pos) : nullptr, qo.data_ptr(), ld(qo, hq.width()), ptr(ko),
        ko.defined() ? ld(ko, hk.width()) : 0, ptr(kc), ptr(vc), c.pages, c.page, c.stride,
        cached ? (const int64_t *)ptr(slots) : nullptr, at_.stream()));
    return THPVariable_Wrap(std::move(qo));
    END_HANDLE_TH_ERRORS
}

// ---- paged_attn(q, k_cache, v_cache, table, lens, scale, window, sinks, max_len, out, ws) --------

PyObject *paged_attn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 11);
    const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                     &table = tensor(a[3], "table"), &lens = tensor(a[4], "lens");
    const int window = (int)integer(a[6], "window"), sinks = (int)integer(a[7], "sinks");
    at::Tensor out = optional(a[9], "out"), ws = optional(a[10], "ws");
    const Heads h = heads_of(q, "q");
    want(kc.dim() == 4, "k_cache must be [pages, kv_heads, page_size, head_dim]");
    const int64_t kv = kc.size(1);
    const Cache c = cache_of(kc, vc, q, kv, h.D);
    want(table.scalar_type() == at::kInt && table.dim() == 2 && table.size(0) == h.rows &&
             (table.stride(1) == 1 || table.size(1) == 1),
         "table must be int32 [B, width]");
    dense(lens, at::kInt, h.rows, "lens");
    const int width = size(table.size(1), "table width");
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)std::max<int64_t>(h.D, 1)) : real(a[5]);
    const int64_t most = (int64_t)width * c.page;
    const int max_len = a[8] == Py_None ? (int)std::min<int64_t>(most, 1 << 30) : (int)integer(a[8], "max_len");
    if (out.defined()) same_heads(out, "out", h);
    const Place at_(q);
    if (!out.defined()) out = at::empty({h.rows, h.heads, h.D}, q.options());
    const int B = size(h.rows, "B"), H = size(h.heads, "heads"), KV = size(kv, "kv_heads"),
              D = size(h.D, "head_dim");
    if (!ws.defined()) {
        const size_t need = w4a4_paged_attn_workspace_bytes(B, H, KV, D, max_len, window, sinks);
        if (need) ws = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    } else {
        want(ws.is_contiguous(), "ws must be contiguous");
    }
    at_.same(kc), at_.same(vc), at_.same(table), at_.same(lens), at_.same(out), at_.same(ws);
    check(w4a4_paged_attn_decode(q.data_ptr(), h.code, B, H, KV, D, ld(q, h.width()), kc.data_ptr(),
                                 vc.data_ptr(), c.pages, c.page, c.stride, (const int32_t *)table.data_ptr(),
                                 width, ld(table, width), (const int32_t *)lens.data_ptr(), max_len,
                                 (float)scale, window, sinks, out.data_ptr(), ld(out, h.width()), ptr(ws),
                                 ws.defined() ? (size_t)ws.nbytes() : 0, at_.stream()));
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// ---- init(W4A4Error) ------------------------------------------------------------------------------

PyObject *init(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XDECREF(error_class);
    error_class = cls;
    Py_RETURN_NONE;
}

template <typename F> PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)); }

PyMethodDef methods[] = {{"gemv", fast(gemv), METH_FASTCALL, nullptr},
                         {"norm_rope", fast(norm_rope), METH_FASTCALL, nullptr},
                         {"paged_attn", fast(paged_attn), METH_FASTCALL, nullptr},
                         {"init", init, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__decode(void) { return PyModule_Create(&module); }
