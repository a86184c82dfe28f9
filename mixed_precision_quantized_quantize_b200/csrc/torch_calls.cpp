// torch_calls.cpp -- the attention operators' Python calls: checks of the
// tensors, allocation of outputs and workspace, and the C call, in one step.
// A decoding step makes these calls for every layer, and their kernels take a
// few microseconds; the same marshalling in Python took 14 to 20 us a call.
// No arithmetic here: everything goes through the C ABI of include/quik.h,
// whose functions are handed over by address (bind), so that the library stays
// free of any dependency on torch.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/quik.h"

namespace {

decltype(&quik_qk_norm_rope) f_qk_norm_rope;
decltype(&quik_kv_append) f_kv_append;
decltype(&quik_kv_gather) f_kv_gather;
decltype(&quik_attention_workspace_size) f_workspace_size;
decltype(&quik_tree_attention) f_tree_attention;
PyObject *g_error;  // QuikError

// Raise QuikError(status, what).
PyObject *fail(quik_status st, const char *what) {
    PyObject *args = Py_BuildValue("(is)", static_cast<int>(st), what);
    if (args != nullptr) {
        PyErr_SetObject(g_error, args);
        Py_DECREF(args);
    }
    return nullptr;
}

// A tensor, or an undefined one for None where that is allowed.
const at::Tensor &tensor(PyObject *o, const char *what, bool optional = false) {
    static const at::Tensor none;
    if (optional && o == Py_None) return none;
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

void check(const at::Tensor &t, const char *what, at::ScalarType type, int dev) {
    TORCH_CHECK_VALUE(t.is_cuda(), what, " must live on a CUDA device");
    TORCH_CHECK_TYPE(t.scalar_type() == type, what, " must be ", type, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.get_device() == dev, what, " is on cuda:", static_cast<int>(t.get_device()),
                      ", others on cuda:", dev);
}

int device_of(const at::Tensor &t, const char *what) {
    TORCH_CHECK_VALUE(t.is_cuda(), what, " must live on a CUDA device");
    return t.get_device();
}

// Rows [tokens, heads, head_dim] fp16: the heads of a token are contiguous, the
// tokens may be any distance apart (a slice of a projection's output).
struct Rows {
    void *p = nullptr;
    int64_t stride = 0;
};
Rows rows(const at::Tensor &t, const char *what, int dev) {
    Rows r;
    if (!t.defined()) return r;
    check(t, what, at::kHalf, dev);
    const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
    TORCH_CHECK_VALUE((t.stride(1) == d || h <= 1) && (t.stride(2) == 1 || d <= 1), what,
                      ": the heads of a token must be contiguous");
    // the stride of a single row says nothing
    r.stride = n == 1 ? (h * d + 7) / 8 * 8 : t.stride(0);
    r.p = t.numel() == 0 ? nullptr : t.data_ptr();
    return r;
}

// Pointer of a contiguous tensor.
void *flat(const at::Tensor &t, const char *what, at::ScalarType type, int dev) {
    if (!t.defined()) return nullptr;
    check(t, what, type, dev);
    TORCH_CHECK_VALUE(t.is_contiguous(), what, " must be contiguous");
    return t.numel() == 0 ? nullptr : t.data_ptr();
}

bool is_rows(const at::Tensor &t) { return t.defined() && t.dim() == 3; }

// rotary_dim and rows of the rotation's tables.
struct Tables {
    int rotary = 0, rows = 0;
};
Tables tables(const at::Tensor &cos, const at::Tensor &sin, const at::Tensor &positions, int64_t tokens) {
    Tables t;
    if (!cos.defined() && !sin.defined()) return t;
    TORCH_CHECK_VALUE(cos.defined() && sin.defined() && positions.defined(),
                      "a rotation needs cos, sin and positions");
    TORCH_CHECK_VALUE(cos.dim() == 2 && cos.sizes() == sin.sizes(),
                      "cos and sin must be [rows, rotary_dim / 2], both alike");
    TORCH_CHECK_VALUE(positions.dim() == 1 && positions.size(0) == tokens, "positions must be [", tokens, "], got ",
                      positions.sizes());
    t.rotary = static_cast<int>(2 * cos.size(1));
    t.rows = static_cast<int>(cos.size(0));
    return t;
}

int to_int(int64_t v, const char *what) {
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, what, " does not fit 32 bits: ", v);
    return static_cast<int>(v);
}

at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
}

bool wants(Py_ssize_t got, Py_ssize_t n) {
    if (got == n) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", n, got);
    return false;
}

// Python's number as a double / an integer (a Python error is thrown on).
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int64_t whole(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
const quik_kv_cache *cache_at(PyObject *o) { return reinterpret_cast<const quik_kv_cache *>(whole(o)); }

// An output to return: the caller's object, or a new one of `t`.
PyObject *given_or(PyObject *o, const at::Tensor &t) {
    if (o != Py_None) {
        Py_INCREF(o);
        return o;
    }
    return THPVariable_Wrap(t);
}
PyObject *pair(PyObject *a, PyObject *b) {
    PyObject *r = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

// (q, k, q_weight, k_weight, eps, cos, sin, positions, interleaved, q_out, k_out)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (!wants(count, 11)) return nullptr;
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k", true);
    const at::Tensor &qw = tensor(a[2], "q_weight", true), &kw = tensor(a[3], "k_weight", true);
    const at::Tensor &cos = tensor(a[5], "cos", true), &sin = tensor(a[6], "sin", true);
    const at::Tensor &pos = tensor(a[7], "positions", true);
    TORCH_CHECK_VALUE(is_rows(q), "q must be [tokens, heads, head_dim], got ", q.sizes());
    const int64_t n = q.size(0), qh = q.size(1), d = q.size(2);
    TORCH_CHECK_VALUE(!k.defined() || (k.dim() == 3 && k.size(0) == n && k.size(2) == d), "k must be [", n,
                      ", heads, ", d, "], got ", k.sizes());
    const Tables t = tables(cos, sin, pos, n);
    for (const at::Tensor *w : {&qw, &kw})
        TORCH_CHECK_VALUE(!w->defined() || (w->dim() == 1 && w->size(0) == d), "weights must be [", d, "], got ",
                          w->sizes());
    const int dev = device_of(q, "q");
    const at::Tensor &gq = tensor(a[9], "q_out", true), &gk = tensor(a[10], "k_out", true);
    TORCH_CHECK_VALUE((!gq.defined() || gq.sizes() == q.sizes()) &&
                          (!gk.defined() || (k.defined() && gk.sizes() == k.sizes())),
                      "an output must have its input's shape");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const at::Tensor qo = gq.defined() ? gq : new_tensor(q.sizes(), at::kHalf, dev);
    const at::Tensor ko = !k.defined() || gk.defined() ? gk : new_tensor(k.sizes(), at::kHalf, dev);
    const quik_heads s{to_int(n, "tokens"), to_int(qh, "heads"),
                       k.defined() ? to_int(k.size(1), "heads") : 0, to_int(d, "head_dim"), t.rotary,
                       truth(a[8]) ? 1 : 0, t.rows};
    const Rows qr = rows(q, "q", dev), kr = rows(k, "k", dev), qor = rows(qo, "q_out", dev),
               kor = rows(ko, "k_out", dev);
    const quik_status st = f_qk_norm_rope(
        &s, qr.p, qr.stride, kr.p, kr.stride, flat(qw, "q_weight", at::kHalf, dev),
        flat(kw, "k_weight", at::kHalf, dev), static_cast<float>(number(a[4])),
        static_cast<const float *>(flat(cos, "cos", at::kFloat, dev)),
        static_cast<const float *>(flat(sin, "sin", at::kFloat, dev)),
        static_cast<const int32_t *>(flat(pos, "positions", at::kInt, dev)), qor.p, qor.stride, kor.p, kor.stride,
        c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != QUIK_OK) return fail(st, "quik_qk_norm_rope");
    PyObject *second = Py_None;
    if (k.defined())
        second = given_or(a[10], ko);
    else
        Py_INCREF(second);
    return pair(given_or(a[9], qo), second);
    END_HANDLE_TH_ERRORS
}

// (cache address, cache device, k, v, slots, cos, sin, positions, interleaved)
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (!wants(count, 9)) return nullptr;
    const quik_kv_cache *c = cache_at(a[0]);
    const int dev = static_cast<int>(whole(a[1]));
    const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &slots = tensor(a[4], "slots");
    const at::Tensor &cos = tensor(a[5], "cos", true), &sin = tensor(a[6], "sin", true);
    const at::Tensor &pos = tensor(a[7], "positions", true);
    TORCH_CHECK_VALUE(is_rows(k) && k.size(1) == c->heads && k.size(2) == c->head_dim && v.sizes() == k.sizes(),
                      "k and v must be [tokens, ", c->heads, ", ", c->head_dim, "], got ", k.sizes(), " and ",
                      v.sizes());
    const int64_t n = k.size(0);
    TORCH_CHECK_VALUE(slots.dim() == 1 && slots.size(0) == n, "slots must be [", n, "], got ", slots.sizes());
    const Tables t = tables(cos, sin, pos, n);
    const quik_heads s{to_int(n, "tokens"), 0, c->heads, c->head_dim, t.rotary, truth(a[8]) ? 1 : 0, t.rows};
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    const Rows kr = rows(k, "k", dev), vr = rows(v, "v", dev);
    const quik_status st =
        f_kv_append(&s, c, kr.p, kr.stride, vr.p, vr.stride,
                    static_cast<const float *>(flat(cos, "cos", at::kFloat, dev)),
                    static_cast<const float *>(flat(sin, "sin", at::kFloat, dev)),
                    static_cast<const int32_t *>(flat(pos, "positions", at::kInt, dev)),
                    static_cast<const int64_t *>(flat(slots, "slots", at::kLong, dev)),
                    c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != QUIK_OK) return fail(st, "quik_kv_append");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (cache address, cache device, slots, k_out, v_out)
PyObject *kv_gather(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (!wants(count, 5)) return nullptr;
    const quik_kv_cache *c = cache_at(a[0]);
    const int dev = static_cast<int>(whole(a[1]));
    const at::Tensor &slots = tensor(a[2], "slots");
    TORCH_CHECK_VALUE(slots.dim() == 1, "slots must be [tokens], got ", slots.sizes());
    const int64_t shape[3] = {slots.size(0), c->heads, c->head_dim};
    const at::Tensor &gk = tensor(a[3], "k_out", true), &gv = tensor(a[4], "v_out", true);
    for (const at::Tensor *o : {&gk, &gv})
        TORCH_CHECK_VALUE(!o->defined() || o->sizes() == at::IntArrayRef(shape), "outputs must be ",
                          at::IntArrayRef(shape), ", got ", o->sizes());
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    const at::Tensor ko = gk.defined() ? gk : new_tensor(shape, at::kHalf, dev);
    const at::Tensor vo = gv.defined() ? gv : new_tensor(shape, at::kHalf, dev);
    const Rows kr = rows(ko, "k_out", dev), vr = rows(vo, "v_out", dev);
    const quik_status st = f_kv_gather(c, to_int(shape[0], "tokens"),
                                       static_cast<const int64_t *>(flat(slots, "slots", at::kLong, dev)), kr.p,
                                       kr.stride, vr.p, vr.stride, c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != QUIK_OK) return fail(st, "quik_kv_gather");
    return pair(given_or(a[3], ko), given_or(a[4], vo));
    END_HANDLE_TH_ERRORS
}

// (q, cache address, cache device, page_table, context, cu_tokens, max_tokens, max_context, mask, scale, out, lse,
//  return_lse)
PyObject *tree_attention(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (!wants(count, 13)) return nullptr;
    const at::Tensor &q = tensor(a[0], "q");
    const quik_kv_cache *c = cache_at(a[1]);
    const int dev = static_cast<int>(whole(a[2]));
    const at::Tensor &table = tensor(a[3], "page_table"), &ctx = tensor(a[4], "context");
    const at::Tensor &cu = tensor(a[5], "cu_tokens"), &mask = tensor(a[8], "mask", true);
    const at::Tensor &go = tensor(a[10], "out", true), &gl = tensor(a[11], "lse", true);
    const bool want_lse = truth(a[12]);
    TORCH_CHECK_VALUE(is_rows(q) && q.size(2) == c->head_dim, "q must be [tokens, heads, ", c->head_dim, "], got ",
                      q.sizes());
    const int64_t n = q.size(0), qh = q.size(1);
    TORCH_CHECK_VALUE(table.dim() == 2 && ctx.dim() == 1 && cu.dim() == 1 && ctx.size(0) == table.size(0) &&
                          cu.size(0) == table.size(0) + 1,
                      "context must be [sequences], page_table [sequences, max_pages], cu_tokens [sequences + 1]");
    TORCH_CHECK_VALUE(!mask.defined() || (mask.dim() == 2 && mask.size(0) == n), "mask must be [", n,
                      ", words], got ", mask.sizes());
    TORCH_CHECK_VALUE(!go.defined() || go.sizes() == q.sizes(), "out must have the shape of q");
    TORCH_CHECK_VALUE(!gl.defined() || (gl.dim() == 2 && gl.size(0) == n && gl.size(1) == qh), "lse must be [", n,
                      ", ", qh, "], got ", gl.sizes());
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    const Rows qr = rows(q, "q", dev);
    const at::Tensor out = go.defined() ? go : new_tensor(q.sizes(), at::kHalf, dev);
    const at::Tensor lse = gl.defined() || !want_lse ? gl : new_tensor({n, qh}, at::kFloat, dev);
    const Rows orow = rows(out, "out", dev);
    quik_attention s{};
    s.tokens = to_int(n, "tokens");
    s.sequences = to_int(table.size(0), "sequences");
    s.q_heads = to_int(qh, "heads");
    s.max_tokens = to_int(whole(a[6]), "max_tokens");
    s.max_pages = to_int(table.size(1), "max_pages");
    s.max_context = to_int(whole(a[7]), "max_context");
    s.mask_words = mask.defined() ? to_int(mask.size(1), "words") : 0;
    s.scale = static_cast<float>(a[9] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c->head_dim)) : number(a[9]));
    const size_t need = f_workspace_size(&s, c);
    // lives until the launch; its memory is reused in the order of this stream only
    at::Tensor ws;
    if (need > 0) ws = new_tensor({static_cast<int64_t>(need)}, at::kByte, dev);
    const quik_status st = f_tree_attention(
        &s, c, qr.p, qr.stride, static_cast<const int32_t *>(flat(table, "page_table", at::kInt, dev)),
        static_cast<const int32_t *>(flat(ctx, "context", at::kInt, dev)),
        static_cast<const int32_t *>(flat(cu, "cu_tokens", at::kInt, dev)),
        static_cast<const uint32_t *>(flat(mask, "mask", at::kInt, dev)), orow.p, orow.stride,
        static_cast<float *>(flat(lse, "lse", at::kFloat, dev)), need > 0 ? ws.data_ptr() : nullptr, need,
        c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != QUIK_OK) return fail(st, "quik_tree_attention");
    if (!want_lse) return given_or(a[10], out);
    return pair(given_or(a[10], out), given_or(a[11], lse));
    END_HANDLE_TH_ERRORS
}

// (QuikError, addresses of quik_qk_norm_rope, quik_kv_append, quik_kv_gather, quik_attention_workspace_size,
//  quik_tree_attention)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (!wants(count, 6)) return nullptr;
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    f_qk_norm_rope = reinterpret_cast<decltype(f_qk_norm_rope)>(whole(a[1]));
    f_kv_append = reinterpret_cast<decltype(f_kv_append)>(whole(a[2]));
    f_kv_gather = reinterpret_cast<decltype(f_kv_gather)>(whole(a[3]));
    f_workspace_size = reinterpret_cast<decltype(f_workspace_size)>(whole(a[4]));
    f_tree_attention = reinterpret_cast<decltype(f_tree_attention)>(whole(a[5]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(qk_norm_rope), METHOD(kv_append), METHOD(kv_gather),
                         METHOD(tree_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
    PyObject *m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", QUIK_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
