// Python binding of the attention half of a decoder layer (the calls declared
// in the last section of include/nvfp4_w4a16.h): checks of the tensors, the
// outputs' allocation and the descriptors, then one library call.
//
// These operators take a few microseconds on the GPU when a step has few
// tokens, and a layer makes several of them, so the marshalling is compiled:
// through ctypes a call costs the host 10 to 16 us (1.7 us an allocation, 1.9
// us the current stream, 0.5 us a tensor's checks, 3.9 us the call with its
// launch), from here 4 to 6 us, most of it the launch.
//
// Every function takes its arguments positionally (attention.py has the
// signatures); wrong ones raise ValueError, a refusal by the library
// Nvfp4Error.
#include <Python.h>

#include <ATen/MemoryOverlap.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/nvfp4_w4a16.h"

namespace {

PyObject* g_error = nullptr;   // the package's Nvfp4Error

void check(nvfp4_status st) {
    if (st == NVFP4_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, nvfp4_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a torch tensor");
    return THPVariable_Unpack(o);
}

bool is_act(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }

void unit_stride(const at::Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.dim() == 0 || t.size(-1) <= 1 || t.stride(-1) == 1, name, " must have unit stride in its last dim");
}

// The tensor a call's type and device come from: bf16 or fp16, `dim` dims.
const at::Tensor& act(PyObject* o, const char* name, int64_t dim) {
    TORCH_CHECK_VALUE(THPVariable_Check(o) && is_act(THPVariable_Unpack(o).scalar_type()), name,
                      " must be a bf16 or fp16 tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be on the GPU");
    TORCH_CHECK_VALUE(t.dim() == dim, name, " must have ", dim, " dims, got shape ", t.sizes());
    unit_stride(t, name);
    return t;
}

// A tensor of a given type and shape on the call's device.
const at::Tensor& same(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
    const at::Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape, name, " must be a ", type, " tensor of shape ", shape);
    TORCH_CHECK_VALUE(t.device() == dev, name, " is on ", t.device(), ", expected ", dev);
    unit_stride(t, name);
    return t;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// What is written to: rows that share memory (an expanded tensor's) would be written by several workgroups at once.
void own_rows(const at::Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(at::has_internal_overlap(t) != at::MemOverlap::Yes, name, " is written to: its rows must not share memory");
}

// `o` as the output of that shape, or a new one if it is None.
at::Tensor output(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
    if (o == Py_None) return fresh(shape, type, dev);
    const at::Tensor& t = same(o, name, type, shape, dev);
    own_rows(t, name);
    return t;
}

void* stream_of(c10::Device dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }

// Strides of dims of one element are of no account.
int64_t step(const at::Tensor& t, int64_t dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }
int64_t leading(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}
int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

void arguments(Py_ssize_t got, Py_ssize_t want) { TORCH_CHECK_VALUE(got == want, "expected ", want, " arguments, got ", got); }

nvfp4_rope rope_of(PyObject* positions, PyObject* inv_freq, PyObject* pair_axis, PyObject* interleaved, int64_t T,
                   c10::Device dev) {
    const at::Tensor& f = tensor(inv_freq, "inv_freq");
    TORCH_CHECK_VALUE(f.dim() == 1, "inv_freq must be a 1-d fp32 tensor (one frequency per rotated pair)");
    const int64_t half = f.size(0);
    same(inv_freq, "inv_freq", at::kFloat, {half}, dev);
    const at::Tensor& p = tensor(positions, "positions");
    TORCH_CHECK_VALUE((p.dim() == 1 || p.dim() == 2) && p.size(-1) == T, "positions must be an int32 tensor [", T, "] or [axes, ",
                      T, "]");
    const int64_t axes = p.dim() == 1 ? 1 : p.size(0);
    same(positions, "positions", at::kInt, p.sizes(), dev);
    nvfp4_rope r = {};
    if (pair_axis != Py_None) r.pair_axis = static_cast<const int32_t*>(same(pair_axis, "pair_axis", at::kInt, {half}, dev).data_ptr());
    else TORCH_CHECK_VALUE(axes <= 1, "positions with several axes need pair_axis");
    r.inv_freq = static_cast<const float*>(f.data_ptr());
    r.positions = static_cast<const int32_t*>(p.data_ptr());
    r.ld_pos = axes > 1 ? p.stride(0) : T;
    TORCH_CHECK_VALUE(axes <= 1024 && half <= 1 << 20, "too many axes or frequencies");
    r.axes = (int32_t)axes;
    r.rotary = (int32_t)(2 * half);
    r.neighbours = truth(interleaved);
    return r;
}

void side_of(const at::Tensor& c, const char* name, bool packed, int64_t (&stride)[3]) {
    TORCH_CHECK_VALUE(c.stride(3) == 1 && (!packed || c.size(2) == 1 || c.stride(2) == c.size(3)), name, " must have contiguous ",
                      packed ? "blocks" : "rows");
    for (int i = 0; i < 3; ++i) stride[i] = step(c, i) * c.element_size();
}

// The cache's description; type: the activations'.
nvfp4_kv_cache cache_of(PyObject* ko, PyObject* vo, PyObject* k_scale, PyObject* v_scale, at::ScalarType type, c10::Device dev) {
    nvfp4_kv_cache c = {};
    const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
    const at::ScalarType kind = k.scalar_type();
    TORCH_CHECK_VALUE(is_act(kind) || kind == at::kFloat8_e4m3fn || kind == at::kByte,
                      "k_cache must be a bf16, fp16, float8_e4m3fn or uint8 (NVFP4) tensor");
    TORCH_CHECK_VALUE(v.scalar_type() == kind && v.sizes() == k.sizes(), "k_cache and v_cache must have one dtype and one shape");
    TORCH_CHECK_VALUE(k.device() == dev && v.device() == dev, "the caches are on ", k.device(), " and ", v.device(), ", expected ", dev);
    TORCH_CHECK_VALUE(k.dim() == 4, "k_cache and v_cache must be [pages, heads, page_size, row]");
    TORCH_CHECK_VALUE(!is_act(kind) || kind == type, "a ", kind, " cache takes ", kind, " activations, got ", type);
    c.format = is_act(kind) ? NVFP4_KV_16BIT : kind == at::kByte ? NVFP4_KV_NVFP4 : NVFP4_KV_E4M3;
    const bool packed = c.format == NVFP4_KV_NVFP4;
    side_of(k, "k_cache", packed, c.k_stride);
    side_of(v, "v_cache", packed, c.v_stride);
    int64_t D = k.size(3);
    if (packed) {
        TORCH_CHECK_VALUE(D % 9 == 0 && D * 16 / 9 % 32 == 0, "an NVFP4 cache row of ", D,
                          " bytes is not 9/16 of a head_dim that is a multiple of 32");
        D = D * 16 / 9;
    }
    TORCH_CHECK_VALUE(k.size(1) < 1 << 30 && k.size(2) < 1 << 30 && D < 1 << 30, "cache shape ", k.sizes(), " is out of range");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.pages = k.size(0);
    c.heads = (int32_t)k.size(1);
    c.page_size = (int32_t)k.size(2);
    c.head_dim = (int32_t)D;
    TORCH_CHECK_VALUE(c.format != NVFP4_KV_16BIT || (k_scale == Py_None && v_scale == Py_None),
                      "a 16-bit cache takes no k_scale or v_scale");
    if (k_scale != Py_None) c.k_scale = static_cast<const float*>(same(k_scale, "k_scale", at::kFloat, {c.heads}, dev).data_ptr());
    if (v_scale != Py_None) c.v_scale = static_cast<const float*>(same(v_scale, "v_scale", at::kFloat, {c.heads}, dev).data_ptr());
    return c;
}

PyObject* none() { Py_RETURN_NONE; }

PyObject* pack(std::initializer_list<PyObject*> items) {
    PyObject* t = PyTuple_New((Py_ssize_t)items.size());
    if (!t) throw python_error();
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}

// ------------------------------------------------------------------- calls --

// rms_norm(x, weight, eps, residual, out, scales, residual_out, fp8) -> (out, h) or (out, scales, h)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& x = act(a[0], "x", 2);
    const at::ScalarType type = x.scalar_type();
    const c10::Device dev = x.device();
    c10::DeviceGuard guard(dev);
    const int64_t T = x.size(0), N = x.size(1);
    const bool fp8 = truth(a[7]), res = a[3] != Py_None;
    const at::Tensor& w = same(a[1], "weight", type, {N}, dev);
    const float eps = number(a[2]);
    TORCH_CHECK_VALUE(res || a[6] == Py_None, "residual_out needs a residual");
    at::Tensor out = output(a[4], "out", fp8 ? at::kFloat8_e4m3fn : type, {T, N}, dev), scales, h;
    if (fp8) scales = output(a[5], "scales", at::kFloat, {T}, dev);
    const at::Tensor* r = res ? &same(a[3], "residual", type, {T, N}, dev) : nullptr;
    if (res) h = output(a[6], "residual_out", type, {T, N}, dev);
    check(nvfp4_rms_norm(x.data_ptr(), leading(x), r ? r->data_ptr() : nullptr, r ? leading(*r) : 0, w.data_ptr(), eps,
                         out.data_ptr(), leading(out), fp8 ? static_cast<float*>(scales.data_ptr()) : nullptr,
                         res ? h.data_ptr() : nullptr, res ? leading(h) : 0, T, N, type == at::kHalf, stream_of(dev)));
    PyObject* ho = res ? THPVariable_Wrap(std::move(h)) : none();
    if (fp8) return pack({THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(scales)), ho});
    return pack({THPVariable_Wrap(std::move(out)), ho});
    END_HANDLE_TH_ERRORS
}

// rope(x, positions, inv_freq, pair_axis, interleaved, out) -> out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const at::Tensor& x = act(a[0], "x", 3);
    const at::ScalarType type = x.scalar_type();
    const c10::Device dev = x.device();
    c10::DeviceGuard guard(dev);
    const int64_t T = x.size(0), H = x.size(1), D = x.size(2);
    const nvfp4_rope r = rope_of(a[1], a[2], a[3], a[4], T, dev);
    at::Tensor out = output(a[5], "out", type, {T, H, D}, dev);
    check(nvfp4_rope_apply(&r, x.data_ptr(), step(x, 0), step(x, 1), out.data_ptr(), step(out, 0), step(out, 1), T, H, D,
                           type == at::kHalf, stream_of(dev)));
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// kv_append(q, k, v, positions, inv_freq, pair_axis, interleaved, k_cache, v_cache, slots, k_scale, v_scale, out)
// -> the rotated queries; q None: keys and values only, not rotated -> None
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 13);
    const bool turn = a[0] != Py_None;
    const at::Tensor& k = act(a[1], "k", 3);
    const at::ScalarType type = k.scalar_type();
    const c10::Device dev = k.device();
    c10::DeviceGuard guard(dev);
    const int64_t T = k.size(0);
    const nvfp4_kv_cache c = cache_of(a[7], a[8], a[10], a[11], type, dev);
    own_rows(tensor(a[7], "k_cache"), "k_cache");
    own_rows(tensor(a[8], "v_cache"), "v_cache");
    same(a[1], "k", type, {T, c.heads, c.head_dim}, dev);
    const at::Tensor& v = same(a[2], "v", type, {T, c.heads, c.head_dim}, dev);
    const at::Tensor& slots = same(a[9], "slots", at::kInt, {T}, dev);
    nvfp4_rope r;
    const at::Tensor* q = nullptr;
    at::Tensor out;
    if (turn) {
        q = &act(a[0], "q", 3);
        same(a[0], "q", type, {T, q->size(1), c.head_dim}, dev);
        r = rope_of(a[3], a[4], a[5], a[6], T, dev);
        out = output(a[12], "out", type, q->sizes(), dev);
    }
    check(nvfp4_kv_append(&c, turn ? &r : nullptr, q ? q->data_ptr() : nullptr, q ? step(*q, 0) : 0, q ? step(*q, 1) : 0,
                          q ? out.data_ptr() : nullptr, q ? step(out, 0) : 0, q ? step(out, 1) : 0, q ? q->size(1) : 0,
                          k.data_ptr(), step(k, 0), step(k, 1), v.data_ptr(), step(v, 0), step(v, 1),
                          static_cast<const int32_t*>(slots.data_ptr()), T, type == at::kHalf, stream_of(dev)));
    return turn ? THPVariable_Wrap(std::move(out)) : none();
    END_HANDLE_TH_ERRORS
}

// kv_read(k_cache, v_cache, slots, fp16 (None: the cache's own type, or bf16), k_scale, v_scale, k_out, v_out) -> (k, v)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& kc = tensor(a[0], "k_cache");
    TORCH_CHECK_VALUE(kc.is_cuda(), "k_cache must be on the GPU");
    const at::ScalarType type = a[3] == Py_None ? (is_act(kc.scalar_type()) ? kc.scalar_type() : at::kBFloat16)
                                                : truth(a[3]) ? at::kHalf : at::kBFloat16;
    const c10::Device dev = kc.device();
    c10::DeviceGuard guard(dev);
    const nvfp4_kv_cache c = cache_of(a[0], a[1], a[4], a[5], type, dev);
    const at::Tensor& slots = tensor(a[2], "slots");
    TORCH_CHECK_VALUE(slots.dim() == 1, "slots must be a 1-d int32 tensor");
    const int64_t T = slots.size(0);
    same(a[2], "slots", at::kInt, {T}, dev);
    at::Tensor k = output(a[6], "out[0]", type, {T, c.heads, c.head_dim}, dev);
    at::Tensor v = output(a[7], "out[1]", type, {T, c.heads, c.head_dim}, dev);
    check(nvfp4_kv_read(&c, static_cast<const int32_t*>(slots.data_ptr()), k.data_ptr(), step(k, 0), step(k, 1), v.data_ptr(),
                        step(v, 0), step(v, 1), T, type == at::kHalf, stream_of(dev)));
    PyObject* ko = THPVariable_Wrap(std::move(k));
    return pack({ko, THPVariable_Wrap(std::move(v))});
    END_HANDLE_TH_ERRORS
}

// paged_attention(q, k_cache, v_cache, page_table, lengths, scale, k_scale, v_scale, window, out, return_lse, workspace)
// -> out or (out, lse)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 12);
    const at::Tensor& q = act(a[0], "q", 3);
    const at::ScalarType type = q.scalar_type();
    const c10::Device dev = q.device();
    c10::DeviceGuard guard(dev);
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    const nvfp4_kv_cache c = cache_of(a[1], a[2], a[6], a[7], type, dev);
    TORCH_CHECK_VALUE(D == c.head_dim, "q has ", D, " columns a head, the cache ", c.head_dim);
    TORCH_CHECK_VALUE(c.heads > 0 && Hq % c.heads == 0, Hq, " query heads are not a multiple of the cache's ", c.heads);
    const at::Tensor& table = tensor(a[3], "page_table");
    TORCH_CHECK_VALUE(table.dim() == 2 && table.size(0) == B, "page_table must be an int32 tensor [", B, ", max_pages]");
    const int64_t max_pages = table.size(1);
    same(a[3], "page_table", at::kInt, table.sizes(), dev);
    const at::Tensor& lengths = same(a[4], "lengths", at::kInt, {B}, dev);
    const float scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : number(a[5]);
    const int64_t window = whole(a[8]);
    const bool want_lse = truth(a[10]);
    at::Tensor out = output(a[9], "out", type, {B, Hq, D}, dev), lse, ws;
    if (want_lse) lse = fresh({B, Hq}, at::kFloat, dev);
    if (a[11] == Py_None) {
        const int64_t need = nvfp4_paged_attention_workspace_bytes(B, Hq, c.heads, D, max_pages * c.page_size);
        if (need < 0) check(NVFP4_ERR_INVALID_ARG);
        ws = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(dev));
        if (need > 0) ws.narrow(0, 0, NVFP4_ATTENTION_COUNTER_BYTES).zero_();
    } else {
        ws = tensor(a[11], "workspace_buf");
        TORCH_CHECK_VALUE(ws.device() == dev && ws.is_contiguous(), "workspace_buf must be a contiguous tensor on ", dev);
    }
    check(nvfp4_paged_attention(&c, q.data_ptr(), step(q, 0), step(q, 1), static_cast<const int32_t*>(table.data_ptr()),
                                leading(table), max_pages, static_cast<const int32_t*>(lengths.data_ptr()), B, Hq, scale, window,
                                out.data_ptr(), step(out, 0), step(out, 1), want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                                ws.data_ptr(), (int64_t)ws.nbytes(), type == at::kHalf, stream_of(dev)));
    PyObject* o = THPVariable_Wrap(std::move(out));
    return want_lse ? pack({o, THPVariable_Wrap(std::move(lse))}) : o;
    END_HANDLE_TH_ERRORS
}

// set_error(class): what a refusal by the library raises
PyObject* set_error(PyObject*, PyObject* cls) {
    Py_XINCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    return none();
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rms_norm), FAST(rope), FAST(kv_append), FAST(kv_read), FAST(paged_attention),
                         {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention(void) { return PyModule_Create(&module); }
