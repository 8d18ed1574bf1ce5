// sv_bind.cpp -- the common form of the paged-cache calls' marshalling as a
// CPython extension: every tensor checked, the outputs allocated and the
// library called without returning to the interpreter between them.
//
// Each function takes the tensors of the api.py function of its name in their
// plain form (no caller-provided outputs, no explicit stream) and returns its
// results, or None when anything about the call is out of the ordinary -- a
// tensor of another type, shape or device, a capture that needs its own
// workspace, a status other than SV_OK -- having launched nothing; api.py
// then goes through its own checks, which say what is wrong.  These calls are
// a few microseconds on the GPU, and the interpreter's share of a call was
// 15 to 25 microseconds against 3 here.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/specverify.h"

namespace {

decltype(&sv_build_block_tables) f_build;
decltype(&sv_release_pages) f_release;
decltype(&sv_append_kv_paged) f_append;
decltype(&sv_chunk_attention_paged) f_chunk;

PyObject *none() { Py_RETURN_NONE; }

// The tensor behind a Python object; null if it is none.
const at::Tensor *tensor(PyObject *o) {
    return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// A contiguous CUDA array of the given type and sizes on device `dev`.
bool array(const at::Tensor *t, at::ScalarType type, int dev, std::initializer_list<int64_t> sizes) {
    return t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type &&
           t->sizes().equals(c10::IntArrayRef(sizes)) && t->is_contiguous();
}

bool i32(const at::Tensor *t, int dev, int64_t n) { return array(t, at::kInt, dev, {n}); }

int32_t *ip(const at::Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); }

// Rows [n, heads, d] whose last two dimensions are dense; elements between
// rows, 0 if they are laid out otherwise.
int64_t row_stride(const at::Tensor &t) {
    const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
    if ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d)) return 0;
    return n == 1 ? h * d : t.stride(0) >= h * d ? t.stride(0) : 0;
}

// The current device, if it is the one that `t` is on; -1 otherwise.
int device_of(const at::Tensor *t) {
    return t && t->is_cuda() && t->get_device() == c10::cuda::current_device() ? (int)t->get_device() : -1;
}

sv_stream_t stream_of(int dev) {
    return reinterpret_cast<sv_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}

// Memory for a call's outputs on the current device and stream, and a tensor of
// `sizes` from element `at` of it on.  Straight from the allocator and as plain
// tensors, without the dispatcher: pages of 8 requests back 4.3 -> 3.8 us a call
// (4.7 on a slower host).
c10::Storage memory(int64_t bytes) {
    c10::Allocator *from = c10::cuda::CUDACachingAllocator::get();
    return c10::Storage(c10::Storage::use_byte_size_t(), (size_t)bytes, from->allocate((size_t)bytes), from, true);
}

at::Tensor part(const c10::Storage &memory, c10::ScalarType type, int64_t at, std::initializer_list<int64_t> sizes) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(memory), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(c10::IntArrayRef(sizes));
    return t;
}

at::Tensor ints(const c10::Storage &memory, int64_t at, int64_t n) { return part(memory, at::kInt, at, {n}); }

at::Tensor empty(std::initializer_list<int64_t> sizes, c10::ScalarType type) {
    int64_t n = 1;
    for (int64_t x : sizes) n *= x;
    return part(memory(n * (int64_t)c10::elementSize(type)), type, 0, sizes);
}

constexpr int64_t kShared = 2048;  // ints of a slot map that shares the others' allocation

// A small non-negative int, -1 if the object is another thing.
int64_t small_int(PyObject *o) {
    if (!PyLong_CheckExact(o)) return -1;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) PyErr_Clear();
    return v >= 0 && v < (1LL << 31) ? v : -1;
}

// An optional status array: its pointer, or `bad` set.
int32_t *status(PyObject *o, int dev, int64_t n, bool &bad) {
    if (o == Py_None) return nullptr;
    const at::Tensor *t = tensor(o);
    if (!i32(t, dev, n)) {
        bad = true;
        return nullptr;
    }
    return ip(*t);
}

// (prefix_lens, new_lens, page_counts, block_table, free_pages, free_count, page_size, num_rows, seq_status)
PyObject *build(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 9 || !f_build) return none();
    const at::Tensor *pre = tensor(a[0]), *nw = tensor(a[1]), *cnt = tensor(a[2]), *tab = tensor(a[3]),
                     *stk = tensor(a[4]), *fc = tensor(a[5]);
    const int64_t ps = small_int(a[6]), rows = small_int(a[7]);
    const int dev = device_of(tab);
    if (dev < 0 || ps <= 0 || rows <= 0 || tab->dim() != 2 || !stk || stk->dim() != 1) return none();
    const int64_t B = tab->size(0), mp = tab->size(1), np = stk->size(0);
    bool bad = B >= (1 << 30) || mp >= (1 << 30) || np >= (1LL << 31);
    int32_t *st = status(a[8], dev, B, bad);
    if (bad || !array(tab, at::kInt, dev, {B, mp}) || !i32(stk, dev, np) || !i32(pre, dev, B) || !i32(nw, dev, B) ||
        !i32(cnt, dev, B) || !i32(fc, dev, 1))
        return none();
    // a short slot map too lies with the others (a long one would keep them all alive, or they it)
    const bool with = rows <= kShared;
    const c10::Storage all = memory((2 * B + 2 + (with ? rows : 0)) * 4);
    at::Tensor slots = with ? ints(all, 2 * B + 2, rows) : empty({rows}, at::kInt);
    at::Tensor starts = ints(all, 0, B + 1), counts = ints(all, B + 1, B), left = ints(all, 2 * B + 1, 1);
    if (f_build(ip(*pre), ip(*nw), ip(*cnt), ip(*stk), ip(*fc), (int)B, (int)ps, (int)mp, (int)np, (int)rows, ip(*tab),
                ip(starts), ip(slots), ip(counts), ip(left), st, stream_of(dev)) != SV_OK)
        return none();
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(std::move(starts)), THPVariable_Wrap(std::move(slots)),
                         THPVariable_Wrap(std::move(counts)), THPVariable_Wrap(std::move(left)));
}

// (keep_lens, page_counts, block_table, free_pages, free_count, page_size, seq_status)
PyObject *release(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 7 || !f_release) return none();
    const at::Tensor *keep = tensor(a[0]), *cnt = tensor(a[1]), *tab = tensor(a[2]), *stk = tensor(a[3]),
                     *fc = tensor(a[4]);
    const int64_t ps = small_int(a[5]);
    const int dev = device_of(tab);
    if (dev < 0 || ps <= 0 || tab->dim() != 2 || !stk || stk->dim() != 1) return none();
    const int64_t B = tab->size(0), mp = tab->size(1), np = stk->size(0);
    bool bad = B >= (1 << 30) || mp >= (1 << 30) || np >= (1LL << 31);
    int32_t *st = status(a[6], dev, B, bad);
    if (bad || !array(tab, at::kInt, dev, {B, mp}) || !i32(stk, dev, np) || !i32(keep, dev, B) || !i32(cnt, dev, B) ||
        !i32(fc, dev, 1))
        return none();
    const c10::Storage all = memory((B + 1) * 4);
    at::Tensor counts = ints(all, 0, B), left = ints(all, B, 1);
    if (f_release(ip(*keep), ip(*cnt), ip(*tab), ip(*stk), ip(*fc), (int)B, (int)ps, (int)mp, (int)np, ip(counts),
                  ip(left), st, stream_of(dev)) != SV_OK)
        return none();
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(counts)), THPVariable_Wrap(std::move(left)));
}

// Caches [num_pages, Hkv, page_size, D] of bf16 on the current device, their sizes below 2^31.
bool caches(const at::Tensor *k, const at::Tensor *v, int dev) {
    if (dev < 0 || k->dim() != 4) return false;
    for (int i = 0; i < 4; ++i)
        if (k->size(i) >= (1LL << 31)) return false;
    const auto s = k->sizes();
    return array(k, at::kBFloat16, dev, {s[0], s[1], s[2], s[3]}) &&
           array(v, at::kBFloat16, dev, {s[0], s[1], s[2], s[3]});
}

// (k_new, v_new, slot_map, k_pages, v_pages, row_status); True when done
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 6 || !f_append) return none();
    const at::Tensor *kn = tensor(a[0]), *vn = tensor(a[1]), *slots = tensor(a[2]), *k = tensor(a[3]), *v = tensor(a[4]);
    const int dev = device_of(k);
    if (!caches(k, v, dev) || !kn || !vn || kn->dim() != 3 || !kn->is_cuda() || kn->get_device() != dev ||
        !vn->is_cuda() || vn->get_device() != dev || vn->scalar_type() != kn->scalar_type() ||
        !vn->sizes().equals(kn->sizes()))
        return none();
    const int64_t rows = kn->size(0);
    const bool f32 = kn->scalar_type() == at::kFloat;
    if ((!f32 && kn->scalar_type() != at::kBFloat16) || kn->size(1) != k->size(1) || kn->size(2) != k->size(3) ||
        rows >= (1LL << 31) || !i32(slots, dev, rows))
        return none();
    bool bad = false;
    int32_t *st = status(a[5], dev, rows, bad);
    const int64_t ks = row_stride(*kn), vs = row_stride(*vn);
    if (bad || !ks || !vs) return none();
    if (f_append(kn->data_ptr(), vn->data_ptr(), f32 ? SV_F32 : SV_BF16, ks, vs, ip(*slots), (int)rows, (int)k->size(1),
                 (int)k->size(3), (int)k->size(2), (int)k->size(0), k->data_ptr(), v->data_ptr(), st,
                 stream_of(dev)) != SV_OK)
        return none();
    Py_RETURN_TRUE;
}

// (q, k_pages, v_pages, block_table, prefix_lens, row_starts, scale, window, return_lse, seq_status, workspaces):
// workspaces is api.py's dict, by (D, device, stream).
PyObject *chunk(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 11 || !f_chunk) return none();
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *tab = tensor(a[3]), *pre = tensor(a[4]),
                     *starts = tensor(a[5]);
    const int dev = device_of(k);
    const int64_t window = small_int(a[7]);
    if (!caches(k, v, dev) || !q || q->dim() != 3 || !q->is_cuda() || q->get_device() != dev ||
        q->scalar_type() != at::kBFloat16 || q->size(2) != k->size(3) || !tab || tab->dim() != 2 || window < 0 ||
        !PyFloat_CheckExact(a[6]) || !PyBool_Check(a[8]) || !PyDict_Check(a[10]))
        return none();
    const int64_t rows = q->size(0), hq = q->size(1), B = tab->size(0), mp = tab->size(1), d = q->size(2);
    bool bad = rows >= (1LL << 31) || hq >= (1LL << 31) || B >= (1 << 30) || mp >= (1 << 30);
    int32_t *st = status(a[9], dev, B, bad);
    const int64_t qs = row_stride(*q);
    if (bad || !qs || !array(tab, at::kInt, dev, {B, mp}) || !i32(pre, dev, B) || !i32(starts, dev, B + 1)) return none();
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) return none();
    PyObject *key = Py_BuildValue("(LiK)", (long long)d, dev, (unsigned long long)(uintptr_t)s);
    PyObject *held = key ? PyDict_GetItemWithError(a[10], key) : nullptr;  // (borrowed)
    Py_XDECREF(key);
    if (PyErr_Occurred()) PyErr_Clear();
    const at::Tensor *ws = held ? tensor(held) : nullptr;
    if (!ws) return none();
    at::Tensor out = empty({rows, hq, d}, at::kBFloat16), lse;
    const bool want_lse = a[8] == Py_True;
    if (want_lse) lse = empty({rows, hq}, at::kFloat);
    if (f_chunk(q->data_ptr(), qs, k->data_ptr(), v->data_ptr(), ip(*tab), (int)mp, (int)k->size(0), (int)k->size(2),
                ip(*pre), ip(*starts), (int)B, (int)rows, (int)hq, (int)k->size(1), (int)d,
                (float)PyFloat_AS_DOUBLE(a[6]), (int)window, out.data_ptr(),
                want_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, st, ws->data_ptr(), (size_t)ws->numel(),
                reinterpret_cast<sv_stream_t>(s)) != SV_OK)
        return none();
    if (!want_lse) return THPVariable_Wrap(std::move(out));
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
}

// No C++ exception (an allocation that fails, say) leaves these functions: the
// interpreted form of the call meets and reports it.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    try {
        return F(self, a, na);
    } catch (...) {
        PyErr_Clear();
        return none();
    }
}

// The addresses of the library's functions: (build, release, append, chunk); zeros turn the module off.
PyObject *use(PyObject *, PyObject *args) {
    unsigned long long b, r, p, c;
    if (!PyArg_ParseTuple(args, "KKKK", &b, &r, &p, &c)) return nullptr;
    f_build = reinterpret_cast<decltype(f_build)>((uintptr_t)b);
    f_release = reinterpret_cast<decltype(f_release)>((uintptr_t)r);
    f_append = reinterpret_cast<decltype(f_append)>((uintptr_t)p);
    f_chunk = reinterpret_cast<decltype(f_chunk)>((uintptr_t)c);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"use", use, METH_VARARGS, nullptr},
                         {"build_block_tables", fast(guarded<build>), METH_FASTCALL, nullptr},
                         {"release_pages", fast(guarded<release>), METH_FASTCALL, nullptr},
                         {"append_kv_paged", fast(guarded<append>), METH_FASTCALL, nullptr},
                         {"chunk_attention_paged", fast(guarded<chunk>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sv_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sv_bind(void) { return PyModule_Create(&module); }
