// fastcall.cpp -- the everyday case of the paged-cache calls of binding.py, as a CPython extension.
//
// These calls are made once per token and layer, and the interpreter's share of one (a dozen attribute
// checks, fifteen converted arguments, two allocations) is longer than a small kernel: a paged_attn call takes
// the host 5.6 us with this and 11.7 without, of which the launch is 2.9.
// Each function here checks the same as its namesake in binding.py and makes the same library
// call; where anything is out of the ordinary (another device or stream, no workspace, tensors given
// for the outputs, a check that fails) it returns NotImplemented and binding.py goes on, with its
// own checks and messages.  It keeps nothing between calls but what setup() gave it.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "streamkl.h"

namespace {

decltype(&streamkl_paged_attn) g_attn = nullptr;
decltype(&streamkl_paged_kl) g_kl = nullptr;
decltype(&streamkl_cache_append) g_append = nullptr;
decltype(&streamkl_cache_gather) g_gather = nullptr;

// What an odd case does: an exception (of an argument that is no number, say) is dropped, so that binding.py meets
// it and words it.
PyObject* go_on() {
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}

// A plain tensor (no subclass) of this type on this device, contiguous, with `dims` dimensions of 1 to 2^31 - 1;
// nullptr otherwise.
const at::Tensor* plain(PyObject* o, at::ScalarType type, long device, int dims) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.scalar_type() != type || t.get_device() != device || t.dim() != dims || !t.is_contiguous())
        return nullptr;
    for (const auto n : t.sizes())
        if (n < 1 || n > 0x7fffffff) return nullptr;
    return &t;
}

// int32 [B] on the device.
const int* ints(PyObject* o, long device, long B) {
    const at::Tensor* t = plain(o, at::kInt, device, 1);
    return t && t->size(0) == B ? static_cast<const int*>(t->data_ptr()) : nullptr;
}

// int32 [B, width] on the device.
const int* page_table(PyObject* o, long device, long B, int* width) {
    const at::Tensor* t = plain(o, at::kInt, device, 2);
    if (!t || t->size(0) != B) return nullptr;
    *width = (int)t->size(1);
    return static_cast<const int*>(t->data_ptr());
}

uint16_t* bf16(const at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }
float* fp32(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// What both attention and divergence take.
struct Common {
    const streamkl_cache* cache;
    long device;
    const at::Tensor *q, *workspace;
    const int *table, *lengths;
    int width, B, Hq, NQ, causal;
    float scale;
    size_t bytes;
    void* stream;

    bool take(PyObject* address, PyObject* index, PyObject* queries, PyObject* pages, PyObject* tokens, PyObject* scale_, PyObject* causal_,
              PyObject* space) {
        cache = static_cast<const streamkl_cache*>(PyLong_AsVoidPtr(address));
        device = PyLong_AsLong(index);
        scale = (float)PyFloat_AsDouble(scale_);
        causal = PyObject_IsTrue(causal_);
        if (PyErr_Occurred() || !cache || causal < 0) return false;
        q = plain(queries, at::kBFloat16, device, 4);
        if (!q || q->size(3) != cache->d || q->size(1) % cache->Hkv) return false;
        B = (int)q->size(0);
        Hq = (int)q->size(1);
        NQ = (int)q->size(2);
        table = page_table(pages, device, B, &width);
        lengths = ints(tokens, device, B);
        if (!table || !lengths || !THPVariable_CheckExact(space)) return false;
        workspace = plain(space, at::kFloat, device, 1);
        if (!workspace || c10::cuda::current_device() != device) return false;
        bytes = (size_t)workspace->numel() * sizeof(float);
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        return true;
    }
    at::Tensor rows() const { return at::empty({B, Hq, NQ}, workspace->options()); }
};

// setup(addresses of attn, kl, append, gather)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "setup takes 4 addresses");
        return nullptr;
    }
    void* f[4];
    for (int i = 0; i < 4; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    g_attn = reinterpret_cast<decltype(g_attn)>(f[0]);
    g_kl = reinterpret_cast<decltype(g_kl)>(f[1]);
    g_append = reinterpret_cast<decltype(g_append)>(f[2]);
    g_gather = reinterpret_cast<decltype(g_gather)>(f[3]);
    Py_RETURN_NONE;
}

// attn(q, cache address, device, table, lengths, scale, causal, workspace): (status, out, lse) or NotImplemented
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        Common c;
        if (n != 8 || !g_attn || !c.take(a[1], a[2], a[0], a[3], a[4], a[5], a[6], a[7]) || !c.cache->v) return go_on();
        at::Tensor out = at::empty(c.q->sizes(), c.q->options()), lse = c.rows();
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = g_attn(c.cache, bf16(*c.q), c.table, c.width, c.lengths, c.B, c.Hq, c.NQ, c.scale, c.causal, bf16(out), fp32(lse),
                    c.workspace->data_ptr(), c.bytes, c.stream);
        Py_END_ALLOW_THREADS
        return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
    } catch (const std::exception&) {      // out of memory, say: binding.py allocates again and words it
        return go_on();
    }
}

// kl(q1, cache1 address, q2, cache2 address, device, table, lengths, scale, causal, workspace):
// (status, (kl, lse1, lse2)) or NotImplemented
PyObject* kl(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        Common c;
        if (n != 10 || !g_kl || !c.take(a[1], a[4], a[0], a[5], a[6], a[7], a[8], a[9])) return go_on();
        const auto* cache2 = static_cast<const streamkl_cache*>(PyLong_AsVoidPtr(a[3]));
        const at::Tensor* q2 = plain(a[2], at::kBFloat16, c.device, 4);
        if (!cache2 || !q2 || q2->sizes() != c.q->sizes() || cache2->pages != c.cache->pages || cache2->Hkv != c.cache->Hkv ||
            cache2->page_size != c.cache->page_size || cache2->d != c.cache->d)
            return go_on();
        at::Tensor out[3] = {c.rows(), c.rows(), c.rows()};
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = g_kl(c.cache, bf16(*c.q), cache2, bf16(*q2), c.table, c.width, c.lengths, c.B, c.Hq, c.NQ, c.scale, c.causal, fp32(out[0]),
                  fp32(out[1]), fp32(out[2]), c.workspace->data_ptr(), c.bytes, c.stream);
        Py_END_ALLOW_THREADS
        return Py_BuildValue("(i(NNN))", rc, THPVariable_Wrap(std::move(out[0])), THPVariable_Wrap(std::move(out[1])),
                             THPVariable_Wrap(std::move(out[2])));
    } catch (const std::exception&) {
        return go_on();
    }
}

// move(cache address, device, append, k, v, table, start or None, count or None): status or NotImplemented
PyObject* move(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        if (n != 8 || !g_append || !g_gather) return go_on();
        const auto* cache = static_cast<const streamkl_cache*>(PyLong_AsVoidPtr(a[0]));
        const long device = PyLong_AsLong(a[1]);
        const int append = PyObject_IsTrue(a[2]);
        if (PyErr_Occurred() || !cache || append < 0 || !cache->v) return go_on();
        const at::Tensor *k = plain(a[3], at::kBFloat16, device, 4), *v = plain(a[4], at::kBFloat16, device, 4);
        if (!k || !v || k->sizes() != v->sizes() || k->size(1) != cache->Hkv || k->size(3) != cache->d) return go_on();
        const int B = (int)k->size(0), NT = (int)k->size(2);
        int width = 0;
        const int *table = page_table(a[5], device, B, &width), *start = nullptr, *count = nullptr;
        if (!table || (a[6] != Py_None && !(start = ints(a[6], device, B))) || (a[7] != Py_None && !(count = ints(a[7], device, B))))
            return go_on();
        if (c10::cuda::current_device() != device) return go_on();
        void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = append ? g_append(cache, bf16(*k), bf16(*v), table, width, start, count, B, NT, stream)
                    : g_gather(cache, table, width, start, count, B, NT, bf16(*k), bf16(*v), stream);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(rc);
    } catch (const std::exception&) {
        return go_on();
    }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<setup>("setup"), method<attn>("attn"), method<kl>("kl"), method<move>("move"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&g_module); }
