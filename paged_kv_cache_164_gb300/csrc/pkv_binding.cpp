// The tree step's Python calls in their usual form, marshalled in C++: every
// tensor given, dense, of the right type, on the current device, launched on its
// current stream.  A call of that form goes straight to the C ABI (reading a
// dozen tensors takes 1 us here and 5 to 9 us in Python, and the kernels of small
// batches take 2); any other form (outputs or a workspace to allocate, another
// stream or device, an argument to refuse) returns None, launches nothing and is
// left to the Python code, whose checks and messages are the binding's.
#include <climits>
#include <cmath>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pkv.h"

namespace {

// The C entry points, of whichever library the Python side has loaded.
decltype(&pkv_norm_rope_append) fn_norm_rope_append = nullptr;
decltype(&pkv_norm_rope_append_fp8) fn_norm_rope_append_fp8 = nullptr;
decltype(&pkv_tree_plan) fn_tree_plan = nullptr;
decltype(&pkv_tree_attention) fn_tree_attention = nullptr;
decltype(&pkv_tree_commit_within) fn_tree_commit = nullptr;

// Reads a call's arguments; `ok` stays true while they have the usual form.
struct Reader {
    bool ok = true;
    int device = -1;

    const at::Tensor* tensor(PyObject* o) {
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    // The call's first tensor: it says the device, which must be the current one.
    const at::Tensor* first(PyObject* o, int64_t dims) {
        const at::Tensor* t = tensor(o);
        if (!ok) return nullptr;
        if (!t->is_cuda() || t->dim() != dims || t->layout() != at::kStrided) {
            ok = false;
            return nullptr;
        }
        device = t->get_device();
        if (c10::cuda::current_device() != device) ok = false;
        return t;
    }
    const at::Tensor* typed(PyObject* o, at::ScalarType type) {
        const at::Tensor* t = tensor(o);
        if (!ok) return nullptr;
        if (!t->is_cuda() || t->scalar_type() != type || t->get_device() != device ||
            t->layout() != at::kStrided)
            ok = false;
        return ok ? t : nullptr;
    }
    // A dense tensor of a type on the call's device, of the given sizes.
    void* dense(PyObject* o, at::ScalarType type, at::IntArrayRef sizes) {
        const at::Tensor* t = typed(o, type);
        if (!ok) return nullptr;
        if (!t->is_contiguous() || t->sizes() != sizes) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void* optional(PyObject* o, at::ScalarType type, at::IntArrayRef sizes) {
        return o == Py_None ? nullptr : dense(o, type, sizes);
    }
    // The optional error word: any dense int32 tensor.
    int32_t* flag(PyObject* o) {
        if (o == Py_None) return nullptr;
        const at::Tensor* t = typed(o, at::kInt);
        if (!ok) return nullptr;
        if (!t->is_contiguous()) ok = false;
        return ok ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
    }
    // [tokens, heads, d] rows whose heads are dense, and the elements between tokens.
    void* rows(PyObject* o, at::ScalarType type, int64_t n, int64_t heads, int64_t d,
               int64_t* stride) {
        const at::Tensor* t = typed(o, type);
        if (!ok) return nullptr;
        if (t->dim() != 3 || t->size(0) != n || t->size(1) != heads || t->size(2) != d ||
            (n > 0 && (t->stride(2) != 1 || (heads > 1 && t->stride(1) != d)))) {
            ok = false;
            return nullptr;
        }
        *stride = n > 1 ? t->stride(0) : heads * d;
        return t->data_ptr();
    }
    int integer(PyObject* o) {
        if (!PyLong_CheckExact(o)) {
            ok = false;
            return 0;
        }
        int overflow = 0;
        const long v = PyLong_AsLongAndOverflow(o, &overflow);
        if (overflow || v < INT_MIN || v > INT_MAX) ok = false;
        return ok ? static_cast<int>(v) : 0;
    }
    float real(PyObject* o) {
        if (!PyFloat_CheckExact(o)) {
            ok = false;
            return 0.f;
        }
        return static_cast<float>(PyFloat_AS_DOUBLE(o));
    }
    int narrow(int64_t v) {
        if (v > INT_MAX) ok = false;
        return static_cast<int>(v);
    }
    bool says(PyObject* o, const char* a, const char* b, bool* is_b) {
        if (PyUnicode_Check(o)) {
            if (PyUnicode_CompareWithASCIIString(o, a) == 0) {
                *is_b = false;
                return true;
            }
            if (PyUnicode_CompareWithASCIIString(o, b) == 0) {
                *is_b = true;
                return true;
            }
        }
        ok = false;
        return false;
    }
};

// A call's two caches and the dtype argument.
struct Caches {
    void *k = nullptr, *v = nullptr;
    int num_blocks = 0, block_size = 0, heads = 0, d = 0;
    pkv_dtype code = PKV_FP16;

    Caches(Reader& r, PyObject* k_obj, PyObject* v_obj, PyObject* layout, at::ScalarType type,
           at::ScalarType activations) {
        bool hnd = false;
        if (!r.ok || !r.says(layout, "nhd", "hnd", &hnd)) return;
        const at::Tensor* t = r.typed(k_obj, type);
        if (!r.ok) return;
        if (t->dim() != 4 || !t->is_contiguous() ||
            (activations != at::kHalf && activations != at::kBFloat16)) {
            r.ok = false;
            return;
        }
        k = t->data_ptr();
        v = r.dense(v_obj, type, t->sizes());
        num_blocks = r.narrow(t->size(0));
        block_size = r.narrow(t->size(hnd ? 2 : 1));
        heads = r.narrow(t->size(hnd ? 1 : 2));
        d = r.narrow(t->size(3));
        code = static_cast<pkv_dtype>((activations == at::kBFloat16 ? PKV_BF16 : PKV_FP16) |
                                      (hnd ? PKV_LAYOUT_HND : 0));
    }
};

// A call of the C ABI without Python's lock: a launch waits where the device's queue
// is full, and other threads go on meanwhile.  (All arguments are read before it.)
struct Unlocked {  // (the lock is back however the call is left)
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
pkv_status run_unlocked(F call) {
    Unlocked u;
    return call();
}
template <typename F>
PyObject* unlocked(F call) {
    return PyLong_FromLong(run_unlocked(call));
}

void* stream_of(int device) {
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
}

// (q, k, v, positions, cos_sin, k_cache, v_cache, slot_mapping, q_weight, k_weight,
//  eps, style, q_out, err_flag, layout[, k_scale, v_scale])
PyObject* norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if ((n != 15 && n != 17) || fn_norm_rope_append == nullptr) Py_RETURN_NONE;
    const bool f8 = n == 17;
    Reader r;
    const at::Tensor* q = r.first(a[0], 3);
    if (!r.ok) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int64_t t = q->size(0), h_q = q->size(1), d = q->size(2);
    const Caches c(r, a[5], a[6], a[14], f8 ? at::kByte : type, type);
    if (!r.ok || c.d != d) Py_RETURN_NONE;
    int64_t qs = 0, ks = 0, vs = 0;
    const void* qp = r.rows(a[0], type, t, h_q, d, &qs);
    const void* kp = r.rows(a[1], type, t, c.heads, d, &ks);
    const void* vp = r.rows(a[2], type, t, c.heads, d, &vs);
    const int64_t one[1] = {t}, width[1] = {d}, out_sizes[3] = {t, h_q, d};
    const void* pos = r.dense(a[3], at::kInt, one);
    const at::Tensor* table = r.typed(a[4], at::kFloat);
    if (!r.ok || table->dim() != 2 || !table->is_contiguous()) Py_RETURN_NONE;
    const void* slots = r.dense(a[7], at::kLong, one);
    const void* qw = r.optional(a[8], type, width);
    const void* kw = r.optional(a[9], type, width);
    const float eps = r.real(a[10]);
    bool inter = false;
    r.says(a[11], "half", "interleaved", &inter);
    void* out = r.dense(a[12], type, out_sizes);
    int32_t* flag = r.flag(a[13]);
    const float k_scale = f8 ? r.real(a[15]) : 1.f, v_scale = f8 ? r.real(a[16]) : 1.f;
    const int tokens = r.narrow(t), heads = r.narrow(h_q), npos = r.narrow(table->size(0)),
              rd = r.narrow(table->size(1));
    if (!r.ok) Py_RETURN_NONE;
    void* st = stream_of(r.device);
    const float* tab = static_cast<const float*>(table->data_ptr());
    const int32_t* ps = static_cast<const int32_t*>(pos);
    const int64_t* sl = static_cast<const int64_t*>(slots);
    return unlocked([&] {
        return f8 ? fn_norm_rope_append_fp8(out, qp, qs, kp, ks, vp, vs, qw, kw, eps, tab, npos,
                                            rd, inter, ps, c.k, c.v, sl, tokens, c.num_blocks,
                                            c.block_size, heads, c.heads, c.d, k_scale, v_scale,
                                            c.code, flag, st)
                  : fn_norm_rope_append(out, qp, qs, kp, ks, vp, vs, qw, kw, eps, tab, npos, rd,
                                        inter, ps, c.k, c.v, sl, tokens, c.num_blocks,
                                        c.block_size, heads, c.heads, c.d, c.code, flag, st);
    });
}

// (parents, context_lens, block_tables, num_blocks, block_size, max_context_len,
//  tree_mask, positions, slot_mapping, err_flag)
PyObject* tree_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 10 || fn_tree_plan == nullptr) Py_RETURN_NONE;
    Reader r;
    const at::Tensor* parents = r.first(a[0], 2);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t b = parents->size(0), t = parents->size(1);
    const int64_t seqs[1] = {b}, nodes[2] = {b, t}, mask_sizes[3] = {b, t, (t + 31) / 32};
    const void* par = r.dense(a[0], at::kInt, nodes);
    const void* lens = r.dense(a[1], at::kInt, seqs);
    const at::Tensor* tables = r.typed(a[2], at::kInt);
    if (!r.ok || tables->dim() != 2 || tables->size(0) != b || !tables->is_contiguous())
        Py_RETURN_NONE;
    const int nb = r.integer(a[3]), bs = r.integer(a[4]), cap = r.integer(a[5]);
    void* mask = r.dense(a[6], at::kInt, mask_sizes);
    void* pos = r.dense(a[7], at::kInt, nodes);
    void* slots = r.dense(a[8], at::kLong, nodes);
    int32_t* flag = r.flag(a[9]);
    const int width = r.narrow(tables->size(1)), batch = r.narrow(b), len = r.narrow(t);
    if (!r.ok) Py_RETURN_NONE;
    const int32_t* tab = static_cast<const int32_t*>(tables->data_ptr());
    void* st = stream_of(r.device);
    return unlocked([&] {
        return fn_tree_plan(static_cast<int32_t*>(mask), static_cast<int32_t*>(pos),
                            static_cast<int64_t*>(slots), static_cast<const int32_t*>(par),
                            static_cast<const int32_t*>(lens), tab, width, cap, batch, len, nb,
                            bs, flag, st);
    });
}

// (q, k_cache, v_cache, block_tables, context_lens, max_context_len, tree_mask,
//  scale, out, workspace, err_flag, layout)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 12 || fn_tree_attention == nullptr) Py_RETURN_NONE;
    Reader r;
    const at::Tensor* q = r.first(a[0], 4);
    if (!r.ok) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int64_t b = q->size(0), t = q->size(1), h_q = q->size(2), d = q->size(3);
    const int64_t words = (t + 31) / 32;
    const Caches c(r, a[1], a[2], a[11], type, type);
    if (!r.ok || c.d != d) Py_RETURN_NONE;
    const int64_t seqs[1] = {b};
    const void* qp = r.dense(a[0], type, q->sizes());
    const at::Tensor* tables = r.typed(a[3], at::kInt);
    if (!r.ok || tables->dim() != 2 || tables->size(0) != b || !tables->is_contiguous())
        Py_RETURN_NONE;
    const void* lens = r.dense(a[4], at::kInt, seqs);
    const int cap = r.integer(a[5]);
    const at::Tensor* mask = r.typed(a[6], at::kInt);
    if (!r.ok || mask->dim() != 3 || (mask->size(0) != b && mask->size(0) != 1) ||
        mask->size(1) != t || mask->size(2) != words ||
        (mask->size(0) > 0 && ((words > 1 && mask->stride(2) != 1) ||
                               (t > 1 && mask->stride(1) != words))))
        Py_RETURN_NONE;
    const int64_t mask_stride = mask->size(0) > 1 ? mask->stride(0) : 0;
    const float scale = a[7] == Py_None && d > 0
                            ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)))
                            : r.real(a[7]);
    void* out = r.dense(a[8], type, q->sizes());
    const at::Tensor* ws = r.ok ? r.tensor(a[9]) : nullptr;
    if (!r.ok || !ws->is_cuda() || ws->get_device() != r.device || !ws->is_contiguous())
        Py_RETURN_NONE;
    int32_t* flag = r.flag(a[10]);
    const int width = r.narrow(tables->size(1)), batch = r.narrow(b), len = r.narrow(t),
              heads = r.narrow(h_q);
    if (!r.ok) Py_RETURN_NONE;
    const int32_t* tab = static_cast<const int32_t*>(tables->data_ptr());
    const int32_t* bits = static_cast<const int32_t*>(mask->data_ptr());
    void* ws_ptr = ws->data_ptr();
    const size_t ws_bytes = ws->nbytes();
    void* st = stream_of(r.device);
    return unlocked([&] {
        return fn_tree_attention(out, qp, c.k, c.v, tab, width, static_cast<const int32_t*>(lens),
                                 cap, bits, mask_stride, batch, len, c.num_blocks, c.block_size,
                                 heads, c.heads, c.d, scale, ws_ptr, ws_bytes, c.code, flag, st);
    });
}

// (k_cache, v_cache, block_tables, context_lens, tree_len, accepted, accepted_lens,
//  new_context_lens, err_flag, layout, max_context_len)
PyObject* tree_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 11 || fn_tree_commit == nullptr) Py_RETURN_NONE;
    Reader r;
    const at::Tensor* k = r.first(a[0], 4);
    if (!r.ok) Py_RETURN_NONE;
    const Caches c(r, a[0], a[1], a[9], k->scalar_type(), k->scalar_type());
    const at::Tensor* tables = r.ok ? r.typed(a[2], at::kInt) : nullptr;
    if (!r.ok || tables->dim() != 2 || !tables->is_contiguous()) Py_RETURN_NONE;
    const int64_t b = tables->size(0);
    const int64_t seqs[1] = {b};
    const void* lens = r.dense(a[3], at::kInt, seqs);
    const int len = r.integer(a[4]);
    const at::Tensor* accepted = r.ok ? r.typed(a[5], at::kInt) : nullptr;
    if (!r.ok || accepted->dim() != 2 || accepted->size(0) != b || !accepted->is_contiguous())
        Py_RETURN_NONE;
    const void* counts = r.dense(a[6], at::kInt, seqs);
    void* fresh = r.dense(a[7], at::kInt, seqs);
    int32_t* flag = r.flag(a[8]);
    const int cap = a[10] == Py_None ? INT_MAX : r.integer(a[10]);
    const int width = r.narrow(tables->size(1)), batch = r.narrow(b),
              most = r.narrow(accepted->size(1));
    if (!r.ok) Py_RETURN_NONE;
    const int32_t* tab = static_cast<const int32_t*>(tables->data_ptr());
    const int32_t* path = static_cast<const int32_t*>(accepted->data_ptr());
    void* st = stream_of(r.device);
    return unlocked([&] {
        return fn_tree_commit(c.k, c.v, tab, width, static_cast<const int32_t*>(lens), cap, len,
                              path, static_cast<const int32_t*>(counts), most,
                              static_cast<int32_t*>(fresh), batch, c.num_blocks, c.block_size,
                              c.heads, c.d, c.code, flag, st);
    });
}

// C++ exceptions (a tensor without storage, a CUDA error) become "not the usual form".
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(self, args, n);
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// bind(addresses of norm_rope_append, norm_rope_append_fp8, tree_plan,
//      tree_attention, tree_commit_within)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    fn_norm_rope_append = reinterpret_cast<decltype(fn_norm_rope_append)>(p[0]);
    fn_norm_rope_append_fp8 = reinterpret_cast<decltype(fn_norm_rope_append_fp8)>(p[1]);
    fn_tree_plan = reinterpret_cast<decltype(fn_tree_plan)>(p[2]);
    fn_tree_attention = reinterpret_cast<decltype(fn_tree_attention)>(p[3]);
    fn_tree_commit = reinterpret_cast<decltype(fn_tree_commit)>(p[4]);
    Py_RETURN_NONE;
}

#define PKV_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", PKV_FAST(bind), nullptr},
    {"norm_rope_append", PKV_FAST(guarded<norm_rope_append>), nullptr},
    {"tree_plan", PKV_FAST(guarded<tree_plan>), nullptr},
    {"tree_attention", PKV_FAST(guarded<tree_attention>), nullptr},
    {"tree_commit", PKV_FAST(guarded<tree_commit>), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pkv_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pkv_binding() {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", PKV_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
