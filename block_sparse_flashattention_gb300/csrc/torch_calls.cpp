// The cache calls as Python functions over torch tensors: what an ordinary call needs of
// checking, output allocation and argument marshalling, in one native call each.
//
// A function returns None when an argument is not of the ordinary kind; kv_cache.py then
// runs the same checks in Python, which name what is wrong or marshal the call through
// ctypes.  Otherwise it calls the C entry (its address given once by bind()) and returns
// the outputs, or the status as an int where that is not BSATTN_OK.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "bsattn.h"

namespace {

decltype(&bsattn_kv_append) g_append = nullptr;
decltype(&bsattn_kv_read) g_read = nullptr;
decltype(&bsattn_decode) g_decode = nullptr;
decltype(&bsattn_decode_shared_prefix) g_prefix = nullptr;

struct Cache {
    const bsattn_kv_cache *c;
    int64_t device;
};

bool tensor(PyObject *o, const at::Tensor **t) {
    if (!THPVariable_Check(o)) return false;
    *t = &THPVariable_Unpack(o);
    return true;
}

bool cache(PyObject *address, PyObject *device, Cache *c) {
    c->c = static_cast<const bsattn_kv_cache *>(PyLong_AsVoidPtr(address));
    c->device = PyLong_AsLongLong(device);
    return c->c && c->device >= 0 && c10::cuda::current_device() == c->device;
}

// A contiguous int32 tensor of `dims` dimensions on the cache's device.
bool ints(const at::Tensor &t, int64_t dims, int64_t device) {
    return t.dim() == dims && t.scalar_type() == at::kInt && t.is_cuda() && t.get_device() == device && t.is_contiguous();
}

const int32_t *int_ptr(const at::Tensor &t) { return static_cast<const int32_t *>(t.data_ptr()); }

// bf16 rows [tokens, H, D] whose [H, D] part is contiguous; *stride: elements from token to token.
bool rows(const at::Tensor &t, int64_t H, int64_t D, int64_t device, int64_t *stride) {
    if (t.dim() != 3 || t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != device) return false;
    if (t.size(1) != H || t.size(2) != D || t.stride(2) != 1 || (t.stride(1) != D && H > 1)) return false;
    *stride = t.size(0) > 1 ? t.stride(0) : H * D;
    return true;
}

bool no(PyObject *o) { return o == Py_None; }

PyObject *none() { Py_RETURN_NONE; }

void *stream_of(int64_t device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

bool small_dims(const at::Tensor &t) {
    for (int64_t i = 0; i < t.dim(); ++i)
        if (t.size(i) > INT32_MAX) return false;
    return true;
}

// Fills *m from a Meta; false where a tensor is not a contiguous int32 one on `device`.
bool fill_meta(PyObject *o, int64_t device, bsattn_meta *m) {
    struct Field {
        const char *name;
        int32_t **to;
    };
    const Field arrays[] = {{"full_cnt", &m->full_cnt}, {"full_idx", &m->full_idx}, {"mask_cnt", &m->mask_cnt},
                            {"mask_idx", &m->mask_idx}, {"cu_total_m_blocks", &m->cu_total_m_blocks},
                            {"cu_block_idx_offsets", &m->cu_block_idx_offsets}};
    for (const Field &f : arrays) {
        PyObject *x = PyObject_GetAttrString(o, f.name);
        if (!x) return false;
        const at::Tensor *t = nullptr;
        const bool none = x == Py_None;
        const bool ok = none || (tensor(x, &t) && t->scalar_type() == at::kInt && t->is_cuda() &&
                                 t->get_device() == device && t->is_contiguous());
        if (ok) *f.to = none ? nullptr : static_cast<int32_t *>(t->data_ptr());
        Py_DECREF(x);
        if (!ok) return false;
    }
    struct Number {
        const char *name;
        int32_t *to;
    };
    const Number numbers[] = {{"varlen", &m->varlen}, {"B", &m->B}, {"H", &m->H}, {"num_m", &m->num_m},
                              {"num_n", &m->num_n}, {"total_m_blocks", &m->total_m_blocks},
                              {"total_n_blocks", &m->total_n_blocks}, {"tile_m", &m->tile_m}, {"tile_n", &m->tile_n}};
    for (const Number &f : numbers) {
        PyObject *x = PyObject_GetAttrString(o, f.name);
        if (!x) return false;
        const long long v = PyLong_AsLongLong(x);
        Py_DECREF(x);
        if (v == -1 && PyErr_Occurred()) return false;
        if (v < INT32_MIN || v > INT32_MAX) return false;
        *f.to = (int32_t)v;
    }
    return true;
}

// bind(append, read, decode, decode_shared_prefix): addresses of the C entries.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind takes 4 addresses");
        return nullptr;
    }
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[0]));
    g_read = reinterpret_cast<decltype(g_read)>(PyLong_AsVoidPtr(a[1]));
    g_decode = reinterpret_cast<decltype(g_decode)>(PyLong_AsVoidPtr(a[2]));
    g_prefix = reinterpret_cast<decltype(g_prefix)>(PyLong_AsVoidPtr(a[3]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// kv_append(cache address, device, k, v, page_table, seqlens, cu_seqlens | None)
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    const at::Tensor *k, *v, *table, *lens, *cu = nullptr;
    if (n != 7 || !cache(a[0], a[1], &c)) return PyErr_Occurred() ? nullptr : none();
    if (!tensor(a[2], &k) || !tensor(a[3], &v) || !tensor(a[4], &table) || !tensor(a[5], &lens)) return none();
    if (!no(a[6]) && !tensor(a[6], &cu)) return none();
    int64_t ks, vs;
    if (!rows(*k, c.c->H, c.c->D, c.device, &ks) || !rows(*v, c.c->H, c.c->D, c.device, &vs)) return none();
    if (!ints(*table, 2, c.device) || !ints(*lens, 1, c.device)) return none();
    const int64_t B = table->size(0);
    if (v->size(0) != k->size(0) || lens->size(0) != B || !small_dims(*k) || !small_dims(*table)) return none();
    if (cu && (!ints(*cu, 1, c.device) || cu->size(0) != B + 1)) return none();
    const int32_t cols = (int32_t)table->size(1);
    const bsattn_status st = g_append(k->data_ptr(), v->data_ptr(), ks, vs, (int32_t)k->size(0), (int32_t)B,
                                      cu ? int_ptr(*cu) : nullptr, int_ptr(*table), cols, cols, int_ptr(*lens), c.c,
                                      nullptr, stream_of(c.device));
    return PyLong_FromLong(st);
}

// kv_read(cache address, device, page_table, cu_seqlens, total) -> (k, v)
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    const at::Tensor *table, *cu;
    if (n != 5 || !cache(a[0], a[1], &c)) return PyErr_Occurred() ? nullptr : none();
    if (!tensor(a[2], &table) || !tensor(a[3], &cu) || !PyLong_Check(a[4])) return none();
    const int64_t total = PyLong_AsLongLong(a[4]);
    if (total < 0 || total > INT32_MAX) {
        PyErr_Clear();
        return none();
    }
    if (!ints(*table, 2, c.device) || !ints(*cu, 1, c.device)) return none();
    const int64_t B = table->size(0);
    if (cu->size(0) != B + 1 || !small_dims(*table)) return none();
    const auto opt = table->options().dtype(at::kBFloat16);
    const int64_t shape[3] = {total, c.c->H, c.c->D};
    at::Tensor k = at::empty(shape, opt), v = at::empty(shape, opt);
    const int32_t cols = (int32_t)table->size(1);
    const bsattn_status st = g_read(c.c, int_ptr(*table), cols, cols, (int32_t)B, int_ptr(*cu), (int32_t)total,
                                    k.data_ptr(), v.data_ptr(), nullptr, stream_of(c.device));
    if (st != BSATTN_OK) return PyLong_FromLong(st);
    return Py_BuildValue("NN", THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v)));
}

// decode(cache address, device, q, page_table | None, seqlens, softmax_scale, workspace,
//        meta | None, prefix_table | None, prefix_len) -> (out, lse)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    const at::Tensor *q, *table = nullptr, *lens, *ws, *pre = nullptr;
    if (n != 10 || !cache(a[0], a[1], &c)) return PyErr_Occurred() ? nullptr : none();
    if (!tensor(a[2], &q) || (!no(a[3]) && !tensor(a[3], &table)) || !tensor(a[4], &lens) || !tensor(a[6], &ws)) return none();
    if ((!no(a[8]) && !tensor(a[8], &pre)) || !PyLong_Check(a[9])) return none();
    const double scale = PyFloat_AsDouble(a[5]);
    const int64_t prefix_len = PyLong_AsLongLong(a[9]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    if (q->dim() != 3) return none();
    const int64_t B = q->size(0), Hq = q->size(1);
    int64_t qs;
    if (!rows(*q, Hq, c.c->D, c.device, &qs) || !small_dims(*q)) return none();
    if (table ? !ints(*table, 2, c.device) || table->size(0) != B || !small_dims(*table) : !pre) return none();
    if (!ints(*lens, 1, c.device) || lens->size(0) != B) return none();
    if (!ws->is_cuda() || ws->get_device() != c.device || !ws->is_contiguous()) return none();
    if (pre && (!ints(*pre, 1, c.device) || prefix_len < 0 || prefix_len > pre->size(0) * c.c->page_size ||
                prefix_len > INT32_MAX))
        return none();
    bsattn_meta meta = {};
    if (!no(a[7]) && !fill_meta(a[7], c.device, &meta)) {
        PyErr_Clear();
        return none();
    }
    const int64_t shape[3] = {B, Hq, c.c->D}, lse_shape[2] = {B, Hq};
    at::Tensor out = at::empty(shape, q->options()), lse = at::empty(lse_shape, q->options().dtype(at::kFloat));
    const bsattn_meta *m = no(a[7]) ? nullptr : &meta;
    const int32_t cols = table ? (int32_t)table->size(1) : 0;
    const int32_t *pages = table ? int_ptr(*table) : nullptr;
    float *l = static_cast<float *>(lse.data_ptr());
    const bsattn_status st =
        pre ? g_prefix(q->data_ptr(), qs, (int32_t)B, (int32_t)Hq, c.c, int_ptr(*pre), (int32_t)prefix_len, pages, cols,
                       cols, int_ptr(*lens), m, nullptr, (float)scale, out.data_ptr(), BSATTN_OUT_BF16, l,
                       ws->data_ptr(), ws->nbytes(), nullptr, stream_of(c.device))
            : g_decode(q->data_ptr(), qs, (int32_t)B, (int32_t)Hq, c.c, pages, cols, cols, int_ptr(*lens), m, nullptr,
                       (float)scale, out.data_ptr(), BSATTN_OUT_BF16, l, ws->data_ptr(), ws->nbytes(), nullptr,
                       stream_of(c.device));
    if (st != BSATTN_OK) return PyLong_FromLong(st);
    return Py_BuildValue("NN", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
}

// The torch release this was compiled against; kv_cache.py uses it with no other.
PyObject *torch_version(PyObject *, PyObject *const *, Py_ssize_t) { return PyUnicode_FromString(TORCH_VERSION); }

// C++ exceptions (an allocation that fails) become torch's Python errors.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    return F(self, a, n);
    END_HANDLE_TH_ERRORS
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(torch_version), ENTRY(bind), ENTRY(kv_append), ENTRY(kv_read), ENTRY(decode), {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
