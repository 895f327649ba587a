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
decltype(&bsattn_prefill) g_prefill = nullptr;
decltype(&bsattn_kv_weigh) g_weigh = nullptr;
decltype(&bsattn_kv_evict) g_evict = nullptr;

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
    if (t.size(1) != H || t.size(2) != D || t.numel() == 0 || t.stride(2) != 1 || (t.stride(1) != D && H > 1)) return false;
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

// bind(append, read, decode, decode_shared_prefix, prefill, kv_weigh, kv_evict): addresses of the C entries.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "bind takes 7 addresses");
        return nullptr;
    }
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[0]));
    g_read = reinterpret_cast<decltype(g_read)>(PyLong_AsVoidPtr(a[1]));
    g_decode = reinterpret_cast<decltype(g_decode)>(PyLong_AsVoidPtr(a[2]));
    g_prefix = reinterpret_cast<decltype(g_prefix)>(PyLong_AsVoidPtr(a[3]));
    g_prefill = reinterpret_cast<decltype(g_prefill)>(PyLong_AsVoidPtr(a[4]));
    g_weigh = reinterpret_cast<decltype(g_weigh)>(PyLong_AsVoidPtr(a[5]));
    g_evict = reinterpret_cast<decltype(g_evict)>(PyLong_AsVoidPtr(a[6]));
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

// A number of an argument or attribute; false where it is none that fits 32 bits.
bool int32_of(PyObject *o, int32_t *x) {
    if (!PyLong_Check(o)) return false;
    const long long v = PyLong_AsLongLong(o);
    if ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX) {
        PyErr_Clear();
        return false;
    }
    *x = (int32_t)v;
    return true;
}

// kind and the numbers of a MaskParams (None: no parameters).
struct Mask {
    int32_t kind;
    bsattn_mask_params params;
    const bsattn_mask_params *given;
};

bool mask(PyObject *kind, PyObject *params, Mask *m) {
    *m = Mask{};
    if (!int32_of(kind, &m->kind)) return false;
    if (no(params)) return true;
    struct Number {
        const char *name;
        int32_t *to;
    };
    const Number numbers[] = {{"window_left", &m->params.window_left}, {"sink_tokens", &m->params.sink_tokens},
                              {"prefix_len", &m->params.prefix_len}};
    for (const Number &f : numbers) {
        PyObject *x = PyObject_GetAttrString(params, f.name);
        if (!x) {
            PyErr_Clear();
            return false;
        }
        const bool ok = int32_of(x, f.to);
        Py_DECREF(x);
        if (!ok) return false;
    }
    m->given = &m->params;
    return true;
}

// What prefill and kv_weigh have in common: queries, page table, lengths, offsets (or none).
struct Chunks {
    const at::Tensor *q, *table, *lens, *cu;
    int64_t stride, total, Hq, B;
    int32_t cols;
};

bool chunks(const Cache &c, PyObject *q, PyObject *table, PyObject *lens, PyObject *cu, Chunks *x) {
    x->cu = nullptr;
    if (!tensor(q, &x->q) || !tensor(table, &x->table) || !tensor(lens, &x->lens) || (!no(cu) && !tensor(cu, &x->cu))) return false;
    if (x->q->dim() != 3) return false;
    x->total = x->q->size(0), x->Hq = x->q->size(1);
    if (!rows(*x->q, x->Hq, c.c->D, c.device, &x->stride) || !small_dims(*x->q)) return false;
    if (!ints(*x->table, 2, c.device) || !ints(*x->lens, 1, c.device) || !small_dims(*x->table)) return false;
    x->B = x->table->size(0);
    if (x->lens->size(0) != x->B) return false;
    if (x->cu ? !ints(*x->cu, 1, c.device) || x->cu->size(0) != x->B + 1 : x->total != x->B) return false;
    x->cols = (int32_t)x->table->size(1);
    return true;
}

// The cache's weights: contiguous fp32 like a scale.
bool weights_of(const Cache &c, PyObject *o, float **w) {
    const at::Tensor *t;
    if (!tensor(o, &t) || t->dim() != 3 || t->scalar_type() != at::kFloat || !t->is_cuda() || t->get_device() != c.device ||
        !t->is_contiguous() || t->size(0) != c.c->num_pages || t->size(1) != c.c->H || t->size(2) != c.c->page_size)
        return false;
    *w = static_cast<float *>(t->data_ptr());
    return true;
}

// prefill(cache address, device, q, page_table, seqlens, cu_seqlens, keys, kind, mask_params | None, softmax_scale,
//         workspace) -> (out, lse)
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    Chunks x;
    Mask m;
    const at::Tensor *ws;
    if (n != 11 || !cache(a[0], a[1], &c)) return PyErr_Occurred() ? nullptr : none();
    if (!chunks(c, a[2], a[3], a[4], a[5], &x) || !x.cu || !PyLong_Check(a[6]) || !mask(a[7], a[8], &m) || !tensor(a[10], &ws)) return none();
    const int64_t keys = PyLong_AsLongLong(a[6]);
    const double scale = PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    if (!ws->is_cuda() || ws->get_device() != c.device || !ws->is_contiguous()) return none();
    const int64_t shape[3] = {x.total, x.Hq, c.c->D}, lse_shape[2] = {x.total, x.Hq};
    at::Tensor out = at::empty(shape, x.q->options()), lse = at::empty(lse_shape, x.q->options().dtype(at::kFloat));
    const bsattn_status st =
        g_prefill(x.q->data_ptr(), x.stride, (int32_t)x.total, (int32_t)x.B, (int32_t)x.Hq, int_ptr(*x.cu), c.c, int_ptr(*x.table),
                  x.cols, x.cols, int_ptr(*x.lens), keys, (bsattn_mask_kind)m.kind, m.given, (float)scale, out.data_ptr(),
                  BSATTN_OUT_BF16, static_cast<float *>(lse.data_ptr()), ws->data_ptr(), ws->nbytes(), nullptr, stream_of(c.device));
    if (st != BSATTN_OK) return PyLong_FromLong(st);
    return Py_BuildValue("NN", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
}

// kv_weigh(cache address, device, q, lse, weights, page_table, seqlens, cu_seqlens | None, accumulate, kind,
//          mask_params | None, softmax_scale)
PyObject *kv_weigh(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    Chunks x;
    Mask m;
    const at::Tensor *lse;
    float *w;
    if (n != 12 || !cache(a[0], a[1], &c)) return PyErr_Occurred() ? nullptr : none();
    if (!chunks(c, a[2], a[5], a[6], a[7], &x) || !tensor(a[3], &lse) || !weights_of(c, a[4], &w) || !mask(a[9], a[10], &m)) return none();
    if (lse->dim() != 2 || lse->scalar_type() != at::kFloat || !lse->is_cuda() || lse->get_device() != c.device ||
        !lse->is_contiguous() || lse->size(0) != x.total || lse->size(1) != x.Hq)
        return none();
    const int add = PyObject_IsTrue(a[8]);
    const double scale = PyFloat_AsDouble(a[11]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    const bsattn_status st =
        g_weigh(x.q->data_ptr(), x.stride, static_cast<const float *>(lse->data_ptr()), (int32_t)x.total, (int32_t)x.B, (int32_t)x.Hq,
                x.cu ? int_ptr(*x.cu) : nullptr, c.c, w, add, int_ptr(*x.table), x.cols, x.cols, int_ptr(*x.lens),
                (bsattn_mask_kind)m.kind, m.given, (float)scale, nullptr, stream_of(c.device));
    return PyLong_FromLong(st);
}

// kv_evict(cache address, device, weights, page_table, seqlens, keep, recent, sinks, out_table | None) -> (kept, lens)
PyObject *kv_evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    float *w;
    const at::Tensor *table, *lens, *out = nullptr;
    int32_t keep, recent, sinks;
    if (n != 9 || !cache(a[0], a[1], &c)) return PyErr_Occurred() ? nullptr : none();
    if (!weights_of(c, a[2], &w) || !tensor(a[3], &table) || !tensor(a[4], &lens) || (!no(a[8]) && !tensor(a[8], &out))) return none();
    if (!int32_of(a[5], &keep) || !int32_of(a[6], &recent) || !int32_of(a[7], &sinks)) return none();
    if (keep <= 0 || recent < 0 || sinks < 0 || (int64_t)recent + sinks > keep) return none();
    if (!ints(*table, 2, c.device) || !ints(*lens, 1, c.device) || !small_dims(*table)) return none();
    const int64_t B = table->size(0);
    if (lens->size(0) != B || (out && (!ints(*out, 2, c.device) || out->size(0) != B || !small_dims(*out)))) return none();
    const int64_t shape[3] = {B, c.c->H, keep}, lens_shape[1] = {B};
    at::Tensor kept = at::empty(shape, lens->options()), now = at::empty(lens_shape, lens->options());
    const int32_t cols = (int32_t)table->size(1), out_cols = out ? (int32_t)out->size(1) : 0;
    const bsattn_status st =
        g_evict(c.c, w, int_ptr(*table), cols, cols, int_ptr(*lens), (int32_t)B, keep, recent, sinks, out ? int_ptr(*out) : nullptr,
                out_cols, out_cols, static_cast<int32_t *>(kept.data_ptr()), static_cast<int32_t *>(now.data_ptr()), nullptr,
                stream_of(c.device));
    if (st != BSATTN_OK) return PyLong_FromLong(st);
    return Py_BuildValue("NN", THPVariable_Wrap(std::move(kept)), THPVariable_Wrap(std::move(now)));
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
PyMethodDef g_methods[] = {ENTRY(torch_version), ENTRY(bind), ENTRY(kv_append), ENTRY(kv_read), ENTRY(decode), ENTRY(prefill),
                           ENTRY(kv_weigh), ENTRY(kv_evict), {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
