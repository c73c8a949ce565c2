// The short way from Python into the token mixers' C entries: checks and marshals the arguments of a
// call whose tensors are all given, in C++, without ctypes (a single-token state update 10.5 -> 3.7 us
// a call, a cache write of 16 tokens 9.8 -> 3.7 us). Every function returns the entry's status, or -1
// where an argument is not what it takes; the caller then goes the long way (mixers.py), which
// allocates, switches devices, or raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w4a16.h"

namespace {

decltype(&w4a16_page_tables) g_page_tables;
decltype(&w4a16_paged_kv_write) g_kv_write;
decltype(&w4a16_paged_attention) g_attention;
decltype(&w4a16_linear_attention) g_linear;
decltype(&w4a16_linear_attention_step) g_step;

// What a call's tensors have to share, and whether one of them did not.
struct Call {
    bool ok = true;
    int device = -1;

    const at::Tensor *any(PyObject *o, int64_t dims)
    {
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || t.dim() != dims) {
            ok = false;
            return nullptr;
        }
        if (device < 0)
            device = t.get_device();
        ok = ok && t.get_device() == device;
        return ok ? &t : nullptr;
    }
    const at::Tensor *typed(PyObject *o, int64_t dims, at::ScalarType type)
    {
        const at::Tensor *t = any(o, dims);
        ok = ok && t->scalar_type() == type;
        return ok ? t : nullptr;
    }
    // Contiguous; None is allowed and gives null where `optional`.
    const at::Tensor *flat(PyObject *o, int64_t dims, at::ScalarType type, bool optional = false)
    {
        if (optional && o == Py_None)
            return nullptr;
        const at::Tensor *t = typed(o, dims, type);
        ok = ok && t->is_contiguous();
        return ok ? t : nullptr;
    }
    // bfloat16 or float16 [rows, heads, dim] with contiguous rows.
    const at::Tensor *rows(PyObject *o, int64_t *ld, int64_t *hs)
    {
        const at::Tensor *t = any(o, 3);
        ok = ok && (t->scalar_type() == at::kBFloat16 || t->scalar_type() == at::kHalf) &&
             (t->stride(2) == 1 || t->size(2) <= 1);
        if (!ok)
            return nullptr;
        *ld = t->size(0) > 1 ? t->stride(0) : 0;
        *hs = t->size(1) > 1 ? t->stride(1) : 0;
        return t;
    }
    void need(bool x) { ok = ok && x; }
    // The current device has to be the tensors'.
    bool ready() { return ok && device >= 0 && device == c10::hip::current_device(); }
    hipStream_t stream() const { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }
};

template <class T = void>
T *ptr(const at::Tensor *t)
{
    return t ? (T *)t->data_ptr() : nullptr;
}
int32_t type_of(const at::Tensor *t)
{
    return t->scalar_type() == at::kBFloat16 ? W4A16_BF16 : t->scalar_type() == at::kHalf ? W4A16_FP16 : W4A16_E4M3;
}
bool fits(int64_t x) { return x >= 0 && x <= INT32_MAX; }

bool read_int(PyObject *o, int64_t *x)
{
    if (!PyLong_CheckExact(o))
        return false;
    int over = 0;
    *x = PyLong_AsLongLongAndOverflow(o, &over);
    return !over && *x >= INT32_MIN && *x <= INT32_MAX;
}
bool read_float(PyObject *o, float *x)
{
    if (!PyFloat_CheckExact(o))
        return false;
    *x = (float)PyFloat_AS_DOUBLE(o);
    return true;
}

bool read_cache(Call &c, PyObject *const *a, at::ScalarType kind, w4a16_paged_cache_t *out)
{
    const at::Tensor *k = c.any(a[0], 4), *v = c.any(a[1], 4);
    if (!c.ok || k->scalar_type() != v->scalar_type() || k->sizes() != v->sizes() ||
        (k->scalar_type() != kind && k->scalar_type() != at::kFloat8_e4m3fn) || k->stride(3) != 1 ||
        v->stride(3) != 1)
        return c.ok = false;
    for (int i = 0; i < 4; ++i)
        if (!fits(k->size(i)))
            return c.ok = false;
    out->k = k->data_ptr();
    out->v = v->data_ptr();
    for (int i = 0; i < 3; ++i) {
        out->k_stride[i] = k->size(i) > 1 ? k->stride(i) : 0;
        out->v_stride[i] = v->size(i) > 1 ? v->stride(i) : 0;
    }
    const at::Tensor *ks = c.flat(a[2], 1, at::kFloat, true), *vs = c.flat(a[3], 1, at::kFloat, true);
    const bool e4m3 = k->scalar_type() == at::kFloat8_e4m3fn;
    c.need((!ks || (e4m3 && ks->size(0) == k->size(2))) && (!vs || (e4m3 && vs->size(0) == k->size(2))));
    out->k_scale = ptr<float>(ks);
    out->v_scale = ptr<float>(vs);
    out->num_pages = (int32_t)k->size(0);
    out->page_size = (int32_t)k->size(1);
    out->heads = (int32_t)k->size(2);
    out->dim = (int32_t)k->size(3);
    out->type = type_of(k);
    return c.ok;
}

PyObject *status(int s) { return PyLong_FromLong(s); }

// (ctx_lens, new_lens, page_table, free_pages, page_size, seq_lens, cu_new, slot_map, positions, counts)
PyObject *page_tables(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c;
    int64_t page = 0;
    if (n != 10 || !read_int(a[4], &page))
        return status(-1);
    const at::Tensor *ctx = c.flat(a[0], 1, at::kInt), *fresh = c.flat(a[1], 1, at::kInt);
    const at::Tensor *table = c.typed(a[2], 2, at::kInt), *free = c.flat(a[3], 1, at::kInt), *out[5];
    for (int i = 0; i < 5; ++i)
        out[i] = c.flat(a[5 + i], 1, at::kInt);
    if (!c.ready())
        return status(-1);
    const int64_t B = ctx->size(0), pages = table->size(1), T = out[2]->size(0);
    c.need(fresh->size(0) == B && table->size(0) == B && (pages <= 1 || table->stride(1) == 1));
    c.need(out[0]->size(0) == B && out[1]->size(0) == B + 1 && out[3]->size(0) == T && out[4]->size(0) == 2);
    c.need(fits(B) && fits(pages) && fits(free->size(0)) && fits(T));
    if (!c.ok)
        return status(-1);
    return status(g_page_tables(ptr<int32_t>(ctx), ptr<int32_t>(fresh), (int32_t)B, ptr<int32_t>(table),
                                B > 1 ? table->stride(0) : pages, (int32_t)pages, ptr<int32_t>(free),
                                (int32_t)free->size(0), (int32_t)page, (int32_t)T, ptr<int32_t>(out[0]),
                                ptr<int32_t>(out[1]), ptr<int32_t>(out[2]), ptr<int32_t>(out[3]),
                                ptr<int32_t>(out[4]), c.stream()));
}

// (k, v, k_cache, v_cache, k_scale, v_scale, slot_map)
PyObject *paged_kv_write(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 7)
        return status(-1);
    Call c;
    int64_t ldk = 0, hsk = 0, ldv = 0, hsv = 0;
    const at::Tensor *k = c.rows(a[0], &ldk, &hsk), *v = c.rows(a[1], &ldv, &hsv);
    const at::Tensor *slots = c.flat(a[6], 1, at::kInt);
    w4a16_paged_cache_t cache;
    if (!c.ok || k->scalar_type() != v->scalar_type() || !read_cache(c, a + 2, k->scalar_type(), &cache) || !c.ready())
        return status(-1);
    const int64_t T = slots->size(0);
    c.need(fits(T) && k->sizes() == v->sizes() && k->size(0) == T && k->size(1) == cache.heads && k->size(2) == cache.dim);
    if (!c.ok)
        return status(-1);
    return status(g_kv_write(ptr(k), ldk, hsk, ptr(v), ldv, hsv, (int32_t)T, type_of(k), ptr<int32_t>(slots), &cache,
                             c.stream()));
}

// (q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, scale, window, out, lse, workspace)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c;
    int64_t ldq = 0, hsq = 0, ldo = 0, hso = 0, window = 0;
    float scale = 0;
    if (n != 12 || !read_float(a[7], &scale) || !read_int(a[8], &window))
        return status(-1);
    const at::Tensor *q = c.rows(a[0], &ldq, &hsq), *table = c.typed(a[5], 2, at::kInt);
    const at::Tensor *lens = c.flat(a[6], 1, at::kInt), *out = c.rows(a[9], &ldo, &hso);
    const at::Tensor *lse = c.flat(a[10], 2, at::kFloat, true), *work = c.flat(a[11], 1, at::kByte);
    w4a16_paged_cache_t cache;
    if (!c.ok || !read_cache(c, a + 1, q->scalar_type(), &cache) || !c.ready())
        return status(-1);
    const int64_t B = q->size(0), Hq = q->size(1), pages = table->size(1);
    c.need(q->size(2) == cache.dim && out->scalar_type() == q->scalar_type() && out->sizes() == q->sizes());
    c.need(table->size(0) == B && lens->size(0) == B && (pages <= 1 || table->stride(1) == 1));
    c.need(!lse || (lse->size(0) == B && lse->size(1) == Hq));
    c.need(fits(B) && fits(Hq) && fits(pages));
    if (!c.ok)
        return status(-1);
    return status(g_attention(ptr(q), ldq, hsq, type_of(q), &cache, ptr<int32_t>(table), B > 1 ? table->stride(0) : pages,
                              (int32_t)pages, ptr<int32_t>(lens), (int32_t)B, (int32_t)Hq, scale, (int32_t)window,
                              ptr(out), ldo, hso, ptr<float>(lse), ptr(work), work->size(0), c.stream()));
}

// What both linear forms share.
struct Mixer {
    const at::Tensor *q, *k, *v, *g, *out;
    int64_t ldq, hsq, ldk, hsk, ldv, hsv, ldg, hsg, ldo, hso, T, Hk, H, Dk, Dv;
};

bool read_mixer(Call &c, PyObject *q, PyObject *k, PyObject *v, PyObject *g, PyObject *out, Mixer *m)
{
    m->q = c.rows(q, &m->ldq, &m->hsq);
    m->k = c.rows(k, &m->ldk, &m->hsk);
    m->v = c.rows(v, &m->ldv, &m->hsv);
    m->out = c.rows(out, &m->ldo, &m->hso);
    if (!c.ok || !THPVariable_Check(g))
        return c.ok = false;
    m->T = m->q->size(0);
    m->Hk = m->q->size(1);
    m->Dk = m->q->size(2);
    m->H = m->v->size(1);
    m->Dv = m->v->size(2);
    const bool each = THPVariable_Unpack(g).dim() == 2;
    m->g = c.typed(g, each ? 2 : 1, at::kFloat);
    c.need(c.ok && m->q->scalar_type() == m->k->scalar_type() && m->q->scalar_type() == m->v->scalar_type() &&
           m->q->scalar_type() == m->out->scalar_type() && m->q->sizes() == m->k->sizes() && m->v->size(0) == m->T &&
           m->v->sizes() == m->out->sizes());
    c.need(c.ok && (each ? m->g->size(0) == m->T && m->g->size(1) == m->H : m->g->size(0) == m->H));
    c.need(fits(m->T) && fits(m->Hk) && fits(m->H) && fits(m->Dk) && fits(m->Dv));
    if (!c.ok)
        return false;
    m->ldg = each ? m->g->stride(0) : 0;
    m->hsg = m->g->stride(each ? 1 : 0);
    return true;
}

const at::Tensor *states(Call &c, PyObject *o, const Mixer &m, bool optional)
{
    const at::Tensor *t = c.flat(o, 4, at::kFloat, optional);
    c.need(!t || (t->size(1) == m.H && t->size(2) == m.Dk && t->size(3) == m.Dv));
    return t;
}

// (q, k, v, log_decay, cu_seqlens, state, state_out, scale, out, workspace)
PyObject *linear_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c;
    Mixer m;
    float scale = 0;
    if (n != 10 || !read_float(a[7], &scale) || !read_mixer(c, a[0], a[1], a[2], a[3], a[8], &m))
        return status(-1);
    const at::Tensor *cu = c.flat(a[4], 1, at::kInt, true), *s0 = states(c, a[5], m, true);
    const at::Tensor *s1 = states(c, a[6], m, false), *work = c.flat(a[9], 1, at::kByte);
    if (!c.ready())
        return status(-1);
    const int64_t seqs = cu ? cu->size(0) - 1 : 1;
    c.need(fits(seqs) && s1->size(0) == seqs && (!s0 || s0->size(0) == seqs));
    if (!c.ok)
        return status(-1);
    return status(g_linear(ptr(m.q), m.ldq, m.hsq, ptr(m.k), m.ldk, m.hsk, ptr(m.v), m.ldv, m.hsv, ptr<float>(m.g),
                           m.ldg, m.hsg, ptr<int32_t>(cu), (int32_t)seqs, (int32_t)m.T, (int32_t)m.Hk, (int32_t)m.H,
                           (int32_t)m.Dk, (int32_t)m.Dv, type_of(m.q), scale, ptr<float>(s0), ptr<float>(s1),
                           ptr(m.out), m.ldo, m.hso, ptr(work), work->size(0), c.stream()));
}

// (q, k, v, log_decay, state, slots, state_out, scale, out)
PyObject *linear_attention_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c;
    Mixer m;
    float scale = 0;
    if (n != 9 || !read_float(a[7], &scale) || !read_mixer(c, a[0], a[1], a[2], a[3], a[8], &m))
        return status(-1);
    const at::Tensor *s0 = states(c, a[4], m, false), *slots = c.flat(a[5], 1, at::kInt, true);
    const at::Tensor *s1 = states(c, a[6], m, false);
    if (!c.ready())
        return status(-1);
    c.need(fits(s0->size(0)) && s1->size(0) == s0->size(0) && (!slots || slots->size(0) == m.T));
    if (!c.ok)
        return status(-1);
    return status(g_step(ptr(m.q), m.ldq, m.hsq, ptr(m.k), m.ldk, m.hsk, ptr(m.v), m.ldv, m.hsv, ptr<float>(m.g), m.ldg,
                         m.hsg, ptr<int32_t>(slots), (int32_t)s0->size(0), (int32_t)m.T, (int32_t)m.Hk, (int32_t)m.H,
                         (int32_t)m.Dk, (int32_t)m.Dv, type_of(m.q), scale, ptr<float>(s0), ptr<float>(s1), ptr(m.out),
                         m.ldo, m.hso, c.stream()));
}

// No C++ exception may leave a function that Python calls.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    try {
        return F(self, a, n);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Addresses of the five C entries, in the order of their declarations.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses are wanted");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    g_page_tables = (decltype(g_page_tables))p[0];
    g_kv_write = (decltype(g_kv_write))p[1];
    g_attention = (decltype(g_attention))p[2];
    g_linear = (decltype(g_linear))p[3];
    g_step = (decltype(g_step))p[4];
    Py_RETURN_NONE;
}

#define ENTRY(name) {#name, (PyCFunction)(void (*)(void))guarded<name>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ENTRY(page_tables),      ENTRY(paged_kv_write),
                          ENTRY(paged_attention),  ENTRY(linear_attention),
                          ENTRY(linear_attention_step), ENTRY(bind),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
