/* The common calls of the windowed, grouped-head, 4-bit and norm entry points, marshalled
 * in C++: outputs and workspace from torch's allocator, the current stream, no buffer of the
 * caller's.  A single-token call is over on the GPU in a few microseconds; the same steps in
 * Python take 22 us of host time for the decode of one sequence, here 8.
 *
 * Every function takes the positional arguments that the Python function of its name
 * passes on, checks all that that function checks, and returns its result, or None when
 * anything is out of the ordinary: the Python function then goes through its own checks
 * and raises what is to be raised.  No computation, and nothing kept between calls but
 * the library's addresses. */
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>

#include "blockattn.h"

namespace {

struct {
    decltype(&::attn_window_fwd) attn_window_fwd;
    decltype(&::attn_window_fwd_workspace_size) attn_window_fwd_workspace_size;
    decltype(&::attn_window_bwd) attn_window_bwd;
    decltype(&::attn_window_bwd_workspace_size) attn_window_bwd_workspace_size;
    decltype(&::attn_window_decode_fwd) attn_window_decode_fwd;
    decltype(&::attn_window_decode_workspace_size) attn_window_decode_workspace_size;
    decltype(&::kv4_append) kv4_append;
    decltype(&::kv4_read) kv4_read;
    decltype(&::attn_decode_kv4_fwd) attn_decode_kv4_fwd;
    decltype(&::attn_decode_kv4_workspace_size) attn_decode_kv4_workspace_size;
    decltype(&::qk_norm_rope_fwd) qk_norm_rope_fwd;
    decltype(&::qk_norm_rope_bwd) qk_norm_rope_bwd;
    decltype(&::qk_norm_rope_bwd_workspace_size) qk_norm_rope_bwd_workspace_size;
} L;

PyObject *s_shape, *s_dev, *s_c;   // attributes of a KV4Cache

// A plain tensor of up to four axes.  code: BA_F32, BA_BF16, 2 for uint8, 3 for int32.
struct Ten {
    int n, code;
    long dev;
    long long size[4], step[4];
    void *ptr;
};

bool read_tensor(PyObject *x, Ten *t) {
    if (!THPVariable_CheckExact(x)) return false;
    const at::Tensor &v = THPVariable_Unpack(x);
    if (!v.is_cuda() || v.layout() != at::kStrided || v.is_neg() || v.dim() > 4) return false;
    switch (v.scalar_type()) {
        case at::kFloat: t->code = BA_F32; break;
        case at::kBFloat16: t->code = BA_BF16; break;
        case at::kByte: t->code = 2; break;
        case at::kInt: t->code = 3; break;
        default: return false;
    }
    t->n = (int)v.dim();
    const auto size = v.sizes(), step = v.strides();
    for (int i = 0; i < t->n; ++i) {
        t->size[i] = size[i];
        t->step[i] = step[i];
    }
    t->dev = v.get_device();
    t->ptr = v.data_ptr();
    return true;
}

ba_tensor view(const Ten *t) {
    const ba_tensor v = {t->ptr, t->step[0], t->step[1], t->step[2]};
    return v;
}

int heads(const Ten *t) { return t->n == 4 && t->code <= BA_BF16 && (t->step[3] == 1 || t->size[3] <= 1); }
int fits(const Ten *t) {   /* sizes that the entry points take as int */
    for (int i = 0; i < t->n; ++i)
        if (t->size[i] > 0x7fffffffLL) return 0;
    return 1;
}
int same(const Ten *a, const Ten *b) {   /* shape, dtype and device */
    if (a->n != b->n || a->code != b->code || a->dev != b->dev) return 0;
    for (int i = 0; i < a->n; ++i)
        if (a->size[i] != b->size[i]) return 0;
    return 1;
}
/* k, v (B, Hkv, L, d) beside q (B, Hq, .., d). */
int grouped(const Ten *q, const Ten *k, const Ten *v) {
    return heads(q) && heads(k) && heads(v) && same(k, v) && k->code == q->code && k->dev == q->dev &&
           k->size[0] == q->size[0] && k->size[3] == q->size[3] && k->size[1] > 0 && q->size[1] % k->size[1] == 0 && fits(q) &&
           fits(k);
}

int whole(PyObject *o, long long lo, int *to) {
    if (!PyLong_CheckExact(o)) return 0;
    const long long v = PyLong_AsLongLong(o);
    if ((v == -1 && PyErr_Occurred()) || v < lo || v > 0x7fffffffLL) return 0;
    *to = (int)v;
    return 1;
}
int real(PyObject *o, float *to) {   /* None: 0 */
    if (o == Py_None) {
        *to = 0.f;
        return 1;
    }
    if (!PyFloat_CheckExact(o)) return 0;
    *to = (float)PyFloat_AS_DOUBLE(o);
    return 1;
}

/* An int32 entry for each of B sequences, or None. */
int per_sequence(PyObject *o, long long B, long dev, const int32_t **to) {
    Ten t;
    *to = nullptr;
    if (o == Py_None) return 1;
    if (!read_tensor(o, &t) || t.code != 3 || t.n != 1 || t.size[0] != B || (B > 1 && t.step[0] != 1) || t.dev != dev) return 0;
    *to = (const int32_t *)t.ptr;
    return 1;
}

/* A key-padding mask of at least B rows and `keys` columns, or None. */
int padding(PyObject *o, long long B, long long keys, long dev, const uint8_t **to, int64_t *ld) {
    Ten t;
    *to = nullptr;
    *ld = 0;
    if (o == Py_None) return 1;
    if (!read_tensor(o, &t) || t.code != 2 || t.n != 2 || t.dev != dev || t.size[0] < B || t.size[1] < keys || t.step[1] != 1 ||
        (t.size[0] > 1 && t.step[0] < keys))
        return 0;
    *to = (const uint8_t *)t.ptr;
    *ld = t.step[0];
    return 1;
}

/* dev is the current device: its current stream. */
int stream_of(long dev, ba_stream_t *to) {
    if (c10::cuda::current_device() != dev) return 0;
    *to = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    return 1;
}

/* A new contiguous tensor and its pointer. */
at::Tensor empty(int n, const long long *size, int code, long dev, void **ptr) {
    int64_t z[4];
    for (int i = 0; i < n; ++i) z[i] = size[i];
    const at::ScalarType type = code == BA_BF16 ? at::kBFloat16 : code == BA_F32 ? at::kFloat : at::kByte;
    at::Tensor t = at::detail::empty_cuda(at::IntArrayRef(z, n), type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
    *ptr = t.data_ptr();
    return t;
}
at::Tensor scratch(size_t need, long dev, void **ptr) {
    const long long n = (long long)need;
    *ptr = nullptr;
    return need ? empty(1, &n, 2, dev, ptr) : at::Tensor();
}

PyObject *other_way(void) {
    PyErr_Clear();
    Py_RETURN_NONE;
}
/* n results as a tuple when the call went well; otherwise None (the Python function calls
 * again and raises). */
PyObject *results(int rc, int n, at::Tensor *r) {
    PyObject *t = rc == BA_OK ? PyTuple_New(n) : nullptr;
    for (int i = 0; t && i < n; ++i) {
        PyObject *x = THPVariable_Wrap(std::move(r[i]));
        if (!x) {
            Py_CLEAR(t);
            break;
        }
        PyTuple_SET_ITEM(t, i, x);
    }
    return t ? t : other_way();
}

/* (q, k, v, window, sinks, q_off, key_padding_mask, scale) -> (out, lse) */
PyObject *window_fwd(PyObject *const *a, Py_ssize_t na) {
    Ten q, k, v;
    int window, sinks, off;
    const uint8_t *kpm;
    int64_t ld;
    float scale;
    ba_stream_t st;
    if (na != 8 || !read_tensor(a[0], &q) || !read_tensor(a[1], &k) || !read_tensor(a[2], &v) || !grouped(&q, &k, &v) ||
        !whole(a[3], 1, &window) || !whole(a[4], 0, &sinks) || !whole(a[5], 0, &off) ||
        !padding(a[6], q.size[0], k.size[2], q.dev, &kpm, &ld) || !real(a[7], &scale) || !stream_of(q.dev, &st))
        return other_way();
    const int B = (int)q.size[0], Hq = (int)q.size[1], Lq = (int)q.size[2], d = (int)q.size[3];
    void *po, *pl, *pw;
    at::Tensor r[2], ws;
    r[0] = empty(4, q.size, q.code, q.dev, &po);
    r[1] = empty(3, q.size, BA_F32, q.dev, &pl);
    int rc;
    const size_t need = L.attn_window_fwd_workspace_size(B, Hq, Lq, d, q.code);
    ws = scratch(need, q.dev, &pw);
    {
        Py_BEGIN_ALLOW_THREADS
        rc = L.attn_window_fwd(view(&q), view(&k), view(&v), B, Hq, (int)k.size[1], Lq, (int)k.size[2], d, q.code, off, window,
                               sinks, kpm, ld, scale, po, q.code, (float *)pl, pw, need, st);
        Py_END_ALLOW_THREADS
    }
    return results(rc, 2, r);
}

/* (q, k, v, out, dout, lse, window, sinks, q_off, key_padding_mask, scale) -> (dq, dk, dv) */
PyObject *window_bwd(PyObject *const *a, Py_ssize_t na) {
    Ten q, k, v, o, g, l;
    int window, sinks, off;
    const uint8_t *kpm;
    int64_t ld;
    float scale;
    ba_stream_t st;
    if (na != 11 || !read_tensor(a[0], &q) || !read_tensor(a[1], &k) || !read_tensor(a[2], &v) || !grouped(&q, &k, &v) ||
        !read_tensor(a[3], &o) || !read_tensor(a[4], &g) || !same(&o, &q) || !same(&g, &q) || !heads(&o) || !heads(&g) ||
        !read_tensor(a[5], &l) || l.code != BA_F32 || l.dev != q.dev || l.n != 3 || l.size[0] != q.size[0] ||
        l.size[1] != q.size[1] || l.size[2] != q.size[2] || l.step[2] != 1 || l.step[1] != l.size[2] ||
        l.step[0] != l.size[1] * l.size[2] || !whole(a[6], 1, &window) || !whole(a[7], 0, &sinks) || !whole(a[8], 0, &off) ||
        !padding(a[9], q.size[0], k.size[2], q.dev, &kpm, &ld) || !real(a[10], &scale) || !stream_of(q.dev, &st))
        return other_way();
    const int B = (int)q.size[0], Hq = (int)q.size[1], Hkv = (int)k.size[1], Lq = (int)q.size[2], Lk = (int)k.size[2],
              d = (int)q.size[3];
    void *p[3], *pw;
    at::Tensor r[3], ws;
    r[0] = empty(4, q.size, q.code, q.dev, &p[0]);
    r[1] = empty(4, k.size, q.code, q.dev, &p[1]);
    r[2] = empty(4, k.size, q.code, q.dev, &p[2]);
    int rc;
    const size_t need = L.attn_window_bwd_workspace_size(B, Hq, Hkv, Lq, Lk, d, off, window, sinks);
    ws = scratch(need, q.dev, &pw);
    {
        Py_BEGIN_ALLOW_THREADS
        rc = L.attn_window_bwd(view(&q), view(&k), view(&v), view(&o), view(&g), (const float *)l.ptr, B, Hq, Hkv, Lq, Lk, d,
                               q.code, off, window, sinks, kpm, ld, scale, p[0], p[1], p[2], q.code, pw, need, st);
        Py_END_ALLOW_THREADS
    }
    return results(rc, 3, r);
}

/* (q, k_cache, v_cache, window, sinks, lengths, scale) -> (out, lse) */
PyObject *window_decode(PyObject *const *a, Py_ssize_t na) {
    Ten q, k, v;
    int window, sinks;
    const int32_t *len;
    float scale;
    ba_stream_t st;
    if (na != 7 || !read_tensor(a[0], &q) || !read_tensor(a[1], &k) || !read_tensor(a[2], &v) || !grouped(&q, &k, &v) ||
        q.size[2] != 1 || !whole(a[3], 1, &window) || !whole(a[4], 0, &sinks) || !per_sequence(a[5], q.size[0], q.dev, &len) ||
        !real(a[6], &scale) || !stream_of(q.dev, &st))
        return other_way();
    const int B = (int)q.size[0], Hq = (int)q.size[1], Hkv = (int)k.size[1], S = (int)k.size[2], d = (int)q.size[3];
    void *po, *pl, *pw;
    at::Tensor r[2], ws;
    r[0] = empty(4, q.size, q.code, q.dev, &po);
    r[1] = empty(3, q.size, BA_F32, q.dev, &pl);
    int rc;
    const size_t need = L.attn_window_decode_workspace_size(B, Hq, Hkv, S, d, window, sinks);
    ws = scratch(need, q.dev, &pw);
    {
        Py_BEGIN_ALLOW_THREADS
        rc = L.attn_window_decode_fwd(view(&q), view(&k), view(&v), B, Hq, Hkv, S, d, q.code, len, window, sinks, scale, po,
                                      q.code, (float *)pl, pw, need, st);
        Py_END_ALLOW_THREADS
    }
    return results(rc, 2, r);
}

int ints(PyObject *t, long long *to) {
    if (!t || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) > 4) return -1;
    const int n = (int)PyTuple_GET_SIZE(t);
    for (int i = 0; i < n; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (to[i] == -1 && PyErr_Occurred()) return -1;
    }
    return n;
}

/* A KV4Cache: its sizes (B, H, S, d), layout and device. */
int read_cache(PyObject *x, long long *size, ba_kv4 *c, long *dev) {
    PyObject *o = PyObject_GetAttr(x, s_shape);
    const int n = ints(o, size);
    Py_XDECREF(o);
    if (n != 4 || !(o = PyObject_GetAttr(x, s_c))) return 0;
    Py_buffer b;
    const int got = PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) == 0;
    Py_DECREF(o);
    if (!got) return 0;
    const int ok = b.len == (Py_ssize_t)sizeof *c;
    if (ok) memcpy(c, b.buf, sizeof *c);
    PyBuffer_Release(&b);
    if (!ok || !(o = PyObject_GetAttr(x, s_dev))) return 0;
    *dev = PyLong_AsLong(o);
    Py_DECREF(o);
    for (int i = 0; i < 4; ++i)
        if (size[i] > 0x7fffffffLL) return 0;
    return !PyErr_Occurred();
}

/* (cache, k, v, start, counts) -> cache */
PyObject *append(PyObject *const *a, Py_ssize_t na) {
    Ten k, v;
    long long z[4];
    ba_kv4 c;
    long dev;
    const int32_t *start, *counts;
    ba_stream_t st;
    if (na != 5 || !read_cache(a[0], z, &c, &dev) || !read_tensor(a[1], &k) || !read_tensor(a[2], &v) || !heads(&k) ||
        !heads(&v) || !same(&k, &v) || !fits(&k) || k.dev != dev || k.size[0] != z[0] || k.size[1] != z[1] || k.size[3] != z[3] ||
        !per_sequence(a[3], z[0], dev, &start) || !per_sequence(a[4], z[0], dev, &counts) || !stream_of(dev, &st))
        return other_way();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = L.kv4_append(view(&k), view(&v), c, (int)z[0], (int)z[1], (int)k.size[2], (int)z[2], (int)z[3], k.code, start, counts, st);
    Py_END_ALLOW_THREADS
    if (rc != BA_OK) return other_way();
    Py_INCREF(a[0]);
    return a[0];
}

/* (cache, T, first, dtype) -> (k, v) */
PyObject *read_back(PyObject *const *a, Py_ssize_t na) {
    long long z[4];
    ba_kv4 c;
    long dev;
    int T, first;
    ba_stream_t st;
    if (na != 4 || !read_cache(a[0], z, &c, &dev) || !whole(a[1], 0, &T) || !whole(a[2], 0, &first) ||
        !THPDtype_Check(a[3]) || !stream_of(dev, &st))
        return other_way();
    const at::ScalarType type = reinterpret_cast<THPDtype *>(a[3])->scalar_type;
    if (type != at::kBFloat16 && type != at::kFloat) return other_way();
    const int code = type == at::kBFloat16 ? BA_BF16 : BA_F32;
    const int S = (int)z[2];
    z[2] = T;
    void *p[2];
    at::Tensor r[2];
    r[0] = empty(4, z, code, dev, &p[0]);
    r[1] = empty(4, z, code, dev, &p[1]);
    int rc;
    {
        Py_BEGIN_ALLOW_THREADS
        rc = L.kv4_read(c, (int)z[0], (int)z[1], S, (int)z[3], first, T, code, p[0], p[1], st);
        Py_END_ALLOW_THREADS
    }
    return results(rc, 2, r);
}

/* (q, cache, lengths, window, sinks, scale) -> (out, lse) */
PyObject *decode_kv4(PyObject *const *a, Py_ssize_t na) {
    Ten q;
    long long z[4];
    ba_kv4 c;
    long dev;
    int window, sinks;
    const int32_t *len;
    float scale;
    ba_stream_t st;
    if (na != 6 || !read_tensor(a[0], &q) || !heads(&q) || !fits(&q) || !read_cache(a[1], z, &c, &dev) || q.dev != dev ||
        q.size[0] != z[0] || q.size[2] != 1 || q.size[3] != z[3] || z[1] < 1 || q.size[1] % z[1] ||
        !per_sequence(a[2], z[0], dev, &len) || !whole(a[3], 0, &window) || !whole(a[4], 0, &sinks) || !real(a[5], &scale) ||
        !stream_of(dev, &st))
        return other_way();
    const int B = (int)z[0], Hq = (int)q.size[1], Hkv = (int)z[1], S = (int)z[2], d = (int)z[3];
    void *po, *pl, *pw;
    at::Tensor r[2], ws;
    r[0] = empty(4, q.size, q.code, dev, &po);
    r[1] = empty(3, q.size, BA_F32, dev, &pl);
    int rc;
    const size_t need = L.attn_decode_kv4_workspace_size(B, Hq, Hkv, S, d, window, sinks);
    ws = scratch(need, dev, &pw);
    {
        Py_BEGIN_ALLOW_THREADS
        rc = L.attn_decode_kv4_fwd(view(&q), c, B, Hq, Hkv, S, d, q.code, len, window, sinks, scale, po, q.code, (float *)pl, pw,
                                   need, st);
        Py_END_ALLOW_THREADS
    }
    return results(rc, 2, r);
}

/* What the norm's two directions share: q, k, wq, wk, eps, positions, base, pos_scale. */
typedef struct {
    Ten q, k, wq, wk;
    float eps, base, scale;
    const int32_t *pos;
    int64_t ld;
    ba_stream_t st;
} Norm;

int read_norm(PyObject *const *a, Norm *n) {
    if (!read_tensor(a[0], &n->q) || !read_tensor(a[1], &n->k) || !heads(&n->q) || !heads(&n->k) || !fits(&n->q) || !fits(&n->k))
        return 0;
    const Ten *q = &n->q, *k = &n->k;
    if (k->code != q->code || k->dev != q->dev || k->size[0] != q->size[0] || k->size[2] != q->size[2] || k->size[3] != q->size[3])
        return 0;
    Ten *w[2] = {&n->wq, &n->wk};
    for (int i = 0; i < 2; ++i)
        if (!read_tensor(a[2 + i], w[i]) || w[i]->n != 1 || w[i]->size[0] != q->size[3] || (w[i]->size[0] > 1 && w[i]->step[0] != 1) ||
            (w[i]->code != q->code && w[i]->code != BA_F32) || w[i]->dev != q->dev)
            return 0;
    if (n->wq.code != n->wk.code || !PyFloat_CheckExact(a[4]) || !PyFloat_CheckExact(a[6]) || !PyFloat_CheckExact(a[7])) return 0;
    n->eps = (float)PyFloat_AS_DOUBLE(a[4]);
    n->base = (float)PyFloat_AS_DOUBLE(a[6]);
    n->scale = (float)PyFloat_AS_DOUBLE(a[7]);
    n->pos = nullptr;
    n->ld = 0;
    if (a[5] != Py_None) {
        Ten p;
        const long long B = q->size[0], T = q->size[2];
        if (!read_tensor(a[5], &p) || p.code != 3 || p.dev != q->dev || p.n < 1 || p.n > 2 || p.size[p.n - 1] != T ||
            (T > 1 && p.step[p.n - 1] != 1) || (p.n == 2 && p.size[0] != B && p.size[0] != 1))
            return 0;
        if (p.n == 2 && p.size[0] == B && B > 1 && p.step[0] != 0) {
            if (p.step[0] < T) return 0;
            n->ld = p.step[0];
        }
        n->pos = (const int32_t *)p.ptr;
    }
    return stream_of(q->dev, &n->st);
}

/* (q, k, wq, wk, eps, positions, base, pos_scale) -> (yq, yk) */
PyObject *norm_fwd(PyObject *const *a, Py_ssize_t na) {
    Norm n;
    if (na != 8 || !read_norm(a, &n)) return other_way();
    void *p[2];
    at::Tensor r[2];
    r[0] = empty(4, n.q.size, n.q.code, n.q.dev, &p[0]);
    r[1] = empty(4, n.k.size, n.q.code, n.q.dev, &p[1]);
    int rc;
    {
        Py_BEGIN_ALLOW_THREADS
        rc = L.qk_norm_rope_fwd(view(&n.q), view(&n.k), n.wq.ptr, n.wk.ptr, n.wq.code, (int)n.q.size[0], (int)n.q.size[1],
                                (int)n.k.size[1], (int)n.q.size[2], (int)n.q.size[3], n.q.code, n.eps, n.pos, n.ld, n.base,
                                n.scale, p[0], p[1], n.st);
        Py_END_ALLOW_THREADS
    }
    return results(rc, 2, r);
}

/* (q, k, wq, wk, eps, positions, base, pos_scale, dyq, dyk) -> (dq, dk, dwq, dwk) */
PyObject *norm_bwd(PyObject *const *a, Py_ssize_t na) {
    Norm n;
    Ten gq, gk;
    if (na != 10 || !read_norm(a, &n) || !read_tensor(a[8], &gq) || !read_tensor(a[9], &gk) || !heads(&gq) || !heads(&gk) ||
        gq.code != gk.code || (gq.code != n.q.code && gq.code != BA_F32) || gq.dev != n.q.dev || gk.dev != n.q.dev)
        return other_way();
    for (int i = 0; i < 4; ++i)
        if (gq.size[i] != n.q.size[i] || gk.size[i] != n.k.size[i]) return other_way();
    const int B = (int)n.q.size[0], Hq = (int)n.q.size[1], Hkv = (int)n.k.size[1], T = (int)n.q.size[2], d = (int)n.q.size[3];
    const long long row = d;
    void *p[4], *pw;
    at::Tensor r[4], ws;
    r[0] = empty(4, n.q.size, n.q.code, n.q.dev, &p[0]);
    r[1] = empty(4, n.k.size, n.q.code, n.q.dev, &p[1]);
    r[2] = empty(1, &row, BA_F32, n.q.dev, &p[2]);
    r[3] = empty(1, &row, BA_F32, n.q.dev, &p[3]);
    int rc;
    const size_t need = L.qk_norm_rope_bwd_workspace_size(B, Hq, Hkv, T, d, n.q.code);
    ws = scratch(need, n.q.dev, &pw);
    {
        Py_BEGIN_ALLOW_THREADS
        rc = L.qk_norm_rope_bwd(view(&n.q), view(&n.k), n.wq.ptr, n.wk.ptr, n.wq.code, view(&gq), view(&gk), gq.code, B, Hq, Hkv,
                                T, d, n.q.code, n.eps, n.pos, n.ld, n.base, n.scale, p[0], p[1], (float *)p[2], (float *)p[3], pw,
                                need, n.st);
        Py_END_ALLOW_THREADS
    }
    return results(rc, 4, r);
}

/* bind({entry point: address}) */
PyObject *bind(PyObject *, PyObject *d) {
    if (!PyDict_Check(d)) return PyErr_Format(PyExc_TypeError, "expected a dict of addresses");
#define ADDRESS(name)                                                                                                    \
    do {                                                                                                                 \
        PyObject *x = PyDict_GetItemString(d, #name);                                                                    \
        if (!x) return PyErr_Format(PyExc_KeyError, "%s", #name);                                                        \
        L.name = reinterpret_cast<decltype(L.name)>(PyLong_AsVoidPtr(x));                                                \
        if (PyErr_Occurred()) return nullptr;                                                                            \
    } while (0)
    ADDRESS(attn_window_fwd);
    ADDRESS(attn_window_fwd_workspace_size);
    ADDRESS(attn_window_bwd);
    ADDRESS(attn_window_bwd_workspace_size);
    ADDRESS(attn_window_decode_fwd);
    ADDRESS(attn_window_decode_workspace_size);
    ADDRESS(kv4_append);
    ADDRESS(kv4_read);
    ADDRESS(attn_decode_kv4_fwd);
    ADDRESS(attn_decode_kv4_workspace_size);
    ADDRESS(qk_norm_rope_fwd);
    ADDRESS(qk_norm_rope_bwd);
    ADDRESS(qk_norm_rope_bwd_workspace_size);
    Py_RETURN_NONE;
}

// No exception passes into the interpreter (torch throws when memory runs out; the Python
// function meets the same and raises it).
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *call(PyObject *, PyObject *const *a, Py_ssize_t na) {
    try {
        return F(a, na);
    } catch (...) {
        return other_way();
    }
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(call<f>)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"attn_window_fwd", FAST(window_fwd)},
                         {"attn_window_bwd", FAST(window_bwd)},
                         {"attn_window_decode_fwd", FAST(window_decode)},
                         {"kv4_append", FAST(append)},
                         {"kv4_read", FAST(read_back)},
                         {"attn_decode_kv4_fwd", FAST(decode_kv4)},
                         {"qk_norm_rope_fwd", FAST(norm_fwd)},
                         {"qk_norm_rope_bwd", FAST(norm_bwd)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void) {
    s_shape = PyUnicode_InternFromString("shape");
    s_dev = PyUnicode_InternFromString("dev");
    s_c = PyUnicode_InternFromString("_c");
    if (!s_shape || !s_dev || !s_c) return nullptr;
    return PyModule_Create(&module);
}
