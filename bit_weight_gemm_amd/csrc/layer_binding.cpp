// Python marshalling of the decoder-layer entry points: checks the tensors'
// types, shapes and strides and calls the C ABI with their addresses.  A
// CPython extension because a decode step makes these calls every few
// microseconds: an append of one token (40 heads) takes 5.2 us a call this way,
// 10.8 us with the same checks in Python and the call through ctypes.  No
// arithmetic, no allocation, no HIP call.
//
// The entry points' addresses come from the loaded library (bind), so the
// extension works with whichever build of it the package has loaded.
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

// The C ABI's types without HIP's headers.
using hipStream_t = void *;
using Status = int32_t;
using AppendFn = Status (*)(uint8_t *, uint8_t *, uint8_t *, uint8_t *, int32_t, int32_t, int32_t, int32_t,
                            const void *, int64_t, const void *, int64_t, const void *, int64_t, int32_t,
                            const int32_t *, int32_t, const uint8_t *, const float *, int32_t, int32_t, int32_t,
                            const int32_t *, const int32_t *, const int32_t *, int32_t, int32_t, int32_t, int32_t,
                            void *, int64_t, hipStream_t);
using AttnFn = Status (*)(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *, int32_t, int32_t,
                          int32_t, int32_t, const void *, int64_t, int32_t, const int32_t *, const int32_t *,
                          const int32_t *, int32_t, int32_t, int32_t, int32_t, int32_t, float, int32_t, int32_t,
                          void *, int64_t, float *, void *, size_t, hipStream_t);
using NormFn = Status (*)(const void *, int64_t, const void *, const void *, int64_t, float, const void *, int64_t,
                          int32_t, const void *, float, float, int32_t, int32_t, void *, int64_t, void *, int64_t,
                          uint8_t *, uint8_t *, hipStream_t);

namespace {

AppendFn g_append;
AttnFn g_attn;
NormFn g_norm;

using at::Tensor;

struct PythonError {};      // an exception is set already

[[noreturn]] void refuse(const char *what, const char *expected) {
    throw std::invalid_argument(std::string(what) + ": " + expected);
}

const Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) refuse(what, "a tensor expected");
    return THPVariable_Unpack(o);
}
const Tensor *maybe(PyObject *o, const char *what) { return o == Py_None ? nullptr : &tensor(o, what); }

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}
int32_t integer32(PyObject *o, const char *what) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) refuse(what, "a 32-bit number expected");
    return (int32_t)v;
}
int32_t size32(int64_t v, const char *what) {
    if (v > INT32_MAX) refuse(what, "fewer than 2^31 rows expected");
    return (int32_t)v;
}
int32_t truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v;
}
float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return (float)v;
}
hipStream_t stream(PyObject *o) {
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) throw PythonError();
    return (hipStream_t)(uintptr_t)v;
}

// The last check: every array that the kernels will touch is a GPU's, the same
// one's, and that GPU is the current one, which the kernels are launched on.
void on_one_gpu(PyObject *current, std::initializer_list<const Tensor *> all) {
    const Tensor *first = nullptr;
    for (const Tensor *t : all) {
        if (!t) continue;
        if (!first) first = t;
        if (!t->is_cuda() || t->get_device() != first->get_device())
            throw std::invalid_argument("tensors of one GPU expected");
    }
    if (first->get_device() != integer(current)) throw std::invalid_argument("tensors of the current GPU expected");
}

template <class... N>
bool shaped(const Tensor &t, N... n) {
    const auto s = t.sizes();
    if (s.size() != sizeof...(n)) return false;
    size_t i = 0;
    return ((s[i++] == (int64_t)n) && ...);
}

struct Cache {
    const Tensor *t[4];
    uint8_t *p[4];
    int32_t pages, heads, page, dim;
};
Cache cache(PyObject *o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse("cache", "a tuple of four tensors expected");
    Cache c;
    const Tensor **t = c.t;
    for (int i = 0; i < 4; ++i) {
        t[i] = &tensor(PyTuple_GET_ITEM(o, i), "cache");
        if (!t[i]->is_contiguous()) refuse("cache", "contiguous arrays expected");
        if (t[i]->scalar_type() != at::kByte) refuse("cache", "uint8 arrays expected");
        c.p[i] = (uint8_t *)t[i]->data_ptr();
    }
    const auto s = t[0]->sizes();
    if (s.size() != 4) refuse("cache", "k_codes [pages][kv_heads][page][dim] expected");
    if (!shaped(*t[1], s[0], s[1], s[2] / 8, s[3], 8) || !shaped(*t[2], s[0], s[1]) || !shaped(*t[3], s[0], s[1]))
        refuse("cache", "arrays of one cache expected");
    c.pages = size32(s[0], "cache");
    c.heads = size32(s[1], "cache");
    c.page = size32(s[2], "cache");
    c.dim = size32(s[3], "cache");
    return c;
}

// Token stride of a bf16 tensor [tokens][heads][dim] whose heads are contiguous.
int64_t token_stride(const Tensor &t, int64_t T, int64_t heads, int64_t dim, const char *what) {
    if (t.scalar_type() != at::kBFloat16 || !shaped(t, T, heads, dim) || t.stride(2) != 1 ||
        (t.stride(1) != dim && heads > 1))
        refuse(what, "bf16 [tokens][heads][dim] with contiguous heads expected");
    return T > 1 ? t.stride(0) : heads * dim;
}
int64_t row_stride(const Tensor &t, int64_t T, int64_t C, at::ScalarType type, const char *what) {
    if (t.scalar_type() != type || !shaped(t, T, C) || (t.stride(1) != 1 && C > 1))
        refuse(what, "[tokens][channels] of its type with contiguous rows expected");
    return T > 1 ? t.stride(0) : C;
}
template <class... N>
const int32_t *ints(const Tensor &t, const char *what, N... n) {
    if (t.scalar_type() != at::kInt || !shaped(t, n...) || !t.is_contiguous())
        refuse(what, "contiguous int32 of its shape expected");
    return (const int32_t *)t.data_ptr();
}
const void *vector(const Tensor *t, int64_t C, const char *what) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kBFloat16 || !shaped(*t, C) || !t->is_contiguous())
        refuse(what, "contiguous bf16 of the channels expected");
    return t->data_ptr();
}
uint8_t *bytes(const Tensor *t, int64_t T, int64_t n, const char *what) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kByte || !shaped(*t, T, n) || !t->is_contiguous())
        refuse(what, "contiguous uint8 of its shape expected");
    return (uint8_t *)t->data_ptr();
}

struct Ragged {
    const int32_t *start, *len, *table;
    int32_t max_pages, B;
};
Ragged ragged(PyObject *q_start, PyObject *kv_len, PyObject *block_table) {
    const Tensor &t = tensor(block_table, "block_table");
    if (t.dim() != 2) refuse("block_table", "[sequences][pages] expected");
    Ragged r;
    r.B = size32(t.size(0), "block_table");
    r.max_pages = size32(t.size(1), "block_table");
    r.table = ints(t, "block_table", t.size(0), t.size(1));
    r.start = ints(tensor(q_start, "q_start"), "q_start", r.B + 1);
    r.len = ints(tensor(kv_len, "kv_len"), "kv_len", r.B);
    return r;
}

Status append(PyObject *const *a) {
    const Cache c = cache(a[0]);
    const Tensor *q = maybe(a[1], "q"), *pos = maybe(a[4], "positions"), *cs = maybe(a[5], "cos_sin"),
                 *out = maybe(a[10], "q_out");
    const Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    if (k.dim() != 3) refuse("k", "[tokens][heads][dim] expected");
    const int64_t T = k.size(0);
    const Ragged r = ragged(a[6], a[7], a[8]);
    int32_t n_pos = 0, rot = 0, axes = 0, heads = 0;
    int64_t sq = 0, so = 0;
    const int32_t *positions = nullptr;
    if (cs) {
        if (cs->dim() != 2 || cs->scalar_type() != at::kFloat || !cs->is_contiguous())
            refuse("cos_sin", "contiguous fp32 [positions][rot_dim] expected");
        if (!pos || pos->dim() != 2) refuse("positions", "int32 [axes][tokens] expected");
        n_pos = size32(cs->size(0), "cos_sin");
        rot = size32(cs->size(1), "cos_sin");
        axes = size32(pos->size(0), "positions");
        positions = ints(*pos, "positions", axes, T);
    }
    const uint8_t *pair_axis = nullptr;
    if (a[11] != Py_None) {
        if (!PyBytes_Check(a[11]) || PyBytes_GET_SIZE(a[11]) != rot / 2)
            refuse("pair_axis", "bytes, one per pair, expected");
        pair_axis = (const uint8_t *)PyBytes_AS_STRING(a[11]);
    }
    if (q) {
        if (q->dim() != 3 || !out) refuse("q", "[tokens][heads][dim] and its output expected");
        heads = size32(q->size(1), "q");
        sq = token_stride(*q, T, heads, c.dim, "q");
        so = token_stride(*out, T, heads, c.dim, "q_out");
    }
    const int32_t interleaved = truth(a[12]);
    const int64_t sk = token_stride(k, T, c.heads, c.dim, "k"), sv = token_stride(v, T, c.heads, c.dim, "v");
    on_one_gpu(a[14], {c.t[0], c.t[1], c.t[2], c.t[3], q, &k, &v, pos, cs, out, &tensor(a[6], "q_start"),
                       &tensor(a[7], "kv_len"), &tensor(a[8], "block_table")});
    return g_append(c.p[0], c.p[1], c.p[2], c.p[3], c.pages, c.heads, c.page, c.dim, q ? q->data_ptr() : nullptr, sq,
                    k.data_ptr(), sk, v.data_ptr(), sv, heads, positions, axes, pair_axis,
                    cs ? (const float *)cs->data_ptr() : nullptr, n_pos, rot, interleaved, r.start, r.len,
                    r.table, r.max_pages, r.B, size32(T, "k"), integer32(a[9], "max_q_len"),
                    q ? out->data_ptr() : nullptr, so, stream(a[13]));
}

Status attn(PyObject *const *a) {
    const Cache c = cache(a[0]);
    const Tensor &q = tensor(a[1], "q"), &out = tensor(a[10], "out"), &ws = tensor(a[12], "workspace");
    if (q.dim() != 3) refuse("q", "[tokens][heads][dim] expected");
    const int64_t T = q.size(0);
    const int32_t heads = size32(q.size(1), "q");
    const Ragged r = ragged(a[2], a[3], a[4]);
    const Tensor *lse = maybe(a[11], "lse");
    if (lse && (lse->scalar_type() != at::kFloat || !shaped(*lse, T, heads) || !lse->is_contiguous()))
        refuse("lse", "contiguous fp32 [tokens][heads] expected");
    if (!ws.is_contiguous()) refuse("workspace", "contiguous memory expected");
    const int64_t sq = token_stride(q, T, heads, c.dim, "q"), so = token_stride(out, T, heads, c.dim, "out");
    on_one_gpu(a[14], {c.t[0], c.t[1], c.t[2], c.t[3], &q, &out, &ws, lse, &tensor(a[2], "q_start"),
                       &tensor(a[3], "kv_len"), &tensor(a[4], "block_table")});
    return g_attn(c.p[0], c.p[1], c.p[2], c.p[3], c.pages, c.heads, c.page, c.dim, q.data_ptr(), sq, heads, r.start,
                  r.len, r.table, r.max_pages, r.B, size32(T, "q"), integer32(a[5], "max_q_len"),
                  integer32(a[6], "max_kv_len"), number(a[7]), integer32(a[8], "window"), integer32(a[9], "sinks"),
                  out.data_ptr(), so, lse ? (float *)lse->data_ptr() : nullptr, ws.data_ptr(), ws.nbytes(),
                  stream(a[13]));
}

Status norm(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x"), &res = tensor(a[1], "res"), &pre = tensor(a[2], "pre_w"),
                 &res_out = tensor(a[8], "res_out"), &h = tensor(a[9], "h");
    const Tensor *post = maybe(a[3], "post_w"), *gate = maybe(a[4], "gate"), *codes = maybe(a[10], "a_codes"),
                 *scales = maybe(a[11], "a_scales");
    if (x.dim() != 2) refuse("x", "[tokens][channels] expected");
    const int64_t T = x.size(0), C = x.size(1);
    const auto kind = res.scalar_type();
    if (kind != at::kFloat && kind != at::kBFloat16) refuse("res", "bf16 or fp32 expected");
    int64_t gate_stride = 0;
    if (gate) {      // one row: of every token
        const bool one = gate->dim() == 2 && gate->size(0) == 1;
        gate_stride = row_stride(*gate, one ? 1 : T, C, at::kBFloat16, "gate");
        if (one) gate_stride = 0;
    }
    const int64_t sx = row_stride(x, T, C, at::kBFloat16, "x"), sr = row_stride(res, T, C, kind, "res"),
                  sro = row_stride(res_out, T, C, kind, "res_out"), sh = row_stride(h, T, C, at::kBFloat16, "h");
    const void *pw = vector(post, C, "post_w"), *w = vector(&pre, C, "pre_w");
    uint8_t *pc = bytes(codes, T, C / 2, "a_codes"), *ps = bytes(scales, T, C / 16, "a_scales");
    on_one_gpu(a[13], {&x, &res, &pre, post, gate, &res_out, &h, codes, scales});
    return g_norm(x.data_ptr(), sx, pw, gate ? gate->data_ptr() : nullptr, gate_stride, number(a[5]), res.data_ptr(),
                  sr, kind == at::kFloat, w, number(a[6]), number(a[7]), size32(T, "x"), size32(C, "x"),
                  res_out.data_ptr(), sro, h.data_ptr(), sh, pc, ps, stream(a[12]));
}

// Calls f with `want` positional arguments; returns the status.
template <Status (*F)(PyObject *const *), int WANT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != WANT) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected", WANT);
        return nullptr;
    }
    if (!g_append || !g_attn || !g_norm) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown exception");
    }
    return nullptr;
}

PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "three addresses expected");
        return nullptr;
    }
    void *p[3];
    for (int i = 0; i < 3; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_append = (AppendFn)p[0];
    g_attn = (AttnFn)p[1];
    g_norm = (NormFn)p[2];
    Py_RETURN_NONE;
}

#define FASTCALL(f) ((PyCFunction)(void (*)(void))(f))
PyMethodDef methods[] = {{"bind", FASTCALL(bind), METH_FASTCALL, "addresses of the three entry points"},
                         {"kv_append", FASTCALL((entry<append, 15>)), METH_FASTCALL, "biloco_kv_append"},
                         {"attn_paged", FASTCALL((entry<attn, 15>)), METH_FASTCALL, "biloco_attn_paged"},
                         {"norm_gate_residual", FASTCALL((entry<norm, 14>)), METH_FASTCALL, "biloco_norm_gate_residual"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding() { return PyModule_Create(&module); }
