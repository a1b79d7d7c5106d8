// Python marshalling of the decoder-layer entry points and of those for several
// answers to one prompt: checks the tensors'
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
using QuantMxFn = Status (*)(const void *, int64_t, int32_t, int32_t, int32_t, uint8_t *, uint8_t *, hipStream_t);
using DequantMxFn = Status (*)(const uint8_t *, const uint8_t *, int32_t, int32_t, void *, int64_t, int32_t, hipStream_t);
using GemmMxFn = Status (*)(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *, int32_t, int32_t, int32_t,
                            void *, int64_t, int32_t, void *, size_t, hipStream_t);
using GemmMxQuantFn = Status (*)(const void *, int64_t, const uint8_t *, const uint8_t *, int32_t, int32_t, int32_t,
                                 void *, int64_t, int32_t, void *, size_t, hipStream_t);
using SampleFn = Status (*)(const void *, int64_t, int32_t, int32_t, int32_t, const float *, const int32_t *,
                            const float *, const float *, const float *, int32_t *, float *, void *, size_t,
                            hipStream_t);
using SharedFn = Status (*)(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *, int32_t, int32_t,
                            int32_t, int32_t, const void *, int64_t, int32_t, const int32_t *, const int32_t *,
                            const int32_t *, int32_t, int32_t, int32_t, int32_t, int32_t, const int32_t *,
                            const int32_t *, int32_t, int32_t, float, int32_t, int32_t, void *, int64_t, float *,
                            void *, size_t, hipStream_t);

namespace {

AppendFn g_append;
AttnFn g_attn;
NormFn g_norm;
QuantMxFn g_quant_mx;
DequantMxFn g_dequant_mx;
GemmMxFn g_gemm_mx;
GemmMxQuantFn g_gemm_mx_quant;
SampleFn g_sample;
SharedFn g_shared;

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

// Rows of bf16 or fp32 with any row stride.
struct RowsOf {
    void *p;
    int64_t n, width, stride;
    int32_t fp32;
};
RowsOf float_rows(const Tensor &t, const char *what) {
    const auto kind = t.scalar_type();
    if (t.dim() != 2 || (kind != at::kFloat && kind != at::kBFloat16)) refuse(what, "bf16 or fp32 [rows][columns] expected");
    return {t.data_ptr(), t.size(0), t.size(1), row_stride(t, t.size(0), t.size(1), kind, what), kind == at::kFloat};
}
// Codes and scales of `rows` rows of K.
struct MxRows {
    const Tensor *c, *s;
    uint8_t *codes, *scales;
    int64_t n, K;
};
MxRows mx_rows(PyObject *codes, PyObject *scales, const char *what_c, const char *what_s) {
    MxRows m{&tensor(codes, what_c), &tensor(scales, what_s), nullptr, nullptr, 0, 0};
    if (m.c->dim() != 2) refuse(what_c, "uint8 [rows][K/2] expected");
    m.n = m.c->size(0);
    m.K = 2 * m.c->size(1);
    m.codes = bytes(m.c, m.n, m.K / 2, what_c);
    m.scales = bytes(m.s, m.n, m.K / 32, what_s);
    return m;
}
const Tensor &space(PyObject *o) {
    const Tensor &t = tensor(o, "workspace");
    if (!t.is_contiguous()) refuse("workspace", "contiguous memory expected");
    return t;
}

Status quant_mx(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    const RowsOf r = float_rows(x, "x");
    const MxRows m = mx_rows(a[1], a[2], "codes", "scales");
    if (m.n != r.n || m.K != r.width) refuse("codes", "uint8 [rows][K/2] of x's rows expected");
    on_one_gpu(a[4], {&x, m.c, m.s});
    return g_quant_mx(r.p, r.stride, r.fp32, size32(r.n, "x"), size32(r.width, "x"), m.codes, m.scales, stream(a[3]));
}

Status dequant_mx(PyObject *const *a) {
    const MxRows m = mx_rows(a[0], a[1], "codes", "scales");
    const Tensor &out = tensor(a[2], "out");
    const RowsOf r = float_rows(out, "out");
    if (m.n != r.n || m.K != r.width) refuse("out", "[rows][K] of the codes' rows expected");
    on_one_gpu(a[4], {m.c, m.s, &out});
    return g_dequant_mx(m.codes, m.scales, size32(m.n, "codes"), size32(m.K, "codes"), r.p, r.stride, r.fp32, stream(a[3]));
}

Status gemm_mx(PyObject *const *a) {
    const MxRows x = mx_rows(a[0], a[1], "a_codes", "a_scales"), w = mx_rows(a[2], a[3], "w_codes", "w_scales");
    const Tensor &y = tensor(a[4], "y"), &ws = space(a[5]);
    const RowsOf r = float_rows(y, "y");
    if (x.K != w.K) refuse("w_codes", "the rows' K expected");
    if (r.n != x.n || r.width != w.n) refuse("y", "[rows of a][rows of w] expected");
    on_one_gpu(a[7], {x.c, x.s, w.c, w.s, &y, &ws});
    return g_gemm_mx(x.codes, x.scales, w.codes, w.scales, size32(x.n, "a_codes"), size32(w.n, "w_codes"),
                     size32(w.K, "w_codes"), r.p, r.stride, r.fp32, ws.data_ptr(), ws.nbytes(), stream(a[6]));
}

Status gemm_mx_quant(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x"), &y = tensor(a[3], "y"), &ws = space(a[4]);
    if (x.dim() != 2) refuse("x", "bf16 [rows][K] expected");
    const MxRows w = mx_rows(a[1], a[2], "w_codes", "w_scales");
    const int64_t M = x.size(0), sx = row_stride(x, M, w.K, at::kBFloat16, "x");
    const RowsOf r = float_rows(y, "y");
    if (r.n != M || r.width != w.n) refuse("y", "[rows of x][rows of w] expected");
    on_one_gpu(a[6], {&x, w.c, w.s, &y, &ws});
    return g_gemm_mx_quant(x.data_ptr(), sx, w.codes, w.scales, size32(M, "x"), size32(w.n, "w_codes"),
                           size32(w.K, "w_codes"), r.p, r.stride, r.fp32, ws.data_ptr(), ws.nbytes(), stream(a[5]));
}

// One number a row, or nothing.
void *per_row(const Tensor *t, int64_t n, at::ScalarType type, const char *what) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || !shaped(*t, n) || !t->is_contiguous())
        refuse(what, type == at::kInt ? "contiguous int32 [rows] expected" : "contiguous fp32 [rows] expected");
    return t->data_ptr();
}

Status sample(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "logits"), &u = tensor(a[1], "u"), &token = tensor(a[6], "token"), &ws = space(a[8]);
    const RowsOf r = float_rows(x, "logits");
    const Tensor *t = maybe(a[2], "temperature"), *k = maybe(a[3], "top_k"), *p = maybe(a[4], "top_p"),
                 *m = maybe(a[5], "min_p"), *lp = maybe(a[7], "logprob");
    const void *pu = per_row(&u, r.n, at::kFloat, "u"), *pt = per_row(t, r.n, at::kFloat, "temperature"),
               *pk = per_row(k, r.n, at::kInt, "top_k"), *pp = per_row(p, r.n, at::kFloat, "top_p"),
               *pm = per_row(m, r.n, at::kFloat, "min_p");
    void *out = per_row(&token, r.n, at::kInt, "token"), *plp = per_row(lp, r.n, at::kFloat, "logprob");
    on_one_gpu(a[10], {&x, &u, t, k, p, m, &token, lp, &ws});
    return g_sample(r.p, r.stride, r.fp32, size32(r.n, "logits"), size32(r.width, "logits"), (const float *)pt,
                    (const int32_t *)pk, (const float *)pp, (const float *)pm, (const float *)pu, (int32_t *)out,
                    (float *)plp, ws.data_ptr(), ws.nbytes(), stream(a[9]));
}

Status shared(PyObject *const *a) {
    const Cache c = cache(a[0]);
    const Tensor &q = tensor(a[1], "q"), &out = tensor(a[13], "out"), &ws = space(a[15]),
                 &groups = tensor(a[5], "group_start"), &lens = tensor(a[6], "shared_len");
    if (q.dim() != 3) refuse("q", "[tokens][heads][dim] expected");
    const int64_t T = q.size(0);
    const int32_t heads = size32(q.size(1), "q");
    const Ragged r = ragged(a[2], a[3], a[4]);
    if (lens.dim() != 1) refuse("shared_len", "int32 [groups] expected");
    const int32_t n = size32(lens.size(0), "shared_len");
    const int32_t *len = ints(lens, "shared_len", n), *start = ints(groups, "group_start", n + 1);
    const Tensor *lse = maybe(a[14], "lse");
    if (lse && (lse->scalar_type() != at::kFloat || !shaped(*lse, T, heads) || !lse->is_contiguous()))
        refuse("lse", "contiguous fp32 [tokens][heads] expected");
    const int64_t sq = token_stride(q, T, heads, c.dim, "q"), so = token_stride(out, T, heads, c.dim, "out");
    on_one_gpu(a[17], {c.t[0], c.t[1], c.t[2], c.t[3], &q, &out, &ws, lse, &groups, &lens, &tensor(a[2], "q_start"),
                       &tensor(a[3], "kv_len"), &tensor(a[4], "block_table")});
    return g_shared(c.p[0], c.p[1], c.p[2], c.p[3], c.pages, c.heads, c.page, c.dim, q.data_ptr(), sq, heads, r.start,
                    r.len, r.table, r.max_pages, r.B, size32(T, "q"), integer32(a[7], "max_q_len"),
                    integer32(a[8], "max_kv_len"), start, len, n, integer32(a[9], "max_shared_len"), number(a[10]),
                    integer32(a[11], "window"), integer32(a[12], "sinks"), out.data_ptr(), so,
                    lse ? (float *)lse->data_ptr() : nullptr, ws.data_ptr(), ws.nbytes(), stream(a[16]));
}

// Calls f with `want` positional arguments; returns the status.
template <Status (*F)(PyObject *const *), int WANT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != WANT) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected", WANT);
        return nullptr;
    }
    if (!g_append) {
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
    constexpr int kEntries = 9;
    if (n != kEntries) {
        PyErr_Format(PyExc_TypeError, "%d addresses expected", kEntries);
        return nullptr;
    }
    void *p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_attn = (AttnFn)p[1];
    g_norm = (NormFn)p[2];
    g_quant_mx = (QuantMxFn)p[3];
    g_dequant_mx = (DequantMxFn)p[4];
    g_gemm_mx = (GemmMxFn)p[5];
    g_gemm_mx_quant = (GemmMxQuantFn)p[6];
    g_sample = (SampleFn)p[7];
    g_shared = (SharedFn)p[8];
    g_append = (AppendFn)p[0];
    Py_RETURN_NONE;
}

#define FASTCALL(f) ((PyCFunction)(void (*)(void))(f))
PyMethodDef methods[] = {{"bind", FASTCALL(bind), METH_FASTCALL, "addresses of the entry points"},
                         {"kv_append", FASTCALL((entry<append, 15>)), METH_FASTCALL, "biloco_kv_append"},
                         {"attn_paged", FASTCALL((entry<attn, 15>)), METH_FASTCALL, "biloco_attn_paged"},
                         {"norm_gate_residual", FASTCALL((entry<norm, 14>)), METH_FASTCALL, "biloco_norm_gate_residual"},
                         {"quant_mxfp4", FASTCALL((entry<quant_mx, 5>)), METH_FASTCALL, "biloco_quant_mxfp4"},
                         {"dequant_mxfp4", FASTCALL((entry<dequant_mx, 5>)), METH_FASTCALL, "biloco_dequant_mxfp4"},
                         {"gemm_mxfp4", FASTCALL((entry<gemm_mx, 8>)), METH_FASTCALL, "biloco_gemm_mxfp4"},
                         {"gemm_mxfp4_quant", FASTCALL((entry<gemm_mx_quant, 7>)), METH_FASTCALL, "biloco_gemm_mxfp4_quant"},
                         {"sample", FASTCALL((entry<sample, 11>)), METH_FASTCALL, "biloco_sample"},
                         {"attn_shared", FASTCALL((entry<shared, 18>)), METH_FASTCALL, "biloco_attn_shared"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding() { return PyModule_Create(&module); }
