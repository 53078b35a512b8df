// Python bindings of the calls whose host time counts (module _calls): the arguments are read from the
// tensors and checked here rather than in Python, where a call's marshalling took 8 to 20 us, several
// times the smallest kernels. Built against the installed torch's headers; the library's entry points
// are handed over by address (bind), so this module links to nothing of it.
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "spec_verify.h"

namespace {

using QkNormRope = decltype(&sv_qk_norm_rope);
using KvAppendRope = decltype(&sv_kv_append_rope);
using AttnScored = decltype(&sv_spec_verify_attn_scored);
using AttnScoredBytes = decltype(&sv_spec_verify_attn_scored_workspace_bytes);
QkNormRope g_heads;
KvAppendRope g_append;
AttnScored g_attn;
AttnScoredBytes g_attn_bytes;

struct TypeError : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void value_error(const std::string &what) { throw std::invalid_argument(what); }

int g_device;  // of the call's tensors; -1 before the first (calls hold the interpreter's lock)

const at::Tensor *tensor(PyObject *o) {  // null for None
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw TypeError("libspecverify takes CUDA tensors only");
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw TypeError("libspecverify takes CUDA tensors only");
  const int device = (int)t.get_device();
  if (g_device >= 0 && device != g_device) value_error("the tensors of a call are on one device");
  g_device = device;
  return &t;
}
const at::Tensor &needed(PyObject *o, const char *what) {
  const at::Tensor *t = tensor(o);
  if (t == nullptr) value_error(std::string(what) + " is missing");
  return *t;
}
void *contiguous(const at::Tensor *t) {
  if (t == nullptr) return nullptr;
  if (!t->is_contiguous()) value_error("libspecverify takes contiguous tensors only");
  return t->data_ptr();
}
template <typename T> T *values(const at::Tensor *t, at::ScalarType type, int64_t n, const char *what) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != type || t->numel() != n)
    value_error(std::string(what) + " holds " + std::to_string(n) + " values of " + c10::toString(type));
  return static_cast<T *>(contiguous(t));
}

// Rows of heads [n, heads, head_dim]: the heads of a row contiguous, the rows possibly parts of wider ones.
struct Rows {
  void *at = nullptr;
  int64_t stride = 0;
};
Rows rows_of(const at::Tensor &t, const at::Tensor *like) {
  if (t.dim() != 3) value_error("expected rows [n, heads, head_dim]");
  const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
  if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && h > 1)) value_error("the heads of a row are contiguous");
  if (like != nullptr && (t.sizes() != like->sizes() || t.scalar_type() != like->scalar_type()))
    value_error("outputs and values have their inputs' shape and type");
  Rows r;
  r.at = t.data_ptr();
  r.stride = n > 1 ? t.stride(0) : h * d;
  return r;
}
int row_type(const at::Tensor &t) {
  if (t.scalar_type() == at::kBFloat16) return SV_DTYPE_BF16;
  if (t.scalar_type() == at::kFloat) return SV_DTYPE_F32;
  throw TypeError(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}
int narrow(int64_t x) {
  if (x < INT32_MIN || x > INT32_MAX) value_error("a size does not fit 32 bits");
  return (int)x;
}
int64_t integer(PyObject *o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw TypeError("");
  return x;
}
float real(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw TypeError("");
  return (float)x;
}

struct Held {  // attributes, released at the end of the call
  PyObject *o[24];
  int n = 0;
  PyObject *get(PyObject *from, PyObject *name) {
    PyObject *x = PyObject_GetAttr(from, name);
    if (x == nullptr) throw TypeError("");
    return o[n++] = x;
  }
  ~Held() {
    while (n > 0) Py_DECREF(o[--n]);
  }
};

PyObject *s_names[16];
enum { kK, kV, kTable, kLens, kFree, kTop, kRef, kKScale, kVScale, kFreq, kQW, kKW, kEps, kOffset, kInter, kNames };

// A PagedKV, with its tensors held.
sv_paged_kv cache_of(PyObject *kv, Held &held) {
  sv_paged_kv p = {};
  auto field = [&](int name) { return tensor(held.get(kv, s_names[name])); };
  const at::Tensor *k = field(kK), *v = field(kV), *table = field(kTable), *lens = field(kLens);
  if (k == nullptr || v == nullptr || table == nullptr || lens == nullptr || k->dim() != 4 || table->dim() != 2)
    value_error("a cache has pools [blocks, heads, block_size, head_dim], a block table and lengths");
  if (v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type()) value_error("the pools have one shape and type");
  p.k_pool = contiguous(k);
  p.v_pool = contiguous(v);
  p.num_blocks = narrow(k->size(0));
  p.num_kv_heads = narrow(k->size(1));
  p.block_size = narrow(k->size(2));
  p.head_dim = narrow(k->size(3));
  p.batch = narrow(lens->numel());
  p.max_blocks_per_seq = narrow(table->size(1));
  p.block_table = values<int32_t>(table, at::kInt, (int64_t)p.batch * p.max_blocks_per_seq, "block_table");
  p.seq_lens = values<int32_t>(lens, at::kInt, p.batch, "seq_lens");
  p.free_list = values<int32_t>(field(kFree), at::kInt, p.num_blocks, "free_list");
  p.free_top = values<int32_t>(field(kTop), at::kInt, 1, "free_top");
  p.ref_count = values<int32_t>(field(kRef), at::kInt, p.num_blocks, "ref_count");
  p.dtype = k->scalar_type() == at::kByte ? SV_DTYPE_E4M3 : row_type(*k);
  p.k_scale = real(held.get(kv, s_names[kKScale]));
  p.v_scale = real(held.get(kv, s_names[kVScale]));
  return p;
}

// A HeadTransform for rows like `rows`, with its tensors held.
sv_head_transform transform_of(PyObject *t, const at::Tensor &rows, Held &held) {
  sv_head_transform p = {};
  auto field = [&](int name) { return held.get(t, s_names[name]); };
  if (const at::Tensor *f = tensor(field(kFreq))) {
    if (f->scalar_type() != at::kFloat) throw TypeError("inv_freq is float32");
    p.rotary_dim = narrow(2 * f->numel());
    p.inv_freq = p.rotary_dim > 0 ? static_cast<const float *>(contiguous(f)) : nullptr;
  }
  p.q_weight = values<void>(tensor(field(kQW)), rows.scalar_type(), rows.size(2), "a norm weight");
  p.k_weight = values<void>(tensor(field(kKW)), rows.scalar_type(), rows.size(2), "a norm weight");
  p.eps = real(field(kEps));
  p.weight_offset = real(field(kOffset));
  p.interleaved = PyObject_IsTrue(field(kInter));
  if (p.interleaved < 0) throw TypeError("");
  return p;
}

void *address(PyObject *stream) { return reinterpret_cast<void *>(static_cast<uintptr_t>(integer(stream))); }

// Every call answers with the library's status.
template <typename F> PyObject *answer(Py_ssize_t n, Py_ssize_t want, F call) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  g_device = -1;
  try {
    return PyLong_FromLong(call());
  } catch (const TypeError &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {  // torch's own, as torch raises them (out of memory among them)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// (transform, q, k, positions, q_out, k_out, stream)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return answer(n, 7, [&] {
    const at::Tensor *q = tensor(a[1]), *k = tensor(a[2]), *some = q != nullptr ? q : k;
    if (some == nullptr) value_error("no rows: q and k are both None");
    Rows rq, rqo, rk, rko;
    int hq = 0, hkv = 0;
    rows_of(*some, nullptr);  // its dimensions are there to be read
    if (q != nullptr) {
      rq = rows_of(*q, nullptr);
      rqo = rows_of(needed(a[4], "q_out"), q);
      hq = narrow(q->size(1));
    }
    if (k != nullptr) {
      rk = rows_of(*k, nullptr);
      rko = rows_of(needed(a[5], "k_out"), k);
      hkv = narrow(k->size(1));
      if (k->size(0) != some->size(0) || k->size(2) != some->size(2) || k->scalar_type() != some->scalar_type())
        value_error("q and k have the same rows, head_dim and type");
    }
    Held held;
    const sv_head_transform t = transform_of(a[0], *some, held);
    const int rows = narrow(some->size(0));
    return g_heads(&t, rq.at, rq.stride, rqo.at, rqo.stride, hq, rk.at, rk.stride, rko.at, rko.stride, hkv,
                   narrow(some->size(2)), row_type(*some), rows, values<int32_t>(tensor(a[3]), at::kInt, rows, "positions"),
                   address(a[6]));
  });
}

// (kv, transform, new_k, new_v, cu_q, status, q, q_out, positions, stream)
PyObject *kv_append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return answer(n, 10, [&] {
    Held held;
    const sv_paged_kv kv = cache_of(a[0], held);
    const at::Tensor &k = needed(a[2], "new_k");
    const Rows rk = rows_of(k, nullptr), rv = rows_of(needed(a[3], "new_v"), &k);
    const int want = kv.dtype == SV_DTYPE_F32 ? SV_DTYPE_F32 : SV_DTYPE_BF16;
    if (row_type(k) != want || k.size(1) != kv.num_kv_heads || k.size(2) != kv.head_dim)
      value_error("new rows are [n, num_kv_heads, head_dim] of the cache's row type");
    const int rows = narrow(k.size(0));
    Rows rq, rqo;
    int hq = 0;
    if (const at::Tensor *q = tensor(a[6])) {
      rq = rows_of(*q, nullptr);
      if (q->size(0) != rows || q->size(2) != kv.head_dim || row_type(*q) != want)
        value_error("queries are [n, heads, head_dim] of the new rows' number and type");
      rqo = rows_of(needed(a[7], "q_out"), q);
      hq = narrow(q->size(1));
    }
    const sv_head_transform t = transform_of(a[1], k, held);
    return g_append(&kv, &t, rk.at, rk.stride, rv.at, rv.stride, rq.at, rq.stride, rqo.at, rqo.stride, hq,
                    values<int32_t>(tensor(a[4]), at::kInt, (int64_t)kv.batch + 1, "cu_q"), rows,
                    values<int32_t>(tensor(a[8]), at::kInt, rows, "positions"),
                    values<int32_t>(tensor(a[5]), at::kInt, 1, "status"), address(a[9]));
  });
}

// (kv, q, out, cu_q, max_q, max_seq_len, scale, softcap, slopes, window, positions, mask_kind, tree_mask, workspace, status,
// stream); without a workspace one is taken here, from the current stream's allocator
PyObject *spec_verify_attn_scored(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return answer(n, 16, [&] {
    Held held;
    const sv_paged_kv kv = cache_of(a[0], held);
    const at::Tensor &q = needed(a[1], "q"), &out = needed(a[2], "out");
    const int want = kv.dtype == SV_DTYPE_F32 ? SV_DTYPE_F32 : SV_DTYPE_BF16;
    if (q.dim() != 3 || row_type(q) != want || q.size(2) != kv.head_dim || out.sizes() != q.sizes() ||
        out.scalar_type() != q.scalar_type())
      value_error("queries and outputs are [n, heads, head_dim] of the cache's row type");
    const int rows = narrow(q.size(0)), hq = narrow(q.size(1)), max_q = narrow(integer(a[4])), max_len = narrow(integer(a[5]));
    const at::Tensor *tree = tensor(a[12]);
    if (tree != nullptr && (tree->element_size() != 8 || tree->numel() != rows))
      value_error("tree_mask holds " + std::to_string(rows) + " 64-bit values");
    sv_score_mod mod = {};
    mod.softcap = real(a[7]);
    mod.slopes = values<const float>(tensor(a[8]), at::kFloat, hq, "slopes");
    mod.window = narrow(integer(a[9]));
    at::Tensor own;
    const at::Tensor *ws = tensor(a[13]);
    if (ws == nullptr) {
      const size_t need = g_attn_bytes(&kv, hq, rows, max_q, max_len);
      own = at::empty({(int64_t)(need > 0 ? need : 1)}, q.options().dtype(at::kByte));
      ws = &own;
    }
    return g_attn(&kv, contiguous(&q), contiguous(&out), values<int32_t>(tensor(a[3]), at::kInt, (int64_t)kv.batch + 1, "cu_q"),
                  hq, rows, max_q, max_len, real(a[6]), &mod, values<int32_t>(tensor(a[10]), at::kInt, rows, "positions"),
                  narrow(integer(a[11])), static_cast<const uint64_t *>(contiguous(tree)), contiguous(ws),
                  (size_t)ws->numel() * ws->element_size(), values<int32_t>(tensor(a[14]), at::kInt, 1, "status"), address(a[15]));
  });
}

// The library's entry points, by address.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return answer(n, 4, [&] {
    g_heads = reinterpret_cast<QkNormRope>(address(a[0]));
    g_append = reinterpret_cast<KvAppendRope>(address(a[1]));
    g_attn = reinterpret_cast<AttnScored>(address(a[2]));
    g_attn_bytes = reinterpret_cast<AttnScoredBytes>(address(a[3]));
    return 0;
  });
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(qk_norm_rope), METH_FASTCALL, nullptr},
    {"kv_append_rope", reinterpret_cast<PyCFunction>(kv_append_rope), METH_FASTCALL, nullptr},
    {"spec_verify_attn_scored", reinterpret_cast<PyCFunction>(spec_verify_attn_scored), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__calls() {
  static const char *names[kNames] = {"k_pool",  "v_pool",  "block_table", "seq_lens", "free_list", "free_top",      "ref_count",  "k_scale",
                                      "v_scale", "inv_freq", "q_weight",    "k_weight", "eps",       "weight_offset", "interleaved"};
  for (int k = 0; k < kNames; ++k)
    if ((s_names[k] = PyUnicode_InternFromString(names[k])) == nullptr) return nullptr;
  return PyModule_Create(&g_module);
}
