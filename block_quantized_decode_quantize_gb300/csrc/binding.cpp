// The quick way into the entry points that run several times a decode step on small data.
//
// A call through ctypes spends most of its time on the argument checks and conversions in
// Python (20 to 40 us on a GB300's host, more than the kernels take); the functions here do
// the same checks on the tensors' C++ objects, take the outputs from torch's allocator and
// call the C ABI.  Each returns the outputs, or None where anything is not as expected: the
// Python function of the same name then takes its long way, which names what is wrong (or
// handles it, as a tensor of another device than the current one).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "memra.h"

namespace {

using at::Tensor;

// A plain tensor on CUDA device `dev` (-1: any, and *dev is set).
inline const Tensor* tensor(PyObject* o, int* dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) return nullptr;
  if (*dev < 0) *dev = t.get_device();
  return t.get_device() == *dev ? &t : nullptr;
}

inline bool dense(const Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
  return t != nullptr && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}

// bf16 or fp32 with a dense last dimension; *code receives the dtype's.
inline bool rows(const Tensor* t, int64_t dims, int32_t* code) {
  if (t == nullptr || t->dim() != dims) return false;
  if (t->scalar_type() == at::kBFloat16) *code = MEMRA_BF16;
  else if (t->scalar_type() == at::kFloat) *code = MEMRA_F32;
  else return false;
  return t->size(dims - 1) <= 1 || t->stride(dims - 1) == 1;
}

// Strides of rows and heads of [rows][heads][D]; those of a single row or head, which reach
// nothing and may be any number, as if dense.
struct Strides {
  int64_t t, h;
  explicit Strides(const Tensor* x)
      : t(x->size(0) > 1 ? x->stride(0) : x->size(1) * x->size(2)),
        h(x->size(1) > 1 ? x->stride(1) : x->size(2)) {}
  bool operator==(const Strides& o) const { return t == o.t && h == o.h; }
};

template <typename V>
inline V* data(const Tensor* t) {
  return t != nullptr ? static_cast<V*>(t->data_ptr()) : nullptr;
}

// An int32 word on `dev`, or None (nullptr).  False: neither.
inline bool word(PyObject* o, int dev, int32_t** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const Tensor* t = tensor(o, &dev);
  if (!dense(t, at::kInt, {1})) return false;
  *p = data<int32_t>(t);
  return true;
}

inline bool whole(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}

inline bool real(PyObject* o, float* v) {
  if (!PyFloat_CheckExact(o)) return false;
  *v = (float)PyFloat_AS_DOUBLE(o);
  return true;
}

inline bool current(int dev) { return c10::cuda::current_device() == dev; }
inline cudaStream_t stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
inline at::TensorOptions on(int dev, at::ScalarType type) {
  return at::TensorOptions().device(at::kCUDA, (c10::DeviceIndex)dev).dtype(type);
}

PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (out == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (o == nullptr) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// A contiguous part of a buffer, from element `at` (of `type`) on, as a tensor that shares its storage: what views of it would be, at a fraction of their cost.
Tensor part(const Tensor& buf, int64_t at, at::IntArrayRef shape, at::ScalarType type) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                      c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(buf.storage_offset() + at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}
Tensor part(const Tensor& buf, int64_t at, at::IntArrayRef shape) { return part(buf, at, shape, buf.scalar_type()); }

struct Cache {
  int8_t *kq, *vq;
  float *kd, *vd;
  int64_t n_pages, heads, page, D, block;
};

inline bool cache(PyObject* const* o, int* dev, Cache* c) {
  const Tensor *kq = tensor(o[0], dev), *kd = tensor(o[1], dev);
  const Tensor *vq = tensor(o[2], dev), *vd = tensor(o[3], dev);
  if (kq == nullptr || kd == nullptr || kq->dim() != 4 || kd->dim() != 3) return false;
  c->n_pages = kq->size(0);
  c->heads = kq->size(1);
  c->page = kq->size(2);
  c->D = kq->size(3);
  const int64_t blocks = kd->size(2);
  if (blocks < 1 || c->page % blocks != 0) return false;
  c->block = c->page / blocks;
  const int64_t scales[3] = {c->n_pages, c->heads, blocks};
  if (!dense(kq, at::kChar, kq->sizes()) || !dense(vq, at::kChar, kq->sizes()) ||
      !dense(kd, at::kFloat, scales) || !dense(vd, at::kFloat, scales))
    return false;
  c->kq = data<int8_t>(kq);
  c->kd = data<float>(kd);
  c->vq = data<int8_t>(vq);
  c->vd = data<float>(vd);
  return true;
}

// plan(ctx_lens, new_lens, page_size, free_pages, block_table, num_tokens, free_head,
//      free_head_out, dev_status): all outputs but, where given, free_head_out are new.
PyObject* plan(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  int dev = -1;
  const Tensor *ctx = tensor(o[0], &dev), *add = tensor(o[1], &dev), *free = tensor(o[3], &dev);
  const Tensor* table = tensor(o[4], &dev);
  int64_t page, T;
  int32_t *head, *head_out, *status;
  if (ctx == nullptr || ctx->dim() != 1 || free == nullptr || free->dim() != 1 ||
      table == nullptr || table->dim() != 2 || !whole(o[2], &page) || !whole(o[5], &T) || T < 0)
    Py_RETURN_NONE;
  const int64_t B = ctx->size(0), max_pages = table->size(1), n_free = free->size(0);
  if (!dense(ctx, at::kInt, {B}) || !dense(add, at::kInt, {B}) || !dense(free, at::kInt, {n_free}) ||
      !dense(table, at::kInt, {B, max_pages}) || !word(o[6], dev, &head) ||
      !word(o[7], dev, &head_out) || !word(o[8], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  // one allocation; slots and positions first, which keeps them 16-byte aligned
  const int64_t pad = (4 - T % 4) % 4;
  const Tensor buf = at::empty({2 * (T + pad) + 2 * B + 2}, on(dev, at::kInt));
  const int64_t sizes[7] = {T, pad, T, pad, B, B + 1, 1};
  const std::vector<Tensor> part = buf.split_with_sizes(sizes);
  if (head_out == nullptr) head_out = data<int32_t>(&part[6]);
  if (memra_kv_plan(data<int32_t>(ctx), data<int32_t>(add), B, page, data<int32_t>(free), n_free,
                    head, data<int32_t>(table), max_pages, T, data<int32_t>(&part[4]),
                    data<int32_t>(&part[5]), data<int32_t>(&part[0]), data<int32_t>(&part[2]),
                    head_out, status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({part[4], part[5], part[0], part[2],
               o[7] == Py_None ? part[6] : THPVariable_Unpack(o[7])});
  END_HANDLE_TH_ERRORS
}

// append(k, v, slots, kq, kd, vq, vd, dev_status): True when done.
PyObject* append(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  int dev = -1;
  Cache c;
  if (!cache(o + 3, &dev, &c)) Py_RETURN_NONE;
  const Tensor *k = tensor(o[0], &dev), *v = tensor(o[1], &dev), *slots = tensor(o[2], &dev);
  int32_t code, code_v, *status;
  if (!rows(k, 3, &code) || !rows(v, 3, &code_v) || code != code_v || k->size(1) != c.heads ||
      k->size(2) != c.D || v->sizes() != k->sizes() || !(Strides(v) == Strides(k)) ||
      !dense(slots, at::kInt, {k->size(0)}) || !word(o[7], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  const Strides step(k);
  if (memra_kv_append_q8(data<void>(k), data<void>(v), code, k->size(0), step.t, step.h,
                         data<int32_t>(slots), c.kq, c.kd, c.vq, c.vd, c.n_pages, c.heads, c.page,
                         c.D, c.block, status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// read(slots, kq, kd, vq, vd, is_bf16, dev_status) -> (k, v)
PyObject* read(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) Py_RETURN_NONE;
  int dev = -1;
  Cache c;
  if (!cache(o + 1, &dev, &c)) Py_RETURN_NONE;
  const Tensor* slots = tensor(o[0], &dev);
  int32_t* status;
  if (slots == nullptr || slots->dim() != 1 || !dense(slots, at::kInt, slots->sizes()) ||
      !word(o[6], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  const bool bf16 = o[5] == Py_True;
  const int64_t N = slots->size(0);
  at::AutoDispatchBelowADInplaceOrView guard;
  const auto opts = on(dev, bf16 ? at::kBFloat16 : at::kFloat);
  const Tensor k = at::empty({N, c.heads, c.D}, opts), v = at::empty({N, c.heads, c.D}, opts);
  if (memra_kv_read_q8(data<int32_t>(slots), N, c.kq, c.kd, c.vq, c.vd, c.n_pages, c.heads, c.page,
                       c.D, c.block, bf16 ? MEMRA_BF16 : MEMRA_F32, k.data_ptr(), v.data_ptr(),
                       status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({k, v});
  END_HANDLE_TH_ERRORS
}

// attention(q, kq, kd, vq, vd, block_table, kv_lens, cu_q, scale, window, workspace,
//           dev_status) -> (out, lse)
PyObject* attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) Py_RETURN_NONE;
  int dev = -1;
  Cache c;
  if (!cache(o + 1, &dev, &c)) Py_RETURN_NONE;
  const Tensor *q = tensor(o[0], &dev), *table = tensor(o[5], &dev), *lens = tensor(o[6], &dev);
  const Tensor *cu = tensor(o[7], &dev), *ws = tensor(o[10], &dev);
  int32_t code, *status;
  int64_t window;
  float scale;
  if (!rows(q, 3, &code) || q->size(2) != c.D || q->size(1) < 1 || c.heads < 1 ||
      q->size(1) % c.heads != 0 || table == nullptr || table->dim() != 2)
    Py_RETURN_NONE;
  const int64_t T = q->size(0), Hq = q->size(1), B = table->size(0), max_pages = table->size(1);
  if (!dense(table, at::kInt, table->sizes()) || !dense(lens, at::kInt, {B}) ||
      !dense(cu, at::kInt, {B + 1}) || !real(o[8], &scale) || !whole(o[9], &window) ||
      ws == nullptr || ws->scalar_type() != at::kByte || !ws->is_contiguous() ||
      ws->numel() < MEMRA_KV_ATTENTION_WORKSPACE_BYTES || !word(o[11], dev, &status) ||
      !current(dev))
    Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const Tensor out = at::empty({T, Hq, c.D}, on(dev, q->scalar_type()));
  const Tensor lse = at::empty({T, Hq}, on(dev, at::kFloat));
  const Strides step(q);
  if (memra_kv_attention_q8(data<void>(q), code, T, Hq, step.t, step.h, c.kq, c.kd,
                            c.vq, c.vd, c.n_pages, c.heads, c.page, c.D, c.block,
                            data<int32_t>(table), B, max_pages, data<int32_t>(lens),
                            data<int32_t>(cu), scale, window, out.data_ptr(),
                            data<float>(&lse), ws->data_ptr(), status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({out, lse});
  END_HANDLE_TH_ERRORS
}

// route(logits, top_k, bias, score, n_groups, topk_groups, group_top, renormalize, scale)
//   -> (ids, gate_w)
PyObject* route(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  int dev = -1;
  const Tensor* x = tensor(o[0], &dev);
  int32_t code;
  int64_t top_k, score, groups, kept, per;
  float scale;
  if (!rows(x, 2, &code) || !whole(o[1], &top_k) || top_k < 1 || !whole(o[3], &score) ||
      !whole(o[4], &groups) || !whole(o[5], &kept) || !whole(o[6], &per) || !PyBool_Check(o[7]) ||
      !real(o[8], &scale) || !current(dev))
    Py_RETURN_NONE;
  const int64_t T = x->size(0), E = x->size(1);
  const Tensor* bias = nullptr;
  if (o[2] != Py_None) {
    bias = tensor(o[2], &dev);
    if (!dense(bias, at::kFloat, {E})) Py_RETURN_NONE;
  }
  at::AutoDispatchBelowADInplaceOrView guard;
  const Tensor ids = at::empty({T, top_k}, on(dev, at::kInt));
  const Tensor gate = at::empty({T, top_k}, on(dev, at::kFloat));
  if (memra_moe_route(data<void>(x), code, T, E, x->stride(0), data<float>(bias), (int32_t)score,
                      groups, kept, per, top_k, o[7] == Py_True ? 1 : 0, scale,
                      data<int32_t>(&ids), data<float>(&gate), stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({ids, gate});
  END_HANDLE_TH_ERRORS
}

// A dense int32 tensor of `dims` dimensions.
inline bool ints(const Tensor* t, int64_t dims) {
  return t != nullptr && t->dim() == dims && t->scalar_type() == at::kInt && t->is_contiguous();
}

// One that may be None (nullptr).  False: neither.
inline bool optional(PyObject* o, int dev, at::ScalarType type, at::IntArrayRef shape, const Tensor** t) {
  *t = nullptr;
  if (o == Py_None) return true;
  *t = tensor(o, &dev);
  return dense(*t, type, shape);
}

// Rows that a call writes.  Given ones have to be like x and of the C library's dtype code `want`
// (-1: any); where there are none (None), their number of bytes is left in *bytes and *type is want,
// or the input's code.
inline bool out_rows(PyObject* o, int* dev, const Tensor* x, int64_t want, int32_t code, Tensor* t, int32_t* type,
                     int64_t* bytes) {
  *bytes = 0;
  if (o == Py_None) {
    *type = (int32_t)(want < 0 ? code : want);
    *bytes = x->numel() * (*type == MEMRA_BF16 ? 2 : 4);
    return true;
  }
  const Tensor* given = tensor(o, dev);
  if (!rows(given, 3, type) || given->sizes() != x->sizes() || (want >= 0 && want != *type)) return false;
  *t = *given;
  return true;
}

// rope(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, q_dtype, k_dtype, q_out, k_out)
//   -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) Py_RETURN_NONE;
  int dev = -1;
  const Tensor *q = tensor(o[0], &dev), *k = tensor(o[1], &dev);
  int32_t code, code_k, qo_type, ko_type;
  int64_t layout, q_type, k_type;
  float eps = -1.0f;
  if (!rows(q, 3, &code) || !rows(k, 3, &code_k) || code != code_k || k->size(0) != q->size(0) ||
      k->size(2) != q->size(2) || (o[6] != Py_None && (!real(o[6], &eps) || !(eps >= 0.0f))) ||
      !whole(o[7], &layout) || !whole(o[8], &q_type) || !whole(o[9], &k_type) || q_type < -1 || k_type < -1 ||
      !current(dev))
    Py_RETURN_NONE;
  const int64_t T = q->size(0), Hq = q->size(1), Hkv = k->size(1), D = q->size(2);
  const Tensor *positions, *freq = nullptr, *qw, *kw;
  if (!optional(o[2], dev, at::kInt, {T}, &positions) || !optional(o[4], dev, at::kFloat, {D}, &qw) ||
      !optional(o[5], dev, at::kFloat, {D}, &kw))
    Py_RETURN_NONE;
  int64_t R = 0;
  if (o[3] != Py_None) {
    freq = tensor(o[3], &dev);
    if (freq == nullptr || freq->dim() != 1 || !dense(freq, at::kDouble, freq->sizes())) Py_RETURN_NONE;
    R = 2 * freq->size(0);
  }
  at::AutoDispatchBelowADInplaceOrView guard;
  Tensor qo, ko;
  int64_t q_bytes, k_bytes;
  if (!out_rows(o[10], &dev, q, q_type, code, &qo, &qo_type, &q_bytes) ||
      !out_rows(o[11], &dev, k, k_type, code, &ko, &ko_type, &k_bytes))
    Py_RETURN_NONE;
  // one allocation for both; k's rows on a boundary of 16 bytes
  const int64_t k_at = (q_bytes + 15) / 16 * 16;
  const auto type_of = [](int32_t t) { return t == MEMRA_BF16 ? at::kBFloat16 : at::kFloat; };
  if (o[10] == Py_None || o[11] == Py_None) {
    const Tensor buf = at::empty({k_at + k_bytes}, on(dev, at::kByte));
    if (o[10] == Py_None) qo = part(buf, 0, q->sizes(), type_of(qo_type));
    if (o[11] == Py_None) ko = part(buf, k_at / (ko_type == MEMRA_BF16 ? 2 : 4), k->sizes(), type_of(ko_type));
  }
  const Strides sq(q), sk(k), so(&qo), sko(&ko);
  if (memra_qk_norm_rope(data<void>(q), data<void>(k), code, T, Hq, Hkv, D, sq.t, sq.h, sk.t, sk.h,
                         data<float>(qw), data<float>(kw), eps, data<int32_t>(positions),
                         data<double>(freq), R, (int32_t)layout, qo.data_ptr(), qo_type, so.t, so.h,
                         ko.data_ptr(), ko_type, sko.t, sko.h, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({qo, ko});
  END_HANDLE_TH_ERRORS
}

// Sequences: lens [B] and block_table [B, max_pages].
struct Sequences {
  int32_t *lens, *table;
  int64_t B, max_pages;
};
inline bool sequences(PyObject* lens, PyObject* table, int* dev, Sequences* s) {
  const Tensor *l = tensor(lens, dev), *t = tensor(table, dev);
  if (!ints(l, 1) || !ints(t, 2) || t->size(0) != l->size(0)) return false;
  s->lens = data<int32_t>(l);
  s->table = data<int32_t>(t);
  s->B = l->size(0);
  s->max_pages = t->size(1);
  return true;
}

// fork(parents, lens, block_table, page_size, refs, prefix_lens, dev_status) -> (lens, table)
PyObject* fork(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) Py_RETURN_NONE;
  int dev = -1;
  Sequences s;
  int64_t page;
  int32_t* status;
  if (!sequences(o[1], o[2], &dev, &s) || !whole(o[3], &page) || !word(o[6], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  const Tensor *parents = tensor(o[0], &dev), *refs = tensor(o[4], &dev), *prefix;
  if (!ints(parents, 1) || !ints(refs, 1)) Py_RETURN_NONE;
  const int64_t C = parents->size(0);
  if (!optional(o[5], dev, at::kInt, {C}, &prefix)) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const Tensor buf = at::empty({C + C * s.max_pages}, on(dev, at::kInt));
  int32_t* at = data<int32_t>(&buf);
  if (memra_kv_fork(data<int32_t>(parents), data<int32_t>(prefix), C, s.lens, s.table, s.B, s.max_pages, page,
                    data<int32_t>(refs), refs->size(0), at, at + C, status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({part(buf, 0, {C}), part(buf, C, {C, s.max_pages})});
  END_HANDLE_TH_ERRORS
}

// unshare(lens, new_lens, page_size, refs, free_pages, block_table, free_head, free_head_out,
//         dev_status) -> (new_lens, src, dst, tokens, free_head)
PyObject* unshare(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  int dev = -1;
  Sequences s;
  int64_t page;
  int32_t *head, *head_out, *status;
  if (!sequences(o[0], o[5], &dev, &s) || !whole(o[2], &page) || !word(o[6], dev, &head) ||
      !word(o[7], dev, &head_out) || !word(o[8], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  const Tensor *add = tensor(o[1], &dev), *refs = tensor(o[3], &dev), *free = tensor(o[4], &dev);
  if (!dense(add, at::kInt, {s.B}) || !ints(refs, 1) || !ints(free, 1)) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const Tensor buf = at::empty({4 * s.B + 1}, on(dev, at::kInt));
  int32_t* at = data<int32_t>(&buf);
  if (memra_kv_unshare(s.lens, data<int32_t>(add), s.B, page, data<int32_t>(refs), refs->size(0),
                       data<int32_t>(free), free->size(0), head, s.table, s.max_pages, at, at + s.B,
                       at + 2 * s.B, at + 3 * s.B, head_out != nullptr ? head_out : at + 4 * s.B, status,
                       stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({part(buf, 0, {s.B}), part(buf, s.B, {s.B}), part(buf, 2 * s.B, {s.B}), part(buf, 3 * s.B, {s.B}),
               o[7] == Py_None ? part(buf, 4 * s.B, {1}) : THPVariable_Unpack(o[7])});
  END_HANDLE_TH_ERRORS
}

// copy_pages(src, dst, caches, tokens, dev_status): True when done.  caches: a list or tuple of
// tuples (kq, kd, vq, vd).
PyObject* copy_pages(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || (!PyList_CheckExact(o[2]) && !PyTuple_CheckExact(o[2]))) Py_RETURN_NONE;
  const Py_ssize_t L = PySequence_Fast_GET_SIZE(o[2]);
  if (L < 1) Py_RETURN_NONE;
  int dev = -1;
  Cache first{}, c;
  std::vector<memra_kv_layer> layers((size_t)L);
  for (Py_ssize_t l = 0; l < L; ++l) {
    PyObject* one = PySequence_Fast_GET_ITEM(o[2], l);
    if (!PyTuple_CheckExact(one) || PyTuple_GET_SIZE(one) != 4) Py_RETURN_NONE;
    if (!cache(PySequence_Fast_ITEMS(one), &dev, &c)) Py_RETURN_NONE;
    if (l == 0) first = c;
    if (c.n_pages != first.n_pages || c.heads != first.heads || c.page != first.page || c.D != first.D ||
        c.block != first.block)
      Py_RETURN_NONE;
    layers[(size_t)l] = {c.kq, c.kd, c.vq, c.vd};
  }
  const Tensor *src = tensor(o[0], &dev), *dst = tensor(o[1], &dev), *tokens;
  int32_t* status;
  if (!ints(src, 1) || !dense(dst, at::kInt, {src->size(0)}) ||
      !optional(o[3], dev, at::kInt, {src->size(0)}, &tokens) || !word(o[4], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  if (memra_kv_copy_pages(data<int32_t>(src), data<int32_t>(dst), data<int32_t>(tokens), src->size(0),
                          layers.data(), L, first.n_pages, first.heads, first.page, first.D, first.block,
                          status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// release(lens, page_size, block_table, refs, free_pages, free_head, keep_lens, free_head_out,
//         dev_status) -> (lens, free_head)
PyObject* release(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  int dev = -1;
  Sequences s;
  int64_t page;
  int32_t *head, *head_out, *status;
  if (!sequences(o[0], o[2], &dev, &s) || !whole(o[1], &page) || !word(o[5], dev, &head) || head == nullptr ||
      !word(o[7], dev, &head_out) || !word(o[8], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  const Tensor *refs = tensor(o[3], &dev), *free = tensor(o[4], &dev), *keep;
  if (!ints(refs, 1) || !ints(free, 1) || !optional(o[6], dev, at::kInt, {s.B}, &keep)) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const Tensor buf = at::empty({s.B + 1}, on(dev, at::kInt));
  int32_t* at = data<int32_t>(&buf);
  if (memra_kv_release(s.lens, data<int32_t>(keep), s.B, page, s.table, s.max_pages, data<int32_t>(refs),
                       refs->size(0), data<int32_t>(free), free->size(0), head, at,
                       head_out != nullptr ? head_out : at + s.B, status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({part(buf, 0, {s.B}), o[7] == Py_None ? part(buf, s.B, {1}) : THPVariable_Unpack(o[7])});
  END_HANDLE_TH_ERRORS
}

// compact(lens, block_table, page_size, n_pages, dev_status) -> (table, refs, free, src, dst, head)
PyObject* compact(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5) Py_RETURN_NONE;
  int dev = -1;
  Sequences s;
  int64_t page, pages;
  int32_t* status;
  if (!sequences(o[0], o[1], &dev, &s) || !whole(o[2], &page) || !whole(o[3], &pages) || pages < 0 ||
      pages > INT32_MAX || !word(o[4], dev, &status) || !current(dev))
    Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const int64_t cells = s.B * s.max_pages, moves = pages / 2;
  const Tensor buf = at::empty({cells + 2 * pages + 2 * moves + 1}, on(dev, at::kInt));
  int32_t *table = data<int32_t>(&buf), *refs = table + cells, *free = refs + pages, *src = free + pages;
  if (memra_kv_compact(s.lens, s.table, s.B, s.max_pages, page, pages, table, refs, free, src, src + moves,
                       src + 2 * moves, status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  int64_t at = cells;
  auto next = [&](int64_t n) {
    at += n;
    return part(buf, at - n, {n});
  };
  const Tensor r = next(pages), f = next(pages), from = next(moves), to = next(moves), head = next(1);
  return pack({part(buf, 0, {s.B, s.max_pages}), r, f, from, to, head});
  END_HANDLE_TH_ERRORS
}

// logprobs(logits, tokens, top_n, dev_status) -> (logprobs or None, entropy, top_ids, top_logprobs)
PyObject* logprobs(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) Py_RETURN_NONE;
  int dev = -1;
  const Tensor* x = tensor(o[0], &dev);
  int32_t code, *status;
  int64_t top;
  if (!rows(x, 2, &code) || !whole(o[2], &top) || top < 0 || top > x->size(1) || !word(o[3], dev, &status) ||
      !current(dev))
    Py_RETURN_NONE;
  const int64_t T = x->size(0), V = x->size(1);
  const Tensor* tokens;
  if (!optional(o[1], dev, at::kInt, {T}, &tokens)) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const int64_t ids_at = 2 * T, best_at = ids_at + T * top;
  const Tensor buf = at::empty({best_at + T * top}, on(dev, at::kFloat));
  float* at = data<float>(&buf);
  if (memra_token_logprobs(data<void>(x), code, T, V, T > 1 ? x->stride(0) : V, data<int32_t>(tokens), top,
                           tokens != nullptr ? at : nullptr, at + T, reinterpret_cast<int32_t*>(at + ids_at),
                           at + best_at, status, stream(dev)) != MEMRA_OK)
    Py_RETURN_NONE;
  return pack({tokens != nullptr ? part(buf, 0, {T}) : Tensor(), part(buf, T, {T}), part(buf, ids_at, {T, top}, at::kInt),
               part(buf, best_at, {T, top})});
  END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(plan), FAST(append), FAST(read), FAST(attention), FAST(route),
                         FAST(rope), FAST(fork), FAST(unshare), FAST(copy_pages), FAST(release),
                         FAST(compact), FAST(logprobs),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_memra_binding",
                          "Quick paths of the package's small calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__memra_binding() { return PyModule_Create(&module_def); }
