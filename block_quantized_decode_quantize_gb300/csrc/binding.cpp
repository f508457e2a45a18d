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

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(plan), FAST(append), FAST(read), FAST(attention), FAST(route),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_memra_binding",
                          "Quick paths of the package's small calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__memra_binding() { return PyModule_Create(&module_def); }
