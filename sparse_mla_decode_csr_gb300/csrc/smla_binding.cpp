// _smla.so: the paged calls of the Python binding, for well-formed arguments.
//
// Some of these calls take less time on the GPU than Python needs to look at a
// dozen tensors (tree masks: 3 us and 7), so the tensors' properties are read here.
// A function returns True when it has made its C call with success.  It returns False, and has
// enqueued nothing, when anything is not as the call wants it or is less common (a stream
// given by hand): the caller then goes through the checks in Python, which name the fault.  A
// launch that failed is returned as its status: an attend has two, the first of which may have
// gone through, so the call is not made again.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>

#include "smla.h"

namespace {

constexpr int64_t kMaxSize = int64_t(1) << 30;  // of a dimension that becomes an int32

// The arguments of a call, in turn; `ok` falls when one is not what is asked for.
struct Args {
  PyObject* const* v;
  Py_ssize_t n, at = 0;
  bool ok = true;
  int device = -2;

  Args(PyObject* const* args, Py_ssize_t count) : v(args), n(count) {}
  PyObject* next() {
    if (at >= n) {
      ok = false;
      return Py_None;
    }
    return v[at++];
  }
  // A tensor on the current device (null: None, where that is allowed).
  const at::Tensor* tensor(bool optional = false) {
    PyObject* o = next();
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) {
      ok = false;
      return nullptr;
    }
    const int d = t.get_device();
    if (device == -2) {
      device = d;
      if (d != c10::cuda::current_device()) ok = false;
    }
    if (d != device) ok = false;
    return ok ? &t : nullptr;
  }
  bool none() { return next() == Py_None; }
  bool flag() {
    const int r = PyObject_IsTrue(next());
    if (r < 0) {
      PyErr_Clear();
      ok = false;
    }
    return r > 0;
  }
  float number() {
    const double d = PyFloat_AsDouble(next());
    if (d == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return float(d);
  }
  // Whether all arguments were as asked for, and there are no more.
  bool fine() const { return ok && at == n; }
  // Fails the call unless `c`.
  bool want(bool c) {
    ok = ok && c;
    return ok;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device)).stream(); }
};

// Type and dimensions of a tensor that is there.
bool is(const at::Tensor* t, at::ScalarType type, int64_t dims) { return t->scalar_type() == type && t->dim() == dims; }
template <typename T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
int32_t* status_of(Args& a, const at::Tensor* t) {
  if (t) a.want(t->scalar_type() == at::kInt && t->numel() >= 1);
  return a.ok ? data<int32_t>(t) : nullptr;
}

// kv_cache, block_table, cu_rows and seq_lens, which come next.
void take_batch(Args& a, smla_paged_batch& b) {
  const at::Tensor *kv = a.tensor(), *table = a.tensor(), *cu = a.tensor(), *lens = a.tensor();
  if (!a.ok) return;
  if (!a.want(is(kv, at::kByte, 3) && is(table, at::kInt, 2) && is(cu, at::kInt, 1) && is(lens, at::kInt, 1))) return;
  b.n_pages = kv->size(0);
  const int64_t page = kv->size(1), seqs = table->size(0), pages = table->size(1);
  if (!a.want(kv->size(2) == SMLA_RECORD_BYTES && page < kMaxSize && seqs < kMaxSize && pages < kMaxSize &&
              lens->size(0) == seqs && cu->size(0) == seqs + 1))
    return;
  if (b.n_pages && page && !a.want(kv->stride(2) == 1 && (page == 1 || kv->stride(1) == SMLA_RECORD_BYTES))) return;
  if (seqs && !a.want((pages <= 1 || table->stride(1) == 1) && cu->stride(0) == 1 && (seqs == 1 || lens->stride(0) == 1)))
    return;
  b.kv_cache = kv->data_ptr();
  b.page_size = int32_t(page);
  b.page_stride = b.n_pages > 1 ? kv->stride(0) : page * SMLA_RECORD_BYTES;
  b.n_seqs = int32_t(seqs);
  b.max_pages = int32_t(pages);
  b.block_table = data<int32_t>(table);
  b.block_table_stride = seqs > 1 ? table->stride(0) : pages;
  b.cu_rows = data<int32_t>(cu);
  b.seq_lens = data<int32_t>(lens);
}

// latent and rope, which come next: rows, strides and type.
struct Rows {
  void *latent = nullptr, *rope = nullptr;
  int64_t n = 0, latent_stride = SMLA_LATENT_DIM, rope_stride = SMLA_ROPE_DIM;
  at::ScalarType type = at::kFloat;
  int32_t dtype = SMLA_DTYPE_F32;
};
void take_rows(Args& a, Rows& r) {
  const at::Tensor *lat = a.tensor(), *rope = a.tensor();
  if (!a.ok) return;
  r.type = lat->scalar_type();
  if (!a.want(r.type == at::kBFloat16 || r.type == at::kHalf || r.type == at::kFloat)) return;
  if (!a.want(lat->dim() == 2 && is(rope, r.type, 2))) return;
  r.n = lat->size(0);
  if (!a.want(lat->size(1) == SMLA_LATENT_DIM && rope->size(0) == r.n && rope->size(1) == SMLA_ROPE_DIM)) return;
  if (r.n && !a.want(lat->stride(1) == 1 && rope->stride(1) == 1)) return;
  if (r.n > 1) r.latent_stride = lat->stride(0), r.rope_stride = rope->stride(0);
  r.latent = lat->data_ptr();
  r.rope = rope->data_ptr();
  r.dtype = r.type == at::kBFloat16 ? SMLA_DTYPE_BF16 : r.type == at::kHalf ? SMLA_DTYPE_F16 : SMLA_DTYPE_F32;
}

// Row and head strides of [n, heads, dims].
bool take_heads(const at::Tensor* t, at::ScalarType type, int64_t n, int64_t heads, int64_t dims, int64_t* row, int64_t* head) {
  if (!is(t, type, 3) || t->size(0) != n || t->size(1) != heads || t->size(2) != dims) return false;
  if (n && heads && t->stride(2) != 1) return false;
  *head = heads > 1 ? t->stride(1) : dims;
  *row = n > 1 ? t->stride(0) : heads * *head;
  return true;
}

// Row stride and words of mask [n, words].
bool take_mask(const at::Tensor* t, int64_t n, int64_t* stride, int32_t* words) {
  if (!is(t, at::kInt, 2) || t->size(0) != n || t->size(1) >= kMaxSize) return false;
  *words = int32_t(t->size(1));
  if (n && *words > 1 && t->stride(1) != 1) return false;
  *stride = n > 1 ? t->stride(0) : *words;
  return true;
}

bool vector_of(const at::Tensor* t, at::ScalarType type, int64_t n) {
  return is(t, type, 1) && t->size(0) == n && (n <= 1 || t->stride(0) == 1);
}

// Lets the other Python threads run while a call is made (a launch may wait for room in its queue, an
// allocation for the driver).  The arguments' properties are read before; the caller keeps them.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// What a call returns: the status of its C call, or that it is not for these functions.
constexpr int kNotTaken = 1;

template <int (*kCall)(Args&)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int rc = kNotTaken;
  try {
    Args a(args, n);
    rc = kCall(a);
  } catch (...) {  // (an allocation: the calls in Python raise it again)
  }
  return rc == SMLA_ERR_LAUNCH ? PyLong_FromLong(rc) : PyBool_FromLong(rc == SMLA_OK);
}

// write and read: kv, table, cu, lens, latent, rope, stream, status
template <bool kWrite>
int copy(Args& a) {
  smla_paged_batch b{};
  Rows r;
  take_batch(a, b);
  if (!a.ok) return kNotTaken;
  take_rows(a, r);
  a.want(a.none());
  b.status = status_of(a, a.tensor(true));
  if (!a.fine()) return kNotTaken;
  b.n_rows = r.n;
  const Unlocked unlocked;
  return kWrite ? smla_paged_write(&b, r.latent, r.latent_stride, r.rope, r.rope_stride, r.dtype, a.stream())
                : smla_paged_read(&b, r.latent, r.latent_stride, r.rope, r.rope_stride, r.dtype, a.stream());
}

// append: kv, table, cu, lens, latent, rope, turns, q_rope, q_out, positions, interleaved, rope_scale,
// stream, status
int append(Args& a) {
  smla_paged_append_params p{};
  Rows r;
  take_batch(a, p.batch);
  if (!a.ok) return kNotTaken;
  take_rows(a, r);
  const at::Tensor *turns = a.tensor(), *q = a.tensor(true), *out = a.tensor(true), *pos = a.tensor(true);
  p.interleaved = a.flag();
  p.rope_scale = a.number();
  a.want(a.none());
  p.batch.status = status_of(a, a.tensor(true));
  if (!a.fine() || !vector_of(turns, at::kLong, SMLA_ROPE_DIM / 2) || (q == nullptr) != (out == nullptr)) return kNotTaken;
  if (pos && !vector_of(pos, at::kInt, r.n)) return kNotTaken;
  if (q) {
    if (q->dim() != 3 || q->size(1) >= kMaxSize) return kNotTaken;
    const int64_t heads = q->size(1);
    if (!take_heads(q, r.type, r.n, heads, SMLA_ROPE_DIM, &p.q_rope_stride_row, &p.q_rope_stride_head) ||
        !take_heads(out, at::kBFloat16, r.n, heads, SMLA_ROPE_DIM, &p.q_out_stride_row, &p.q_out_stride_head))
      return kNotTaken;
    p.num_heads = int32_t(heads);
    p.q_rope = q->data_ptr();
    p.q_out = out->data_ptr();
  }
  p.batch.n_rows = r.n;
  p.latent = r.latent;
  p.latent_stride = r.latent_stride;
  p.rope = r.rope;
  p.rope_stride = r.rope_stride;
  p.dtype = r.dtype;
  p.turns = static_cast<const uint64_t*>(turns->data_ptr());
  p.positions = data<int32_t>(pos);
  const Unlocked unlocked;
  return smla_paged_append(&p, a.stream());
}

// tree: parents, cu, lens, mask, positions, stream, status
int tree(Args& a) {
  const at::Tensor *parents = a.tensor(), *cu = a.tensor(), *lens = a.tensor(), *mask = a.tensor(true), *pos = a.tensor(true);
  a.want(a.none());
  int32_t* status = status_of(a, a.tensor(true));
  if (!a.fine() || parents->dim() != 1 || lens->dim() != 1) return kNotTaken;
  const int64_t n = parents->size(0), seqs = lens->size(0);
  if (seqs >= kMaxSize || !vector_of(parents, at::kInt, n) || !vector_of(lens, at::kInt, seqs) ||
      !vector_of(cu, at::kInt, seqs + 1) || (pos && !vector_of(pos, at::kInt, n)))
    return kNotTaken;
  int64_t stride = 0;
  int32_t words = 0;
  if (mask && !take_mask(mask, n, &stride, &words)) return kNotTaken;
  const Unlocked unlocked;
  return smla_paged_tree(data<int32_t>(parents), data<int32_t>(cu), data<int32_t>(lens), n, int32_t(seqs),
                         data<uint32_t>(mask), stride, words, data<int32_t>(pos), status, a.stream());
}

// attend and attend_tree: kv, table, cu, lens, q, sm_scale, sink, out, lse, causal, stream, status,
// workspace, mask (None: attend)
int attend(Args& a) {
  smla_paged_attend_params p{};
  take_batch(a, p.batch);
  if (!a.ok) return kNotTaken;
  const at::Tensor* q = a.tensor();
  p.sm_scale = a.number();
  const at::Tensor *sink = a.tensor(true), *out = a.tensor(), *lse = a.tensor(true);
  p.causal = a.flag();
  a.want(a.none());
  p.batch.status = status_of(a, a.tensor(true));
  const at::Tensor *given = a.tensor(true), *mask = a.tensor(true);
  if (!a.fine() || q->dim() != 3 || q->size(1) >= kMaxSize) return kNotTaken;
  const int64_t n = q->size(0), heads = q->size(1);
  if (!take_heads(q, at::kBFloat16, n, heads, SMLA_QK_DIM, &p.q_stride_row, &p.q_stride_head) ||
      !take_heads(out, at::kBFloat16, n, heads, SMLA_LATENT_DIM, &p.out_stride_row, &p.out_stride_head))
    return kNotTaken;
  if (sink && !vector_of(sink, at::kFloat, heads)) return kNotTaken;
  if (lse && !(is(lse, at::kFloat, 2) && lse->size(0) == n && lse->size(1) == heads && lse->is_contiguous())) return kNotTaken;
  if (given && !given->is_contiguous()) return kNotTaken;
  int64_t mask_stride = 0;
  int32_t words = 0;
  if (mask && !take_mask(mask, n, &mask_stride, &words)) return kNotTaken;
  p.batch.n_rows = n;
  p.num_heads = int32_t(heads);
  p.q = q->data_ptr();
  p.sink = data<float>(sink);
  p.out = out->data_ptr();
  p.lse = data<float>(lse);
  // without a workspace a block of this call's own, on its stream: calls on other streams and
  // other captured graphs never share it
  const Unlocked unlocked;
  at::Tensor own;
  void* workspace = given ? given->data_ptr() : nullptr;
  size_t bytes = given ? given->nbytes() : 0;
  if (!given) {
    bytes = smla_paged_attend_workspace_size(&p);
    if (bytes) {
      own = at::empty({int64_t(bytes)}, q->options().dtype(at::kByte));
      workspace = own.data_ptr();
    }
  }
  return mask ? smla_paged_attend_tree(&p, data<uint32_t>(mask), mask_stride, words, workspace, bytes, a.stream())
              : smla_paged_attend(&p, workspace, bytes, a.stream());
}

// accept: kv, table, cu, lens, path, new_lens, n_rows, stream, status
int accept(Args& a) {
  smla_paged_batch b{};
  take_batch(a, b);
  const at::Tensor *path = a.tensor(), *lens = a.tensor();
  b.n_rows = PyLong_AsLongLong(a.next());
  if (b.n_rows == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return kNotTaken;
  }
  a.want(a.none());
  b.status = status_of(a, a.tensor(true));
  if (!a.fine() || !is(path, at::kInt, 2) || path->size(0) != b.n_seqs || path->size(1) >= kMaxSize ||
      !vector_of(lens, at::kInt, b.n_seqs))
    return kNotTaken;
  const int64_t width = path->size(1);
  if (b.n_seqs && width > 1 && path->stride(1) != 1) return kNotTaken;
  const Unlocked unlocked;
  return smla_paged_accept(&b, data<int32_t>(path), b.n_seqs > 1 ? path->stride(0) : width, int32_t(width),
                           data<int32_t>(lens), a.stream());
}

template <int (*kCall)(Args&)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<kCall>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<copy<true>>("write"), method<copy<false>>("read"), method<append>("append"),
                           method<tree>("tree"),        method<attend>("attend"),    method<accept>("accept"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_smla", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__smla() { return PyModule_Create(&g_module); }
