// binding.cpp -- the Python side of the operators that use the selection:
// checks of the tensors, outputs, the structures of include/mm3idx.h, one
// library call each.  A small batch's kernel takes 5 to 10 us, and a whole call
// in Python, one attribute at a time, took 9 us for paged attention, 15 for
// verification and 26 for eviction on the card's host; here 3, 5 and 7.
// Nothing is computed and nothing is kept between calls.
//
// Arguments are positional (the package's functions have the names and
// defaults); None stands for an argument that was not given.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>

#include "../../include/mm3idx.h"

namespace {

PyObject* g_error = nullptr;   // Mm3idxError(status, what)

// A Python exception is set.
struct Raised : std::exception {};

[[noreturn]] void refuse(const char* why) {
  PyErr_SetString(PyExc_ValueError, why);
  throw Raised();
}
void need(bool ok, const char* why) {
  if (!ok) refuse(why);
}

void check(int status, const char* what) {
  if (status == MM3IDX_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", status, what);
  if (e) {
    PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
    Py_DECREF(e);
  }
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw Raised();
  }
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}
int32_t integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument outside the 32-bit integers");
    throw Raised();
  }
  return static_cast<int32_t>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

int64_t blocks_of(int64_t tokens) { return (tokens + 127) / 128; }
// Elements between the rows of a matrix (free when it has one row).
int64_t row_stride(const at::Tensor& t) {
  return t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.size(1), 1);
}
bool unit_inner(const at::Tensor& t) { return t.size(t.dim() - 1) <= 1 || t.stride(t.dim() - 1) == 1; }
bool is(const at::Tensor& t, at::ScalarType type, int64_t dims) {
  return t.scalar_type() == type && t.dim() == dims;
}
bool shaped(const at::Tensor& t, std::initializer_list<int64_t> sizes) {
  return t.sizes() == at::IntArrayRef(sizes.begin(), sizes.size());
}
void same_gpu(const at::Tensor& ref, std::initializer_list<const at::Tensor*> others) {
  bool ok = ref.is_cuda();
  for (const at::Tensor* t : others) ok = ok && (!t || t->device() == ref.device());
  need(ok, "all inputs must be on the same GPU");
}
at::Tensor make(const at::Tensor& like, at::ScalarType type, std::initializer_list<int64_t> sizes) {
  return at::empty(at::IntArrayRef(sizes.begin(), sizes.size()), like.options().dtype(type));
}
// Several outputs of a call in one allocation, 256 bytes apart: an allocation
// costs the host 0.6 us, a tensor on a part of one a tenth of that.
template <int N>
class Outputs {
 public:
  void add(int k, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    int64_t count = 1;
    for (const int64_t x : sizes) count *= x;
    parts_[k] = Part{type, at::DimVector(sizes.begin(), sizes.end()), bytes_};
    bytes_ += (count * static_cast<int64_t>(c10::elementSize(type)) + 255) & ~int64_t{255};
  }
  void allocate(const at::Tensor& like, at::Tensor* out) {
    const at::Tensor base = at::empty({bytes_}, like.options().dtype(at::kByte));
    for (int k = 0; k < N; ++k) {
      const Part& p = parts_[k];
      if (p.offset < 0) continue;
      out[k] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(),
                                                        c10::scalarTypeToTypeMeta(p.type));
      c10::TensorImpl* t = out[k].unsafeGetTensorImpl();
      t->set_sizes_contiguous(p.sizes);
      t->set_storage_offset(p.offset / static_cast<int64_t>(c10::elementSize(p.type)));
    }
  }

 private:
  struct Part {
    at::ScalarType type = at::kByte;
    at::DimVector sizes;
    int64_t offset = -1;
  };
  Part parts_[N];
  int64_t bytes_ = 0;
};
void* stream_of(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}
int32_t type_of(at::ScalarType t) {
  return t == at::kBFloat16 ? MM3IDX_TYPE_BF16 : t == at::kHalf ? MM3IDX_TYPE_FP16
         : t == at::kFloat ? MM3IDX_TYPE_FP32 : MM3IDX_TYPE_E4M3;
}

PyObject* paged_attention(PyObject* const* args) {
  const at::Tensor &q = tensor(args[0], "q"), &k = tensor(args[1], "k_cache"),
                   &v = tensor(args[2], "v_cache"), &table = tensor(args[3], "page_table"),
                   &lens = tensor(args[4], "seq_lens");
  const int32_t query_len = integer(args[5]), max_seq_len = integer(args[6]);
  const at::Tensor *given = maybe(args[10], "out"), *lse = maybe(args[11], "lse"),
                   *weights = maybe(args[12], "block_weights");
  const at::ScalarType type = q.scalar_type(), kv = k.scalar_type();
  need(q.dim() == 3 && (type == at::kBFloat16 || type == at::kHalf) && unit_inner(q),
       "queries must be bf16 or fp16 [tokens, heads, head_dim] with contiguous head_dim");
  const int64_t rows = q.size(0), heads = q.size(1), dim = q.size(2);
  need(k.dim() == 4 && k.sizes() == v.sizes() && kv == v.scalar_type() &&
           (kv == type || kv == at::kFloat8_e4m3fn) && k.size(3) == dim && unit_inner(k) &&
           unit_inner(v),
       "caches must be [pages, page_size, kv_heads, head_dim] with contiguous head_dim, of the "
       "queries' type or float8_e4m3fn");
  need(is(table, at::kInt, 2) && unit_inner(table) && is(lens, at::kInt, 1) && lens.is_contiguous(),
       "page table and lengths must be int32 with unit stride");
  same_gpu(q, {&k, &v, &table, &lens});
  const int64_t reqs = lens.size(0);
  need(rows == reqs * query_len && table.size(0) == reqs,
       "queries must have batch * query_len rows and the page table one row per request");
  need(!given || (given->sizes() == q.sizes() && given->scalar_type() == type &&
                  given->device() == q.device() && unit_inner(*given)),
       "out must be like the queries");
  need(!lse || (is(*lse, at::kFloat, 2) && lse->size(0) >= rows && lse->size(1) == heads &&
                unit_inner(*lse) && lse->device() == q.device()),
       "lse must be fp32 [>= rows, heads] with unit inner stride");
  need(!weights || (is(*weights, at::kFloat, 2) && weights->size(0) >= rows &&
                    weights->size(1) >= blocks_of(max_seq_len) && unit_inner(*weights) &&
                    weights->device() == q.device()),
       "block_weights must be fp32 [>= rows, >= cdiv(max_seq_len, 128)] with unit inner stride");
  const c10::cuda::CUDAGuard guard(q.device());
  at::Tensor out = given ? *given : make(q, type, {rows, heads, dim});

  mm3idx_attention_t a{};
  const int64_t pages = k.size(0), size = k.size(1), kv_heads = k.size(2);
  // strides of dimensions of one are free
  a.q = q.data_ptr();
  a.q_token_stride = rows > 1 ? q.stride(0) : heads * dim;
  a.q_head_stride = heads > 1 ? q.stride(1) : dim;
  a.q_heads = static_cast<int32_t>(heads);
  a.kv_heads = static_cast<int32_t>(kv_heads);
  a.head_dim = static_cast<int32_t>(dim);
  a.q_type = type_of(type);
  a.kv_type = type_of(kv);
  a.k_cache = k.data_ptr();
  a.k_page_stride = pages > 1 ? k.stride(0) : size * kv_heads * dim;
  a.k_token_stride = size > 1 ? k.stride(1) : kv_heads * dim;
  a.k_head_stride = kv_heads > 1 ? k.stride(2) : dim;
  a.v_cache = v.data_ptr();
  a.v_page_stride = pages > 1 ? v.stride(0) : size * kv_heads * dim;
  a.v_token_stride = size > 1 ? v.stride(1) : kv_heads * dim;
  a.v_head_stride = kv_heads > 1 ? v.stride(2) : dim;
  a.sm_scale = static_cast<float>(number(args[7]));
  a.k_scale = static_cast<float>(number(args[8]));
  a.v_scale = static_cast<float>(number(args[9]));
  need(pages <= INT32_MAX, "more pages than 32 bits count");
  a.num_pages = static_cast<int32_t>(pages);
  a.page_size = static_cast<int32_t>(size);
  a.page_table = static_cast<const int32_t*>(table.data_ptr());
  a.table_stride = row_stride(table);
  a.table_width = static_cast<int32_t>(table.size(1));
  a.seq_lens = static_cast<const int32_t*>(lens.data_ptr());
  a.num_reqs = static_cast<int32_t>(reqs);
  a.query_len = query_len;
  a.max_seq_len = max_seq_len;
  a.out = out.data_ptr();
  a.out_token_stride = rows > 1 ? out.stride(0) : heads * dim;
  a.out_head_stride = heads > 1 ? out.stride(1) : dim;
  if (lse) {
    a.lse = static_cast<float*>(lse->data_ptr());
    a.lse_token_stride = row_stride(*lse);
  }
  if (weights) {
    a.block_weights = static_cast<float*>(weights->data_ptr());
    a.block_weights_stride = row_stride(*weights);
  }
  at::Tensor workspace;
  if (args[13] == Py_None) {
    size_t bytes = 0;
    check(mm3idx_attention_workspace_bytes(a.q_heads, a.kv_heads, a.head_dim, a.num_reqs, query_len,
                                           max_seq_len, weights ? 1 : 0, &bytes),
          "mm3idx_attention_workspace_bytes");
    workspace = at::zeros({static_cast<int64_t>(std::max<size_t>(bytes, 256))},
                          q.options().dtype(at::kByte));
  } else {
    workspace = tensor(args[13], "workspace");
    need(workspace.device() == q.device() && workspace.is_contiguous(),
         "workspace must be a contiguous tensor on the inputs' GPU");
  }
  check(mm3idx_paged_attention(&a, workspace.data_ptr(), workspace.nbytes(), stream_of(q)),
        "mm3idx_paged_attention");
  return THPVariable_Wrap(std::move(out));
}

// The checks of mm3idx_weights_t.
mm3idx_weights_t weights_of(const at::Tensor& acc, const at::Tensor& lens, const at::Tensor* w,
                            const at::Tensor* ids, int32_t query_len, int32_t max_seq_len,
                            double decay) {
  const int64_t width = blocks_of(max_seq_len);
  need(is(lens, at::kInt, 1) && lens.is_contiguous(), "lengths must be contiguous int32");
  const int64_t reqs = lens.size(0);
  need(is(acc, at::kFloat, 2) && acc.size(0) == reqs && acc.size(1) >= width && unit_inner(acc),
       "weights must be fp32 [num_reqs, >= cdiv(max_seq_len, 128)] with unit inner stride");
  same_gpu(acc, {&lens, w, ids});
  mm3idx_weights_t a{};
  a.acc = static_cast<float*>(acc.data_ptr());
  a.acc_stride = row_stride(acc);
  a.seq_lens = static_cast<const int32_t*>(lens.data_ptr());
  a.num_reqs = static_cast<int32_t>(reqs);
  a.query_len = query_len;
  a.max_seq_len = max_seq_len;
  a.decay = decay;
  if (w) {
    need(is(*w, at::kFloat, 2) && w->size(0) >= reqs * query_len && unit_inner(*w) &&
             w->size(1) >= (ids ? ids->size(ids->dim() - 1) : width),
         "block_weights must be fp32 [>= num_reqs * query_len, a column per block or id] with unit "
         "inner stride");
    a.block_weights = static_cast<const float*>(w->data_ptr());
    a.weights_stride = row_stride(*w);
  }
  if (ids) {
    // [rows, topk], or [1, rows, topk] as decode returns the ids of one head
    const int64_t d = ids->dim();
    need(w && ids->scalar_type() == at::kInt && (d == 2 || (d == 3 && ids->size(0) == 1)) &&
             ids->size(d - 2) >= reqs * query_len && unit_inner(*ids),
         "ids must be int32 [>= num_reqs * query_len, topk] of one index head with unit inner "
         "stride, with their block_weights");
    a.ids = static_cast<const int32_t*>(ids->data_ptr());
    a.topk = static_cast<int32_t>(ids->size(d - 1));
    a.ids_stride = ids->size(d - 2) > 1 ? ids->stride(d - 2) : std::max<int32_t>(a.topk, 1);
  }
  return a;
}

PyObject* accumulate_weights(PyObject* const* args) {
  const at::Tensor& acc = tensor(args[0], "acc");
  const mm3idx_weights_t w =
      weights_of(acc, tensor(args[2], "seq_lens"), maybe(args[1], "block_weights"),
                 maybe(args[3], "ids"), integer(args[4]), integer(args[5]), number(args[6]));
  const c10::cuda::CUDAGuard guard(acc.device());
  check(mm3idx_accumulate_weights(&w, stream_of(acc)), "mm3idx_accumulate_weights");
  Py_RETURN_NONE;
}

// (ids, seq_lens, weights, block_table, freed, attention table, its freed)
PyObject* evict_blocks(PyObject* const* args) {
  const at::Tensor &acc = tensor(args[0], "acc"), &lens = tensor(args[1], "seq_lens"),
                   &table = tensor(args[2], "block_table");
  const at::Tensor* second = maybe(args[3], "attention_block_table");
  const int32_t budget = integer(args[6]), max_seq_len = integer(args[9]);
  const bool in_place = truth(args[12]);
  mm3idx_weights_t w = weights_of(acc, lens, maybe(args[4], "block_weights"), maybe(args[5], "ids"),
                                  integer(args[10]), max_seq_len, number(args[11]));
  const int64_t width = blocks_of(max_seq_len), reqs = lens.size(0);
  const int64_t gone = std::max<int64_t>(1, width - budget);
  need(budget >= 1, "budget must be at least 1");
  for (const at::Tensor* t : {&table, second}) {
    if (!t) continue;
    need(is(*t, at::kInt, 2) && t->size(0) == reqs && t->size(1) >= width && unit_inner(*t) &&
             t->device() == acc.device(),
         "block tables must be int32 [num_reqs, >= cdiv(max_seq_len, 128)] with unit inner stride, "
         "on the weights' GPU");
    need(!in_place || t->size(1) >= budget, "in-place tables must have at least budget columns");
  }
  const c10::cuda::CUDAGuard guard(acc.device());
  at::Tensor out[7];      // in the order of the result
  const int64_t columns[7] = {budget, 0, width, budget, gone, budget, gone};
  if (args[13] != Py_None) {
    need(!in_place, "out and in_place exclude each other");
    need(PyTuple_Check(args[13]) && PyTuple_GET_SIZE(args[13]) == 7, "out must be an Eviction");
    for (int k = 0; k < 7; ++k) {
      PyObject* o = PyTuple_GET_ITEM(args[13], k);
      need((o == Py_None) == (k >= 5 && !second), "out must be an Eviction of these shapes");
      if (o == Py_None) continue;
      out[k] = tensor(o, "out");
      const at::Tensor& t = out[k];
      need(t.device() == acc.device() && t.scalar_type() == (k == 2 ? at::kFloat : at::kInt) &&
               (k == 1 ? t.sizes() == lens.sizes() && t.is_contiguous()
                       : t.dim() == 2 && t.size(0) == reqs && t.size(1) >= columns[k] &&
                             unit_inner(t)),
           "out must be an Eviction of these shapes");
    }
  } else {
    Outputs<7> made;
    for (int k = 0; k < 7; ++k) {
      if (k >= 5 && !second) continue;
      if (in_place && (k == 1 || k == 2 || k == 3 || k == 5))
        out[k] = k == 1 ? lens : k == 2 ? acc : k == 3 ? table : *second;
      else if (k == 1) made.add(k, at::kInt, {reqs});
      else made.add(k, k == 2 ? at::kFloat : at::kInt, {reqs, columns[k]});
    }
    made.allocate(acc, out);
  }
  mm3idx_eviction_t e{};
  e.budget = budget;
  e.init_blocks = integer(args[7]);
  e.local_blocks = integer(args[8]);
  for (int k = 0; k < 2; ++k) {
    const at::Tensor* from = k ? second : &table;
    if (!from) continue;
    const at::Tensor &to = out[k ? 5 : 3], &freed = out[k ? 6 : 4];
    e.tables[k] = mm3idx_evict_table_t{
        static_cast<const int32_t*>(from->data_ptr()), row_stride(*from),
        static_cast<int32_t*>(to.data_ptr()), row_stride(to),
        static_cast<int32_t*>(freed.data_ptr()), row_stride(freed)};
  }
  e.ids = static_cast<int32_t*>(out[0].data_ptr());
  e.ids_stride = row_stride(out[0]);
  e.acc_out = static_cast<float*>(out[2].data_ptr());
  e.acc_out_stride = row_stride(out[2]);
  e.seq_lens_out = static_cast<int32_t*>(out[1].data_ptr());
  check(mm3idx_evict_blocks(&w, &e, stream_of(acc)), "mm3idx_evict_blocks");
  PyObject* result = PyTuple_New(7);
  if (!result) throw Raised();
  for (int k = 0; k < 7; ++k) {
    PyObject* o = out[k].defined() ? THPVariable_Wrap(std::move(out[k])) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(result);
      throw Raised();
    }
    PyTuple_SET_ITEM(result, k, o);
  }
  return result;
}

// (tokens, accepted)
PyObject* verify_drafts(PyObject* const* args) {
  const at::Tensor &target = tensor(args[0], "target_probs"), &tokens = tensor(args[1], "draft_tokens"),
                   &u = tensor(args[2], "uniforms");
  const at::Tensor *draft = maybe(args[3], "draft_probs"), *lens = maybe(args[4], "draft_lens"),
                   *out_given = maybe(args[5], "out"), *acc_given = maybe(args[6], "accepted");
  const at::ScalarType type = target.scalar_type();
  need(target.dim() == 3 && (type == at::kFloat || type == at::kBFloat16 || type == at::kHalf) &&
           unit_inner(target) && target.size(1) >= 1,
       "target_probs must be fp32, bf16 or fp16 [num_reqs, drafts + 1, vocab] with contiguous vocab");
  const int64_t reqs = target.size(0), rows = target.size(1), vocab = target.size(2), k = rows - 1;
  need(vocab <= INT32_MAX, "more tokens than 32 bits count");
  need(is(tokens, at::kInt, 2) && shaped(tokens, {reqs, k}) && unit_inner(tokens),
       "draft_tokens must be int32 [num_reqs, drafts] with unit inner stride");
  need(is(u, at::kFloat, 2) && shaped(u, {reqs, rows}) && unit_inner(u),
       "uniforms must be fp32 [num_reqs, drafts + 1] with unit inner stride");
  need(!draft || (draft->scalar_type() == type && shaped(*draft, {reqs, k, vocab}) && unit_inner(*draft)),
       "draft_probs must be [num_reqs, drafts, vocab] of target_probs' type with contiguous vocab");
  need(!lens || (is(*lens, at::kInt, 1) && lens->is_contiguous() && lens->size(0) == reqs),
       "draft_lens must be contiguous int32 [num_reqs]");
  same_gpu(target, {&tokens, &u, draft, lens, out_given, acc_given});
  const c10::cuda::CUDAGuard guard(target.device());
  at::Tensor results[2];
  Outputs<2> made;
  if (out_given) results[0] = *out_given;
  else made.add(0, at::kInt, {reqs, rows});
  if (acc_given) results[1] = *acc_given;
  else made.add(1, at::kInt, {reqs});
  if (!out_given || !acc_given) made.allocate(target, results);
  at::Tensor &out = results[0], &accepted = results[1];
  need(is(out, at::kInt, 2) && shaped(out, {reqs, rows}) && unit_inner(out) &&
           is(accepted, at::kInt, 1) && accepted.size(0) == reqs && accepted.is_contiguous(),
       "out must be int32 [num_reqs, drafts + 1] with unit inner stride, accepted int32 [num_reqs]");
  mm3idx_drafts_t d{};
  d.target = target.data_ptr();
  d.target_req_stride = target.stride(0);
  d.target_row_stride = target.stride(1);
  if (draft) {
    d.draft = draft->data_ptr();
    d.draft_req_stride = draft->stride(0);
    d.draft_row_stride = draft->stride(1);
  }
  d.type = type_of(type);
  d.tokens = static_cast<const int32_t*>(tokens.data_ptr());
  d.tokens_stride = row_stride(tokens);
  d.draft_lens = lens ? static_cast<const int32_t*>(lens->data_ptr()) : nullptr;
  d.uniforms = static_cast<const float*>(u.data_ptr());
  d.uniforms_stride = row_stride(u);
  d.num_reqs = static_cast<int32_t>(reqs);
  d.drafts = static_cast<int32_t>(k);
  d.vocab = static_cast<int32_t>(vocab);
  d.out = static_cast<int32_t*>(out.data_ptr());
  d.out_stride = row_stride(out);
  d.accepted = static_cast<int32_t*>(accepted.data_ptr());
  check(mm3idx_verify_drafts(&d, stream_of(target)), "mm3idx_verify_drafts");
  PyObject* a = THPVariable_Wrap(std::move(out));
  PyObject* b = a ? THPVariable_Wrap(std::move(accepted)) : nullptr;
  PyObject* result = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  if (!result) throw Raised();
  return result;
}

// Every exception becomes Python's; `N` positional arguments.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"set_error", set_error, METH_O, nullptr},
    {"paged_attention", fast(entry<paged_attention, 14>), METH_FASTCALL, nullptr},
    {"accumulate_weights", fast(entry<accumulate_weights, 7>), METH_FASTCALL, nullptr},
    {"evict_blocks", fast(entry<evict_blocks, 14>), METH_FASTCALL, nullptr},
    {"verify_drafts", fast(entry<verify_drafts, 7>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
