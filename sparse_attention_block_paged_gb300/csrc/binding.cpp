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

// Scales of an e4m3 cache's pages: none, or both.
bool scales_of(PyObject* ko, PyObject* vo, const at::Tensor& cache, mm3idx_kv_scales_t* out) {
  const at::Tensor *k = maybe(ko, "k_scales"), *v = maybe(vo, "v_scales");
  if (!k && !v) return false;
  need(k && v && cache.scalar_type() == at::kFloat8_e4m3fn,
       "k_scales and v_scales go together, with float8_e4m3fn caches");
  for (const at::Tensor* t : {k, v})
    need(is(*t, at::kFloat, 2) && t->size(0) == cache.size(0) && t->size(1) == cache.size(2) &&
             t->device() == cache.device(),
         "k_scales and v_scales must be fp32 [pages, kv_heads] on the caches' GPU");
  *out = mm3idx_kv_scales_t{static_cast<float*>(k->data_ptr()), k->stride(0), k->stride(1),
                            static_cast<float*>(v->data_ptr()), v->stride(0), v->stride(1)};
  return true;
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
  mm3idx_kv_scales_t scales{};
  if (scales_of(args[14], args[15], k, &scales))
    check(mm3idx_paged_attention_scaled(&a, &scales, workspace.data_ptr(), workspace.nbytes(),
                                        stream_of(q)),
          "mm3idx_paged_attention_scaled");
  else
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

PyObject* append_kv(PyObject* const* args) {
  const at::Tensor &k = tensor(args[0], "k"), &v = tensor(args[1], "v"),
                   &kc = tensor(args[2], "k_cache"), &vc = tensor(args[3], "v_cache"),
                   &table = tensor(args[4], "page_table"), &lens = tensor(args[5], "seq_lens");
  const int32_t query_len = integer(args[6]), max_seq_len = integer(args[7]);
  const at::Tensor* cu = maybe(args[12], "cu_seqlens_q");
  const at::ScalarType type = k.scalar_type(), kv = kc.scalar_type();
  need(k.dim() == 3 && (type == at::kBFloat16 || type == at::kHalf) && v.scalar_type() == type &&
           k.sizes() == v.sizes() && unit_inner(k) && unit_inner(v),
       "new keys and values must be bf16 or fp16 [tokens, kv_heads, head_dim] with contiguous "
       "head_dim");
  const int64_t rows = k.size(0), heads = k.size(1), dim = k.size(2);
  need(kc.dim() == 4 && kc.sizes() == vc.sizes() && kv == vc.scalar_type() &&
           (kv == type || kv == at::kFloat8_e4m3fn) && kc.size(2) == heads && kc.size(3) == dim &&
           unit_inner(kc) && unit_inner(vc),
       "caches must be [pages, page_size, kv_heads, head_dim] with contiguous head_dim, of the new "
       "tokens' type or float8_e4m3fn");
  need(is(table, at::kInt, 2) && unit_inner(table) && is(lens, at::kInt, 1) && lens.is_contiguous(),
       "page table and lengths must be int32 with unit stride");
  same_gpu(k, {&v, &kc, &vc, &table, &lens, cu});
  const int64_t reqs = lens.size(0);
  need(table.size(0) == reqs, "the page table must have one row per request");
  need(!cu || (is(*cu, at::kInt, 1) && cu->size(0) == reqs + 1 && cu->is_contiguous()),
       "cu_seqlens_q must be contiguous int32 [num_reqs + 1]");
  need(cu ? rows <= reqs * query_len : rows == reqs * query_len,
       cu ? "more new tokens than num_reqs * query_len"
          : "new keys and values must have batch * query_len rows");
  const int64_t pages = kc.size(0), size = kc.size(1);
  need(pages <= INT32_MAX, "more pages than 32 bits count");
  const c10::cuda::CUDAGuard guard(k.device());
  mm3idx_append_t a{};
  a.k = k.data_ptr();
  a.k_token_stride = rows > 1 ? k.stride(0) : heads * dim;
  a.k_head_stride = heads > 1 ? k.stride(1) : dim;
  a.v = v.data_ptr();
  a.v_token_stride = rows > 1 ? v.stride(0) : heads * dim;
  a.v_head_stride = heads > 1 ? v.stride(1) : dim;
  a.type = type_of(type);
  a.kv_type = type_of(kv);
  a.kv_heads = static_cast<int32_t>(heads);
  a.head_dim = static_cast<int32_t>(dim);
  a.k_cache = kc.data_ptr();
  a.k_page_stride = pages > 1 ? kc.stride(0) : size * heads * dim;
  a.k_page_token_stride = size > 1 ? kc.stride(1) : heads * dim;
  a.k_page_head_stride = heads > 1 ? kc.stride(2) : dim;
  a.v_cache = vc.data_ptr();
  a.v_page_stride = pages > 1 ? vc.stride(0) : size * heads * dim;
  a.v_page_token_stride = size > 1 ? vc.stride(1) : heads * dim;
  a.v_page_head_stride = heads > 1 ? vc.stride(2) : dim;
  a.k_scale = static_cast<float>(number(args[8]));
  a.v_scale = static_cast<float>(number(args[9]));
  scales_of(args[10], args[11], kc, &a.scales);
  a.num_pages = static_cast<int32_t>(pages);
  a.page_size = static_cast<int32_t>(size);
  a.page_table = static_cast<const int32_t*>(table.data_ptr());
  a.table_stride = row_stride(table);
  a.table_width = static_cast<int32_t>(table.size(1));
  a.seq_lens = static_cast<const int32_t*>(lens.data_ptr());
  a.num_reqs = static_cast<int32_t>(reqs);
  a.query_len = query_len;
  a.max_seq_len = max_seq_len;
  a.cu_seqlens_q = cu ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr;
  a.total_q = static_cast<int32_t>(rows);
  check(mm3idx_append_kv(&a, stream_of(k)), "mm3idx_append_kv");
  Py_RETURN_NONE;
}

// The checks of mm3idx_pool_t.
mm3idx_pool_t pool_of(const at::Tensor& refs, const at::Tensor& table, const at::Tensor* lens,
                      int32_t page_size) {
  need(is(refs, at::kInt, 1) && refs.is_contiguous() && refs.size(0) <= INT32_MAX,
       "reference counts must be contiguous int32 [num_pages]");
  need(is(table, at::kInt, 2) && unit_inner(table) && table.size(0) <= INT32_MAX &&
           table.size(1) <= INT32_MAX,
       "page tables must be int32 [num_reqs, columns] with unit inner stride");
  need(!lens || (is(*lens, at::kInt, 1) && lens->is_contiguous() && lens->size(0) == table.size(0)),
       "lengths must be contiguous int32, one per row of the page table");
  same_gpu(refs, {&table, lens});
  mm3idx_pool_t p{};
  p.refs = static_cast<int32_t*>(refs.data_ptr());
  p.num_pages = static_cast<int32_t>(refs.size(0));
  p.page_size = page_size;
  p.page_table = static_cast<int32_t*>(table.data_ptr());
  p.table_stride = row_stride(table);
  p.table_width = static_cast<int32_t>(table.size(1));
  p.seq_lens = lens ? static_cast<const int32_t*>(lens->data_ptr()) : nullptr;
  p.num_reqs = static_cast<int32_t>(table.size(0));
  return p;
}

// A sequence of caches: tensors whose first dimension is the page, the rest of a
// page without gaps, in any order.
struct Caches {
  mm3idx_cache_t at[MM3IDX_MAX_CACHES];
  int32_t count = 0, pages = 0;   // pages: of the first one
  Caches(PyObject* o, const at::Tensor& like, int64_t num_pages) {
    const bool list = PyList_Check(o) || PyTuple_Check(o);
    need(list, "caches must be a list or tuple of tensors");
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
    need(n <= MM3IDX_MAX_CACHES, "more caches than a call takes");
    for (Py_ssize_t k = 0; k < n; ++k) {
      const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(o, k), "caches");
      if (num_pages < 0) num_pages = t.dim() >= 1 ? t.size(0) : 0;
      need(t.dim() >= 1 && t.size(0) == num_pages && t.device() == like.device() &&
               t.layout() == at::kStrided && t.numel() > 0 && num_pages <= INT32_MAX,
           "caches must be tensors of the pool's number of pages on its GPU");
      const int64_t count_of_page = t.numel() / num_pages;
      int64_t dense = 1;                       // the dimensions of a page, innermost first
      for (;;) {
        int64_t d = 1;
        while (d < t.dim() && !(t.stride(d) == dense && t.size(d) > 1)) ++d;
        if (d == t.dim()) break;
        dense *= t.size(d);
      }
      need(dense == count_of_page && (num_pages == 1 || t.stride(0) >= count_of_page),
           "a cache's page must lie in memory without gaps, and pages must not overlap");
      const int64_t size = t.element_size();
      at[k] = mm3idx_cache_t{t.data_ptr(), (num_pages > 1 ? t.stride(0) : count_of_page) * size,
                             count_of_page * size};
      pages = static_cast<int32_t>(num_pages);
    }
    count = static_cast<int32_t>(n);
  }
};

at::Tensor pages_workspace(PyObject* given, const at::Tensor& refs, int32_t forks) {
  if (given == Py_None) {
    size_t bytes = 0;
    check(mm3idx_pages_workspace_bytes(static_cast<int32_t>(refs.size(0)), forks, &bytes),
          "mm3idx_pages_workspace_bytes");
    return at::empty({static_cast<int64_t>(bytes)}, refs.options().dtype(at::kByte));
  }
  const at::Tensor& t = tensor(given, "workspace");
  need(t.device() == refs.device() && t.is_contiguous(),
       "workspace must be a contiguous tensor on the inputs' GPU");
  return t;
}

PyObject* allocate_pages(PyObject* const* args) {
  const at::Tensor &refs = tensor(args[0], "refs"), &table = tensor(args[1], "page_table"),
                   &lens = tensor(args[2], "seq_lens");
  const mm3idx_pool_t p = pool_of(refs, table, &lens, integer(args[4]));
  const c10::cuda::CUDAGuard guard(refs.device());
  const at::Tensor ws = pages_workspace(args[5], refs, 0);
  check(mm3idx_allocate_pages(&p, integer(args[3]), ws.data_ptr(), ws.nbytes(), stream_of(refs)),
        "mm3idx_allocate_pages");
  Py_RETURN_NONE;
}

PyObject* release_pages(PyObject* const* args) {
  const at::Tensor &refs = tensor(args[0], "refs"), &table = tensor(args[1], "page_table");
  const at::Tensor* lens = maybe(args[2], "seq_lens");
  need((args[3] == Py_None) == !lens, "seq_lens and page_size go together");
  const mm3idx_pool_t p = pool_of(refs, table, lens, lens ? integer(args[3]) : 1);
  const c10::cuda::CUDAGuard guard(refs.device());
  check(mm3idx_release_pages(&p, stream_of(refs)), "mm3idx_release_pages");
  Py_RETURN_NONE;
}

PyObject* pair_of(at::Tensor first, at::Tensor second) {
  PyObject* a = THPVariable_Wrap(std::move(first));
  PyObject* b = a ? THPVariable_Wrap(std::move(second)) : nullptr;
  PyObject* result = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  if (!result) throw Raised();
  return result;
}

// (table, lengths)
PyObject* fork_pages(PyObject* const* args) {
  const at::Tensor &refs = tensor(args[0], "refs"), &table = tensor(args[1], "page_table"),
                   &lens = tensor(args[2], "seq_lens"), &parents = tensor(args[3], "parents");
  const at::Tensor *out = maybe(args[6], "out"), *out_lens = maybe(args[7], "out_lens");
  const mm3idx_pool_t p = pool_of(refs, table, &lens, integer(args[5]));
  need(is(parents, at::kInt, 1) && parents.is_contiguous() && parents.size(0) <= INT32_MAX,
       "parents must be contiguous int32 [forks]");
  const int64_t n = parents.size(0), width = table.size(1);
  need(!out || (is(*out, at::kInt, 2) && shaped(*out, {n, width}) && unit_inner(*out)),
       "out must be int32 [forks, columns of the page table] with unit inner stride");
  need(!out_lens || (is(*out_lens, at::kInt, 1) && out_lens->size(0) == n && out_lens->is_contiguous()),
       "out_lens must be contiguous int32 [forks]");
  same_gpu(refs, {&parents, out, out_lens});
  const Caches caches(args[4], refs, refs.size(0));
  const c10::cuda::CUDAGuard guard(refs.device());
  at::Tensor results[2];
  Outputs<2> made;
  if (out) results[0] = *out;
  else made.add(0, at::kInt, {n, width});
  if (out_lens) results[1] = *out_lens;
  else made.add(1, at::kInt, {n});
  if (!out || !out_lens) made.allocate(refs, results);
  const at::Tensor ws = pages_workspace(args[8], refs, static_cast<int32_t>(n));
  check(mm3idx_fork_pages(&p, static_cast<const int32_t*>(parents.data_ptr()),
                          static_cast<int32_t>(n), static_cast<int32_t*>(results[0].data_ptr()),
                          row_stride(results[0]), static_cast<int32_t*>(results[1].data_ptr()),
                          caches.at, caches.count, ws.data_ptr(), ws.nbytes(), stream_of(refs)),
        "mm3idx_fork_pages");
  return pair_of(std::move(results[0]), std::move(results[1]));
}

// (refs, table, live)
PyObject* compact_pages(PyObject* const* args) {
  const at::Tensor &refs = tensor(args[0], "refs"), &table = tensor(args[1], "page_table");
  const bool in_place = truth(args[3]);
  const mm3idx_pool_t p = pool_of(refs, table, nullptr, 1);
  const Caches caches(args[2], refs, refs.size(0));
  const c10::cuda::CUDAGuard guard(refs.device());
  at::Tensor out[3];
  Outputs<3> made;
  if (in_place) {
    out[0] = refs;
    out[1] = table;
  } else {
    made.add(0, at::kInt, {refs.size(0)});
    made.add(1, at::kInt, {table.size(0), table.size(1)});
  }
  made.add(2, at::kInt, {1});
  made.allocate(refs, out);
  const at::Tensor ws = pages_workspace(args[4], refs, 0);
  check(mm3idx_compact_pages(&p, static_cast<int32_t*>(out[0].data_ptr()),
                             static_cast<int32_t*>(out[1].data_ptr()), row_stride(out[1]),
                             static_cast<int32_t*>(out[2].data_ptr()), caches.at, caches.count,
                             ws.data_ptr(), ws.nbytes(), stream_of(refs)),
        "mm3idx_compact_pages");
  PyObject* result = PyTuple_New(3);
  if (!result) throw Raised();
  for (int k = 0; k < 3; ++k) {
    PyObject* o = THPVariable_Wrap(std::move(out[k]));
    if (!o) {
      Py_DECREF(result);
      throw Raised();
    }
    PyTuple_SET_ITEM(result, k, o);
  }
  return result;
}

PyObject* copy_pages(PyObject* const* args) {
  const at::Tensor &src = tensor(args[1], "src"), &dst = tensor(args[2], "dst");
  need(is(src, at::kInt, 1) && is(dst, at::kInt, 1) && src.sizes() == dst.sizes() &&
           src.is_contiguous() && dst.is_contiguous() && src.size(0) <= INT32_MAX,
       "src and dst must be contiguous int32 of one length");
  same_gpu(src, {&dst});
  const Caches caches(args[0], src, -1);
  need(caches.count > 0, "at least one cache");
  const c10::cuda::CUDAGuard guard(src.device());
  check(mm3idx_copy_pages(caches.at, caches.count, caches.pages,
                          static_cast<const int32_t*>(src.data_ptr()),
                          static_cast<const int32_t*>(dst.data_ptr()),
                          static_cast<int32_t>(src.size(0)), stream_of(src)),
        "mm3idx_copy_pages");
  Py_RETURN_NONE;
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
    {"paged_attention", fast(entry<paged_attention, 16>), METH_FASTCALL, nullptr},
    {"accumulate_weights", fast(entry<accumulate_weights, 7>), METH_FASTCALL, nullptr},
    {"evict_blocks", fast(entry<evict_blocks, 14>), METH_FASTCALL, nullptr},
    {"verify_drafts", fast(entry<verify_drafts, 7>), METH_FASTCALL, nullptr},
    {"append_kv", fast(entry<append_kv, 13>), METH_FASTCALL, nullptr},
    {"allocate_pages", fast(entry<allocate_pages, 6>), METH_FASTCALL, nullptr},
    {"release_pages", fast(entry<release_pages, 4>), METH_FASTCALL, nullptr},
    {"fork_pages", fast(entry<fork_pages, 9>), METH_FASTCALL, nullptr},
    {"compact_pages", fast(entry<compact_pages, 5>), METH_FASTCALL, nullptr},
    {"copy_pages", fast(entry<copy_pages, 3>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
