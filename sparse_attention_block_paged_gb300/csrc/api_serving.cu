// api_serving.cu -- the extern "C" boundary of the operators that use the
// selection (include/mm3idx.h: paged attention, accumulated block weights and
// eviction, draft verification): argument checks and dispatch.  No device
// memory is allocated or freed here.
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/mm3idx.h"
#include "serving.h"

using namespace mm3idx;

namespace {

constexpr float kLog2e = 1.4426950408889634f;   // the kernel's scores are base 2

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// int32 and fp32 arrays (null is aligned)
template <class... P>
bool aligned4(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) == 0;
}
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MM3IDX_OK : MM3IDX_ERR_CUDA; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

bool head_shape_ok(int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  return kv_heads >= 1 && q_heads >= kv_heads && q_heads % kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128);
}

// Positive strides of `bytes`-sized elements that are multiples of 16 bytes.
bool stride16(int64_t stride, int bytes) { return stride > 0 && stride * bytes % 16 == 0; }

int check_attention(const mm3idx_attention_t* a) {
  if (!a || a->num_reqs < 0) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (a->query_len < 1 || a->max_seq_len < a->query_len) return MM3IDX_ERR_QUERY_LEN;
  if (static_cast<int64_t>(a->num_reqs) * a->query_len >= INT_MAX / 2)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if (cdiv(a->max_seq_len, kBlock) >= 0xFFFF) return MM3IDX_ERR_TOO_MANY_BLOCKS;
  if (!(a->sm_scale > 0.0f) || !std::isfinite(a->sm_scale) || !(a->k_scale > 0.0f) ||
      !std::isfinite(a->k_scale) || !std::isfinite(a->v_scale) ||
      !std::isnormal(a->sm_scale * a->k_scale) ||
      !std::isfinite(a->sm_scale * a->k_scale * kLog2e))
    return MM3IDX_ERR_INVALID_ARGUMENT;
  const bool half = a->q_type == MM3IDX_TYPE_BF16 || a->q_type == MM3IDX_TYPE_FP16;
  if (!half || (a->kv_type != a->q_type && a->kv_type != MM3IDX_TYPE_E4M3) ||
      !head_shape_ok(a->q_heads, a->kv_heads, a->head_dim) ||
      (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128))
    return MM3IDX_ERR_ATTENTION_SHAPE;
  if (static_cast<int64_t>(a->q_heads) * a->num_reqs * a->query_len >= INT_MAX)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  // A CTA counts its share of the work list in 32 bits: 2^37 / SMs < 2^30.
  const int64_t group = a->q_heads / a->kv_heads;
  if (static_cast<int64_t>(a->num_reqs) * a->kv_heads * cdiv(group * a->query_len, 64) >
      (int64_t{1} << 37) / (cdiv(a->max_seq_len, kBlock) + kTaskCost))
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if (a->num_reqs == 0) return MM3IDX_OK;
  if (!a->q || !a->k_cache || !a->v_cache || !a->page_table || !a->seq_lens || !a->out)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!aligned4(a->seq_lens)) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!aligned4(a->page_table)) return MM3IDX_ERR_TABLE_LAYOUT;
  if (!aligned4(a->lse, a->block_weights)) return MM3IDX_ERR_ATTENTION_LAYOUT;
  if (a->num_pages < 1) return MM3IDX_ERR_CACHE_LAYOUT;
  const int kb = a->kv_type == MM3IDX_TYPE_E4M3 ? 1 : 2;
  if (!aligned16(a->q) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned16(a->out) ||
      !stride16(a->q_token_stride, 2) || !stride16(a->q_head_stride, 2) ||
      !stride16(a->k_page_stride, kb) || !stride16(a->k_token_stride, kb) ||
      !stride16(a->k_head_stride, kb) || !stride16(a->v_page_stride, kb) ||
      !stride16(a->v_token_stride, kb) || !stride16(a->v_head_stride, kb) ||
      !stride16(a->out_token_stride, 2) || !stride16(a->out_head_stride, 2))
    return MM3IDX_ERR_ATTENTION_LAYOUT;
  // [rows, heads, d] or [heads, rows, d] order, without overlap
  const int64_t rows = static_cast<int64_t>(a->num_reqs) * a->query_len;
  const int64_t ot = a->out_token_stride, oh = a->out_head_stride, D = a->head_dim;
  const bool by_row = (a->q_heads == 1 || oh >= D) && (rows == 1 || ot >= (a->q_heads - 1) * oh + D);
  const bool by_head = (rows == 1 || ot >= D) && (a->q_heads == 1 || oh >= (rows - 1) * ot + D);
  if (!by_row && !by_head) return MM3IDX_ERR_ATTENTION_LAYOUT;
  if (a->lse && a->lse_token_stride < a->q_heads) return MM3IDX_ERR_ATTENTION_LAYOUT;
  if (a->block_weights && a->block_weights_stride < cdiv(a->max_seq_len, kBlock))
    return MM3IDX_ERR_ATTENTION_LAYOUT;
  if (a->table_width < cdiv(a->max_seq_len, a->page_size) || a->table_stride < a->table_width)
    return MM3IDX_ERR_TABLE_LAYOUT;
  return MM3IDX_OK;
}

int check_scales(const mm3idx_kv_scales_t* s) {
  if (!s || !s->k || !s->v) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!aligned4(s->k, s->v) || s->k_page_stride < 0 || s->k_head_stride < 0 ||
      s->v_page_stride < 0 || s->v_head_stride < 0)
    return MM3IDX_ERR_ATTENTION_LAYOUT;
  return MM3IDX_OK;
}

// Workspace: [a ticket an SM][partial references and sums][partial outputs], for
// block weights [rows' log-sum-exps][tiles' log-sum-exps], each 256-aligned.
// Tickets have to be zero when a call starts; they come first and are as many
// for every problem, so that calls of any shapes can share a workspace.
struct AttentionWs {
  size_t ml, o, row, tile, total;   // offsets (of the tickets: 0), sum
};

AttentionWs attention_ws(int sms, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                         int32_t num_reqs, int32_t query_len, int32_t max_seq_len, bool weights) {
  const int64_t rows = static_cast<int64_t>(q_heads / kv_heads) * query_len;  // of a kv head
  const size_t tasks = static_cast<size_t>(num_reqs) * kv_heads * cdiv(rows, 64);
  const int r = static_cast<int>(rows < 64 ? rows : 64);
  AttentionWs w{};
  w.ml = align256(static_cast<size_t>(sms) * 4);
  w.o = w.ml + static_cast<size_t>(2 * sms) * 64 * 8;
  w.row = w.o + static_cast<size_t>(2 * sms) * 64 * head_dim * 4;
  w.tile = w.row + (weights ? align256(static_cast<size_t>(num_reqs) * query_len * q_heads * 4) : 0);
  w.total = w.tile +
            (weights ? align256(tasks * cdiv(max_seq_len, kBlock) * 16 *
                                attention_row_tiles16(r) * 4)
                     : 0);
  return w;
}

// [pages, heads, tokens, d] of one cache: boxes of one page and kv head, at
// most 128 bytes of d.
int make_cache_map(const mm3idx_attention_t* p, bool values, CUtensorMap* m) {
  TensorMapEncode enc = tensor_map_encoder();
  if (!enc) return MM3IDX_ERR_CUDA;
  const cuuint64_t size = p->kv_type == MM3IDX_TYPE_E4M3 ? 1 : 2;
  const CUtensorMapDataType type = p->kv_type == MM3IDX_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : p->kv_type == MM3IDX_TYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const cuuint32_t row = static_cast<cuuint32_t>(p->head_dim * size > 128 ? 128 : p->head_dim * size);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p->head_dim),
                              static_cast<cuuint64_t>(p->page_size),
                              static_cast<cuuint64_t>(p->kv_heads),
                              static_cast<cuuint64_t>(p->num_pages)};
  const cuuint64_t strides[3] = {
      static_cast<cuuint64_t>(values ? p->v_token_stride : p->k_token_stride) * size,
      static_cast<cuuint64_t>(values ? p->v_head_stride : p->k_head_stride) * size,
      static_cast<cuuint64_t>(values ? p->v_page_stride : p->k_page_stride) * size};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(row / size),
                             static_cast<cuuint32_t>(p->page_size), 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, type, 4, const_cast<void*>(values ? p->v_cache : p->k_cache), dims,
                         strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MM3IDX_OK : MM3IDX_ERR_ATTENTION_LAYOUT;
}

// The launch of a checked problem that has requests.
int attend(const mm3idx_attention_t* p, const mm3idx_kv_scales_t* s, void* workspace,
           size_t workspace_bytes, void* stream) {
  int sms = 0;
  int32_t* status = nullptr;
  int rc = library_device(&sms, &status);
  if (rc) return rc;
  const AttentionWs w = attention_ws(sms, p->q_heads, p->kv_heads, p->head_dim, p->num_reqs,
                                     p->query_len, p->max_seq_len, p->block_weights != nullptr);
  if (!workspace || workspace_bytes < w.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return MM3IDX_ERR_WORKSPACE;
  AttentionArgs a{};
  a.q = p->q;
  a.q_tok = p->q_token_stride;
  a.q_head = p->q_head_stride;
  a.kv_heads = p->kv_heads;
  a.group = p->q_heads / p->kv_heads;
  a.head_dim = p->head_dim;
  a.q_type = p->q_type;
  a.kv_type = p->kv_type;
  a.num_pages = p->num_pages;
  a.page_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.table_width = p->table_width;
  a.seq_lens = p->seq_lens;
  a.num_reqs = p->num_reqs;
  a.query_len = p->query_len;
  a.max_seq_len = p->max_seq_len;
  a.scale = p->sm_scale * p->k_scale;
  a.v_scale = p->v_scale;
  if (s) {
    a.k_scales = s->k;
    a.v_scales = s->v;
    a.ks_page = s->k_page_stride;
    a.ks_head = s->k_head_stride;
    a.vs_page = s->v_page_stride;
    a.vs_head = s->v_head_stride;
  }
  a.out = p->out;
  a.o_tok = p->out_token_stride;
  a.o_head = p->out_head_stride;
  a.lse = p->lse;
  a.lse_tok = p->lse_token_stride;
  a.weights = p->block_weights;
  a.w_stride = p->block_weights_stride;
  a.w_width = static_cast<int32_t>(cdiv(p->max_seq_len, kBlock));
  a.status = status;
  const int rows = a.group * a.query_len;
  a.row_tiles = static_cast<int32_t>(cdiv(rows, 64));
  // The most kv heads side by side that leave no more than one SM in 25 idle.
  a.gang = 1;
  for (int g = 2; g <= a.kv_heads && g <= sms; ++g)
    if (a.kv_heads % g == 0 && sms / g * g * 25 >= sms * 24) a.gang = g;
  a.tasks = a.kv_heads / a.gang * a.row_tiles;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.tickets = reinterpret_cast<unsigned int*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  if (p->block_weights) {
    a.row_lse = reinterpret_cast<float*>(ws + w.row);
    a.tile_lse = reinterpret_cast<float*>(ws + w.tile);
  }
  CUtensorMap kmap, vmap;
  if ((rc = make_cache_map(p, false, &kmap)) || (rc = make_cache_map(p, true, &vmap))) return rc;
  // One CTA an SM; no more than there can be tiles.
  const int64_t most = static_cast<int64_t>(p->num_reqs) * a.tasks * (cdiv(p->max_seq_len, kBlock) + 2);
  const int gangs = static_cast<int>(most < sms / a.gang ? most : sms / a.gang);
  const int grid = gangs * a.gang;
  const int32_t deal = (a.num_reqs + gangs - 1) / gangs;
  a.deal = Divisor(deal);
  a.deal_full = a.num_reqs / deal;
  a.deal_rest = a.num_reqs % deal;
  a.by_tasks = Divisor(a.tasks);
  a.by_row_tiles = Divisor(a.row_tiles);
  a.by_group = Divisor(a.group);
  const int64_t list = static_cast<int64_t>(p->num_reqs) * a.tasks *
                       (cdiv(p->max_seq_len, kBlock) + kTaskCost);
  a.few = p->num_reqs <= 32 && list <= UINT32_MAX / gangs;
  return cuda_status(launch_attention(kmap, vmap, a, grid, static_cast<cudaStream_t>(stream)));
}

int check_weights(const mm3idx_weights_t* w) {
  if (!w || w->num_reqs < 0 || w->topk < 0) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (w->query_len < 1 || w->max_seq_len < 1) return MM3IDX_ERR_QUERY_LEN;
  if (static_cast<int64_t>(w->num_reqs) * w->query_len >= INT_MAX) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (cdiv(w->max_seq_len, kBlock) >= 0xFFFF) return MM3IDX_ERR_TOO_MANY_BLOCKS;
  if (!(w->decay >= 0.0 && w->decay <= 1.0)) return MM3IDX_ERR_BUDGET;
  if (w->num_reqs == 0) return MM3IDX_OK;
  const int64_t width = cdiv(w->max_seq_len, kBlock);
  if (!w->acc || !w->seq_lens) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!aligned4(w->seq_lens)) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!aligned4(w->block_weights, w->ids)) return MM3IDX_ERR_TABLE_LAYOUT;
  if (w->acc_stride < width || !aligned4(w->acc)) return MM3IDX_ERR_OUT_LAYOUT;
  if (!w->block_weights) return w->ids ? MM3IDX_ERR_INVALID_ARGUMENT : MM3IDX_OK;
  if (!w->ids) return w->weights_stride < width ? MM3IDX_ERR_TABLE_LAYOUT : MM3IDX_OK;
  if (w->topk < 1) return MM3IDX_ERR_TOPK;
  if (w->weights_stride < w->topk || w->ids_stride < w->topk) return MM3IDX_ERR_TABLE_LAYOUT;
  if (static_cast<int64_t>(w->query_len) * w->topk > MM3IDX_MAX_WEIGHT_ENTRIES)
    return MM3IDX_ERR_UNSUPPORTED;
  return MM3IDX_OK;
}

WeightArgs weight_args(const mm3idx_weights_t* w, int32_t* status) {
  WeightArgs a{};
  a.acc = w->acc;
  a.acc_stride = w->acc_stride;
  a.w = w->block_weights;
  a.w_stride = w->weights_stride;
  a.ids = w->ids;
  a.ids_stride = w->ids_stride;
  a.topk = w->topk;
  a.seq_lens = w->seq_lens;
  a.num_reqs = w->num_reqs;
  a.query_len = w->query_len;
  a.max_seq_len = w->max_seq_len;
  a.decay = static_cast<float>(w->decay);
  a.decay_low = static_cast<float>(w->decay - static_cast<double>(a.decay));
  a.status = status;
  return a;
}

}  // namespace

extern "C" {

int mm3idx_attention_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                     int32_t num_reqs, int32_t query_len, int32_t max_seq_len,
                                     int32_t block_weights, size_t* bytes) {
  if (!bytes || num_reqs < 0) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (query_len < 1 || max_seq_len < 1) return MM3IDX_ERR_QUERY_LEN;
  if (!head_shape_ok(q_heads, kv_heads, head_dim)) return MM3IDX_ERR_ATTENTION_SHAPE;
  int sms = 0;
  int32_t* status = nullptr;
  const int rc = library_device(&sms, &status);
  if (rc) return rc;
  *bytes = attention_ws(sms, q_heads, kv_heads, head_dim, num_reqs, query_len, max_seq_len,
                        block_weights != 0)
               .total;
  return MM3IDX_OK;
}

int mm3idx_paged_attention(const mm3idx_attention_t* p, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const int rc = check_attention(p);
  return rc || p->num_reqs == 0 ? rc : attend(p, nullptr, workspace, workspace_bytes, stream);
}

int mm3idx_paged_attention_scaled(const mm3idx_attention_t* p, const mm3idx_kv_scales_t* s,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_attention(p);
  if (rc) return rc;
  if (p->kv_type != MM3IDX_TYPE_E4M3) return MM3IDX_ERR_ATTENTION_SHAPE;
  if (p->num_reqs == 0) return MM3IDX_OK;
  if ((rc = check_scales(s))) return rc;
  return attend(p, s, workspace, workspace_bytes, stream);
}

int mm3idx_accumulate_weights(const mm3idx_weights_t* w, void* stream) {
  int rc = check_weights(w);
  if (rc) return rc;
  if (w->num_reqs == 0) return MM3IDX_OK;
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  return cuda_status(launch_accumulate(weight_args(w, status), w->acc, w->acc_stride,
                                       static_cast<cudaStream_t>(stream)));
}

int mm3idx_evict_blocks(const mm3idx_weights_t* w, const mm3idx_eviction_t* e, void* stream) {
  int rc = check_weights(w);
  if (rc) return rc;
  if (!e) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (e->init_blocks < 0 || e->local_blocks < 1 ||
      static_cast<int64_t>(e->init_blocks) + e->local_blocks > e->budget)
    return MM3IDX_ERR_BUDGET;
  if (w->num_reqs == 0) return MM3IDX_OK;
  const int64_t width = cdiv(w->max_seq_len, kBlock);
  if (!e->acc_out || !e->seq_lens_out) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (e->acc_out_stride < width || (e->acc_out == w->acc && e->acc_out_stride != w->acc_stride) ||
      (e->ids && e->ids_stride < e->budget) || !aligned4(e->ids, e->acc_out, e->seq_lens_out))
    return MM3IDX_ERR_OUT_LAYOUT;
  const int64_t gone = width > e->budget ? width - e->budget : 1;
  for (const mm3idx_evict_table_t& t : e->tables) {
    if (!t.in) {
      if (t.out || t.freed) return MM3IDX_ERR_INVALID_ARGUMENT;
      continue;
    }
    if (!t.out) return MM3IDX_ERR_INVALID_ARGUMENT;
    if (t.in_stride < width || !aligned4(t.in)) return MM3IDX_ERR_TABLE_LAYOUT;
    if (t.out_stride < e->budget || (t.out == t.in && t.out_stride != t.in_stride) ||
        (t.freed && t.freed_stride < gone) || !aligned4(t.out, t.freed))
      return MM3IDX_ERR_OUT_LAYOUT;
  }
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  EvictArgs a{};
  a.w = weight_args(w, status);
  a.budget = e->budget;
  a.init_blocks = e->init_blocks;
  a.local_blocks = e->local_blocks;
  a.width = static_cast<int32_t>(width);
  for (int k = 0; k < 2; ++k) {
    const mm3idx_evict_table_t& t = e->tables[k];
    a.t[k] = EvictTable{t.in, t.in_stride, t.out, t.out_stride, t.freed, t.freed_stride};
  }
  a.ids = e->ids;
  a.ids_stride = e->ids_stride;
  a.acc_out = e->acc_out;
  a.acc_out_stride = e->acc_out_stride;
  a.seq_out = e->seq_lens_out;
  return cuda_status(launch_evict(a, static_cast<cudaStream_t>(stream)));
}

int mm3idx_verify_drafts(const mm3idx_drafts_t* d, void* stream) {
  if (!d || d->num_reqs < 0) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (d->vocab < 1 || d->vocab > (1 << 30) || d->drafts < 0 || d->drafts > MM3IDX_MAX_DRAFTS) return MM3IDX_ERR_VOCAB;
  if (d->type != MM3IDX_TYPE_FP32 && d->type != MM3IDX_TYPE_BF16 && d->type != MM3IDX_TYPE_FP16)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if (d->num_reqs == 0) return MM3IDX_OK;
  if (!d->target || (d->drafts > 0 && !d->tokens) || !d->uniforms || !d->out || !d->accepted)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  const int size = d->type == MM3IDX_TYPE_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(d->target) | reinterpret_cast<uintptr_t>(d->draft)) % size)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if ((d->drafts > 0 && d->target_row_stride < d->vocab) ||
      (d->num_reqs > 1 && d->target_req_stride < d->vocab) ||
      (d->draft && ((d->drafts > 1 && d->draft_row_stride < d->vocab) ||
                    (d->num_reqs > 1 && d->draft_req_stride < d->vocab))))
    return MM3IDX_ERR_VOCAB;
  if ((d->drafts > 0 && d->num_reqs > 1 && d->tokens_stride < d->drafts) ||
      (d->num_reqs > 1 && d->uniforms_stride < d->drafts + 1) ||
      !aligned4(d->tokens, d->draft_lens, d->uniforms))
    return MM3IDX_ERR_TABLE_LAYOUT;
  if (d->out_stride < d->drafts + 1 || !aligned4(d->out, d->accepted)) return MM3IDX_ERR_OUT_LAYOUT;
  int sms = 0;
  int32_t* status = nullptr;
  const int rc = library_device(&sms, &status);
  if (rc) return rc;
  DraftArgs a{};
  a.target = d->target;
  a.t_req = d->target_req_stride;
  a.t_row = d->target_row_stride;
  a.draft = d->draft;
  a.d_req = d->draft_req_stride;
  a.d_row = d->draft_row_stride;
  a.type = d->type;
  a.tokens = d->tokens;
  a.tok_stride = d->tokens_stride;
  a.lens = d->draft_lens;
  a.u = d->uniforms;
  a.u_stride = d->uniforms_stride;
  a.num_reqs = d->num_reqs;
  a.drafts = d->drafts;
  a.vocab = d->vocab;
  a.out = d->out;
  a.out_stride = d->out_stride;
  a.accepted = d->accepted;
  a.status = status;
  return cuda_status(launch_verify(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
