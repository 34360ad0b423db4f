// api_pages.cu -- the extern "C" boundary of the operators of a cache's pages
// (include/mm3idx.h: new tokens' keys and values; allocation, release, forks,
// compaction, copies): argument checks and dispatch.  No device memory is
// allocated or freed here.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <numeric>

#include "pages.h"

using namespace mm3idx;

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <class... P>
bool aligned4(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ... | uintptr_t{0}) & 3u) == 0;
}
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MM3IDX_OK : MM3IDX_ERR_CUDA; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }
bool stride16(int64_t stride, int bytes) { return stride > 0 && stride * bytes % 16 == 0; }

constexpr int32_t kMaxPages = 1 << 30, kMaxReqs = 1 << 20;

// One side's scales [pages, heads]: are they all different floats?  The first two
// pairs that meet are hs / g pages and ps / g heads apart, g the strides' common divisor.
bool own_floats(int64_t pages, int64_t heads, int64_t ps, int64_t hs) {
  if (pages == 1) ps = 0;
  if (heads == 1) hs = 0;
  const int64_t g = std::gcd(ps, hs);
  return g == 0 ? pages * heads == 1 : hs / g >= pages || ps / g >= heads;
}

// Keys' and values' scales, each of own floats: is no float one of both?  Sides of
// unlike strides have to lie in ranges of their own.
bool no_common_float(const mm3idx_kv_scales_t& s, int64_t pages, int64_t heads) {
  const int64_t ps = pages > 1 ? s.k_page_stride : 0, hs = heads > 1 ? s.k_head_stride : 0;
  const int64_t pv = pages > 1 ? s.v_page_stride : 0, hv = heads > 1 ? s.v_head_stride : 0;
  const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(s.v) -
                                           reinterpret_cast<uintptr_t>(s.k)) / 4;
  if (off > (pages - 1) * ps + (heads - 1) * hs || -off > (pages - 1) * pv + (heads - 1) * hv)
    return true;
  if (ps != pv || hs != hv) return false;
  for (int64_t h = 1 - heads; h < heads; ++h) {      // a head apart, and how many pages?
    const int64_t rest = off - h * hs;
    if (rest == 0 || (ps != 0 && rest % ps == 0 && std::abs(rest / ps) < pages)) return false;
  }
  return true;
}

int check_append(const mm3idx_append_t* a) {
  if (!a || a->num_reqs < 0) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (a->query_len < 1 || a->max_seq_len < a->query_len) return MM3IDX_ERR_QUERY_LEN;
  if (cdiv(a->max_seq_len, kBlock) >= 0xFFFF) return MM3IDX_ERR_TOO_MANY_BLOCKS;
  for (const float s : {a->k_scale, a->v_scale})
    if (!(s > 0.0f) || !std::isnormal(s)) return MM3IDX_ERR_INVALID_ARGUMENT;
  const bool half = a->type == MM3IDX_TYPE_BF16 || a->type == MM3IDX_TYPE_FP16;
  const bool scaled = a->scales.k || a->scales.v;
  if (!half || (a->kv_type != a->type && a->kv_type != MM3IDX_TYPE_E4M3) || a->kv_heads < 1 ||
      (a->head_dim != 64 && a->head_dim != 128) ||
      (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128) ||
      (scaled && a->kv_type != MM3IDX_TYPE_E4M3))
    return MM3IDX_ERR_ATTENTION_SHAPE;
  if (static_cast<int64_t>(a->num_reqs) * a->query_len >= INT_MAX / 2)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  // a group of threads for every (request, page, side, head)
  if (static_cast<int64_t>(a->num_reqs) * (cdiv(a->query_len - 1, a->page_size) + 1) >
      (INT_MAX / 2 - 8) / a->kv_heads)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if (a->num_reqs == 0) return MM3IDX_OK;
  if (a->cu_seqlens_q ? a->total_q < 0 || a->total_q > a->num_reqs * a->query_len
                      : a->total_q != a->num_reqs * a->query_len)
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!a->k_cache || !a->v_cache || !a->page_table || !a->seq_lens ||
      (a->total_q > 0 && (!a->k || !a->v)) || (scaled && (!a->scales.k || !a->scales.v)))
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!aligned4(a->seq_lens, a->cu_seqlens_q)) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (!aligned4(a->page_table)) return MM3IDX_ERR_TABLE_LAYOUT;
  if (a->num_pages < 1) return MM3IDX_ERR_CACHE_LAYOUT;
  const int kb = a->kv_type == MM3IDX_TYPE_E4M3 ? 1 : 2;
  if (!aligned16(a->k) || !aligned16(a->v) || !aligned16(a->k_cache) || !aligned16(a->v_cache) ||
      !stride16(a->k_token_stride, 2) || !stride16(a->k_head_stride, 2) ||
      !stride16(a->v_token_stride, 2) || !stride16(a->v_head_stride, 2) ||
      !stride16(a->k_page_stride, kb) || !stride16(a->k_page_token_stride, kb) ||
      !stride16(a->k_page_head_stride, kb) || !stride16(a->v_page_stride, kb) ||
      !stride16(a->v_page_token_stride, kb) || !stride16(a->v_page_head_stride, kb))
    return MM3IDX_ERR_ATTENTION_LAYOUT;
  if (scaled && (!aligned4(a->scales.k, a->scales.v) || a->scales.k_page_stride < 0 ||
                 a->scales.k_head_stride < 0 || a->scales.v_page_stride < 0 ||
                 a->scales.v_head_stride < 0 ||
                 !own_floats(a->num_pages, a->kv_heads, a->scales.k_page_stride, a->scales.k_head_stride) ||
                 !own_floats(a->num_pages, a->kv_heads, a->scales.v_page_stride, a->scales.v_head_stride)))
    return MM3IDX_ERR_ATTENTION_LAYOUT;
  if (a->table_width < cdiv(a->max_seq_len, a->page_size) || a->table_stride < a->table_width)
    return MM3IDX_ERR_TABLE_LAYOUT;
  return MM3IDX_OK;
}

// `sized`: the call needs page_size; `tabled`: and seq_lens.
int check_pool(const mm3idx_pool_t* p, bool sized, bool tabled) {
  if (!p || p->num_reqs < 0 || p->num_reqs > kMaxReqs) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (p->num_pages < 1 || p->num_pages > kMaxPages || (sized && p->page_size < 1))
    return MM3IDX_ERR_PAGES;
  if (p->table_width < 0 || (p->num_reqs > 1 && p->table_stride < p->table_width) ||
      !aligned4(p->page_table))
    return MM3IDX_ERR_TABLE_LAYOUT;
  if (sized && static_cast<int64_t>(p->table_width) * p->page_size > INT_MAX / 2)
    return MM3IDX_ERR_PAGES;
  if (!p->refs || !aligned4(p->refs, p->seq_lens) ||
      (p->num_reqs > 0 && p->table_width > 0 && !p->page_table) ||
      (p->num_reqs > 0 && tabled && !p->seq_lens))
    return MM3IDX_ERR_INVALID_ARGUMENT;
  return MM3IDX_OK;
}

int check_caches(const mm3idx_cache_t* c, int32_t n, int32_t num_pages) {
  if (n < 0 || n > MM3IDX_MAX_CACHES || num_pages < 1 || num_pages > kMaxPages)
    return MM3IDX_ERR_PAGES;
  if (n > 0 && !c) return MM3IDX_ERR_INVALID_ARGUMENT;
  for (int k = 0; k < n; ++k) {
    if (!c[k].data) return MM3IDX_ERR_INVALID_ARGUMENT;
    if (c[k].page_bytes < 1 || c[k].page_stride < c[k].page_bytes ||
        c[k].page_bytes > (int64_t{1} << 24))
      return MM3IDX_ERR_PAGES;
  }
  return MM3IDX_OK;
}

// Copies by 16 bytes where base, stride and size allow it, by 4, or by 1; a warp
// takes 256 elements at a time.
void set_caches(MoveArgs& m, const mm3idx_cache_t* c, int32_t n, int32_t num_pages) {
  m.num_caches = n;
  m.num_pages = num_pages;
  int32_t end = 0;
  for (int k = 0; k < n; ++k) {
    const uint64_t all = reinterpret_cast<uintptr_t>(c[k].data) |
                         static_cast<uint64_t>(c[k].page_stride) |
                         static_cast<uint64_t>(c[k].page_bytes);
    const int unit = (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : 1;
    end += static_cast<int32_t>(cdiv(c[k].page_bytes, 256 * unit));
    m.caches[k] = Cache{static_cast<uint8_t*>(c[k].data), c[k].page_stride, c[k].page_bytes, unit, end};
  }
  m.chunks = end;
}

// Workspace: [counts][a list or map][sources][destinations], each 256-aligned.
struct PagesWs {
  size_t list, src, dst, total;
};
PagesWs pages_ws(int32_t num_pages, int32_t num_forks) {
  const size_t one = align256(4 * static_cast<size_t>(num_pages > num_forks ? num_pages : num_forks));
  return PagesWs{256, 256 + one, 256 + 2 * one, 256 + 3 * one};
}
bool workspace_ok(const void* p, size_t bytes, size_t need) {
  return p && bytes >= need && (reinterpret_cast<uintptr_t>(p) & 255u) == 0;
}

ScanArgs scan_args(const mm3idx_pool_t* p, const PagesWs& w, void* workspace, int32_t* status) {
  ScanArgs a{};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.refs = p->refs;
  a.num_pages = p->num_pages;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.width = p->table_width;
  a.page_size = p->page_size;
  a.seq_lens = p->seq_lens;
  a.num_reqs = p->num_reqs;
  a.by_columns = Divisor(1);
  a.list = reinterpret_cast<int32_t*>(ws + w.list);
  a.src = reinterpret_cast<int32_t*>(ws + w.src);
  a.dst = reinterpret_cast<int32_t*>(ws + w.dst);
  a.moves = reinterpret_cast<int32_t*>(ws);
  a.status = status;
  return a;
}

}  // namespace

extern "C" {

int mm3idx_append_kv(const mm3idx_append_t* p, void* stream) {
  int rc = check_append(p);
  if (rc) return rc;
  if (p->num_reqs == 0 || p->total_q == 0) return MM3IDX_OK;
  // the codes of a page follow its scale: what another group writes too ends up wrong
  if (p->scales.k && (p->k_cache == p->v_cache || !no_common_float(p->scales, p->num_pages, p->kv_heads)))
    return MM3IDX_ERR_ATTENTION_LAYOUT;
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  AppendArgs a{};
  const int64_t kb = p->kv_type == MM3IDX_TYPE_E4M3 ? 1 : 2;
  a.side[0] = AppendSide{static_cast<const uint16_t*>(p->k), p->k_token_stride, p->k_head_stride,
                         static_cast<uint8_t*>(p->k_cache), p->k_page_stride * kb,
                         p->k_page_token_stride * kb, p->k_page_head_stride * kb, p->k_scale,
                         p->scales.k, p->scales.k_page_stride, p->scales.k_head_stride};
  a.side[1] = AppendSide{static_cast<const uint16_t*>(p->v), p->v_token_stride, p->v_head_stride,
                         static_cast<uint8_t*>(p->v_cache), p->v_page_stride * kb,
                         p->v_page_token_stride * kb, p->v_page_head_stride * kb, p->v_scale,
                         p->scales.v, p->scales.v_page_stride, p->scales.v_head_stride};
  a.type = p->type;
  a.kv_type = p->kv_type;
  a.kv_heads = p->kv_heads;
  a.head_dim = p->head_dim;
  a.num_pages = p->num_pages;
  a.page_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.seq_lens = p->seq_lens;
  a.num_reqs = p->num_reqs;
  a.query_len = p->query_len;
  a.max_seq_len = p->max_seq_len;
  a.cu = p->cu_seqlens_q;
  a.total_q = p->total_q;
  // query_len tokens from any slot on: this many pages at most
  a.touched = static_cast<int32_t>(cdiv(p->query_len - 1, p->page_size)) + 1;
  a.units = p->num_reqs * a.touched * 2 * p->kv_heads;
  a.by_heads = Divisor(p->kv_heads);
  a.by_touched = Divisor(a.touched);
  a.status = status;
  return cuda_status(launch_append(a, static_cast<cudaStream_t>(stream)));
}

int mm3idx_pages_workspace_bytes(int32_t num_pages, int32_t num_forks, size_t* bytes) {
  if (!bytes || num_forks < 0 || num_forks > kMaxReqs) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (num_pages < 1 || num_pages > kMaxPages) return MM3IDX_ERR_PAGES;
  *bytes = pages_ws(num_pages, num_forks).total;
  return MM3IDX_OK;
}

int mm3idx_allocate_pages(const mm3idx_pool_t* p, int32_t query_len, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int rc = check_pool(p, true, true);
  if (rc) return rc;
  if (query_len < 1) return MM3IDX_ERR_QUERY_LEN;
  const int64_t columns = cdiv(query_len - 1, p->page_size) + 1;
  const int64_t most = columns < p->table_width ? columns : p->table_width;
  if (most * p->num_reqs > INT_MAX / 2) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (p->num_reqs == 0 || p->table_width == 0) return MM3IDX_OK;
  const PagesWs w = pages_ws(p->num_pages, 0);
  if (!workspace_ok(workspace, workspace_bytes, w.total)) return MM3IDX_ERR_WORKSPACE;
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  ScanArgs a = scan_args(p, w, workspace, status);
  a.query_len = query_len;
  a.columns = static_cast<int32_t>(most);
  a.by_columns = Divisor(a.columns);
  a.items = most * p->num_reqs;
  return cuda_status(launch_allocate(a, static_cast<cudaStream_t>(stream)));
}

int mm3idx_release_pages(const mm3idx_pool_t* p, void* stream) {
  int rc = check_pool(p, p && p->seq_lens, false);
  if (rc) return rc;
  if (p->num_reqs == 0 || p->table_width == 0) return MM3IDX_OK;
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  const ReleaseArgs a{p->refs, p->num_pages, p->page_size, p->page_table, p->table_stride,
                      p->table_width, p->seq_lens, p->num_reqs, status};
  return cuda_status(launch_release(a, sms, static_cast<cudaStream_t>(stream)));
}

int mm3idx_fork_pages(const mm3idx_pool_t* p, const int32_t* parents, int32_t num_forks,
                      int32_t* out, int64_t out_stride, int32_t* out_lens,
                      const mm3idx_cache_t* caches, int32_t num_caches, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc = check_pool(p, true, true);
  if (rc || (rc = check_caches(caches, num_caches, p->num_pages))) return rc;
  if (num_forks < 0 || num_forks > kMaxReqs) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (num_forks == 0) return MM3IDX_OK;
  if (!parents || !out_lens || (!out && p->table_width > 0) || !aligned4(parents))
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if ((num_forks > 1 && out_stride < p->table_width) || !aligned4(out, out_lens))
    return MM3IDX_ERR_OUT_LAYOUT;
  const PagesWs w = pages_ws(p->num_pages, num_forks);
  if (!workspace_ok(workspace, workspace_bytes, w.total)) return MM3IDX_ERR_WORKSPACE;
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  ScanArgs a = scan_args(p, w, workspace, status);
  a.parents = parents;
  a.items = num_forks;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((rc = cuda_status(launch_fork_plan(a, s)))) return rc;
  MoveArgs m{};
  set_caches(m, caches, num_caches, p->num_pages);
  m.src = a.src;
  m.dst = a.dst;
  m.pairs = num_forks;
  m.refs = p->refs;
  m.table = p->page_table;
  m.table_stride = p->table_stride;
  m.width = p->table_width;
  m.page_size = p->page_size;
  m.seq_lens = p->seq_lens;
  m.num_reqs = p->num_reqs;
  m.parents = parents;
  m.out = out;
  m.out_stride = out_stride;
  m.out_lens = out_lens;
  m.status = status;
  return cuda_status(launch_move(m, sms, s));
}

int mm3idx_compact_pages(const mm3idx_pool_t* p, int32_t* refs_out, int32_t* table_out,
                         int64_t table_out_stride, int32_t* live, const mm3idx_cache_t* caches,
                         int32_t num_caches, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_pool(p, false, false);
  if (rc || (rc = check_caches(caches, num_caches, p->num_pages))) return rc;
  if (!refs_out || !live || (p->num_reqs > 0 && p->table_width > 0 && !table_out))
    return MM3IDX_ERR_INVALID_ARGUMENT;
  if ((p->num_reqs > 1 && table_out_stride < p->table_width) ||
      (table_out == p->page_table && p->num_reqs > 1 && table_out_stride != p->table_stride) ||
      !aligned4(refs_out, table_out, live))
    return MM3IDX_ERR_OUT_LAYOUT;
  const PagesWs w = pages_ws(p->num_pages, 0);
  if (!workspace_ok(workspace, workspace_bytes, w.total)) return MM3IDX_ERR_WORKSPACE;
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  ScanArgs a = scan_args(p, w, workspace, status);
  a.refs_out = refs_out;
  a.map = a.list;
  a.live = live;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((rc = cuda_status(launch_compact_plan(a, s)))) return rc;
  MoveArgs m{};
  set_caches(m, caches, num_caches, p->num_pages);
  m.src = a.src;
  m.dst = a.dst;
  m.count = a.moves;
  m.table = p->page_table;
  m.table_stride = p->table_stride;
  m.width = p->table_width;
  m.num_reqs = p->table_width > 0 ? p->num_reqs : 0;
  m.out = table_out;
  m.out_stride = table_out_stride;
  m.map = a.map;
  m.live = live;
  m.status = status;
  return cuda_status(launch_move(m, sms, s));
}

int mm3idx_copy_pages(const mm3idx_cache_t* caches, int32_t num_caches, int32_t num_pages,
                      const int32_t* src, const int32_t* dst, int32_t count, void* stream) {
  int rc = check_caches(caches, num_caches, num_pages);
  if (rc) return rc;
  if (count < 0) return MM3IDX_ERR_INVALID_ARGUMENT;
  if (count == 0 || num_caches == 0) return MM3IDX_OK;
  if (!src || !dst || !aligned4(src, dst)) return MM3IDX_ERR_INVALID_ARGUMENT;
  int sms = 0;
  int32_t* status = nullptr;
  if ((rc = library_device(&sms, &status))) return rc;
  MoveArgs m{};
  set_caches(m, caches, num_caches, num_pages);
  m.src = src;
  m.dst = dst;
  m.pairs = count;
  m.status = status;
  return cuda_status(launch_move(m, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
