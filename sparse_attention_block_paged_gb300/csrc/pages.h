// pages.h -- argument blocks and launcher declarations of the operators of a
// cache's pages (writing new tokens; allocation, forks, release, compaction,
// copies), shared by their C ABI (api_pages.cu) and kernels.
#pragma once

#include "../../include/mm3idx.h"
#include "serving.h"

namespace mm3idx {

struct AppendSide {             // keys or values
  const uint16_t* x;            // new tokens; strides in elements
  int64_t x_tok, x_head;
  uint8_t* cache;               // strides in bytes
  int64_t c_page, c_tok, c_head;
  float scale;                  // elements are stored divided by it
  float* scales;                // of a page and head; null: none
  int64_t s_page, s_head;
};

struct AppendArgs {
  AppendSide side[2];
  int32_t type, kv_type;
  int32_t kv_heads, head_dim;
  int32_t num_pages, page_shift;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* seq_lens;
  int32_t num_reqs, query_len, max_seq_len;
  const int32_t* cu;            // null: query_len rows each
  int32_t total_q;
  int32_t touched;              // most pages that a request's new tokens lie in
  int32_t units;                // num_reqs * touched * 2 * kv_heads
  Divisor by_heads, by_touched;
  int32_t* status;
};

struct Cache {
  uint8_t* data;
  int64_t page_stride, page_bytes;
  int32_t unit;                 // bytes of a copy's element: 16, 4 or 1
  int32_t end;                  // chunks of a page in the caches up to this one
};

// Copies of pages, and what a fork or a compaction does with the tables.
struct MoveArgs {
  Cache caches[MM3IDX_MAX_CACHES];
  int32_t num_caches;
  int32_t chunks;               // of a page in all caches
  int32_t num_pages;
  const int32_t* src;
  const int32_t* dst;           // pairs with an entry < 0 are none
  const int32_t* count;         // on the device; null: `pairs`
  int32_t pairs;
  // fork: rows of `out` from the parents' rows (out null: none)
  int32_t* refs;
  const int32_t* table;
  int64_t table_stride;
  int32_t width, page_size;
  const int32_t* seq_lens;
  int32_t num_reqs;
  const int32_t* parents;
  int32_t* out;
  int64_t out_stride;
  int32_t* out_lens;
  // compaction: entries from live on through the map (map null: none), into out
  const int32_t* map;
  const int32_t* live;
  int32_t* status;
};

// The ordered scans: allocation and forks (`claim`), compaction (`plan`).
struct ScanArgs {
  int32_t* refs;
  int32_t num_pages;
  int32_t* table;
  int64_t table_stride;
  int32_t width, page_size;
  const int32_t* seq_lens;
  int32_t num_reqs, query_len;
  int32_t columns;              // allocation: columns of a request that new tokens can lie in
  Divisor by_columns;
  const int32_t* parents;       // fork
  int64_t items;                // entries that may take a page
  int32_t* list;                // [num_pages] workspace
  int32_t* src;                 // [num_forks] or [num_pages]
  int32_t* dst;
  // compaction
  int32_t* refs_out;
  int32_t* map;
  int32_t* live;
  int32_t* moves;               // number of pairs
  int32_t* status;
};

struct ReleaseArgs {
  int32_t* refs;
  int32_t num_pages, page_size;
  const int32_t* table;
  int64_t table_stride;
  int32_t width;
  const int32_t* seq_lens;      // null: all columns
  int32_t num_reqs;
  int32_t* status;
};

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);
cudaError_t launch_allocate(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_fork_plan(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_compact_plan(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_move(const MoveArgs& a, int sms, cudaStream_t s);
cudaError_t launch_release(const ReleaseArgs& a, int sms, cudaStream_t s);

// cudaLaunchKernelEx as a programmatic dependent of the kernel before it (every
// kernel here waits for that one's end before it reads or writes), in clusters
// of `cluster` CTAs.
template <class K, class A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int cluster, const A& a,
                             cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace mm3idx
