// serving.h -- argument blocks and launcher declarations of the operators
// that use the selection (paged attention, block eviction, draft
// verification), shared by their C ABI (api_serving.cu) and kernels.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace mm3idx {

// Defined in api.cu: the current device's SM count and status word, and the
// driver's tensor-map encoder (nullptr when the driver has none).
int library_device(int* sms, int32_t** status);
using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                     const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                     const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncode tensor_map_encoder();

// Positions that a (request, kv head) takes in the list beyond its tiles (its
// start and its join cost time, too), and the fewest positions worth a CTA.
// Measured over 3, 4, 5, 6: 64 x 4 rows of 4K-32K tokens 189.0, 189.4, 190.3,
// 191.5 us; 300 rows of 16 selected blocks 189.6, 189.2, 188.9, 188.2; two
// requests of 300-700 tokens with 2, 3, 4 positions at least 9.8, 10.2, 10.6.
constexpr int kTaskCost = 4;
constexpr int kMinShare = 2;

// Division by a number that the host knows: a product and a correction (with
// divisions in the kernel 4096 requests of up to 400 tokens took 318 us instead
// of 304, and 16 long ones 242 instead of 237).
struct Divisor {
  uint32_t d, m;
  Divisor() = default;
  explicit Divisor(int32_t x) : d(static_cast<uint32_t>(x)), m(0xFFFFFFFFu / d) {}
#ifdef __CUDACC__
  // n / d for 0 <= n < 2^31.  n m / 2^32 is short of it by less than n / 2^32,
  // so its whole part by 1 at most.
  __device__ __forceinline__ int quotient(int n) const {
    const uint32_t u = static_cast<uint32_t>(n), q = __umulhi(u, m);
    return static_cast<int>(q + (u - q * d >= d));
  }
#endif
};

struct AttentionArgs {
  const void* q;
  int64_t q_tok, q_head;      // element strides
  int32_t kv_heads;
  int32_t group;              // query heads per kv head
  int32_t head_dim;
  int32_t q_type, kv_type;    // MM3IDX_TYPE_*
  int32_t row_tiles;          // 64-row tiles of a kv head's group * query_len rows
  int32_t gang;               // kv heads that as many CTAs work on side by side (a divisor)
  int32_t tasks;              // kv_heads / gang * row_tiles, of a request
  int32_t num_pages;
  int32_t page_shift;         // log2 of the page's tokens
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t* seq_lens;
  int32_t num_reqs, query_len, max_seq_len;
  Divisor deal;               // places of the list that a gang gets: requests are dealt in so many turns
  int32_t deal_full, deal_rest;  // num_reqs / deal, num_reqs % deal
  Divisor by_tasks, by_row_tiles, by_group;
  bool few;                   // at most 32 requests, and a list whose positions times gangs fit 32 bits
  float scale;                // sm_scale * k_scale
  float v_scale;
  const float* k_scales;      // of a page and kv head, by the strides below; null: none
  const float* v_scales;
  int64_t ks_page, ks_head, vs_page, vs_head;
  void* out;
  int64_t o_tok, o_head;
  float* lse;                 // may be null
  int64_t lse_tok;
  float* weights;             // [rows, w_stride] fp32, may be null
  int64_t w_stride;
  int32_t w_width;            // cdiv(max_seq_len, 128)
  // workspace
  unsigned int* tickets;      // [grid], 0 between calls
  float2* part_ml;            // [2 * grid][64]: reference and sum of a CTA's share of a task
  float* part_o;              // [2 * grid][64][head_dim]
  float* row_lse;             // with weights: [rows, q heads], base 2
  float* tile_lse;            // with weights: [num_reqs * kv_heads * row_tiles][w_width][rows of
                              // the kernel], base 2
  int32_t* status;
};

// 16-row tiles that the kernel works on at a time: 1, 2 or 4.
inline int attention_row_tiles16(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

struct WeightArgs {
  float* acc;
  int64_t acc_stride;
  const float* w;             // null: nothing to add
  int64_t w_stride;
  const int32_t* ids;         // null: dense
  int64_t ids_stride;
  int32_t topk;
  const int32_t* seq_lens;
  int32_t num_reqs, query_len, max_seq_len;
  float decay, decay_low;     // the decay as a sum
  int32_t* status;
};

struct EvictTable {
  const int32_t* in;
  int64_t in_stride;
  int32_t* out;
  int64_t out_stride;
  int32_t* freed;
  int64_t freed_stride;
};

struct EvictArgs {
  WeightArgs w;
  int32_t budget, init_blocks, local_blocks;
  int32_t width;              // cdiv(max_seq_len, 128)
  EvictTable t[2];
  int32_t* ids;
  int64_t ids_stride;
  float* acc_out;
  int64_t acc_out_stride;
  int32_t* seq_out;
};

struct DraftArgs {
  const void* target;
  int64_t t_req, t_row;
  const void* draft;          // null: drafted tokens had probability 1
  int64_t d_req, d_row;
  int32_t type;
  const int32_t* tokens;
  int64_t tok_stride;
  const int32_t* lens;        // null: drafts each
  const float* u;
  int64_t u_stride;
  int32_t num_reqs, drafts, vocab;
  int32_t* out;
  int64_t out_stride;
  int32_t* accepted;
  int32_t* status;
};

// Runs f, which sets a kernel's attributes, once for each device (`done`: a
// bit a device, one word a kernel); the attributes stay with the device.
template <class F>
cudaError_t once_per_device(std::atomic<uint64_t>& done, F f) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  if ((e = f()) == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_attention(const CUtensorMap& kmap, const CUtensorMap& vmap,
                             const AttentionArgs& a, int grid, cudaStream_t s);
cudaError_t launch_attention_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  const AttentionArgs& a, int grid, cudaStream_t s);
cudaError_t launch_attention_fp16(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  const AttentionArgs& a, int grid, cudaStream_t s);
cudaError_t launch_attention_bf16_e4m3(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                       const AttentionArgs& a, int grid, cudaStream_t s);
cudaError_t launch_attention_fp16_e4m3(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                       const AttentionArgs& a, int grid, cudaStream_t s);
cudaError_t launch_attention_bf16_e4m3_scaled(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                              const AttentionArgs& a, int grid, cudaStream_t s);
cudaError_t launch_attention_fp16_e4m3_scaled(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                              const AttentionArgs& a, int grid, cudaStream_t s);
// dst may be a.acc itself.
cudaError_t launch_accumulate(const WeightArgs& a, float* dst, int64_t dst_stride, cudaStream_t s);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);
cudaError_t launch_verify(const DraftArgs& a, int sms, cudaStream_t s);

}  // namespace mm3idx
