// attention.cu -- attention of a few new tokens a request over the paged
// key-value cache (include/mm3idx.h, mm3idx_paged_attention).
//
// One warp per (query row, query head): the row's tokens one after another,
// each lane holding head_dim / 32 elements of q and of the output, with the
// running maximum m and sum l of the softmax:
//   m' = max(m, s);  l' = l e^(m-m') + e^(s-m');  o' = o e^(m-m') + e^(s-m') v.
// The block weights come from a second kernel that takes the scores again
// and weighs them with the row's log-sum-exp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../../include/mm3idx.h"
#include "serving.h"

namespace mm3idx {
namespace {

constexpr int kWarps = 4;

template <int TYPE>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if (TYPE == MM3IDX_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (TYPE == MM3IDX_TYPE_FP16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(p)[i]);
}

template <int TYPE>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float x) {
  if (TYPE == MM3IDX_TYPE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else static_cast<__half*>(p)[i] = __float2half_rn(x);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The length that row j of request i sees (0: nothing).
__device__ __forceinline__ int visible(const AttentionArgs& a, int i, int j, bool report) {
  const int raw = a.seq_lens[i];
  if (report && threadIdx.x == 0) {
    int bits = 0;
    if (raw > a.max_seq_len) bits |= MM3IDX_DEV_SEQ_TOO_LONG;
    if (raw < 0 || (raw > 0 && raw < a.query_len)) bits |= MM3IDX_DEV_SEQ_TOO_SHORT;
    if (bits) atomicOr(a.status, bits);
  }
  const int seq = min(max(raw, 0), a.max_seq_len);
  return max(0, seq - a.query_len + j + 1);
}

// The score of token t (on every lane), -inf for a page outside the cache.
template <int QT, int KT, int D>
__device__ __forceinline__ float score_of(const AttentionArgs& a, const float (&q)[D / 32], int i,
                                          int kvh, int t, int lane, int& page) {
  page = a.table[static_cast<int64_t>(i) * a.table_stride + (t >> a.page_shift)];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) atomicOr(a.status, MM3IDX_DEV_BAD_PAGE);
    page = -1;
    return -INFINITY;
  }
  const int64_t at = page * a.k_page + (t & ((1 << a.page_shift) - 1)) * a.k_tok + kvh * a.k_head;
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s += q[c] * load_elem<KT>(a.k, at + lane * (D / 32) + c);
  return warp_sum(s);
}

template <int QT, int KT, int D>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttentionArgs a) {
  const int lane = threadIdx.x & 31;
  const int heads = a.kv_heads * a.group;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.num_reqs) * a.query_len * heads) return;
  const int64_t row = w / heads;
  const int h = static_cast<int>(w - row * heads), kvh = h / a.group;
  const int i = static_cast<int>(row / a.query_len), j = static_cast<int>(row % a.query_len);
  const int n = visible(a, i, j, true);
  float q[D / 32], o[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    q[c] = a.scale * load_elem<QT>(a.q, row * a.q_tok + h * a.q_head + lane * (D / 32) + c);
    o[c] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int t = 0; t < n; ++t) {
    int page;
    const float s = score_of<QT, KT, D>(a, q, i, kvh, t, lane, page);
    if (page < 0 || s == -INFINITY) continue;
    const float mn = fmaxf(m, s), f = __expf(m - mn), p = __expf(s - mn);
    const int64_t at =
        page * a.v_page + (t & ((1 << a.page_shift) - 1)) * a.v_tok + kvh * a.v_head;
    l = l * f + p;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      o[c] = o[c] * f + p * load_elem<KT>(a.v, at + lane * (D / 32) + c);
    m = mn;
  }
  const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
  const float lse = l == 0.0f ? -INFINITY : m + logf(l);
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    store_elem<QT>(a.out, row * a.o_tok + h * a.o_head + lane * (D / 32) + c, o[c] * inv);
  if (lane == 0) {
    if (a.lse) a.lse[row * a.lse_tok + h] = lse;
    a.lse_ws[row * heads + h] = lse;
  }
}

// One warp per (row, block).
template <int QT, int KT, int D>
__global__ void __launch_bounds__(kWarps * 32) block_weight_kernel(const AttentionArgs a) {
  const int lane = threadIdx.x & 31;
  const int heads = a.kv_heads * a.group;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.num_reqs) * a.query_len * a.w_width) return;
  const int64_t row = w / a.w_width;
  const int b = static_cast<int>(w - row * a.w_width);
  const int i = static_cast<int>(row / a.query_len), j = static_cast<int>(row % a.query_len);
  const int n = min(visible(a, i, j, false), (b + 1) * kBlock);
  float sum = 0.0f;
  for (int h = 0; h < heads; ++h) {
    const float lse = a.lse_ws[row * heads + h];
    if (lse == -INFINITY) continue;
    float q[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      q[c] = a.scale * load_elem<QT>(a.q, row * a.q_tok + h * a.q_head + lane * (D / 32) + c);
    for (int t = b * kBlock; t < n; ++t) {
      int page;
      const float s = score_of<QT, KT, D>(a, q, i, h / a.group, t, lane, page);
      if (page >= 0) sum += __expf(s - lse);
    }
  }
  if (lane == 0) a.weights[row * a.w_stride + b] = sum;
}

template <int QT, int KT, int D>
cudaError_t launch_typed(const AttentionArgs& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.num_reqs) * a.query_len;
  const int64_t warps = rows * a.kv_heads * a.group;
  attention_kernel<QT, KT, D>
      <<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
  if (a.weights)
    block_weight_kernel<QT, KT, D>
        <<<static_cast<unsigned>((rows * a.w_width + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs& a, int sms, cudaStream_t s) {
  (void)sms;
  constexpr int B = MM3IDX_TYPE_BF16, H = MM3IDX_TYPE_FP16, E = MM3IDX_TYPE_E4M3;
  const bool wide = a.head_dim == 128;
  if (a.q_type == B)
    return a.kv_type == B ? (wide ? launch_typed<B, B, 128>(a, s) : launch_typed<B, B, 64>(a, s))
                          : (wide ? launch_typed<B, E, 128>(a, s) : launch_typed<B, E, 64>(a, s));
  return a.kv_type == H ? (wide ? launch_typed<H, H, 128>(a, s) : launch_typed<H, H, 64>(a, s))
                        : (wide ? launch_typed<H, E, 128>(a, s) : launch_typed<H, E, 64>(a, s));
}

}  // namespace mm3idx
