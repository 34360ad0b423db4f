// verify.cu -- verification of drafted tokens against the target's
// probabilities (include/mm3idx.h, mm3idx_verify_drafts).
//
// One CTA per request.  The accepted drafts need one probability of each row;
// only the row of the first rejected draft (or the last row) is read whole,
// twice: once for its total weight, once for the token whose cumulative
// weight passes u * total.  Weights are 64-bit integers in units of 2^-52, so
// sums are exact whatever their order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mm3idx.h"
#include "serving.h"

namespace mm3idx {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

template <int TYPE>
__device__ __forceinline__ float prob_at(const void* p, int64_t i) {
  if (TYPE == MM3IDX_TYPE_FP32) return __ldg(static_cast<const float*>(p) + i);
  if (TYPE == MM3IDX_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// A probability in units of 2^-52: clamped to 0..1, NaN as 0.
__device__ __forceinline__ int64_t fixed(float p) {
  p = fminf(fmaxf(p, 0.0f), 1.0f);   // fmaxf(NaN, 0) is 0
  return __float2ll_rn(p * 4503599627370496.0f);
}

// floor(u * total) for u in [0, 1) (clamped, NaN as 0).
__device__ __forceinline__ uint64_t target_of(float u, uint64_t total) {
  u = fminf(fmaxf(u, 0.0f), 0.99999994f);
  return __umul64hi(__float2ull_rz(u * 18446744073709551616.0f), total);
}

// What is left of the row at token v: p, or max(p - q, 0).
template <int TYPE>
struct Row {
  const void* p;
  const void* q;     // null: nothing is taken off
  int without;       // a token whose weight is dropped, -1: none
  __device__ __forceinline__ uint64_t weight(int v) const {
    int64_t w = fixed(prob_at<TYPE>(p, v));
    if (q) w = max(w - fixed(prob_at<TYPE>(q, v)), static_cast<int64_t>(0));
    return v == without ? 0 : static_cast<uint64_t>(w);
  }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The row's weight from token v on to each warp's share: warp w has tokens
// [w * share, (w + 1) * share).
template <int TYPE>
__device__ __forceinline__ uint64_t total_of(const Row<TYPE>& r, int vocab, int share,
                                             uint64_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int end = min(vocab, (warp + 1) * share);
  uint64_t s = 0;
  for (int v = warp * share + lane; v < end; v += 32) s += r.weight(v);
  s = warp_sum(s);
  __syncthreads();
  if (lane == 0) sums[warp] = s;
  __syncthreads();
  uint64_t total = 0;
  for (int w = 0; w < kWarps; ++w) total += sums[w];
  return total;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) verify_kernel(const DraftArgs a) {
  __shared__ uint64_t sums[kWarps];
  __shared__ int s_count;
  const int i = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = a.lens ? min(max(a.lens[i], 0), a.drafts) : a.drafts;
  constexpr int kSize = TYPE == MM3IDX_TYPE_FP32 ? 4 : 2;
  const char* target = static_cast<const char*>(a.target) + i * a.t_req * kSize;
  const char* draft = static_cast<const char*>(a.draft) + i * a.d_req * kSize;
  if (warp == 0) {
    bool ok = true;
    if (lane < len) {
      const int d = a.tokens[i * a.tok_stride + lane];
      if (d < 0 || d >= a.vocab) {
        atomicOr(a.status, MM3IDX_DEV_BAD_TOKEN);
        ok = false;
      } else {
        const float p = prob_at<TYPE>(target, lane * a.t_row + d);
        const float q = a.draft ? prob_at<TYPE>(draft, lane * a.d_row + d) : 1.0f;
        ok = static_cast<double>(a.u[i * a.u_stride + lane]) * q < static_cast<double>(p);
      }
    }
    const unsigned no = __ballot_sync(0xffffffffu, !ok);
    if (lane == 0) s_count = no ? __ffs(no) - 1 : len;
  }
  __syncthreads();
  const int count = s_count;
  Row<TYPE> r{target + count * a.t_row * kSize, nullptr, -1};
  if (count < len) {
    if (a.draft) r.q = draft + count * a.d_row * kSize;
    else r.without = a.tokens[i * a.tok_stride + count];
  }
  const int share = (a.vocab + kWarps - 1) / kWarps;
  uint64_t total = total_of(r, a.vocab, share, sums);
  if (total == 0 && count < len) {
    r = Row<TYPE>{r.p, nullptr, -1};
    total = total_of(r, a.vocab, share, sums);
  }
  // The warp whose share holds the point finds it.
  const uint64_t x = target_of(a.u[i * a.u_stride + a.drafts], total);
  uint64_t before = 0;
  int owner = -1;
  for (int w = 0; w < kWarps && owner < 0; ++w) {
    if (before + sums[w] > x) owner = w;
    else before += sums[w];
  }
  int32_t* out = a.out + i * a.out_stride;
  if (threadIdx.x == 0) {
    a.accepted[i] = count;
    for (int j = 0; j < count; ++j) out[j] = a.tokens[i * a.tok_stride + j];
    for (int j = count + 1; j <= a.drafts; ++j) out[j] = -1;
    if (owner < 0) out[count] = a.vocab - 1;
  }
  if (warp != owner) return;
  const int end = min(a.vocab, (warp + 1) * share);
  for (int v0 = warp * share; v0 < end; v0 += 32) {
    const int v = v0 + lane;
    uint64_t incl = v < end ? r.weight(v) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + incl > x);
    if (hit) {
      if (lane == 0) out[count] = v0 + __ffs(hit) - 1;
      return;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

}  // namespace

cudaError_t launch_verify(const DraftArgs& a, int sms, cudaStream_t s) {
  (void)sms;
  if (a.type == MM3IDX_TYPE_FP32) verify_kernel<MM3IDX_TYPE_FP32><<<a.num_reqs, kThreads, 0, s>>>(a);
  else if (a.type == MM3IDX_TYPE_BF16) verify_kernel<MM3IDX_TYPE_BF16><<<a.num_reqs, kThreads, 0, s>>>(a);
  else verify_kernel<MM3IDX_TYPE_FP16><<<a.num_reqs, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mm3idx
