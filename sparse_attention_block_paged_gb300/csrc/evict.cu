// evict.cu -- the weight that a request's blocks have taken, and eviction of
// the lightest of them (include/mm3idx.h, mm3idx_accumulate_weights,
// mm3idx_evict_blocks).
//
// One CTA per request.  The weights are ordered by the unsigned image of
// their fp32 bits (ordered_bits), so the threshold, the weight of the last
// block that stays, is found bit by bit from the top: 32 counts of the
// weights at or above a trial value.  Of the blocks at the threshold the ones
// with the lowest ids stay.  Both the order and the counts are whole numbers:
// the result depends on nothing but the weights.
#include "../../include/mm3idx.h"
#include "ptx.cuh"
#include "serving.h"

namespace mm3idx {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kEntries = MM3IDX_MAX_WEIGHT_ENTRIES;

// The block's place in the weight order: higher is heavier, NaN above all.
__device__ __forceinline__ uint32_t rank_bits(float w) {
  return w != w ? 0xFFFFFFFFu : ordered_bits(w);
}

struct Shared {
  int32_t ids[kEntries];
  float w[kEntries];
  uint32_t touched[(0xFFFF + 31) / 32];  // blocks that the ids name, a bit each
  int sums[kWarps];
  int total;
};

// Sum over the CTA, on every thread (called by all of them).
__device__ __forceinline__ int block_sum(int x, Shared& sh) {
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.sums[threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, sh.sums[threadIdx.x & 31]);
}

// Sum over the threads below this one, and over all (called by all threads).
__device__ __forceinline__ int block_scan(int x, Shared& sh, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) sh.sums[warp] = incl;
  __syncthreads();
  const int s = sh.sums[lane];
  total = __reduce_add_sync(0xffffffffu, s);
  return incl - x + __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
}

__device__ __forceinline__ int request_len(const WeightArgs& a, int i) {
  const int raw = a.seq_lens[i];
  if (threadIdx.x == 0 && (raw > a.max_seq_len || raw < 0))
    atomicOr(a.status, raw < 0 ? MM3IDX_DEV_SEQ_TOO_SHORT : MM3IDX_DEV_SEQ_TOO_LONG);
  return min(max(raw, 0), a.max_seq_len);
}

// dst[0..n) = the weights of request i brought up to date (dst may be acc).
__device__ __forceinline__ void accumulate(const WeightArgs& a, int i, int n, float* dst,
                                           Shared& sh) {
  const float* acc = a.acc + i * a.acc_stride;
  const double decay = a.decay;
  const int64_t row0 = static_cast<int64_t>(i) * a.query_len;
  const int rows = a.w ? a.query_len : 0;
  if (!a.ids) {
    for (int b = threadIdx.x; b < n; b += kThreads) {
      double s = decay * acc[b];
      for (int j = 0; j < rows; ++j) s += a.w[(row0 + j) * a.w_stride + b];
      dst[b] = static_cast<float>(s);
    }
    return;
  }
  // An entry whose id appears for the first time sums all entries of that id.
  const int entries = rows * a.topk;
  for (int k = threadIdx.x; k < (n + 31) / 32; k += kThreads) sh.touched[k] = 0;
  for (int e = threadIdx.x; e < entries; e += kThreads) {
    const int64_t row = row0 + e / a.topk;
    const int b = a.ids[row * a.ids_stride + e % a.topk];
    sh.ids[e] = b >= 0 && b < n ? b : -1;
    sh.w[e] = a.w[row * a.w_stride + e % a.topk];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < entries; e += kThreads) {
    const int b = sh.ids[e];
    bool first = b >= 0;
    for (int x = 0; x < e && first; ++x) first = sh.ids[x] != b;
    if (!first) continue;
    double s = decay * acc[b];
    for (int x = e; x < entries; ++x)
      if (sh.ids[x] == b) s += sh.w[x];
    dst[b] = static_cast<float>(s);
    atomicOr(&sh.touched[b >> 5], 1u << (b & 31));
  }
  __syncthreads();
  if (a.decay != 1.0 || dst != acc)
    for (int b = threadIdx.x; b < n; b += kThreads)
      if (!((sh.touched[b >> 5] >> (b & 31)) & 1u)) dst[b] = static_cast<float>(decay * acc[b]);
}

__global__ void __launch_bounds__(kThreads) accumulate_kernel(const WeightArgs a) {
  __shared__ Shared sh;
  const int i = blockIdx.x;
  accumulate(a, i, (request_len(a, i) + kBlock - 1) / kBlock, a.acc + i * a.acc_stride, sh);
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs e) {
  __shared__ Shared sh;
  const int i = blockIdx.x;
  const int seq = request_len(e.w, i), n = (seq + kBlock - 1) / kBlock;
  float* acc = e.acc_out + i * e.acc_out_stride;   // up to date here, then compacted in place
  accumulate(e.w, i, n, acc, sh);
  __syncthreads();
  const int kept = min(n, e.budget), f_lo = e.init_blocks, l_lo = n - e.local_blocks;
  // The threshold among the blocks [f_lo, l_lo): `picks` of them stay.
  const int picks = kept - (n - max(0, l_lo - f_lo));
  uint32_t cut = 0;       // weights above it stay, and the first `ties` of those at it
  int ties = 0;
  if (n > e.budget) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = cut | (1u << bit);
      int c = 0;
      for (int b = f_lo + threadIdx.x; b < l_lo; b += kThreads) c += rank_bits(acc[b]) >= trial;
      if (block_sum(c, sh) >= picks) cut = trial;
    }
    int c = 0;
    for (int b = f_lo + threadIdx.x; b < l_lo; b += kThreads) c += rank_bits(acc[b]) > cut;
    ties = picks - block_sum(c, sh);
  }
  // Compaction, kThreads blocks at a time: a kept block moves to a column at
  // or before its own, so in place each chunk is read before it is written.
  int done = 0, gone = 0, tied = 0;
  for (int b0 = 0; b0 < n; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const float w = b < n ? acc[b] : 0.0f;
    const bool free = b >= f_lo && b < l_lo && n > e.budget;
    const uint32_t r = rank_bits(w);
    int all;
    const int tie_at = tied + block_scan(free && r == cut, sh, all);
    tied += all;
    const bool stays = b < n && (!free || r > cut || (r == cut && tie_at < ties));
    const int at = done + block_scan(stays, sh, all);
    const int gone_at = gone + b - b0 - (at - done);
    done += all;
    gone += min(kThreads, n - b0) - all;
    int32_t entry[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (e.t[k].in && b < n) entry[k] = e.t[k].in[i * e.t[k].in_stride + b];
    __syncthreads();
    if (stays) {
      if (e.ids) e.ids[i * e.ids_stride + at] = b;
      acc[at] = w;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!e.t[k].in || b >= n) continue;
      if (stays) e.t[k].out[i * e.t[k].out_stride + at] = entry[k];
      else if (e.t[k].freed) e.t[k].freed[i * e.t[k].freed_stride + gone_at] = entry[k];
    }
  }
  __syncthreads();
  const int room = max(1, e.width - e.budget);
  for (int c = threadIdx.x; c < max(e.width, e.budget); c += kThreads) {
    if (c >= kept && c < e.width) acc[c] = 0.0f;
    if (c >= kept && c < e.budget && e.ids) e.ids[i * e.ids_stride + c] = -1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!e.t[k].in) continue;
      if (c >= kept && c < e.budget) e.t[k].out[i * e.t[k].out_stride + c] = -1;
      if (c >= n - kept && c < room && e.t[k].freed)
        e.t[k].freed[i * e.t[k].freed_stride + c] = -1;
    }
  }
  if (threadIdx.x == 0) e.seq_out[i] = seq - kBlock * (n - kept);
}

}  // namespace

cudaError_t launch_accumulate(const WeightArgs& a, cudaStream_t s) {
  if (!a.w && a.decay == 1.0) return cudaSuccess;
  accumulate_kernel<<<a.num_reqs, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  evict_kernel<<<a.w.num_reqs, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mm3idx
