// verify.cu -- verification of drafted tokens against the target's
// probabilities (include/mm3idx.h, mm3idx_verify_drafts).
//
// Mathematics.  Draft j (token d) is accepted while u_j q_j(d) < p_j(d), both
// products exact in fp64.  That needs one number of each row; only one row a
// request is read whole: with w(v) = p(v), or max(p(v) - q(v), 0) at the first
// rejected draft, the drawn token is the smallest v with
// w(0) + .. + w(v) > floor(u W), W the row's total.  Weights are 64-bit integers
// in units of 2^-46, so the sums are exact in any order and the token depends
// on neither the split nor the card (fp32 sums of 10^5 terms would move it in
// about 2 of 100 draws, and fp64 adds run at a fiftieth of the integer rate).
//
// What bounds it.  One pass over a row of p and one of q from HBM; for a few
// requests the chain of dependent loads (lengths, tokens, probabilities, row,
// token).  A cluster of CTAs takes a request, each a contiguous part of the
// row, its warps chunks of it whose sums stay in shared memory; the CTAs
// exchange their totals through distributed shared memory, and the one whose
// part holds the point reads the one chunk again that holds it.  One launch, no
// workspace, nothing read twice but that chunk.  It measured 45 us for 256
// requests x 131072 fp32 (85 % of the measured copy rate if every draft is
// refused somewhere), 21 us for 64 x 200000 and 5.6 us for 4 x 32000.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mm3idx.h"
#include "serving.h"

namespace mm3idx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 4;          // 16-byte loads of a lane and row in flight
constexpr int kMaxChunks = 512;     // of a CTA's part
constexpr int kMaxCluster = 16;

template <int TYPE>
struct Elem {
  static constexpr int kSize = TYPE == MM3IDX_TYPE_FP32 ? 4 : 2;
  static constexpr int kPer = 16 / kSize;          // elements of a 16-byte load
  static constexpr int kStep = 32 * kPer * kGroups;  // elements of a warp step
};

template <int TYPE>
__device__ __forceinline__ float prob_at(const char* p, int64_t i) {
  if constexpr (TYPE == MM3IDX_TYPE_FP32) return __ldg(reinterpret_cast<const float*>(p) + i);
  const uint16_t x = __ldg(reinterpret_cast<const uint16_t*>(p) + i);
  if constexpr (TYPE == MM3IDX_TYPE_BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
  return __half2float(__ushort_as_half(x));
}

// Element e of a 16-byte load.
template <int TYPE>
__device__ __forceinline__ float elem_of(const uint4& v, int e) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (TYPE == MM3IDX_TYPE_FP32) return __uint_as_float(w[e]);
  const uint32_t x = w[e >> 1];
  if constexpr (TYPE == MM3IDX_TYPE_BF16) return __uint_as_float((e & 1) ? x & 0xffff0000u : x << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>((e & 1) ? x >> 16 : x & 0xffffu)));
}

// A probability (clamped to 0..1, NaN as 0) in units of 2^-46, as two whole
// numbers: high 2^23 + low.  Adding 2^23 leaves a whole number in a float's
// mantissa, so both are differences of float images; fp32 instructions run at
// 128 a clock and SM where a conversion to 64 bits takes the slow pipe
// (256 requests x 131072: 131 us with it).
struct Limbs {
  float value;           // clamped
  uint32_t high, low;    // images: 0x4B000000 stands for 0
};
__device__ __forceinline__ Limbs limbs(float p) {
  constexpr float kBase = 8388608.0f;                      // 2^23
  p = __saturatef(p);
  const float h = __fmaf_rz(p, kBase, kBase);
  const float rest = __fmaf_rn(kBase - h, 1.0f / kBase, p);  // exact: p's bits below 2^-23
  const float l = __fmaf_rn(rest, kBase * kBase, kBase);
  return Limbs{p, __float_as_uint(h), __float_as_uint(l)};
}
// The weight of p, or of max(p - q, 0), added to two running sums of up to
// 2^8 elements.
template <bool Q>
__device__ __forceinline__ void add_weight(float p, float q, int32_t& high, int32_t& low) {
  constexpr uint32_t kZero = 0x4B000000u;                  // the image of 2^23
  const Limbs a = limbs(p);
  if constexpr (Q) {
    const Limbs b = limbs(q);
    if (a.value > b.value) {
      high += static_cast<int32_t>(a.high - b.high);
      low += static_cast<int32_t>(a.low - b.low);
    }
  } else {
    high += static_cast<int32_t>(a.high - kZero);
    low += static_cast<int32_t>(a.low - kZero);
  }
}

// floor(u * total) for u in [0, 1) (clamped, NaN as 0).
__device__ __forceinline__ uint64_t point_of(float u, uint64_t total) {
  u = fminf(fmaxf(u, 0.0f), 0.99999994f);
  return __umul64hi(__float2ull_rz(u * 18446744073709551616.0f), total);
}

// The weights of a row.  Elements are addressed by x = token + skew, so that
// x a multiple of kPer is a 16-byte boundary of p, whatever the row's address.
template <int TYPE>
struct Row {
  using E = Elem<TYPE>;
  const char* p;     // token 0
  const char* q;     // null: nothing is taken off
  int skew, end;     // tokens are x in [skew, end)
  int shift;         // bytes from a 16-byte boundary of q to q's elements of p's boundaries

  __device__ __forceinline__ Row(const char* p_, const char* q_, int vocab) : p(p_), q(q_) {
    skew = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / E::kSize;
    end = skew + vocab;
    shift = q ? static_cast<int>(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) & 15
              : 0;
  }
  // kPer elements from x, 0 outside the row, one by one.
  __device__ __forceinline__ uint4 gather(const char* row, int x) const {
    const char* at = row + static_cast<int64_t>(x - skew) * E::kSize;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E::kPer; ++e) {
      if (x + e < skew || x + e >= end) continue;
      if constexpr (E::kSize == 4) w[e] = __ldg(reinterpret_cast<const uint32_t*>(at) + e);
      else w[e >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(at) + e)) << (16 * (e & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // 16 bytes from byte `shift` of the two vectors v, next.
  __device__ __forceinline__ uint4 shifted(const uint4& v, const uint4& next) const {
    uint32_t w[8] = {v.x, v.y, v.z, v.w, next.x, next.y, next.z, next.w};
    if (shift & 8)
#pragma unroll
      for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    if (shift & 4)
#pragma unroll
      for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    const int bits = (shift & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
  }
  // One warp's elements of a step: kGroups x 32 x kPer from x0.  In rows of odd
  // lengths q's boundaries lie elsewhere than p's.  16-bit vectors of q are then
  // put together from two aligned ones, a lane's own and the next lane's (256 x
  // 131073 bf16: 48 us, 68 element by element; four fp32 elements one by one
  // cost no more than that: 57 us, 55).
  template <bool Q>
  __device__ __forceinline__ void load(int x0, uint4 (&vp)[kGroups], uint4 (&vq)[kGroups]) const {
    const int lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(x0 + lane * E::kPer - skew) * E::kSize;
    if (shift == 0 && x0 >= skew && x0 + E::kStep <= end) {
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        vp[k] = stream(p + at + k * 512);
        if constexpr (Q) vq[k] = stream(q + at + k * 512);
      }
    } else if (Q && E::kSize == 2 && x0 - E::kPer >= skew && x0 + E::kStep + E::kPer <= end) {
      const char* from = q + at - shift;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        vp[k] = stream(p + at + k * 512);
        vq[k] = stream(from + k * 512);
      }
      uint4 after = make_uint4(0, 0, 0, 0);          // what follows the last lane's vector
      if (lane == 0) after = stream(from + kGroups * 512);
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const uint4 give = lane ? vq[k] : k + 1 < kGroups ? vq[k + 1 < kGroups ? k + 1 : k] : after;
        const int src = (lane + 1) & 31;
        const uint4 next = make_uint4(__shfl_sync(0xffffffffu, give.x, src),
                                      __shfl_sync(0xffffffffu, give.y, src),
                                      __shfl_sync(0xffffffffu, give.z, src),
                                      __shfl_sync(0xffffffffu, give.w, src));
        vq[k] = shifted(vq[k], next);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        vp[k] = gather(p, x0 + (k * 32 + lane) * E::kPer);
        if constexpr (Q) vq[k] = gather(q, x0 + (k * 32 + lane) * E::kPer);
      }
    }
  }
  static __device__ __forceinline__ uint4 stream(const char* at) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
    return v;
  }
  // The lane's part of the weight of steps [s, end_step).
  template <bool Q>
  __device__ __forceinline__ uint64_t sum(int s, int end_step) const {
    uint64_t total = 0;   // unsigned: wraps as the signed low sums need
    for (; s < end_step; ++s) {
      uint4 vp[kGroups], vq[kGroups];
      load<Q>(s * E::kStep, vp, vq);
      int32_t high = 0, low = 0;
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int e = 0; e < E::kPer; ++e)
          add_weight<Q>(elem_of<TYPE>(vp[k], e), Q ? elem_of<TYPE>(vq[k], e) : 0.0f, high, low);
      total += static_cast<uint64_t>((static_cast<int64_t>(high) << 23) + low);
    }
    return total;
  }
};

template <bool Q>
__device__ __forceinline__ uint64_t weight_of(float p, float q) {
  int32_t high = 0, low = 0;
  add_weight<Q>(p, q, high, low);
  return static_cast<uint64_t>((static_cast<int64_t>(high) << 23) + low);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ uint64_t warp_scan(uint64_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t remote_u64(const uint64_t* mine, int rank) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), there;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(there) : "memory");
  return v;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const DraftArgs a, int cluster) {
  using E = Elem<TYPE>;
  __shared__ uint64_t chunks[kMaxChunks];
  __shared__ uint64_t totals[2], groups[kGroups];
  __shared__ int s_count;
  const int rank = cluster_rank(), i = blockIdx.x / cluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const char* target = static_cast<const char*>(a.target) + i * a.t_req * E::kSize;
  const char* draft = static_cast<const char*>(a.draft) + i * a.d_req * E::kSize;
  const int32_t* tokens = a.tokens + i * a.tok_stride;
  if (warp == 0) {
    const int len = a.lens ? min(max(__ldg(a.lens + i), 0), a.drafts) : a.drafts;
    bool ok = true;
    if (lane < a.drafts) {              // loaded for all, judged up to len
      const int d = __ldg(tokens + lane);
      const float u = __ldg(a.u + i * a.u_stride + lane);
      if (lane < len) {
        if (d < 0 || d >= a.vocab) {
          atomicOr(a.status, MM3IDX_DEV_BAD_TOKEN);
          ok = false;
        } else {
          const float p = prob_at<TYPE>(target, lane * a.t_row + d);
          const float q = a.draft ? prob_at<TYPE>(draft, lane * a.d_row + d) : 1.0f;
          ok = static_cast<double>(u) * q < static_cast<double>(p);
        }
      }
    }
    const unsigned no = __ballot_sync(0xffffffffu, !ok);
    // the rejected draft, or minus 1 minus the length when all are accepted
    if (lane == 0) s_count = no ? __ffs(no) - 1 : -1 - len;
  }
  __syncthreads();
  const bool rejected = s_count >= 0;
  const int count = rejected ? s_count : -1 - s_count;
  const char* p = target + count * a.t_row * E::kSize;
  const char* q = rejected && a.draft ? draft + count * a.d_row * E::kSize : nullptr;
  const int without = rejected && !a.draft ? __ldg(tokens + count) : -1;
  const float u = __ldg(a.u + i * a.u_stride + a.drafts);

  for (int pass = 0;; ++pass) {
    const Row<TYPE> r(p, pass ? nullptr : q, a.vocab);
    // The token whose weight is dropped (-1: none), as an element.
    const int drop = pass == 0 && without >= 0 && without < a.vocab ? without + r.skew : -1;
    const uint64_t dropped = drop >= 0 ? weight_of<false>(prob_at<TYPE>(p, without), 0.0f) : 0;
    // This CTA's part, in whole warp steps, and its chunks of whole steps.
    const int steps = (r.end + E::kStep - 1) / E::kStep;
    const int part = (steps + cluster - 1) / cluster;
    const int s0 = min(rank * part, steps), s1 = min(s0 + part, steps);
    const int per = (part + kMaxChunks - 1) / kMaxChunks;
    const int n = (s1 - s0 + per - 1) / per;
    for (int c = warp; c < n; c += kWarps) {
      const int from = s0 + c * per, to = min(from + per, s1);
      uint64_t sum = warp_sum(r.q ? r.template sum<true>(from, to) : r.template sum<false>(from, to));
      if (drop >= from * E::kStep && drop < to * E::kStep) sum -= dropped;
      if (lane == 0) chunks[c] = sum;
    }
    __syncthreads();
    // Chunk sums to sums up to and with each; the part's total to the others.
    if (warp == 0) {
      uint64_t before = 0;
      for (int c0 = 0; c0 < n; c0 += 32) {
        const uint64_t x = warp_scan(c0 + lane < n ? chunks[c0 + lane] : 0) + before;
        if (c0 + lane < n) chunks[c0 + lane] = x;
        before = __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) totals[pass] = before;
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    // (every warp for itself: lane k asks rank k)
    const uint64_t theirs = lane < cluster ? remote_u64(&totals[pass], lane) : 0;
    const uint64_t upto = warp_scan(theirs);
    const uint64_t total = __shfl_sync(0xffffffffu, upto, 31);
    if (total == 0 && rejected && pass == 0) continue;     // nothing left: the target's own row
    const uint64_t mine = __shfl_sync(0xffffffffu, theirs, rank);
    const uint64_t before = __shfl_sync(0xffffffffu, upto, rank) - mine;
    const uint64_t x = point_of(u, total);
    int32_t* out = a.out + i * a.out_stride;
    if (rank == 0 && warp == 1) {
      if (lane == 0) a.accepted[i] = count;
      if (lane <= a.drafts && lane != count) out[lane] = lane < count ? __ldg(tokens + lane) : -1;
      if (lane == 0 && total == 0) out[count] = a.vocab - 1;
    }
    if (x >= before && x < before + mine) {    // one CTA of the cluster, all of it
      // The first chunk whose sum, with all before it, is above the point.
      int c = 0;
      uint64_t below = before;
      for (int c0 = 0; c0 < n; c0 += 32) {
        const uint64_t y = c0 + lane < n ? chunks[c0 + lane] : 0;
        const unsigned hit = __ballot_sync(0xffffffffu, c0 + lane < n && before + y > x);
        if (hit) {
          c = c0 + __ffs(hit) - 1;
          if (c > 0) below = before + chunks[c - 1];
          break;
        }
      }
      // Warp k takes group k of each of its steps.
      bool found = false;
      for (int s = s0 + c * per; s < min(s0 + (c + 1) * per, s1) && !found; ++s) {
        const int x0 = s * E::kStep + threadIdx.x * E::kPer;
        uint64_t own = 0, upto = 0;
        uint4 vp = {}, vq = {};
        auto weight = [&](int e) {
          if (x0 + e == drop) return static_cast<uint64_t>(0);
          const float fp = elem_of<TYPE>(vp, e);
          return r.q ? weight_of<true>(fp, elem_of<TYPE>(vq, e)) : weight_of<false>(fp, 0.0f);
        };
        if (warp < kGroups) {
          vp = r.gather(p, x0);
          if (r.q) vq = r.gather(r.q, x0);
#pragma unroll
          for (int e = 0; e < E::kPer; ++e) own += weight(e);
          upto = warp_scan(own);
          if (lane == 31) groups[warp] = upto;
        }
        __syncthreads();
        uint64_t at = below;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          if (k < warp) at += groups[k];
          below += groups[k];
        }
        found = below > x;
        const unsigned hit = __ballot_sync(0xffffffffu, at + upto > x);
        if (warp < kGroups && at <= x && hit && lane == __ffs(hit) - 1) {
          at += upto - own;
          int e = 0;
#pragma unroll
          for (int y = 0; y < E::kPer; ++y) {
            at += weight(y);
            if (at <= x) e = y + 1;
          }
          out[count] = x0 + e - r.skew;
        }
        __syncthreads();
      }
    }
    break;
  }
  cluster_arrive();      // no CTA leaves while another may read its total
  cluster_wait();
}

template <int TYPE>
cudaError_t launch_t(const DraftArgs& a, int cluster, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(verify_kernel<TYPE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_reqs) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<TYPE>, a, cluster);
}

}  // namespace

cudaError_t launch_verify(const DraftArgs& a, int sms, cudaStream_t s) {
  // CTAs a request: as many as run at once (four an SM; 64 x 200000: 25.5 us
  // with 8, 32.2 with 16, half of them in a second wave), each with a step a
  // warp at least.
  const int step = a.type == MM3IDX_TYPE_FP32 ? Elem<MM3IDX_TYPE_FP32>::kStep
                                              : Elem<MM3IDX_TYPE_BF16>::kStep;
  const int most = a.vocab / (kWarps * step);
  int cluster = 1;
  while (2 * cluster <= kMaxCluster && cluster < most &&
         static_cast<int64_t>(a.num_reqs) * 2 * cluster <= 4 * sms)
    cluster *= 2;
  if (a.type == MM3IDX_TYPE_FP32) return launch_t<MM3IDX_TYPE_FP32>(a, cluster, s);
  if (a.type == MM3IDX_TYPE_BF16) return launch_t<MM3IDX_TYPE_BF16>(a, cluster, s);
  return launch_t<MM3IDX_TYPE_FP16>(a, cluster, s);
}

}  // namespace mm3idx
