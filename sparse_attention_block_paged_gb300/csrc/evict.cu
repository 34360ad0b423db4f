// evict.cu -- the weight that a request's blocks have taken, and eviction of
// the lightest of them (include/mm3idx.h, mm3idx_accumulate_weights,
// mm3idx_evict_blocks).
//
// Mathematics.  acc' = decay acc + sum of the step's weights, carried as an
// unevaluated sum of two floats (products by fma, sums by the two-sum of Knuth),
// good to about 2^-46 of the terms' magnitudes, then rounded once to fp32.  The
// order of the terms is fixed (query rows, then places), so a call repeats
// itself; another order can move a result next to a rounding border by a step.
// (fp64 instructions would do the same at a sixtieth of the rate:
// 128 requests of 8192 blocks took 52 us with them, most of it there.)  The
// weights are ordered by the unsigned image of their bits (ordered_bits).  The
// weight of the last block that stays is found in two steps: the keys between
// the lowest and the highest are counted in 256 bins (again within the bin that
// holds it while more than 256 keys are left), then the keys of that bin are
// compared with each other: the threshold is the lowest with fewer above it
// than have to stay.  Of blocks at the threshold the lowest ids stay.  Whole
// numbers throughout: the result depends on the weights alone.  (Two bits a
// round over all keys took 18.4 us where this takes 14.0.)
//
// What bounds it.  A few bytes a block: latency, of one round of loads, of the
// counts and of a dozen barriers.  One CTA takes a request; every load is issued
// before the first is used, and a thread keeps its blocks' weights and table
// entries in registers (blocks blockDim.x apart, so that a warp's accesses are
// one line: 16 neighbouring blocks a thread took 39 us for 128 x 8192 blocks).
// With many blocks a thread the issue of instructions bounds it.  Wider tables
// than the registers hold (kFastWidth) go through global memory.  It measured
// 14.0 us for 128 requests of 1K to 8K blocks (sums 3.4, counts 3.8, columns
// 1.2, stores 2.7) and 4.6 us for 64 of 32 to 256 blocks with the entries of a
// step of 4 rows x 16 blocks (7.2 with a branch an entry in sum_block and rounds
// of counts).
#include "../../include/mm3idx.h"
#include "ptx.cuh"
#include "serving.h"

namespace mm3idx {
namespace {

constexpr int kEntries = MM3IDX_MAX_WEIGHT_ENTRIES;
constexpr int kWideThreads = 1024;
constexpr int kSumThreads = 256;
constexpr int kFew = 256;      // keys that are compared with each other
constexpr int kBins = 256;
constexpr int kMaxItems = 8;
constexpr int kFastThreads = 1024;
constexpr int kFastWidth = kMaxItems * kFastThreads;   // blocks: a million tokens

// The block's place in the weight order: higher is heavier, NaN above all.
__device__ __forceinline__ uint32_t rank_bits(float w) {
  return w != w ? 0xFFFFFFFFu : ordered_bits(w);
}
// The weight of a place (NaN for all NaNs; -0 comes back as 0).
__device__ __forceinline__ float weight_at(uint32_t r) {
  return __uint_as_float((r & 0x80000000u) ? r ^ 0x80000000u : ~r);
}

// high + low, a sum in about twice fp32's digits.
struct Sum {
  float high, low;
  // decay * x, decay given as a sum of two floats
  __device__ __forceinline__ Sum(float x, float decay_high, float decay_low) {
    high = __fmul_rn(x, decay_high);
    low = __fmaf_rn(x, decay_low, __fmaf_rn(x, decay_high, -high));
  }
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(high, x), b = __fsub_rn(s, high);
    low = __fadd_rn(low, __fadd_rn(__fsub_rn(high, __fsub_rn(s, b)), __fsub_rn(x, b)));
    high = s;
  }
  // (an infinite or NaN sum has no second part)
  __device__ __forceinline__ float value() const {
    return isfinite(high) ? __fadd_rn(high, low) : high;
  }
};

// The step's entries (query row, place) of a request, in shared memory.
struct Entries {
  int32_t id[kEntries];
  float w[kEntries];
};

__device__ __forceinline__ int load_entries(const WeightArgs& a, int i, Entries& en) {
  const int count = a.w ? a.query_len * a.topk : 0, padded = (count + 31) & ~31;
  const int64_t row0 = static_cast<int64_t>(i) * a.query_len;
  for (int e = threadIdx.x; e < padded; e += blockDim.x) {
    const int64_t row = row0 + e / a.topk;
    const int k = e % a.topk;
    en.id[e] = e < count ? __ldg(a.ids + row * a.ids_stride + k) : -1;
    en.w[e] = e < count ? __ldg(a.w + row * a.w_stride + k) : 0.0f;
  }
  return padded;
}

// Adds to `s` every entry of e's block from e on, in order; false if an
// earlier entry has that block (which then is its to sum).
__device__ __forceinline__ bool sum_block(const Entries& en, int count, int e, Sum& s) {
  const int b = en.id[e];
  for (int x = 0; x < count; x += 32) {
    uint32_t same = 0;               // the entries of this block among 32, without a branch each
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int4 v = *reinterpret_cast<const int4*>(en.id + x + 4 * k);
      same |= (v.x == b ? 1u : 0u) << (4 * k) | (v.y == b ? 2u : 0u) << (4 * k) |
              (v.z == b ? 4u : 0u) << (4 * k) | (v.w == b ? 8u : 0u) << (4 * k);
    }
    if (x <= e) {
      const uint32_t before = e - x < 32 ? (1u << (e - x)) - 1u : 0xFFFFFFFFu;
      if (same & before) return false;
    }
    for (; same; same &= same - 1) s.add(en.w[x + __ffs(same) - 1]);
  }
  return true;
}

__device__ __forceinline__ int request_len(const WeightArgs& a, int i, bool report) {
  const int raw = __ldg(a.seq_lens + i);
  if (report && (raw > a.max_seq_len || raw < 0))
    atomicOr(a.status, raw < 0 ? MM3IDX_DEV_SEQ_TOO_SHORT : MM3IDX_DEV_SEQ_TOO_LONG);
  return min(max(raw, 0), a.max_seq_len);
}

__device__ __forceinline__ int blocks_of(int len) { return (len + kBlock - 1) / kBlock; }

// dst = the weights brought up to date: kSumThreads blocks a CTA.
__global__ void __launch_bounds__(kSumThreads)
    accumulate_kernel(const WeightArgs a, float* dst, int64_t dst_stride) {
  __shared__ __align__(16) Entries en;
  __shared__ int touched[kSumThreads];
  const int i = blockIdx.x, b0 = blockIdx.y * kSumThreads, b = b0 + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = blocks_of(request_len(a, i, threadIdx.x == 0 && b0 == 0));
  if (b0 >= n) return;
  const float* acc = a.acc + i * a.acc_stride;
  float* out = dst + i * dst_stride;
  const float old = b < n ? acc[b] : 0.0f;
  Sum s(old, a.decay, a.decay_low);
  if (a.ids && a.w) {
    const int count = load_entries(a, i, en);
    touched[threadIdx.x] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < count; e += kSumThreads) {
      const int at = en.id[e];
      if (at < b0 || at >= min(n, b0 + kSumThreads)) continue;
      Sum t(acc[at], a.decay, a.decay_low);
      if (!sum_block(en, count, e, t)) continue;
      touched[at - b0] = 1;
      out[at] = t.value();
    }
    __syncthreads();
    if (b >= n || touched[threadIdx.x]) return;
  } else if (a.w && b < n) {
    const float* w = a.w + static_cast<int64_t>(i) * a.query_len * a.w_stride + b;
    for (int j = 0; j < a.query_len; ++j) s.add(__ldg(w + j * a.w_stride));
  }
  if (b < n) out[b] = s.value();
}

// ------------------------------------------------------------ block-wide sums

// Sums over the warps (buffers alternate, so one barrier a call) and the
// search for the threshold.
struct Exchange {
  uint32_t word[2][32];
  uint32_t top[32], bottom[32];
  __align__(16) int bins[kBins];           // the highest first
  int bin, above, left;                    // the threshold's
  __align__(16) uint32_t list[kFew + 32];   // the keys left in the search
  int few;
  uint32_t low[kFew / 32];                 // of the list's warps
  int most[kFew / 32], count[kFew / 32];
};

// Exclusive sum of x over the threads before this one, and the total.
__device__ __forceinline__ int block_scan(int x, Exchange& ex, int turn, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) ex.word[turn & 1][warp] = incl;
  __syncthreads();
  const int s = lane < warps ? static_cast<int>(ex.word[turn & 1][lane]) : 0;
  total = __reduce_add_sync(0xffffffffu, s);
  return incl - x + __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
}

// at[k] = how many of the CTA's flags come before this thread's k-th, blocks
// in order (the k-th block of thread t is k * blockDim.x + t).
template <int ITEMS>
__device__ __forceinline__ void block_rank(uint32_t flags, int* counts, int (&at)[ITEMS]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const unsigned before = (1u << lane) - 1u;
  __syncthreads();                       // `counts` may still be read
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const unsigned set = __ballot_sync(0xffffffffu, (flags >> k) & 1u);
    at[k] = __popc(set & before);
    if (lane == 0) counts[k * warps + warp] = __popc(set);
  }
  __syncthreads();
  if (warp == 0) {                       // exclusive sums of ITEMS * warps <= 256 counts
    constexpr int kEach = ITEMS;
    int c[kEach], sum = 0;
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int p = lane * kEach + x;
      c[x] = p < ITEMS * warps ? counts[p] : 0;
      sum += c[x];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int run = incl - sum;
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int p = lane * kEach + x;
      if (p < ITEMS * warps) counts[p] = run;
      run += c[x];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) at[k] += counts[k * warps + warp];
}

// The threshold among this CTA's n keys (0: none, which no weight has): `picks`
// of them stay, those above `cut` and the first `ties` at it.  LIST: at most
// kFew threads of one key, compared with each other at once.
template <int ITEMS, bool LIST>
__device__ __forceinline__ void threshold(const uint32_t (&key)[ITEMS], int n, int picks, Exchange& ex,
                                          uint32_t& cut, int& ties) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, T = blockDim.x, warps = T >> 5;
  cut = 0xFFFFFFFFu;
  ties = 0;
  if (picks == 0) return;
  int left = min(T, (n + 31) & ~31);     // keys in the list, `picks` of which stay
  if constexpr (LIST) {
    ex.list[threadIdx.x] = key[0];
  } else {
    uint32_t top = 0, bottom = 0xFFFFFFFFu;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      top = max(top, key[k]);
      if (key[k]) bottom = min(bottom, key[k]);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    bottom = __reduce_min_sync(0xffffffffu, bottom);
    if (lane == 0) {
      ex.top[warp] = top;
      ex.bottom[warp] = bottom;
    }
    for (int x = threadIdx.x; x < kBins; x += T) ex.bins[x] = 0;
    if (threadIdx.x == 0) ex.few = 0;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < warps ? ex.top[lane] : 0u);
    bottom = __reduce_min_sync(0xffffffffu, lane < warps ? ex.bottom[lane] : 0xFFFFFFFFu);
    cut = top;
    ties = picks;
    if (top == bottom) return;
    // The threshold lies in [base, base + 2^size): how many keys in each 256th of it?
    int size = 32 - __clz(top ^ bottom);
    uint32_t base = size == 32 ? 0u : top >> size << size;
    for (;;) {
      const int shift = max(size - 8, 0);
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        const uint32_t d = key[k] - base;
        const bool in = key[k] >= base && key[k] && (size == 32 || (d >> size) == 0);
        const uint32_t bin = in ? d >> shift : 0xFFFFFFFFu;
        // (a warp's keys in one bin are one addition: equal weights are common)
        const uint32_t one = __shfl_sync(0xffffffffu, bin, 0);
        if (__all_sync(0xffffffffu, bin == one)) {
          if (in && lane == 0) atomicAdd(&ex.bins[kBins - 1 - bin], 32);
        } else if (in) {
          atomicAdd(&ex.bins[kBins - 1 - bin], 1);
        }
      }
      __syncthreads();
      if (warp == 0) {                   // from the top, eight bins a lane
        const int4 u = *reinterpret_cast<const int4*>(ex.bins + 8 * lane);
        const int4 v = *reinterpret_cast<const int4*>(ex.bins + 8 * lane + 4);
        const int c[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        const int sum = u.x + u.y + u.z + u.w + v.x + v.y + v.z + v.w;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int above = incl - sum;
        if (above < picks && picks <= incl) {
          int x = 0;
#pragma unroll
          for (int k = 0; k < 7; ++k)
            if (x == k && above + c[k] < picks) {
              above += c[k];
              ++x;
            }
          ex.bin = kBins - 1 - (8 * lane + x);
          ex.above = above;
          ex.left = ex.bins[8 * lane + x];
        }
      }
      __syncthreads();
      picks -= ex.above;
      left = ex.left;
      base += static_cast<uint32_t>(ex.bin) << shift;
      size = shift;
      if (left == picks) {               // all of them stay
        cut = base - 1;
        ties = 0;
        return;
      }
      if (size == 0) {                   // they are equal
        cut = base;
        ties = picks;
        return;
      }
      if (left <= kFew) break;
      for (int x = threadIdx.x; x < kBins; x += T) ex.bins[x] = 0;
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      // (key 0, none, is at base 0 in the interval of weights from -inf on: not of the list)
      if (key[k] && key[k] >= base && ((key[k] - base) >> size) == 0)
        ex.list[atomicAdd(&ex.few, 1)] = key[k];     // their order does not count
    if (threadIdx.x < 32) ex.list[left + threadIdx.x] = 0;
  }
  __syncthreads();
  // Every key of the list against all of them.  Those with fewer than `picks`
  // above them stay, at least in part: the lowest of them is the threshold.
  const uint32_t mine = static_cast<int>(threadIdx.x) < left ? ex.list[threadIdx.x] : 0u;
  int over = 0;
  if (warp * 32 < left) {
#pragma unroll 1
    for (int x = 0; x < left; x += 32) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(ex.list + x + 4 * k);
        over += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
      }
    }
    const bool in = mine && over < picks;
    const unsigned all = __ballot_sync(0xffffffffu, in);
    const uint32_t low = __reduce_min_sync(0xffffffffu, in ? mine : 0xFFFFFFFFu);
    const int most = __reduce_max_sync(0xffffffffu, in ? over : -1);
    if (lane == 0) {
      ex.low[warp] = low;
      ex.most[warp] = most;
      ex.count[warp] = __popc(all);
    }
  }
  __syncthreads();
  const bool part = lane * 32 < left;              // (a warp's results a lane)
  const uint32_t found = __reduce_min_sync(0xffffffffu, part ? ex.low[lane] : 0xFFFFFFFFu);
  const int from = __reduce_add_sync(0xffffffffu, part ? ex.count[lane] : 0);
  over = __reduce_max_sync(0xffffffffu, part ? ex.most[lane] : -1);
  cut = from == picks ? found - 1 : found;         // all equal ones stay
  ties = from == picks ? 0 : picks - over;
}

// ---------------------------------------------------------------- eviction

// Columns behind the kept blocks, and the new length.
__device__ __forceinline__ void finish(const EvictArgs& e, int i, int seq, int n, int kept) {
  const int room = max(1, e.width - e.budget);
  float* acc = e.acc_out + i * e.acc_out_stride;
  for (int c = kept + threadIdx.x; c < max(e.width, e.budget); c += blockDim.x) {
    if (c < e.width) acc[c] = 0.0f;
    if (c >= e.budget) continue;
    if (e.ids) e.ids[i * e.ids_stride + c] = -1;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (e.t[k].in) e.t[k].out[i * e.t[k].out_stride + c] = -1;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (e.t[k].in && e.t[k].freed)
      for (int c = n - kept + threadIdx.x; c < room; c += blockDim.x)
        e.t[k].freed[i * e.t[k].freed_stride + c] = -1;
  if (threadIdx.x == 0) e.seq_out[i] = seq - kBlock * (n - kept);
}

// ITEMS blocks a thread, blockDim.x apart.
template <int ITEMS, bool LIST>
__global__ void __launch_bounds__(kFastThreads) evict_kernel(const EvictArgs e) {
  __shared__ Exchange ex;
  __shared__ __align__(16) Entries en;
  __shared__ uint32_t touched[kFastWidth / 32];
  __shared__ int counts[kMaxItems * kFastThreads / 32];
  extern __shared__ float staged[];              // sparse steps: the weights by block
  const int i = blockIdx.x, T = blockDim.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const WeightArgs& a = e.w;
  const float* acc = a.acc + i * a.acc_stride;
  const int seq = request_len(a, i, threadIdx.x == 0), n = blocks_of(seq);
  // Up to e.width, not n: none of these loads waits for the length.
  float w[ITEMS];
  int32_t entry[2][ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int b = k * T + threadIdx.x;
    const bool in = b < e.width;
    w[k] = in ? __ldcg(acc + b) : 0.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      entry[t][k] = in && e.t[t].in ? __ldcg(e.t[t].in + i * e.t[t].in_stride + b) : 0;
  }
  if (a.w && a.ids) {
    const int count = load_entries(a, i, en);
    for (int k = threadIdx.x; k < (e.width + 31) / 32; k += T) touched[k] = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      if (k * T + threadIdx.x < e.width) staged[k * T + threadIdx.x] = w[k];
    __syncthreads();
    for (int x = threadIdx.x; x < count; x += T) {
      const int b = en.id[x];
      if (b < 0 || b >= n) continue;
      Sum s(staged[b], a.decay, a.decay_low);
      if (!sum_block(en, count, x, s)) continue;
      staged[b] = s.value();       // no other thread has this block
      atomicOr(&touched[b >> 5], 1u << (b & 31));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int b = k * T + threadIdx.x;
      if (b >= e.width) continue;
      const bool fresh = (touched[b >> 5] >> (b & 31)) & 1u;
      w[k] = fresh ? staged[b] : Sum(w[k], a.decay, a.decay_low).value();
    }
  } else {
    float x0[ITEMS];                             // the first row's, all in flight at once
    const float* x = a.w + static_cast<int64_t>(i) * a.query_len * a.w_stride + threadIdx.x;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      x0[k] = a.w && k * T + threadIdx.x < e.width ? __ldg(x + k * T) : 0.0f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      Sum s(w[k], a.decay, a.decay_low);
      if (a.w && k * T + threadIdx.x < e.width) {
        s.add(x0[k]);
        for (int j = 1; j < a.query_len; ++j) s.add(__ldg(x + j * a.w_stride + k * T));
      }
      w[k] = s.value();
    }
  }
  const int kept = min(n, e.budget), f_lo = e.init_blocks, l_lo = n - e.local_blocks;
  uint32_t place[ITEMS], key[ITEMS], cut = 0, stays = 0, tied = 0;
  int ties = 0;
  const bool full = n > e.budget;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int b = k * T + threadIdx.x;
    place[k] = rank_bits(w[k]);
    key[k] = full && b >= f_lo && b < l_lo ? place[k] : 0u;
  }
  const int open = max(0, l_lo - f_lo);
  if (full) threshold<ITEMS, LIST>(key, n, kept - (n - open), ex, cut, ties);
  // Which blocks stay, and the columns they move to.
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (k * T + threadIdx.x < n && (!key[k] || key[k] > cut)) stays |= 1u << k;
    if (full && key[k] == cut) tied |= 1u << k;
  }
  int at[ITEMS];
  if (ties > 0) {
    block_rank<ITEMS>(tied, counts, at);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      if (((tied >> k) & 1u) && at[k] < ties) stays |= 1u << k;
  }
  // (its barriers also part the loads of every thread from the stores below)
  block_rank<ITEMS>(stays, counts, at);
  int32_t* ids = e.ids ? e.ids + i * e.ids_stride : nullptr;
  float* acc_out = e.acc_out + i * e.acc_out_stride;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if ((stays >> k) & 1u) {
      if (ids) ids[at[k]] = k * T + threadIdx.x;
      acc_out[at[k]] = weight_at(place[k]);
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if (!e.t[t].in) continue;
    int32_t* out = e.t[t].out + i * e.t[t].out_stride;
    int32_t* freed = e.t[t].freed ? e.t[t].freed + i * e.t[t].freed_stride : nullptr;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int b = k * T + threadIdx.x;
      const bool stay = (stays >> k) & 1u;
      int32_t* to = stay ? out + at[k] : freed + (b - at[k]);
      if (b < n && (stay || freed)) *to = entry[t][k];
    }
  }
  finish(e, i, seq, n, kept);
}

// Any width; the weights are up to date in acc_out and compacted in place.
__global__ void __launch_bounds__(kWideThreads) evict_wide_kernel(const EvictArgs e) {
  __shared__ Exchange ex;
  const int i = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int seq = request_len(e.w, i, false), n = blocks_of(seq);
  float* acc = e.acc_out + i * e.acc_out_stride;
  const int kept = min(n, e.budget), f_lo = e.init_blocks, l_lo = n - e.local_blocks;
  uint32_t cut = 0;
  int ties = 0, turn = 0;
  const bool full = n > e.budget;
  if (full) {
    // one bit a round: a thread's count has no bound that a packed field holds
    const int picks = kept - (n - max(0, l_lo - f_lo));
    int total;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = cut | (1u << bit);
      int c = 0;
      for (int b = f_lo + threadIdx.x; b < l_lo; b += kWideThreads) c += rank_bits(acc[b]) >= trial;
      block_scan(c, ex, turn++, total);
      if (total >= picks) cut = trial;
    }
    int c = 0;
    for (int b = f_lo + threadIdx.x; b < l_lo; b += kWideThreads) c += rank_bits(acc[b]) > cut;
    block_scan(c, ex, turn++, total);
    ties = picks - total;
  }
  // kWideThreads blocks at a time: a kept block moves to a column at or before
  // its own, so each chunk is read before it is written.
  int done = 0, gone = 0, tied = 0;
  for (int c0 = 0; c0 < n; c0 += kWideThreads) {
    const int b = c0 + threadIdx.x;
    const float w = b < n ? acc[b] : 0.0f;
    const bool open = b >= f_lo && b < l_lo && full;
    const uint32_t r = rank_bits(w);
    int32_t entry[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (e.t[k].in && b < n) entry[k] = e.t[k].in[i * e.t[k].in_stride + b];
    int all;
    const int tie_at = tied + block_scan(open && r == cut, ex, turn++, all);
    tied += all;
    const bool stays = b < n && (!open || r > cut || (r == cut && tie_at < ties));
    const int at = done + block_scan(stays, ex, turn++, all);
    const int gone_at = gone + b - c0 - (at - done);
    done += all;
    gone += min(kWideThreads, n - c0) - all;
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
  finish(e, i, seq, n, kept);
}

template <class Kernel, class... Args>
cudaError_t launch(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t s,
                   const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int ITEMS, bool LIST = false>
cudaError_t launch_items(const EvictArgs& a, cudaStream_t s) {
  const int threads = ((a.width + ITEMS - 1) / ITEMS + 31) / 32 * 32;
  return launch(evict_kernel<ITEMS, LIST>, dim3(a.w.num_reqs), threads,
                a.w.w && a.w.ids ? static_cast<size_t>(a.width) * 4 : 0, s, a);
}

}  // namespace

cudaError_t launch_accumulate(const WeightArgs& a, float* dst, int64_t dst_stride, cudaStream_t s) {
  const int chunks = ((a.max_seq_len + kBlock - 1) / kBlock + kSumThreads - 1) / kSumThreads;
  return launch(accumulate_kernel, dim3(a.num_reqs, chunks), kSumThreads, 0, s, a, dst, dst_stride);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  // As many threads as it takes, up to kFastThreads, then more blocks a thread.
  if (a.width <= kFew) return launch_items<1, true>(a, s);
  if (a.width <= kFastThreads) return launch_items<1>(a, s);
  if (a.width <= 2 * kFastThreads) return launch_items<2>(a, s);
  if (a.width <= 4 * kFastThreads) return launch_items<4>(a, s);
  if (a.width <= kFastWidth) return launch_items<8>(a, s);
  const cudaError_t e = launch_accumulate(a.w, a.acc_out, a.acc_out_stride, s);
  if (e != cudaSuccess) return e;
  return launch(evict_wide_kernel, dim3(a.w.num_reqs), kWideThreads, 0, s, a);
}

}  // namespace mm3idx
