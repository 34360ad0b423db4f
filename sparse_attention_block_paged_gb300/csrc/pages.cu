// pages.cu -- pages of a cache taken, shared, given back, moved
// (include/mm3idx.h: mm3idx_allocate_pages, _release_pages, _fork_pages,
// _compact_pages, _copy_pages).
//
// The pool's state is one array of reference counts; a page is free where its
// count is 0, so there is no list of free pages to keep in step with them, and
// what a call does depends on nothing but its inputs: free pages are taken in
// ascending order, by entries in ascending order.
//
// What bounds it.  Counts (4 bytes a page) and tables are small: a cluster of
// CTAs reads them once or twice from L2 and finds every place by counting
// (a ballot a 32 entries, a prefix over warps, then over the cluster's CTAs).
// What is left is the copy of page data, at HBM's rate: a warp moves up to 4 KB
// of a page at a time, eight 16-byte loads a lane in flight before the first store.
//
// What it measured (GB300, calls captured in a CUDA graph): half of 16384 pages of
// 128 KB live, compacted: 171 us (92 % of the measured copy rate); 8 requests forked
// into 64, four layers of 128 KB a page: 15 us with the release before it (HBM needs
// 10); 1024 pages of 128 KB copied: 41.7 us (95 %); the smallest calls: release 1.8 us,
// allocation 3.3 where nothing is wanted and about 4 where it gives pages (512 or 4096
// pages; 5 of 16384), a fork 5.6, a compaction of 512 pages 7.6, all latency of one or
// two dependent kernels.  Issued from Python one after another: release 2.5, allocation
// as above, a compaction of 512 pages 8.9 to 10.
#include "pages.h"

namespace mm3idx {
namespace {

// Loads that name L2 (__ldcg): what another CTA of the same kernel wrote (lists, pairs)
// has to be read there.  Counts, tables and lengths, which only kernels before
// this one wrote, need not: griddepcontrol.wait makes those writes seen by any load
// behind it.  They are read once, so L1 has nothing to give, and alike here.

// ------------------------------------------------------------ ordered scans

constexpr int kScanThreads = 1024, kScanWarps = kScanThreads / 32;
constexpr int kCluster = 8;
constexpr int kAhead = 8;               // loads of a lane in flight
constexpr int kNear = 2048;             // entries of a list in shared memory
// Pages and entries that one CTA scans (allocation of 16 pages and compaction without
// caches, one CTA and a cluster, us: 512 pages 5.8 and 7.4, 6.9 and 9.0; 8192 7.6 and 8.6,
// 9.3 and 10.0; 16384 8.6 and 8.5, 16.4 and 10.8; 65536 17.9 and 9.5, 52 and 12.4).
constexpr int64_t kSmall = 8192;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of the cluster; what they wrote before is seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int64_t remote(const int64_t* p, uint32_t rank) {
  uint32_t at;
  int64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}

// One of a kernel's scans over [0, n): the part of one of `warps` warps a CTA (a CTA's
// first warps, or those after others), the marked entries before it and in all, and
// what the first round found (parts longer than a round look again).
struct Part {
  int64_t lo, hi, before, total;
  int found[kAhead];
};

struct Counts {
  int64_t warp[kScanWarps];
  int64_t cta;
};

// `first`: the first of the CTA's warps that share it; others get an empty part.
__device__ __forceinline__ void split(Part& p, int64_t n, int first, int warps) {
  const int w = static_cast<int>(threadIdx.x >> 5) - first;
  const int64_t all = static_cast<int64_t>(gridDim.x) * warps;
  const int64_t per = ((n + all - 1) / all + 31) & ~int64_t{31};
  const int64_t at = static_cast<int64_t>(cluster_rank()) * warps + w;
  const bool mine = w >= 0 && w < warps;
  p.lo = mine ? min(at * per, n) : 0;
  p.hi = mine ? min(p.lo + per, n) : 0;
  p.before = p.total = 0;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) p.found[k] = -1;
}

// f(entry) is what a marked entry stands for (>= 0), or -1.
template <class F>
__device__ __forceinline__ void look(const Part& p, int64_t i, F f, int (&found)[kAhead]) {
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t at = i + 32 * k + (threadIdx.x & 31);
    found[k] = at < p.hi ? f(at) : -1;
  }
}

// The number of marked entries in the warp's part, the first round's known.
template <class F>
__device__ __forceinline__ int64_t count_rest(const Part& p, F f) {
  int64_t sum = 0;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) sum += __popc(__ballot_sync(0xffffffffu, p.found[k] >= 0));
  for (int64_t i = p.lo + 32 * kAhead; i < p.hi; i += 32 * kAhead) {
    int found[kAhead];
    look(p, i, f, found);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) sum += __popc(__ballot_sync(0xffffffffu, found[k] >= 0));
  }
  return sum;
}

template <class F>
__device__ __forceinline__ int64_t count(Part& p, F f) {
  if (p.lo < p.hi) look(p, p.lo, f, p.found);
  return count_rest(p, f);
}

// g(entry, what it stands for, its rank) of the marked entries below rank `most`.
template <class F, class G>
__device__ __forceinline__ void each(const Part& p, int64_t most, F f, G g) {
  const int lane = threadIdx.x & 31;
  int64_t rank = p.before;
  for (int64_t i = p.lo; i < p.hi && rank < most; i += 32 * kAhead) {
    int found[kAhead];
    if (i == p.lo) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) found[k] = p.found[k];
    } else {
      look(p, i, f, found);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const unsigned all = __ballot_sync(0xffffffffu, found[k] >= 0);
      const int64_t r = rank + __popc(all & ((1u << lane) - 1u));
      if (found[k] >= 0 && r < most) g(i + 32 * k + lane, found[k], r);
      rank += __popc(all);
    }
  }
}

// The prefixes of N scans' counts over the warps of the cluster.
template <int N>
__device__ __forceinline__ void prefixes(Counts* c, const int64_t (&mine)[N], Part* (&parts)[N]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) c[k].warp[warp] = mine[k];
  __syncthreads();
  if (warp < N) {
    int64_t v = c[warp].warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    c[warp].warp[lane] = v;             // inclusive
    if (lane == 31) c[warp].cta = v;
  }
  cluster_sync();
  const uint32_t rank = cluster_rank();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    int64_t before = warp > 0 ? c[k].warp[warp - 1] : 0, total = 0;
    if (gridDim.x == 1) {
      total = c[k].cta;
    } else {
      const int64_t theirs = lane < static_cast<int>(gridDim.x) ? remote(&c[k].cta, lane) : 0;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) {
        const int64_t x = __shfl_sync(0xffffffffu, theirs, r);
        total += x;
        if (r < static_cast<int>(rank)) before += x;
      }
    }
    parts[k]->before = before;
    parts[k]->total = total;
  }
}

__device__ __forceinline__ int clamped_len(const ScanArgs& a, int i, bool* over) {
  const int raw = max(__ldcg(a.seq_lens + i), 0);
  const int64_t most = static_cast<int64_t>(a.width) * a.page_size;
  *over = raw > most;
  return static_cast<int>(min(static_cast<int64_t>(raw), most));
}

// Entry k of an allocation: request k / columns, one of the columns that its new
// tokens lie in; null where there is none.
__device__ __forceinline__ int32_t* allocation_entry(const ScanArgs& a, int64_t k) {
  const int i = a.by_columns.quotient(static_cast<int>(k));
  const int turn = static_cast<int>(k) - i * a.columns;
  bool over;
  const int len = clamped_len(a, i, &over);
  if (over && turn == 0) atomicOr(a.status, MM3IDX_DEV_SEQ_TOO_LONG);
  const int first = max(len - a.query_len, 0) / a.page_size, end = (len + a.page_size - 1) / a.page_size;
  return first + turn < end ? a.table + i * a.table_stride + first + turn : nullptr;
}

// The partly filled last page of fork k's parent, or -1.
__device__ __forceinline__ int last_page(const ScanArgs& a, int64_t k) {
  const int i = __ldcg(a.parents + k);
  if (i < 0 || i >= a.num_reqs) return -1;
  bool over;
  const int len = clamped_len(a, i, &over), full = len / a.page_size;
  if (full * a.page_size == len) return -1;
  const int page = __ldcg(a.table + i * a.table_stride + full);
  return page >= 0 && page < a.num_pages ? page : -1;
}

// Free pages for the entries that want one.  FORK: (source, new page) pairs.  An
// entry hangs on two or three loads in a row, a count on one: half of the warps
// each.
template <bool FORK>
__global__ void __launch_bounds__(kScanThreads) claim_kernel(const __grid_constant__ ScanArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ Counts counts[2];
  __shared__ int32_t near[kNear];        // a single CTA's list
  Part items, pages;
  split(items, a.items, 0, kScanWarps / 2);
  split(pages, a.num_pages, kScanWarps / 2, kScanWarps / 2);
  auto wants = [&](int64_t k) {
    if constexpr (FORK) return last_page(a, k);
    const int32_t* e = allocation_entry(a, k);
    return e && __ldcg(e) < 0 ? 0 : -1;
  };
  auto is_free = [&](int64_t p) { return __ldcg(a.refs + p) == 0 ? static_cast<int>(p) : -1; };
  const int64_t mine[2] = {count(items, wants), count(pages, is_free)};
  Part* parts[2] = {&items, &pages};
  prefixes(counts, mine, parts);
  const int64_t most = min(items.total, pages.total);
  int32_t* list = gridDim.x == 1 && most <= kNear ? near : a.list;
  each(pages, most, is_free, [&](int64_t p, int, int64_t r) {
    list[r] = static_cast<int32_t>(p);
    a.refs[p] = 1;
  });
  if (threadIdx.x == 0 && cluster_rank() == 0 && items.total > pages.total)
    atomicOr(a.status, MM3IDX_DEV_NO_PAGES);
  cluster_sync();
  auto entry = [&](int64_t r) { return list == near ? near[r] : __ldcg(list + r); };
  if constexpr (FORK) {
    for (int64_t k = items.lo + (threadIdx.x & 31); k < items.hi; k += 32) a.src[k] = a.dst[k] = -1;
    __syncwarp();
    each(items, most, wants, [&](int64_t k, int from, int64_t r) {
      a.src[k] = from;
      a.dst[k] = entry(r);
    });
  } else {
    each(items, items.total, wants, [&](int64_t k, int, int64_t r) {
      *allocation_entry(a, k) = r < most ? entry(r) : -1;
    });
  }
  cluster_sync();                        // no CTA leaves while its counts may be read
}

// A compaction's pairs, counts and map.
__global__ void __launch_bounds__(kScanThreads) plan_kernel(const __grid_constant__ ScanArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ Counts first[1], second[2];
  Part all;
  split(all, a.num_pages, 0, kScanWarps);
  auto used = [&](int64_t p) { return __ldcg(a.refs + p) != 0 ? static_cast<int>(p) : -1; };
  {
    const int64_t mine[1] = {count(all, used)};
    Part* parts[1] = {&all};
    prefixes(first, mine, parts);
  }
  const int64_t live = all.total;
  Part holes = all, movers = all;
  auto hole = [&](int64_t p) { return p < live && __ldcg(a.refs + p) == 0 ? static_cast<int>(p) : -1; };
  auto mover = [&](int64_t p) { return p >= live && __ldcg(a.refs + p) != 0 ? static_cast<int>(p) : -1; };
  // a warp's part lies before `live`, behind it, or is the one around it
  if (holes.lo >= live) holes.lo = holes.hi;
  if (movers.hi <= live) movers.lo = movers.hi;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t p = all.lo + 32 * k + (threadIdx.x & 31);
    const bool in = p < all.hi, free = all.found[k] < 0;
    holes.found[k] = in && free && p < live ? static_cast<int>(p) : -1;
    movers.found[k] = in && !free && p >= live ? static_cast<int>(p) : -1;
  }
  const int64_t mine[2] = {count_rest(holes, hole), count_rest(movers, mover)};
  Part* parts[2] = {&holes, &movers};
  prefixes(second, mine, parts);
  const int64_t none = int64_t{1} << 62;
  each(holes, none, hole, [&](int64_t, int p, int64_t r) { a.dst[r] = p; });
  each(movers, none, mover, [&](int64_t, int p, int64_t r) { a.src[r] = p; });
  if (threadIdx.x == 0 && cluster_rank() == 0) {
    *a.live = static_cast<int32_t>(live);
    *a.moves = static_cast<int32_t>(movers.total);
  }
  // Pages that stay keep their count (or their place in the map, behind `live`).
  for (int64_t i = all.lo + (threadIdx.x & 31); i < all.hi; i += 32 * kAhead) {
    int32_t n[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) n[k] = i + 32 * k < all.hi ? __ldcg(a.refs + i + 32 * k) : 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t p = i + 32 * k;
      if (p >= all.hi) break;
      if (p < live && n[k] != 0) a.refs_out[p] = n[k];
      if (p >= live && n[k] == 0) {
        a.refs_out[p] = 0;
        a.map[p] = static_cast<int32_t>(p);
      }
    }
  }
  cluster_sync();
  // As many holes as movers: the live pages before `live` and the holes are `live` many.
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x; k < movers.total;
       k += static_cast<int64_t>(gridDim.x) * kScanThreads) {
    const int32_t from = __ldcg(a.src + k), to = __ldcg(a.dst + k);
    const int32_t n = __ldcg(a.refs + from);
    a.refs_out[to] = n;
    a.refs_out[from] = 0;
    a.map[from] = to;
  }
}

// ------------------------------------------------------------------- copies

// CTAs an SM at most (half of 16384 pages of 128 KB live: with 3 or 5 of them
// compaction takes 7 or 2 us more; registers allow 3 at a time).
constexpr int kMoveThreads = 256, kMoveCtas = 8;
constexpr int kPieces = 8;               // of a lane, in flight

template <class T>
__device__ __forceinline__ void copy_chunk(uint8_t* to, const uint8_t* from, int64_t at, int64_t end) {
  const int lane = threadIdx.x & 31;
  T v[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t o = at + (k * 32 + lane) * static_cast<int64_t>(sizeof(T));
    if (o < end) v[k] = __ldcs(reinterpret_cast<const T*>(from + o));
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t o = at + (k * 32 + lane) * static_cast<int64_t>(sizeof(T));
    if (o < end) __stcs(reinterpret_cast<T*>(to + o), v[k]);
  }
}

// (The tables fall to the last CTAs first: the first ones have the copies.)
__device__ __forceinline__ void fork_rows(const MoveArgs& a) {
  const unsigned last = gridDim.x - 1 - blockIdx.x;
  const int64_t all = static_cast<int64_t>(a.pairs) * max(a.width, 1);
  int bits = 0;
  for (int64_t e = static_cast<int64_t>(last) * kMoveThreads + threadIdx.x; e < all;
       e += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
    const int k = static_cast<int>(e / max(a.width, 1)), c = static_cast<int>(e - static_cast<int64_t>(k) * max(a.width, 1));
    const int i = __ldcg(a.parents + k);
    int len = 0;
    if (i >= a.num_reqs) bits |= MM3IDX_DEV_BAD_ROWS;
    if (i >= 0 && i < a.num_reqs) {
      const int64_t raw = max(__ldcg(a.seq_lens + i), 0);
      const int64_t most = static_cast<int64_t>(a.width) * a.page_size;
      if (raw > most) bits |= MM3IDX_DEV_SEQ_TOO_LONG;
      len = static_cast<int>(min(raw, most));
    }
    if (c == 0) a.out_lens[k] = len;
    if (c >= a.width) continue;
    const int full = len / a.page_size;
    int32_t page = -1;
    if (c < full || (c == full && full * a.page_size < len)) {
      page = __ldcg(a.table + i * a.table_stride + c);
      if (page < 0 || page >= a.num_pages) {
        bits |= MM3IDX_DEV_BAD_PAGE;
        page = -1;
      } else if (c < full) {
        atomicAdd(a.refs + page, 1);
      } else {
        page = __ldcg(a.dst + k);
      }
    }
    a.out[k * a.out_stride + c] = page;
  }
  if (bits) atomicOr(a.status, bits);
}

__device__ __forceinline__ void mapped_rows(const MoveArgs& a) {
  const unsigned last = gridDim.x - 1 - blockIdx.x;
  const int64_t all = static_cast<int64_t>(a.num_reqs) * a.width;
  const int live = __ldcg(a.live);
  for (int64_t e = static_cast<int64_t>(last) * kMoveThreads + threadIdx.x; e < all;
       e += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
    const int64_t i = e / a.width, c = e - i * a.width;
    int32_t page = __ldcg(a.table + i * a.table_stride + c);
    if (page >= live && page < a.num_pages) page = __ldcg(a.map + page);
    a.out[i * a.out_stride + c] = page;
  }
}

// A warp's items are (pair, chunk of a page in one of the caches), chunks of a
// pair next to each other.
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ MoveArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t pairs = a.count ? __ldcg(a.count) : a.pairs;
  const int64_t items = pairs * a.chunks;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kMoveThreads / 32);
  int bits = 0;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
       w < items; w += warps) {
    const int64_t k = (w >> 32) == 0 ? static_cast<uint32_t>(w) / static_cast<uint32_t>(a.chunks)
                                     : w / a.chunks;
    const int chunk = static_cast<int>(w - k * a.chunks);
    const int from = __ldcg(a.src + k), to = __ldcg(a.dst + k);
    if (from < 0 || to < 0) continue;
    if (from >= a.num_pages || to >= a.num_pages) {
      bits |= MM3IDX_DEV_BAD_PAGE;
      continue;
    }
    int c = 0;
    while (chunk >= a.caches[c].end) ++c;
    const Cache& cache = a.caches[c];
    const int64_t at = static_cast<int64_t>(chunk - (c ? a.caches[c - 1].end : 0)) *
                       (kPieces * 32 * cache.unit);
    const int64_t end = min(at + kPieces * 32 * cache.unit, cache.page_bytes);
    const uint8_t* src = cache.data + from * cache.page_stride;
    uint8_t* dst = cache.data + to * cache.page_stride;
    if (cache.unit == 16) copy_chunk<uint4>(dst, src, at, end);
    else if (cache.unit == 4) copy_chunk<uint32_t>(dst, src, at, end);
    else copy_chunk<uint8_t>(dst, src, at, end);
  }
  if (bits && (threadIdx.x & 31) == 0) atomicOr(a.status, bits);
  if (a.parents) fork_rows(a);
  else if (a.map) mapped_rows(a);
}

__global__ void __launch_bounds__(kMoveThreads) release_kernel(const __grid_constant__ ReleaseArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t all = static_cast<int64_t>(a.num_reqs) * a.width;
  int bits = 0;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; e < all;
       e += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
    const int64_t i = e / a.width, c = e - i * a.width;
    if (a.seq_lens) {
      const int64_t len = max(__ldcg(a.seq_lens + i), 0);
      if (c >= (len + a.page_size - 1) / a.page_size) continue;
    }
    const int32_t page = __ldcg(a.table + i * a.table_stride + c);
    if (page < 0) continue;
    if (page >= a.num_pages) {
      bits |= MM3IDX_DEV_BAD_PAGE;
      continue;
    }
    // Below 0 it goes back up at once: exactly `count` of the releases find a
    // reference, in any order.
    if (atomicSub(a.refs + page, 1) <= 0) {
      atomicAdd(a.refs + page, 1);
      bits |= MM3IDX_DEV_NOT_HELD;
    }
  }
  if (bits) atomicOr(a.status, bits);
}

}  // namespace

// A small pool is scanned by one CTA (which does without the cluster's barriers and
// its list's way through global memory), others by a cluster.
template <class K>
cudaError_t launch_scan(K kernel, const ScanArgs& a, cudaStream_t s) {
  const int cluster = a.num_pages + a.items <= kSmall ? 1 : kCluster;
  return launch_dependent(kernel, dim3(cluster), kScanThreads, cluster, a, s);
}

cudaError_t launch_allocate(const ScanArgs& a, cudaStream_t s) {
  return launch_scan(claim_kernel<false>, a, s);
}

cudaError_t launch_fork_plan(const ScanArgs& a, cudaStream_t s) {
  return launch_scan(claim_kernel<true>, a, s);
}

cudaError_t launch_compact_plan(const ScanArgs& a, cudaStream_t s) {
  return launch_scan(plan_kernel, a, s);
}

// CTAs for the most items and table entries that there can be, as many as fit at
// most.
cudaError_t launch_move(const MoveArgs& a, int sms, cudaStream_t s) {
  const int64_t pairs = a.count ? a.num_pages / 2 : a.pairs;
  const int64_t rows = a.parents ? static_cast<int64_t>(a.pairs) * (a.width > 0 ? a.width : 1)
                       : a.map ? static_cast<int64_t>(a.num_reqs) * a.width : 0;
  const int64_t warps = kMoveThreads / 32;
  const int64_t ctas = (pairs * a.chunks + warps - 1) / warps + (rows + kMoveThreads - 1) / kMoveThreads;
  const int64_t most = static_cast<int64_t>(sms) * kMoveCtas;
  return launch_dependent(move_kernel, dim3(static_cast<unsigned>(ctas < 1 ? 1 : ctas < most ? ctas : most)),
                          kMoveThreads, 1, a, s);
}

cudaError_t launch_release(const ReleaseArgs& a, int sms, cudaStream_t s) {
  const int64_t all = static_cast<int64_t>(a.num_reqs) * a.width;
  const int64_t ctas = (all + kMoveThreads - 1) / kMoveThreads;
  return launch_dependent(release_kernel, dim3(static_cast<unsigned>(ctas < sms * 8 ? ctas : sms * 8)),
                          kMoveThreads, 1, a, s);
}

}  // namespace mm3idx
