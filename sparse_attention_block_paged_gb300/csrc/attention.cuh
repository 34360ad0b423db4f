// attention.cuh -- attention of a few new tokens a request over the paged
// key-value cache (include/mm3idx.h, mm3idx_paged_attention), one kernel per
// pair of types, head size and row count; the types' instances are compiled in
// attention_<types>.cu.
//
// Mathematics.  For a query row and the tokens it sees, taken in any order and
// any grouping, three numbers are enough: the reference m, the sum
// l = sum 2^(x_t - m) and the vector o = sum 2^(x_t - m) v_t, with
// x_t = scale log2(e) q.k_t.  Two such triples join to m = max(m1, m2),
// l = l1 2^(m1-m) + l2 2^(m2-m), o alike; the result is o / l, and
// m + log2 l is the (base 2) log-sum-exp.  A maximum passes over NaN, so scores
// that are all NaN (or all masked) leave m = -inf; l and o tell them apart, and
// every join carries them on: NaN times a factor of 0 is NaN.  Every warp keeps a triple of its
// own over its part of the tokens, CTAs join their warps' through shared
// memory, and a (request, kv head) that several CTAs share is joined by the
// last of them to finish, in a fixed order, so a result never depends on timing.
//
// What bounds it.  K and V of the visible tokens are read once: 4 D bytes a
// token in 16 bits against 4 D flops a query head, 2 to 16 flops a byte for
// the group sizes in use, far below what the tensor cores need: the kernel is
// a stream of pages from HBM.  So:
//
//   * Work partition.  The list of all (request, 128-token tile) is cut into
//     equal shares on the device, one a gang of CTAs, one CTA an SM; lengths
//     need no host round trip and cost no imbalance.  The CTAs of a gang walk
//     the same pages at the same time, each for its own kv head: a page whose
//     tokens hold all heads next to each other is then read from HBM in long
//     pieces (16 e4m3 requests of 32K-128K tokens, 4 heads of 128 bytes a
//     token: 326 us with each head's share elsewhere in time).  Where a gang
//     gets several requests, the list holds them dealt out in turns, so that
//     neighbours (rows of one request over their sparse tables, requests with a
//     common beginning) are read at about the same time and their common pages
//     once (64 requests x 4 rows, 64 heads, 16 selected blocks a row: 149 us,
//     165 in their own order; with 4 rows that select the same 129 and 162).
//   * Pages go through a ring of slots in shared memory (192 KB for 16-bit
//     D = 128: six slots of 128 tokens, keys and values in turn), filled with
//     4-D tiled TMA copies, so strides and page sizes cost nothing and about
//     three tiles are in flight.  Keys and values have a producer warp each:
//     a copy takes one about 50 ns to issue, and pages of 16 tokens are 16 of
//     them a tile (one request of 128K tokens, head_dim 64: 70 us with one
//     producer, 48 with two).
//   * Eight warps consume it.  The query rows of one kv head (group x
//     query_len) are rows of 16-row matrix products (mma.sync m16n8k16: up to
//     32 rows need less than that rate's half, and a warp that owns its scores
//     needs no exchange with others inside the loop).  A warp owns one of RT
//     16-row tiles and one part of the tokens: of every tile, or with few rows
//     of every second or fourth one, so that it has two or four 16-token
//     slices whose products interleave (one slice a warp: 1058 ns a tile from
//     L2 against 787).  Registers go from the other warps to these
//     (setmaxnreg).
//   * The reference m moves only when a score passes the largest so far by 8
//     (fp16 weights: 4), a factor that fp32 sums and 16-bit weights hold
//     without loss, so the accumulators are rarely rescaled.
//   * Weights for the second product are held as the sum of two 16-bit numbers
//     (one would cost an error as large as the output's own rounding; the
//     extra products hide behind the copies up to 32 rows).  Over e4m3 values
//     and for bf16 output one fp16 number is enough: its step is 1/8 of the
//     output's.
//   * e4m3 pages are widened to fp16 (exact) in registers.  The query is then
//     fp16 as well, scaled by a power of two so that its largest element is
//     in [1, 2): what this loses is below 2^-25 of that element.
//
// What it measured (GB300, tables and caches dealt at random; K and V bytes
// over the measured copy rate in brackets): 64 requests x 4 rows over 4K-32K
// tokens, 8 heads a kv head, bf16: 189 us (94 %); 16 x 32K-128K e4m3: 214 us
// (93 %); 64 x 4 rows of 16 selected blocks: 145 us; one request of 128K
// tokens, head_dim 64, pages of 16: 48 us (82 %; 9 us of it start and join);
// 8 x 128K: 310 us (100 %).  From L2 (no HBM) a 64 KB tile takes 0.80 us with
// up to 16 rows, 1.41 with 32 and 2.26 with 64, against 1.47 us at the HBM
// rate: 64 rows are bound by the products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "../../include/mm3idx.h"
#include "ptx.cuh"
#include "serving.h"

namespace mm3idx {
namespace attn {

constexpr int kConsumers = 8;                    // warps
constexpr int kProducer = kConsumers;            // warp of the keys' copies; the next: the values'
constexpr int kWeigher = kConsumers + 2;         // warp that writes the tiles' weights
constexpr int kSpare = kConsumers + 3;           // warp that sees to empty requests
constexpr int kThreads = (kConsumers + 4) * 32;  // three warpgroups
// Registers a thread: the launch's, and the split of them (setmaxnreg) between
// the consumers' two warpgroups and the third, whose sum is the launch's.
constexpr int kRegsLaunch = 168, kRegsConsumer = 216, kRegsOther = 72;
static_assert(2 * kRegsConsumer + kRegsOther == 3 * kRegsLaunch, "register split");
constexpr int kTile = kBlock;                    // tokens of a tile
constexpr int kRedStride = 40;                   // floats of a 32-column row in the join buffer
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int KV, int D>
struct Cfg {
  static constexpr bool kByte = KV == MM3IDX_TYPE_E4M3;
  static constexpr int kElem = kByte ? 1 : 2;
  static constexpr int kRow = D * kElem > 128 ? 128 : D * kElem;  // bytes of a row in a copy
  static constexpr int kHalves = D * kElem / kRow;                // copies of a page
  static constexpr int kHalf = kTile * kRow;
  static constexpr int kSlot = kHalves * kHalf;
  static constexpr int kSlots = kSlot == 32768 ? 6 : kSlot == 16384 ? 12 : 16;  // even: keys, values
  // Barriers per kind.  A slot that warps take turns at (every second tile is
  // one group's) has one barrier a group: a group that skips a slot's phase
  // cannot tell the phase before it from the phase after it by their parity.
  static constexpr int kBars = kSlots / 2 % 4 ? 2 * kSlots : kSlots;
  static constexpr uint32_t kSwizzle = kRow == 128 ? 0x70 : 0x30;
  static constexpr int oRed = kSlots * kSlot;
  static constexpr int oMl = oRed + kConsumers * 16 * kRedStride * 4;
  static constexpr int oFin = oMl + kConsumers * 16 * 8;
  static constexpr int oSlice = oFin + 64 * 8;
  static constexpr int oBar = oSlice + kSlots / 2 * kConsumers * 16 * 4;
  static constexpr int oMask = oBar + 3 * kBars * 8;
  static constexpr int oMisc = oMask + kSlots * 4;
  static constexpr int kSmem = oMisc + 128 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

template <int V>
struct Const {
  static constexpr int value = V;
};

// A gang's share [lo, hi) of the list of `total` positions that `grid` gangs
// share, its first and last task and their first positions.
struct Share {
  long long lo, hi, total, p0, pl;
  int t0, tl, grid;
};

struct Misc {
  Share share;
  int abort, last;
  long long scan[kConsumers];
};

__device__ __forceinline__ int request_len(const AttentionArgs& a, int i) {
  return min(max(__ldg(a.seq_lens + i), 0), a.max_seq_len);
}

// The CTAs of a gang are neighbours: x is the kv head that one works on, of the
// gang's, y the gang.
__device__ __forceinline__ int cta() {
  return static_cast<int>(blockIdx.y * gridDim.x + blockIdx.x);
}

// The request at place k of the list (see the work partition above).
__device__ __forceinline__ int dealt(const AttentionArgs& a, int k) {
  const int round = a.deal.quotient(k), turn = k - round * static_cast<int>(a.deal.d);
  return turn * a.deal_full + min(turn, a.deal_rest) + round;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Positions of one task (request, a gang's kv heads, 64-row tile) in the list.
__device__ __forceinline__ long long task_slots(int len) {
  return len > 0 ? tiles_of(len) + kTaskCost : 0;
}

// a / b of non-negative numbers, in 32 bits where they allow it (a 64-bit
// division takes several hundred cycles).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

__device__ __forceinline__ int length_bits(const AttentionArgs& a, int raw) {
  return (raw > a.max_seq_len ? MM3IDX_DEV_SEQ_TOO_LONG : 0) |
         (raw != 0 && raw < a.query_len ? MM3IDX_DEV_SEQ_TOO_SHORT : 0);
}

// This gang's bounds in a list of `total` positions.  No share is empty: at
// most one gang per kMinShare positions takes part.
__device__ __forceinline__ void bounds(const AttentionArgs& a, long long total, Share& s) {
  const long long most = total / kMinShare;
  const int gangs = static_cast<int>(gridDim.y);
  s.grid = static_cast<int>(most < 1 ? 1 : most < gangs ? most : gangs);
  const long long c = blockIdx.y;
  s.total = total;
  s.lo = c < s.grid ? quotient(total * c, s.grid) : 0;
  s.hi = c < s.grid ? quotient(total * (c + 1), s.grid) : 0;
}

// Up to 32 requests, one a lane, in a list that times the grid stays below
// 2^32: every warp finds the share by itself, without a barrier.
__device__ __forceinline__ Share share_of_few(const AttentionArgs& a, bool report) {
  const int lane = threadIdx.x & 31;
  const int raw = lane < a.num_reqs ? __ldg(a.seq_lens + dealt(a, lane)) : 0;
  const uint32_t one = static_cast<uint32_t>(task_slots(min(max(raw, 0), a.max_seq_len)));
  const uint32_t mine = one * static_cast<uint32_t>(a.tasks);
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (report) {
    const int bits = lane < a.num_reqs ? length_bits(a, raw) : 0;
    if (bits) atomicOr(a.status, bits);
  }
  const uint32_t total = __shfl_sync(0xffffffffu, incl, 31), before = incl - mine;
  const uint32_t grid = max(min(total / kMinShare, gridDim.y), 1u), c = blockIdx.y;
  const uint32_t lo = c < grid ? total * c / grid : 0, hi = c < grid ? total * (c + 1) / grid : 0;
  Share s;
  s.lo = lo;
  s.hi = hi;
  s.total = total;
  s.grid = static_cast<int>(grid);
  auto find = [&](uint32_t x, int& task, long long& pos) {
    const unsigned here = __ballot_sync(0xffffffffu, before <= x && x < incl);
    const uint32_t h = here >> lane & 1u ? (x - before) / one : 0;
    const int src = here ? __ffs(here) - 1 : 0;
    task = __shfl_sync(0xffffffffu, lane * a.tasks + static_cast<int>(h), src);
    pos = __shfl_sync(0xffffffffu, before + h * one, src);
  };
  find(lo, s.t0, s.p0);
  find(hi - 1, s.tl, s.pl);
  return s;
}

// Any number of requests, by the consumer threads, into shared memory.
__device__ __forceinline__ void share_of_many(const AttentionArgs& a, Misc* m) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.num_reqs + kConsumers * 32 - 1) / (kConsumers * 32);
  const int first = min(tid * per, a.num_reqs), end = min(first + per, a.num_reqs);
  long long mine = 0;
  int bits = 0;
  for (int i = first; i < end; ++i) {
    const int raw = __ldg(a.seq_lens + dealt(a, i));
    bits |= length_bits(a, raw);
    mine += task_slots(min(max(raw, 0), a.max_seq_len));
  }
  if (bits && cta() == 0) atomicOr(a.status, bits);
  mine *= a.tasks;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) m->scan[warp] = incl;
  consumer_sync();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kConsumers; ++w) {
    const long long s = m->scan[w];
    if (w < warp) before += s;
    total += s;
  }
  Share s;
  bounds(a, total, s);
  if (tid == 0) {
    m->share.lo = s.lo;
    m->share.hi = s.hi;
    m->share.total = s.total;
    m->share.grid = s.grid;
  }
  if (s.hi <= s.lo || mine == 0) return;
  const bool has_lo = before <= s.lo && s.lo < before + mine;
  const bool has_hi = before <= s.hi - 1 && s.hi - 1 < before + mine;
  if (!has_lo && !has_hi) return;
  long long P = before;
  for (int i = first; i < end; ++i) {
    const long long one = task_slots(request_len(a, dealt(a, i)));
    const long long all = one * a.tasks;
    if (has_lo && P <= s.lo && s.lo < P + all) {
      const int h = static_cast<int>(quotient(s.lo - P, one));
      m->share.t0 = i * a.tasks + h;
      m->share.p0 = P + h * one;
    }
    if (has_hi && P <= s.hi - 1 && s.hi - 1 < P + all) {
      const int h = static_cast<int>(quotient(s.hi - 1 - P, one));
      m->share.tl = i * a.tasks + h;
      m->share.pl = P + h * one;
    }
    P += all;
  }
}

// Lines of the lengths, the page table and the queries on their way to L2
// (one a lane of one warp in every CTA) while the kernel before this one ends:
// they are read again, as they then are, after it.
__device__ __forceinline__ void prefetch_inputs(const AttentionArgs& a) {
  const int64_t line = (static_cast<int64_t>(cta()) * 32 + (threadIdx.x & 31)) * 128;
  auto pull = [&](const void* p, int64_t bytes) {
    if (line < bytes)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + line));
  };
  pull(a.seq_lens, 4 * static_cast<int64_t>(a.num_reqs));
  pull(a.table, 4 * ((a.num_reqs - 1) * a.table_stride + a.table_width));
  if (a.q_tok > 0 && a.q_head <= a.q_tok)
    pull(a.q, 2 * ((static_cast<int64_t>(a.num_reqs) * a.query_len - 1) * a.q_tok + a.head_dim));
}

// One stretch of a CTA's share: tiles [b0, b1) of a task.
struct Segment {
  int req, len;
  int head, row0;      // this CTA's kv head, the first of its 64 rows
  int unit;            // index of (request, kv head, 64-row tile)
  int b0, b1, nb;
  int pos;             // the task's first position, from the share's start
};

// The stretches of the share, the two that other CTAs may share first.  (One
// copy of the code a role: four of them, inlined, took 168.5 us where this
// takes 164.5 over 256 rows of 16 selected blocks, and spilled registers.)
struct Walker {
  int size, p0, pl, P;         // positions from the share's start (2^31 tiles would take one CTA
  int t0, tl, t, stage;        // half an hour)
  __device__ explicit Walker(const Share& s)
      : size(static_cast<int>(s.hi - s.lo)), p0(static_cast<int>(s.p0 - s.lo)),
        pl(static_cast<int>(s.pl - s.lo)), P(0), t0(s.t0), tl(s.tl), t(0), stage(0) {}
  __device__ bool next(const AttentionArgs& a, Segment& s) {
    if (size <= 0) return false;
    for (;;) {
      const int step = stage;
      if (step < 2) stage = step + 1;
      else if (t >= tl) return false;
      if (step == 1 && tl == t0) continue;
      const int task = step == 0 ? t0 : step == 1 ? tl : t;
      const int pos = step == 0 ? p0 : step == 1 ? pl : P;
      const int place = a.by_tasks.quotient(task), sub = task - place * a.tasks;
      const int head = a.by_row_tiles.quotient(sub), tile = sub - head * a.row_tiles;
      s.req = dealt(a, place);
      s.head = head * a.gang + static_cast<int>(blockIdx.x);
      s.row0 = tile * 64;
      s.unit = (s.req * a.kv_heads + s.head) * a.row_tiles + tile;
      s.len = request_len(a, s.req);
      s.nb = tiles_of(s.len);
      s.pos = pos;
      if (step != 1) {
        t = task + 1;
        P = pos + static_cast<int>(task_slots(s.len));
      }
      const int pb = pos + kTaskCost, from = max(pb, 0), to = min(pb + s.nb, size);
      if (s.nb == 0 || to <= from) continue;
      s.b0 = from - pb;
      s.b1 = to - pb;
      return true;
    }
  }
};

// The gang whose share holds position x.
__device__ __forceinline__ int gang_of(long long x, long long total, int grid) {
  return static_cast<int>(quotient((x + 1) * grid - 1, total));
}

// Arrivals at a task: the count before this one, back to 0 after `wrap`.
__device__ __forceinline__ int ticket(unsigned int* p, unsigned int wrap) {
  unsigned int old;
  asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
               : "=r"(old)
               : "l"(p), "r"(wrap)
               : "memory");
  return static_cast<int>(old);
}

// ------------------------------------------------------------- instructions

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// D += A B: A 16x16 (row), B 16x8 (col), D 16x8 fp32.
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Every lane's view of a phase's end; the bounded wait where it is not there yet.
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats as a pair of 16-bit numbers (lo in the low half), and what the
// rounding left as a second pair.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2_rest(float lo, float hi, uint32_t packed) {
  float a, b;
  if constexpr (BF16) {
    a = __uint_as_float(packed << 16);
    b = __uint_as_float(packed & 0xffff0000u);
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&packed);
    a = __low2float(h);
    b = __high2float(h);
  }
  return pack2<BF16>(lo - a, hi - b);
}

// Two e4m3 numbers (the low 16 bits, or the high ones) as two fp16.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// The halves of a pair (tokens t and t + 1) that lie below `end`.
__device__ __forceinline__ uint32_t below(int t, int end) {
  return (t < end ? 0x0000ffffu : 0u) | (t + 1 < end ? 0xffff0000u : 0u);
}

// ------------------------------------------------------------------- kernel
//
// Fragments (thread t of a warp, c = t & 3, g = t >> 2).  Scores of 16 tokens:
// s[0], s[1] row g, tokens 2c, 2c+1; s[2], s[3] row g+8; s[4..7] the same for
// tokens 8+2c, 9+2c.  As the A operand of the second product they are, packed,
// in place.  16-bit caches: d runs in order; e4m3: the thread's 2 D/16 k-steps
// walk the D/4 bytes from c D/4 of a token's key (queries alike), and column n
// of output tile 4 t + i is d = 32 t + 4 n + i, so that a thread loads four
// neighbouring bytes of a value row.

template <int KV, int D>
struct State {
  float o[D / 8][4];
  float m0, m1, l0, l1;
};

// Q: type of the queries and the output.  KV: of the cache, Q or e4m3.
template <int Q, int KV, int D, int RT>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const AttentionArgs a) {
  using C = Cfg<KV, D>;
  constexpr int S = C::kSlots, NB = C::kBars;       // data slots; barriers (a multiple of them)
  constexpr bool kByte = C::kByte;
  constexpr bool kBf = KV == MM3IDX_TYPE_BF16;      // bf16 products (else fp16)
  constexpr bool kOutBf = Q == MM3IDX_TYPE_BF16;
  // The reference lies kHead (base 2) below the largest score at its last move
  // and moves again when a score is kRaise above that one: fp16 weights then
  // reach 2^15 and those down to 2^-36 of the largest still count.
  constexpr float kHead = kBf ? 0.0f : 11.0f, kRaise = kBf ? 8.0f : 4.0f;
  constexpr int TJ = kConsumers / RT;               // warps that share a row tile
  // A warp takes every ALT-th tile, so that it has 32 tokens of a tile with
  // 16-bit D = 128 and 64 where a tile is half the bytes (or RT = 4).
  constexpr int ALT = (C::kSlot == 32768 ? 2 : 4) / RT > 1 ? (C::kSlot == 32768 ? 2 : 4) / RT : 1;
  static_assert(NB / 2 % ALT == 0, "a barrier belongs to one group of warps");
  constexpr int TG = TJ / ALT;                      // token groups of a tile
  constexpr int NS = 8 / TG;                        // 16-token slices of a warp
  constexpr int NT = D / 8;                         // output tiles of 8 columns
  constexpr int KS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(sm + C::oRed);
  float2* ml = reinterpret_cast<float2*>(sm + C::oMl);     // [warp][16]
  float2* fin = reinterpret_cast<float2*>(sm + C::oFin);   // [row of the task]
  float* slice = reinterpret_cast<float*>(sm + C::oSlice); // [slot / 2][warp][16]
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::oBar);
  uint64_t* empty = full + NB;
  uint64_t* done = empty + NB;                             // values' barriers: the tile's weights are there
  uint32_t* mask = reinterpret_cast<uint32_t*>(sm + C::oMask);
  Misc* misc = reinterpret_cast<Misc*>(sm + C::oMisc);
  volatile int* abort_flag = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool weigh = a.tile_lse != nullptr;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NB; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumers / ALT + ((s & 1) && weigh ? 1 : 0));
      mbar_init(&done[s], kConsumers / ALT);
    }
    misc->abort = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == kProducer * 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == kSpare) prefetch_inputs(a);
  __syncthreads();
  // A programmatic dependent launch: what the kernel before it wrote is read
  // (and the workspace it used is written) only after this.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Share share;
  if (a.few) {
    share = share_of_few(a, cta() == 0 && warp == 0);
    if (threadIdx.x == 0) misc->share = share;    // for the joins, behind their barriers
  } else {
    if (warp < kConsumers) share_of_many(a, misc);
    __syncthreads();
    share = misc->share;
  }
  Walker walk(share);
  Segment sg;

  if (warp >= kConsumers) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp < kWeigher) {
      // ------------------------------------------- producers: keys, values
      const int kv = warp - kProducer;
      const CUtensorMap* map = kv ? &vmap : &kmap;
      const int per = kTile >> a.page_shift;       // pages of a tile
      const int batch = 32 * (1 << a.page_shift) / kTile;                  // tiles whose page ids one register holds
      const int box = C::kRow << a.page_shift;
      uint32_t slot = kv, bar = kv, items = 0;
      uint32_t wait = kv, wait_phase = 0;          // the barrier of the tile S / 2 before
      bool ok = true;
      while (ok && walk.next(a, sg)) {
        const int head = sg.head;
        const int32_t* table = a.table + static_cast<int64_t>(sg.req) * a.table_stride;
        const int pages = (sg.len + (1 << a.page_shift) - 1) >> a.page_shift;
        auto ids_from = [&](int p) { return p + lane < pages ? __ldg(table + p + lane) : -1; };
        int cur = ids_from(sg.b0 * per), nxt = ids_from(sg.b0 * per + 32), k = 0;
        for (int b = sg.b0; b < sg.b1; ++b, ++k) {
          if (k == batch) {
            k = 0;
            cur = nxt;
            nxt = ids_from(b * per + 32);
          }
          const int id = __shfl_sync(0xffffffffu, cur, (k * per + lane) & 31);
          const bool need = lane < per && b * per + lane < pages;
          const uint32_t good = __ballot_sync(0xffffffffu, need && id >= 0 && id < a.num_pages);
          if (__ballot_sync(0xffffffffu, need) != good && lane == 0)
            atomicOr(a.status, MM3IDX_DEV_BAD_PAGE);
          const int p = lane / C::kHalves, half = lane % C::kHalves;
          const int page = __shfl_sync(0xffffffffu, id, p);
          const bool issue = lane < per * C::kHalves && ((good >> p) & 1u);
          const uint32_t bytes = __popc(good) * C::kHalves * box;
          if (items >= S / 2) {
            ok = warp_wait(&empty[wait], wait_phase, abort_flag);
            if (!ok) break;
            wait += 2;
            if (wait >= NB) {
              wait = kv;
              wait_phase ^= 1;
            }
          }
          if (lane == 0) {
            if (kv == 0) mask[slot] = good;
            if (bytes) mbar_arrive_expect_tx(&full[bar], bytes);
            else mbar_arrive(&full[bar]);
          }
          __syncwarp();
          if (issue)
            tma_load_4d(smem_u32(sm) + slot * C::kSlot + half * C::kHalf + p * box, map, &full[bar],
                        half * (C::kRow / C::kElem), 0, head, page);
          ++items;
          slot += 2;
          if (slot >= S) slot = kv;
          bar += 2;
          if (bar >= NB) bar = kv;
        }
      }
      // Every copy that was started lands before the CTA can exit.
      if (lane == 0) {
        const uint32_t pending = items < S / 2 ? items : S / 2;
        for (uint32_t k = 0; k < pending; ++k) {
          const uint32_t idx = 2 * (items - 1 - k);
          int dummy = 0;
          mbar_wait(&full[idx % NB + kv], (idx / NB) & 1, &dummy);
        }
      }
      __syncwarp();
    } else if (warp == kWeigher) {
      // ------------------------------------- log-sum-exp of each tile's rows
      if (weigh) {
        uint32_t slot = 1, bar = 1, phase = 0, turn = 0;
        bool ok = true;
        while (ok && walk.next(a, sg)) {
          for (int b = sg.b0; b < sg.b1 && ok; ++b, turn = (turn + 1) % ALT) {
            ok = warp_wait(&done[bar], phase, abort_flag);
            if (!ok) break;
            const float* from = slice + ((slot >> 1) * kConsumers + turn * TG * RT) * 16;
            float* to = a.tile_lse + (static_cast<int64_t>(sg.unit) * a.w_width + b) * (RT * 16);
            for (int r = lane; r < RT * 16; r += 32) {
              float x[TG], top = -INFINITY, sum = 0.0f;
#pragma unroll
              for (int t = 0; t < TG; ++t) {
                x[t] = from[(t * RT + (r >> 4)) * 16 + (r & 15)];
                top = fmaxf(top, x[t]);
              }
              const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
              for (int t = 0; t < TG; ++t) sum += ex2(x[t] - ref);
              to[r] = ref + lg2(sum);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[bar]);
            slot += 2;
            if (slot > S) slot = 1;
            bar += 2;
            if (bar > NB) {
              bar = 1;
              phase ^= 1;
            }
          }
        }
      }
    } else if (warp == kSpare) {
      // ------------------------------------------- rows of empty requests
      // (a request's rows dealt out to the CTAs where there are fewer requests:
      // one CTA takes seconds for 2^20 rows of 128 heads)
      const int heads = a.kv_heads * a.group;
      const int64_t pieces = static_cast<int64_t>(heads) * (D / 8);   // of a row, 16 bytes each
      const int ctas = static_cast<int>(gridDim.x * gridDim.y);
      const int share = a.num_reqs < ctas ? ctas / a.num_reqs : 1;
      for (int i = cta() / share; i < a.num_reqs; i += ctas / share) {
        if (request_len(a, i) > 0) continue;
        for (int j = cta() % share; j < a.query_len; j += share) {
          const int64_t row = static_cast<int64_t>(i) * a.query_len + j;
          for (int64_t e = lane; e < pieces; e += 32) {
            const int h = static_cast<int>(e / (D / 8)), d = static_cast<int>(e % (D / 8)) * 8;
            uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.o_tok + h * a.o_head + d;
            *reinterpret_cast<uint4*>(out) = make_uint4(0, 0, 0, 0);
            if (d == 0) {
              if (a.lse) a.lse[row * a.lse_tok + h] = -INFINITY;
              if (weigh) a.row_lse[row * heads + h] = -INFINITY;
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsConsumer));
    // ---------------------------------------------------------- consumers
    const int c = lane & 3, g = lane >> 2;
    const int rt = warp % RT, tj = warp / RT, tg = tj % TG, alt = tj / TG;
    const uint32_t ring = smem_u32(sm);
    State<KV, D> st;
    uint32_t slot = 0, bar = 0, phase = 0, turn = 0;
    bool dead = false;       // a wait gave up: go through the motions to the end
    // Weights as pairs.  (Known to the compiler: the second numbers' registers and
    // instructions, unused, cost the e4m3 batch above 236 us instead of 223.)
    constexpr bool rest = !kByte || Q == MM3IDX_TYPE_FP16;

    // Offsets of this lane in a slot for slice 0 of its tokens.  A 16-byte
    // piece p of a row lies at p xor (row mod 8) (swizzled copies); slices and
    // k-steps only add rows or flip bits of p, so the rest are constants.
    auto twisted = [](uint32_t off) { return off ^ ((off >> 3) & C::kSwizzle); };
    const uint32_t first = tg * NS * 16;
    uint32_t koff, voff0, voff1 = 0;
    if constexpr (!kByte) {
      koff = twisted((first + ((lane >> 4) << 3) + (lane & 7)) * C::kRow + ((lane >> 3) & 1) * 16);
      voff0 = twisted((first + (lane & 15)) * C::kRow + (lane >> 4) * 16);
    } else {
      koff = twisted((first + g) * C::kRow + c * (D / 4));
      voff0 = twisted((first + 2 * c) * C::kRow + g * 4);
      voff1 = twisted((first + 2 * c + 1) * C::kRow + g * 4);
    }

    const int R = a.group * a.query_len;
    // The queries of a segment, as they lie in memory: 16-bit caches, the A
    // operands; e4m3, D/4 elements from c D/4 of rows g and g + 8.
    uint32_t q[KS][4];
    auto load_queries = [&](const Segment& s) {
      const int ra = s.row0 + rt * 16 + g, rb = ra + 8;
      const uint16_t* base = static_cast<const uint16_t*>(a.q) +
                             static_cast<int64_t>(s.req) * a.query_len * a.q_tok +
                             static_cast<int64_t>(s.head) * a.group * a.q_head;
      auto row_at = [&](int r) {
        r = min(r, R - 1);
        const int j = a.by_group.quotient(r);
        return base + j * a.q_tok + (r - j * a.group) * a.q_head;
      };
      const uint16_t* qa = row_at(ra);
      const uint16_t* qb = row_at(rb);
      const bool va = ra < R, vb = rb < R;
      if constexpr (!kByte) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int d = ks * 16 + 2 * c;
          q[ks][0] = va ? __ldg(reinterpret_cast<const uint32_t*>(qa + d)) : 0u;
          q[ks][1] = vb ? __ldg(reinterpret_cast<const uint32_t*>(qb + d)) : 0u;
          q[ks][2] = va ? __ldg(reinterpret_cast<const uint32_t*>(qa + d + 8)) : 0u;
          q[ks][3] = vb ? __ldg(reinterpret_cast<const uint32_t*>(qb + d + 8)) : 0u;
        }
      } else {
#pragma unroll
        for (int u = 0; u < KS / 2; ++u) {
          const uint4 none = make_uint4(0, 0, 0, 0);
          const uint4 x = va ? __ldg(reinterpret_cast<const uint4*>(qa + c * (D / 4)) + u) : none;
          const uint4 y = vb ? __ldg(reinterpret_cast<const uint4*>(qb + c * (D / 4)) + u) : none;
          q[2 * u][0] = x.x; q[2 * u][1] = y.x; q[2 * u][2] = x.y; q[2 * u][3] = y.y;
          q[2 * u + 1][0] = x.z; q[2 * u + 1][1] = y.z; q[2 * u + 1][2] = x.w; q[2 * u + 1][3] = y.w;
        }
      }
    };

    bool more = walk.next(a, sg);
    if (more) load_queries(sg);
    while (more) {
      const int head = sg.head, row0 = sg.row0;
      const int rows = min(64, R - row0);                  // of this task
      const int64_t tok0 = static_cast<int64_t>(sg.req) * a.query_len;
      // Row r of the kv head is query token r / group, query head r % group.
      const int ra = row0 + rt * 16 + g, rb = ra + 8;
      const int ja = a.by_group.quotient(min(ra, R - 1)), jb = a.by_group.quotient(min(rb, R - 1));
      const int shift = sg.len - a.query_len + 1;          // query token j sees [0, shift + j)
      const int j_lo = a.by_group.quotient(min(row0 + rt * 16, R - 1));
      const int j_hi = a.by_group.quotient(min(row0 + rt * 16 + 15, R - 1));
      const int lim_a = shift + ja, lim_b = shift + jb;
      const int lim_lo = shift + j_lo, lim_hi = shift + j_hi;
      const bool idle = row0 + rt * 16 >= R;               // no row of this 16-row tile

      float sc_a = a.scale * kLog2e, sc_b = sc_a;
      if constexpr (kByte) {
        // fp16 queries, each row scaled by the power of two that brings its
        // largest element into [1, 2) (not at all where that is 0).  The factor of
        // the scores stays finite and normal: infinity and 0 would make NaN of a
        // score of 0 and of a masked one's -inf.
        float top[2] = {0.0f, 0.0f}, down[2];
        auto floats = [&](uint32_t w) {
          if constexpr (kOutBf)
            return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
          return __half22float2(*reinterpret_cast<const __half2*>(&w));
        };
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = floats(q[ks][e]);
            top[e & 1] = max3(top[e & 1], fabsf(f.x), fabsf(f.y));
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
          const int e = min(static_cast<int>(__float_as_uint(top[x]) >> 23), 253);
          down[x] = e == 0 ? 1.0f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
          const float up = e == 0 ? 1.0f : __uint_as_float(static_cast<uint32_t>(e) << 23);
          if (x) sc_b = fminf(fmaxf(sc_b * up, FLT_MIN), FLT_MAX);
          else sc_a = fminf(fmaxf(sc_a * up, FLT_MIN), FLT_MAX);
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = floats(q[ks][e]);
            q[ks][e] = pack2<false>(f.x * down[e & 1], f.y * down[e & 1]);
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[n][e] = 0.0f;
      st.m0 = st.m1 = -INFINITY;
      st.l0 = st.l1 = 0.0f;

      for (int b = sg.b0; b < sg.b1; ++b) {
        auto next_slot = [&] {      // to the next tile's keys
          if (++slot >= S) slot = 0;
          if (++bar >= NB) {
            bar = 0;
            phase ^= 1;
          }
        };
        if constexpr (ALT > 1) {
          const bool mine = turn == alt;
          turn = (turn + 1) % ALT;
          if (!mine) {
            ++slot;
            ++bar;
            next_slot();
            continue;
          }
        }
        // ------------------------------------------------------- scores
        if (!dead) dead = !all_wait(&full[bar], phase, abort_flag);
        const bool live = !idle && !dead;
        const uint32_t pages = mask[slot];
        const int t0 = b * kTile + static_cast<int>(first);
        // Whether every row sees every token of this warp's part.
        const bool inside = t0 + NS * 16 <= lim_lo &&
                            pages == (0xffffffffu >> (32 - (kTile >> a.page_shift)));
        float s[NS][2][4];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.0f;
        if (live) {
          // All slices at once: 2 NS chains of products.  What lies behind the
          // last token may be anything; its scores are replaced below.
          const uint32_t kbase = ring + slot * C::kSlot + koff;
          if constexpr (!kByte) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              uint32_t r[NS][4];
#pragma unroll
              for (int n = 0; n < NS; ++n)
                ldmatrix4((kbase ^ ((2 * ks & 7) << 4)) + (ks >> 2) * C::kHalf + n * 16 * C::kRow,
                          r[n]);
#pragma unroll
              for (int n = 0; n < NS; ++n) {
                mma<kBf>(s[n][0], q[ks], r[n][0], r[n][1]);
                mma<kBf>(s[n][1], q[ks], r[n][2], r[n][3]);
              }
            }
          } else {
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
              uint4 w[NS][2];
#pragma unroll
              for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  w[n][x] = lds128((kbase ^ (16 * u)) + (n * 16 + 8 * x) * C::kRow);
#pragma unroll
              for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint32_t k4 = e == 0 ? w[n][x].x : e == 1 ? w[n][x].y
                                        : e == 2 ? w[n][x].z : w[n][x].w;
                    mma<false>(s[n][x], q[u * 4 + e], widen_lo(k4), widen_hi(k4));
                  }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[bar]);
        ++slot;      // the values' (both counts are even)
        ++bar;

        // ------------------------------------------------------ softmax
        uint32_t act = (1u << NS) - 1u;          // slices with a token that some row sees
        if (!inside || !live) {
          // tokens that a row does not see: -inf before the (positive) scale
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            const bool on = live && t0 + n * 16 < lim_hi &&
                            ((pages >> ((first + n * 16) >> a.page_shift)) & 1u);
            if (!on) act &= ~(1u << n);
            const int t = t0 + n * 16 + 2 * c;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!on || t + 8 * x + (e & 1) >= (e < 2 ? lim_a : lim_b)) s[n][x][e] = -INFINITY;
          }
        }
        float top_a = -INFINITY, top_b = -INFINITY;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            top_a = max3(top_a, s[n][x][0], s[n][x][1]);
            top_b = max3(top_b, s[n][x][2], s[n][x][3]);
          }
        top_a *= sc_a;
        top_b *= sc_b;
        if (__any_sync(0xffffffffu, top_a > st.m0 + kHead + kRaise || top_b > st.m1 + kHead + kRaise)) {
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            top_a = fmaxf(top_a, __shfl_xor_sync(0xffffffffu, top_a, o));
            top_b = fmaxf(top_b, __shfl_xor_sync(0xffffffffu, top_b, o));
          }
          const float na = fmaxf(st.m0, top_a - kHead), nb = fmaxf(st.m1, top_b - kHead);
          const float fa = na == -INFINITY ? 0.0f : ex2(st.m0 - na);
          const float fb = nb == -INFINITY ? 0.0f : ex2(st.m1 - nb);
          st.m0 = na;
          st.m1 = nb;
          st.l0 *= fa;
          st.l1 *= fb;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            st.o[n][0] *= fa;
            st.o[n][1] *= fa;
            st.o[n][2] *= fb;
            st.o[n][3] *= fb;
          }
        }
        const float ref_a = st.m0 == -INFINITY ? 0.0f : st.m0;
        const float ref_b = st.m1 == -INFINITY ? 0.0f : st.m1;
        uint32_t p[NS][4], pr[NS][4];
        float sum_a = 0.0f, sum_b = 0.0f;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float w0 = ex2(fmaf(s[n][x][0], sc_a, -ref_a));
            const float w1 = ex2(fmaf(s[n][x][1], sc_a, -ref_a));
            const float w2 = ex2(fmaf(s[n][x][2], sc_b, -ref_b));
            const float w3 = ex2(fmaf(s[n][x][3], sc_b, -ref_b));
            sum_a += w0 + w1;
            sum_b += w2 + w3;
            p[n][2 * x] = pack2<kBf>(w0, w1);
            p[n][2 * x + 1] = pack2<kBf>(w2, w3);
            if (rest) {
              pr[n][2 * x] = pack2_rest<kBf>(w0, w1, p[n][2 * x]);
              pr[n][2 * x + 1] = pack2_rest<kBf>(w2, w3, p[n][2 * x + 1]);
            }
          }
        st.l0 += sum_a;
        st.l1 += sum_b;

        // ------------------------------------------------------- values
        if (!dead) dead = !all_wait(&full[bar], phase, abort_flag);
        const uint32_t vbase = ring + slot * C::kSlot;
        if (weigh) {
          // (the values' arrival says that the slot's last weights were read)
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            sum_a += __shfl_xor_sync(0xffffffffu, sum_a, o);
            sum_b += __shfl_xor_sync(0xffffffffu, sum_b, o);
          }
          if (c == 0) {
            float* to = slice + ((slot >> 1) * kConsumers + warp) * 16;
            to[g] = ref_a + lg2(sum_a);
            to[g + 8] = ref_b + lg2(sum_b);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&done[bar]);
        }
        // B operands of output tiles 2u, 2u+1 (16-bit) or 4u .. 4u+3 (e4m3),
        // 16 tokens from row `at` of this warp's part
        constexpr int TU = kByte ? 4 : 2, NU = NT / TU, UG = kByte ? 2 : 4;
        auto load_v = [&](int u, int at, uint32_t(&r)[2 * TU]) {
          if constexpr (!kByte) {
            ldmatrix4_trans(((vbase + voff0) ^ ((2 * u & 7) << 4)) + (u >> 2) * C::kHalf +
                                at * C::kRow, r);
          } else {
            const uint32_t even = (vbase + voff0) ^ (u * 32), odd = (vbase + voff1) ^ (u * 32);
            uint32_t w[4];
            w[0] = lds32(even + at * C::kRow);
            w[1] = lds32(odd + at * C::kRow);
            w[2] = lds32(even + (at + 8) * C::kRow);
            w[3] = lds32(odd + (at + 8) * C::kRow);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t x = __byte_perm(w[2 * k], w[2 * k + 1], 0x5140);
              const uint32_t y = __byte_perm(w[2 * k], w[2 * k + 1], 0x7362);
              r[0 + k] = widen_lo(x);
              r[2 + k] = widen_hi(x);
              r[4 + k] = widen_lo(y);
              r[6 + k] = widen_hi(y);
            }
          }
        };
        if (live && inside) {
          // Two slices and UG loads at a time, products on one accumulator
          // eight apart.
#pragma unroll
          for (int n = 0; n < NS; n += 2)
#pragma unroll
            for (int u0 = 0; u0 < NU; u0 += UG) {
              uint32_t r[2][UG][2 * TU];
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int u = 0; u < UG; ++u) load_v(u0 + u, (n + x) * 16, r[x][u]);
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int u = 0; u < UG; ++u)
#pragma unroll
                  for (int k = 0; k < TU; ++k)
                    mma<kBf>(st.o[(u0 + u) * TU + k], p[n + x], r[x][u][2 * k], r[x][u][2 * k + 1]);
              if (rest) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                  for (int u = 0; u < UG; ++u)
#pragma unroll
                    for (int k = 0; k < TU; ++k)
                      mma<kBf>(st.o[(u0 + u) * TU + k], pr[n + x], r[x][u][2 * k],
                               r[x][u][2 * k + 1]);
              }
            }
        } else if (live) {
          // The last tokens, or a page outside the cache: values that a row
          // does not see do not meet its weights (0 times NaN), so the rows of
          // each query token take their product with the values behind its
          // limit zeroed.
#pragma unroll 1
          for (int n = 0; n < NS; ++n) {
            if (!((act >> n) & 1u)) continue;
            uint32_t pn[4], prn[4] = {0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < NS; ++x)
              if (x == n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  pn[e] = p[x][e];
                  if (rest) prn[e] = pr[x][e];
                }
              }
            const int t = t0 + n * 16 + 2 * c;
#pragma unroll 1
            for (int j = j_lo; j <= j_hi; ++j) {
              const int end = shift + j;
              const uint32_t k0 = below(t, end), k1 = below(t + 8, end);
#pragma unroll
              for (int u = 0; u < NU; ++u) {
                uint32_t r[2 * TU];
                load_v(u, n * 16, r);
#pragma unroll
                for (int k = 0; k < TU; ++k) {
                  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma<kBf>(x, pn, r[2 * k] & k0, r[2 * k + 1] & k1);
                  if (rest) mma<kBf>(x, prn, r[2 * k] & k0, r[2 * k + 1] & k1);
                  if (ja == j) {
                    st.o[u * TU + k][0] += x[0];
                    st.o[u * TU + k][1] += x[1];
                  }
                  if (jb == j) {
                    st.o[u * TU + k][2] += x[2];
                    st.o[u * TU + k][3] += x[3];
                  }
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[bar]);
        next_slot();
      }
      // The next segment's queries are under way during the join.
      Segment after;
      more = walk.next(a, after);
      if (more) load_queries(after);

      // ------------------------------------------------ join of the warps
      // Quad sums of l, then the warps' triples through shared memory, 32
      // columns at a time: the result, or this CTA's partial one.
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, o);
        st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, o);
      }
      const bool whole = sg.b0 == 0 && sg.b1 == sg.nb;
      if (c == 0) {
        ml[warp * 16 + g] = make_float2(st.m0, st.l0);
        ml[warp * 16 + g + 8] = make_float2(st.m1, st.l1);
      }
      consumer_sync();
      float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
      for (int t = 0; t < TJ; ++t) {
        ma = fmaxf(ma, ml[(t * RT + rt) * 16 + g].x);
        mb = fmaxf(mb, ml[(t * RT + rt) * 16 + g + 8].x);
      }
      const float fa = ma == -INFINITY ? 0.0f : ex2(st.m0 - ma);
      const float fb = mb == -INFINITY ? 0.0f : ex2(st.m1 - mb);
      const int64_t part = 2 * cta() + (sg.pos > 0 ? 1 : 0);
      const int heads = a.kv_heads * a.group;
      if (threadIdx.x < RT * 16) {
        const int r = threadIdx.x;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int t = 0; t < TJ; ++t) top = fmaxf(top, ml[(t * RT + (r >> 4)) * 16 + (r & 15)].x);
#pragma unroll
        for (int t = 0; t < TJ; ++t) {
          const float2 x = ml[(t * RT + (r >> 4)) * 16 + (r & 15)];
          sum += top == -INFINITY ? x.y : x.y * ex2(x.x - top);
        }
        if (r < rows) {
          if (whole) {
            const int j = a.by_group.quotient(row0 + r);
            const int64_t row = tok0 + j;
            const int h = head * a.group + row0 + r - j * a.group;
            const float lse2 = sum == 0.0f ? -INFINITY : top + lg2(sum);
            if (a.lse) a.lse[row * a.lse_tok + h] = lse2 * kLn2;
            if (weigh) a.row_lse[row * heads + h] = lse2;
          } else {
            __stcg(a.part_ml + part * 64 + r, make_float2(top, sum));
          }
        }
        fin[r].x = sum == 0.0f ? 0.0f : a.v_scale / sum;
      }
      // This thread's two columns of rows q2 * 16 + tid / 16.
      uint16_t* out_at[RT];
#pragma unroll
      for (int q2 = 0; q2 < RT; ++q2) {
        const int r = min(q2 * 16 + static_cast<int>(threadIdx.x >> 4), rows - 1);
        const int j = a.by_group.quotient(row0 + r);
        out_at[q2] = static_cast<uint16_t*>(a.out) + (tok0 + j) * a.o_tok +
                     (head * a.group + row0 + r - j * a.group) * a.o_head + (threadIdx.x & 15) * 2;
      }
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        float* mine = red + warp * 16 * kRedStride;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          if (u != ch) continue;             // static register indices
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float(&o)[4] = st.o[u * 4 + k];
            if constexpr (!kByte) {
              *reinterpret_cast<float2*>(mine + g * kRedStride + 8 * k + 2 * c) =
                  make_float2(o[0] * fa, o[1] * fa);
              *reinterpret_cast<float2*>(mine + (g + 8) * kRedStride + 8 * k + 2 * c) =
                  make_float2(o[2] * fb, o[3] * fb);
            } else {
              mine[g * kRedStride + 8 * c + k] = o[0] * fa;
              mine[g * kRedStride + 8 * c + 4 + k] = o[1] * fa;
              mine[(g + 8) * kRedStride + 8 * c + k] = o[2] * fb;
              mine[(g + 8) * kRedStride + 8 * c + 4 + k] = o[3] * fb;
            }
          }
        }
        consumer_sync();
#pragma unroll
        for (int q2 = 0; q2 < RT; ++q2) {
          const int r = q2 * 16 + (threadIdx.x >> 4), col = (threadIdx.x & 15) * 2;
          if (r >= rows) continue;
          float2 v[TJ];
#pragma unroll
          for (int t = 0; t < TJ; ++t)
            v[t] = *reinterpret_cast<const float2*>(
                red + ((t * RT + q2) * 16 + (threadIdx.x >> 4)) * kRedStride + col);
          float x = 0.0f, y = 0.0f;
#pragma unroll
          for (int t = 0; t < TJ; ++t) {
            x += v[t].x;
            y += v[t].y;
          }
          if (whole) {
            const float f = fin[r].x;
            *reinterpret_cast<uint32_t*>(out_at[q2] + ch * 32) =
                pack2<kOutBf>(x * f, y * f);
          } else {
            __stcg(reinterpret_cast<float2*>(a.part_o + (part * 64 + r) * D + ch * 32 + col),
                   make_float2(x, y));
          }
        }
        consumer_sync();
      }
      if (!whole) {
        // Publish; the last CTA of the task joins the partial results.  (The
        // barrier orders the CTA's stores before thread 0's release.)  The ticket
        // is the one of the CTA that has the task's first tile: only one task
        // goes on past the end of its share.
        const long long pos = misc->share.lo + sg.pos, pb = pos + kTaskCost;
        const int lead = gang_of(pb, misc->share.total, misc->share.grid);
        const int parts = gang_of(pb + sg.nb - 1, misc->share.total, misc->share.grid) - lead + 1;
        if (threadIdx.x == 0)
          misc->last = !dead && ticket(a.tickets + lead * a.gang + static_cast<int>(blockIdx.x),
                                       parts - 1) == parts - 1;
        consumer_sync();
        if (misc->last) {
          // Four columns of a row are a unit.  A thread takes up to UB units, their
          // partial results in order, UB x PB = 16 loads in flight.
          constexpr int kStride = kConsumers * 32;
          const int member = static_cast<int>(blockIdx.x);
          const bool second = pos > quotient(misc->share.total * lead, misc->share.grid);
          const int units = rows * (D / 4);
          auto gather = [&](auto ub, auto pb, int u0, int t_first, int t_step, float* m, float* l,
                            float4* o) {
            constexpr int UB = decltype(ub)::value, PB = decltype(pb)::value;
#pragma unroll
            for (int u = 0; u < UB; ++u) {
              m[u] = -INFINITY;
              l[u] = 0.0f;
              o[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll 1
            for (int t0 = t_first; t0 < parts; t0 += t_step) {
              float2 x[UB][PB];
              float4 v[UB][PB];
#pragma unroll
              for (int k = 0; k < PB; ++k) {
                const int64_t at = 2 * static_cast<int64_t>((lead + t0 + k) * a.gang + member) +
                                   (t0 + k == 0 && second);
#pragma unroll
                for (int u = 0; u < UB; ++u) {
                  const int unit = u0 + u * kStride;
                  x[u][k] = make_float2(-INFINITY, 0.0f);
                  v[u][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                  if (t0 + k < parts && unit < units) {
                    x[u][k] = __ldcg(a.part_ml + at * 64 + unit / (D / 4));
                    v[u][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * 64 * D) + unit);
                  }
                }
              }
#pragma unroll
              for (int u = 0; u < UB; ++u) {
                float top = m[u];
#pragma unroll
                for (int k = 0; k < PB; ++k) top = fmaxf(top, x[u][k].x);
                const float ref = top == -INFINITY ? 0.0f : top;
                const float f = ex2(m[u] - ref);
                m[u] = top;
                l[u] *= f;
                o[u].x *= f; o[u].y *= f; o[u].z *= f; o[u].w *= f;
#pragma unroll
                for (int k = 0; k < PB; ++k) {
                  const float w = ex2(x[u][k].x - ref);
                  l[u] += x[u][k].y * w;
                  o[u].x += v[u][k].x * w; o[u].y += v[u][k].y * w;
                  o[u].z += v[u][k].z * w; o[u].w += v[u][k].w * w;
                }
              }
            }
          };
          auto finish = [&](int unit, float m, float l, float4 o) {
            const int r = unit / (D / 4), col = unit % (D / 4) * 4;
            const int j = a.by_group.quotient(row0 + r);
            const int64_t row = tok0 + j;
            const int h = head * a.group + row0 + r - j * a.group;
            const float f = l == 0.0f ? 0.0f : a.v_scale / l;
            const uint2 w =
                make_uint2(pack2<kOutBf>(o.x * f, o.y * f), pack2<kOutBf>(o.z * f, o.w * f));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.o_tok + h * a.o_head +
                                      col) = w;
            if (col == 0) {
              const float lse2 = l == 0.0f ? -INFINITY : m + lg2(l);
              if (a.lse) a.lse[row * a.lse_tok + h] = lse2 * kLn2;
              if (weigh) a.row_lse[row * heads + h] = lse2;
            }
          };
          if (units > kStride) {
            constexpr int UB = 4;
#pragma unroll 1
            for (int u0 = threadIdx.x; u0 < units; u0 += UB * kStride) {
              float m[UB], l[UB];
              float4 o[UB];
              gather(Const<UB>{}, Const<4>{}, u0, 0, 4, m, l, o);
#pragma unroll
              for (int u = 0; u < UB; ++u)
                if (u0 + u * kStride < units) finish(u0 + u * kStride, m[u], l[u], o[u]);
            }
          } else {
            // Few columns: with many parts `turns` threads a unit, every
            // turns-th eight parts each, joined through shared memory in order.
            const int split = parts <= 8 || units > kStride / 2 ? 0 : units > kStride / 4 ? 1 : 2;
            const int turns = 1 << split, each = kStride >> split;
            const int unit = threadIdx.x & (each - 1), turn = threadIdx.x * turns / kStride;
            float m, l;
            float4 o;
            gather(Const<1>{}, Const<8>{}, unit, turn * 8, turns * 8, &m, &l, &o);
            if (turns > 1) {
              float* mine = red + threadIdx.x * 6;
              mine[0] = m; mine[1] = l; mine[2] = o.x; mine[3] = o.y; mine[4] = o.z; mine[5] = o.w;
              consumer_sync();
              for (int t = 1; t < turns && turn == 0; ++t) {
                const float* from = red + (t * each + unit) * 6;
                const float top = fmaxf(m, from[0]), ref = top == -INFINITY ? 0.0f : top;
                const float f = ex2(m - ref), w = ex2(from[0] - ref);
                m = top;
                l = l * f + from[1] * w;
                o.x = o.x * f + from[2] * w; o.y = o.y * f + from[3] * w;
                o.z = o.z * f + from[4] * w; o.w = o.w * f + from[5] * w;
              }
              consumer_sync();      // `red` is free again
            }
            if (turn == 0 && unit < units) finish(unit, m, l, o);
          }
        }
      }
      sg = after;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && misc->abort) atomicOr(a.status, MM3IDX_DEV_TIMEOUT);
}

template <int Q, int KV, int D, int RT>
cudaError_t launch_rt(const CUtensorMap& kmap, const CUtensorMap& vmap, const AttentionArgs& a,
                      int grid, cudaStream_t s) {
  using C = Cfg<KV, D>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    // The register split waits for what the launch does not have: never
    // launch a build that got fewer.
    cudaFuncAttributes at;
    const cudaError_t err = cudaFuncGetAttributes(&at, attention_kernel<Q, KV, D, RT>);
    if (err != cudaSuccess) return err;
    if (at.numRegs < kRegsLaunch) return cudaErrorLaunchOutOfResources;
    return cudaFuncSetAttribute(attention_kernel<Q, KV, D, RT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.gang, grid / a.gang);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_kernel<Q, KV, D, RT>, kmap, vmap, a);
}

template <int Q, int KV, int D>
cudaError_t launch_d(const CUtensorMap& kmap, const CUtensorMap& vmap, const AttentionArgs& a,
                     int grid, cudaStream_t s) {
  const int tiles = attention_row_tiles16(a.group * a.query_len);
  if (tiles == 1) return launch_rt<Q, KV, D, 1>(kmap, vmap, a, grid, s);
  if (tiles == 2) return launch_rt<Q, KV, D, 2>(kmap, vmap, a, grid, s);
  return launch_rt<Q, KV, D, 4>(kmap, vmap, a, grid, s);
}

template <int Q, int KV>
cudaError_t launch_kv(const CUtensorMap& kmap, const CUtensorMap& vmap, const AttentionArgs& a,
                      int grid, cudaStream_t s) {
  return a.head_dim == 128 ? launch_d<Q, KV, 128>(kmap, vmap, a, grid, s)
                           : launch_d<Q, KV, 64>(kmap, vmap, a, grid, s);
}

}  // namespace attn
}  // namespace mm3idx
