// append.cu -- new tokens' keys and values into their requests' pages
// (include/mm3idx.h, mm3idx_append_kv).
//
// Mathematics.  y = x / k_scale.  With a scale a page and head: A = max |y| of the
// page's finite new elements, need = the least power of two with A / need <= 448;
// the scale S is need in a page that starts with them, else max(need, old S).
// Codes are y / S to the nearest e4m3.  A power of two costs no precision (e4m3
// is a floating type) but at most one of its 18 binades, and makes growing
// exact: older codes times old / new only move their exponents, until they
// meet e4m3's subnormals.
//
// What bounds it.  2 bytes read and 1 (2) written an element: HBM for prompts,
// for a decode step a chain of dependent loads (length, page, old scale).  So a
// (page, head) of the keys or of the values is one group of threads' that holds
// its new elements in registers between the maximum and the rounding: one pass
// over the data, nothing exchanged between CTAs.  Elements are asked for as soon as
// the length is known, before the page table; what is rare (an infinity, an old
// scale that is no power of two) reads them again instead of holding registers.
//
// What it measured (GB300, calls captured in a CUDA graph): four prompts of 8192 tokens,
// 8 heads of 128, into e4m3 pages of 64: 32 us (92 % of the measured copy rate; with the
// page first, 107 registers and two CTAs an SM 104 us), 31 us without page scales; pieces
// of 32 prompts, 134 MB, in 16 bits: 22 us (90 %); a decode step's tokens (64 x 1, 2
// heads): 2.0 us (3.1 to 3.5 issued from Python, the host's time); 256 x 4 drafts, 8
// heads of 64: 3.5 us, both a chain of four dependent loads.
//
// Where it is slow.  Groups are dealt out by the most rows that a request may have: one
// prompt chunk beside many single tokens launches a chunk's groups for every request
// (64 x 1 and 8192 tokens, pages of 128: 234 us where the bytes need 8).  Tensors' scales
// other than 1 with page scales: 64 us (a power of two) or 111 for the prompts above.
//
// Plain loads of what kernels before this one wrote (lengths, table, older codes) lie
// behind griddepcontrol.wait, which makes those writes seen.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pages.h"

namespace mm3idx {
namespace {

constexpr int kThreads = 256;
constexpr float kLowScale = 0x1p-60f, kHighScale = 0x1p60f;

template <bool BF16>
__device__ __forceinline__ float2 floats(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The larger of two pairs; a NaN loses.
template <bool BF16>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t halves(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four floats as e4m3, to the nearest, saturated at 448 (infinities too); NaN
// stays NaN.
__device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ float2 widen(uint16_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The least power of two, in the scales' range, that brings `top` to 448 or
// less: 448 = 1.75 2^8, so it is the exponent of top less 8, or less 7 where its
// fraction is above 1.75.
__device__ __forceinline__ float least_scale(float top) {
  const uint32_t bits = __float_as_uint(top);
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(min(max(e, 127 - 60), 127 + 60)) << 23);
}

// Division by a number: a product with its reciprocal where that is exact.
struct By {
  float d, inv;
  bool exact;
  __device__ __forceinline__ float operator()(float x) const { return exact ? x * inv : x / d; }
};

__device__ __forceinline__ By division(float x) {
  return By{x, 1.0f / x, (__float_as_uint(x) & 0x7fffffu) == 0};
}

enum { kCopy = 0, kCodes = 1, kScaled = 2 };

// BF16: type of the new elements.  MODE: a cache of that type, of e4m3, or of e4m3
// with scales.  UNIT: both divisors are 1.  G: threads a (page, head).  N: pieces of
// 16 bytes a thread.
template <bool BF16, int MODE, bool UNIT, int G, int N>
__global__ void __launch_bounds__(kThreads, N > 4 ? 4 : MODE == kScaled ? 5 : 6)
    append_kernel(const __grid_constant__ AppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float tops[kThreads / 32];
  const int unit = static_cast<int>(blockIdx.x) * (kThreads / G) + static_cast<int>(threadIdx.x) / G;
  const int t = threadIdx.x % G;
  // unit = ((request * touched + page) * 2 + side) * kv_heads + head: neighbours
  // read neighbouring heads of the same tokens
  const int outer = a.by_heads.quotient(min(unit, a.units - 1));
  const int head = unit - outer * a.kv_heads, which = outer & 1;
  const int req = a.by_touched.quotient(outer >> 1), turn = (outer >> 1) - req * a.touched;
  const AppendSide& side = a.side[which];
  const int shift = a.head_dim == 128 ? 4 : 3;           // pieces of a row, log2
  const int mask = (1 << shift) - 1;

  // The page's new slots [from, to) and the row of the first of them.
  int from = 0, pieces = 0, column = 0, bits = 0;
  int64_t row = 0;
  if (unit < a.units) {
    const int raw = a.seq_lens[req];
    const int len = min(max(raw, 0), a.max_seq_len);
    int rows = a.query_len;
    bits = raw > a.max_seq_len ? MM3IDX_DEV_SEQ_TOO_LONG : 0;
    int64_t row0 = static_cast<int64_t>(req) * a.query_len;
    if (a.cu) {
      const int c0 = a.cu[req], c1 = a.cu[req + 1];
      const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.total_q && c1 - c0 <= a.query_len;
      if (!ok || (req == 0 && c0 != 0) || (req == a.num_reqs - 1 && c1 != a.total_q))
        bits |= MM3IDX_DEV_BAD_ROWS;
      rows = ok ? c1 - c0 : 0;
      row0 = c0;
    }
    const int begin = max(len - rows, 0);               // first new position
    column = (begin >> a.page_shift) + turn;            // page of the request
    const int lo = max(begin, column << a.page_shift), hi = min(len, (column + 1) << a.page_shift);
    if (lo < hi) {
      from = lo & ((1 << a.page_shift) - 1);
      pieces = (hi - lo) << shift;
      row = row0 + (lo - (len - rows));
    }
  }
  const uint16_t* x = side.x + row * side.x_tok + head * side.x_head;
  auto load = [&](int m) {
    const int k = t + m * G;
    if (k >= pieces) return make_uint4(0, 0, 0, 0);
    return __ldg(reinterpret_cast<const uint4*>(x + (k >> shift) * side.x_tok) + (k & mask));
  };
  uint4 v[N];
#pragma unroll
  for (int m = 0; m < N; ++m) v[m] = load(m);
  int page = -1;
  if (pieces > 0) {
    page = a.table[req * a.table_stride + column];
    if (page < 0 || page >= a.num_pages) {
      bits |= MM3IDX_DEV_BAD_PAGE;
      pieces = 0;
    }
  }
  if (bits && t == 0 && head == 0 && which == 0) atomicOr(a.status, bits);

  const By by = division(side.scale);
  auto pair = [&](uint32_t w) {
    const float2 f = floats<BF16>(w);
    if constexpr (UNIT) return f;
    return make_float2(by(f.x), by(f.y));
  };
  uint8_t* base = side.cache + page * side.c_page + head * side.c_head;
  if constexpr (MODE == kCopy) {
#pragma unroll
    for (int m = 0; m < N; ++m) {
      const int k = t + m * G;
      if (k >= pieces) continue;
      uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
      if constexpr (!UNIT)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = pair(w[e]);
          w[e] = halves<BF16>(f.x, f.y);
        }
      *reinterpret_cast<uint4*>(base + (from + (k >> shift)) * side.c_tok + (k & mask) * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
  By to_codes{1.0f, 1.0f, true};
  if constexpr (MODE == kScaled) {
    float* at = side.scales + page * side.s_page + head * side.s_head;
    const float old = pieces > 0 && from > 0 ? fminf(fmaxf(__ldcg(at), kLowScale), kHighScale) : 0.0f;
    // The largest magnitude (a maximum passes over NaN); where that is infinite,
    // once more without the infinities, from memory (registers are not indexed).
    auto larger = [&](float top, uint4 q, bool finite) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 f = pair(w[e]);
        f = make_float2(fabsf(f.x), fabsf(f.y));
        if (finite) f = make_float2(f.x < INFINITY ? f.x : 0.0f, f.y < INFINITY ? f.y : 0.0f);
        top = fmaxf(top, fmaxf(f.x, f.y));
      }
      return top;
    };
    auto joined = [&](float top) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if constexpr (G > 32) {
        __syncthreads();               // (the last use of tops)
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < G / 32; ++k)
          top = fmaxf(top, tops[(threadIdx.x / G) * (G / 32) + k]);
      }
      return top;
    };
    float top = 0.0f;
    if constexpr (UNIT) {              // as they came, two at a time
      uint32_t two = 0;
#pragma unroll
      for (int m = 0; m < N; ++m) {
        const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) two = larger2<BF16>(two, w[e] & 0x7fff7fffu);
      }
      const float2 f = floats<BF16>(two);
      top = fmaxf(f.x, f.y);
    } else {
#pragma unroll
      for (int m = 0; m < N; ++m) top = larger(top, v[m], false);
    }
    top = joined(top);
    bool again = top == INFINITY;
    if constexpr (G > 32) again = __syncthreads_or(again);
    if (again) {
      float without = 0.0f;
#pragma unroll 1
      for (int m = 0; m < N; ++m) without = larger(without, load(m), true);
      without = joined(without);
      if (top == INFINITY) top = without;
    }
    const float scale = fmaxf(least_scale(top), old);
    __syncwarp();                      // every lane has the old scale (larger groups met above)
    if (pieces > 0) {
      if (from > 0 && scale != old) {
        // the older tokens' codes, 16 of them a piece
        const float f = old / scale;
        for (int k = t; k < from << (shift - 1); k += G) {
          uint4* c = reinterpret_cast<uint4*>(base + (k >> (shift - 1)) * side.c_tok) +
                     (k & (mask >> 1));
          uint4 q = *c;
          uint32_t* w = &q.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 l = widen(static_cast<uint16_t>(w[e])), h = widen(static_cast<uint16_t>(w[e] >> 16));
            w[e] = codes(l.x * f, l.y * f, h.x * f, h.y * f);
          }
          *c = q;
        }
      }
      if (t == 0) *at = scale;
    }
    to_codes = division(scale);
  }
  auto store = [&](int m, uint4 q, auto scaled) {
    const int k = t + m * G;
    if (k >= pieces) return;
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 lo = pair(w[2 * h]), hi = pair(w[2 * h + 1]);
      c[h] = codes(scaled(lo.x), scaled(lo.y), scaled(hi.x), scaled(hi.y));
    }
    *reinterpret_cast<uint2*>(base + (from + (k >> shift)) * side.c_tok + (k & mask) * 8) =
        make_uint2(c[0], c[1]);
  };
  if (MODE == kScaled && !to_codes.exact) {
    // an old scale that is no power of two: divisions, from memory again
#pragma unroll 1
    for (int m = 0; m < N; ++m) store(m, load(m), [&](float f) { return f / to_codes.d; });
    return;
  }
#pragma unroll
  for (int m = 0; m < N; ++m)
    store(m, v[m], [&](float f) { return MODE == kScaled ? f * to_codes.inv : f; });
}

template <bool BF16, int MODE, bool UNIT, int G, int N>
cudaError_t launch_group(const AppendArgs& a, cudaStream_t s) {
  constexpr int per = kThreads / G;
  return launch_dependent(append_kernel<BF16, MODE, UNIT, G, N>, dim3((a.units - 1) / per + 1),
                          kThreads, 1, a, s);
}

// The threads that hold the most new tokens of a page, eight pieces each (few
// tokens: one or four pieces of one warp).  Four prompts of 8192 tokens, pages of
// 64: 256 threads with four pieces 35.7 us, 128 with eight 32.1, 512 with two 64.
template <bool BF16, int MODE, bool UNIT>
cudaError_t launch_mode(const AppendArgs& a, cudaStream_t s) {
  const int page = 1 << a.page_shift;
  const int pieces = (a.query_len < page ? a.query_len : page) * (a.head_dim / 8);
  if (pieces <= 32) return launch_group<BF16, MODE, UNIT, 32, 1>(a, s);
  if (pieces <= 128) return launch_group<BF16, MODE, UNIT, 32, 4>(a, s);
  if (pieces <= 256) return launch_group<BF16, MODE, UNIT, 32, 8>(a, s);
  if (pieces <= 512) return launch_group<BF16, MODE, UNIT, 64, 8>(a, s);
  if (pieces <= 1024) return launch_group<BF16, MODE, UNIT, 128, 8>(a, s);
  return launch_group<BF16, MODE, UNIT, 256, 8>(a, s);
}

template <bool BF16, bool UNIT>
cudaError_t launch_cache(const AppendArgs& a, cudaStream_t s) {
  if (a.kv_type != MM3IDX_TYPE_E4M3) return launch_mode<BF16, kCopy, UNIT>(a, s);
  if (a.side[0].scales) return launch_mode<BF16, kScaled, UNIT>(a, s);
  return launch_mode<BF16, kCodes, UNIT>(a, s);
}

template <bool BF16>
cudaError_t launch_type(const AppendArgs& a, cudaStream_t s) {
  return a.side[0].scale == 1.0f && a.side[1].scale == 1.0f ? launch_cache<BF16, true>(a, s)
                                                            : launch_cache<BF16, false>(a, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  return a.type == MM3IDX_TYPE_BF16 ? launch_type<true>(a, s) : launch_type<false>(a, s);
}

}  // namespace mm3idx
