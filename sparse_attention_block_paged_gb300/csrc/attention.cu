// attention.cu -- dispatch of the paged attention (attention.cuh) and the
// block weights made from what it leaves in the workspace.
#include "../../include/mm3idx.h"
#include "serving.h"

namespace mm3idx {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;

// block_weights[row, b] = sum over the heads of 2^(tile - row), the base-2
// log-sum-exps of the row's scores in the block and in all: one thread per
// (row, block), 0 past the row's last block.  A dependent of the attention.
__global__ void __launch_bounds__(kThreads) block_weight_kernel(const AttentionArgs a, int pitch) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = blockIdx.x;
  const int b = blockIdx.y * kThreads + threadIdx.x;
  if (b >= a.w_width) return;
  const int i = static_cast<int>(row / a.query_len), j = static_cast<int>(row % a.query_len);
  const int len = min(max(__ldg(a.seq_lens + i), 0), a.max_seq_len);
  float sum = 0.0f;
  if (b * kBlock < len - a.query_len + j + 1) {
    const int first = j * a.group;                 // rows of the kv head, 64 a task
    for (int h = 0; h < a.kv_heads; ++h) {
      const float* lse = a.row_lse + (row * a.kv_heads + h) * a.group;
      const float* tile = a.tile_lse +
                          ((static_cast<int64_t>(i) * a.kv_heads + h) * a.row_tiles * a.w_width + b) * pitch;
      const int64_t next = static_cast<int64_t>(a.w_width) * pitch;
      for (int k0 = 0; k0 < a.group; k0 += kAhead) {
        float x[kAhead], all[kAhead];              // in flight together
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int r = first + k0 + k;
          const bool in = k0 + k < a.group;
          all[k] = in ? __ldcg(lse + k0 + k) : -INFINITY;
          x[k] = in ? __ldcg(tile + (r >> 6) * next + (r & 63)) : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (all[k] != -INFINITY) sum += exp2f(x[k] - all[k]);
      }
    }
  }
  a.weights[row * a.w_stride + b] = sum;
}

}  // namespace

cudaError_t launch_attention(const CUtensorMap& kmap, const CUtensorMap& vmap,
                             const AttentionArgs& a, int grid, cudaStream_t s) {
  cudaError_t e;
  if (a.kv_type == MM3IDX_TYPE_BF16) e = launch_attention_bf16(kmap, vmap, a, grid, s);
  else if (a.kv_type == MM3IDX_TYPE_FP16) e = launch_attention_fp16(kmap, vmap, a, grid, s);
  else if (a.k_scales) e = a.q_type == MM3IDX_TYPE_BF16
                               ? launch_attention_bf16_e4m3_scaled(kmap, vmap, a, grid, s)
                               : launch_attention_fp16_e4m3_scaled(kmap, vmap, a, grid, s);
  else if (a.q_type == MM3IDX_TYPE_BF16) e = launch_attention_bf16_e4m3(kmap, vmap, a, grid, s);
  else e = launch_attention_fp16_e4m3(kmap, vmap, a, grid, s);
  if (e != cudaSuccess || !a.weights) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_reqs) * a.query_len,
                     (a.w_width + kThreads - 1) / kThreads);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_weight_kernel, a,
                            16 * attention_row_tiles16(a.group * a.query_len));
}

}  // namespace mm3idx
