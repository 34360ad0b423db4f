// attention_bf16_e4m3.cu -- the paged attention kernels (attention.cuh) of bf16
// queries over e4m3 keys and values.
#include "attention.cuh"

namespace mm3idx {

cudaError_t launch_attention_bf16_e4m3(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                       const AttentionArgs& a, int grid, cudaStream_t s) {
  return attn::launch_kv<MM3IDX_TYPE_BF16, MM3IDX_TYPE_E4M3>(kmap, vmap, a, grid, s);
}

}  // namespace mm3idx
