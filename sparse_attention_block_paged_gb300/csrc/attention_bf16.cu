// attention_bf16.cu -- the paged attention kernels (attention.cuh) over bf16
// keys and values.
#include "attention.cuh"

namespace mm3idx {

cudaError_t launch_attention_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  const AttentionArgs& a, int grid, cudaStream_t s) {
  return attn::launch_kv<MM3IDX_TYPE_BF16, MM3IDX_TYPE_BF16>(kmap, vmap, a, grid, s);
}

}  // namespace mm3idx
