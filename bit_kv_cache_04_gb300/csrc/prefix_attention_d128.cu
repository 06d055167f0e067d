// Attention over shared prefixes, head dim 128, more than 32 rows a group.
#include "chunk_kernel.cuh"

namespace kvq {

cudaError_t launch_prefix_d128(const ChunkArgs& a, int mode, int grid, cudaStream_t s) {
  const bool paired = mode == kChunkPaired;
  if (a.lo.dtype == KVQ_DT_F16)
    return paired ? launch_chunk<128, KVQ_DT_F16, kChunkPaired, true>(a, grid, s)
                  : launch_chunk<128, KVQ_DT_F16, kChunkShared, true>(a, grid, s);
  return paired ? launch_chunk<128, KVQ_DT_BF16, kChunkPaired, true>(a, grid, s)
                : launch_chunk<128, KVQ_DT_BF16, kChunkShared, true>(a, grid, s);
}

}  // namespace kvq
