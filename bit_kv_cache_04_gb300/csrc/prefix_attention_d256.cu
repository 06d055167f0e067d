// Attention over shared prefixes, head dim 256.
#include "chunk_kernel.cuh"

namespace kvq {

cudaError_t launch_prefix_d256(const ChunkArgs& a, int grid, cudaStream_t s) {
  if (a.lo.dtype == KVQ_DT_F16) return launch_chunk<256, KVQ_DT_F16, kChunkShared, true>(a, grid, s);
  return launch_chunk<256, KVQ_DT_BF16, kChunkShared, true>(a, grid, s);
}

}  // namespace kvq
