// Chunk attention, head dim 256.
#include "chunk_kernel.cuh"

namespace kvq {

cudaError_t launch_chunk_d256(const ChunkArgs& a, int grid, cudaStream_t s) {
  if (a.lo.dtype == KVQ_DT_F16) return launch_chunk<256, KVQ_DT_F16, kChunkShared>(a, grid, s);
  return launch_chunk<256, KVQ_DT_BF16, kChunkShared>(a, grid, s);
}

}  // namespace kvq
