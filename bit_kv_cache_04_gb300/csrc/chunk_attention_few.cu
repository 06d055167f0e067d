// Chunk attention, head dim 128, at most 32 rows a sequence (single tokens, drafts).
#include "chunk_kernel.cuh"

namespace kvq {

cudaError_t launch_chunk_few(const ChunkArgs& a, int grid, cudaStream_t s) {
  if (a.lo.dtype == KVQ_DT_F16) return launch_chunk<128, KVQ_DT_F16, kChunkFew>(a, grid, s);
  return launch_chunk<128, KVQ_DT_BF16, kChunkFew>(a, grid, s);
}

}  // namespace kvq
