// Chunk attention, head dim 128.
#include "chunk_kernel.cuh"

namespace kvq {

cudaError_t launch_chunk_d128(const ChunkArgs& a, bool paired, int grid, cudaStream_t s) {
  if (a.lo.dtype == KVQ_DT_F16)
    return paired ? launch_chunk<128, KVQ_DT_F16, true>(a, grid, s) : launch_chunk<128, KVQ_DT_F16, false>(a, grid, s);
  return paired ? launch_chunk<128, KVQ_DT_BF16, true>(a, grid, s) : launch_chunk<128, KVQ_DT_BF16, false>(a, grid, s);
}

}  // namespace kvq
