// Chunk attention over 2-bit caches: one instance per head dim and number of row tiles.
#include "chunk_attn.cuh"

namespace kvq {
namespace chunk {

cudaError_t launch_i2(int head_dim, int nt, const Params& p, int grid, size_t smem, cudaStream_t stream) {
  if (head_dim == 64) return nt == 2 ? launch_instance<2, 64, 2>(p, grid, smem, stream)
                                     : launch_instance<2, 64, 1>(p, grid, smem, stream);
  if (head_dim == 128) return nt == 2 ? launch_instance<2, 128, 2>(p, grid, smem, stream)
                                      : launch_instance<2, 128, 1>(p, grid, smem, stream);
  return launch_instance<2, 256, 1>(p, grid, smem, stream);
}

}  // namespace chunk
}  // namespace kvq
