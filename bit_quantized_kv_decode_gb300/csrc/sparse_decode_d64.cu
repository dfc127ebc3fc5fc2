// Decode over lists of blocks: kernel instances for head dim 64, 4 query heads per unit.
#include "decode_general.cuh"

namespace kvq {

cudaError_t launch_listed_d64(int bits, bool kcw, bool vcw, int group, const ListParams& p, int grid,
                                const GenLaunch& shape, cudaStream_t s) {
  if (bits == 4) {
    if (group == 32) return gen::launch_schemes<4, 64, 32, false, 4>(kcw, vcw, p, grid, shape, s);
    if (group == 64) return gen::launch_schemes<4, 64, 64, false, 4>(kcw, vcw, p, grid, shape, s);
  }
  if (bits == 2) {
    if (group == 32) return gen::launch_schemes<2, 64, 32, false, 4>(kcw, vcw, p, grid, shape, s);
    if (group == 64) return gen::launch_schemes<2, 64, 64, false, 4>(kcw, vcw, p, grid, shape, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
