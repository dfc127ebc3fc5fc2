// Append with the position rotation: instances for 2-bit codes.
#include "append_rotary.cuh"

namespace kvq {

cudaError_t launch_append_rotary_i2(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  return launch_bits<2>(p, rows, stream);
}

}  // namespace kvq
