// Append with the position rotation: instances for 4-bit codes.
#include "append_rotary.cuh"

namespace kvq {

cudaError_t launch_append_rotary_i4(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  return launch_bits<4>(p, rows, stream);
}

}  // namespace kvq
