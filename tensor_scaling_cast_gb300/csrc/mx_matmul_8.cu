// mx_matmul of 8-bit operands (see mx_matmul.cuh).
#include "mx_matmul.cuh"

namespace fp8q {

cudaError_t launch_mx_matmul_8(const MxProduct& p, cudaStream_t s, int* launches) {
  return launch_format<false>(p, s, launches);
}
cudaError_t read_mm8_wait_timeouts(unsigned int* count) { return read_timeouts(count); }

}  // namespace fp8q
