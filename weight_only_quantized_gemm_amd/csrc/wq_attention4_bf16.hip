// The 4-bit cache's attention for bf16 tensors.
#include "wq_attention4_kernel.h"

namespace wq {

hipError_t launch_attn4_bf16(const Attn4Args& p, const Columns& c, dim3 grid, hipStream_t stream) {
  return launch_attn4<true>(p, c, grid, stream);
}

}  // namespace wq
