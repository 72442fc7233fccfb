// Backward pass of the norms for a block's output in bf16.
#define MOE_NORM_BACK_KERNELS
#include "norm_back.h"

namespace moe {

void launch_norm_back_bf16(const NormBackArgs& a, hipStream_t s, bool sf, bool of, bool pf, bool bias) {
  pick_norm_back<false>(a, s, sf, of, pf, bias);
}

}  // namespace moe
