// head_dim 64 instances of the tensor-core attention over many query rows.
#include "flash_tc.cuh"

namespace vsk {

fa::FaFn kernel_fa_64(int mode) {
  return mode == fa::kPrompt ? static_cast<fa::FaFn>(fa_kernel<64, fa::kPrompt>)
         : mode == fa::kSharedBf16 ? static_cast<fa::FaFn>(fa_kernel<64, fa::kSharedBf16>)
                                   : static_cast<fa::FaFn>(fa_kernel<64, fa::kSharedE4m3>);
}

}  // namespace vsk
