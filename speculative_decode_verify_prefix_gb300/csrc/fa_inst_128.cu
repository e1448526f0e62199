// head_dim 128 instances of the tensor-core attention over many query rows.
#include "flash_tc.cuh"

namespace vsk {

fa::FaFn kernel_fa_128(int mode) {
  return mode == fa::kPrompt ? static_cast<fa::FaFn>(fa_kernel<128, fa::kPrompt>)
         : mode == fa::kSharedBf16 ? static_cast<fa::FaFn>(fa_kernel<128, fa::kSharedBf16>)
                                   : static_cast<fa::FaFn>(fa_kernel<128, fa::kSharedE4m3>);
}

}  // namespace vsk
