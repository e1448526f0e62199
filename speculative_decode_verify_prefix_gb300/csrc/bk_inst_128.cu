// Instances of the block-scaled cache's stream and of its joining launch, head_dim 128.
#include "block_combine.cuh"

namespace vsk {

bk::BkFn kernel_block_stream_128(int nr) {
  return nr == 8 ? block_stream_kernel<128, 8> : nr == 16 ? block_stream_kernel<128, 16> : block_stream_kernel<128, 32>;
}
bk::BkJoinFn kernel_block_combine_128(bool split) { return split ? block_combine_kernel<128, true> : block_combine_kernel<128, false>; }

}  // namespace vsk
