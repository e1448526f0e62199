// Instances of the block-scaled cache's stream and of its joining launch, head_dim 64.
#include "block_combine.cuh"

namespace vsk {

bk::BkFn kernel_block_stream_64(int nr) {
  return nr == 8 ? block_stream_kernel<64, 8> : nr == 16 ? block_stream_kernel<64, 16> : block_stream_kernel<64, 32>;
}
bk::BkJoinFn kernel_block_combine_64(bool split) { return split ? block_combine_kernel<64, true> : block_combine_kernel<64, false>; }

}  // namespace vsk
