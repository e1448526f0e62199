// Instances of the block-scaled cache's stream and of its joining launch, head_dim 256.
#include "block_combine.cuh"

namespace vsk {

bk::BkFn kernel_block_stream_256(int nr) {
  return nr == 8 ? block_stream_kernel<256, 8> : nr == 16 ? block_stream_kernel<256, 16> : block_stream_kernel<256, 32>;
}
bk::BkJoinFn kernel_block_combine_256(bool split) { return split ? block_combine_kernel<256, true> : block_combine_kernel<256, false>; }

}  // namespace vsk
