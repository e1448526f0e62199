// Instances of the block-scaled cache's stream and of its joining launch, head_dim 64.
#include "block_combine.cuh"

namespace vsk {

bk::BkFn kernel_block_stream_64() { return block_stream_kernel<64>; }
bk::BkJoinFn kernel_block_combine_64() { return block_combine_kernel<64>; }

}  // namespace vsk
