// Instances of the block-scaled cache's stream and of its joining launch, head_dim 256.
#include "block_combine.cuh"

namespace vsk {

bk::BkFn kernel_block_stream_256() { return block_stream_kernel<256>; }
bk::BkJoinFn kernel_block_combine_256() { return block_combine_kernel<256>; }

}  // namespace vsk
