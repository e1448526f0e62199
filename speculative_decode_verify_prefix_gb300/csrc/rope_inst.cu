// Instances of the rotary and append kernels.
#include "rope_append.cuh"

namespace vsk {

template <int D>
static rp::RopeFn rope_of(int pool) {
  return pool == 0   ? static_cast<rp::RopeFn>(rope_kernel<D, 0>)
         : pool == 1 ? static_cast<rp::RopeFn>(rope_kernel<D, 1>)
                     : static_cast<rp::RopeFn>(rope_kernel<D, 2>);
}
rp::RopeFn kernel_rope(int D, int pool) {
  return D == 64 ? rope_of<64>(pool) : D == 128 ? rope_of<128>(pool) : rope_of<256>(pool);
}
rp::RopeFn kernel_rope_block(int D) {
  return D == 64 ? static_cast<rp::RopeFn>(rope_block_kernel<64>)
         : D == 128 ? static_cast<rp::RopeFn>(rope_block_kernel<128>)
                    : static_cast<rp::RopeFn>(rope_block_kernel<256>);
}

}  // namespace vsk
