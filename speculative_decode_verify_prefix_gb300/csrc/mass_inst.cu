// Instances of the key-weight kernel.
#include "key_mass.cuh"

namespace vsk {

km::MassFn kernel_mass(int D, bool fp8, bool qreg) {
  if (D == 64) {
    if (qreg) return fp8 ? static_cast<km::MassFn>(mass_kernel<64, true, true>) : static_cast<km::MassFn>(mass_kernel<64, false, true>);
    return fp8 ? static_cast<km::MassFn>(mass_kernel<64, true, false>) : static_cast<km::MassFn>(mass_kernel<64, false, false>);
  }
  if (D == 128) {
    if (qreg) return fp8 ? static_cast<km::MassFn>(mass_kernel<128, true, true>) : static_cast<km::MassFn>(mass_kernel<128, false, true>);
    return fp8 ? static_cast<km::MassFn>(mass_kernel<128, true, false>) : static_cast<km::MassFn>(mass_kernel<128, false, false>);
  }
  // head_dim 256: the query fragments of a tile take as many registers as a stage of keys
  return fp8 ? static_cast<km::MassFn>(mass_kernel<256, true, false>) : static_cast<km::MassFn>(mass_kernel<256, false, false>);
}

}  // namespace vsk
