// Instantiations of the masked tensor-memory query-split kernel for int8 caches, in a translation unit of their own so
// that they compile in parallel with the other kernel families.
#include "pkv_decode_kernel.cuh"
#include "pkv_i8_tc5.cuh"

namespace pkv {

LaunchFn pick_mask_i8_tc5(int D)
{
    if (D == 64) return launch_decode<64, 16, kI8, true, true, true>;
    if (D == 128) return launch_decode<128, 16, kI8, true, true, true>;
    return nullptr;
}

}  // namespace pkv
