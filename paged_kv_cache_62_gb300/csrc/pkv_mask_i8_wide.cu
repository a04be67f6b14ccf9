// Instantiations of the masked decode kernel for int8 caches, 9 to 16 virtual heads, in a translation unit of their
// own so that they compile in parallel with the other kernel families.
#include "pkv_decode_kernel.cuh"
#include "pkv_i8_tile.cuh"

namespace pkv {

LaunchFn pick_mask_i8_wide(int D, int G)
{
    if (D == 64) return pick_wide_group<64, kI8, true>(G);
    if (D == 128) return pick_wide_group<128, kI8, true>(G);
    return nullptr;
}

}  // namespace pkv
