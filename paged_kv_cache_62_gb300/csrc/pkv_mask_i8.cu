// Instantiations of the masked decode kernel for int8 caches, 1 to 8 virtual heads, in a translation unit of their own
// so that they compile in parallel with the other kernel families.
#include "pkv_decode_kernel.cuh"
#include "pkv_i8_tile.cuh"

namespace pkv {

LaunchFn pick_mask_i8(int D, int G)
{
    if (D == 64) return pick_group<64, kI8, false, true>(G);
    if (D == 128) return pick_group<128, kI8, false, true>(G);
    return nullptr;
}

}  // namespace pkv
