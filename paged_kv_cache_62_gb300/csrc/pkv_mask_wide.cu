// Instantiations of the masked decode kernel for 9 to 16 virtual heads (bf16 caches), in a translation unit of their
// own so that they compile in parallel with the other kernel families.
#include "pkv_decode_kernel.cuh"

namespace pkv {

LaunchFn pick_mask_wide(int D, int G)
{
    if (D == 64) return pick_wide_group<64, kBf16, true>(G);
    if (D == 128) return pick_wide_group<128, kBf16, true>(G);
    return nullptr;
}

}  // namespace pkv
