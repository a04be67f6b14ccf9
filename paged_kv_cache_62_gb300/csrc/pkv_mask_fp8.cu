// Instantiations of the masked decode kernel for E4M3 caches, in a translation unit of their own so that they compile
// in parallel with the other kernel families.
#include "pkv_decode_kernel.cuh"

namespace pkv {

LaunchFn pick_mask_fp8(int D, int G)
{
    if (D == 64) return pick_group<64, kE4m3, false, true>(G);
    if (D == 128) return pick_group<128, kE4m3, false, true>(G);
    return nullptr;
}

}  // namespace pkv
