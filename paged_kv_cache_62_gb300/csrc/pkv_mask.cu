// Instantiations of the masked decode kernel (sliding windows with sinks, trees of drafted tokens; bf16 caches, 1 to 8
// virtual heads), in a translation unit of their own so that they compile in parallel with the other kernel
// families.
#include "pkv_decode_kernel.cuh"

namespace pkv {

LaunchFn pick_mask(int D, int G)
{
    if (D == 64) return pick_group<64, kBf16, false, true>(G);
    if (D == 128) return pick_group<128, kBf16, false, true>(G);
    return nullptr;
}

}  // namespace pkv
