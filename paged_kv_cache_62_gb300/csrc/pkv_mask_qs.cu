// Instantiations of the masked query-split kernels (bf16 caches; warp-level tiles and tensor-memory CTAs), in a
// translation unit of their own so that they compile in parallel with the other kernel families.
#include "pkv_decode_kernel.cuh"

namespace pkv {

template <int D>
static LaunchFn pick_qs(int G)
{
    switch (G) {
    case 12: return launch_decode<D, 12, kBf16, true, false, true>;
    case 14: return launch_decode<D, 14, kBf16, true, false, true>;
    case 15: return launch_decode<D, 15, kBf16, true, false, true>;
    case 16: return launch_decode<D, 16, kBf16, true, false, true>;
    default: return nullptr;
    }
}

LaunchFn pick_mask_qs(int D, int G)
{
    if (D == 64) return pick_qs<64>(G);
    if (D == 128) return pick_qs<128>(G);
    return nullptr;
}

LaunchFn pick_mask_tc5(int D)
{
    if (D == 64) return launch_decode<64, 16, kBf16, true, true, true>;
    if (D == 128) return launch_decode<128, 16, kBf16, true, true, true>;
    return nullptr;
}

}  // namespace pkv
