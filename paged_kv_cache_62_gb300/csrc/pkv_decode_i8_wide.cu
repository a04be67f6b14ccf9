// Instantiations of the decode kernel for int8 caches with 9 to 16 virtual heads (both 8-row halves of the MMA
// tile), in a translation unit of their own so that they compile in parallel with the other kernel families.
#include "pkv_decode_kernel.cuh"
#include "pkv_i8_tile.cuh"

namespace pkv {

template <int D>
static LaunchFn pick_wide(int G)
{
    switch (G) {
    case 9: return launch_decode<D, 9, kI8, false>;
    case 10: return launch_decode<D, 10, kI8, false>;
    case 11: return launch_decode<D, 11, kI8, false>;
    case 12: return launch_decode<D, 12, kI8, false>;
    case 13: return launch_decode<D, 13, kI8, false>;
    case 14: return launch_decode<D, 14, kI8, false>;
    case 15: return launch_decode<D, 15, kI8, false>;
    case 16: return launch_decode<D, 16, kI8, false>;
    default: return nullptr;
    }
}

LaunchFn pick_decode_i8_wide(int D, int G)
{
    if (D == 64) return pick_wide<64>(G);
    if (D == 128) return pick_wide<128>(G);
    return nullptr;
}

}  // namespace pkv
