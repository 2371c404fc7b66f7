// Attention over FP8 (E4M3) caches: half the bytes per tile, so more blocks
// per SM keep as much in flight.
#include "attention.cuh"

namespace dvl {
namespace attn {

cudaError_t config_fp8(int D, int rows, AttnConfig *out)
{
    if (D <= 64)
        return config_rows<64, true, 4>(rows, out);
    if (D <= 128)
        return config_rows<128, true, 3>(rows, out);
    return config_rows<256, true, 3>(rows, out);
}

}  // namespace attn
}  // namespace dvl
