// Attention over bf16 caches.  Ring depth: what fills the SM's shared memory
// (two blocks per SM at width 128, one at 256).
#include "attention.cuh"

namespace dvl {
namespace attn {

cudaError_t config_bf16(int D, int rows, AttnConfig *out)
{
    if (D <= 64)
        return config_rows<64, false, 4>(rows, out);
    if (D <= 128)
        return config_rows<128, false, 3>(rows, out);
    return config_rows<256, false, 3>(rows, out);
}

}  // namespace attn
}  // namespace dvl
