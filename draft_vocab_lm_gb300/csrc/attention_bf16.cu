// Attention over bf16 caches.
#include "attention.cuh"

namespace dvl {
namespace attn {

// Eight warps or more per SM, each with one chunk in flight: 32 tokens at
// widths up to 128, 16 at 256 (16 KB either way).
cudaError_t config_bf16(int D, int rows, AttnConfig *out)
{
    if (D <= 64)
        return rows <= 8    ? config<64, kBf16, 0, 32, 1, 4, 3>(out)
               : rows <= 16 ? config<64, kBf16, 1, 32, 1, 4, 3>(out)
               : rows <= 32 ? config<64, kBf16, 2, 32, 1, 4, 1>(out)
                            : config<64, kBf16, 4, 32, 1, 2, 1>(out);
    if (D <= 128)
        return rows <= 8    ? config<128, kBf16, 0, 32, 1, 4, 2>(out)
               : rows <= 16 ? config<128, kBf16, 1, 32, 1, 4, 2>(out)
               : rows <= 32 ? config<128, kBf16, 2, 32, 1, 4, 1>(out)
                            : config<128, kBf16, 4, 32, 1, 2, 1>(out);
    return rows <= 8    ? config<256, kBf16, 0, 16, 1, 8, 1>(out)
           : rows <= 16 ? config<256, kBf16, 1, 16, 1, 8, 1>(out)
           : rows <= 32 ? config<256, kBf16, 2, 16, 1, 4, 1>(out)
                        : config<256, kBf16, 4, 16, 1, 2, 1>(out);
}

}  // namespace attn
}  // namespace dvl
