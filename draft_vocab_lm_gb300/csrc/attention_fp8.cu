// Attention over FP8 (E4M3) caches.
#include "attention.cuh"

namespace dvl {
namespace attn {

// Half the bytes per token and twice the instructions per byte of bf16: more
// warps per SM.
cudaError_t config_fp8(int D, int rows, AttnConfig *out)
{
    if (D <= 64)
        return rows <= 8    ? config<64, true, 0, 32, 1, 4, 4>(out)
               : rows <= 16 ? config<64, true, 1, 32, 1, 4, 3>(out)
               : rows <= 32 ? config<64, true, 2, 32, 1, 4, 1>(out)
                            : config<64, true, 4, 32, 1, 2, 1>(out);
    if (D <= 128)
        return rows <= 8    ? config<128, true, 0, 32, 1, 4, 3>(out)
               : rows <= 16 ? config<128, true, 1, 32, 1, 4, 2>(out)
               : rows <= 32 ? config<128, true, 2, 32, 1, 4, 1>(out)
                            : config<128, true, 4, 32, 1, 2, 1>(out);
    return rows <= 8    ? config<256, true, 0, 16, 1, 4, 2>(out)
           : rows <= 16 ? config<256, true, 1, 16, 1, 4, 2>(out)
           : rows <= 32 ? config<256, true, 2, 16, 1, 4, 1>(out)
                        : config<256, true, 4, 16, 1, 2, 1>(out);
}

}  // namespace attn
}  // namespace dvl
