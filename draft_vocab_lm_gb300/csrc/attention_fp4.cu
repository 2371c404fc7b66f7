// Attention over NVFP4 caches: E2M1 codes, one E4M3 scale per 16 values.
#include "attention.cuh"

namespace dvl {
namespace attn {

cudaError_t config_fp4(int D, int rows, AttnConfig *out)
{
    if (D <= 64)
        return rows <= 8    ? config<64, kFp4, 0, 32, 1, 4, 3>(out)
               : rows <= 16 ? config<64, kFp4, 1, 32, 1, 4, 2>(out)
               : rows <= 32 ? config<64, kFp4, 2, 32, 1, 4, 1>(out)
                            : config<64, kFp4, 4, 32, 1, 2, 1>(out);
    if (D <= 128)
        return rows <= 8    ? config<128, kFp4, 0, 32, 1, 4, 3>(out)
               : rows <= 16 ? config<128, kFp4, 1, 32, 1, 4, 2>(out)
               : rows <= 32 ? config<128, kFp4, 2, 32, 1, 4, 1>(out)
                            : config<128, kFp4, 4, 32, 1, 2, 1>(out);
    return rows <= 8    ? config<256, kFp4, 0, 32, 1, 4, 2>(out)
           : rows <= 16 ? config<256, kFp4, 1, 16, 1, 4, 2>(out)
           : rows <= 32 ? config<256, kFp4, 2, 16, 1, 4, 1>(out)
                        : config<256, kFp4, 4, 16, 1, 2, 1>(out);
}

}  // namespace attn
}  // namespace dvl
