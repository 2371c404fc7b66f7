// Attention over NVFP4 caches: E2M1 codes, one E4M3 scale per 16 values.
#include "attention.cuh"

namespace dvl {
namespace attn {

// One chunk in flight per group: with 4.5 KB a chunk (128) an SM's twelve groups
// have 54 KB on their way, and more chunks or more blocks change nothing (64 x <=
// 16,381 tokens, 128: 1, 2 and 3 chunks 184, 185 and 186 us, four blocks an SM
// 183; 16 tokens a chunk 242).  At 256 and up to 8 query rows 32 tokens a chunk
// against 16: 262,139 tokens 55 against 62 us; 64 tokens a chunk at 128 was slower
// (216 against 187).  With 9 to 16 rows three blocks an SM at 64 (32 x <= 8,189
// tokens, 3 new ones, 40 / 8 heads: 49 us against 56 with two), two at 128, whose
// registers three do not hold (73 against 80).
cudaError_t config_fp4(int D, int rows, AttnConfig *out)
{
    if (D <= 64)
        return rows <= 8    ? config<64, kFp4, 0, 32, 1, 4, 3>(out)
               : rows <= 16 ? config<64, kFp4, 1, 32, 1, 4, 3>(out)
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
