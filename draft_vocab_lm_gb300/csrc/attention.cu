// Attention over a paged cache: the choice of the kernel and its launch.
#include <cuda_runtime.h>

#include "dvl_attention.h"

namespace dvl {
namespace attn {

cudaError_t grid_blocks(int dtype, int D, int rows, AttnConfig *cfg, int *blocks)
{
    cudaError_t e = dtype == DVL_FP8     ? config_fp8(D, rows, cfg)
                    : dtype == DVL_NVFP4 ? config_fp4(D, rows, cfg)
                                         : config_bf16(D, rows, cfg);
    DeviceInfo di;
    if (e == cudaSuccess)
        e = device_info(&di);
    int per_sm = 0;
    if (e == cudaSuccess)
        e = blocks_per_sm(cfg->func, cfg->threads, cfg->smem, &per_sm);
    if (e != cudaSuccess)
        return e;
    if (per_sm < 1)
        return cudaErrorInvalidConfiguration;
    *blocks = per_sm * di.sms;
    if (*blocks > kMaxCtas)
        *blocks = kMaxCtas;
    return cudaSuccess;
}

cudaError_t launch_attention(AttnArgs &a, const AttnConfig &cfg, cudaStream_t s)
{
    // lanes: the most heads, up to eight, that divide all of them evenly
    a.lanes = a.heads < 8 ? a.heads : 8;
    while (a.heads % a.lanes != 0)
        --a.lanes;
    using Kernel = void (*)(AttnArgs);
    return launch_pdl(reinterpret_cast<Kernel>(const_cast<void *>(cfg.func)), (unsigned)a.blocks,
                      (unsigned)cfg.threads, cfg.smem, s, a);
}

}  // namespace attn
}  // namespace dvl
