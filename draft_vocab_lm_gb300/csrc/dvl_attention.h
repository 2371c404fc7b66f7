// Declarations shared by the attention kernels, their join and the argument
// checks.
#pragma once

#include "dvl_internal.h"

namespace dvl {
namespace attn {

constexpr int kTile = 64;  // tokens per unit of work

struct AttnArgs {
    const uint16_t *q;        // bf16
    int64_t qb, qt, qh;       // strides in elements: sequence, token, head
    const unsigned char *k, *v;
    int64_t kp, kt, kh;       // strides in bytes: page, token, head
    int64_t vp, vt, vh;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lengths;
    uint16_t *out;            // bf16 [B][T][Hq][D]
    float *lse;               // [B][T][Hq] or nullptr
    unsigned char *ws;        // its header holds the status word
    float *parts;             // [2 * blocks][part_floats]
    int64_t part_floats;      // rows * D sums, then (maximum, sum) per row
    int B, T, Hq, heads, G, D;
    int rows;                 // T * G: query rows per cached head
    int pages, page_size;
    int max_len;              // tokens a table row can name
    uint32_t page_mul;        // pos / page_size = pos * page_mul >> page_shift
    int page_shift;
    float qk_scale;           // scale * k_scale * log2(e)
    float v_scale;
    int blocks;               // of the attention kernel

#ifdef __CUDACC__
    __device__ __forceinline__ int page_of(int pos) const
    {
        return (int)((uint64_t)(uint32_t)pos * page_mul >> page_shift);
    }
#endif
};

#ifdef __CUDACC__
// Blocks that hold units: with fewer units than blocks, one unit each, so
// that every block between a pair's first and last holds a part of it.
__device__ __forceinline__ int64_t used_blocks(int blocks, int64_t units)
{
    return units < blocks ? units : blocks;
}

// Natural logarithm of a sum of weights relative to 2^m; -inf for an empty row.
__device__ __forceinline__ float log_sum(float m, float sum)
{
    constexpr float kLn2 = 0.69314718055994531f;
    return sum == 0.f ? -__builtin_huge_valf() : fmaf(m, kLn2, logf(sum));
}
#endif

struct AttnConfig {
    const void *func;
    size_t smem;
};
// The kernel for padded head widths of 64, 128 and 256, by cache type.
cudaError_t config_bf16(int D, int rows, AttnConfig *out);
cudaError_t config_fp8(int D, int rows, AttnConfig *out);

// Blocks of the attention kernel on the current device.
cudaError_t grid_blocks(bool fp8, int D, int rows, AttnConfig *cfg, int *blocks);
cudaError_t launch_attention(AttnArgs &a, bool fp8, cudaStream_t s);

}  // namespace attn
}  // namespace dvl
