// Declarations shared by the attention kernels, their join and the argument
// checks.
#pragma once

#include "dvl_internal.h"

namespace dvl {
namespace attn {

struct AttnArgs {
    const uint16_t *q;        // bf16
    int64_t qb, qt, qh;       // strides in elements: sequence, token, head
    const unsigned char *k, *v;
    const unsigned char *kb, *vb;  // NVFP4: the scales
    int64_t kp, vp;           // strides in bytes: page
    uint32_t kt, kh, vt, vh;  // token, head (within a page)
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lengths;
    uint16_t *out;            // bf16 [B][T][Hq][D]
    float *lse;               // [B][T][Hq] or nullptr
    unsigned char *ws;        // its header holds the status word
    unsigned int *tickets;    // one per part slot; top_tickets on, one per joined pair
    int top_tickets;
    float *parts;             // [2 * blocks][part_floats]
    int64_t part_floats;      // rows * D sums, (maximum, sum) per row, the same of a joined group
    int B, T, Hq, heads, G, D;
    int rows;                 // T * G: query rows per cached head
    uint32_t token_mul;       // row / G = row * token_mul >> 16, for up to 64 rows
    int pages, page_size;
    int max_len;              // tokens a table row can name
    uint32_t page_mul;        // pos / page_size = pos * page_mul >> page_shift
    int page_shift;
    float qk_scale;           // scale * k_scale * log2(e)
    float v_scale;
    int blocks;               // of the grid
    int lanes;                // blocks that walk the same tokens, one head each

#ifdef __CUDACC__
    __device__ __forceinline__ int page_of(int pos) const
    {
        return (int)((uint64_t)(uint32_t)pos * page_mul >> page_shift);
    }
    __device__ __forceinline__ int token_of(int row) const { return row * token_mul >> 16; }
#endif
};

#ifdef __CUDACC__
// Shares that hold units: with fewer units than blocks of a lane, one unit
// each, so that every share between a pair's first and last holds a part.
__device__ __forceinline__ int used_shares(const AttnArgs &a, int64_t units)
{
    const int n = a.blocks / a.lanes;
    return units < n ? (int)units : n;
}

// Cached tokens of sequence b, cut to what its table row can name, and the
// units of one cached head of it.
__device__ __forceinline__ int seq_len(const AttnArgs &a, int b)
{
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.max_len ? a.max_len : n;
}
template <int TILE>
__device__ __forceinline__ int seq_tiles(const AttnArgs &a, int b)
{
    return (seq_len(a, b) + TILE - 1) / TILE;
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
    int threads;
    int tile;  // tokens per unit
};
// The kernel for padded head widths of 64, 128 and 256, by cache type.
cudaError_t config_bf16(int D, int rows, AttnConfig *out);
cudaError_t config_fp8(int D, int rows, AttnConfig *out);
cudaError_t config_fp4(int D, int rows, AttnConfig *out);

// The kernel and its grid on the current device.
cudaError_t grid_blocks(int dtype, int D, int rows, AttnConfig *cfg, int *blocks);
cudaError_t launch_attention(AttnArgs &a, const AttnConfig &cfg, cudaStream_t s);

}  // namespace attn
}  // namespace dvl
