// Attention over a paged cache: the launch, and the join of the parts of
// (sequence, head) pairs that were cut between blocks.
#include <cuda_runtime.h>

#include "dvl_attention.h"
#include "dvl_device.cuh"

namespace dvl {
namespace attn {
namespace {

constexpr int kJoinThreads = 256;

// One block per (sequence, query row of a cached head).  It finds the
// units of its (sequence, head) from the lengths, as the attention blocks
// did, hence which blocks hold a part and where; a pair that one block
// finished is left alone.  Thread = (group of parts, 4 columns); each adds
// its parts with weight 2^(m_part - m), and the groups meet in shared memory.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnArgs a)
{
    __shared__ int64_t s_before[kJoinThreads / 32], s_all[kJoinThreads / 32];
    __shared__ float4 s_acc[kJoinThreads];
    __shared__ float s_m[kJoinThreads / 32], s_l[kJoinThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kW = kJoinThreads / 32;
    const int r = blockIdx.x % a.rows;
    const int bh = blockIdx.x / a.rows;
    const int b = bh / a.heads, h = bh - b * a.heads;
    int64_t before = 0, all = 0;
    int len = 0;
    for (int i = threadIdx.x; i < a.B; i += kJoinThreads) {
        const int n = min(max(a.lengths[i], 0), a.max_len);
        const int tiles = (n + kTile - 1) / kTile;
        all += tiles;
        before += i < b ? tiles : 0;
    }
    len = min(max(a.lengths[b], 0), a.max_len);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        before += __shfl_xor_sync(kFull, before, off);
        all += __shfl_xor_sync(kFull, all, off);
    }
    if (lane == 0) {
        s_before[warp] = before;
        s_all[warp] = all;
    }
    __syncthreads();
    before = all = 0;
    for (int w = 0; w < kW; ++w) {
        before += s_before[w];
        all += s_all[w];
    }
    const int tiles = (len + kTile - 1) / kTile;
    const int t = r / a.G;
    const int64_t at = ((int64_t)b * a.T + t) * a.Hq + h * a.G + (r - t * a.G);
    if (tiles == 0) {  // an empty sequence
        for (int d = threadIdx.x; d < a.D; d += kJoinThreads)
            a.out[at * a.D + d] = 0;
        if (a.lse && threadIdx.x == 0)
            a.lse[at] = -__builtin_huge_valf();
        return;
    }
    const int64_t units = all * a.heads;
    const int64_t first = before * a.heads + (int64_t)h * tiles, last = first + tiles - 1;
    // block c holds unit u when floor(c U / blocks) <= u < floor((c + 1) U / blocks)
    const int64_t blocks = used_blocks(a.blocks, units);
    const int c0 = (int)(((first + 1) * blocks - 1) / units);
    const int c1 = (int)(((last + 1) * blocks - 1) / units);
    if (c0 == c1)
        return;
    auto part_of = [&](int c) {
        // a block's first pair is in its slot 0, a later one in slot 1
        const int slot = c == c0 && c * units / blocks < first ? 1 : 0;
        return a.parts + (2 * (int64_t)c + slot) * a.part_floats;
    };

    const int stat = a.rows * a.D + 2 * r;
    float m = -__builtin_huge_valf();
    for (int c = c0 + threadIdx.x; c <= c1; c += kJoinThreads)
        m = fmaxf(m, part_of(c)[stat]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    if (lane == 0)
        s_m[warp] = m;
    __syncthreads();
    m = s_m[0];
    for (int w = 1; w < kW; ++w)
        m = fmaxf(m, s_m[w]);
    const float ref = m == -__builtin_huge_valf() ? 0.f : m;
    float l = 0.f;
    for (int c = c0 + threadIdx.x; c <= c1; c += kJoinThreads) {
        const float *p = part_of(c) + stat;
        l += p[1] * exp2f(p[0] - ref);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        l += __shfl_xor_sync(kFull, l, off);
    if (lane == 0)
        s_l[warp] = l;

    const int cols = a.D / 4;
    const int groups = kJoinThreads / cols;
    const int grp = threadIdx.x / cols, col = threadIdx.x - grp * cols;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp < groups)
#pragma unroll 4
        for (int c = c0 + grp; c <= c1; c += groups) {
            const float *p = part_of(c);
            const float w = exp2f(p[stat] - ref);
            const float4 x = *reinterpret_cast<const float4 *>(p + r * a.D + 4 * col);
            acc.x = fmaf(w, x.x, acc.x);
            acc.y = fmaf(w, x.y, acc.y);
            acc.z = fmaf(w, x.z, acc.z);
            acc.w = fmaf(w, x.w, acc.w);
        }
    s_acc[threadIdx.x] = acc;
    __syncthreads();
    l = 0.f;
    for (int w = 0; w < kW; ++w)
        l += s_l[w];
    if (grp == 0) {
        for (int i = 1; i < groups; ++i) {
            const float4 x = s_acc[i * cols + col];
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
        }
        // a row without positions (or of -inf scores only): 0
        const float f = l == 0.f ? 0.f : a.v_scale / l;
        uint32_t lo, hi;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(acc.y * f), "f"(acc.x * f));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(acc.w * f), "f"(acc.z * f));
        *reinterpret_cast<uint2 *>(a.out + at * a.D + 4 * col) = make_uint2(lo, hi);
        if (a.lse && threadIdx.x == 0)
            a.lse[at] = log_sum(m, l);
    }
}

}  // namespace

cudaError_t grid_blocks(bool fp8, int D, int rows, AttnConfig *cfg, int *blocks)
{
    cudaError_t e = fp8 ? config_fp8(D, rows, cfg) : config_bf16(D, rows, cfg);
    DeviceInfo di;
    if (e == cudaSuccess)
        e = device_info(&di);
    int per_sm = 0;
    if (e == cudaSuccess)
        e = blocks_per_sm(cfg->func, 128, cfg->smem, &per_sm);
    if (e != cudaSuccess)
        return e;
    if (per_sm < 1)
        return cudaErrorInvalidConfiguration;
    *blocks = per_sm * di.sms;
    return cudaSuccess;
}

cudaError_t launch_attention(AttnArgs &a, bool fp8, cudaStream_t s)
{
    AttnConfig cfg;
    cudaError_t e = grid_blocks(fp8, a.D, a.rows, &cfg, &a.blocks);
    if (e != cudaSuccess)
        return e;
    using Kernel = void (*)(AttnArgs);
    e = launch_pdl(reinterpret_cast<Kernel>(const_cast<void *>(cfg.func)), (unsigned)a.blocks, 128,
                   cfg.smem, s, a);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(join_kernel, (unsigned)((int64_t)a.B * a.heads * a.rows), kJoinThreads, 0, s,
                      a);
}

}  // namespace attn
}  // namespace dvl
