// Cached tokens that stay move together, in place: for every sequence, token
// first + keep[i] to place first + i, i < count, keep rising.
//
// Pure data movement, bound by HBM for long lists and by a chain of dependent
// loads (count, keep -> page -> row) for the few tokens of a verification.
//
// Order.  A row may be another's target (keep[j] = i, j < i: row i is read for
// place j and written from keep[i]), so it is read first.  keep rises, hence
// keep[i] >= i: what a step of consecutive i reads lies at or past what it and
// every earlier step writes, and one barrier between a step's reads and its
// writes is all the order there is to keep -- among the threads that touch the
// same bytes.  Those are one block: a block owns 32 columns (16 bytes each) of
// a token, of one sequence, and walks its list, so blocks never meet.
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 8;  // of a warp's step

template <typename U>
__device__ __forceinline__ void keep_columns(const KeepArgs &a, const KeepPool &pool, int b, int col)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int count = max(0, min(a.counts[b], a.M));
    const int first = max(0, a.first[b]);
    const int64_t length = min((int64_t)a.lengths[b], (int64_t)a.width * a.page_size);
    const bool mine = col < pool.cols;
    const int head = col / pool.units;
    unsigned char *at = pool.base + (int64_t)head * pool.head + (col - head * pool.units) * (int)sizeof(U);
    for (int i0 = 0; i0 < count; i0 += kWarps * kRows) {
        // lanes 0 .. kRows - 1 look up where the warp's rows are, the next
        // kRows where they go
        const int i = i0 + warp * kRows + lane % kRows;
        int64_t place = -1, other = -1;
        if (lane < 2 * kRows && i < count) {
            const int from = a.keep[b * a.keep_stride + i];
            const int64_t source = from < 0 ? -1 : (int64_t)first + from;
            place = lane < kRows ? source : (int64_t)first + i;
            other = lane < kRows ? (int64_t)first + i : source;
        }
        int page = -1, slot = 0;
        if (place >= 0 && place != other && place < length) {
            const int entry = (int)place / a.page_size;
            slot = (int)place - entry * a.page_size;
            page = a.table[b * a.table_stride + entry];
            if ((unsigned)page >= (unsigned)a.pages)
                page = -1;
        }
        U v[kRows];
        unsigned char *dst[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int sp = __shfl_sync(kFull, page, j), ss = __shfl_sync(kFull, slot, j);
            const int dp = __shfl_sync(kFull, page, kRows + j), ds = __shfl_sync(kFull, slot, kRows + j);
            dst[j] = nullptr;
            if (mine && sp >= 0 && dp >= 0) {
                dst[j] = at + dp * pool.page + (int64_t)ds * pool.token;
                v[j] = *reinterpret_cast<const U *>(at + sp * pool.page + (int64_t)ss * pool.token);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (dst[j])
                *reinterpret_cast<U *>(dst[j]) = v[j];
    }
}

__global__ void __launch_bounds__(kThreads) cache_keep_kernel(const __grid_constant__ KeepArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x / a.blocks, blk = blockIdx.x - b * a.blocks;
    if (blk == 0 && threadIdx.x == 0 && a.lengths_out)
        a.lengths_out[b] = max(0, a.first[b]) + max(0, min(a.counts[b], a.M));
    int p = a.n_pools - 1;
    while (blk < a.pool[p].first_block)
        --p;
    const KeepPool &pool = a.pool[p];
    const int col = (blk - pool.first_block) * 32 + (threadIdx.x & 31);
    if (pool.wide)
        keep_columns<uint4>(a, pool, b, col);
    else
        keep_columns<uint32_t>(a, pool, b, col);
}

}  // namespace

cudaError_t launch_cache_keep(KeepArgs &a, cudaStream_t s)
{
    a.blocks = 0;
    for (int p = 0; p < a.n_pools; ++p) {
        a.pool[p].first_block = a.blocks;
        a.blocks += (a.pool[p].cols + 31) / 32;
    }
    if ((int64_t)a.blocks * a.B > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(cache_keep_kernel, (unsigned)(a.blocks * a.B), kThreads, 0, s, a);
}

}  // namespace dvl
