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
// same bytes.  Those are one block: a block owns a few columns (16 bytes each)
// of a token, of one sequence, and walks its list, so blocks never meet.
//
// Measured (GB300, wall time a call back to back): half of 16 x 16,381 tokens of
// 8 x 128 in 4 bits 52 us (228 MB, 0.65 of the copy rate; with 512 threads and four
// loads a lane 59), in E4M3 78-82 (0.7), in bf16 148 (0.77).  A block's 16 steps of a
// read, a barrier and a write follow each other here; by the order above they need
// not: what step s + 1 reads lies at or past what step s writes, so its loads could
// be in flight across the barrier.  One such list: 18, 25 and 19 us, the same steps
// on few blocks.  A path of 7 of one request's tree 3.2 us and 64 requests' 3.1 to
// 3.3, the host's side of the call.
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 8;  // loads in flight per lane

// Where a row of the list lies and goes in the block's columns, in bytes from
// the pool's start; from < 0: nowhere.
struct Move {
    int64_t from, to;
};

// A step: every warp moves kRows * (32 / COLS) rows, 32 / COLS at a time.
template <typename U, int COLS>
__device__ __forceinline__ void keep_columns(const KeepArgs &a, const KeepPool &pool, int b, int col0)
{
    constexpr int kAtOnce = 32 / COLS;             // rows of a load
    constexpr int kMine = kRows * kAtOnce;         // rows of a warp's step
    constexpr int kLook = (kMine + 31) / 32;       // looked up by a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int count = max(0, min(a.counts[b], a.M));
    const int first = max(0, a.first[b]);
    const int64_t length = min((int64_t)a.lengths[b], (int64_t)a.width * a.page_size);
    const int32_t *keep = a.keep + b * a.keep_stride, *table = a.table + b * a.table_stride;
    const int col = col0 + lane % COLS;
    const bool mine = col < pool.cols;
    const int head = col / pool.units;
    unsigned char *at = pool.base + head * pool.head + (col - head * pool.units) * (int)sizeof(U);

    auto place = [&](int64_t pos) -> int64_t {
        const int entry = (int)((uint64_t)(uint32_t)pos * a.page_mul >> a.page_shift);
        const int page = table[entry];
        return (unsigned)page < (unsigned)a.pages ? page * pool.page + (pos - entry * a.page_size) * pool.token
                                                  : -1;
    };
    // the list's entries of a step, and from them its places
    auto entries = [&](int64_t i0, int (&from)[kLook]) {
#pragma unroll
        for (int k = 0; k < kLook; ++k) {
            const int r = 32 * k + lane;
            const int64_t i = i0 + warp * kMine + r;
            from[k] = -1;
            if ((kMine >= 32 || r < kMine) && i < count)
                from[k] = keep[i];
        }
    };
    auto places = [&](int64_t i0, const int (&from)[kLook], Move (&m)[kLook]) {
#pragma unroll
        for (int k = 0; k < kLook; ++k) {
            const int64_t src = (int64_t)first + from[k], dst = first + i0 + warp * kMine + 32 * k + lane;
            m[k].from = m[k].to = -1;
            if (from[k] >= 0 && src != dst && src < length && dst < length) {
                m[k].from = place(src);
                m[k].to = place(dst);
                if (m[k].to < 0)
                    m[k].from = -1;
            }
        }
    };
    constexpr int kStep = kWarps * kMine;
    Move now[kLook];
    int from[kLook];
    entries(0, from);
    places(0, from, now);
    entries(kStep, from);
    for (int64_t i0 = 0; i0 < count; i0 += kStep) {
        U v[kRows];
        int64_t to[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int r = j * kAtOnce + lane / COLS;  // of the warp's rows
            const int64_t at_row = __shfl_sync(kFull, now[j * kAtOnce / 32].from, r & 31);
            to[j] = __shfl_sync(kFull, now[j * kAtOnce / 32].to, r & 31);
            if (at_row < 0 || !mine)
                to[j] = -1;
            else
                v[j] = *reinterpret_cast<const U *>(at + at_row);
        }
        // while its rows are on their way, the next step's places are looked up
        // and the entries of the one after read (past the list's end: none)
        if (i0 + kStep < count) {
            places(i0 + kStep, from, now);
            entries(i0 + 2 * kStep, from);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (to[j] >= 0)
                *reinterpret_cast<U *>(at + to[j]) = v[j];
    }
}

template <int COLS>
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
    const int col = (blk - pool.first_block) * COLS;
    if (pool.wide)
        keep_columns<uint4, COLS>(a, pool, b, col);
    else
        keep_columns<uint32_t, COLS>(a, pool, b, col);
}

}  // namespace

cudaError_t launch_cache_keep(KeepArgs &a, cudaStream_t s)
{
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    auto blocks = [&](int cols) {
        int64_t n = 0;
        for (int p = 0; p < a.n_pools; ++p)
            n += (a.pool[p].cols + cols - 1) / cols;
        return n;
    };
    // Columns per block: 32 (512 bytes a row) where a list is one step of a block,
    // else as many of 32, 8, 4 or 2 as leave two blocks an SM.  Half of B x 16,381
    // tokens of 8 x 128, us with 32, 8, 4 and 2 columns (* what the rule gives):
    //   4 bits  16: 172, 72, 52*, 72   4: 123, 45, 42, 27*   1: 76, 21, 16, 18*
    //   E4M3    16: 214, 86, 82*, 94   4: 163, 67, 47, 34*   1: 108, 30, 21, 25*
    //   bf16    16: 251, 149*, 140, 180   4: 144, 67, 47, 55*   1: 91, 29, 28, 19*
    // and of 64 x 4,095: 4 bits 66, 45*, 48, 72, bf16 142*, 129, 134, 198.  So it is
    // within 18 % of the best of them.
    int cols = 32;
    if (a.M > kRows * kWarps)
        while (cols > 2 && a.B * blocks(cols) < 2 * di.sms)
            cols = cols == 32 ? 8 : cols / 2;
    int64_t n = 0;
    for (int p = 0; p < a.n_pools; ++p) {
        a.pool[p].first_block = (int)n;
        n += (a.pool[p].cols + cols - 1) / cols;
    }
    if (n * a.B > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    a.blocks = (int)n;
    const auto kernel = cols == 32  ? cache_keep_kernel<32>
                        : cols == 8 ? cache_keep_kernel<8>
                        : cols == 4 ? cache_keep_kernel<4>
                                    : cache_keep_kernel<2>;
    return launch_pdl(kernel, (unsigned)(n * a.B), kThreads, 0, s, a);
}

}  // namespace dvl
