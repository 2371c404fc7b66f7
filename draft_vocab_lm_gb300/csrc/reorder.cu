// Reordering of per-beam rows after a selection, and the private copy of
// each new beam's partly filled cache page, in one launch.
//
// Pure data movement, bound by HBM (or by the launch, for a few rows).  One
// block copies one piece of at most kPiece bytes of one destination row:
// every thread keeps four 16-byte loads in flight (two: 29.0 us for 128 rows
// of 517 KB and their pages, against 22.1 of HBM time).  The block index walks the
// states, the page table and the lengths (ReorderItem.first_block), then the
// pages; a page's blocks read how many of its tokens are filled and leave if
// their piece lies past that.
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;                       // per thread
constexpr int kPiece = kThreads * 16 * kLoads;  // bytes per block

// The source row of new beam r = b * k + i, or -1 for an unused slot.
__device__ __forceinline__ int64_t source_row(const ReorderArgs &a, int64_t r)
{
    const int parent = __ldg(a.parents + r);
    return (unsigned)parent < (unsigned)a.beams ? r / a.k * a.beams + parent : -1;
}

__device__ __forceinline__ void copy_piece(const ReorderArgs &a, const ReorderItem &it, int64_t blk)
{
    const int64_t r = blk / it.pieces;
    const int64_t off = (blk - r * it.pieces) * kPiece;
    const int n = (int)(it.row_bytes - off < kPiece ? it.row_bytes - off : kPiece);
    const int64_t from = source_row(a, r);
    const unsigned char *src = it.src + from * it.src_stride + off;
    unsigned char *dst = it.dst + r * it.dst_stride + off;
    if (it.wide) {
        uint4 v[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int i = (j * kThreads + (int)threadIdx.x) * 16;
            v[j] = from >= 0 && i < n ? *reinterpret_cast<const uint4 *>(src + i)
                                      : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int i = (j * kThreads + (int)threadIdx.x) * 16;
            if (i < n)
                *reinterpret_cast<uint4 *>(dst + i) = v[j];
        }
    } else {
        for (int i = threadIdx.x; i < n; i += kThreads)
            dst[i] = from >= 0 ? src[i] : (unsigned char)0;
    }
}

// The page table row of new beam r: the parent's, with the spare page at the
// slot that the next token goes to.
__device__ __forceinline__ void copy_table(const ReorderArgs &a, const ReorderItem &it, int64_t blk)
{
    const int64_t r = blk / it.pieces;
    const int w0 = (int)(blk - r * it.pieces) * (kPiece / 4);
    const int w1 = min(w0 + kPiece / 4, a.pages.width);
    const int64_t from = source_row(a, r);
    const int32_t *src = a.pages.table + from * a.pages.width;
    int32_t *dst = a.pages.table_out + r * a.pages.width;
    const int slot = from >= 0 ? max(a.pages.lengths[from], 0) / a.cache.page_size : -1;
    for (int i = w0 + threadIdx.x; i < w1; i += kThreads)
        dst[i] = from < 0 ? 0 : i == slot ? a.pages.spare[r] : src[i];
}

// Piece `blk` of the pages of new beam r: keys, then values, of the rows; of an
// NVFP4 cache also of their scales, which lie as the rows do, in an eighth of
// the room, 4 bytes at a time.
template <typename U, bool SCALES>
__device__ __forceinline__ void copy_page(const ReorderArgs &a, int64_t blk, int pieces)
{
    const dvl_kv_cache &c = a.cache;
    const int64_t r = blk / (2 * pieces);
    const int piece = (int)(blk - r * (2 * pieces));
    const bool values = piece >= pieces;
    const int64_t from = source_row(a, r);
    if (from < 0)
        return;
    const int length = max(a.pages.lengths[from], 0);
    const int slot = length / c.page_size;
    constexpr int kDown = SCALES ? 3 : 0;
    const int units = (a.head_bytes >> kDown) / (int)sizeof(U);  // of one head of one token
    const int total = length % c.page_size * c.heads * units;
    const int u0 = (piece - (values ? pieces : 0)) * (kThreads * kLoads);
    if (u0 >= total || slot >= a.pages.width)
        return;
    const int src_page = a.pages.table[from * a.pages.width + slot];
    const int dst_page = a.pages.spare[r];
    if ((unsigned)src_page >= (unsigned)c.pages || (unsigned)dst_page >= (unsigned)c.pages)
        return;
    const int64_t ps = a.strides[values].page >> kDown;
    // (offsets within a page are below 2^31)
    const uint32_t ts = (uint32_t)(a.strides[values].token >> kDown);
    const uint32_t hs = (uint32_t)(a.strides[values].head >> kDown);
    unsigned char *base = static_cast<unsigned char *>(
        SCALES ? (values ? c.v_blocks : c.k_blocks) : (values ? c.v : c.k));
    U v[kLoads];
    uint32_t at[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int u = u0 + (int)threadIdx.x + j * kThreads;
        if (u < total) {
            const int th = u / units, unit = u - th * units;
            const int tok = th / c.heads, head = th - tok * c.heads;
            at[j] = tok * ts + head * hs + unit * (int)sizeof(U);
            v[j] = *reinterpret_cast<const U *>(base + src_page * ps + at[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
        if (u0 + (int)threadIdx.x + j * kThreads < total)
            *reinterpret_cast<U *>(base + dst_page * ps + at[j]) = v[j];
}

// FOUR: the cache is NVFP4.  (Copies live from the threads an SM holds: 32
// registers let it hold all 2,048; at 36, 128 rows of 517 KB took 2 % longer,
// with the scales' code in the same kernel 4 %.)
template <bool FOUR>
__global__ void __launch_bounds__(kThreads, 8) beam_reorder_kernel(const __grid_constant__ ReorderArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t blk = blockIdx.x;
    if (blk >= a.copy_blocks) {
        const int64_t at = blk - a.copy_blocks;
        if constexpr (FOUR) {
            const int64_t rows = (int64_t)a.batch * a.k * 2 * a.page_pieces;
            if (at >= rows) {
                copy_page<uint32_t, true>(a, at - rows, a.block_pieces);
                return;
            }
        }
        copy_page<uint4, false>(a, at, a.page_pieces);
        return;
    }
    int i = a.n_items - 1;
    while (blk < a.item[i].first_block)
        --i;
    const ReorderItem &it = a.item[i];
    if (a.pages.table && it.dst == reinterpret_cast<unsigned char *>(a.pages.table_out))
        copy_table(a, it, blk - it.first_block);
    else
        copy_piece(a, it, blk - it.first_block);
}

}  // namespace

cudaError_t launch_beam_reorder(ReorderArgs &a, cudaStream_t s)
{
    const int64_t rows = (int64_t)a.batch * a.k;
    int64_t blocks = 0;
    for (int i = 0; i < a.n_items; ++i) {
        ReorderItem &it = a.item[i];
        it.pieces = (int)((it.row_bytes + kPiece - 1) / kPiece);
        it.wide = aligned(it.src, 16) && aligned(it.dst, 16) && it.row_bytes % 16 == 0 &&
                  it.src_stride % 16 == 0 && it.dst_stride % 16 == 0;
        it.first_block = blocks;
        blocks += rows * it.pieces;
    }
    a.copy_blocks = blocks;
    a.page_pieces = a.block_pieces = 0;
    if (a.pages.table) {
        const int64_t bytes = (int64_t)(a.cache.page_size - 1) * a.cache.heads * a.head_bytes;
        a.page_pieces = (int)((bytes + kPiece - 1) / kPiece);
        if (a.cache.dtype == DVL_NVFP4)
            a.block_pieces = (int)((bytes / 8 + kPiece / 4 - 1) / (kPiece / 4));
        blocks += rows * 2 * (a.page_pieces + a.block_pieces);
    }
    if (blocks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    if (blocks == 0)
        return cudaSuccess;
    const auto kernel = a.block_pieces ? beam_reorder_kernel<true> : beam_reorder_kernel<false>;
    return launch_pdl(kernel, (unsigned)blocks, kThreads, 0, s, a);
}

}  // namespace dvl
