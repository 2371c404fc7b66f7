// Attention of the newest tokens of many sequences over a paged key-value
// cache, split over the caches' lengths and joined.  Per sequence, cached
// head and query row (token t, head g of the group; n visible positions):
//   s_j = scale q . k_j,   out = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m}.
//
// Bound by HBM: a cached token costs 2 D values and 4 D flops per query row,
// so with up to 64 rows per cached head the tensor cores idle most of the
// time.  The rows of one cached head share every load: they are the M rows
// of the matrix products (16 per MMA).
//
// Work split.  The unit is a tile of TOK G tokens of one (sequence, cached
// head).  The blocks of a grid that is resident at once form lanes, one per
// head of a set of up to eight; a lane's units in a row (by sequence, set,
// tile) are cut into one equal share per block, so unequal lengths balance by
// themselves and the host needs to know none of them, and the blocks of one
// share index walk the same tokens of neighbouring heads at the same time
// (in the usual layout the heads of a token are neighbours in memory: 64
// sequences of up to 16,381 tokens, 8 FP8 heads of 64, all lanes apart: 195
// us; heads first in memory: 131).  A block walks its share through a ring of
// chunks in shared memory, filled by 16-byte asynchronous copies that run
// ahead across sequence boundaries.
//
// Joining.  A (sequence, head) that lies in one share is finished by its
// block.  The parts of one that was cut go to the workspace as
// (unnormalised sums, maximum, sum of weights); the last block of every
// kJoin consecutive parts (by a wrapping ticket, as in the reducing
// kernels) adds them in order of the shares, and where there are more, the
// last of those adds the groups' sums, so the result does not depend on
// timing and no second launch is needed.
//
// Warps.  A group of warps (one per 16 query rows) owns TOK consecutive tokens
// of every tile: it finds their pages, copies their rows, and runs its own
// softmax over them -- running maximum, sum and output rows stay in
// registers, the weights go from the score accumulators straight into the
// operand registers of the second product -- so no warp waits for another
// within a (sequence, head); the groups' results meet in shared memory at its
// end.  (Sharing a tile across the block, each warp with a slice of the
// columns, took three block barriers per tile.)  The group's ring holds keys
// and values of P + 1 chunks less one entry, keys and values as entries of
// their own: the next chunk's keys load while this chunk's scores are formed,
// its values while the values are used, which keeps P chunks per group in
// flight in the least shared memory, hence the most warps per SM.
// Up to 8 query rows (RT = 0) the upper half of every MMA is padding: its
// softmax is left out and its accumulators are not kept.
//
// Weights are rounded to the MMA operand type, at most 2^-8 relative for bf16
// and 2^-11 for f16, independently per position; sums and statistics stay
// fp32.  That keeps the second product on the tensor cores and costs little
// next to the output's own rounding to bf16 (error against 64 bits 1.00 to
// 1.07 of that with fp32 weights over short to long caches).  f16 weights are
// multiplied by 2^15 first (the largest is 1): they are normal numbers down to
// 2^-29 of the largest and lie on a grid of 2^-39 below, so a long tail far
// under one position keeps its share, which unscaled it lost (40,000 positions
// 18 nats down: all of it).  Output sums are in that unit until they are
// divided.  Scores are kept in units of log2 (the scale carries log2 e), so a
// weight is one ex2.
//
// Operands.  bf16 cache: mma m16n8k16 bf16, K and V by ldmatrix (V
// transposed).  FP8 cache: E4M3 pairs are widened to f16 (exact) in
// registers, mma m16n8k16 f16; a query row is multiplied by a power of two
// that puts its largest value in [2^14, 2^15), which keeps every bf16 value
// down to 2^-29 of the row's largest exact in f16 (smaller ones round to the
// f16 subnormal grid, at most 2^-38 of the largest), and the power is taken
// out of the score's fp32 scale.  The order of the D values inside an MMA is
// permuted so that a lane's FP8 bytes are consecutive; Q is stored in the same
// order.
//
// Masks.  Row t sees n = length - (T - 1 - t) positions.  Scores at or past
// n are replaced, not added to, so nothing a masked key holds can show; a
// row without positions keeps the sum 0 and gives 0.  Positions that only
// some rows see (the last T - 1) are added value by value for the rows that
// see them, and their V rows zeroed before the MMA: 0 times a NaN or an
// infinity in V would otherwise reach the rows that do not.  Rows past the
// length are zeros from the copy.
#pragma once

#include <cuda_runtime.h>

#include "dvl_async.cuh"
#include "dvl_attention.h"
#include "dvl_device.cuh"

namespace dvl {
namespace attn {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kJoin = 16;  // parts per first-level join
constexpr float kF16Weight = 32768.f;  // a weight of 1 among f16 operands (FP8 caches)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint16_t lds8(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint16_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// D += A B, m16n8k16, fp32 accumulators; FP8 caches run it on f16 operands.
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1)
{
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same where only rows g (NJ = 1) or rows g and g + 8 are kept.
template <bool F16, int NJ>
__device__ __forceinline__ void mma_rows(float (&o)[2 * NJ], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    float c[4] = {o[0], o[1], NJ == 2 ? o[2 * NJ - 2] : 0.f, NJ == 2 ? o[2 * NJ - 1] : 0.f};
    mma16<F16>(c, a, b0, b1);
    o[0] = c[0];
    o[1] = c[1];
    if constexpr (NJ == 2) {
        o[2] = c[2];
        o[3] = c[3];
    }
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool F16>
__device__ __forceinline__ float unpack1(uint16_t x)
{
    if constexpr (F16) {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(x));
        return f;
    } else {
        return __uint_as_float((uint32_t)x << 16);
    }
}

// Two weights as operands of the second product: f16 ones in units of 2^-15.
template <bool F16>
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi)
{
    return F16 ? pack2<true>(lo * kF16Weight, hi * kF16Weight) : pack2<false>(lo, hi);
}

// Two E4M3 bytes -> two f16 (exact); four bytes -> two such pairs.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t x)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    return r;
}
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Walks a lane's units from (sequence b, head h, tile t) on.
template <int TILE>
struct Cursor {
    int b, h, t, len, tiles;
    __device__ __forceinline__ void next(const AttnArgs &a)
    {
        if (b >= a.B || ++t < tiles)
            return;
        t = 0;
        h += a.lanes;
        if (h < a.heads)
            return;
        h %= a.lanes;
        do {
            if (++b >= a.B)
                return;  // past the last unit
            len = seq_len(a, b);
        } while (len == 0);
        tiles = (len + TILE - 1) / TILE;
    }
};

// DP: head width padded to 64, 128 or 256.  RT: 16-row tiles of query rows; 0
// for at most 8 rows.  TOK: tokens per group and tile.  P: chunks in flight.
// G: groups, so G TOK tokens per tile.
constexpr int max_of(int x, int y) { return x > y ? x : y; }

// The most columns (DP halved as often as needed) of `bytes` each that fit.
constexpr int round_columns(int dp, int bytes, int room)
{
    return dp * bytes <= room ? dp : round_columns(dp / 2, bytes, room);
}

template <int DP, bool FP8, int RT, int TOK, int P, int G>
struct Shape {
    static constexpr int kElem = FP8 ? 1 : 2;
    static constexpr int kTile = TOK * G;
    static_assert(kTile <= 128, "lengths are limited so that a tile more fits 32 bits");
    static constexpr int kGroup = RT == 0 ? 32 : 32 * RT;  // threads
    static constexpr int kThreads = kGroup * G;
    // Rows that one access phase touches lie on distinct banks.  bf16: the
    // 16-byte units of a row are permuted by its lowest three bits (8 rows of
    // an ldmatrix).  FP8: padded pitches (8-byte loads of 4 rows for K, 4-byte
    // loads of every other row for V).
    static constexpr int kKPitch = FP8 ? DP + 32 : DP * 2;
    static constexpr int kVPitch = FP8 ? DP + 16 : DP * 2;
    static constexpr int kQPitch = DP * 2 + 16;
    static constexpr int kRows = RT == 0 ? 8 : 16 * RT;    // query rows kept
    static constexpr int kQRows = RT == 0 ? 16 : 16 * RT;  // rows of the operand
    // One ring entry: a chunk's keys or values; also 32 columns of the rows.
    static constexpr int kEntry = max_of(TOK * kKPitch, kRows * 4 * 32);
    static constexpr int kEntries = 2 * P + 1;
    static constexpr int kRing = kEntries * kEntry;        // per group
    // At a pair's end every group lays its output rows, kRound columns at a
    // time, into the ring entry that is free then.
    static constexpr int kRound = round_columns(DP, kRows * 4, kEntry);
    static_assert(kRound >= 32 && kEntry % 16 == 0, "rows are permuted within 32 columns");
    static constexpr int kQ = G * kRing;
    static constexpr int kStat = kQ + kQRows * kQPitch;    // float2[G][kRows]: maximum, sum
    static constexpr int kScale = kStat + G * kRows * 8;   // float[kQRows]
    static constexpr int kAddr = kScale + kQRows * 4;      // pointers [G][P + 1][2][TOK]
    static constexpr int kBytes = kAddr + G * (P + 1) * 2 * TOK * 8;
};

// The output column of accumulator e (of a row) of column tile n.
template <bool FP8>
__device__ __forceinline__ int out_col(int n, int c, int e)
{
    return FP8 ? n / 4 * 32 + 4 * (2 * c + e) + n % 4 : 8 * n + 2 * c + e;
}

// The permutation of a row's columns while the groups' rows are joined.
template <bool FP8>
__device__ __forceinline__ int swizzle(int r)
{
    return FP8 ? (r & 1) << 2 : (r & 3) << 3;
}

// Where a token's row starts, found by one thread per token a chunk before the
// copies need it: the page id is read from the table one chunk earlier still,
// so no copy waits for the table.
struct RowAddress {
    uint32_t k, v;  // byte offsets within the page
    int id;         // page id, not yet checked
    bool has;       // a cached token

    template <int TILE>
    __device__ __forceinline__ void fetch(const AttnArgs &a, const Cursor<TILE> &it, int r)
    {
        const int pos = it.t * TILE + r;
        has = it.b < a.B && pos < it.len;
        if (!has)
            return;
        const int page = a.page_of(pos);
        id = __ldg(a.table + it.b * a.table_stride + page);
        const uint32_t slot = pos - page * a.page_size;
        k = slot * a.kt + it.h * a.kh;
        v = slot * a.vt + it.h * a.vh;
    }
    // The row's addresses.  A page outside the pool is reported, and read as
    // page 0; past the length nothing is read through the address.
    __device__ __forceinline__ void resolve(const AttnArgs &a, const unsigned char **rows,
                                            int tok) const
    {
        const unsigned char *pk = a.k, *pv = a.v;
        if (has) {
            int page = id;
            if ((unsigned)page >= (unsigned)a.pages) {
                set_status(a.ws, 1u << DVL_ERR_OUT_OF_RANGE);
                page = 0;
            }
            pk += page * a.kp + k;
            pv += page * a.vp + v;
        }
        rows[0] = pk;
        rows[tok] = pv;
    }
};

// Copy a chunk's rows (keys or values) into a ring entry, `live` of them; the
// others become zeros, and so do the padding columns of keys: they meet zeros
// of Q and must hold no NaN, which whatever the entry held before may be.
// at: the thread's place among the group's N threads.
template <int DP, bool FP8, int TOK, int N, bool KEYS>
__device__ __forceinline__ void load_rows(int row_bytes, const unsigned char *const *rows, int live,
                                          int at, uint32_t dst, int pitch)
{
    constexpr int kCols = DP * (FP8 ? 1 : 2) / 16;  // 16-byte units of a padded row
    constexpr int kStep = N / kCols;                // rows per pass
    const int col = at % kCols, r0 = at / kCols;
    int from = col * 16;
    if (from >= row_bytes) {
        if (!KEYS)
            return;
        from = live = 0;
    }
    if (r0 >= TOK)
        return;
#pragma unroll
    for (int i = 0; i < (kStep < TOK ? TOK / kStep : 1); ++i) {
        const int r = r0 + i * kStep;
        const int unit = FP8 ? col : col ^ (r & 7);
        cp_async16(dst + r * pitch + unit * 16, rows[r] + from, r < live);
    }
}

// Barrier of one group's N threads.
template <int N>
__device__ __forceinline__ void group_sync(int group)
{
    if constexpr (N == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(N) : "memory");
}

// A block's share of its lane: units [u0, u1) of `units`, cut into `shares`,
// and the sequence that holds unit u0 with u0's place in it.
struct Share {
    int64_t u0, u1, units;
    int shares, b;
    int64_t off;
};

// floor(i n / d) for i <= d < 2^10.
__device__ __forceinline__ int64_t cut(int64_t n, int i, int d)
{
    if (n >> 22 == 0)
        return (uint32_t)n * (uint32_t)i / (uint32_t)d;
    return n * i / d;
}

// The share that holds unit u.
__device__ __forceinline__ int holder(int64_t u, int64_t units, int shares)
{
    const int64_t x = (u + 1) * shares - 1;
    return x >> 32 == 0 && units >> 32 == 0 ? (int)((uint32_t)x / (uint32_t)units)
                                            : (int)(x / units);
}

// Every thread calls it; scratch: 16 + 8 THREADS / 32 bytes.
template <int THREADS, int TILE>
__device__ __forceinline__ Share locate(const AttnArgs &a, int64_t *scratch)
{
    constexpr int kW = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sets = a.heads / a.lanes;
    int64_t *s_off = scratch, *s_b = scratch + 1, *s_warp = scratch + 2;
    Share s;
    int64_t total = 0;
    if (a.B > THREADS) {  // the units of all sequences, before the scan by parts
        for (int b0 = 0; b0 < a.B; b0 += THREADS) {
            const int b = b0 + (int)threadIdx.x;
            // at most 2^26 tiles per sequence
            total += __reduce_add_sync(kFull, b < a.B ? (unsigned)seq_tiles<TILE>(a, b) : 0u);
        }
        if (lane == 0)
            s_warp[warp] = total;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w)
            total += s_warp[w];
        __syncthreads();
    }
    s.shares = 0;
    int64_t carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
        const int b = b0 + (int)threadIdx.x;
        const unsigned mine = b < a.B ? (unsigned)seq_tiles<TILE>(a, b) : 0u;
        unsigned scan = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned o = __shfl_up_sync(kFull, scan, off);
            if (lane >= off)
                scan += o;
        }
        if (lane == 31)
            s_warp[warp] = scan;
        __syncthreads();
        int64_t end = carry + scan;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (w < warp)
                end += s_warp[w];
            carry += s_warp[w];
        }
        if (s.shares == 0) {
            s.units = (a.B > THREADS ? total : carry) * sets;
            s.shares = used_shares(a, s.units);
            const int share = (int)blockIdx.x / a.lanes;
            s.u0 = s.u1 = 0;
            if (share < s.shares) {
                s.u0 = cut(s.units, share, s.shares);
                s.u1 = cut(s.units, share + 1, s.shares);
            }
        }
        end *= sets;
        const int64_t begin = end - (int64_t)mine * sets;
        if (begin <= s.u0 && s.u0 < end) {
            *s_b = b;
            *s_off = s.u0 - begin;
        }
        __syncthreads();
    }
    s.b = (int)*s_b;
    s.off = *s_off;
    return s;
}

// Sequences without tokens: zeros, written by whichever block their index names.
template <int THREADS>
__device__ __forceinline__ void write_empty(const AttnArgs &a)
{
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (threadIdx.x == 0 && a.lengths[b] > a.max_len)
            set_status(a.ws, 1u << DVL_ERR_OUT_OF_RANGE);
        if (seq_len(a, b) != 0)
            continue;
        const int64_t n = (int64_t)a.T * a.Hq;
        for (int64_t i = threadIdx.x; i < n * a.D / 8; i += THREADS)
            reinterpret_cast<uint4 *>(a.out + b * n * a.D)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int64_t i = threadIdx.x; i < n; i += THREADS)
                a.lse[b * n + i] = kNegInf;
    }
}

// Four columns of a finished row: the sums over their weights' sum.
template <bool FP8>
__device__ __forceinline__ void put_row(const AttnArgs &a, int b, int h, int r, int d,
                                        const float4 &acc, float m, float sum)
{
    const int t = a.token_of(r);
    const int64_t to = ((int64_t)b * a.T + t) * a.Hq + h * a.G + (r - t * a.G);
    // a row without positions (or of -inf scores only): 0
    const float inv = sum == 0.f ? 0.f : a.v_scale / (FP8 ? sum * kF16Weight : sum);
    *reinterpret_cast<uint2 *>(a.out + to * a.D + d) =
        make_uint2(pack2<false>(acc.x * inv, acc.y * inv), pack2<false>(acc.z * inv, acc.w * inv));
    if (a.lse && d == 0)
        a.lse[to] = log_sum(m, sum);
}

// Add n parts in order: slot `first`, then second, second + stride, ..  Their
// statistics lie at `stats`.  With `last` the result is the (sequence, head)'s
// output, else its sums replace the first part's and its statistics go behind
// that part's own.  Every thread takes 4 columns of R rows at a time and runs
// through the parts with a running maximum, kBatch parts' loads in flight; no
// shared memory and no barrier.
template <int DP, bool FP8, int THREADS, int R>
__device__ __forceinline__ void join_parts(const AttnArgs &a, int n, int first, int second,
                                           int stride, int stats, bool last, int b, int h)
{
    constexpr int kBatch = 8;
    constexpr int kCols = DP / 4;
    const int d = 4 * ((int)threadIdx.x % kCols);
    if (d >= a.D)
        return;
    constexpr int kStep = THREADS / kCols;  // rows per pass
    float *to_part = a.parts + (int64_t)first * a.part_floats;
    for (int r0 = (int)threadIdx.x / kCols; r0 < a.rows; r0 += R * kStep) {
        float m[R], sum[R];
        float4 acc[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            m[k] = kNegInf;
            sum[k] = 0.f;
            acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            float2 ml[R][kBatch];
            float4 x[R][kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int slot = i0 + i == 0 ? first : second + (i0 + i - 1) * stride;
                const float *p = a.parts + (int64_t)slot * a.part_floats;
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const int r = r0 + k * kStep;
                    ml[k][i] = make_float2(kNegInf, 0.f);
                    x[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i0 + i < n && r < a.rows) {
                        ml[k][i] = __ldcg(reinterpret_cast<const float2 *>(p + stats) + r);
                        x[k][i] = __ldcg(reinterpret_cast<const float4 *>(p + r * a.D + d));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                float big = m[k];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    big = fmaxf(big, ml[k][i].x);
                const float ref = big == kNegInf ? 0.f : big;
                const float alpha = ex2(m[k] - ref);
                m[k] = big;
                sum[k] *= alpha;
                acc[k].x *= alpha, acc[k].y *= alpha, acc[k].z *= alpha, acc[k].w *= alpha;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float w = ex2(ml[k][i].x - ref);
                    sum[k] = fmaf(w, ml[k][i].y, sum[k]);
                    acc[k].x = fmaf(w, x[k][i].x, acc[k].x);
                    acc[k].y = fmaf(w, x[k][i].y, acc[k].y);
                    acc[k].z = fmaf(w, x[k][i].z, acc[k].z);
                    acc[k].w = fmaf(w, x[k][i].w, acc[k].w);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int r = r0 + k * kStep;
            if (r >= a.rows)
                continue;
            if (last) {
                put_row<FP8>(a, b, h, r, d, acc[k], m[k], sum[k]);
            } else {
                // (the part's own statistics may still be read by other threads)
                *reinterpret_cast<float4 *>(to_part + r * a.D + d) = acc[k];
                if (d == 0)
                    reinterpret_cast<float2 *>(to_part + stats + 2 * a.rows)[r] =
                        make_float2(m[k], sum[k]);
            }
        }
    }
}

// A part of a (sequence, head) that this block has written to the workspace.
struct Part {
    int64_t first;  // the pair's first unit in its lane
    int tiles, b, h;
};

// Count the part in; the last block of a group of parts joins them, the last
// of the groups those.  Every thread calls it, after the part's last write.
template <int DP, bool FP8, int THREADS, int R>
__device__ __forceinline__ void finish_part(const AttnArgs &a, const Share &share, const Part &p,
                                            int *s_last)
{
    // The shares that hold the pair: those of its first and last unit (s
    // holds unit u when floor(s U / n) <= u < floor((s + 1) U / n)).
    const int64_t last = p.first + p.tiles - 1;
    const int n = share.shares, mine = (int)blockIdx.x / a.lanes;
    const int s0 = holder(p.first, share.units, n), s1 = holder(last, share.units, n);
    const int lane_of = blockIdx.x % a.lanes;
    // a share's first pair is in its slot 0, a later one in slot 1
    const int slot0 = 2 * (s0 * a.lanes + lane_of) + (cut(share.units, s0, n) < p.first ? 1 : 0);
    auto slot_of = [&](int s) { return s == s0 ? slot0 : 2 * (s * a.lanes + lane_of); };
    const int count = s1 - s0 + 1, index = mine - s0;
    const int from = index / kJoin * kJoin;  // first part of this part's group
    const int size = min(kJoin, count - from);
    const int groups = (count + kJoin - 1) / kJoin;
    const int step = 2 * a.lanes;            // slots from a share to the next
    int stats = a.rows * a.D;
    int parts = size, slot_a = slot_of(s0 + from), slot_b = slot_of(s0 + from + 1), stride = step;
    unsigned int *ticket = a.tickets + slot_a;
    // (one copy of the code for both levels: a short call waits for most of
    // its instructions as it waits for its data)
#pragma unroll 1
    for (int level = 0;; ++level) {
        __syncthreads();
        if (threadIdx.x == 0)
            *s_last = ticket_inc(ticket, parts - 1) == (unsigned)parts - 1;
        __syncthreads();
        if (!*s_last)
            return;
        const bool last_level = level == 1 || groups == 1;
        join_parts<DP, FP8, THREADS, R>(a, parts, slot_a, slot_b, stride, stats, last_level, p.b, p.h);
        if (last_level)
            return;
        parts = groups;
        slot_a = slot0;
        slot_b = slot_of(s0 + kJoin);
        stride = step * kJoin;
        stats += 2 * a.rows;
        ticket = a.tickets + a.top_tickets + slot0;
    }
}

template <int DP, bool FP8, int RT, int TOK, int P, int G, int BLOCKS>
__global__ void __launch_bounds__(Shape<DP, FP8, RT, TOK, P, G>::kThreads, BLOCKS)
    attention_kernel(const __grid_constant__ AttnArgs a)
{
    using S = Shape<DP, FP8, RT, TOK, P, G>;
    constexpr int kThreads = S::kThreads;
    constexpr int kGroup = S::kGroup;
    constexpr int kWarps = kThreads / 32;
    constexpr int NJ = RT == 0 ? 1 : 2;  // row halves kept per MMA (rows g, g + 8)
    constexpr int kNT = DP / 8;          // MMA column tiles of the output
    constexpr int kSN = TOK / 8;         // MMA column tiles of the scores
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_scan[2 + kWarps];
    __shared__ int s_last;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = threadIdx.x / kGroup, at = threadIdx.x % kGroup;  // place in the group
    const int mt = at / 32;                                             // row tile
    const int g = lane >> 2, c = lane & 3;
    const uint32_t base = smem_u32(smem);
    float2 *stat = reinterpret_cast<float2 *>(smem + S::kStat);
    float *row_scale = reinterpret_cast<float *>(smem + S::kScale);

    const Share share = locate<kThreads, S::kTile>(a, s_scan);
    if (share.u0 >= share.u1) {
        write_empty<kThreads>(a);
        return;
    }
    Cursor<S::kTile> cur;
    cur.b = share.b;
    cur.len = seq_len(a, cur.b);
    cur.tiles = (cur.len + S::kTile - 1) / S::kTile;
    const int set = a.heads == a.lanes ? 0 : (int)(share.off / cur.tiles);
    cur.h = set * a.lanes + blockIdx.x % a.lanes;
    cur.t = (int)(share.off - (int64_t)set * cur.tiles);
    const int64_t n_units = share.u1 - share.u0;

    // Q of a (sequence, cached head): row t * G + g; a thread takes 8 values of
    // a row, all of its loads in flight at once -- the block's first ones
    // before the ring's copies fill the memory system's queues.
    constexpr int kUnits = DP / 8;
    constexpr int kPasses = (S::kQRows * kUnits + kThreads - 1) / kThreads;
    uint4 qv[kPasses];
    auto load_q = [&](int b, int h) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = (i * kThreads + (int)threadIdx.x) / kUnits;
            const int d = ((int)threadIdx.x % kUnits) * 8;
            qv[i] = make_uint4(0, 0, 0, 0);
            if (r < a.rows && d < a.D) {
                const int t = a.token_of(r);
                qv[i] = *reinterpret_cast<const uint4 *>(
                    a.q + b * a.qb + t * a.qt + (int64_t)(h * a.G + (r - t * a.G)) * a.qh + d);
            }
        }
    };
    auto store_q = [&]() {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = (i * kThreads + (int)threadIdx.x) / kUnits;
            const int d = ((int)threadIdx.x % kUnits) * 8;
            unsigned char *dst = smem + S::kQ + r * S::kQPitch;
            if constexpr (FP8) {
                const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
                uint32_t big = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    big = max(big, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
#pragma unroll
                for (int off = kUnits / 2; off >= 1; off >>= 1)
                    big = max(big, __shfl_xor_sync(kFull, big, off));
                int e2 = (int)(big >> 23) - 127;
                e2 = e2 < -100 ? -100 : e2 > 127 ? 127 : e2;
                const float up = __uint_as_float((uint32_t)(127 + 14 - e2) << 23);
                if (r < S::kQRows) {
                    // place of value d in the permuted order: block of 32, lane
                    // quarter (d / 8 % 4), step (d / 4 % 2), half (d / 2 % 2)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint32_t *>(
                            dst + 2 * ((d & ~31) + (e >> 1) * 16 + (e & 1) * 8 + ((d >> 3) & 3) * 2)) =
                            pack2<true>(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
                    if (d == 0)
                        row_scale[r] = a.qk_scale * __uint_as_float((uint32_t)(127 + e2 - 14) << 23);
                }
            } else if (r < S::kQRows) {
                *reinterpret_cast<uint4 *>(dst + 2 * d) = qv[i];
                if (d == 0)
                    row_scale[r] = a.qk_scale;
            }
        }
    };
    load_q(cur.b, cur.h);

    // Row addresses are known P + 1 chunks ahead of the chunk in work, page
    // ids one more.
    const unsigned char **addr = reinterpret_cast<const unsigned char **>(smem + S::kAddr) +
                                 group * (P + 1) * 2 * TOK;
    const uint32_t ring = base + group * S::kRing;
    const int row_bytes = a.D * S::kElem;
    RowAddress row;
    Cursor<S::kTile> ahead = cur;  // of the row addresses
    Cursor<S::kTile> load = cur;   // of the copies
    const bool finds = at < TOK;
    if (finds) {
        RowAddress first[P + 1];
#pragma unroll
        for (int i = 0; i < P + 1; ++i) {
            first[i].fetch(a, ahead, TOK * group + at);
            ahead.next(a);
        }
        row.fetch(a, ahead, TOK * group + at);
        ahead.next(a);
#pragma unroll
        for (int i = 0; i < P + 1; ++i)
            first[i].resolve(a, addr + i * 2 * TOK + at, TOK);
    }
    group_sync<kGroup>(group);
    int64_t to_load = n_units;
    int load_slot = 0, load_entry = 0;  // of addr, of the ring
    auto load_keys = [&]() {
        if (to_load > 0)
            load_rows<DP, FP8, TOK, kGroup, true>(row_bytes, addr + load_slot * 2 * TOK,
                                            load.len - load.t * S::kTile - TOK * group, at,
                                            ring + load_entry * S::kEntry, S::kKPitch);
        cp_async_commit();
        load_entry = load_entry + 1 == S::kEntries ? 0 : load_entry + 1;
    };
    auto load_values = [&]() {
        if (to_load > 0)
            load_rows<DP, FP8, TOK, kGroup, false>(row_bytes, addr + load_slot * 2 * TOK + TOK,
                                            load.len - load.t * S::kTile - TOK * group, at,
                                            ring + load_entry * S::kEntry, S::kVPitch);
        cp_async_commit();
        load_entry = load_entry + 1 == S::kEntries ? 0 : load_entry + 1;
        load_slot = load_slot + 1 == P + 1 ? 0 : load_slot + 1;
        --to_load;
        load.next(a);
    };
#pragma unroll
    for (int i = 0; i < P; ++i) {
        load_keys();
        load_values();
    }

    float o[kNT][2 * NJ];
    float m[NJ], l[NJ];
    int sees[NJ], sees_least = 0;
    auto reset = [&]() {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            m[j] = kNegInf;
            l[j] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int e = 0; e < 2 * NJ; ++e)
                o[n][e] = 0.f;
    };
    // Visible positions per row of the (sequence, head) that starts.
    auto start_pair = [&](int len) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int r = 16 * mt + 8 * j + g;
            sees[j] = r < a.rows ? len - (a.T - 1 - a.token_of(r)) : 0;
        }
        sees_least = len - (a.T - 1);
    };
    reset();
    start_pair(cur.len);
    store_q();
    __syncthreads();
    bool first_part = true;  // still in the block's first (sequence, head)
    int t_first = cur.t;
    int entry = 0;
    for (int64_t left = n_units; left > 0; --left) {
        const int pos0 = cur.t * S::kTile + TOK * group;

        // keys
        cp_async_wait<2 * P - 1>();
        group_sync<kGroup>(group);
        load_keys();  // into the entry of the previous values
        const uint32_t k_smem = ring + entry * S::kEntry;
        entry = entry + 1 == S::kEntries ? 0 : entry + 1;
        uint32_t pa[TOK / 16][4];  // the weights as the second product's operand
        float s[kSN][2 * NJ];
        if (pos0 < cur.len) {
            // scores
            float acc[kSN][4];
#pragma unroll
            for (int n = 0; n < kSN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[n][e] = 0.f;
            const uint32_t q_row =
                base + S::kQ + (16 * mt + (lane & 15)) * S::kQPitch + (lane >> 4) * 16;
            if constexpr (FP8) {
                const uint32_t k_row = k_smem + g * S::kKPitch + 8 * c;
#pragma unroll
                for (int d = 0; d < DP; d += 32) {
                    uint32_t qa[2][4];
                    ldsm4(qa[0], q_row + d * 2);
                    ldsm4(qa[1], q_row + d * 2 + 32);
#pragma unroll
                    for (int n = 0; n < kSN; ++n) {
                        const uint2 x = lds64(k_row + 8 * n * S::kKPitch + d);
                        uint32_t kb[4];
                        e4m3x4_f16x4(x.x, kb[0], kb[1]);
                        e4m3x4_f16x4(x.y, kb[2], kb[3]);
                        mma16<true>(acc[n], qa[0], kb[0], kb[1]);
                        mma16<true>(acc[n], qa[1], kb[2], kb[3]);
                    }
                }
            } else {
                const uint32_t k_row = k_smem + ((lane & 7) + (lane >> 4) * 8) * S::kKPitch;
                const int half = (lane >> 3) & 1;
#pragma unroll
                for (int d = 0; d < DP; d += 16) {
                    uint32_t qa[4];
                    ldsm4(qa, q_row + d * 2);
#pragma unroll
                    for (int n = 0; n < kSN; n += 2) {
                        uint32_t kb[4];
                        ldsm4(kb, k_row + n * 8 * S::kKPitch +
                                      (((d / 8 + half) ^ (lane & 7)) << 4));
                        mma16<false>(acc[n], qa, kb[0], kb[1]);
                        mma16<false>(acc[n + 1], qa, kb[2], kb[3]);
                    }
                }
            }

            // scale, mask, running maximum, weights
            bool raised = false;
            float alpha[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float sc = row_scale[16 * mt + 8 * j + g];
#pragma unroll
                for (int n = 0; n < kSN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        s[n][2 * j + e] = acc[n][2 * j + e] * sc;
            }
            if (pos0 + TOK > sees_least) {  // some position is masked for some row
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int n = 0; n < kSN; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (pos0 + 8 * n + 2 * c + e >= sees[j])
                                s[n][2 * j + e] = kNegInf;
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float big = m[j];
#pragma unroll
                for (int n = 0; n < kSN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        big = fmaxf(big, s[n][2 * j + e]);
                big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
                big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
                const float ref = big == kNegInf ? 0.f : big;
                raised |= big != m[j];
                alpha[j] = ex2(m[j] - ref);
                m[j] = big;
                float sum = l[j] * alpha[j];
#pragma unroll
                for (int n = 0; n < kSN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s[n][2 * j + e];
                        x = ex2(x - ref);
                        sum += x;
                    }
                l[j] = sum;
            }
            // most chunks raise no maximum: then the output rows stay as they are
            if (__any_sync(kFull, raised)) {
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int e = 0; e < 2 * NJ; ++e)
                        o[n][e] *= alpha[e >> 1];
            }
#pragma unroll
            for (int k = 0; k < TOK / 16; ++k) {
                pa[k][0] = pack_weights<FP8>(s[2 * k][0], s[2 * k][1]);
                pa[k][1] =
                    NJ == 2 ? pack_weights<FP8>(s[2 * k][2 * NJ - 2], s[2 * k][2 * NJ - 1]) : 0u;
                pa[k][2] = pack_weights<FP8>(s[2 * k + 1][0], s[2 * k + 1][1]);
                pa[k][3] = NJ == 2 ? pack_weights<FP8>(s[2 * k + 1][2 * NJ - 2],
                                                       s[2 * k + 1][2 * NJ - 1])
                                   : 0u;
            }
        }

        // values
        cp_async_wait<2 * P - 1>();
        group_sync<kGroup>(group);
        load_values();  // into the entry of these keys
        if (finds) {    // the chunk after: its addresses are read after the next barrier
            row.resolve(a, addr + load_slot * 2 * TOK + at, TOK);
            row.fetch(a, ahead, TOK * group + at);
            ahead.next(a);
        }
        const uint32_t v_smem = ring + entry * S::kEntry;
        entry = entry + 1 == S::kEntries ? 0 : entry + 1;
        if (pos0 < cur.len) {
            // positions only some rows see: added value by value, then zeroed
            if (a.T > 1 && pos0 + TOK > sees_least) {
                const int from = max(max(sees_least, 0) - pos0, 0);
                const int to = min(cur.len - pos0, TOK);
                for (int tok = from; tok < to; ++tok) {
                    const int src = (lane & ~3) + ((tok & 7) >> 1);
                    float w[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        float pair[kSN];
#pragma unroll
                        for (int n = 0; n < kSN; ++n)
                            pair[n] = tok & 1 ? s[n][2 * j + 1] : s[n][2 * j];
                        float mine = tok & 8 ? pair[1] : pair[0];
                        if constexpr (kSN == 4)
                            mine = tok & 16 ? (tok & 8 ? pair[3] : pair[2]) : mine;
                        w[j] = __shfl_sync(kFull, FP8 ? mine * kF16Weight : mine, src);
                    }
#pragma unroll
                    for (int n = 0; n < kNT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = out_col<FP8>(n, c, e);
                            float v;
                            if constexpr (FP8)
                                v = unpack1<true>((uint16_t)e4m3x2_f16x2(
                                    lds8(v_smem + tok * S::kVPitch + d)));
                            else
                                v = unpack1<false>(lds16(v_smem + tok * S::kVPitch +
                                                         (((d / 8) ^ (tok & 7)) << 4) + (d & 7) * 2));
#pragma unroll
                            for (int j = 0; j < NJ; ++j)
                                if (pos0 + tok < sees[j])
                                    o[n][2 * j + e] = fmaf(w[j], v, o[n][2 * j + e]);
                        }
                }
                group_sync<kGroup>(group);
                for (int u = at; u < (to - from) * (S::kVPitch / 16); u += kGroup)
                    sts128(v_smem + from * S::kVPitch + u * 16, make_uint4(0, 0, 0, 0));
                group_sync<kGroup>(group);
            }
#pragma unroll
            for (int k = 0; k < TOK / 16; ++k) {
                if constexpr (FP8) {
                    // lane (g, c): tokens 2c, 2c + 1, 2c + 8, 2c + 9, columns
                    // 4 g .. 4 g + 3 of each block of 32; column tile j of a
                    // block is columns 4 n + j
                    const uint32_t v_row = v_smem + (16 * k + 2 * c) * S::kVPitch + 4 * g;
#pragma unroll
                    for (int nb = 0; nb < kNT; nb += 4) {
                        // bytes of two tokens interleaved before they are widened
                        uint32_t w[4], x[2][4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            w[q] = lds32(v_row + ((q & 1) + (q >> 1) * 8) * S::kVPitch + nb * 8);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            e4m3x4_f16x4(__byte_perm(w[2 * q], w[2 * q + 1], 0x5140), x[q][0],
                                         x[q][1]);
                            e4m3x4_f16x4(__byte_perm(w[2 * q], w[2 * q + 1], 0x7362), x[q][2],
                                         x[q][3]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_rows<true, NJ>(o[nb + j], pa[k], x[0][j], x[1][j]);
                    }
                } else {
                    const uint32_t v_row = v_smem + (16 * k + (lane & 15)) * S::kVPitch;
#pragma unroll
                    for (int n = 0; n < kNT; n += 2) {
                        uint32_t vb[4];
                        ldsm4_trans(vb, v_row + (((n + (lane >> 4)) ^ (lane & 7)) << 4));
                        mma_rows<false, NJ>(o[n], pa[k], vb[0], vb[1]);
                        mma_rows<false, NJ>(o[n + 1], pa[k], vb[2], vb[3]);
                    }
                }
            }
        }

        const bool ends = cur.t + 1 == cur.tiles;
        if (ends || left == 1) {
            // This block's part of the (sequence, head) is complete: join the
            // groups in order, through the ring entry of the values just used.
            // The next one's Q is on its way meanwhile.
            Cursor<S::kTile> after = cur;
            if (left > 1) {
                after.next(a);
                load_q(after.b, after.h);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                l[j] += __shfl_xor_sync(kFull, l[j], 1);
                l[j] += __shfl_xor_sync(kFull, l[j], 2);
                if (c == 0)
                    stat[group * S::kRows + 16 * mt + 8 * j + g] = make_float2(m[j], l[j]);
            }
            __syncthreads();
            float f[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float big = kNegInf;
#pragma unroll
                for (int w = 0; w < G; ++w)
                    big = fmaxf(big, stat[w * S::kRows + 16 * mt + 8 * j + g].x);
                f[j] = ex2(m[j] - (big == kNegInf ? 0.f : big));
            }
            const bool whole = ends && t_first == 0;
            float *part = a.parts + (2 * (int64_t)blockIdx.x + (first_part ? 0 : 1)) * a.part_floats;
            unsigned char *free_entry =
                smem + (entry == 0 ? S::kEntries - 1 : entry - 1) * S::kEntry;
#pragma unroll
            for (int c0 = 0; c0 < DP; c0 += S::kRound) {
                float *mine = reinterpret_cast<float *>(free_entry + group * S::kRing);
                // columns are permuted by the row so that a store's lanes hit
                // distinct banks
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int r = 16 * mt + 8 * j + g;
                    float *dst = mine + r * S::kRound;
#pragma unroll
                    for (int n0 = c0 / 8; n0 < (c0 + S::kRound) / 8; n0 += FP8 ? 4 : 1) {
                        if constexpr (FP8) {
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                *reinterpret_cast<float4 *>(
                                    dst + ((out_col<true>(n0, c, e) - c0) ^ swizzle<true>(r))) =
                                    make_float4(o[n0][2 * j + e] * f[j], o[n0 + 1][2 * j + e] * f[j],
                                                o[n0 + 2][2 * j + e] * f[j],
                                                o[n0 + 3][2 * j + e] * f[j]);
                        } else {
                            *reinterpret_cast<float2 *>(
                                dst + ((out_col<false>(n0, c, 0) - c0) ^ swizzle<false>(r))) =
                                make_float2(o[n0][2 * j] * f[j], o[n0][2 * j + 1] * f[j]);
                        }
                    }
                }
                __syncthreads();
                constexpr int kCols = S::kRound / 4;
                const int d = 4 * ((int)threadIdx.x % kCols);
                if (c0 + d < a.D) {
#pragma unroll 2
                    for (int r = (int)threadIdx.x / kCols; r < a.rows; r += kThreads / kCols) {
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                        float big = kNegInf, sum = 0.f;
#pragma unroll
                        for (int w = 0; w < G; ++w) {
                            const float4 x = *reinterpret_cast<const float4 *>(
                                free_entry + w * S::kRing +
                                (r * S::kRound + (d ^ swizzle<FP8>(r))) * 4);
                            acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
                            big = fmaxf(big, stat[w * S::kRows + r].x);
                        }
                        const float ref = big == kNegInf ? 0.f : big;
#pragma unroll
                        for (int w = 0; w < G; ++w)
                            sum = fmaf(stat[w * S::kRows + r].y,
                                       ex2(stat[w * S::kRows + r].x - ref), sum);
                        if (whole) {
                            put_row<FP8>(a, cur.b, cur.h, r, c0 + d, acc, big, sum);
                        } else {
                            *reinterpret_cast<float4 *>(part + r * a.D + c0 + d) = acc;
                            if (c0 + d == 0)
                                reinterpret_cast<float2 *>(part + a.rows * a.D)[r] =
                                    make_float2(big, sum);
                        }
                    }
                }
                if (c0 + S::kRound < DP)
                    __syncthreads();
            }
            if (!whole)
                finish_part<DP, FP8, kThreads, BLOCKS >= 3 ? 1 : 2>(
                    a, share, {share.u1 - left - cur.t, cur.tiles, cur.b, cur.h}, &s_last);
            if (left == 1)
                break;
            // (all scores with the old Q are done since the first barrier)
            store_q();
            start_pair(after.len);
            __syncthreads();
            first_part = false;
            t_first = after.t;
            reset();
            cur = after;
            continue;
        }
        cur.next(a);
    }
    write_empty<kThreads>(a);
}

template <int DP, bool FP8, int RT, int TOK, int P, int G, int BLOCKS>
cudaError_t config(AttnConfig *out)
{
    using S = Shape<DP, FP8, RT, TOK, P, G>;
    static_assert(BLOCKS * (S::kBytes + 1024 + 256) <= 228 * 1024, "shared memory per SM");
    out->func = reinterpret_cast<const void *>(attention_kernel<DP, FP8, RT, TOK, P, G, BLOCKS>);
    out->smem = S::kBytes;
    out->threads = S::kThreads;
    out->tile = S::kTile;
    return cudaSuccess;
}

}  // namespace attn
}  // namespace dvl
