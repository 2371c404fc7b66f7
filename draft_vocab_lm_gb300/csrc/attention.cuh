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
// softmax is left out and its accumulators are not kept.  With an NVFP4 cache
// the products are turned round: tokens are the 16 rows of the first
// (S^T = K Q^T), columns of V those of the second (O^T = V^T P^T), 8 query rows
// the columns, so no half is padding and no accumulator is moved in and out.
// The weights change places between the two by an 8 x 8 transposition of
// registers.
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
// NVFP4 cache: a byte's two E2M1 codes are widened to f16 (exact) and multiplied
// by their group's E4M3 scale as f16: the product has at most 6 significant bits
// and lies in [2^-10, 2688] (or is 0), so it is exact; Q as with FP8.  A lane
// holds 16 consecutive values of a token of K, one group, so that it needs one
// scale for them.  Not bound by HBM: 842 instructions for 32 tokens of a head of
// 128 (widening 144, scales 128, products 32, the rest finds pages, copies and
// weighs; without the multiplications by the scales 64 sequences took 158 us
// instead of 185).  61 % of the issue slots, the ALU pipe 54 % and HBM 48 % are
// busy: with 2.8 warps a scheduler the rest is waiting for a warp's own last
// result.  Measured: 64 x <= 16,381 tokens, 40 / 8 heads of 128: 180 us (692 MB,
// 0.57 of the copy rate; the same in FP8, with 1.78 times the bytes: 187-200).
//
// Masks.  Row t sees n = length - (T - 1 - t) positions.  Scores at or past
// n are replaced, not added to, so nothing a masked key holds can show; a
// row without positions keeps the sum 0 and gives 0.  Positions that only
// some rows see (the last T - 1) are added value by value for the rows that
// see them, and their V rows zeroed before the MMA: 0 times a NaN or an
// infinity in V would otherwise reach the rows that do not.  (Over an NVFP4 cache
// only those with a NaN among their scales: there is no other such value.)  Rows
// past the length are zeros from the copy.
#pragma once

#include <cuda_runtime.h>

#include "dvl_async.cuh"
#include "dvl_attention.h"
#include "dvl_device.cuh"

namespace dvl {
namespace attn {

constexpr int kBf16 = 0, kFp8 = 1, kFp4 = 2;  // what a cache holds (FMT)
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kJoin = 16;  // parts per first-level join
constexpr float kF16Weight = 32768.f;  // 2^15: a weight of 1 among f16 operands (FP8 and NVFP4 caches)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
template <int BYTES>  // 4 or 8
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? BYTES : 0), "n"(BYTES)
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
// N words (1, 2 or 4) at once.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N])
{
    if constexpr (N == 1)
        w[0] = lds32(addr);
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr)
                     : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint16_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// D += A B, m16n8k16, fp32 accumulators; FP8 and NVFP4 caches run it on f16 operands.
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

// Four of an array of accumulators.
template <int N>
__device__ __forceinline__ float (&tile(float (&x)[N], int i))[4]
{
    return *reinterpret_cast<float(*)[4]>(x + 4 * i);
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

// The two values of a byte of E2M1 codes as f16 (exact), of a word's four bytes.
__device__ __forceinline__ void e2m1x8_f16x8(uint32_t w, uint32_t (&f)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// An 8 x 8 matrix of f16, row g's values 2c and 2c + 1 with lane (g, c), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
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

template <int DP, int FMT, int RT, int TOK, int P, int G>
struct Shape {
    static constexpr int kTile = TOK * G;
    static_assert(kTile <= 128, "lengths are limited so that a tile more fits 32 bits");
    static constexpr int kGroup = RT == 0 ? 32 : 32 * RT;  // threads
    static constexpr int kThreads = kGroup * G;
    static constexpr bool kTurned = FMT == kFp4;  // S^T and O^T
    // Rows that one access phase touches lie on distinct banks.  bf16: the
    // 16-byte units of a row are permuted by its lowest three bits (8 rows of
    // an ldmatrix).  FP8: padded pitches (8-byte loads of 4 rows for K, 4-byte
    // loads of every other row for V).  NVFP4: rows without padding, in which
    // the four 32-byte pieces of every 128 bytes change places (fp4_place()).
    static constexpr int kKPitch = FMT == kFp4 ? DP / 2 : FMT == kFp8 ? DP + 32 : DP * 2;
    static constexpr int kVPitch = FMT == kFp4 ? DP / 2 : FMT == kFp8 ? DP + 16 : DP * 2;
    // Behind the rows of an NVFP4 entry: their scales.
    static constexpr int kBlocks = FMT == kFp4 ? DP / 16 : 0;  // bytes per row
    static constexpr int kQPitch = DP * 2 + 16;
    static constexpr int kRows = RT == 0 ? 8 : 16 * RT;    // query rows kept
    static constexpr int kQRows = kTurned ? kRows : RT == 0 ? 16 : 16 * RT;  // rows of the operand
    // One ring entry: a chunk's keys or values; also 32 columns of the rows.
    static constexpr int kEntry = max_of(TOK * (kKPitch + kBlocks), kRows * 4 * 32);
    static_assert(FMT != kFp4 || kEntry % 128 == 0, "fp4_place() permutes within 128 bytes");
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

// Where byte x of an NVFP4 entry's rows lies: its 32-byte piece is permuted by
// the 128-byte line, so that four rows that follow each other, and four that
// are two apart, lie on distinct banks at any width.  The permutation of a sum
// of rows is the permutations one after the other where the sum carries into
// neither's bits (rows of less than a step of 4 or 8, and steps of that), so
// that an address takes one xor with a constant: fp4_step().
__host__ __device__ constexpr int fp4_step(int x) { return (((x >> 7) ^ (x >> 9)) & 3) << 5; }
__device__ __forceinline__ int fp4_place(int x) { return x ^ fp4_step(x); }

// The output column of accumulator e (of a row) of column tile n.
template <int FMT>
__device__ __forceinline__ int out_col(int n, int c, int e)
{
    return FMT == kFp8 ? n / 4 * 32 + 4 * (2 * c + e) + n % 4 : 8 * n + 2 * c + e;
}
// The output column at place v of the joined ones.  They are the same but for
// NVFP4, where a lane holds eight columns of a block of 64 and a round joins
// four of each.
template <int FMT>
__device__ __forceinline__ int real_col(int v)
{
    return FMT == kFp4 ? (v & ~63) + ((v & 28) << 1) + ((v & 32) >> 3) + (v & 3) : v;
}

// The permutation of a row's columns while the groups' rows are joined.
template <int FMT>
__device__ __forceinline__ int swizzle(int r)
{
    return FMT == kFp4 ? (r >> 1 & 3) << 3 : FMT == kFp8 ? (r & 1) << 2 : (r & 3) << 3;
}

// Where a token's row starts, found by one thread per token a chunk before the
// copies need it: the page id is read from the table one chunk earlier still,
// so no copy waits for the table.
struct RowAddress {
    uint32_t k, v;  // byte offsets within the page
    int id;         // page id, not yet checked
    bool has;       // a cached token

    // (Straight-line code: what depends on `has` is chosen, not branched
    // around, and a bad page is reported once, at the block's end.)
    template <int TILE>
    __device__ __forceinline__ void fetch(const AttnArgs &a, const Cursor<TILE> &it, int r)
    {
        const int pos = it.t * TILE + r;
        has = it.b < a.B && pos < it.len;
        const int page = a.page_of(pos);
        id = 0;
        if (has)
            id = __ldg(a.table + it.b * a.table_stride + page);
        const uint32_t slot = pos - page * a.page_size;
        k = has ? slot * a.kt + it.h * a.kh : 0u;
        v = has ? slot * a.vt + it.h * a.vh : 0u;
    }
    // The row's addresses.  A page outside the pool is reported, and read as
    // page 0; past the length nothing is read through the address.
    __device__ __forceinline__ void resolve(const AttnArgs &a, const unsigned char **rows, int tok,
                                            bool &bad) const
    {
        const bool in = (unsigned)id < (unsigned)a.pages;
        bad |= !in;
        const int page = in ? id : 0;
        rows[0] = a.k + page * a.kp + k;
        rows[tok] = a.v + page * a.vp + v;
    }
};

// Copy a chunk's rows (keys or values) into a ring entry, `live` of them; the
// others become zeros, and so do the padding columns of keys: they meet zeros
// of Q and must hold no NaN, which whatever the entry held before may be.
// at: the thread's place among the group's N threads.
// pool, blocks: of an NVFP4 cache, the rows' pool and their scales'.
template <int DP, int FMT, int TOK, int N, bool KEYS>
__device__ __forceinline__ void load_rows(int row_bytes, const unsigned char *const *rows, int live,
                                          int at, uint32_t dst, int pitch, const unsigned char *pool,
                                          const unsigned char *blocks)
{
    if constexpr (FMT == kFp4) {
        // a row's scales, 8 bytes at a time at a width of 128, else 4 (192 has
        // 12); the padding's are zeros, too
        constexpr int kBytes = DP == 128 ? 8 : 4;
        constexpr int kUnits = DP / 16 / kBytes;
#pragma unroll
        for (int u0 = 0; u0 < TOK * kUnits; u0 += N) {
            const int u = u0 + at, r = u / kUnits, unit = u % kUnits;
            if (u < TOK * kUnits) {
                const bool have = r < live && unit * 8 * kBytes < row_bytes;
                const unsigned char *from = blocks + ((rows[r] - pool) >> 3) + unit * kBytes;
                cp_async_small<kBytes>(dst + TOK * pitch + u * kBytes, have ? from : blocks, have);
            }
        }
    }
    constexpr int kCols = DP * (FMT == kFp4 ? 1 : FMT == kFp8 ? 2 : 4) / 32;  // 16-byte units of a padded row
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
        const int unit = FMT == kBf16 ? col ^ (r & 7) : col;
        const uint32_t to = FMT == kFp4
                                ? ((dst + fp4_place(r0 * pitch + unit * 16)) ^ fp4_step(i * kStep * pitch)) +
                                      i * kStep * pitch
                                : dst + r * pitch + unit * 16;
        cp_async16(to, rows[r] + from, r < live);
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
template <int FMT>
__device__ __forceinline__ void put_row(const AttnArgs &a, int b, int h, int r, int d,
                                        const float4 &acc, float m, float sum)
{
    const int t = a.token_of(r);
    const int64_t to = ((int64_t)b * a.T + t) * a.Hq + h * a.G + (r - t * a.G);
    // a row without positions (or of -inf scores only): 0
    const float inv = sum == 0.f ? 0.f : a.v_scale / (FMT != kBf16 ? sum * kF16Weight : sum);
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
template <int DP, int FMT, int THREADS, int R>
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
                put_row<FMT>(a, b, h, r, d, acc[k], m[k], sum[k]);
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
template <int DP, int FMT, int THREADS, int R>
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
        join_parts<DP, FMT, THREADS, R>(a, parts, slot_a, slot_b, stride, stats, last_level, p.b, p.h);
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

template <int DP, int FMT, int RT, int TOK, int P, int G, int BLOCKS>
__global__ void __launch_bounds__(Shape<DP, FMT, RT, TOK, P, G>::kThreads, BLOCKS)
    attention_kernel(const __grid_constant__ AttnArgs a)
{
    using S = Shape<DP, FMT, RT, TOK, P, G>;
    constexpr int kThreads = S::kThreads;
    constexpr int kGroup = S::kGroup;
    constexpr int kWarps = kThreads / 32;
    constexpr bool F16 = FMT != kBf16;   // the operands' type, else bf16
    constexpr bool kTurned = S::kTurned;
    constexpr int NJ = RT == 0 ? 1 : 2;  // row halves kept per MMA (rows g, g + 8)
    // rows whose softmax a lane takes part in: 16 mt + 8 j + g, or turned two of
    // every column tile of 8, 16 mt + 8 (j / 2) + 2 c + j % 2
    constexpr int NQ = RT == 0 ? 1 : 2;  // column tiles
    constexpr int NS = kTurned ? 2 * NQ : NJ;
    constexpr int kNT = DP / 8;          // MMA column tiles of the output
    constexpr int kOT = kTurned ? DP / 16 : kNT;  // its tiles
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
            if constexpr (F16) {
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
                float up = __uint_as_float((uint32_t)(127 + 14 - e2) << 23);
                float down = a.qk_scale * __uint_as_float((uint32_t)(127 + e2 - 14) << 23);
                if constexpr (kTurned) {
                    // maxima are taken before the scale, which has to keep their
                    // order: Q takes its sign, and a masked score's -inf times it
                    // must not be NaN
                    if (a.qk_scale < 0.f) {
                        up = -up;
                        down = -down;
                    }
                    down = fmaxf(down, 0x1p-120f);
                }
                if (r < S::kQRows) {
                    // place of value d in the permuted order.  FP8: block of 32, lane
                    // quarter (d / 8 % 4), step (d / 4 % 2), half (d / 2 % 2).  NVFP4:
                    // block of 64, lane quarter (d / 16 % 4), step (d / 4 % 4), half
                    const int to = FMT == kFp4 ? (d & ~63) + ((d >> 3) & 1) * 32 + ((d >> 4) & 3) * 2
                                               : (d & ~31) + ((d >> 3) & 3) * 2;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint32_t *>(dst + 2 * (to + (e >> 1) * 16 + (e & 1) * 8)) =
                            pack2<true>(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
                    if (d == 0)
                        row_scale[r] = down;
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
    const int row_bytes = FMT == kFp4 ? a.D / 2 : FMT == kFp8 ? a.D : a.D * 2;
    RowAddress row;
    Cursor<S::kTile> ahead = cur;  // of the row addresses
    Cursor<S::kTile> load = cur;   // of the copies
    const bool finds = at < TOK;
    bool bad_page = false;
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
            first[i].resolve(a, addr + i * 2 * TOK + at, TOK, bad_page);
    }
    group_sync<kGroup>(group);
    int64_t to_load = n_units;
    int load_slot = 0, load_entry = 0;  // of addr, of the ring
    auto load_keys = [&]() {
        if (to_load > 0)
            load_rows<DP, FMT, TOK, kGroup, true>(row_bytes, addr + load_slot * 2 * TOK,
                                            load.len - load.t * S::kTile - TOK * group, at,
                                            ring + load_entry * S::kEntry, S::kKPitch, a.k, a.kb);
        cp_async_commit();
        load_entry = load_entry + 1 == S::kEntries ? 0 : load_entry + 1;
    };
    auto load_values = [&]() {
        if (to_load > 0)
            load_rows<DP, FMT, TOK, kGroup, false>(row_bytes, addr + load_slot * 2 * TOK + TOK,
                                            load.len - load.t * S::kTile - TOK * group, at,
                                            ring + load_entry * S::kEntry, S::kVPitch, a.v, a.vb);
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

    constexpr int kOE = kTurned ? 4 * NQ : 2 * NJ;  // accumulators kept of a tile
    float o[kOT][kOE];
    float m[NS], l[NS];
    int sees[NS], sees_least = 0;
    bool far = false;  // (NVFP4) some row's maximum is large: turned_weights()
    auto row_of = [&](int j) { return 16 * mt + (kTurned ? 8 * (j >> 1) + 2 * c + (j & 1) : 8 * j + g); };
    auto reset = [&]() {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            m[j] = kNegInf;
            l[j] = 0.f;
        }
        far = false;
#pragma unroll
        for (int n = 0; n < kOT; ++n)
#pragma unroll
            for (int e = 0; e < kOE; ++e)
                o[n][e] = 0.f;
    };
    // Visible positions per row of the (sequence, head) that starts.
    auto start_pair = [&](int len) {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int r = row_of(j);
            sees[j] = r < a.rows ? len - (a.T - 1 - a.token_of(r)) : 0;
        }
        sees_least = len - (a.T - 1);
    };
    reset();
    start_pair(cur.len);
    store_q();
    __syncthreads();
    // Value d of token tok of an NVFP4 entry.
    auto fp4_value = [&](uint32_t entry, int tok, int d) {
        const uint16_t code = lds8(entry + fp4_place(tok * S::kVPitch + d / 2)) >> 4 * (d & 1);
        uint32_t x[4];
        e2m1x8_f16x8(code & 15u, x);
        return unpack1<true>((uint16_t)mul_f16x2(
            x[0], e4m3x2_f16x2(lds8(entry + TOK * S::kVPitch + tok * S::kBlocks + d / 16))));
    };
    // The scores of a chunk's tokens with tokens as rows -- lane (g, c) holds
    // tokens g and g + 8 of every 16 for query rows 2 c and 2 c + 1 -- and their
    // weights in units of 2^-15, also as the second product's operand.  The
    // lanes of a row compare their maxima only where one is above the running
    // maximum, which after the first chunks is rare.  A weight's exponent is one
    // fma, s sc + (15 - m), of the unrounded product with roundings of m and of
    // 15 - m: up to |m| = 2^20 it exceeds 15 by less than 1/8, and f16 holds
    // 2^15.9.  From 2^23 on it would not (16.99, and at 2^28 the maximum's own
    // weight could be 2^32 or 2^-32), so larger maxima subtract from the rounded
    // product, which lies nowhere above m.
    auto turned_weights = [&](uint32_t k_smem, int pos0, auto &s, auto &pa) {
        constexpr int kTM = TOK / 16;
#pragma unroll
        for (int t = 0; t < kTM; ++t)
#pragma unroll
            for (int e = 0; e < kOE; ++e)
                s[t][e] = 0.f;
        const uint32_t q_row = base + S::kQ + (16 * mt + (lane & 7)) * S::kQPitch + (lane >> 3) * 16;
        const uint32_t k_row = k_smem + fp4_place(g * S::kKPitch) + 8 * c;
        uint32_t scales[kTM][2][DP / 64];
#pragma unroll
        for (int t = 0; t < kTM; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                lds_words(k_smem + TOK * S::kKPitch + (16 * t + 8 * h + g) * S::kBlocks, scales[t][h]);
#pragma unroll
        for (int blk = 0; blk < DP / 64; ++blk) {
            uint32_t qb[NQ][2][4];  // two steps each
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                ldsm4(qb[q][0], q_row + 8 * q * S::kQPitch + 128 * blk);
                ldsm4(qb[q][1], q_row + 8 * q * S::kQPitch + 128 * blk + 64);
            }
#pragma unroll
            for (int t = 0; t < kTM; ++t) {
                uint32_t f[2][2][4];  // token half, word, pair of codes
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int step = (16 * t + 8 * h) * S::kKPitch;
                    const uint2 x = lds64((k_row ^ (fp4_step(step) ^ blk << 5)) + step);
                    const uint32_t sc = e4m3x2_f16x2((uint16_t)__byte_perm(scales[t][h][blk], 0, c * 0x11));
                    e2m1x8_f16x8(x.x, f[h][0]);
                    e2m1x8_f16x8(x.y, f[h][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[h][0][i] = mul_f16x2(f[h][0][i], sc);
                        f[h][1][i] = mul_f16x2(f[h][1][i], sc);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int w = j / 2, i = 2 * (j & 1);
                    const uint32_t ka[4] = {f[0][w][i], f[1][w][i], f[0][w][i + 1], f[1][w][i + 1]};
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
                        mma16<true>(tile(s[t], q), ka, qb[q][w][i], qb[q][w][i + 1]);
                }
            }
        }
        // accumulator 4 q + e: token 16 t + 8 (e / 2) + g, row 2 q + e % 2 of the lane's
        if (pos0 + TOK > sees_least) {  // some position is masked for some row
#pragma unroll
            for (int t = 0; t < kTM; ++t)
#pragma unroll
                for (int e = 0; e < kOE; ++e)
                    if (pos0 + 16 * t + 8 * (e >> 1 & 1) + g >= sees[2 * (e >> 2) + (e & 1)])
                        s[t][e] = kNegInf;
        }
        float big[NS], sc[NS];
        bool raised = false;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            sc[j] = row_scale[row_of(j)];
            big[j] = kNegInf;
#pragma unroll
            for (int t = 0; t < kTM; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    big[j] = fmaxf(big[j], s[t][4 * (j >> 1) + 2 * h + (j & 1)]);
            big[j] *= sc[j];
            raised |= big[j] > m[j];
        }
        if (__any_sync(kFull, raised)) {
            float alpha[NS];
            bool large = false;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                big[j] = fmaxf(big[j], m[j]);
                big[j] = fmaxf(big[j], __shfl_xor_sync(kFull, big[j], 4));
                big[j] = fmaxf(big[j], __shfl_xor_sync(kFull, big[j], 8));
                big[j] = fmaxf(big[j], __shfl_xor_sync(kFull, big[j], 16));
                alpha[j] = ex2(m[j] - (big[j] == kNegInf ? 0.f : big[j]));
                m[j] = big[j];
                l[j] *= alpha[j];
                large |= fabsf(m[j]) >= 0x1p20f && m[j] != kNegInf;
            }
            far = __any_sync(kFull, large);
#pragma unroll
            for (int n = 0; n < kOT; ++n)
#pragma unroll
                for (int e = 0; e < kOE; ++e)
                    o[n][e] *= alpha[2 * (e >> 2) + (e & 1)];
        }
        float up[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j)
            up[j] = m[j] == kNegInf ? 0.f : 15.f - m[j];
        if (far) {
#pragma unroll
            for (int t = 0; t < kTM; ++t)
#pragma unroll
                for (int e = 0; e < kOE; ++e) {
                    const int j = 2 * (e >> 2) + (e & 1);
                    s[t][e] = __fmul_rn(s[t][e], sc[j]) - (m[j] == kNegInf ? 0.f : m[j]);
                }
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                sc[j] = 1.f;
                up[j] = 15.f;
            }
        }
#pragma unroll
        for (int t = 0; t < kTM; ++t) {
#pragma unroll
            for (int e = 0; e < kOE; ++e) {
                const int j = 2 * (e >> 2) + (e & 1);
                s[t][e] = ex2(fmaf(s[t][e], sc[j], up[j]));
                l[j] += s[t][e];
            }
#pragma unroll
            for (int i = 0; i < 2 * NQ; ++i)
                pa[t][i] = transpose8(pack2<true>(s[t][2 * i], s[t][2 * i + 1]));
        }
    };
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
        uint32_t pa[TOK / 16][kTurned ? 2 * NQ : 4];  // the weights as the second product's operand
        float s[kTurned ? TOK / 16 : kSN][kTurned ? 4 * NQ : 2 * NJ];
        if constexpr (kTurned) {
            if (pos0 < cur.len) {
                turned_weights(k_smem, pos0, s, pa);
            }
        } else if (pos0 < cur.len) {
            // scores
            float acc[kSN][4];
#pragma unroll
            for (int n = 0; n < kSN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[n][e] = 0.f;
            const uint32_t q_row =
                base + S::kQ + (16 * mt + (lane & 15)) * S::kQPitch + (lane >> 4) * 16;
            if constexpr (FMT == kFp8) {
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
                pa[k][0] = pack_weights<F16>(s[2 * k][0], s[2 * k][1]);
                pa[k][1] =
                    NJ == 2 ? pack_weights<F16>(s[2 * k][2 * NJ - 2], s[2 * k][2 * NJ - 1]) : 0u;
                pa[k][2] = pack_weights<F16>(s[2 * k + 1][0], s[2 * k + 1][1]);
                pa[k][3] = NJ == 2 ? pack_weights<F16>(s[2 * k + 1][2 * NJ - 2],
                                                       s[2 * k + 1][2 * NJ - 1])
                                   : 0u;
            }
        }

        // values
        cp_async_wait<2 * P - 1>();
        group_sync<kGroup>(group);
        load_values();  // into the entry of these keys
        if (finds) {    // the chunk after: its addresses are read after the next barrier
            row.resolve(a, addr + load_slot * 2 * TOK + at, TOK, bad_page);
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
                if constexpr (kTurned) {
                    // Only where a scale is a NaN: codes are numbers, and there are
                    // no infinities among the scales, so a weight of 0 does for the
                    // others.
                    const uint32_t scales = v_smem + TOK * S::kVPitch;
                    unsigned nans = 0u;  // tokens, from `from` on
                    for (int tok = from; tok < to; ++tok) {
                        const uint32_t x = lds32(scales + tok * S::kBlocks + lane % (S::kBlocks / 4) * 4);
                        if (!__any_sync(kFull, __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u))
                            continue;
                        nans |= 1u << (tok - from);
                        float w[NS];
#pragma unroll
                        for (int j = 0; j < NS; ++j) {
                            const int at = 4 * (j >> 1) + (j & 1);
                            float mine = tok & 8 ? s[0][at + 2] : s[0][at];
                            if constexpr (TOK == 32)
                                mine = tok & 16 ? (tok & 8 ? s[1][at + 2] : s[1][at]) : mine;
                            w[j] = __shfl_sync(kFull, mine, (tok & 7) * 4 + c);
                        }
#pragma unroll
                        for (int n = 0; n < kOT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float v =
                                    fp4_value(v_smem, tok, n / 4 * 64 + 8 * g + 2 * (n % 4) + e);
#pragma unroll
                                for (int j = 0; j < NS; ++j) {
                                    float &sum = o[n][4 * (j >> 1) + 2 * e + (j & 1)];
                                    if (pos0 + tok < sees[j])
                                        sum = fmaf(w[j], v, sum);
                                }
                            }
                    }
                    if (nans != 0u) {  // a scale of 0 makes a token's values 0
                        group_sync<kGroup>(group);
                        for (int u = at; u < (to - from) * (S::kBlocks / 4); u += kGroup)
                            if (nans >> u / (S::kBlocks / 4) & 1u)
                                sts32(scales + from * S::kBlocks + u * 4, 0u);
                        group_sync<kGroup>(group);
                    }
                } else {
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
                            w[j] = __shfl_sync(kFull, F16 ? mine * kF16Weight : mine, src);
                        }
#pragma unroll
                        for (int n = 0; n < kNT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int d = out_col<FMT>(n, c, e);
                                float v;
                                if constexpr (FMT == kFp8)
                                    v = unpack1<true>((uint16_t)e4m3x2_f16x2(
                                        lds8(v_smem + tok * S::kVPitch + d)));
                                else
                                    v = unpack1<false>(
                                        lds16(v_smem + tok * S::kVPitch +
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
            }
#pragma unroll
            for (int k = 0; k < TOK / 16; ++k) {
                if constexpr (FMT == kFp4) {
                    // lane (g, c): tokens 2c, 2c + 1, 2c + 8, 2c + 9, columns
                    // 8 g .. 8 g + 7 of each block of 64; row tile j of a block is
                    // columns 8 n + 2 j and 8 n + 2 j + 1.  The codes of two tokens
                    // are paired before they are widened, so that a byte holds both.
                    const uint32_t v_row[2] = {v_smem + fp4_place(2 * c * S::kVPitch) + 4 * g,
                                               v_smem + fp4_place((2 * c + 1) * S::kVPitch) + 4 * g};
                    uint32_t scales[2][2][DP / 64];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            lds_words(v_smem + TOK * S::kVPitch + (16 * k + 8 * q + 2 * c + t) * S::kBlocks,
                                      scales[q][t]);
#pragma unroll
                    for (int blk = 0; blk < DP / 64; ++blk) {
                        uint32_t x[2][2][4];  // pair of tokens, odd column, half the column
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int step = (16 * k + 8 * q) * S::kVPitch;
                            const uint32_t w0 = lds32((v_row[0] ^ (fp4_step(step) ^ blk << 5)) + step);
                            const uint32_t w1 = lds32((v_row[1] ^ (fp4_step(step) ^ blk << 5)) + step);
                            const uint32_t sc = e4m3x2_f16x2((uint16_t)__byte_perm(
                                scales[q][0][blk], scales[q][1][blk], (g >> 1) * 0x11 + 0x40));
                            e2m1x8_f16x8((w0 & 0x0f0f0f0fu) | (w1 & 0x0f0f0f0fu) << 4, x[q][0]);
                            e2m1x8_f16x8((w0 >> 4 & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), x[q][1]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                x[q][0][j] = mul_f16x2(x[q][0][j], sc);
                                x[q][1][j] = mul_f16x2(x[q][1][j], sc);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t va[4] = {x[0][0][j], x[0][1][j], x[1][0][j], x[1][1][j]};
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
                                mma16<true>(tile(o[4 * blk + j], q), va, pa[k][2 * q], pa[k][2 * q + 1]);
                        }
                    }
                } else if constexpr (FMT == kFp8) {
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
            for (int j = 0; j < NS; ++j) {
                if constexpr (kTurned) {
                    l[j] += __shfl_xor_sync(kFull, l[j], 4);
                    l[j] += __shfl_xor_sync(kFull, l[j], 8);
                    l[j] += __shfl_xor_sync(kFull, l[j], 16);
                    l[j] *= 1.f / kF16Weight;
                } else {
                    l[j] += __shfl_xor_sync(kFull, l[j], 1);
                    l[j] += __shfl_xor_sync(kFull, l[j], 2);
                }
                if ((kTurned ? g : c) == 0)
                    stat[group * S::kRows + row_of(j)] = make_float2(m[j], l[j]);
            }
            __syncthreads();
            float f[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                float big = kNegInf;
#pragma unroll
                for (int w = 0; w < G; ++w)
                    big = fmaxf(big, stat[w * S::kRows + row_of(j)].x);
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
                for (int j = 0; j < NS; ++j) {
                    const int r = row_of(j);
                    float *dst = mine + r * S::kRound;
                    if constexpr (kTurned) {
                        // tiles n and n + 1: four columns of 8 g .. 8 g + 7
#pragma unroll
                        for (int n = c0 / 16; n < (c0 + S::kRound) / 16; n += 2)
                            *reinterpret_cast<float4 *>(dst + ((16 * n - c0 + 4 * g) ^ swizzle<FMT>(r))) =
                                make_float4(o[n][4 * (j >> 1) + (j & 1)] * f[j],
                                            o[n][4 * (j >> 1) + 2 + (j & 1)] * f[j],
                                            o[n + 1][4 * (j >> 1) + (j & 1)] * f[j],
                                            o[n + 1][4 * (j >> 1) + 2 + (j & 1)] * f[j]);
                    } else {
#pragma unroll
                        for (int n0 = c0 / 8; n0 < (c0 + S::kRound) / 8; n0 += F16 ? 4 : 1) {
                            if constexpr (F16) {
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    *reinterpret_cast<float4 *>(
                                        dst + ((out_col<FMT>(n0, c, e) - c0) ^ swizzle<FMT>(r))) =
                                        make_float4(o[n0][2 * j + e] * f[j], o[n0 + 1][2 * j + e] * f[j],
                                                    o[n0 + 2][2 * j + e] * f[j],
                                                    o[n0 + 3][2 * j + e] * f[j]);
                            } else {
                                *reinterpret_cast<float2 *>(
                                    dst + ((out_col<FMT>(n0, c, 0) - c0) ^ swizzle<FMT>(r))) =
                                    make_float2(o[n0][2 * j] * f[j], o[n0][2 * j + 1] * f[j]);
                            }
                        }
                    }
                }
                __syncthreads();
                constexpr int kCols = S::kRound / 4;
                const int d = 4 * ((int)threadIdx.x % kCols);
                const int col = real_col<FMT>(c0 + d);
                if (col < a.D) {
#pragma unroll 2
                    for (int r = (int)threadIdx.x / kCols; r < a.rows; r += kThreads / kCols) {
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                        float big = kNegInf, sum = 0.f;
#pragma unroll
                        for (int w = 0; w < G; ++w) {
                            const float4 x = *reinterpret_cast<const float4 *>(
                                free_entry + w * S::kRing +
                                (r * S::kRound + (d ^ swizzle<FMT>(r))) * 4);
                            acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
                            big = fmaxf(big, stat[w * S::kRows + r].x);
                        }
                        const float ref = big == kNegInf ? 0.f : big;
#pragma unroll
                        for (int w = 0; w < G; ++w)
                            sum = fmaf(stat[w * S::kRows + r].y,
                                       ex2(stat[w * S::kRows + r].x - ref), sum);
                        if (whole) {
                            put_row<FMT>(a, cur.b, cur.h, r, col, acc, big, sum);
                        } else {
                            *reinterpret_cast<float4 *>(part + r * a.D + col) = acc;
                            if (col == 0)
                                reinterpret_cast<float2 *>(part + a.rows * a.D)[r] =
                                    make_float2(big, sum);
                        }
                    }
                }
                if (c0 + S::kRound < DP)
                    __syncthreads();
            }
            if (!whole)
                finish_part<DP, FMT, kThreads, BLOCKS >= 3 ? 1 : 2>(
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
    if (bad_page)
        set_status(a.ws, 1u << DVL_ERR_OUT_OF_RANGE);
    write_empty<kThreads>(a);
}

template <int DP, int FMT, int RT, int TOK, int P, int G, int BLOCKS>
cudaError_t config(AttnConfig *out)
{
    using S = Shape<DP, FMT, RT, TOK, P, G>;
    static_assert(BLOCKS * (S::kBytes + 1024 + 256) <= 228 * 1024, "shared memory per SM");
    out->func = reinterpret_cast<const void *>(attention_kernel<DP, FMT, RT, TOK, P, G, BLOCKS>);
    out->smem = S::kBytes;
    out->threads = S::kThreads;
    out->tile = S::kTile;
    return cudaSuccess;
}

}  // namespace attn
}  // namespace dvl
