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
// Work split.  The unit is a tile of 64 tokens of one (sequence, cached
// head); all units in a row (by sequence, head, tile) are cut into one equal
// share per block of a grid that is resident at once, so unequal lengths
// balance by themselves and the host needs to know none of them.  A block
// walks its share through a ring of tiles in shared memory, filled by
// 16-byte asynchronous copies that run ahead across sequence boundaries.  A
// (sequence, head) that lies in one share is finished by its block; the
// parts of one that was cut go to the workspace as (unnormalised sums,
// maximum, sum of weights), and the join kernel adds them in order of the
// shares, so the result does not depend on timing.
//
// One tile, four warps:
//   1. scores: warp w takes tokens 16 w .. 16 w + 15 against all rows;
//   2. the warps' row maxima meet in shared memory (barrier), every thread
//      keeps the running maximum of its rows and scales sums by 2^(old-new);
//   3. the weights go to shared memory in the MMA operand type (barrier): a
//      16-bit weight is the tensor cores' operand; its rounding (2^-9
//      relative for bf16, 2^-12 for f16) is random per position and averages
//      over the positions that matter, while the sums stay fp32;
//   4. values: warp w takes columns D / 4 w .. of V for all 64 tokens, so
//      the output sums of a row are spread over the block and never have to
//      be added across warps.
// Scores are kept in units of log2 (the scale carries log2 e), so a weight
// is one ex2.
//
// Operands.  bf16 cache: mma m16n8k16 bf16, K and V by ldmatrix (V
// transposed).  FP8 cache: E4M3 pairs are widened to f16 (exact) in
// registers, mma m16n8k16 f16; a query row is multiplied by a power of two
// that puts its largest value in [2^14, 2^15), which keeps every bf16 value
// down to 2^-29 of the row's largest exact in f16 (smaller ones round to the
// f16 subnormal grid, 2^-39 of the largest), and the power is taken out of
// the score's fp32 scale.  The order of the D values inside an MMA is
// permuted so that a lane's FP8 bytes are consecutive; Q is stored in the
// same order.
//
// Masks.  Row t sees n = length - (T - 1 - t) positions.  Scores at or past
// n are replaced, not added to, so nothing a masked key holds can show; a
// row without positions keeps the sum 0 and gives 0.  Positions that only
// some rows see (the last T - 1) stay out of the V tile (zeros there) and
// are added value by value for the rows that see them: 0 times a NaN or an
// infinity in V would otherwise reach the rows that do not.
#pragma once

#include <cuda_runtime.h>

#include "dvl_async.cuh"
#include "dvl_attention.h"
#include "dvl_device.cuh"

namespace dvl {
namespace attn {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kNegInf = -__builtin_huge_valf();

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

// Two E4M3 bytes -> two f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t x)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Cached tokens of sequence b, cut to what its table row can name.
__device__ __forceinline__ int seq_len(const AttnArgs &a, int b)
{
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.max_len ? a.max_len : n;
}
__device__ __forceinline__ int seq_tiles(const AttnArgs &a, int b)
{
    return (seq_len(a, b) + kTile - 1) / kTile;
}

// Walks the units from (b, h, t) on.
struct Cursor {
    int b, h, t, len, tiles;
    __device__ __forceinline__ void next(const AttnArgs &a)
    {
        if (++t < tiles)
            return;
        t = 0;
        if (++h < a.heads)
            return;
        h = 0;
        do {
            if (++b >= a.B)
                return;  // past the last unit: never loaded
            len = seq_len(a, b);
        } while (len == 0);
        tiles = (len + kTile - 1) / kTile;
    }
};

template <int DP, bool FP8, int MT, int STAGES>
struct Shape {
    static constexpr int kElem = FP8 ? 1 : 2;
    // Pitches keep the rows that one access phase touches on distinct banks:
    // ldmatrix (8 rows of 16 bytes), 8-byte loads of 4 rows, 4-byte loads of
    // every other row.
    static constexpr int kKPitch = FP8 ? DP + 32 : DP * 2 + 16;
    static constexpr int kVPitch = FP8 ? DP + 16 : DP * 2 + 16;
    static constexpr int kQPitch = DP * 2 + 16;
    static constexpr int kPPitch = kTile * 2 + 16;
    static constexpr int kRows = 16 * MT;
    static constexpr int kStage = kTile * (kKPitch + kVPitch);
    static constexpr int kQ = STAGES * kStage;
    static constexpr int kP = kQ + kRows * kQPitch;
    static constexpr int kRed = kP + kRows * kPPitch;              // float[kWarps][kRows]
    static constexpr int kSum = kRed + kWarps * kRows * 4;         // float[kWarps][kRows]
    static constexpr int kScale = kSum + kWarps * kRows * 4;       // float[kRows]
    static constexpr int kBytes = kScale + kRows * 4;
};

// Copy tile `it` into a ring stage.
template <int DP, bool FP8>
__device__ __forceinline__ void load_tile(const AttnArgs &a, const Cursor &it, uint32_t k_smem,
                                          uint32_t v_smem, int k_pitch, int v_pitch)
{
    constexpr int kElem = FP8 ? 1 : 2;
    constexpr int kCols = DP * kElem / 16;       // 16-byte units of a padded row
    constexpr int kStep = kThreads / kCols;      // rows per pass
    const int col = threadIdx.x % kCols;
    if (col * 16 >= a.D * kElem)
        return;
    const int32_t *table = a.table + it.b * a.table_stride;
    const int whole = it.len - (a.T - 1);        // positions every row sees
#pragma unroll
    for (int i = 0; i < kTile / kStep; ++i) {
        const int r = (int)threadIdx.x / kCols + i * kStep;
        const int pos = it.t * kTile + r;
        bool valid = pos < it.len;
        const int page = valid ? a.page_of(pos) : 0;
        const int id = valid ? __ldg(table + page) : 0;
        if ((unsigned)id >= (unsigned)a.pages) {
            valid = false;
            set_status(a.ws, 1u << DVL_ERR_OUT_OF_RANGE);
        }
        const int64_t slot = pos - (int64_t)page * a.page_size;
        const unsigned char *k = a.k, *v = a.v;
        if (valid) {
            k += id * a.kp + slot * a.kt + it.h * a.kh + col * 16;
            v += id * a.vp + slot * a.vt + it.h * a.vh + col * 16;
        }
        cp_async16(k_smem + r * k_pitch + col * 16, k, valid);
        cp_async16(v_smem + r * v_pitch + col * 16, v, valid && pos < whole);
    }
}

// One cached value of V at (position, column), for the positions only some
// rows see.
template <bool FP8>
__device__ __forceinline__ float value_at(const AttnArgs &a, int b, int h, int pos, int d)
{
    const int page = a.page_of(pos);
    const int id = a.table[b * a.table_stride + page];
    if ((unsigned)id >= (unsigned)a.pages)
        return 0.f;
    const unsigned char *p =
        a.v + id * a.vp + (pos - (int64_t)page * a.page_size) * a.vt + h * a.vh;
    if constexpr (FP8)
        return unpack1<true>((uint16_t)(e4m3x2_f16x2(p[d]) & 0xffffu));
    else
        return unpack1<false>(reinterpret_cast<const uint16_t *>(p)[d]);
}

// The block's first unit: the sequence that holds unit u0 and u0's place in
// it, and the number of units in all.  Every thread calls it.
__device__ __forceinline__ int64_t locate(const AttnArgs &a, int *s_b, int64_t *s_off,
                                          int64_t *s_warp, int64_t *u0, int64_t *u1)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t total = 0;
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
        if (a.lengths[b] > a.max_len)
            set_status(a.ws, 1u << DVL_ERR_OUT_OF_RANGE);
        total += seq_tiles(a, b);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        total += __shfl_xor_sync(kFull, total, off);
    if (lane == 0)
        s_warp[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        total += s_warp[w];
    const int64_t units = total * a.heads;
    const int64_t blocks = used_blocks(a.blocks, units);
    *u0 = blockIdx.x * units / (blocks > 0 ? blocks : 1);
    *u1 = blockIdx.x < blocks ? (blockIdx.x + 1ll) * units / blocks : *u0;
    int64_t carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const int64_t mine = b < a.B ? seq_tiles(a, b) : 0;
        int64_t scan = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(kFull, scan, off);
            if (lane >= off)
                scan += o;
        }
        __syncthreads();
        if (lane == 31)
            s_warp[warp] = scan;
        __syncthreads();
        for (int w = 0; w < warp; ++w)
            scan += s_warp[w];
        const int64_t end = (carry + scan) * a.heads, begin = end - mine * a.heads;
        if (begin <= *u0 && *u0 < end) {
            *s_b = b;
            *s_off = *u0 - begin;
        }
        for (int w = 0; w < kWarps; ++w)
            carry += s_warp[w];
    }
    __syncthreads();
    return units;
}

template <int DP, bool FP8, int MT, int STAGES>
__global__ void __launch_bounds__(kThreads) attention_kernel(const __grid_constant__ AttnArgs a)
{
    using S = Shape<DP, FP8, MT, STAGES>;
    constexpr int kCols = DP / 4;        // output columns per warp
    constexpr int kNT = kCols / 8;       // MMA column tiles per warp
    constexpr int kJ = kNT < 4 ? kNT : 4;  // FP8: column tiles that share a V load
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_b;
    __shared__ int64_t s_off, s_warp[kWarps];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const uint32_t base = smem_u32(smem);
    float *red = reinterpret_cast<float *>(smem + S::kRed);
    float *sums = reinterpret_cast<float *>(smem + S::kSum);
    float *row_scale = reinterpret_cast<float *>(smem + S::kScale);

    int64_t u0, u1;
    locate(a, &s_b, &s_off, s_warp, &u0, &u1);
    if (u0 >= u1)
        return;
    Cursor cur;
    cur.b = s_b;
    cur.len = seq_len(a, cur.b);
    cur.tiles = (cur.len + kTile - 1) / kTile;
    cur.h = (int)(s_off / cur.tiles);
    cur.t = (int)(s_off - (int64_t)cur.h * cur.tiles);
    const int64_t n_units = u1 - u0;

    // Padding columns of K meet zeros of Q: they must hold no NaN.
    if (a.D < DP)
        for (int i = threadIdx.x * 16; i < S::kQ; i += kThreads * 16)
            *reinterpret_cast<uint4 *>(smem + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();

    Cursor ahead = cur;
    int64_t loaded = 0;
    auto load_next = [&]() {
        if (loaded < n_units) {
            const uint32_t st = base + (uint32_t)(loaded % STAGES) * S::kStage;
            load_tile<DP, FP8>(a, ahead, st, st + kTile * S::kKPitch, S::kKPitch, S::kVPitch);
            ahead.next(a);
        }
        ++loaded;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        load_next();

    float o[MT][kNT][4];
    float m[MT][2], l[MT][2];
    int sees[MT][2];
    bool fresh = true;       // the next tile starts a (sequence, head)
    bool first_part = true;  // still in the block's first (sequence, head)
    int t_first = 0;
    for (int64_t i = 0; i < n_units; ++i) {
        if (fresh) {
            fresh = false;
            t_first = cur.t;
            // Q of this (sequence, cached head): row t * G + g
            for (int r = warp; r < S::kRows; r += kWarps) {
                const int t = r / a.G;
                const uint16_t *q = a.q + cur.b * a.qb + t * a.qt +
                                    (int64_t)(cur.h * a.G + (r - t * a.G)) * a.qh;
                unsigned char *dst = smem + S::kQ + r * S::kQPitch;
                if constexpr (FP8) {
                    constexpr int kPer = DP / 32 < 2 ? 2 : DP / 32;  // values per lane
                    float v[kPer];
                    uint32_t big = 0u;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const int d = lane + 32 * e;
                        v[e] = r < a.rows && d < a.D ? __uint_as_float((uint32_t)q[d] << 16) : 0.f;
                        big = max(big, __float_as_uint(v[e]) & 0x7fffffffu);
                    }
                    big = __reduce_max_sync(kFull, big);
                    int e2 = (int)(big >> 23) - 127;
                    e2 = e2 < -100 ? -100 : e2 > 127 ? 127 : e2;
                    const float up = __uint_as_float((uint32_t)(127 + 14 - e2) << 23);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const int d = lane + 32 * e;
                        if (d < DP) {
                            // place of d in the permuted order: block of 32,
                            // lane quarter (d / 8 % 4), step (d / 4 % 2),
                            // half (d / 2 % 2)
                            const int p = (d & ~31) + ((d >> 2) & 1) * 16 + ((d >> 1) & 1) * 8 +
                                          ((d >> 3) & 3) * 2 + (d & 1);
                            reinterpret_cast<uint16_t *>(dst)[p] =
                                (uint16_t)(pack2<true>(v[e] * up, 0.f) & 0xffffu);
                        }
                    }
                    if (lane == 0)
                        row_scale[r] = a.qk_scale * __uint_as_float((uint32_t)(127 + e2 - 14) << 23);
                } else {
                    for (int d = 2 * lane; d < DP; d += 64)
                        *reinterpret_cast<uint32_t *>(dst + 2 * d) =
                            r < a.rows && d < a.D ? *reinterpret_cast<const uint32_t *>(q + d) : 0u;
                    if (lane == 0)
                        row_scale[r] = a.qk_scale;
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 16 * mt + 8 * j + g;
                    sees[mt][j] = r < a.rows ? cur.len - (a.T - 1 - r / a.G) : 0;
                    m[mt][j] = kNegInf;
                    l[mt][j] = 0.f;
                }
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[mt][n][e] = 0.f;
            }
        }
        cp_async_wait<STAGES - 2>();
        __syncthreads();
        load_next();  // into the stage the previous tile used

        const uint32_t k_smem = base + (uint32_t)(i % STAGES) * S::kStage;
        const uint32_t v_smem = k_smem + kTile * S::kKPitch;
        const int pos0 = cur.t * kTile;

        // 1. scores of this warp's 16 tokens
        float s[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[mt][n][e] = 0.f;
        const uint32_t q_row = base + S::kQ + (lane & 15) * S::kQPitch + (lane >> 4) * 16;
        if constexpr (FP8) {
            const uint32_t k_row = k_smem + (16 * warp + g) * S::kKPitch + 8 * c;
#pragma unroll
            for (int d = 0; d < DP; d += 32) {
                uint32_t kb[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint2 x = lds64(k_row + 8 * n * S::kKPitch + d);
                    kb[n][0] = e4m3x2_f16x2((uint16_t)x.x);
                    kb[n][1] = e4m3x2_f16x2((uint16_t)(x.x >> 16));
                    kb[n][2] = e4m3x2_f16x2((uint16_t)x.y);
                    kb[n][3] = e4m3x2_f16x2((uint16_t)(x.y >> 16));
                }
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t qa[4];
                        ldsm4(qa, q_row + 16 * mt * S::kQPitch + (d + 16 * st) * 2);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            mma16<true>(s[mt][n], qa, kb[n][2 * st], kb[n][2 * st + 1]);
                    }
            }
        } else {
            const uint32_t k_row = k_smem +
                                   (16 * warp + (lane & 7) + (lane >> 4) * 8) * S::kKPitch +
                                   ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int d = 0; d < DP; d += 16) {
                uint32_t kb[4];
                ldsm4(kb, k_row + d * 2);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t qa[4];
                    ldsm4(qa, q_row + 16 * mt * S::kQPitch + d * 2);
                    mma16<false>(s[mt][0], qa, kb[0], kb[1]);
                    mma16<false>(s[mt][1], qa, kb[2], kb[3]);
                }
            }
        }

        // 2. scale, mask, row maxima
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 16 * mt + 8 * j + g;
                const float sc = row_scale[r];
                float big = kNegInf;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int pos = pos0 + 16 * warp + 8 * n + 2 * c + e;
                        float &x = s[mt][n][2 * j + e];
                        x = pos < sees[mt][j] ? x * sc : kNegInf;
                        big = fmaxf(big, x);
                    }
                big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
                big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
                if (c == 0)
                    red[warp * S::kRows + r] = big;
            }
        __syncthreads();

        // 3. weights
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 16 * mt + 8 * j + g;
                float big = m[mt][j];
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    big = fmaxf(big, red[w * S::kRows + r]);
                const float ref = big == kNegInf ? 0.f : big;
                const float alpha = ex2(m[mt][j] - ref);
                m[mt][j] = big;
                float sum = l[mt][j] * alpha;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2(s[mt][n][2 * j] - ref);
                    const float p1 = ex2(s[mt][n][2 * j + 1] - ref);
                    sum += p0 + p1;
                    *reinterpret_cast<uint32_t *>(smem + S::kP + r * S::kPPitch +
                                                  (16 * warp + 8 * n + 2 * c) * 2) =
                        pack2<FP8>(p0, p1);
                }
                l[mt][j] = sum;
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    o[mt][n][2 * j] *= alpha;
                    o[mt][n][2 * j + 1] *= alpha;
                }
            }
        __syncthreads();

        // 4. values
        const uint32_t p_row = base + S::kP + (lane & 15) * S::kPPitch + (lane >> 4) * 16;
#pragma unroll
        for (int kk = 0; kk < kTile; kk += 16) {
            uint32_t pa[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                ldsm4(pa[mt], p_row + 16 * mt * S::kPPitch + kk * 2);
            if constexpr (FP8) {
                // lane (g, c): tokens 2c, 2c + 1, 2c + 8, 2c + 9, columns
                // kJ g .. kJ g + kJ - 1 of each 8 kJ-wide block; column tile j
                // of the block is columns kJ n + j
                const uint32_t v_row = v_smem + (kk + 2 * c) * S::kVPitch + warp * kCols + kJ * g;
#pragma unroll
                for (int nb = 0; nb < kNT; nb += kJ) {
                    uint32_t x[4][kJ / 2];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t at =
                            v_row + ((q & 1) + (q >> 1) * 8) * S::kVPitch + nb * 8;
                        if constexpr (kJ == 4) {
                            const uint32_t w = lds32(at);
                            x[q][0] = e4m3x2_f16x2((uint16_t)w);
                            x[q][1] = e4m3x2_f16x2((uint16_t)(w >> 16));
                        } else {
                            x[q][0] = e4m3x2_f16x2(lds16(at));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
                        const uint32_t b0 = __byte_perm(x[0][j / 2], x[1][j / 2], sel);
                        const uint32_t b1 = __byte_perm(x[2][j / 2], x[3][j / 2], sel);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            mma16<true>(o[mt][nb + j], pa[mt], b0, b1);
                    }
                }
            } else {
                const uint32_t v_row = v_smem +
                                       (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * S::kVPitch +
                                       (warp * kCols + (lane >> 4) * 8) * 2;
#pragma unroll
                for (int n = 0; n < kNT; n += 2) {
                    uint32_t vb[4];
                    ldsm4_trans(vb, v_row + n * 16);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16<false>(o[mt][n], pa[mt], vb[0], vb[1]);
                        mma16<false>(o[mt][n + 1], pa[mt], vb[2], vb[3]);
                    }
                }
            }
        }
        // the column of o[.][n][e] is col(n, e) (+ 2 j rows)
        auto col = [&](int n, int e) {
            if constexpr (FP8)
                return warp * kCols + n / kJ * kJ * 8 + kJ * (2 * c + e) + n % kJ;
            else
                return warp * kCols + 8 * n + 2 * c + e;
        };
        // positions only some rows see
        if (a.T > 1 && pos0 + kTile > cur.len - (a.T - 1)) {
            const int from = max(pos0, max(cur.len - (a.T - 1), 0));
            const int to = min(pos0 + kTile, cur.len);
            for (int pos = from; pos < to; ++pos)
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = col(n, e);
                        if (d >= a.D)
                            continue;
                        const float v = value_at<FP8>(a, cur.b, cur.h, pos, d);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (pos < sees[mt][j]) {
                                    const float p = unpack1<FP8>(*reinterpret_cast<const uint16_t *>(
                                        smem + S::kP + (16 * mt + 8 * j + g) * S::kPPitch +
                                        (pos - pos0) * 2));
                                    o[mt][n][2 * j + e] = fmaf(p, v, o[mt][n][2 * j + e]);
                                }
                    }
        }

        const bool ends = cur.t + 1 == cur.tiles;
        if (ends || i + 1 == n_units) {
            // this block's part of the (sequence, head) is complete
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = l[mt][j];
                    x += __shfl_xor_sync(kFull, x, 1);
                    x += __shfl_xor_sync(kFull, x, 2);
                    if (c == 0)
                        sums[warp * S::kRows + 16 * mt + 8 * j + g] = x;
                }
            __syncthreads();
            const bool whole = ends && t_first == 0;
            float *part = a.parts + (2 * (int64_t)blockIdx.x + (first_part ? 0 : 1)) * a.part_floats;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 16 * mt + 8 * j + g;
                    if (r >= a.rows)
                        continue;
                    float x = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        x += sums[w * S::kRows + r];
                    if (whole) {
                        const int t = r / a.G;
                        const int64_t at = ((int64_t)cur.b * a.T + t) * a.Hq + cur.h * a.G +
                                           (r - t * a.G);
                        // a row without positions (or of -inf scores only): 0
                        const float f = x == 0.f ? 0.f : a.v_scale / x;
#pragma unroll
                        for (int n = 0; n < kNT; ++n) {
                            if constexpr (FP8) {
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (col(n, e) < a.D)
                                        a.out[at * a.D + col(n, e)] =
                                            (uint16_t)(pack2<false>(o[mt][n][2 * j + e] * f, 0.f));
                            } else if (col(n, 0) < a.D) {
                                *reinterpret_cast<uint32_t *>(a.out + at * a.D + col(n, 0)) =
                                    pack2<false>(o[mt][n][2 * j] * f, o[mt][n][2 * j + 1] * f);
                            }
                        }
                        if (a.lse && warp == 0 && c == 0)
                            a.lse[at] = log_sum(m[mt][j], x);
                    } else {
#pragma unroll
                        for (int n = 0; n < kNT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (col(n, e) < a.D)
                                    part[r * a.D + col(n, e)] = o[mt][n][2 * j + e];
                        if (warp == 0 && c == 0) {
                            part[a.rows * a.D + 2 * r] = m[mt][j];
                            part[a.rows * a.D + 2 * r + 1] = x;
                        }
                    }
                }
            first_part = false;
            fresh = true;
        }
        cur.next(a);
    }
}

// STAGES tiles in the ring, or one fewer where they and Q exceed a block's
// shared memory (227 KB less the static part).
template <int DP, bool FP8, int MT, int STAGES>
cudaError_t config(AttnConfig *out)
{
    constexpr int kFit = Shape<DP, FP8, MT, STAGES>::kBytes <= 227 * 1024 - 128 ? STAGES : STAGES - 1;
    static_assert(kFit >= 2, "the ring needs two stages");
    out->func = reinterpret_cast<const void *>(attention_kernel<DP, FP8, MT, kFit>);
    out->smem = Shape<DP, FP8, MT, kFit>::kBytes;
    return cudaSuccess;
}

template <int DP, bool FP8, int STAGES>
cudaError_t config_rows(int rows, AttnConfig *out)
{
    if (rows <= 16)
        return config<DP, FP8, 1, STAGES>(out);
    if (rows <= 32)
        return config<DP, FP8, 2, STAGES>(out);
    return config<DP, FP8, 4, STAGES>(out);
}

}  // namespace attn
}  // namespace dvl
