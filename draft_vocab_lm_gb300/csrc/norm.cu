// Residual addition, root-mean-square norm, and the 8-bit codes of the
// result, in one pass over a row:
//   u = x + residual,  y = u w / sqrt(mean(u^2) + eps),
//   per group: a = max |y|, scale = a / 448, code = RNE_e4m3(y (448 / a)).
//
// Bound by HBM (6 flops per element against 5 to 13 bytes).  A team takes one
// row: a warp for short rows (eight per block: a block per row of 80 took 10.6
// us for 9,999 rows, a warp 3), else a block of up to 1,024
// threads.  A thread owns 8 values per step (one 16-byte load of a bf16
// tensor), keeps u in registers between the sum and the output, and reads
// every input once.  Many small teams hide each other's latencies; a loop over
// rows with the next row's inputs in flight cost the registers of the teams it
// replaced (20,011 rows of 2,560, fp32 residual: 86.5 to 92 us against 87 then;
// 80 now).
//   - The sum of squares: per thread, butterfly per warp, then every warp
//     adds the warps' partial sums itself (one block barrier).  fp32
//     throughout.
//   - The group maximum stays within a warp, which owns 256 consecutive
//     values; one scale per row takes a second barrier.  Maxima compare the
//     bit patterns of |y| as unsigned integers: the order is that of the
//     values, with NaN above infinity, so a NaN reaches the scale instead of
//     being dropped.
//   - Divisions are few, for the issue slots bound what HBM does not (67 % of
//     them in use, at 0.64 of the copy rate, with IEEE divisions): the
//     reciprocal root is the hardware's approximation (2^-22 relative), 448 / a
//     is 448 times one rounded reciprocal per thread and group, so it is rounded
//     twice (up to 2^-23 relative): a value within that of the middle between
//     two codes can take either.
//   - The codes are cut from the fp32 y, not from its bf16 rounding.
// Rows that 16-byte accesses do not fit (K % 8 != 0, an odd stride, a pointer
// off a 16-byte boundary) run the same kernel with element accesses, a lane
// taking every 32nd value of its warp's 256 so that a warp reads one run of
// bytes (8 consecutive values per lane: 111 us for 12,001 rows of 2,001, bf16 in
// and out; every 32nd 58; without a bounds test per access where the warp's 256
// values lie inside the row 43, 0.67 of the copy rate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kVals = 8;          // values per thread and step
constexpr int kRowsPerBlock = 8;  // where a warp takes a row

struct None {};  // no residual

struct NormArgs {
    dvl_norm a;
    int groups;   // per row
    float inv_k;  // 1 / K
    int group_shift;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two E4M3 codes (lo in the low byte), nearest even, saturating at 448.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The 8 values of a thread.  WIDE: values 8 lane .. of the warp's 256, else
// lane, lane + 32, ..; p points at the warp's first, n values of the row are
// left from there.
template <bool WIDE>
__device__ __forceinline__ int place(int lane, int i)
{
    return WIDE ? kVals * lane + i : 32 * i + lane;
}

// op(i) for the thread's values inside the row; most warps hold no others.
template <typename Op>
__device__ __forceinline__ void for_values(int lane, int n, Op op)
{
    if (n >= 32 * kVals) {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            op(i);
    } else {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            if (32 * i + lane < n)
                op(i);
    }
}

// Inputs as they are stored, so that those in flight take few registers.
template <typename T, bool WIDE>
struct Raw;
template <>
struct Raw<uint16_t, true> {
    uint4 q;
    __device__ __forceinline__ void load(const uint16_t *p, int lane, int)
    {
        q = *reinterpret_cast<const uint4 *>(p + kVals * lane);
    }
    __device__ __forceinline__ void get(float (&v)[kVals]) const
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <>
struct Raw<float, true> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p, int lane, int)
    {
        a = reinterpret_cast<const float4 *>(p + kVals * lane)[0];
        b = reinterpret_cast<const float4 *>(p + kVals * lane)[1];
    }
    __device__ __forceinline__ void get(float (&v)[kVals]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <>
struct Raw<uint16_t, false> {
    uint16_t e[kVals];
    __device__ __forceinline__ void load(const uint16_t *p, int lane, int n)
    {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            e[i] = 0;
        for_values(lane, n, [&](int i) { e[i] = p[32 * i + lane]; });
    }
    __device__ __forceinline__ void get(float (&v)[kVals]) const
    {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            v[i] = __uint_as_float((uint32_t)e[i] << 16);
    }
};
template <>
struct Raw<float, false> {
    float e[kVals];
    __device__ __forceinline__ void load(const float *p, int lane, int n)
    {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            e[i] = 0.f;
        for_values(lane, n, [&](int i) { e[i] = p[32 * i + lane]; });
    }
    __device__ __forceinline__ void get(float (&v)[kVals]) const
    {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            v[i] = e[i];
    }
};

template <bool WIDE>
__device__ __forceinline__ void store8(uint16_t *p, int lane, int n, const float (&v)[kVals])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if constexpr (WIDE) {
        *reinterpret_cast<uint4 *>(p + kVals * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        for_values(lane, n, [&](int i) {
            p[32 * i + lane] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        });
    }
}

template <bool WIDE>
__device__ __forceinline__ void store8(float *p, int lane, int n, const float (&v)[kVals])
{
    if constexpr (WIDE) {
        reinterpret_cast<float4 *>(p + kVals * lane)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p + kVals * lane)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        for_values(lane, n, [&](int i) { p[32 * i + lane] = v[i]; });
    }
}

template <bool WIDE>
__device__ __forceinline__ void store8_codes(uint8_t *p, int lane, int n, const float (&v)[kVals])
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = pack_e4m3(v[4 * i], v[4 * i + 1]) | pack_e4m3(v[4 * i + 2], v[4 * i + 3]) << 16;
    if constexpr (WIDE) {
        *reinterpret_cast<uint2 *>(p + kVals * lane) = make_uint2(w[0], w[1]);
    } else {
        for_values(lane, n, [&](int i) {
            p[32 * i + lane] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
        });
    }
}

// The larger of |y| and m, NaN above all.
__device__ __forceinline__ float max_abs(float m, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(y)));
    return r;
}
// (of numbers without a sign, which order like their bits)
__device__ __forceinline__ float warp_max(float m)
{
    return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)));
}

// The multiplier 448 / a of a group whose largest |y| is a, and its scale
// a / 448.  Below 2^-119 the multiplier is no fp32 number: codes 0.
__device__ __forceinline__ float code_factor(float a, float *scale)
{
    *scale = a * (1.f / 448.f);
    return a < 0x1p-119f ? 0.f : 448.f * __frcp_rn(a);
}

// Scale a warp's 256 values (8 per thread) by their groups' factors and write
// the groups' scales; n values of the row are left; group is 2^shift.
template <bool WIDE>
__device__ __forceinline__ void scale_groups(float (&y)[kVals], int group, int shift, int lane, int n,
                                             float *scales)
{
    float scale;
    if constexpr (WIDE) {  // a group is group / 8 consecutive lanes
        float amax = 0.f;
        if (kVals * lane < n)
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                amax = max_abs(amax, y[i]);
        if (group == 256)
            amax = warp_max(amax);
        else
            for (int off = group / (2 * kVals); off >= 1; off >>= 1)
                amax = max_abs(amax, __shfl_xor_sync(kFull, amax, off));
        const float f = code_factor(amax, &scale);
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            y[i] *= f;
        if ((kVals * lane & (group - 1)) == 0 && kVals * lane < n)
            scales[kVals * lane >> shift] = scale;
    } else {  // a group is group / 32 values of every lane, or half the lanes' one
        float amax[kVals];
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            amax[i] = 0.f;
        for_values(lane, n, [&](int i) { amax[i] = max_abs(0.f, y[i]); });
        if (group == 16) {
#pragma unroll
            for (int i = 0; i < kVals; ++i)
#pragma unroll
                for (int off = 8; off >= 1; off >>= 1)
                    amax[i] = max_abs(amax[i], __shfl_xor_sync(kFull, amax[i], off));
        } else {
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                amax[i] = warp_max(amax[i]);
            for (int span = 1; 32 * span < group; span *= 2)
#pragma unroll
                for (int i = 0; i < kVals; ++i) {
                    // value i's partner group: constant indexes after unrolling
                    if (span == 1 && !(i & 1))
                        amax[i] = amax[i + 1] = max_abs(amax[i], amax[i + 1]);
                    if (span == 2 && !(i & 3))
                        amax[i] = amax[i + 1] = amax[i + 2] = amax[i + 3] =
                            max_abs(amax[i], amax[i + 2]);
                    if (span == 4 && i == 0) {
                        const float all = max_abs(amax[0], amax[4]);
#pragma unroll
                        for (int j = 0; j < kVals; ++j)
                            amax[j] = all;
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            y[i] *= code_factor(amax[i], &scale);
            const int k = 32 * i + lane;
            if ((k & (group - 1)) == 0 && k < n)
                scales[k >> shift] = scale;
        }
    }
}

// R: the residual's storage (uint16_t: bf16), or None.  NC: 256-value steps per warp of
// the team.  TEAM: whether a block is one team (else each of its warps is).
template <typename R, bool WIDE, int NC, bool TEAM>
__global__ void __launch_bounds__(TEAM ? kMaxThreads : 32 * kRowsPerBlock)
    add_rmsnorm_kernel(const NormArgs p)
{
    __shared__ float part[32], part_max[32];
    pdl_launch_dependents();
    pdl_wait();
    const dvl_norm &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int K = a.K;
    const int64_t row = TEAM ? blockIdx.x : (int64_t)blockIdx.x * kRowsPerBlock + warp;
    if (row >= a.rows)  // (a whole warp of a block without barriers)
        return;
    // the warp's values of step c: first .. first + 255
    auto first = [&](int c) { return 256 * (TEAM ? c * warps + warp : c); };
    // whether the thread has values there
    auto live = [&](int c) { return first(c) + place<WIDE>(lane, 0) < K; };

    const uint16_t *px = static_cast<const uint16_t *>(a.x) + row * a.x_stride;
    Raw<uint16_t, WIDE> x[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (live(c))
            x[c].load(px + first(c), lane, K - first(c));
    const uint16_t *pw = static_cast<const uint16_t *>(a.weight);
    // Weights are loaded with the row where that takes few registers (1 row of
    // 2,560: 1.6 us without, 1.5 with; element accesses, 12,001 rows of 2,001:
    // 39.5 and 43).
    Raw<uint16_t, WIDE> w[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (WIDE && live(c))
            w[c].load(pw + first(c), lane, K - first(c));
    float u[NC][kVals];
    float ss = 0.f;
    if constexpr (!std::is_same_v<R, None>) {
        const R *pr = static_cast<const R *>(a.residual) + row * a.residual_stride;
        R *to = static_cast<R *>(a.residual_out) + row * a.residual_out_stride;
        Raw<R, WIDE> r[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (live(c))
                r[c].load(pr + first(c), lane, K - first(c));
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (live(c)) {
                float v[kVals];
                x[c].get(u[c]);
                r[c].get(v);
#pragma unroll
                for (int i = 0; i < kVals; ++i)
                    u[c][i] += v[i];
                store8<WIDE>(to + first(c), lane, K - first(c), u[c]);
            }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (live(c))
                x[c].get(u[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (live(c))
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                ss = fmaf(u[c][i], u[c][i], ss);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        ss += __shfl_xor_sync(kFull, ss, off);
    if constexpr (TEAM) {
        if (lane == 0)
            part[warp] = ss;
        __syncthreads();
        ss = lane < warps ? part[lane] : 0.f;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            ss += __shfl_xor_sync(kFull, ss, off);
    }
    const float inv = rsqrtf(fmaf(ss, p.inv_k, a.eps));

    float row_max = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (live(c)) {
            float wv[kVals];
            if (!WIDE)
                w[c].load(pw + first(c), lane, K - first(c));
            w[c].get(wv);
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                u[c][i] = u[c][i] * inv * wv[i];
            if (a.out)
                store8<WIDE>(static_cast<uint16_t *>(a.out) + row * a.out_stride + first(c), lane,
                             K - first(c), u[c]);
        }
        if (!a.codes)
            continue;
        if (a.group == 0) {
            if (live(c))
#pragma unroll
                for (int i = 0; i < kVals; ++i)
                    row_max = max_abs(row_max, u[c][i]);
            continue;
        }
        if (first(c) >= K)
            continue;
        scale_groups<WIDE>(u[c], a.group, p.group_shift, lane, K - first(c),
                           a.scales + row * p.groups + (first(c) >> p.group_shift));
        if (live(c))
            store8_codes<WIDE>(a.codes + row * a.codes_stride + first(c), lane, K - first(c), u[c]);
    }
    if (!a.codes || a.group != 0)
        return;
    row_max = warp_max(row_max);
    if constexpr (TEAM) {
        if (lane == 0)
            part_max[warp] = row_max;
        __syncthreads();
        row_max = warp_max(lane < warps ? part_max[lane] : 0.f);
    }
    float scale;
    const float f = code_factor(row_max, &scale);
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (live(c)) {
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                u[c][i] *= f;
            store8_codes<WIDE>(a.codes + row * a.codes_stride + first(c), lane, K - first(c), u[c]);
        }
    if (TEAM ? threadIdx.x == 0 : lane == 0)
        a.scales[row] = scale;
}

template <typename R, bool WIDE>
cudaError_t launch(const NormArgs &p, cudaStream_t s)
{
    const int steps = (p.a.K + 255) / 256;  // of 256 values
    // A warp takes a row of up to 256 values, and one of up to 512 when the
    // rows are many: 7,737 rows of 504 4.7 us, a block each 8.2; 99 rows 1.8
    // and 1.6.  With element accesses a warp issues eight times as many, and
    // the turn comes later: 999 rows of 511 4.3 and 3.2, 7,737 of 331 7.0 and
    // 8.7.  (A warp per row of 1,001 values: 43.7 us for 7,737 rows, 10.1 for
    // 99; a block each 19.5 and 3.0.)
    if (steps == 1 || (steps == 2 && p.a.rows >= (WIDE ? 768 : 4096))) {
        const unsigned grid = (unsigned)((p.a.rows + kRowsPerBlock - 1) / kRowsPerBlock);
        const int threads = 32 * kRowsPerBlock;
        if (steps == 1)
            return launch_pdl(add_rmsnorm_kernel<R, WIDE, 1, false>, grid, threads, 0, s, p);
        return launch_pdl(add_rmsnorm_kernel<R, WIDE, 2, false>, grid, threads, 0, s, p);
    }
    // Many rows without a residual: two steps per thread, for more bytes in
    // flight per SM (19,317 rows of 2,560 -> codes: 43.7 and 38.9 us; 12,001 of
    // 2,001: 29.8 and 24.2; 1,893 of 1,376: 3.6 and 3.8).  With one, its loads
    // do as much (20,011 of 2,560, fp32: 80.1 and 80.3).
    const bool two = std::is_same_v<R, None> && p.a.rows >= 4096;
    const int nc = steps <= 32 ? 1 + two : (steps + 31) / 32;
    const int threads = 32 * ((steps + nc - 1) / nc);
    const unsigned grid = (unsigned)p.a.rows;
    if (nc == 1)
        return launch_pdl(add_rmsnorm_kernel<R, WIDE, 1, true>, grid, threads, 0, s, p);
    if (nc == 2)
        return launch_pdl(add_rmsnorm_kernel<R, WIDE, 2, true>, grid, threads, 0, s, p);
    return launch_pdl(add_rmsnorm_kernel<R, WIDE, 3, true>, grid, threads, 0, s, p);
}

// Whether every row of a tensor (elements of `size` bytes) starts on a
// boundary of its 8-value accesses: 16 bytes, 8 for codes.
bool rows_wide(const void *p, int64_t stride, int64_t rows, int size)
{
    const uintptr_t unit = size == 1 ? 8 : 16;
    return aligned(p, unit) && (rows == 1 || (stride * size) % (int64_t)unit == 0);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const dvl_norm &a, cudaStream_t s)
{
    NormArgs p;
    p.a = a;
    p.inv_k = 1.f / (float)a.K;
    p.group_shift = 0;
    while ((1 << p.group_shift) < a.group)
        ++p.group_shift;
    p.groups = a.group ? (a.K + a.group - 1) / a.group : 1;
    const int rsize = a.residual_dtype == DVL_F32 ? 4 : 2;
    const bool wide = a.K % kVals == 0 && rows_wide(a.x, a.x_stride, a.rows, 2) &&
                      aligned(a.weight, 16) &&
                      rows_wide(a.residual, a.residual_stride, a.rows, rsize) &&
                      rows_wide(a.residual_out, a.residual_out_stride, a.rows, rsize) &&
                      rows_wide(a.out, a.out_stride, a.rows, 2) &&
                      rows_wide(a.codes, a.codes_stride, a.rows, 1);
    if (!a.residual)
        return wide ? launch<None, true>(p, s) : launch<None, false>(p, s);
    if (a.residual_dtype == DVL_F32)
        return wide ? launch<float, true>(p, s) : launch<float, false>(p, s);
    return wide ? launch<uint16_t, true>(p, s) : launch<uint16_t, false>(p, s);
}

}  // namespace dvl
