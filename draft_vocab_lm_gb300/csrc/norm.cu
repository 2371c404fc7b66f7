// Residual addition, root-mean-square norm, and the 8-bit codes of the
// result, in one pass over a row:
//   u = x + residual,  y = u w / sqrt(mean(u^2) + eps),
//   per group: a = max |y|, scale = a / 448, code = RNE_e4m3(y (448 / a)).
//
// Bound by HBM (6 flops per element against 5 to 13 bytes).  One block per
// row; a thread owns 8 consecutive values per step (one 16-byte load of a
// bf16 tensor), keeps u in registers between the sum and the output, and
// reads every input once.  Up to 8,192 values per row a thread owns one such
// chunk; wider rows take two or three.
//   - The sum of squares: per thread, butterfly per warp, then every warp
//     adds the warps' partial sums itself (one block barrier).  fp32
//     throughout.
//   - The group maximum: a group of 16 .. 256 values is 2 .. 32 consecutive
//     lanes of one warp (a warp's lanes own 256 consecutive values), so it is
//     a butterfly of that width; one scale per row takes a second barrier.
//     Maxima compare the bit patterns of |y| as unsigned integers: the order
//     is that of the values, with NaN above infinity, so a NaN reaches the
//     scale instead of being dropped.
//   - The codes are cut from the fp32 y, not from its bf16 rounding.
// Rows that 16-byte accesses do not fit (K % 8 != 0, an odd stride, a
// pointer off a 16-byte boundary) run the same kernel with element accesses.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kVals = 8;  // consecutive values per thread and step

struct NormArgs {
    dvl_norm a;
    int groups;  // per row
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

template <bool WIDE>
__device__ __forceinline__ void load8(const uint16_t *p, int n, float (&v)[kVals])
{
    if constexpr (WIDE) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            v[i] = i < n ? __uint_as_float((uint32_t)p[i] << 16) : 0.f;
    }
}

template <bool WIDE>
__device__ __forceinline__ void load8(const float *p, int n, float (&v)[kVals])
{
    if constexpr (WIDE) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0];
        const float4 b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            v[i] = i < n ? p[i] : 0.f;
    }
}

template <bool WIDE>
__device__ __forceinline__ void store8(uint16_t *p, int n, const float (&v)[kVals])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if constexpr (WIDE) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            if (i < n)
                p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

template <bool WIDE>
__device__ __forceinline__ void store8(float *p, int n, const float (&v)[kVals])
{
    if constexpr (WIDE) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            if (i < n)
                p[i] = v[i];
    }
}

template <bool WIDE>
__device__ __forceinline__ void store8_codes(uint8_t *p, int n, const float (&v)[kVals])
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = pack_e4m3(v[4 * i], v[4 * i + 1]) | pack_e4m3(v[4 * i + 2], v[4 * i + 3]) << 16;
    if constexpr (WIDE) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            if (i < n)
                p[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
    }
}

// The multiplier 448 / a of a group whose |y| has the bits amax, and its
// scale.  Below 2^-119 the multiplier is no fp32 number: codes 0.
__device__ __forceinline__ float code_factor(uint32_t amax, float *scale)
{
    const float a = __uint_as_float(amax);
    *scale = a / 448.f;
    return amax < 0x04000000u ? 0.f : 448.f / a;  // 0x04000000 is 2^-119
}

// R: the residual's storage (uint16_t: bf16).  NC: chunks per thread.
template <typename R, bool WIDE, int NC>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_kernel(const NormArgs p)
{
    __shared__ float part[32];
    __shared__ uint32_t part_max[32];
    pdl_launch_dependents();
    pdl_wait();
    const dvl_norm &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int K = a.K;
    const int64_t row = blockIdx.x;
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + row * a.x_stride;
    const uint16_t *w = static_cast<const uint16_t *>(a.weight);

    float u[NC][kVals];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = kVals * (c * blockDim.x + threadIdx.x);
        if (k < K) {
            load8<WIDE>(x + k, K - k, u[c]);
            if (a.residual) {
                float r[kVals];
                load8<WIDE>(static_cast<const R *>(a.residual) + row * a.residual_stride + k,
                            K - k, r);
#pragma unroll
                for (int i = 0; i < kVals; ++i)
                    u[c][i] += r[i];
                store8<WIDE>(static_cast<R *>(a.residual_out) + row * a.residual_out_stride + k,
                             K - k, u[c]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                u[c][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            ss = fmaf(u[c][i], u[c][i], ss);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        ss += __shfl_xor_sync(kFull, ss, off);
    if (lane == 0)
        part[warp] = ss;
    __syncthreads();
    ss = lane < warps ? part[lane] : 0.f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        ss += __shfl_xor_sync(kFull, ss, off);
    const float inv = 1.f / sqrtf(ss / (float)K + a.eps);

    uint32_t row_max = 0u;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = kVals * (c * blockDim.x + threadIdx.x);
        const bool live = k < K;
        uint32_t amax = 0u;
        if (live) {
            float wv[kVals];
            load8<WIDE>(w + k, K - k, wv);
#pragma unroll
            for (int i = 0; i < kVals; ++i) {
                u[c][i] = u[c][i] * inv * wv[i];
                if (WIDE || i < K - k)
                    amax = max(amax, __float_as_uint(u[c][i]) & 0x7fffffffu);
            }
            if (a.out)
                store8<WIDE>(static_cast<uint16_t *>(a.out) + row * a.out_stride + k, K - k, u[c]);
        }
        if (!a.codes)
            continue;
        if (a.group == 0) {
            row_max = max(row_max, amax);
            continue;
        }
        for (int off = a.group / (2 * kVals); off >= 1; off >>= 1)
            amax = max(amax, __shfl_xor_sync(kFull, amax, off));
        if (live) {
            float scale;
            const float f = code_factor(amax, &scale);
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                u[c][i] *= f;
            store8_codes<WIDE>(a.codes + row * a.codes_stride + k, K - k, u[c]);
            if (k % a.group == 0)
                a.scales[row * p.groups + k / a.group] = scale;
        }
    }
    if (a.codes && a.group == 0) {
        row_max = __reduce_max_sync(kFull, row_max);
        if (lane == 0)
            part_max[warp] = row_max;
        __syncthreads();
        row_max = __reduce_max_sync(kFull, lane < warps ? part_max[lane] : 0u);
        float scale;
        const float f = code_factor(row_max, &scale);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = kVals * (c * blockDim.x + threadIdx.x);
            if (k < K) {
#pragma unroll
                for (int i = 0; i < kVals; ++i)
                    u[c][i] *= f;
                store8_codes<WIDE>(a.codes + row * a.codes_stride + k, K - k, u[c]);
            }
        }
        if (threadIdx.x == 0)
            a.scales[row] = scale;
    }
}

template <typename R, bool WIDE>
cudaError_t launch(const NormArgs &p, cudaStream_t s)
{
    const int chunks = (p.a.K + kVals - 1) / kVals;
    const int nc = (chunks + kMaxThreads - 1) / kMaxThreads;
    const int threads = ((chunks + nc - 1) / nc + 31) / 32 * 32;
    const unsigned grid = (unsigned)p.a.rows;
    if (nc == 1)
        return launch_pdl(add_rmsnorm_kernel<R, WIDE, 1>, grid, threads, 0, s, p);
    if (nc == 2)
        return launch_pdl(add_rmsnorm_kernel<R, WIDE, 2>, grid, threads, 0, s, p);
    return launch_pdl(add_rmsnorm_kernel<R, WIDE, 3>, grid, threads, 0, s, p);
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
    p.groups = a.group ? (a.K + a.group - 1) / a.group : 1;
    const int rsize = a.residual_dtype == DVL_F32 ? 4 : 2;
    const bool wide = a.K % kVals == 0 && rows_wide(a.x, a.x_stride, a.rows, 2) &&
                      aligned(a.weight, 16) &&
                      rows_wide(a.residual, a.residual_stride, a.rows, rsize) &&
                      rows_wide(a.residual_out, a.residual_out_stride, a.rows, rsize) &&
                      rows_wide(a.out, a.out_stride, a.rows, 2) &&
                      rows_wide(a.codes, a.codes_stride, a.rows, 1);
    if (a.residual_dtype == DVL_F32)
        return wide ? launch<float, true>(p, s) : launch<float, false>(p, s);
    return wide ? launch<uint16_t, true>(p, s) : launch<uint16_t, false>(p, s);
}

}  // namespace dvl
