// Norm of the new tokens' queries and keys for each head, rotation by their
// position, and the new keys and values to their places of a paged cache:
//   y = x w / sqrt(mean x^2 + eps),
//   (y1, y2) -> (y1 cos t - y2 sin t, y2 cos t + y1 sin t),  t = position freq.
//
// Pure streaming: every value is read once and written once, a dozen flops
// each, so many rows are bound by HBM and a few by the chain of dependent
// loads (sequence -> length -> page -> store).
//
// Split.  A head takes D / 16 lanes (rounded up to a power of two), two chunks
// of 8 values each: of the rotated ones a chunk and the one rot / 2 values on,
// so that both values of every pair are in one lane (of the others one of each
// half of them: 16 bytes of neighbouring lanes are neighbours), and the sum of
// squares is a butterfly over the lanes.  (One chunk to a lane, the pair's
// other half fetched by shuffles, took 62 million warp instructions against 47
// for 16,381 rows of 40 + 2 x 8 heads of 128.)  A warp walks heads of ONE row,
// queries, then keys, then values, because a lane's cos and sin depend on the
// row and on its place in the head alone: computed once, they serve all of the
// row's heads.  Where rows are few, several warps share a row's heads, each
// with its own cos and sin, up to 16 warps an SM.
//
// Measured (GB300, wall time a call back to back): those 16,381 rows, bf16, 82
// us (460 MB, 0.83 of the copy rate; 75 with the arithmetic left out), E4M3 81,
// NVFP4 93, without a cache 69; 192 rows to an E4M3 cache 4.4 us, to an NVFP4 one
// 5.6; one row 3.1, the host's side of the call.  8,191 rows of 16 + 2 x 2 heads of
// 256, a quarter rotated, E4M3, no norm: 37 us (0.62; with one chunk to a lane 33).
// Ten steps of such a row are four batches of loads, because a batch ends with its
// kind of head, and a row's end and the next one's start are not overlapped within
// a warp.  Where a row has few heads its fixed cost (place, sines, three loops)
// is the time and most lanes idle: 16,001 rows of 1 + 2 x 1 heads of 64 28 us (12
// MB).  Equal or slower: 3 or 5 blocks an SM, two warps a row, loads of the next
// step before a step's arithmetic, rows looked up 32 at a time.
//
// Angles.  freq is in turns per position, as a 64-bit fraction, so position x
// freq modulo one turn is an integer product that wraps: its upper 32 bits are
// the angle to 2^-32 of a turn however far the position, with no reduction (as
// exact as the fraction is: half a unit of it is 2^-34 of a turn at 2^31).
// cos and sin then come from the fast units, which are good to 2^-21 within
// half a turn; the result is rounded to 8 bits or fewer.
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 4;  // per SM: 128 registers a thread
// Steps whose values a lane has in flight, 32 bytes each.  A row's steps of a kind
// of head go in batches of this many: with heads of 128 (four a step) 20 and 40
// heads fill batches of 5, 16, 32 and 64 batches of 4.  16,381 rows with 16, 20, 28,
// 32, 40 and 64 query heads: 5 54.9, 52.6, 64.1, 74.7, 82.3 and 115.0 us; 4 54.4,
// 55.7, 63.2, 73.4, 84.9 and 112.9; 3, 6 and 8 slower than the better of the two.
// Fewer rows, wide heads and few heads: 4 faster by 1 to 3 %.
constexpr int kLoads = 5;

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float e4m3_value(uint16_t code)
{
    float f;
    asm("{\n\t.reg .b32 p;\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.f16x2.e4m3x2 p, %1;\n\t"
        "mov.b32 {l, h}, p;\n\t"
        "cvt.f32.f16 %0, l;\n\t}"
        : "=f"(f)
        : "h"(code));
    return f;
}

// Eight values -> four bytes of E2M1 codes, value 2i in the low nibble of byte i.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}

// The sequence of row r: the last b with starts[b] <= r, found by 32 probes at
// a time (`starts` rises).  False for a row past the last sequence.
__device__ __forceinline__ bool find_sequence(const QkArgs &a, int64_t r, int lane, int *b, int64_t *end)
{
    if (!a.starts) {
        *b = (int)((uint32_t)r / (uint32_t)a.per_sequence);
        *end = (int64_t)(*b + 1) * a.per_sequence;
        return true;
    }
    int lo = 0, hi = a.B;  // the answer lies in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool below = at < hi && a.starts[at] <= r;
        const int n = __popc(__ballot_sync(kFull, below));
        lo += n * step;
        hi = min(hi, lo + step);
    }
    *b = lo;
    *end = a.starts[lo + 1];
    return r < *end && r >= a.starts[lo];
}

// A lane's place in a head: its two chunks of 8 values, and for NVFP4 where the
// other halves of their groups of 16 are: the lane, and which of its chunks.
struct Chunks {
    int first, second;
    bool live;
    int lane[2];
    bool of_second[2];
};
template <int LPH>
__device__ __forceinline__ Chunks chunks_of(int D, int rot, int lane)
{
    const int l = lane % LPH, turned = rot / 16;  // lanes with pairs
    Chunks c;
    c.live = 16 * l < D;
    const int rest = D / 16 - turned;  // lanes without
    c.first = l < turned ? l : turned + l;
    c.second = c.first + (l < turned ? turned : rest);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int mate = (i ? c.second : c.first) ^ 1;
        const bool pairs = mate < 2 * turned;
        const int half = pairs ? turned : rest, at = pairs ? mate : mate - 2 * turned;
        c.of_second[i] = at >= half;
        c.lane[i] = c.live ? lane - l + (pairs ? 0 : turned) + (c.of_second[i] ? at - half : at) : lane;
    }
    return c;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    return e4m3x2(a, b) | (uint32_t)e4m3x2(c, d) << 16;
}

// A lane's sixteen values of a head in the cache's type.  NVFP4: the quotients of
// the codes are rounded once, as middles between two codes are common among values
// of 8 bits, and a product with the reciprocal can lie on either side of one.  That
// product is corrected by its residual (P. Markstein, 1990: with a rounded
// reciprocal the result is the rounded quotient), two operations a value, where
// fp32 holds the residual: not for a block that saturates, nor for a tiny unit.
// 16,381 rows of 40 + 2 x 8 heads of 128: 93 us, with divisions 100, uncorrected
// 87; 192 rows 5.6, 6.1 and 4.8.
// at: the place of the row's head in the pool, in bytes (of NVFP4: of codes).
__device__ __forceinline__ void to_cache(const QkArgs &a, unsigned char *pool, unsigned char *blocks,
                                         int64_t at, const Chunks &c, bool put, const float (&y)[2][8],
                                         float inv_scale, float scale)
{
    const int chunk[2] = {c.first, c.second};
    if (a.dtype == DVL_BF16) {
        if (put) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<uint4 *>(pool + at + 16 * chunk[i]) = pack8(y[i]);
        }
    } else if (a.dtype == DVL_FP8) {
        if (put) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<uint2 *>(pool + at + 8 * chunk[i]) = make_uint2(
                    e4m3x4(y[i][0] * inv_scale, y[i][1] * inv_scale, y[i][2] * inv_scale, y[i][3] * inv_scale),
                    e4m3x4(y[i][4] * inv_scale, y[i][5] * inv_scale, y[i][6] * inv_scale, y[i][7] * inv_scale));
        }
    } else {
        // a NaN's bits are above every number's, so a maximum of bits keeps it
        uint32_t big[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                big[i] = max(big[i], __float_as_uint(y[i][e]) & 0x7fffffffu);
        uint32_t mate[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x0 = __shfl_sync(kFull, big[0], c.lane[i]);
            const uint32_t x1 = __shfl_sync(kFull, big[1], c.lane[i]);
            mate[i] = c.of_second[i] ? x1 : x0;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float m = __uint_as_float(max(big[i], mate[i]));
            const uint16_t s = e4m3x2(m / (6.f * scale), 0.f) & 0xff;  // NaN stays NaN
            const float unit = e4m3_value(s) * scale;
            float z[8];
            if (unit >= 0x1p-90f && m <= 8.f * unit) {
                const float inv = 1.f / unit;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z0 = y[i][e] * inv;
                    z[e] = fmaf(fmaf(z0, unit, -y[i][e]), -inv, z0);  // (these signs keep -0)
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    z[e] = s == 0 ? 0.f : y[i][e] / unit;
            }
            const uint32_t w = e2m1x8(z);
            if (put) {
                *reinterpret_cast<uint32_t *>(pool + at + 4 * chunk[i]) = w;
                if ((chunk[i] & 1) == 0)
                    blocks[(at >> 3) + (chunk[i] >> 1)] = (unsigned char)s;
            }
        }
    }
}

// PAIRS: the other value of a pair is its neighbour, not rot / 2 away.
template <int LPH, bool PAIRS>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_kernel(const __grid_constant__ QkArgs a)
{
    constexpr int kHeads = 32 / LPH;  // heads of a warp's step
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t row = unit / a.parts;
    const int part = (int)(unit - row * a.parts);
    if (row >= a.rows)
        return;
    const int sub = lane / LPH;
    const Chunks c = chunks_of<LPH>(a.D, a.rot, lane);
    const bool turned = 16 * (lane % LPH) < a.rot;

    // the steps of a row: queries, keys, values, kHeads heads each
    const int nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.H + kHeads - 1) / kHeads;
    const int steps = nq + (a.dtype >= 0 ? 2 * nk : nk);
    const int from = (int)((int64_t)steps * part / a.parts), to = (int)((int64_t)steps * (part + 1) / a.parts);

    // the first heads' values are on their way while the row's place is found
    uint4 x[kLoads][2];
    auto load = [&](int i, int last, int heads, const uint16_t *at, int64_t stride) {
        const int head = i * kHeads + sub;
        at += head * stride;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
            if (i + u < last && c.live && head + u * kHeads < heads) {
                x[u][0] = *reinterpret_cast<const uint4 *>(at + 8 * c.first);
                x[u][1] = *reinterpret_cast<const uint4 *>(at + 8 * c.second);
            }
            at += kHeads * stride;
        }
    };
    if (from < nq)
        load(from, min(to, nq), a.Hq, a.q + row * a.qs, a.qh);

    // place in the sequence and in the cache
    int position = 0;
    int64_t k_at = 0, v_at = 0;
    bool put = false;
    if (a.dtype >= 0) {
        int b;
        int64_t end;
        if (!find_sequence(a, row, lane, &b, &end))
            return;
        const int64_t place = a.lengths[b] - (end - row);
        position = (int)place;
        if (place >= 0 && place < (int64_t)a.width * a.page_size) {
            const int entry = (int)place / a.page_size, slot = (int)place - entry * a.page_size;
            const int page = a.table[b * a.table_stride + entry];
            put = (unsigned)page < (unsigned)a.pages;
            k_at = page * a.kp + slot * a.kt;
            v_at = page * a.vp + slot * a.vt;
        }
    }
    if (a.positions)
        position = a.positions[row];

    // cos and sin of the lane's eight pairs; values that are not rotated keep
    // 1 and 0
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (turned) {
            const int pair = PAIRS ? 4 * (e < 4 ? c.first : c.second) + (e & 3) : 8 * c.first + e;
            const uint64_t turns = (uint64_t)(int64_t)position * __ldg(a.freq + pair);
            constexpr float kTurn = 6.283185307179586f / 4294967296.f;
            __sincosf((float)(int32_t)(turns >> 32) * kTurn, &sn[e], &cs[e]);
        }
    }

    // Queries, then keys: the heads of steps [first, last) of `heads`.  With the
    // weights in them, a pair's four coefficients are A and B:
    //   y1 = (x1 A1 + x2 B1) / rms,  y2 = (x2 A2 + x1 B2) / rms.
    const float per = 1.f / (float)a.D;
    auto normed = [&](bool loaded, int first, int last, int heads, const uint16_t *from, int64_t stride,
                      const uint16_t *weight, auto &&store) {
        float A[2][8], B[2][8];
        {
            float w[2][8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 p = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);  // ones
                if (weight && c.live)
                    p = __ldg(reinterpret_cast<const uint4 *>(weight) + (i ? c.second : c.first));
                unpack8(p, w[i]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // the pair, and whether this is its second value
                    const int pair = PAIRS ? 4 * i + e / 2 : e;
                    const bool second = PAIRS ? e & 1 : i;
                    const float other = PAIRS ? w[i][e ^ 1] : w[1 - i][e];
                    A[i][e] = w[i][e] * cs[pair];
                    B[i][e] = other * (second ? sn[pair] : -sn[pair]);
                }
        }
        int head = first * kHeads + sub;
        for (int i = first; i < last; i += kLoads) {
            if (!loaded)
                load(i, last, heads, from, stride);
            loaded = false;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                if (i + u >= last)
                    break;
                float v[2][8], y[2][8];
                unpack8(x[u][0], v[0]);
                unpack8(x[u][1], v[1]);
                float inv = 1.f;
                if (weight) {
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sum[0] = fmaf(v[0][e], v[0][e], sum[0]);
                        sum[1] = fmaf(v[1][e], v[1][e], sum[1]);
                    }
                    sum[0] += sum[1];
#pragma unroll
                    for (int off = LPH / 2; off >= 1; off >>= 1)
                        sum[0] += __shfl_xor_sync(kFull, sum[0], off);
                    inv = rsqrtf(fmaf(sum[0], per, a.eps));
                }
                if (turned) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[k][e] = fmaf(PAIRS ? v[k][e ^ 1] : v[1 - k][e], B[k][e], v[k][e] * A[k][e]) * inv;
                } else {  // a value that is not rotated meets no other: 0 times an infinity is no 0
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[k][e] = v[k][e] * A[k][e] * inv;
                }
                store(head, c.live && head < heads, y);
                head += kHeads;
            }
        }
    };
    auto put_bf16 = [&](uint16_t *to, const float (&y)[2][8]) {
        *reinterpret_cast<uint4 *>(to + 8 * c.first) = pack8(y[0]);
        *reinterpret_cast<uint4 *>(to + 8 * c.second) = pack8(y[1]);
    };
    if (from < nq)
        normed(true, from, min(to, nq), a.Hq, a.q + row * a.qs, a.qh, a.q_weight,
               [&](int head, bool have, const float (&y)[2][8]) {
                   if (have)
                       put_bf16(a.q_out + row * a.qos + head * a.qoh, y);
               });
    if (to > nq && from < nq + nk)
        normed(false, max(from, nq) - nq, min(to, nq + nk) - nq, a.H, a.k + row * a.ks, a.kh, a.k_weight,
               [&](int head, bool have, const float (&y)[2][8]) {
                   if (a.k_out && have)
                       put_bf16(a.k_out + row * a.kos + head * a.koh, y);
                   if (a.dtype >= 0)
                       to_cache(a, a.ck, a.ckb, k_at + head * a.khead, c, put && have, y, a.k_inv, a.k_scale);
               });
    if (to > nq + nk) {
        const int first = max(from, nq + nk) - nq - nk, last = to - nq - nk;
        for (int i = first; i < last; i += kLoads) {
            load(i, last, a.H, a.v + row * a.vs, a.vh);
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                if (i + u >= last)
                    break;
                const int head = (i + u) * kHeads + sub;
                float y[2][8];
                unpack8(x[u][0], y[0]);
                unpack8(x[u][1], y[1]);
                to_cache(a, a.cv, a.cvb, v_at + head * a.vhead, c, put && c.live && head < a.H, y, a.v_inv,
                         a.v_scale);
            }
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(QkArgs &a, cudaStream_t s)
{
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    int lanes = 1, at = 0;
    for (; 16 * lanes < a.D; ++at)
        lanes *= 2;
    const int per = 32 / lanes;
    const int steps = (a.Hq + per - 1) / per + (a.dtype >= 0 ? 2 : 1) * ((a.H + per - 1) / per);
    const int64_t wanted = (int64_t)di.sms * 16 / a.rows;
    a.parts = wanted < 1 ? 1 : wanted > steps ? steps : (int)wanted;
    const int64_t blocks = (a.rows * a.parts + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    void (*const kernels[2][5])(QkArgs) = {
        {qk_kernel<1, false>, qk_kernel<2, false>, qk_kernel<4, false>, qk_kernel<8, false>, qk_kernel<16, false>},
        {qk_kernel<1, true>, qk_kernel<2, true>, qk_kernel<4, true>, qk_kernel<8, true>, qk_kernel<16, true>}};
    const auto kernel = kernels[a.interleaved][at];
    return launch_pdl(kernel, (unsigned)blocks, kThreads, 0, s, a);
}

}  // namespace dvl
