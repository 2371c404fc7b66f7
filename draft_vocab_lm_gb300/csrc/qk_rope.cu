// Norm of the new tokens' queries and keys for each head, rotation by their
// position, and the new keys and values to their places of a paged cache:
//   y = x w / sqrt(mean x^2 + eps),
//   (y1, y2) -> (y1 cos t - y2 sin t, y2 cos t + y1 sin t),  t = position freq.
//
// Pure streaming: every value is read once and written once, a dozen flops
// each, so many rows are bound by HBM and a few by the chain of dependent
// loads (sequence -> length -> page -> store).
//
// Split.  A head takes D / 8 lanes (rounded up to a power of two), 8 values
// each: the sum of squares is a butterfly over them and the other half of a
// pair (rot / 2 values away) lies in another lane's register.  A warp walks
// heads of ONE row, queries, then keys, then values, because a lane's cos and
// sin depend on the row and on its place in the head alone: computed once,
// they serve all of the row's heads.  Where rows are few, several warps share
// a row's heads, each with its own cos and sin.
//
// Angles.  freq is in turns per position, as a 64-bit fraction, so position x
// freq modulo one turn is an integer product that wraps: its upper 32 bits are
// the angle to 2^-32 of a turn however far the position, with no reduction.
// cos and sin then come from the fast units, which are good to 2^-21 within
// half a turn; the result is rounded to 8 bits or fewer.
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 4;  // 16-byte loads in flight per lane

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

// Eight values of a head, `live` ones, in the cache's type.
// at: the place of the row's head in the pool, in bytes (of NVFP4: of codes).
__device__ __forceinline__ void to_cache(const QkArgs &a, unsigned char *pool, unsigned char *blocks,
                                         int64_t at, int l, bool put, const float (&y)[8],
                                         float inv_scale, float scale)
{
    if (a.dtype == DVL_BF16) {
        if (put)
            *reinterpret_cast<uint4 *>(pool + at + 16 * l) = pack8(y);
    } else if (a.dtype == DVL_FP8) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = e4m3x2(y[4 * i] * inv_scale, y[4 * i + 1] * inv_scale) |
                   (uint32_t)e4m3x2(y[4 * i + 2] * inv_scale, y[4 * i + 3] * inv_scale) << 16;
        if (put)
            *reinterpret_cast<uint2 *>(pool + at + 8 * l) = make_uint2(w[0], w[1]);
    } else {
        float big = 0.f;
        bool nan = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            big = fmaxf(big, fabsf(y[e]));
            nan |= y[e] != y[e];
        }
        // 16 values are two lanes'
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
        nan = __shfl_xor_sync(kFull, (int)nan, 1) | (int)nan;
        const uint16_t s = nan ? 0x7f : e4m3x2(big * (inv_scale * (1.f / 6.f)), 0.f) & 0xff;
        const float unit = e4m3_value(s) * scale;
        const float inv = s == 0 ? 0.f : 1.f / unit;
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            z[e] = s == 0 ? 0.f : y[e] * inv;
        const uint32_t w = e2m1x8(z);
        if (put) {
            *reinterpret_cast<uint32_t *>(pool + at + 4 * l) = w;
            if ((l & 1) == 0)
                blocks[(at >> 3) + (l >> 1)] = (unsigned char)s;
        }
    }
}

// PAIRS: the other value of a pair is its neighbour, not rot / 2 away.
template <int LPH, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 5) qk_kernel(const __grid_constant__ QkArgs a)
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
    const int sub = lane / LPH, l = lane % LPH, d = 8 * l;
    const bool live = d < a.D;

    // the steps of a row: queries, keys, values, kHeads heads each
    const int nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.H + kHeads - 1) / kHeads;
    const int steps = nq + (a.dtype >= 0 ? 2 * nk : nk);
    const int from = (int)((int64_t)steps * part / a.parts), to = (int)((int64_t)steps * (part + 1) / a.parts);

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

    // cos and sin of the lane's values; the partner's sign goes with the sine
    const int half = a.rot / 2;
    const bool turned = d < a.rot;
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (PAIRS && (e & 1)) {
                cs[e] = cs[e - 1];
                sn[e] = -sn[e - 1];
                continue;
            }
            const int j = PAIRS ? (d + e) / 2 : d < half ? d + e : d + e - half;
            const uint64_t turns = (uint64_t)(int64_t)position * __ldg(a.freq + j);
            constexpr float kTurn = 6.283185307179586f / 4294967296.f;
            float s, c;
            __sincosf((float)(int32_t)(turns >> 32) * kTurn, &s, &c);
            cs[e] = c;
            sn[e] = PAIRS || d < half ? -s : s;
        }
    }
    const int partner = PAIRS || !turned ? lane : d < half ? lane + half / 8 : lane - half / 8;
    // a value that is not rotated meets no other (0 times an infinity is no 0)
    const uint32_t meets = turned ? 0xffffffffu : 0u;
    auto others = [&](const uint4 &x, const float (&own)[8], float (&other)[8]) {
        if constexpr (PAIRS) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                other[e] = turned ? own[e ^ 1] : 0.f;
        } else {
            uint4 o;
            o.x = __shfl_sync(kFull, x.x, partner) & meets;
            o.y = __shfl_sync(kFull, x.y, partner) & meets;
            o.z = __shfl_sync(kFull, x.z, partner) & meets;
            o.w = __shfl_sync(kFull, x.w, partner) & meets;
            unpack8(o, other);
        }
    };

    // Queries, then keys: the heads of steps [first, last) of `heads`.  Each
    // value is (x A + partner B) / rms, with the weights in A and B.
    const float per = 1.f / (float)a.D;
    auto normed = [&](int first, int last, int heads, const uint16_t *from, int64_t stride,
                      const uint16_t *weight, auto &&store) {
        float A[8], B[8];
        if (weight) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live)
                w = __ldg(reinterpret_cast<const uint4 *>(weight + d));
            float own[8], other[8];
            unpack8(w, own);
            others(w, own, other);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                A[e] = own[e] * cs[e];
                B[e] = other[e] * sn[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                A[e] = cs[e];
                B[e] = sn[e];
            }
        }
        int head = first * kHeads + sub;
        const uint16_t *at = from + head * stride + d;
        for (int i = first; i < last; i += kLoads) {
            uint4 x[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                x[u] = make_uint4(0, 0, 0, 0);
                if (i + u < last && live && head + u * kHeads < heads)
                    x[u] = *reinterpret_cast<const uint4 *>(at);
                at += kHeads * stride;
            }
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                if (i + u >= last)
                    break;
                float y[8], p[8];
                unpack8(x[u], y);
                others(x[u], y, p);
                float inv = 1.f;
                if (weight) {
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum = fmaf(y[e], y[e], sum);
#pragma unroll
                    for (int off = LPH / 2; off >= 1; off >>= 1)
                        sum += __shfl_xor_sync(kFull, sum, off);
                    inv = rsqrtf(fmaf(sum, per, a.eps));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = fmaf(p[e], B[e], y[e] * A[e]) * inv;
                store(head, live && head < heads, y);
                head += kHeads;
            }
        }
    };
    if (from < nq)
        normed(from, min(to, nq), a.Hq, a.q + row * a.qs, a.qh, a.q_weight,
               [&](int head, bool have, const float (&y)[8]) {
                   if (have)
                       *reinterpret_cast<uint4 *>(a.q_out + row * a.qos + head * a.qoh + d) = pack8(y);
               });
    if (to > nq && from < nq + nk)
        normed(max(from, nq) - nq, min(to, nq + nk) - nq, a.H, a.k + row * a.ks, a.kh, a.k_weight,
               [&](int head, bool have, const float (&y)[8]) {
                   if (a.k_out && have)
                       *reinterpret_cast<uint4 *>(a.k_out + row * a.kos + head * a.koh + d) = pack8(y);
                   if (a.dtype >= 0)
                       to_cache(a, a.ck, a.ckb, k_at + head * a.khead, l, put && have, y, a.k_inv, a.k_scale);
               });
    if (to > nq + nk) {
        const int first = max(from, nq + nk) - nq - nk, last = to - nq - nk;
        for (int i = first; i < last; i += kLoads) {
            uint4 x[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int head = (i + u) * kHeads + sub;
                x[u] = make_uint4(0, 0, 0, 0);
                if (i + u < last && live && head < a.H)
                    x[u] = *reinterpret_cast<const uint4 *>(a.v + row * a.vs + head * a.vh + d);
            }
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                if (i + u >= last)
                    break;
                const int head = (i + u) * kHeads + sub;
                float y[8];
                unpack8(x[u], y);
                to_cache(a, a.cv, a.cvb, v_at + head * a.vhead, l, put && live && head < a.H, y, a.v_inv,
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
    int lanes = 2;
    while (8 * lanes < a.D)
        lanes *= 2;
    const int per = 32 / lanes;
    const int steps = (a.Hq + per - 1) / per + (a.dtype >= 0 ? 2 : 1) * ((a.H + per - 1) / per);
    const int64_t wanted = (int64_t)di.sms * 16 / a.rows;
    a.parts = wanted < 1 ? 1 : wanted > steps ? steps : (int)wanted;
    const int64_t blocks = (a.rows * a.parts + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    void (*const kernels[2][5])(QkArgs) = {
        {qk_kernel<2, false>, qk_kernel<4, false>, qk_kernel<8, false>, qk_kernel<16, false>, qk_kernel<32, false>},
        {qk_kernel<2, true>, qk_kernel<4, true>, qk_kernel<8, true>, qk_kernel<16, true>, qk_kernel<32, true>}};
    int at = 0;
    while (2 << at < lanes)
        ++at;
    const auto kernel = kernels[a.interleaved][at];
    return launch_pdl(kernel, (unsigned)blocks, kThreads, 0, s, a);
}

}  // namespace dvl
