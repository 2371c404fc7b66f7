// Beam selection: log-softmax of every beam's logits, the beam's score added,
// and the k best (beam, row) pairs of a request:
//   score(j, n) = scores[j] + (x[j][n] - lse_j),  lse_j = m + ln sum e^{x - m}.
//
// Bound by HBM: each logit is read once and costs one exponential and a few
// comparisons.  Two kernels:
//   1. beam_scan_kernel, one block per chunk of a row, the chunk in
//      registers: the chunk's maximum and sum of exponentials, and its best
//      rows as packed (logit, row) keys.  Within one beam the order of the
//      scores is that of the logits, so no score is needed here.  The k best
//      of the chunk are found without sorting it: the k-th largest of the
//      threads' own maxima is a lower bound of the k-th largest key, and at
//      most k threads hold keys at or above it (keys are distinct), so a few
//      keys (k * E at the very most) go through shared memory to one warp.
//   2. beam_pick_kernel, one block per request: per beam the chunks' sums
//      join into lse and the chunks' lists merge into the beam's best; then
//      the beams' lists, now as (score, beam, place) keys, merge into the k
//      best of the request.
// Lists are 32 keys, one per lane of a warp, in descending order; two merge
// by the elementwise maximum of one and the other reversed (which holds the
// 32 largest of both as a bitonic sequence) and a five-step bitonic merge.
// Empty places are key 0.  Nothing depends on the order blocks run in.
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

static_assert(kBeamKeys == 32 && DVL_MAX_BEAMS <= 32, "one key per lane");

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;

// One compare-exchange step across the warp: this lane keeps the larger key
// of the pair when `high`.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int stride, bool high)
{
    const uint64_t o = __shfl_xor_sync(kFull, v, stride);
    return (o > v) == high ? o : v;
}

// Descending order across the lanes of a bitonic sequence.
__device__ __forceinline__ uint64_t warp_bitonic_merge(uint64_t v, int lane)
{
#pragma unroll
    for (int stride = 16; stride >= 1; stride >>= 1)
        v = exchange(v, stride, (lane & stride) == 0);
    return v;
}

__device__ __forceinline__ uint64_t warp_sort(uint64_t v, int lane)
{
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int stride = size / 2; stride >= 1; stride >>= 1)
            v = exchange(v, stride, ((lane & size) == 0) == ((lane & stride) == 0));
    return v;
}

// The 32 largest of two descending lists.
__device__ __forceinline__ uint64_t warp_merge_lists(uint64_t a, uint64_t b, int lane)
{
    const uint64_t r = __shfl_xor_sync(kFull, b, 31);
    return warp_bitonic_merge(a > r ? a : r, lane);
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        x += __shfl_xor_sync(kFull, x, off);
    return x;
}

__device__ __forceinline__ float exp_diff(float d)  // e^d, d <= 0
{
    return exp2f(d * kLog2e);
}

// One 16-byte vector of logits as fp32.
__device__ __forceinline__ void widen(const uint4 &q, float (&v)[4])
{
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void widen(const uint4 &q, float (&v)[8])
{
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ float widen1(float x) { return x; }
__device__ __forceinline__ float widen1(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// T: float, or uint16_t holding bf16.  E: logits per thread.  A row may start
// anywhere: the chunks are cut at 16-byte boundaries, row index n is place
// n + lead of the aligned sequence, and the vectors that reach over an end of
// the row are read element by element.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const BeamArgs a)
{
    constexpr int V = 16 / sizeof(T);
    constexpr int NV = E / V;
    constexpr int kMost = 32 * E;  // keys that can reach the threshold
    __shared__ uint64_t lists[kWarps][32];
    __shared__ uint64_t passed[kMost];
    __shared__ uint64_t s_thr;
    __shared__ float s_sum[kWarps];
    __shared__ int s_n;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / a.chunks;
    const int chunk = (int)(blockIdx.x - row * a.chunks);
    uint64_t *out = a.keys + (row * a.chunks + chunk) * kBeamKeys;
    if (!(a.scores[row] > kNegInf)) {  // a dead beam
        if (threadIdx.x < kBeamKeys)
            out[threadIdx.x] = 0ull;
        return;
    }
    const int64_t b = row / a.beams;
    const T *x = static_cast<const T *>(a.logits) + b * a.batch_stride +
                 (row - b * a.beams) * a.beam_stride;
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % V);
    const int first = chunk * (kThreads * E) - lead + (int)threadIdx.x * V;

    float v[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int n = first + j * kThreads * V;
        if (n >= 0 && n + V <= a.N) {
            widen(ld_stream16(x + n), v[j]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[j][e] = n + e >= 0 && n + e < a.N ? widen1(x[n + e]) : kNegInf;
        }
    }

    // the thread's best key: the lowest row among equal logits; -inf and NaN
    // are no candidates
    float best = kNegInf;
    int at = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (v[j][e] > best) {
                best = v[j][e];
                at = first + j * kThreads * V + e;
            }
    const uint64_t mine = best > kNegInf ? make_key(best, at) : 0ull;
    lists[warp][lane] = warp_sort(mine, lane);
    if (threadIdx.x == 0)
        s_n = 0;
    __syncthreads();

    uint64_t top = lists[0][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
        top = lists[w][0] > top ? lists[w][0] : top;
    const float m = top ? key_logit(top) : kNegInf;
    const float m_use = top ? m : 0.f;
    if (warp == 0) {
        uint64_t l = lists[0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            l = warp_merge_lists(l, lists[w][lane], lane);
        if (lane == a.k - 1)
            s_thr = l;
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
            sum += exp_diff(v[j][e] - m_use);
    sum = warp_sum(sum);
    if (lane == 0)
        s_sum[warp] = sum;
    __syncthreads();

    const uint64_t thr = s_thr;
    if (mine && mine >= thr) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (v[j][e] > kNegInf) {
                    const uint64_t key = make_key(v[j][e], first + j * kThreads * V + e);
                    if (key >= thr)
                        passed[atomicAdd(&s_n, 1)] = key;
                }
    }
    __syncthreads();
    if (warp == 0) {
        const int n = s_n;
        uint64_t l = warp_sort(lane < n ? passed[lane] : 0ull, lane);
        for (int i = 32; i < n; i += 32)
            l = warp_merge_lists(l, warp_sort(i + lane < n ? passed[i + lane] : 0ull, lane), lane);
        out[lane] = l;
        const float s = warp_sum(lane < kWarps ? s_sum[lane] : 0.f);
        if (lane == 0)
            a.sums[row * a.chunks + chunk] = make_float2(m, s);
    }
}

__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamArgs a)
{
    __shared__ uint64_t lists[kPickWarps][32];
    __shared__ int rows[DVL_MAX_BEAMS][32];
    __shared__ float s_lse[DVL_MAX_BEAMS];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    const int per_beam = kPickWarps / a.beams;  // warps per beam, >= 1
    const int beam = warp / per_beam, sub = warp - beam * per_beam;
    const bool live = beam < a.beams && a.scores[row0 + beam] > kNegInf;

    uint64_t l = 0ull;
    if (live) {
        const uint64_t *src = a.keys + (row0 + beam) * a.chunks * kBeamKeys + lane;
        for (int c = sub; c < a.chunks; c += per_beam)
            l = warp_merge_lists(l, src[(int64_t)c * kBeamKeys], lane);
        if (sub == 0) {
            const float2 *ms = a.sums + (row0 + beam) * a.chunks;
            float m = kNegInf, s = 0.f;
            for (int c = lane; c < a.chunks; c += 32)
                m = fmaxf(m, ms[c].x);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
                m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
            // a row of -inf only: m - m is NaN, and so are its scores
            for (int c = lane; c < a.chunks; c += 32)
                s += ms[c].y * exp_diff(ms[c].x - m);
            s = warp_sum(s);
            if (lane == 0)
                s_lse[beam] = m + logf(s);
        }
    }
    lists[warp][lane] = l;
    __syncthreads();

    // warp j: beam j's best, as (score, beam, place) keys
    l = 0ull;
    if (warp < a.beams) {
        for (int w = 0; w < per_beam; ++w) {
            const uint64_t o = lists[warp * per_beam + w][lane];
            l = w == 0 ? o : warp_merge_lists(l, o, lane);
        }
        rows[warp][lane] = key_id(l);
        if (l) {
            const float score = a.scores[row0 + warp] + (key_logit(l) - s_lse[warp]);
            l = score > kNegInf ? make_key(score, warp * 32 + lane) : 0ull;
        }
    }
    __syncthreads();
    if (warp < a.beams)
        lists[warp][lane] = l;
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < a.beams; ++w)
            l = warp_merge_lists(l, lists[w][lane], lane);
        if (lane < a.k) {
            const int64_t o = (int64_t)blockIdx.x * a.k + lane;
            if (l) {
                const int place = key_id(l);
                const int n = rows[place >> 5][place & 31];
                a.out_scores[o] = key_logit(l);
                a.parents[o] = place >> 5;
                a.tokens[o] = a.d2t ? a.d2t[n] : n;
            } else {
                a.out_scores[o] = kNegInf;
                a.parents[o] = -1;
                a.tokens[o] = -1;
            }
        }
    }
}

constexpr int kLong = 32, kShort = 8;  // logits per thread

template <typename T>
cudaError_t launch_scan(const BeamArgs &a, cudaStream_t s)
{
    const int64_t rows = (int64_t)a.batch * a.beams;
    const unsigned grid = (unsigned)(rows * a.chunks);
    if (beam_chunk(rows, a.N) == kThreads * kLong)
        return launch_pdl(beam_scan_kernel<T, kLong>, grid, kThreads, 0, s, a);
    return launch_pdl(beam_scan_kernel<T, kShort>, grid, kThreads, 0, s, a);
}

}  // namespace

// Long chunks cost fewer lists; short ones spread a small call over more SMs.
int beam_chunk(int64_t rows, int N)
{
    return kThreads * (rows * N >= (1 << 20) ? kLong : kShort);
}

int beam_chunks(int64_t rows, int N)
{
    const int c = beam_chunk(rows, N);
    return (int)(((int64_t)N + 7 + c - 1) / c);  // up to 7 places before a row's start
}

cudaError_t launch_beam_select(const BeamArgs &a, int dtype, cudaStream_t s)
{
    const cudaError_t e =
        dtype == DVL_F32 ? launch_scan<float>(a, s) : launch_scan<uint16_t>(a, s);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(beam_pick_kernel, (unsigned)a.batch, kPickThreads, 0, s, a);
}

}  // namespace dvl
