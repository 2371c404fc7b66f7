// Beam selection: log-softmax of every beam's logits, the beam's score added,
// and the k best (beam, row) pairs of a request:
//   score(j, n) = scores[j] + (x[j][n] - lse_j),  lse_j = m + ln sum e^{x - m}.
//
// Bound by HBM: each logit is read once and costs one exponential and a
// maximum.  One launch:
//   - A block takes one segment of a row, in chunks that sit in registers.
//     Every thread keeps the maximum and the sum of exponentials of what it
//     has seen.  Within one beam the order of the scores is that of the
//     logits, so the segment's best rows are found as packed (logit, row)
//     keys: of the first chunk, 32 groups of 8 threads compare their maxima,
//     and the k-th largest of those bounds the k-th largest key from below;
//     what lies at or above the bound (a few more than k) goes to a buffer in
//     shared memory, as does what exceeds it in later chunks.  At the end the
//     buffer's keys count their betters, and the k best are written out.
//   - The last block of a request (a wrapping ticket) joins the segments' sums
//     into lse, turns keys into scores, and picks: a segment list whose head
//     has r better heads can give its first k - r keys only.
// Ties are exact: bounds carry the place of their logit, rows are read in
// order, and later rows have to exceed a bound, not to reach it, so rows of
// equal logits (a constant row, a mask of the type's lowest value) pass in
// limited number.  A segment that overflows the buffer all the same (rising
// logits) is read again in slices that fit, with the buffer cut back to its
// k best after each.  After chunk 1, 2, 4, 8 .. the block looks at the buffer:
// cutting it back gives a higher bound for the chunks to come (a chunk passes
// about k / c keys after c chunks).  No other barrier stands in the loop.
// Nothing depends on the order blocks run in.
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

static_assert(DVL_MAX_BEAMS <= 32 && kBeamKeys >= DVL_MAX_BEAMS, "one warp's lanes cover k");

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBuffer = 8 * kThreads + kBeamKeys;  // a slice of 8 logits per thread, and the best so far
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_diff(float d)  // e^d
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d * kLog2e));
    return y;
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
// The vector at row index n, -inf outside [0, end).
__device__ __forceinline__ uint4 load_vector(const float *x, int n, int end)
{
    if (n >= 0 && n + 4 <= end)
        return ld_stream16(x + n);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = n + e >= 0 && n + e < end ? __float_as_uint(x[n + e]) : 0xff800000u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load_vector(const uint16_t *x, int n, int end)
{
    if (n >= 0 && n + 8 <= end)
        return ld_stream16(x + n);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = n + 2 * e;
        w[e] = (i >= 0 && i < end ? x[i] : 0xff80u) |
               (uint32_t)(i + 1 >= 0 && i + 1 < end ? x[i + 1] : 0xff80u) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int N>
__device__ __forceinline__ float max_of(const float (&v)[N])
{
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        m = fmaxf(m, v[i]);
    return m;
}

struct Groups {
    uint64_t key[32];
    int rank[32];
};

struct Shared {
    uint64_t buffer[kBuffer];
    Groups groups;
    uint64_t best[kBeamKeys];
    float2 sums[kWarps];
    int n;           // keys in the buffer (may exceed its size: then it overflowed)
    unsigned ticket;
};

// The second half's view of the same shared memory.
constexpr int kPairs = DVL_MAX_BEAMS * (DVL_MAX_BEAMS + 1) / 2;  // keys r lists of k can give
struct PickShared {
    uint64_t hi[kBeamLists], lo[kBeamLists];  // heads: (score, beam), (logit, row)
    int16_t list_of[kBeamLists];
    uint64_t c_hi[kPairs], c_lo[kPairs];  // candidates
    Groups groups;
    float lse[DVL_MAX_BEAMS], base[DVL_MAX_BEAMS];  // per beam, its score
    int head[DVL_MAX_BEAMS];              // the k best heads, in order
    int n_heads, n;
};

// Cut the buffer's n keys back to the k best, in order, and return the k-th
// (0 when there are fewer).  Every thread calls it.
__device__ __forceinline__ uint64_t prune(Shared &s, int n, int k)
{
    if (threadIdx.x < kBeamKeys)
        s.best[threadIdx.x] = 0ull;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t key = s.buffer[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j)
            rank += s.buffer[j] > key;
        if (rank < k)
            s.best[rank] = key;
    }
    __syncthreads();
    if (threadIdx.x < k)
        s.buffer[threadIdx.x] = s.best[threadIdx.x];
    if (threadIdx.x == 0)
        s.n = n < k ? n : k;
    const uint64_t last = s.best[k - 1];
    __syncthreads();
    return last;
}

// A bound from below of the k-th largest of the block's keys `mine` (0: none):
// the k-th largest of the maxima of 32 groups of 8 threads; 0 when fewer than
// k groups have a key.  The warps share the comparisons, a warp taking four
// groups against all.  Every thread calls it; g.rank is zero before.
__device__ __forceinline__ uint64_t group_bound(Groups &g, uint64_t mine, int k)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const uint64_t o = __shfl_xor_sync(kFull, mine, off);
        mine = o > mine ? o : mine;
    }
    if ((lane & 7) == 0)
        g.key[threadIdx.x >> 3] = mine;
    __syncthreads();
    mine = g.key[lane];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 32 / kWarps; ++i) {
        const int j = warp * (32 / kWarps) + i;
        const uint64_t o = g.key[j];
        rank += o > mine || (o == mine && j < lane);  // (empty groups are equal)
    }
    if (rank)
        atomicAdd(&g.rank[lane], rank);
    __syncthreads();
    return __shfl_sync(kFull, mine, __ffs(__ballot_sync(kFull, g.rank[lane] == k - 1)) - 1);
}

// (score, beam) as a key whose order is the result's: higher score, lower beam.
__device__ __forceinline__ uint64_t score_key(float score, int beam)
{
    return score > kNegInf ? make_key(score, beam) : 0ull;  // -inf and NaN: no candidate
}
__device__ __forceinline__ bool better(uint64_t hi, uint64_t lo, uint64_t hi2, uint64_t lo2)
{
    return hi > hi2 || (hi == hi2 && lo > lo2);
}

// The k best of a request, from its segments' lists.  One block.
__device__ __forceinline__ void pick(const BeamArgs &a, int64_t request, PickShared &s)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = request * a.beams;
    const int heads = a.beams * a.segments;
    const uint64_t *keys = a.keys + row0 * a.segments * kBeamKeys;
    constexpr int kHeads = (kBeamLists + kThreads - 1) / kThreads;  // per thread
    const float base = threadIdx.x < a.beams ? a.scores[row0 + threadIdx.x] : 0.f;
    uint64_t head[kHeads];  // in flight while the sums are joined
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int list = i * kThreads + (int)threadIdx.x;
        head[i] = list < heads ? __ldcg(keys + (int64_t)list * kBeamKeys) : 0ull;
    }
    for (int beam = warp; beam < a.beams; beam += kWarps) {
        const float2 *ms = a.sums + (row0 + beam) * a.segments;
        const float2 mine =
            lane < a.segments ? __ldcg(ms + lane) : make_float2(kNegInf, 0.f);
        float m = mine.x, sum = 0.f;
        for (int c = lane + 32; c < a.segments; c += 32)
            m = fmaxf(m, __ldcg(&ms[c].x));
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        // a row of -inf only: m - m is NaN, and so are its scores
        if (lane < a.segments)
            sum = mine.y * exp_diff(mine.x - m);
        for (int c = lane + 32; c < a.segments; c += 32) {
            const float2 x = __ldcg(&ms[c]);
            sum += x.y * exp_diff(x.x - m);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            sum += __shfl_xor_sync(kFull, sum, off);
        if (lane == 0)
            s.lse[beam] = m + logf(sum);
    }
    if (threadIdx.x < DVL_MAX_BEAMS) {
        s.head[threadIdx.x] = -1;
        s.groups.rank[threadIdx.x] = 0;
        s.base[threadIdx.x] = base;
    }
    if (threadIdx.x == 0)
        s.n = s.n_heads = 0;
    __syncthreads();
    auto score_of = [&](uint64_t key, int beam) {
        return score_key(s.base[beam] + (key_logit(key) - s.lse[beam]), beam);
    };
    uint64_t head_hi[kHeads], top = 0ull;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int list = i * kThreads + (int)threadIdx.x;
        head_hi[i] = head[i] ? score_of(head[i], list / a.segments) : 0ull;
        top = head_hi[i] > top ? head_hi[i] : top;
    }
    const uint64_t bound = group_bound(s.groups, top, a.k);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (head_hi[i] && head_hi[i] >= bound) {
            const int at = atomicAdd(&s.n_heads, 1);
            s.hi[at] = head_hi[i];
            s.lo[at] = head[i];
            s.list_of[at] = (int16_t)(i * kThreads + threadIdx.x);
        }
    __syncthreads();
    // the k best of them in order
    const int n_heads = s.n_heads;
    for (int i = threadIdx.x; i < n_heads; i += kThreads) {
        const uint64_t hi = s.hi[i], lo = s.lo[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n_heads; ++j)
            rank += better(s.hi[j], s.lo[j], hi, lo);
        if (rank < a.k)
            s.head[rank] = i;
    }
    __syncthreads();
    // what is no better than the k-th head is none of the k best
    const int last = s.head[a.k - 1];
    const uint64_t floor_hi = last >= 0 ? s.hi[last] : 1ull, floor_lo = last >= 0 ? s.lo[last] : 0ull;
    for (int i = threadIdx.x; i < a.k * a.k; i += kThreads) {
        const int r = i / a.k, j = i - r * a.k, h = s.head[r];
        if (r + j >= a.k || h < 0)
            continue;
        const int list = s.list_of[h];
        const uint64_t key = __ldcg(keys + (int64_t)list * kBeamKeys + j);
        const uint64_t hi = key ? score_of(key, list / a.segments) : 0ull;
        if (hi && !better(floor_hi, floor_lo, hi, key)) {
            const int at = atomicAdd(&s.n, 1);
            s.c_hi[at] = hi;
            s.c_lo[at] = key;
        }
    }
    __syncthreads();
    const int n = s.n;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t hi = s.c_hi[i], lo = s.c_lo[i];
        const int row = key_id(lo);
        const int token = a.d2t ? a.d2t[row] : row;  // in flight while the rank is counted
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j)
            rank += better(s.c_hi[j], s.c_lo[j], hi, lo);
        if (rank < a.k) {
            const int64_t o = request * a.k + rank;
            a.out_scores[o] = key_logit(hi);
            a.parents[o] = key_id(hi);
            a.tokens[o] = token;
        }
    }
    for (int i = n + threadIdx.x; i < a.k; i += kThreads) {
        const int64_t o = request * a.k + i;
        a.out_scores[o] = kNegInf;
        a.parents[o] = -1;
        a.tokens[o] = -1;
    }
}

// T: float, or uint16_t holding bf16.  NV: 16-byte vectors per thread and chunk,
// one chunk in work and one in flight.  A row
// may start anywhere: row index n is place n + lead of a sequence aligned to
// 16 bytes, segments are cut at such boundaries, and the vectors that reach
// over an end of the row are read element by element.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const BeamArgs a)
{
    constexpr int V = 16 / sizeof(T);
    constexpr int E = NV * V;  // logits per thread and chunk
    static_assert(V * kThreads + kBeamKeys <= kBuffer, "a slice fits the buffer");
    __shared__ union {
        Shared scan;
        PickShared pick;
    } sm;
    Shared &s = sm.scan;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / a.segments;
    const int segment = (int)(blockIdx.x - row * a.segments);
    const int64_t request = row / a.beams;
    const int k = a.k;
    uint64_t *out = a.keys + (int64_t)blockIdx.x * kBeamKeys;

    const T *x = static_cast<const T *>(a.logits) + request * a.batch_stride +
                 (row - request * a.beams) * a.beam_stride;
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % V);
    const int begin = segment * a.length - lead;  // of the segment, a multiple of V past the lead
    const int end = min(begin + a.length, a.N);
    // the chunk after the one in work; the first is in flight before the
    // beam's score says whether it is needed
    uint4 next[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        next[j] = load_vector(x, begin + (j * kThreads + (int)threadIdx.x) * V, end);
    if (a.scores[row] > kNegInf) {
        float m = kNegInf, sum = 0.f;
        float bound = kNegInf;  // later rows must exceed it
        int chunk = 0;
        if (threadIdx.x == 0)
            s.n = 0;
        if (threadIdx.x < 32)
            s.groups.rank[threadIdx.x] = 0;
        for (int base = begin; base < end; base += kThreads * E) {
            const int first = base + (int)threadIdx.x * V;
            float v[NV][V];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                widen(next[j], v[j]);
                next[j] = load_vector(x, first + kThreads * E + j * kThreads * V, end);
            }
            float top = max_of(v[0]);
            int top_j = 0;
#pragma unroll
            for (int j = 1; j < NV; ++j) {
                const float t = max_of(v[j]);
                if (t > top) {
                    top = t;
                    top_j = j;
                }
            }
            // the place up to which logits equal to the bound pass
            int place = -1;
            if (base == begin) {
                const uint64_t key = group_bound(
                    s.groups, top > kNegInf ? make_key(top, top_j * kThreads + threadIdx.x) : 0ull, k);
                if (key) {
                    bound = key_logit(key);
                    place = key_id(key);
                }
            }

            const float m_new = fmaxf(m, top);
            const float ref = m_new == kNegInf ? 0.f : m_new;
            sum *= exp_diff(m - ref);
            m = m_new;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum += exp_diff(v[j][e] - ref);

            // keys past the bound into the buffer; with no bound yet, all of them
            auto passes = [&](float t, int j) {
                return t > bound || (t == bound && j * kThreads + (int)threadIdx.x <= place);
            };
            if (top >= bound) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (max_of(v[j]) >= bound)
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (passes(v[j][e], j)) {
                                const int at = atomicAdd(&s.n, 1);
                                if (at < kBuffer)
                                    s.buffer[at] = make_key(v[j][e], first + j * kThreads * V + e);
                            }
            }
            ++chunk;
            if ((chunk & (chunk - 1)) == 0 && base + kThreads * E < end) {
                __syncthreads();
                const int count = s.n;
                __syncthreads();
                if (count > 2 * k + 16 && count <= kBuffer) {
                    const uint64_t kth = prune(s, count, k);
                    if (kth)
                        bound = key_logit(kth);
                }
            }
        }
        __syncthreads();
        const int count = s.n;
        __syncthreads();
        if (count > kBuffer) {
            prune(s, 0, k);
            float least = kNegInf;
            for (int n0 = begin; n0 < end; n0 += kThreads * V) {
                const int n = n0 + (int)threadIdx.x * V;
                float v[V];
                widen(load_vector(x, n, end), v);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (v[e] > least)
                        s.buffer[atomicAdd(&s.n, 1)] = make_key(v[e], n + e);
                __syncthreads();
                const int held = s.n;
                __syncthreads();
                if (held > kBeamKeys || n0 == begin) {
                    const uint64_t kth = prune(s, held, k);
                    least = kth ? key_logit(kth) : kNegInf;
                }
            }
        }
        // the block's sum relative to its maximum
        float big = m;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            big = fmaxf(big, __shfl_xor_sync(kFull, big, off));
        sum *= exp_diff(m - (big == kNegInf ? 0.f : big));
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            sum += __shfl_xor_sync(kFull, sum, off);
        if (lane == 0)
            s.sums[warp] = make_float2(big, sum);
        if (threadIdx.x < kBeamKeys)
            out[threadIdx.x] = 0ull;
        __syncthreads();
        // the buffer's k best, each key at the place of its rank
        const int n = s.n;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t key = s.buffer[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j)
                rank += s.buffer[j] > key;
            if (rank < k)
                out[rank] = key;
        }
        if (threadIdx.x == 0) {
            big = kNegInf;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                big = fmaxf(big, s.sums[w].x);
            sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += s.sums[w].y * exp_diff(s.sums[w].x - (big == kNegInf ? 0.f : big));
            a.sums[blockIdx.x] = make_float2(big, sum);
        }
    } else {  // a dead beam
        if (threadIdx.x < kBeamKeys)
            out[threadIdx.x] = 0ull;
        if (threadIdx.x == 0)
            a.sums[blockIdx.x] = make_float2(kNegInf, 0.f);
    }
    __syncthreads();
    const unsigned blocks = (unsigned)(a.beams * a.segments);
    if (threadIdx.x == 0)
        s.ticket = ticket_inc(a.tickets + request, blocks - 1);
    __syncthreads();
    const bool last = s.ticket == blocks - 1;
    __syncthreads();
    if (last)
        pick(a, request, sm.pick);
}

constexpr int kLeast = 8 * kThreads;  // logits of a segment, at least

}  // namespace

// Segments of a row: as many as fill the SMs, of kLeast logits at least.
int beam_segments(int64_t rows, int N)
{
    const int64_t most = ((int64_t)N + 7 + kLeast - 1) / kLeast;
    const int64_t n = rows > 0 && rows < kBeamLists ? kBeamLists / rows : 1;
    return (int)(n < most ? n : most);
}

template <typename T>
static cudaError_t launch(const BeamArgs &a, unsigned grid, cudaStream_t s)
{
    // Four vectors per thread keep 64 KB per SM in flight; a segment of the
    // least length runs through less code in a chunk of its own size.
    if (a.length > 2 * kLeast)
        return launch_pdl(beam_select_kernel<T, 4>, grid, kThreads, 0, s, a);
    return launch_pdl(beam_select_kernel<T, 8 * sizeof(T) / 16>, grid, kThreads, 0, s, a);
}

cudaError_t launch_beam_select(BeamArgs &a, int dtype, cudaStream_t s)
{
    const int64_t rows = (int64_t)a.batch * a.beams;
    // up to 7 places before a row's start; lengths are multiples of a vector
    a.length = (int)((((int64_t)a.N + 7 + a.segments - 1) / a.segments + 7) / 8 * 8);
    const unsigned grid = (unsigned)(rows * a.segments);
    return dtype == DVL_F32 ? launch<float>(a, grid, s) : launch<uint16_t>(a, grid, s);
}

}  // namespace dvl
