// Beam selection: log-softmax of every beam's logits, the beam's score added,
// and the k best (beam, row) pairs of a request:
//   score(j, n) = scores[j] + ((x[j][n] - m_j) - ln sum_n e^{x[j][n] - m_j}),
// m_j the row's largest logit.  m and the logarithm stay apart: their sum would
// lose the logarithm in a row of large numbers, wholly in one of the type's
// lowest value (a mask), whose rows are uniform and score -ln N, not 0.
//
// Each logit is read once and costs one exponential and a maximum: HBM bounds
// many long fp32 rows (512 rows of 248,320: 0.91 of the copy rate), issue slots
// many bf16 rows (1,024 of them, k = 8: 94 us, 0.81; with one logit per
// instruction and every key pushed by its own thread 142 us), and a chain of
// dependent steps few rows: about 5 us until the last segment has left its
// keys and 2 to 4 us to pick (64 rows of 248,320, k = 16: 20.7 us of which
// 9.5 are HBM time; 4 rows of 16,000: 6.2 us).  One launch:
//   - A block takes one segment of a row, in chunks that sit in registers.
//     Every thread keeps the maximum and the sum of exponentials of what it
//     has seen, two logits per instruction.  Within one beam the order of the
//     scores is that of the logits, so the segment's best rows are found as
//     packed (logit, row) keys: of the first chunk, 32 groups of 8 threads
//     compare their maxima, and the k-th largest of those bounds the k-th
//     largest key from below; vectors with a logit at or above the bound (a few
//     more than k) are kept aside in shared memory, as are those that exceed it
//     in later chunks.  At the end their keys count their betters, and the k
//     best are written out.  (A whole vector is put aside because a warp with
//     one passing logit in eight runs through all eight tests: on short
//     segments, which pass few, that costs less than the second look.)
//   - The last block of a request (a wrapping ticket) joins the segments'
//     maxima and sums, turns keys into scores, and picks: a segment list whose
//     head has r better heads can give its first k - r keys only.  Four keys of
//     every list come with its head, more only where the fourth is good enough.
// Ties are exact: bounds carry the place of their logit, rows are read in
// order, and later rows have to exceed a bound, not to reach it, so rows of
// equal logits (a constant row, a mask of the type's lowest value) pass in
// limited number.  A segment that overflows its room all the same (rising
// logits) is read again in slices that fit, with the keys cut back to the k
// best after each.  After chunk 1, 2, 4, 8 .. the block looks at what it
// holds: cutting it back to k gives a higher bound for the chunks to come (a
// chunk passes about k / c keys after c chunks).  No other barrier stands in
// the loop.  Nothing depends on the order blocks run in.
// Segments: four blocks per SM where the rows allow, never more than one round
// of them (before the paired instructions, 64 rows of 248,320: 9 segments 22.6
// us, 7 24.7, 12 29.8; 800 rows of 52,755: 1 segment 46, 2 51, 5 67).
#include <cuda_runtime.h>

#include "dvl_device.cuh"
#include "dvl_step.h"

namespace dvl {
namespace {

static_assert(DVL_MAX_BEAMS <= 32 && kBeamKeys >= DVL_MAX_BEAMS, "one warp's lanes cover k");

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBuffer = 8 * kThreads + kBeamKeys;  // a slice of 8 logits per thread, and the best so far
constexpr int kVectors = 512;                      // vectors kept aside between two looks
constexpr int kVectorsPerChunk = 4;                // per thread, in long segments
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_diff(float d)  // e^d
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d * kLog2e));
    return y;
}

// Two fp32 values in one register pair, and the instructions that work on both.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi)
{
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(Pair p, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// e^(v - ref) of both values
__device__ __forceinline__ Pair exp_diff2(Pair v, Pair minus_ref)
{
    float lo, hi;
    unpair(mul2(add2(v, minus_ref), pair(kLog2e, kLog2e)), lo, hi);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(lo));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(hi));
    return pair(lo, hi);
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
// Its values two by two (the type selects the width), and their maximum.
__device__ __forceinline__ void pairs(const uint4 &q, Pair (&p)[2])
{
    p[0] = pair(__uint_as_float(q.x), __uint_as_float(q.y));
    p[1] = pair(__uint_as_float(q.z), __uint_as_float(q.w));
}
__device__ __forceinline__ void pairs(const uint4 &q, Pair (&p)[4])
{
    p[0] = pair(bf16_lo(q.x), bf16_hi(q.x)), p[1] = pair(bf16_lo(q.y), bf16_hi(q.y));
    p[2] = pair(bf16_lo(q.z), bf16_hi(q.z)), p[3] = pair(bf16_lo(q.w), bf16_hi(q.w));
}
__device__ __forceinline__ float max_of(const float *, const uint4 &q)
{
    float m = __uint_as_float(q.x);
    asm("max.f32 %0, %0, %1, %2;"
        : "+f"(m)
        : "f"(__uint_as_float(q.y)), "f"(__uint_as_float(q.z)));
    return fmaxf(m, __uint_as_float(q.w));
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_of(const uint16_t *, const uint4 &q)
{
    const uint32_t m = max_bf16x2(max_bf16x2(q.x, q.y), max_bf16x2(q.z, q.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
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

struct Groups {
    uint64_t key[32];
    int rank[32];
};

struct Shared {
    uint64_t buffer[kBuffer];
    uint4 vector[kVectors];
    int row[kVectors];  // of a vector's first logit
    Groups groups;
    uint64_t best[kBeamKeys];
    float2 sums[kWarps];
    int n;           // keys in the buffer (may exceed its size: then it overflowed)
    int vectors;     // likewise
    unsigned ticket;
};

// The second half's view of the same shared memory.
constexpr int kPairs = DVL_MAX_BEAMS * (DVL_MAX_BEAMS + 1) / 2;  // keys r lists of k can give
constexpr int kFront = 4;  // keys of a list that are read with its head
struct PickShared {
    uint64_t hi[kBeamLists];          // of the heads: (score, beam)
    uint64_t lo[kBeamLists][kFront];  // of the lists' first keys: (logit, row)
    int16_t list_of[kBeamLists];
    uint64_t c_hi[kPairs], c_lo[kPairs];  // candidates
    Groups groups;
    // per beam: the largest logit, the logarithm of the sum, the beam's score
    float big[DVL_MAX_BEAMS], log_sum[DVL_MAX_BEAMS], base[DVL_MAX_BEAMS];
    int head[DVL_MAX_BEAMS];              // the k best heads, in order
    int n_heads, n;
};

// The k best of the buffer's n keys, each to the place of its rank in `out`.
// Up to eight threads share a key's comparisons.  Every thread calls it.
__device__ __forceinline__ void rank_keys(const Shared &s, int n, int k, uint64_t *out)
{
    const int shift = n <= kThreads / 8 ? 3 : n <= kThreads / 4 ? 2 : n <= kThreads / 2 ? 1 : 0;
    const int share = threadIdx.x & ((1 << shift) - 1);
    for (int first = 0; first < n; first += kThreads >> shift) {
        const int i = first + (threadIdx.x >> shift);
        const uint64_t key = i < n ? s.buffer[i] : 0ull;
        int rank = 0;
#pragma unroll 4
        for (int j = share; j < n; j += 1 << shift)
            rank += s.buffer[j] > key;
        for (int off = 1 << shift >> 1; off >= 1; off >>= 1)
            rank += __shfl_xor_sync(kFull, rank, off);
        if (i < n && rank < k && share == 0)
            out[rank] = key;
    }
}

// Cut the buffer's n keys back to the k best, in order, and return the k-th
// (0 when there are fewer).  Every thread calls it.
__device__ __forceinline__ uint64_t prune(Shared &s, int n, int k)
{
    if (threadIdx.x < kBeamKeys)
        s.best[threadIdx.x] = 0ull;
    __syncthreads();
    rank_keys(s, n, k, s.best);
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
    ulonglong2 front[kHeads][kFront / 2];  // in flight while the sums are joined
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int list = i * kThreads + (int)threadIdx.x;
#pragma unroll
        for (int j = 0; j < kFront / 2; ++j)
            front[i][j] = list < heads ? __ldcg(reinterpret_cast<const ulonglong2 *>(
                                             keys + (int64_t)list * kBeamKeys) + j)
                                       : make_ulonglong2(0ull, 0ull);
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
        if (lane == 0) {
            s.big[beam] = m;
            s.log_sum[beam] = logf(sum);
        }
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
        return score_key(s.base[beam] + ((key_logit(key) - s.big[beam]) - s.log_sum[beam]), beam);
    };
    uint64_t head_hi[kHeads], top = 0ull;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int list = i * kThreads + (int)threadIdx.x;
        head_hi[i] = front[i][0].x ? score_of(front[i][0].x, list / a.segments) : 0ull;
        top = head_hi[i] > top ? head_hi[i] : top;
    }
    const uint64_t bound = group_bound(s.groups, top, a.k);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (head_hi[i] && head_hi[i] >= bound) {
            const int at = atomicAdd(&s.n_heads, 1);
            s.hi[at] = head_hi[i];
#pragma unroll
            for (int j = 0; j < kFront / 2; ++j) {
                s.lo[at][2 * j] = front[i][j].x;
                s.lo[at][2 * j + 1] = front[i][j].y;
            }
            s.list_of[at] = (int16_t)(i * kThreads + threadIdx.x);
        }
    __syncthreads();
    // the k best of them in order
    const int n_heads = s.n_heads;
    for (int i = threadIdx.x; i < n_heads; i += kThreads) {
        const uint64_t hi = s.hi[i], lo = s.lo[i][0];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n_heads; ++j)
            rank += better(s.hi[j], s.lo[j][0], hi, lo);
        if (rank < a.k)
            s.head[rank] = i;
    }
    __syncthreads();
    // what is no better than the k-th head is none of the k best
    const int last = s.head[a.k - 1];
    const uint64_t floor_hi = last >= 0 ? s.hi[last] : 1ull, floor_lo = last >= 0 ? s.lo[last][0] : 0ull;
    auto enough = [&](uint64_t hi, uint64_t key) {
        return hi && !better(floor_hi, floor_lo, hi, key);
    };
    for (int i = threadIdx.x; i < a.k * a.k; i += kThreads) {
        const int r = i / a.k, j = i - r * a.k, h = s.head[r];
        if (r + j >= a.k || h < 0)
            continue;
        const int list = s.list_of[h], beam = list / a.segments;
        uint64_t key = s.lo[h][j < kFront ? j : kFront - 1];
        uint64_t hi = key ? score_of(key, beam) : 0ull;
        if (j >= kFront && enough(hi, key)) {  // (lists descend)
            key = __ldcg(keys + (int64_t)list * kBeamKeys + j);
            hi = key ? score_of(key, beam) : 0ull;
        }
        if (enough(hi, key)) {
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
        // in flight while the rank is counted; a row past N is a key that another
        // call left behind (a stale ticket lets the pick start too early)
        const int token = (unsigned)row >= (unsigned)a.N ? -1 : a.d2t ? a.d2t[row] : row;
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

// The keys of one vector past a bound (ties: or at it) into the buffer.
template <typename T>
__device__ __forceinline__ void put_keys(Shared &s, const uint4 &q, int row, float bound, bool ties)
{
    constexpr int V = 16 / sizeof(T);
    float v[V];
    widen(q, v);
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (v[e] > bound || (v[e] == bound && ties)) {
            const int at = atomicAdd(&s.n, 1);
            if (at < kBuffer)
                s.buffer[at] = make_key(v[e], row + e);
        }
}
// Those of the n vectors kept aside, past the bound they were kept for; `begin`
// is the row index of place 0.
template <typename T>
__device__ __forceinline__ void take_keys(Shared &s, int n, float bound, int place, int begin)
{
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int row = s.row[i];
        put_keys<T>(s, s.vector[i], row, bound, (row - begin) / (16 / (int)sizeof(T)) <= place);
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
    constexpr bool kAside = NV == kVectorsPerChunk;
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
        float m = kNegInf;
        Pair sum = 0ull;
        float bound = kNegInf;  // keys must exceed it,
        int place = -1;         // or reach it up to this place of the first chunk
        int chunk = 0;
        if (threadIdx.x == 0)
            s.n = s.vectors = 0;
        if (threadIdx.x < 32)
            s.groups.rank[threadIdx.x] = 0;
        for (int base = begin; base < end; base += kThreads * E) {
            const int first = base + (int)threadIdx.x * V;
            uint4 work[NV];
            float top_of[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                work[j] = next[j];
                top_of[j] = max_of(x, work[j]);
            }
            if (kAside && base + 2 * kThreads * E <= end) {  // (base + kThreads * E is above 0)
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    next[j] = ld_stream16(x + first + kThreads * E + j * kThreads * V);
            } else {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    next[j] = load_vector(x, first + kThreads * E + j * kThreads * V, end);
            }
            float top = top_of[0];
            int top_j = 0;
#pragma unroll
            for (int j = 1; j < NV; ++j)
                if (top_of[j] > top) {
                    top = top_of[j];
                    top_j = j;
                }
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
            const float scale = exp_diff(m - ref);
            sum = mul2(sum, pair(scale, scale));
            m = m_new;
            const Pair minus_ref = pair(-ref, -ref);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                Pair v[V / 2];
                pairs(work[j], v);
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    sum = add2(sum, exp_diff2(v[e], minus_ref));
            }

            // vectors with keys past the bound; with no bound yet, all of them
            const int ties = base == begin ? place : -1;
            if (top >= bound) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int row0 = first + j * kThreads * V;
                    const bool tie = j * kThreads + (int)threadIdx.x <= ties;
                    if (top_of[j] > bound || (top_of[j] == bound && tie)) {
                        if constexpr (kAside) {
                            const int at = atomicAdd(&s.vectors, 1);
                            if (at < kVectors) {
                                s.vector[at] = work[j];
                                s.row[at] = row0;
                            }
                        } else {
                            put_keys<T>(s, work[j], row0, bound, tie);
                        }
                    }
                }
            }
            ++chunk;
            if ((chunk & (chunk - 1)) == 0 && base + kThreads * E < end) {
                __syncthreads();
                const int held = s.vectors;
                int count = s.n;
                __syncthreads();
                if (held + count > 2 * k + 16 && held <= kVectors) {
                    if constexpr (kAside) {
                        take_keys<T>(s, held, bound, place, begin);
                        if (threadIdx.x == 0)
                            s.vectors = 0;
                        __syncthreads();
                        count = s.n;
                        __syncthreads();
                    }
                    if (count <= kBuffer) {
                        const uint64_t kth = prune(s, count, k);
                        if (kth) {
                            bound = key_logit(kth);
                            place = -1;
                        }
                    }
                }
            }
        }
        __syncthreads();
        const int held = s.vectors;
        if (kAside && held <= kVectors) {
            take_keys<T>(s, held, bound, place, begin);
            __syncthreads();
        }
        const int count = s.n;
        __syncthreads();
        if (held > kVectors || count > kBuffer) {
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
                const int held_now = s.n;
                __syncthreads();
                if (held_now > kBeamKeys || n0 == begin) {
                    const uint64_t kth = prune(s, held_now, k);
                    least = kth ? key_logit(kth) : kNegInf;
                }
            }
        }
        // the block's sum relative to its maximum
        float big = m;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            big = fmaxf(big, __shfl_xor_sync(kFull, big, off));
        float even, odd;
        unpair(sum, even, odd);
        float total = (even + odd) * exp_diff(m - (big == kNegInf ? 0.f : big));
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            total += __shfl_xor_sync(kFull, total, off);
        if (lane == 0)
            s.sums[warp] = make_float2(big, total);
        if (threadIdx.x < kBeamKeys)
            out[threadIdx.x] = 0ull;
        __syncthreads();
        rank_keys(s, s.n, k, out);
        if (threadIdx.x == 0) {
            big = kNegInf;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                big = fmaxf(big, s.sums[w].x);
            total = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                total += s.sums[w].y * exp_diff(s.sums[w].x - (big == kNegInf ? 0.f : big));
            a.sums[blockIdx.x] = make_float2(big, total);
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
        return launch_pdl(beam_select_kernel<T, kVectorsPerChunk>, grid, kThreads, 0, s, a);
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
