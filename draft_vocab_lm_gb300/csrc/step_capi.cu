// The C ABI of the drafting step's operators: argument checks and dispatch.
// Every check runs on the host before anything is enqueued; nothing here
// allocates, frees or synchronizes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstring>
#include <utility>

#include "dvl_attention.h"
#include "dvl_step.h"

namespace dvl {
namespace {

dvl_status done(cudaError_t e) { return e == cudaSuccess ? DVL_OK : cuda_failed(e); }

// A row tensor of the norm: pointer alignment, and the stride when it matters.
bool row_ok(const void *p, int64_t stride, int64_t rows, int64_t least, int size)
{
    return !p || (aligned(p, (uintptr_t)size) && (rows <= 1 || stride >= least));
}

dvl_status check_cache(const dvl_kv_cache *c)
{
    if (!c || (c->dtype != DVL_BF16 && c->dtype != DVL_FP8 && c->dtype != DVL_NVFP4) || c->reserved != 0)
        return DVL_ERR_INVALID_ARG;
    if (c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->D < 16 || c->D % 16 != 0 ||
        c->D > DVL_MAX_HEAD_DIM)
        return DVL_ERR_INVALID_ARG;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
        return DVL_ERR_INVALID_ARG;
    if (c->dtype == DVL_NVFP4 && (c->D % 64 != 0 || !c->k_blocks || !c->v_blocks ||
                                  !aligned(c->k_blocks, 16) || !aligned(c->v_blocks, 16)))
        return DVL_ERR_INVALID_ARG;
    // elements in 16 bytes; NVFP4 rows of scales start on their own size
    const int64_t unit = c->dtype == DVL_BF16 ? 8 : c->dtype == DVL_FP8 ? 16 : c->D;
    const int64_t strides[6] = {c->k_page_stride, c->k_token_stride, c->k_head_stride,
                                c->v_page_stride, c->v_token_stride, c->v_head_stride};
    for (int64_t s : strides)
        if (s < 0 || s % unit != 0)
            return DVL_ERR_INVALID_ARG;
    // one page spans less than 2 GB: offsets within a page are 32-bit
    for (int i = 0; i < 6; i += 3)
        if ((double)strides[i + 1] * c->page_size + (double)strides[i + 2] * c->heads > 1e9)
            return DVL_ERR_INVALID_ARG;
    if (!std::isfinite(c->k_scale) || !std::isfinite(c->v_scale))
        return DVL_ERR_INVALID_ARG;
    return DVL_OK;
}

// Half bytes per cached value.
int half_bytes(const dvl_kv_cache *c)
{
    return c->dtype == DVL_BF16 ? 4 : c->dtype == DVL_FP8 ? 2 : 1;
}

// pos / page_size for 0 <= pos < 2^31: multiply by 2^(31 + s) / page_size
// rounded up, s = ceil(log2 page_size); the error stays below one unit.
void page_division(int page_size, uint32_t *mul, int *shift)
{
    int s = 0;
    while ((1ll << s) < page_size)
        ++s;
    *shift = 31 + s;
    *mul = (uint32_t)((1ull << *shift) / (uint64_t)page_size + 1);
}

// Query rows per cached head, or 0 when T and Hq are outside the limits.
int query_rows(const dvl_kv_cache *c, int32_t T, int32_t Hq)
{
    if (T < 1 || T > DVL_MAX_QUERY || Hq < 1 || Hq % c->heads != 0)
        return 0;
    const int64_t rows = (int64_t)T * (Hq / c->heads);
    return rows <= DVL_MAX_QUERY_ROWS ? (int)rows : 0;
}

// Floats of one part: the rows' sums, then maximum and weight sum per row, and
// room for those of a joined group.
int64_t part_floats(int rows, int D) { return (int64_t)rows * (D + 4); }

// Both workspaces begin with the header and a fixed number of tickets, so that
// calls of different sizes can share one: no call's data lies where another
// expects its tickets at zero.
constexpr size_t kTicketBytes = 4 * kMaxCtas * sizeof(unsigned int);
constexpr int kBeamRequests = 4 * kMaxCtas;  // requests per launch

size_t attention_bytes(int blocks, int rows, int D)
{
    return kWsSlots + kTicketBytes + (size_t)2 * blocks * part_floats(rows, D) * sizeof(float);
}

// `rows` rows of `bytes` consecutive bytes each, `stride` apart.
struct Rows {
    uintptr_t at;
    int64_t rows, bytes, stride;
    uintptr_t end() const { return at + (uintptr_t)(rows - 1) * (uintptr_t)stride + (uintptr_t)bytes; }
};

// Whether a byte lies in a row of both.  Rows of two tensors may lie between
// each other's; only where the spans meet is row compared with row.
bool overlap(const Rows &a, const Rows &b)
{
    if (a.rows < 1 || b.rows < 1 || a.end() <= b.at || b.end() <= a.at)
        return false;
    const Rows &few = a.rows <= b.rows ? a : b, &many = a.rows <= b.rows ? b : a;
    for (int64_t i = 0; i < few.rows; ++i) {
        const uintptr_t x = few.at + (uintptr_t)i * (uintptr_t)few.stride;
        // the first of the other's rows that ends past x
        int64_t j = 0;
        if (x >= many.at + (uintptr_t)many.bytes)
            j = (int64_t)((x - many.at - (uintptr_t)many.bytes) / (uintptr_t)many.stride) + 1;
        if (j < many.rows &&
            many.at + (uintptr_t)j * (uintptr_t)many.stride < x + (uintptr_t)few.bytes)
            return true;
    }
    return false;
}

// A tensor [rows][heads][D] of bf16 as dvl_qk has it, and the bytes of its rows.
struct HeadRows {
    const void *p;
    int64_t stride, head_stride;  // elements
    int heads;
};
bool heads_ok(const HeadRows &t, bool optional)
{
    if (!t.p)
        return optional;
    return aligned(t.p, 16) && t.stride % 8 == 0 && t.head_stride % 8 == 0 && t.stride >= 0 && t.head_stride >= 0;
}
// Whether no value of an output is another's: heads within rows, or rows
// within heads.
bool apart(const HeadRows &t, int64_t rows, int D)
{
    const int64_t in_row = (t.heads - 1) * t.head_stride + D, in_head = (rows - 1) * t.stride + D;
    return (t.heads == 1 || t.head_stride >= D) && (rows == 1 || t.stride >= D) &&
           (rows == 1 || t.heads == 1 || t.stride >= in_row || t.head_stride >= in_head);
}
bool same(const HeadRows &x, const HeadRows &y, int64_t rows)
{
    return x.p == y.p && (rows == 1 || x.stride == y.stride) &&
           (x.heads == 1 || x.head_stride == y.head_stride) && x.heads == y.heads;
}
// Floor of x / d, d > 0.
int64_t floor_div(int64_t x, int64_t d) { return x / d - (x % d < 0); }

// The differences lo .. hi of two tensors' indices along an axis, `stride` bytes each.
struct Axis {
    int64_t lo, hi, stride;
};
// Whether runs of bx bytes of one tensor and of by bytes of another meet: whether
// some off + i a.stride + j b.stride lies in (-by, bx), off the distance of the
// first runs.  Only differences along the longer stride that the other axis can
// make up for are tried: a few, where one axis lies within the other.
bool runs_meet(int64_t off, int64_t bx, int64_t by, Axis a, Axis b)
{
    if (off + a.hi * a.stride + b.hi * b.stride <= -by || off + a.lo * a.stride + b.lo * b.stride >= bx)
        return false;  // (nearly every call)
    if (a.stride < b.stride)
        std::swap(a, b);
    if (b.stride == 0)
        b = {0, 0, 1};
    if (a.stride == 0)
        a = {0, 0, 1};
    const int64_t first = -floor_div(off + b.hi * b.stride + by - 1, a.stride);
    const int64_t last = floor_div(bx - 1 - off - b.lo * b.stride, a.stride);
    for (int64_t i = std::max(first, a.lo); i <= std::min(last, a.hi); ++i) {
        const int64_t at = off + i * a.stride;
        if (std::max(-floor_div(at + by - 1, b.stride), b.lo) <= std::min(floor_div(bx - 1 - at, b.stride), b.hi))
            return true;
    }
    return false;
}

// Whether two of these tensors share a byte.  Where their strides differ: whether
// they may, by rows where the heads of a row lie together, else by the span of all.
bool meet(const HeadRows &x, const HeadRows &y, int64_t rows, int D)
{
    if (!x.p || !y.p)
        return false;
    const Axis r = {1 - rows, rows - 1, rows == 1 ? 0 : 2 * x.stride};
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(y.p) - reinterpret_cast<uintptr_t>(x.p));
    if ((rows == 1 || x.stride == y.stride) &&
        (x.heads == 1 || y.heads == 1 || x.head_stride == y.head_stride)) {
        const Axis h = {1 - x.heads, y.heads - 1,
                        x.heads > 1 ? 2 * x.head_stride : y.heads > 1 ? 2 * y.head_stride : 0};
        return runs_meet(off, 2 * D, 2 * D, r, h);
    }
    auto bytes = [&](const HeadRows &t) {
        const int64_t row = 2 * ((t.heads - 1) * t.head_stride + D);
        const uintptr_t at = reinterpret_cast<uintptr_t>(t.p);
        if (rows == 1 || 2 * t.stride >= row)
            return Rows{at, rows, row, rows == 1 ? row : 2 * t.stride};
        const int64_t span = row + 2 * (rows - 1) * t.stride;
        return Rows{at, 1, span, span};
    };
    const Rows a = bytes(x), b = bytes(y);
    if (a.rows == rows && b.rows == rows && a.stride == b.stride)
        return runs_meet(off, a.bytes, b.bytes, r, {0, 0, 0});
    return overlap(a, b);
}

// The outputs of a call, and whether what it reads reaches into them.  Nearly
// nothing lies between their first and last bytes: that is asked first.
class Written {
    const HeadRows out_[2];
    const int64_t rows_;
    const int D_;
    uintptr_t from_[2] = {}, end_[2] = {};

public:
    Written(const HeadRows &x, const HeadRows &y, int64_t rows, int D) : out_{x, y}, rows_(rows), D_(D)
    {
        for (int i = 0; i < 2; ++i)
            if (out_[i].p && rows > 0) {
                from_[i] = reinterpret_cast<uintptr_t>(out_[i].p);
                end_[i] = from_[i] + 2 * ((rows - 1) * out_[i].stride + (out_[i].heads - 1) * out_[i].head_stride + D);
            }
    }
    // `count` rows of `bytes` from p on, `stride` bytes apart.
    bool meets(const void *p, int64_t count, int64_t bytes, int64_t stride) const
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p), last = at + (count - 1) * stride;
        for (int i = 0; i < 2; ++i)
            if (at < end_[i] && last + bytes > from_[i] && p && count > 0 && bytes > 0 &&
                look(i, at, count, bytes, stride))
                return true;
        return false;
    }
    // A cache's pages, each counted whole.
    bool meets(const dvl_kv_cache &c) const
    {
        const int64_t half = half_bytes(&c);
        for (int i = 0; i < (c.dtype == DVL_NVFP4 ? 4 : 2); ++i) {
            const bool values = i & 1;
            const int shift = i < 2 ? 1 : 4;
            const int64_t page = values ? c.v_page_stride : c.k_page_stride,
                          token = values ? c.v_token_stride : c.k_token_stride,
                          head = values ? c.v_head_stride : c.k_head_stride;
            if (meets(i < 2 ? (values ? c.v : c.k) : (values ? c.v_blocks : c.k_blocks), c.pages,
                      ((c.page_size - 1) * token + (c.heads - 1) * head + c.D) * half >> shift, page * half >> shift))
                return true;
        }
        return false;
    }

private:
    bool look(int i, uintptr_t p, int64_t count, int64_t bytes, int64_t stride) const
    {
        const HeadRows &x = out_[i];
        const Axis r = {1 - rows_, 0, rows_ == 1 ? 0 : 2 * x.stride};
        const Axis h = {1 - x.heads, 0, x.heads == 1 ? 0 : 2 * x.head_stride};
        const int64_t at = (int64_t)(p - from_[i]), end = (int64_t)(end_[i] - from_[i]);
        if (count > 1 && stride <= bytes) {
            bytes += (count - 1) * stride;
            count = 1;
        }
        // only the rows that reach into the output's span
        for (int64_t k = count > 1 ? std::max<int64_t>(0, floor_div(-at - bytes, stride) + 1) : 0;
             k < count && at + k * stride < end; ++k)
            if (runs_meet(at + k * stride, 2 * D_, bytes, r, h))
                return true;
        return false;
    }
};

bool beam_sizes_ok(int32_t batch, int32_t beams, int32_t N)
{
    return batch >= 0 && beams >= 1 && beams <= DVL_MAX_BEAMS && N >= 1 &&
           N <= 0x7fffffff - 65536 && (int64_t)batch * beams <= 0x7fffffffLL;
}

// Lists of one launch: at least kBeamLists, so that the size grows with the
// batch although fewer rows are cut into more segments.
int64_t beam_lists(int32_t batch, int32_t beams)
{
    const int64_t rows = (int64_t)(batch < kBeamRequests ? batch : kBeamRequests) * beams;
    return rows > kBeamLists ? rows : kBeamLists;
}

}  // namespace
}  // namespace dvl

using namespace dvl;

extern "C" {

dvl_status dvl_add_rmsnorm(const dvl_norm *p, void *stream)
{
    if (!p || p->rows < 0 || p->rows > 0x7fffffffLL || p->K < 1 || p->K > DVL_MAX_K)
        return DVL_ERR_INVALID_ARG;
    if (p->residual_dtype != DVL_BF16 && p->residual_dtype != DVL_F32)
        return DVL_ERR_INVALID_ARG;
    if (p->group != 0 && p->group != 16 && p->group != 32 && p->group != 64 && p->group != 128 &&
        p->group != 256)
        return DVL_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || !std::isfinite(p->eps))
        return DVL_ERR_INVALID_ARG;
    if (!p->x || !p->weight || !aligned(p->weight, 2) || (!p->out && !p->codes) ||
        !p->codes != !p->scales || !p->residual != !p->residual_out || !aligned(p->scales, 4))
        return DVL_ERR_INVALID_ARG;
    const int rsize = p->residual_dtype == DVL_F32 ? 4 : 2;
    if (!row_ok(p->x, p->x_stride, p->rows, 0, 2) ||
        !row_ok(p->residual, p->residual_stride, p->rows, 0, rsize) ||
        !row_ok(p->residual_out, p->residual_out_stride, p->rows, p->K, rsize) ||
        !row_ok(p->out, p->out_stride, p->rows, p->K, 2) ||
        !row_ok(p->codes, p->codes_stride, p->rows, p->K, 1))
        return DVL_ERR_INVALID_ARG;
    if (p->rows == 0)
        return DVL_OK;
    return done(launch_add_rmsnorm(*p, static_cast<cudaStream_t>(stream)));
}

size_t dvl_attention_workspace_bytes(const dvl_kv_cache *cache, int32_t T, int32_t Hq)
{
    if (check_cache(cache) != DVL_OK)
        return 0;
    const int rows = query_rows(cache, T, Hq);
    attn::AttnConfig cfg;
    int blocks = 0;
    if (rows == 0 || attn::grid_blocks(cache->dtype, cache->D, rows, &cfg, &blocks) !=
                         cudaSuccess)
        return 0;
    return attention_bytes(blocks, rows, cache->D);
}

dvl_status dvl_paged_attention(const dvl_kv_cache *cache, const void *q, int64_t q_batch_stride,
                               int64_t q_token_stride, int64_t q_head_stride, int32_t B, int32_t T,
                               int32_t Hq, const int32_t *table, int64_t table_stride,
                               int32_t table_width, const int32_t *lengths, float scale, void *out,
                               float *lse, void *ws, size_t ws_bytes, void *stream)
{
    dvl_status st = check_cache(cache);
    if (st != DVL_OK)
        return st;
    const int rows = query_rows(cache, T, Hq);
    if (rows == 0 || B < 0 || (int64_t)B * cache->heads * rows > 0x7fffffffLL)
        return DVL_ERR_INVALID_ARG;
    if (table_width < 1 || table_stride < 0 ||
        (int64_t)table_width * cache->page_size > 0x7fffffffLL - 127)  // rounding up to a tile fits
        return DVL_ERR_INVALID_ARG;
    if (!q || !aligned(q, 16) || !table || !aligned(table, 4) || !lengths || !aligned(lengths, 4) ||
        !out || !aligned(out, 16) || !aligned(lse, 4))
        return DVL_ERR_INVALID_ARG;
    if (q_batch_stride % 8 != 0 || q_token_stride % 8 != 0 || q_head_stride % 8 != 0 ||
        !std::isfinite(scale))
        return DVL_ERR_INVALID_ARG;
    attn::AttnArgs a;
    std::memset(&a, 0, sizeof a);
    attn::AttnConfig cfg;
    const cudaError_t e = attn::grid_blocks(cache->dtype, cache->D, rows, &cfg, &a.blocks);
    if (e != cudaSuccess)
        return cuda_failed(e);
    if (!ws || !aligned(ws, 16) || ws_bytes < attention_bytes(a.blocks, rows, cache->D))
        return DVL_ERR_WORKSPACE;
    if (B == 0)
        return DVL_OK;
    const int64_t half = half_bytes(cache);
    a.q = static_cast<const uint16_t *>(q);
    a.qb = q_batch_stride;
    a.qt = q_token_stride;
    a.qh = q_head_stride;
    a.k = static_cast<const unsigned char *>(cache->k);
    a.v = static_cast<const unsigned char *>(cache->v);
    a.kp = cache->k_page_stride * half / 2;
    a.kt = (uint32_t)(cache->k_token_stride * half / 2);
    a.kh = (uint32_t)(cache->k_head_stride * half / 2);
    a.vp = cache->v_page_stride * half / 2;
    a.vt = (uint32_t)(cache->v_token_stride * half / 2);
    a.vh = (uint32_t)(cache->v_head_stride * half / 2);
    if (cache->dtype == DVL_NVFP4) {
        a.kb = static_cast<const unsigned char *>(cache->k_blocks);
        a.vb = static_cast<const unsigned char *>(cache->v_blocks);
    }
    a.table = table;
    a.table_stride = table_stride;
    a.lengths = lengths;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.ws = static_cast<unsigned char *>(ws);
    a.tickets = reinterpret_cast<unsigned int *>(a.ws + kWsSlots);
    a.top_tickets = 2 * kMaxCtas;
    a.parts = reinterpret_cast<float *>(a.ws + kWsSlots + kTicketBytes);
    a.part_floats = part_floats(rows, cache->D);
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.heads = cache->heads;
    a.G = Hq / cache->heads;
    a.D = cache->D;
    a.rows = rows;
    a.token_mul = (uint32_t)((65536 + a.G - 1) / a.G);
    a.pages = cache->pages;
    a.page_size = cache->page_size;
    a.max_len = table_width * cache->page_size;
    page_division(cache->page_size, &a.page_mul, &a.page_shift);
    a.qk_scale = scale * cache->k_scale * 1.4426950408889634f;
    a.v_scale = cache->v_scale;
    return done(attn::launch_attention(a, cfg, static_cast<cudaStream_t>(stream)));
}

size_t dvl_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t N)
{
    if (!beam_sizes_ok(batch, beams, N))
        return 0;
    return kWsSlots + kTicketBytes +
           (size_t)beam_lists(batch, beams) * (kBeamKeys * sizeof(uint64_t) + sizeof(float2));
}

dvl_status dvl_beam_select(const void *logits, int32_t dtype, int64_t batch_stride,
                           int64_t beam_stride, const float *scores, int32_t batch, int32_t beams,
                           int32_t N, int32_t k, const int32_t *d2t, float *out_scores,
                           int32_t *parents, int32_t *tokens, void *ws, size_t ws_bytes,
                           void *stream)
{
    if (dtype != DVL_BF16 && dtype != DVL_F32)
        return DVL_ERR_INVALID_ARG;
    if (!beam_sizes_ok(batch, beams, N) || k < 1 || k > DVL_MAX_BEAMS)
        return DVL_ERR_INVALID_ARG;
    if (batch_stride < 0 || beam_stride < 0)
        return DVL_ERR_INVALID_ARG;
    if (!logits || !aligned(logits, dtype == DVL_F32 ? 4 : 2) || !scores || !aligned(scores, 4) ||
        !aligned(d2t, 4) || !out_scores || !aligned(out_scores, 4) || !parents ||
        !aligned(parents, 4) || !tokens || !aligned(tokens, 4))
        return DVL_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 16) || ws_bytes < dvl_beam_workspace_bytes(batch, beams, N))
        return DVL_ERR_WORKSPACE;
    if (batch == 0)
        return DVL_OK;
    for (int32_t b0 = 0; b0 < batch; b0 += kBeamRequests) {
        BeamArgs a;
        a.batch = batch - b0 < kBeamRequests ? batch - b0 : kBeamRequests;
        a.logits = static_cast<const unsigned char *>(logits) +
                   (int64_t)b0 * batch_stride * (dtype == DVL_F32 ? 4 : 2);
        a.batch_stride = batch_stride;
        a.beam_stride = beam_stride;
        a.scores = scores + (int64_t)b0 * beams;
        a.d2t = d2t;
        a.out_scores = out_scores + (int64_t)b0 * k;
        a.parents = parents + (int64_t)b0 * k;
        a.tokens = tokens + (int64_t)b0 * k;
        a.beams = beams;
        a.N = N;
        a.k = k;
        const int64_t rows = (int64_t)a.batch * beams;
        a.segments = beam_segments(rows, N);
        unsigned char *at = static_cast<unsigned char *>(ws) + kWsSlots;
        a.tickets = reinterpret_cast<unsigned int *>(at);
        a.keys = reinterpret_cast<uint64_t *>(at + kTicketBytes);
        a.sums = reinterpret_cast<float2 *>(a.keys + rows * a.segments * kBeamKeys);
        const cudaError_t e = launch_beam_select(a, dtype, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess)
            return cuda_failed(e);
    }
    return DVL_OK;
}

dvl_status dvl_beam_reorder(const dvl_state *states, int32_t n_states, const dvl_beam_pages *pages,
                            const dvl_kv_cache *cache, const int32_t *parents, int32_t batch,
                            int32_t beams, int32_t k, void *stream)
{
    if (n_states < 0 || n_states > DVL_MAX_STATES || (n_states > 0 && !states) ||
        !pages != !cache || !parents || !aligned(parents, 4))
        return DVL_ERR_INVALID_ARG;
    if (batch < 0 || beams < 1 || beams > DVL_MAX_BEAMS || k < 1 || k > DVL_MAX_BEAMS)
        return DVL_ERR_INVALID_ARG;
    ReorderArgs a;
    std::memset(&a, 0, sizeof a);
    for (int i = 0; i < n_states; ++i) {
        const dvl_state &s = states[i];
        if (!s.src || !s.dst || s.row_bytes < 1 || s.row_bytes > 0x7fffffffLL ||
            s.src_stride < s.row_bytes || s.dst_stride < s.row_bytes)
            return DVL_ERR_INVALID_ARG;
        ReorderItem &it = a.item[a.n_items++];
        it.src = static_cast<const unsigned char *>(s.src);
        it.dst = static_cast<unsigned char *>(s.dst);
        it.row_bytes = s.row_bytes;
        it.src_stride = s.src_stride;
        it.dst_stride = s.dst_stride;
    }
    if (pages) {
        const dvl_status st = check_cache(cache);
        if (st != DVL_OK)
            return st;
        if (pages->reserved != 0 || pages->width < 1 || !pages->table || !pages->table_out ||
            !pages->lengths || !pages->lengths_out || !pages->spare ||
            !aligned(pages->table, 4) || !aligned(pages->table_out, 4) ||
            !aligned(pages->lengths, 4) || !aligned(pages->lengths_out, 4) ||
            !aligned(pages->spare, 4))
            return DVL_ERR_INVALID_ARG;
        const int64_t half = half_bytes(cache);
        a.head_bytes = (int)(cache->D * half / 2);
        a.strides[0] = {cache->k_page_stride * half / 2, cache->k_token_stride * half / 2,
                        cache->k_head_stride * half / 2};
        a.strides[1] = {cache->v_page_stride * half / 2, cache->v_token_stride * half / 2,
                        cache->v_head_stride * half / 2};
        if ((int64_t)cache->page_size * cache->heads * a.head_bytes > 0x7fffffffLL ||
            (int64_t)pages->width * 4 > 0x7fffffffLL)
            return DVL_ERR_INVALID_ARG;
        a.pages = *pages;
        // (a caller's struct without the scales' pointers ends before them)
        std::memcpy(&a.cache, cache, cache->dtype == DVL_NVFP4 ? sizeof a.cache : offsetof(dvl_kv_cache, k_blocks));
        const void *src[2] = {pages->table, pages->lengths};
        void *dst[2] = {pages->table_out, pages->lengths_out};
        const int64_t bytes[2] = {4ll * pages->width, 4};
        for (int i = 0; i < 2; ++i) {
            ReorderItem &it = a.item[a.n_items++];
            it.src = static_cast<const unsigned char *>(src[i]);
            it.dst = static_cast<unsigned char *>(dst[i]);
            it.row_bytes = it.src_stride = it.dst_stride = bytes[i];
        }
    }
    a.parents = parents;
    a.batch = batch;
    a.beams = beams;
    a.k = k;
    if (batch == 0 || a.n_items == 0)
        return DVL_OK;
    // rows are copied in no order: an output meets neither an input nor another
    // output
    Rows in[DVL_MAX_STATES + 4], out[DVL_MAX_STATES + 2];
    int n_in = 0;
    for (int i = 0; i < a.n_items; ++i) {
        const ReorderItem &it = a.item[i];
        in[n_in++] = {reinterpret_cast<uintptr_t>(it.src), (int64_t)batch * beams, it.row_bytes,
                      it.src_stride};
        out[i] = {reinterpret_cast<uintptr_t>(it.dst), (int64_t)batch * k, it.row_bytes, it.dst_stride};
    }
    in[n_in++] = {reinterpret_cast<uintptr_t>(parents), 1, 4ll * batch * k, 4ll * batch * k};
    if (pages)
        in[n_in++] = {reinterpret_cast<uintptr_t>(pages->spare), 1, 4ll * batch * k, 4ll * batch * k};
    for (int i = 0; i < a.n_items; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j]))
                return DVL_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return DVL_ERR_INVALID_ARG;
    }
    return done(launch_beam_reorder(a, static_cast<cudaStream_t>(stream)));
}

dvl_status dvl_qk_norm_rope(const dvl_qk *p, void *stream)
{
    if (!p || p->rows < 0 || p->rows > 0x7fffffffLL || p->Hq < 1 || p->H < 1 || p->Hq > 65536 || p->H > 65536 ||
        p->D < 16 || p->D % 16 != 0 || p->D > DVL_MAX_HEAD_DIM || p->rot < 0 || p->rot % 16 != 0 || p->rot > p->D ||
        (p->interleaved != 0 && p->interleaved != 1) || !(p->eps >= 0.f) || !std::isfinite(p->eps))
        return DVL_ERR_INVALID_ARG;
    const HeadRows q = {p->q, p->q_stride, p->q_head_stride, p->Hq}, k = {p->k, p->k_stride, p->k_head_stride, p->H},
                   v = {p->v, p->v_stride, p->v_head_stride, p->H},
                   qo = {p->q_out, p->q_out_stride, p->q_out_head_stride, p->Hq},
                   ko = {p->k_out, p->k_out_stride, p->k_out_head_stride, p->H};
    if (!heads_ok(q, false) || !heads_ok(k, false) || !heads_ok(v, !p->cache) || !heads_ok(qo, false) ||
        !heads_ok(ko, p->cache != nullptr) || (!p->cache && p->v) || !aligned(p->q_weight, 16) ||
        !aligned(p->k_weight, 16) || !aligned(p->positions, 4) || !aligned(p->freq, 8) || (p->rot > 0 && !p->freq) ||
        (p->rot > 0 && !p->cache && !p->positions))
        return DVL_ERR_INVALID_ARG;
    const int64_t rows = p->rows;
    if (rows > 0 &&
        (!apart(qo, rows, p->D) || (ko.p && !apart(ko, rows, p->D)) ||
         (!same(qo, q, rows) && meet(qo, q, rows, p->D)) || meet(qo, k, rows, p->D) || meet(qo, v, rows, p->D) ||
         meet(qo, ko, rows, p->D) || meet(ko, q, rows, p->D) ||
         (ko.p && !same(ko, k, rows) && meet(ko, k, rows, p->D)) || meet(ko, v, rows, p->D)))
        return DVL_ERR_INVALID_ARG;
    const Written written(qo, ko, rows, p->D);
    if (written.meets(p->q_weight, 1, 2 * p->D, 0) || written.meets(p->k_weight, 1, 2 * p->D, 0) ||
        written.meets(p->freq, 1, 4 * p->rot, 0) || written.meets(p->positions, 1, 4 * rows, 0))
        return DVL_ERR_INVALID_ARG;
    QkArgs a;
    std::memset(&a, 0, sizeof a);
    a.dtype = -1;
    if (const dvl_kv_cache *c = p->cache) {
        const dvl_status st = check_cache(c);
        if (st != DVL_OK)
            return st;
        if (c->heads != p->H || c->D != p->D || p->B < 0 || !aligned(p->starts, 4) ||
            (p->B == 0 ? rows > 0 && !p->starts : !p->starts && rows % p->B != 0))
            return DVL_ERR_INVALID_ARG;
        if (p->B > 0 &&
            (p->table_width < 1 || p->table_stride < 0 ||
             (int64_t)p->table_width * c->page_size > 0x7fffffffLL || !p->table || !aligned(p->table, 4) ||
             !p->lengths || !aligned(p->lengths, 4)))
            return DVL_ERR_INVALID_ARG;
        if (written.meets(*c) || written.meets(p->table, p->B, 4ll * p->table_width, 4 * p->table_stride) ||
            written.meets(p->lengths, 1, 4ll * p->B, 0) || written.meets(p->starts, 1, 4ll * p->B + 4, 0))
            return DVL_ERR_INVALID_ARG;
        // reciprocals of the scales, and products with an E4M3 scale, stay normal numbers
        for (float s : {c->k_scale, c->v_scale})
            if (c->dtype != DVL_BF16 && !(s >= 0x1p-100f && s <= 0x1p100f))
                return DVL_ERR_INVALID_ARG;
        if (p->B == 0)
            return DVL_OK;
        const int64_t half = half_bytes(c);
        a.dtype = c->dtype;
        a.ck = static_cast<unsigned char *>(c->k);
        a.cv = static_cast<unsigned char *>(c->v);
        if (c->dtype == DVL_NVFP4) {
            a.ckb = static_cast<unsigned char *>(c->k_blocks);
            a.cvb = static_cast<unsigned char *>(c->v_blocks);
        }
        a.kp = c->k_page_stride * half / 2;
        a.kt = c->k_token_stride * half / 2;
        a.khead = c->k_head_stride * half / 2;
        a.vp = c->v_page_stride * half / 2;
        a.vt = c->v_token_stride * half / 2;
        a.vhead = c->v_head_stride * half / 2;
        a.pages = c->pages;
        a.page_size = c->page_size;
        a.width = p->table_width;
        a.B = p->B;
        a.table = p->table;
        a.table_stride = p->table_stride;
        a.lengths = p->lengths;
        a.starts = p->starts;
        a.per_sequence = p->starts ? 0 : (int)(rows / p->B);
        a.k_scale = c->k_scale;
        a.v_scale = c->v_scale;
        a.k_inv = 1.f / c->k_scale;
        a.v_inv = 1.f / c->v_scale;
    }
    if (rows == 0)
        return DVL_OK;
    a.rows = rows;
    a.Hq = p->Hq;
    a.H = p->H;
    a.D = p->D;
    a.rot = p->rot;
    a.interleaved = p->interleaved;
    a.eps = p->eps;
    a.q = static_cast<const uint16_t *>(p->q);
    a.k = static_cast<const uint16_t *>(p->k);
    a.v = static_cast<const uint16_t *>(p->v);
    a.qs = q.stride, a.qh = q.head_stride;
    a.ks = k.stride, a.kh = k.head_stride;
    a.vs = v.stride, a.vh = v.head_stride;
    a.q_weight = static_cast<const uint16_t *>(p->q_weight);
    a.k_weight = static_cast<const uint16_t *>(p->k_weight);
    a.freq = p->freq;
    a.positions = p->positions;
    a.q_out = static_cast<uint16_t *>(p->q_out);
    a.k_out = static_cast<uint16_t *>(p->k_out);
    a.qos = qo.stride, a.qoh = qo.head_stride;
    a.kos = ko.stride, a.koh = ko.head_stride;
    return done(launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

dvl_status dvl_cache_keep(const dvl_kv_cache *cache, const int32_t *table, int64_t table_stride,
                          int32_t table_width, const int32_t *lengths, const int32_t *first,
                          const int32_t *keep, int64_t keep_stride, const int32_t *counts,
                          int32_t B, int32_t M, int32_t *lengths_out, void *stream)
{
    const dvl_status st = check_cache(cache);
    if (st != DVL_OK)
        return st;
    if (B < 0 || M < 0 || M > 0x7fffffff - 65536 || table_width < 1 || table_stride < 0 || (B > 1 && keep_stride < 0) ||
        (int64_t)table_width * cache->page_size > 0x7fffffffLL || !table || !aligned(table, 4) || !lengths ||
        !aligned(lengths, 4) || !first || !aligned(first, 4) || (M > 0 && !keep) || !aligned(keep, 4) || !counts ||
        !aligned(counts, 4) || !aligned(lengths_out, 4))
        return DVL_ERR_INVALID_ARG;
    if (B == 0)
        return DVL_OK;
    if (lengths_out) {
        const Rows to = {reinterpret_cast<uintptr_t>(lengths_out), 1, 4ll * B, 4ll * B};
        auto span = [&](const int32_t *p, int64_t width, int64_t stride) {
            const int64_t n = 4 * ((B - 1) * stride + width);
            return Rows{reinterpret_cast<uintptr_t>(p), n > 0, n, n};
        };
        if (overlap(to, span(lengths, B, 0)) || overlap(to, span(first, B, 0)) || overlap(to, span(counts, B, 0)) ||
            (M > 0 && overlap(to, span(keep, M, keep_stride))) || overlap(to, span(table, table_width, table_stride)))
            return DVL_ERR_INVALID_ARG;
    }
    KeepArgs a;
    std::memset(&a, 0, sizeof a);
    const int64_t half = half_bytes(cache);
    const int row = (int)(cache->D * half / 2);  // bytes of a head of a token
    // values that are the keys themselves move with them, once
    const bool shared = cache->k == cache->v && cache->k_page_stride == cache->v_page_stride &&
                        cache->k_token_stride == cache->v_token_stride &&
                        cache->k_head_stride == cache->v_head_stride;
    for (int i = 0; i < (cache->dtype == DVL_NVFP4 ? 4 : 2); ++i) {
        const bool values = i & 1, scales = i >= 2;
        if (values && shared && (!scales || cache->k_blocks == cache->v_blocks))
            continue;
        KeepPool &p = a.pool[a.n_pools++];
        const int64_t down = scales ? 16 : 2;
        p.base = static_cast<unsigned char *>(scales ? (values ? cache->v_blocks : cache->k_blocks)
                                                     : (values ? cache->v : cache->k));
        p.page = (values ? cache->v_page_stride : cache->k_page_stride) * half / down;
        p.token = (values ? cache->v_token_stride : cache->k_token_stride) * half / down;
        p.head = (values ? cache->v_head_stride : cache->k_head_stride) * half / down;
        p.wide = !scales;
        p.units = scales ? row / 8 / 4 : row / 16;
        if ((int64_t)p.units * cache->heads > 0x7fffffffLL - 32)
            return DVL_ERR_INVALID_ARG;
        p.cols = p.units * cache->heads;
    }
    a.pages = cache->pages;
    a.page_size = cache->page_size;
    a.width = table_width;
    a.B = B;
    a.M = M;
    a.table = table;
    a.table_stride = table_stride;
    a.lengths = lengths;
    a.first = first;
    a.keep = keep;
    a.keep_stride = keep_stride;
    a.counts = counts;
    a.lengths_out = lengths_out;
    page_division(cache->page_size, &a.page_mul, &a.page_shift);
    return done(launch_cache_keep(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
