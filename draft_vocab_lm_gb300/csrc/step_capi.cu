// The C ABI of the drafting step's operators: argument checks and dispatch.
// Every check runs on the host before anything is enqueued; nothing here
// allocates, frees or synchronizes.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

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
    if (!c || (c->dtype != DVL_BF16 && c->dtype != DVL_FP8) || c->reserved != 0)
        return DVL_ERR_INVALID_ARG;
    if (c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->D < 16 || c->D % 16 != 0 ||
        c->D > DVL_MAX_HEAD_DIM)
        return DVL_ERR_INVALID_ARG;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
        return DVL_ERR_INVALID_ARG;
    const int64_t unit = c->dtype == DVL_BF16 ? 8 : 16;  // elements in 16 bytes
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
    if (rows == 0 || attn::grid_blocks(cache->dtype == DVL_FP8, cache->D, rows, &cfg, &blocks) !=
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
    const bool fp8 = cache->dtype == DVL_FP8;
    attn::AttnArgs a;
    std::memset(&a, 0, sizeof a);
    attn::AttnConfig cfg;
    const cudaError_t e = attn::grid_blocks(fp8, cache->D, rows, &cfg, &a.blocks);
    if (e != cudaSuccess)
        return cuda_failed(e);
    if (!ws || !aligned(ws, 16) || ws_bytes < attention_bytes(a.blocks, rows, cache->D))
        return DVL_ERR_WORKSPACE;
    if (B == 0)
        return DVL_OK;
    const int64_t size = fp8 ? 1 : 2;
    a.q = static_cast<const uint16_t *>(q);
    a.qb = q_batch_stride;
    a.qt = q_token_stride;
    a.qh = q_head_stride;
    a.k = static_cast<const unsigned char *>(cache->k);
    a.v = static_cast<const unsigned char *>(cache->v);
    a.kp = cache->k_page_stride * size;
    a.kt = (uint32_t)(cache->k_token_stride * size);
    a.kh = (uint32_t)(cache->k_head_stride * size);
    a.vp = cache->v_page_stride * size;
    a.vt = (uint32_t)(cache->v_token_stride * size);
    a.vh = (uint32_t)(cache->v_head_stride * size);
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
    // pos / page_size for 0 <= pos < 2^31: multiply by 2^(31 + s) / page_size
    // rounded up, s = ceil(log2 page_size); the error stays below one unit
    int s = 0;
    while ((1ll << s) < cache->page_size)
        ++s;
    a.page_shift = 31 + s;
    a.page_mul = (uint32_t)((1ull << a.page_shift) / (uint64_t)cache->page_size + 1);
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
        a.elem = cache->dtype == DVL_FP8 ? 1 : 2;
        if ((int64_t)cache->page_size * cache->heads * cache->D * a.elem > 0x7fffffffLL ||
            (int64_t)pages->width * 4 > 0x7fffffffLL)
            return DVL_ERR_INVALID_ARG;
        a.pages = *pages;
        a.cache = *cache;
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

}  // extern "C"
