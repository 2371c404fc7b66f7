// Host-side declarations of the drafting step's operators (norms, attention,
// beam selection and reordering, kept tokens), shared by their argument checks
// and their kernel files.
#pragma once

#include "dvl_internal.h"

namespace dvl {

// Residual addition and norm; the arguments are dvl_norm's, checked.
cudaError_t launch_add_rmsnorm(const dvl_norm &a, cudaStream_t s);

// Beam selection.  A row of logits is cut into segments, each leaving its best
// keys and its part of the row's sum of exponentials.
constexpr int kBeamKeys = 32;    // keys per segment list (>= DVL_MAX_BEAMS)
constexpr int kBeamLists = 608;  // blocks the segments are cut for: four per SM
struct BeamArgs {
    const void *logits;
    int64_t batch_stride, beam_stride;  // elements
    const float *scores;                // [batch][beams]
    const int32_t *d2t;                 // [N] or nullptr
    float *out_scores;                  // [batch][k]
    int32_t *parents, *tokens;          // [batch][k]
    int batch, beams, N, k;
    int segments, length;               // per row; logits of one
    unsigned int *tickets;              // [batch]
    uint64_t *keys;                     // [batch * beams][segments][kBeamKeys]
    float2 *sums;                       // [batch * beams][segments]: maximum, sum
};
int beam_segments(int64_t rows, int N);
cudaError_t launch_beam_select(BeamArgs &a, int dtype, cudaStream_t s);

// Reordering: every copied row is cut into pieces of at most kPiece bytes,
// one thread block each.
struct ReorderItem {
    const unsigned char *src;
    unsigned char *dst;
    int64_t row_bytes, src_stride, dst_stride;
    int pieces;                         // per row
    int wide;                           // 16-byte accesses
    int64_t first_block;
};
struct ReorderArgs {
    ReorderItem item[DVL_MAX_STATES + 2];  // the states, then table and lengths
    int n_items;
    int64_t copy_blocks;                // blocks of the items
    const int32_t *parents;             // [batch][k]
    int batch, beams, k;
    // the partly filled pages (pages.table == nullptr: none)
    dvl_beam_pages pages;
    dvl_kv_cache cache;
    struct {
        int64_t page, token, head;
    } strides[2];                       // of keys and values, in bytes
    int head_bytes;                     // of one head of one token
    int page_pieces, block_pieces;      // per new beam, keys and values each: of the
                                        // rows, of an NVFP4 cache's scales
};
cudaError_t launch_beam_reorder(ReorderArgs &a, cudaStream_t s);

// Norm and rotation of queries and keys, and the cache's new rows: dvl_qk's
// arguments, checked, strides of tensors in elements, of the cache in bytes.
struct QkArgs {
    int64_t rows;
    int Hq, H, D, rot, interleaved;
    float eps;
    const uint16_t *q, *k, *v;
    int64_t qs, qh, ks, kh, vs, vh;     // row, head
    const uint16_t *q_weight, *k_weight;
    const uint64_t *freq;
    const int32_t *positions;
    uint16_t *q_out, *k_out;
    int64_t qos, qoh, kos, koh;
    // the cache; dtype -1: none
    int dtype;
    unsigned char *ck, *cv, *ckb, *cvb; // pools, NVFP4 scales
    int64_t kp, kt, khead, vp, vt, vhead;
    int pages, page_size, width, B;
    const int32_t *table, *lengths, *starts;
    int64_t table_stride;
    int per_sequence;                   // rows of each without starts
    float k_scale, v_scale, k_inv, v_inv;
    int parts;                          // warps that share a row
};
cudaError_t launch_qk_norm_rope(QkArgs &a, cudaStream_t s);

// Kept tokens.  A token of a pool is `cols` columns of 16 bytes (wide) or 4.
struct KeepPool {
    unsigned char *base;
    int64_t page, token, head;          // strides in bytes
    int units, cols;                    // columns per head, per token
    int wide;
    int first_block;
};
struct KeepArgs {
    KeepPool pool[4];                   // keys, values, their NVFP4 scales
    int n_pools;
    int pages, page_size, width, B, M;
    const int32_t *table, *lengths, *first, *keep, *counts;
    int64_t table_stride, keep_stride;
    int32_t *lengths_out;
    uint32_t page_mul;                  // pos / page_size = pos * page_mul >> page_shift
    int page_shift;
    int blocks;                         // per sequence
};
cudaError_t launch_cache_keep(KeepArgs &a, cudaStream_t s);

}  // namespace dvl
