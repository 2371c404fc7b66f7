// Host-side declarations of the drafting step's operators (norm, attention,
// beam selection and reordering), shared by their argument checks and their
// kernel files.
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
    int elem;                           // bytes per cached value
    int page_pieces;                    // per new beam, keys and values each
};
cudaError_t launch_beam_reorder(ReorderArgs &a, cudaStream_t s);

}  // namespace dvl
