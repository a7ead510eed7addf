// evict.h -- parameters and launchers of cache eviction: which rows stay, and the
// records moved (internal).
#pragma once

#include "launch.h"

namespace psk {

struct SelectParams {
    const float* weights;
    int64_t w_stride;
    const int32_t* seq_lens;
    const int32_t* keep_lens;
    int32_t num_reqs, width;
    const int32_t* positions;  // nullable: row j is at position j
    int64_t pos_stride;
    int32_t num_first, num_recent;
    float* weights_out;        // nullable
    int64_t wo_stride;
    int32_t* positions_out;    // nullable
    int64_t po_stride;
    int2* moves;               // (from, to)
    int64_t moves_stride;      // in moves
    int32_t* num_moves;
    int32_t* seq_lens_out;
    int32_t* err;              // nullable
};

cudaError_t launch_select_evictions(const SelectParams& p, cudaStream_t stream);

struct MoveParams {
    uint8_t* cache;
    int64_t num_pages, page_stride;
    int32_t block_size, shift;     // shift: log2(block_size) or -1; set by the launcher
    int32_t data_bytes, scale_bytes;  // of a record
    const int32_t* bt;
    int64_t bt_stride;
    int32_t bt_width;
    const int32_t* base;           // nullable
    int32_t num_reqs;
    const int2* moves;
    int64_t moves_stride;
    int32_t max_moves;
    const int32_t* num_moves;
    int32_t* err;                  // nullable
};

cudaError_t launch_move_rows(MoveParams p, cudaStream_t stream);

}  // namespace psk
