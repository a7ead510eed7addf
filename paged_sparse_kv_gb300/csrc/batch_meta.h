// batch_meta.h -- parameters and launchers of the batch-metadata kernels: slot
// maps and block tables from request lengths (internal).
#pragma once

#include "launch.h"

namespace psk {

struct SlotMapTable {
    const int32_t* bt;
    int64_t stride;
    int32_t width;
    const int32_t* base;  // nullable
    int32_t block_size;
    int32_t shift;        // log2(block_size) or -1; set by the launcher
};

struct SlotMapParams {
    const int32_t* qsl;
    const int32_t* seq_lens;
    int32_t num_reqs;
    int64_t num_tokens;
    SlotMapTable main, comp;
    int32_t compress_ratio;
    int32_t ratio_shift;  // log2(compress_ratio) or -1; set by the launcher
    int64_t* positions;     // the four outputs are nullable
    int32_t* token_to_req;
    int64_t* slots;
    int64_t* comp_slots;
};

cudaError_t launch_slot_mappings(SlotMapParams p, cudaStream_t stream);

struct ExtendParams {
    const int32_t* seq_lens;
    int32_t num_reqs;
    int32_t block_size;
    int32_t compress_ratio;
    const int32_t* page_counts;  // nullable
    const int32_t* pool;
    int64_t pool_size;
    const int32_t* pool_head;    // nullable
    int32_t* bt;
    int64_t bt_stride;
    int32_t bt_width;
    int32_t* page_counts_out;
    int32_t* pool_head_out;
    int32_t* err_count;          // nullable
    int32_t rows_per_cta, ratio_shift, block_shift;  // set by the launcher
};

cudaError_t launch_extend_block_tables(ExtendParams p, cudaStream_t stream);

}  // namespace psk
