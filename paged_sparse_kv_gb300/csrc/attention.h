// attention.h -- parameters and launchers of the attention kernels over paged
// fp8_ds_mla caches (internal).
#pragma once

#include "launch.h"

namespace psk {

struct AttnCache {
    const uint8_t* base;
    int64_t num_pages;
    int64_t page_stride;
    int32_t block_size;
    int32_t shift;  // log2(block_size) or -1; set by the launcher
};

struct AttnParams {
    const uint16_t* q;
    int64_t q_stride_t, q_stride_h;
    int64_t num_tokens;
    int32_t num_heads;
    int32_t head_dim, rope_dim;
    AttnCache cache;
    float scale;
    const float* sink;  // nullable
    uint16_t* out;
    int64_t out_stride_t, out_stride_h;
    float* lse;  // nullable
    int64_t lse_stride_t;
    void* workspace;

    // index form: columns [0, split) name slots of `cache`, the others of `extra`
    AttnCache extra;
    const int32_t* idx;
    int64_t idx_stride;
    int32_t cols, split;

    // position form: the visible positions of a token through its block table
    const int32_t* qsl;
    const int32_t* seq_lens;
    const int32_t* t2r;
    const int32_t* replay;  // nullable
    const uint8_t* valid;   // nullable
    int32_t num_reqs;
    const int32_t* bt;
    int64_t bt_stride;
    int32_t bt_width;
    const int32_t* base_off;  // nullable
    int32_t window;           // 0: the whole context
};

// Bytes of workspace a call of these sizes needs on the current device; max_keys
// is the largest number of rows one token can see.
int64_t attention_workspace_bytes(int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                                  int64_t max_keys, bool indexed, int32_t num_reqs);

cudaError_t launch_attention_indexed(AttnParams p, cudaStream_t stream);
cudaError_t launch_attention_chunk(AttnParams p, cudaStream_t stream);

// Count of expired bounded waits in the attention kernels.
cudaError_t read_attention_wait_timeouts(uint32_t* count);

}  // namespace psk
