// attn_weights.h -- parameters and launcher of the accumulation of attention
// weights per cached row (internal).
#pragma once

#include "attention.h"

namespace psk {

struct WeightParams {
    const uint16_t* q;
    int64_t q_stride_t, q_stride_h;
    int64_t num_tokens;
    int32_t num_heads, head_dim, rope_dim;
    const float* lse;
    int64_t lse_stride_t;
    const float* sink;        // nullable
    float scale;
    AttnCache cache;
    const int32_t* qsl;
    const int32_t* seq_lens;
    const int32_t* replay;    // nullable
    const uint8_t* valid;     // nullable
    int32_t num_reqs;
    const int32_t* bt;
    int64_t bt_stride;
    int32_t bt_width;
    const int32_t* base_off;  // nullable
    int32_t window;           // 0: the whole context
    const float* weights;     // may be null where decay is 0
    int64_t w_stride;
    int32_t width;
    float decay;
    float* out;               // may be `weights`
    int64_t out_stride;
    void* workspace;
};

// Bytes of workspace a call needs on the current device.
int64_t attn_weights_workspace_bytes();

cudaError_t launch_attn_weights(WeightParams p, cudaStream_t stream);

// Count of expired bounded waits in the kernel.
cudaError_t read_attn_weights_wait_timeouts(uint32_t* count);

}  // namespace psk
