// rotary.h -- parameters and launchers of the rotary-position kernels (internal).
#pragma once

#include "launch.h"

namespace psk {

constexpr int kMaxTablePairs = 256;  // rope_dim up to 512
constexpr int32_t kMostRotaryHeads = 0x7FFFFFFF - (1 << 20);  // of queries and keys together

struct RopeTableParams {
    float* out;
    int64_t stride;
    int64_t first_pos, num_pos;
    int32_t pairs;
    float factor;                   // multiplies every value
    uint64_t turn[kMaxTablePairs];  // 2^64 times the fraction of a turn a position adds
};

cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream);

struct RotaryTensor {
    const uint8_t* in;
    uint8_t* out;
    int64_t in_stride_t, in_stride_h, out_stride_t, out_stride_h;  // bytes
};

struct RotaryParams {
    RotaryTensor q, k;
    int32_t heads, all_heads;  // of q; of both
    int64_t num_tokens;
    int32_t dtype;             // psk_dtype
    int32_t head_dim, offset, rope_dim;
    int32_t half, inverse;
    int32_t copy_q, copy_k;    // not in place: what is not rotated is copied
    const int64_t* positions;
    const float* cos_sin;
    int64_t cs_stride, max_pos;
    int32_t* err;              // nullable
};

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream);

}  // namespace psk
