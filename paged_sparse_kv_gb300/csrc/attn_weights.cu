// attn_weights.cu -- attention weights summed per cached row over new tokens and
// heads: what eviction ranks rows by.
//
//   sum_j = sum over tokens t that see row j, heads h, of exp(s_thj - L_th)
//   s = scale q.k_j,  L = log(exp(lse) + exp(sink)),  out_j = decay w_j + sum_j
//
// A CTA takes 32 rows of a request, dequantised to binary32 in shared memory.  A warp
// takes a (token, head) at a time: 16 dims of the query a lane, one row after another.
#include "attn_weights.h"
#include "psk_common.cuh"
#include "umma.cuh"

namespace psk {
namespace {

constexpr int kRows = 32, kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(kThreads) attn_weights_kernel(const WeightParams p, const int32_t tiles) {
    extern __shared__ float s_k[];  // [row][dim]
    __shared__ float s_sum[kThreads / kWarp][kRows];
    __shared__ const uint8_t* s_data[kRows];
    __shared__ const uint8_t* s_scale[kRows];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const int32_t r = (int32_t)(blockIdx.x / tiles), first = (int32_t)(blockIdx.x % tiles) * kRows;
    const int32_t rows = p.seq_lens[r], end = min(rows, p.width);
    if (first >= end) return;
    const int D = p.head_dim, nope = D - p.rope_dim;
    if (tid < kRows) {
        const int32_t j = first + tid;
        s_data[tid] = nullptr;
        if (j < end) {
            int32_t off;
            const int64_t logical =
                (int64_t)div_block32(j, p.cache.block_size, p.cache.shift, off) - (p.base_off ? p.base_off[r] : 0);
            if (logical >= 0 && logical < p.bt_width) {
                const int32_t page = p.bt[(int64_t)r * p.bt_stride + logical];
                if (page >= 0 && page < p.cache.num_pages) {
                    const uint8_t* pg = p.cache.base + (int64_t)page * p.cache.page_stride;
                    s_data[tid] = pg + (int64_t)off * (D + p.rope_dim);
                    s_scale[tid] = pg + (int64_t)p.cache.block_size * (D + p.rope_dim) + (int64_t)off * (D / 64);
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kThreads) {
        const int row = i / D, d = i % D;
        float x = 0.0f;
        if (s_data[row] != nullptr) {
            if (d < nope) {
                const float v = f16_lo(cvt_e4m3x2_to_f16x2(s_data[row][d]));
                x = bf16_lo(pack_bf16x2(v * ue8m0_scale(s_scale[row][d / 64]), 0.0f));
            } else {
                x = bf16_lo(*reinterpret_cast<const uint16_t*>(s_data[row] + nope + 2 * (d - nope)));
            }
        }
        s_k[i] = x;
    }
    __syncthreads();
    const bool there = s_data[lane] != nullptr;
    const int64_t q0 = p.qsl[r], q1 = min((int64_t)p.qsl[r + 1], p.num_tokens);
    const int64_t at0 = (int64_t)rows - ((int64_t)p.qsl[r + 1] - q0);  // row of token q0
    const float c = p.scale * kLog2e;
    const int32_t j = first + lane;
    float sum = 0.0f, low = 0.0f;  // Kahan's compensation in `low`
    for (int64_t t = max(q0, (int64_t)0) ; t < q1; ++t) {
        const int64_t pos = at0 + (t - q0);
        if (pos < first || (p.valid && !p.valid[t])) continue;
        int64_t from = p.window > 0 ? pos - p.window + 1 : 0;
        if (p.replay) from = max(from, (int64_t)p.replay[r]);
        if (from >= first + kRows) continue;
        const bool sees = there && j <= pos && j >= from;
        for (int h = warp; h < p.num_heads; h += kThreads / kWarp) {
            const float a = p.lse[t * p.lse_stride_t + h] * kLog2e, b = p.sink ? p.sink[h] * kLog2e : -INFINITY;
            const float top = fmaxf(a, b);
            if (top == -INFINITY && !(a != a) && !(b != b)) continue;  // a token that saw nothing
            const float L = a != a || b != b ? NAN : isinf(top) ? top : top + log2f(1.0f + exp2f(-fabsf(a - b)));
            const uint16_t* q = p.q + t * p.q_stride_t + h * p.q_stride_h;
            float mine = 0.0f;
            for (int row = 0; row < kRows; ++row) {
                float s = 0.0f;
                for (int d = lane; d < D; d += kWarp) s = fmaf(bf16_lo(q[d]), s_k[row * D + d], s);
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                if (row == lane) mine = s;
            }
            const float w = sees ? exp2f(fmaf(mine, c, -L)) : 0.0f;
            const float y = w - low, z = sum + y;
            low = isfinite(z) ? (z - sum) - y : 0.0f;
            sum = z;
        }
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && j < end) {
        float all = 0.0f;
        for (int i = 0; i < kThreads / kWarp; ++i) all += s_sum[i][lane];
        float* out = p.out + (int64_t)r * p.out_stride + j;
        *out = p.decay == 0.0f ? all : fmaf(p.decay, p.weights[(int64_t)r * p.w_stride + j], all);
    }
    pdl_launch_dependents();
}

}  // namespace

int64_t attn_weights_workspace_bytes() { return 0; }

cudaError_t launch_attn_weights(WeightParams p, cudaStream_t stream) {
    p.cache.shift = log2_if_pow2(p.cache.block_size);
    const int32_t tiles = p.width / kRows + (p.width % kRows != 0);
    const int smem = kRows * p.head_dim * (int)sizeof(float);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_limit_per_device(attn_weights_kernel, kRows * 512 * (int)sizeof(float), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_weights_kernel, dim3((unsigned)((int64_t)tiles * p.num_reqs)), dim3(kThreads), smem, stream, p,
                      tiles);
}

}  // namespace psk
