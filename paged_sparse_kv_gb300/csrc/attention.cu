// attention.cu -- attention over the rows of paged fp8_ds_mla caches.
//
// For a token and a head with query q and visible rows k_j (each row is key and
// value at once):
//   s_j = scale * q.k_j,  m = max_j s_j,  p_j = exp(s_j - m),  l = sum_j p_j
//   out = sum_j p_j k_j / (l + exp(sink - m)),  lse = m + log(l)
// in one pass with a running maximum: when m grows, l and the weighted sum are
// multiplied by exp(m_old - m_new).
#include "attention.h"
#include "psk_common.cuh"

namespace psk {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPerLane = 16;  // head_dim 512 / 32 lanes

// One warp per (token, head); lane i holds dims i, i + 32, ...
template <bool kIndexed>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttnParams p) {
    pdl_wait();
    const int lane = threadIdx.x % kWarp;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / kWarp) + threadIdx.x / kWarp;
    if (unit >= p.num_tokens * p.num_heads) return;
    const int64_t t = unit / p.num_heads;
    const int32_t h = (int32_t)(unit % p.num_heads);
    const int32_t D = p.head_dim, nope = D - p.rope_dim, per = D / kWarp;

    float q[kMaxPerLane], acc[kMaxPerLane];
    for (int i = 0; i < per; ++i) {
        q[i] = __uint_as_float((uint32_t)p.q[t * p.q_stride_t + h * p.q_stride_h + lane + 32 * i] << 16);
        acc[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;

    int64_t n = p.cols, lo = 0;
    int32_t r = 0;
    if (!kIndexed) {
        r = p.t2r[t];
        n = 0;
        if (r >= 0 && r < p.num_reqs && (!p.valid || p.valid[t])) {
            const int64_t pos = (int64_t)p.seq_lens[r] - ((int64_t)p.qsl[r + 1] - p.qsl[r]) +
                                (t - p.qsl[r]);
            if (p.window > 0) lo = pos - p.window + 1;
            if (p.replay && p.replay[r] > lo) lo = p.replay[r];
            if (lo < 0) lo = 0;
            n = pos + 1 > lo ? pos + 1 - lo : 0;
        }
    }
    for (int64_t j = 0; j < n; ++j) {
        const AttnCache& c = kIndexed && j >= p.split ? p.extra : p.cache;
        int64_t page, off;
        if (kIndexed) {
            const int32_t s = p.idx[t * p.idx_stride + j];
            if (s < 0 || s >= c.num_pages * c.block_size) continue;
            page = s / c.block_size;
            off = s % c.block_size;
        } else {
            const int64_t logical = (lo + j) / c.block_size - (p.base_off ? p.base_off[r] : 0);
            off = (lo + j) % c.block_size;
            if (logical < 0 || logical >= p.bt_width) continue;
            page = p.bt[(int64_t)r * p.bt_stride + logical];
            if (page < 0 || page >= c.num_pages) continue;
        }
        const uint8_t* pg = c.base + page * c.page_stride;
        const uint8_t* row = pg + off * (nope + 2 * p.rope_dim);
        const uint8_t* sc = pg + (int64_t)c.block_size * (nope + 2 * p.rope_dim) + off * (D / 64);
        float k[kMaxPerLane], s = 0.0f;
        for (int i = 0; i < per; ++i) {
            const int d = lane + 32 * i;
            if (d < nope) {
                const float x = f16_lo(cvt_e4m3x2_to_f16x2(row[d])) * ue8m0_scale(sc[d / 64]);
                k[i] = bf16_lo(pack_bf16x2(x, 0.0f));
            } else {
                const uint8_t* b = row + nope + 2 * (d - nope);
                k[i] = __uint_as_float((uint32_t)b[0] << 16 | (uint32_t)b[1] << 24);
            }
            s = fmaf(q[i], k[i], s);
        }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        s *= p.scale;
        const float mn = s > m || s != s ? s : m;
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float a = expf(m - ref), e = expf(s - ref);
        l = l * a + e;
        for (int i = 0; i < per; ++i) acc[i] = acc[i] * a + e * k[i];
        m = mn;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    const float total = l + (p.sink ? expf(p.sink[h] - ref) : 0.0f);
    const float inv = l == 0.0f ? 0.0f : 1.0f / total;
    for (int i = 0; i < per; ++i)
        p.out[t * p.out_stride_t + h * p.out_stride_h + lane + 32 * i] =
            (uint16_t)pack_bf16x2(acc[i] * inv, 0.0f);
    if (p.lse && lane == 0) p.lse[t * p.lse_stride_t + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <bool kIndexed>
cudaError_t launch(const AttnParams& p, cudaStream_t stream) {
    const int64_t units = p.num_tokens * p.num_heads;
    const int64_t ctas = (units + kThreads / kWarp - 1) / (kThreads / kWarp);
    return launch_pdl(attention_kernel<kIndexed>, dim3((unsigned)ctas), dim3(kThreads), 0, stream, p);
}

}  // namespace

int64_t attention_workspace_bytes(int64_t, int32_t, int32_t, int64_t) { return 0; }

cudaError_t launch_attention_indexed(AttnParams p, cudaStream_t stream) {
    return launch<true>(p, stream);
}

cudaError_t launch_attention_chunk(AttnParams p, cudaStream_t stream) {
    return launch<false>(p, stream);
}

}  // namespace psk
