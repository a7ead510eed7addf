// attention.cu -- attention over the rows of paged fp8_ds_mla caches on the
// 5th-generation tensor cores.
//
// For a token and a head with query q and visible rows k_j (each row is key and
// value at once):
//   s_j = scale * q.k_j,  m = max_j s_j,  p_j = exp(s_j - m),  l = sum_j p_j
//   out = sum_j p_j k_j / (l + exp(sink - m)),  lse = m + log(l)
//
// Layout.  All heads of a token share its rows, so the work of a CTA is one
// token with up to 64 heads (a "unit"; a small head count takes several
// neighbouring tokens of one request), walked in tiles of 128 rows:
//   S^T [128 rows x N columns]  = K [128 x D] Q^T         (D/16 MMAs of M = 128)
//   O^T [D x N]                += K^T [D x 128] P^T       (D/128 x 8 MMAs)
// A column is one (token, head).  Rows on the M side let every head count use
// full 128-row MMAs and keep O^T for head_dim 512 in 4 * 64 of the 512 columns
// of tensor memory, which the untransposed form (128 heads x 512 dims) would
// fill alone.  K is dequantised once per tile into one 128-byte-swizzled bf16
// tile that both products read: with the dims contiguous as the K-major A
// operand of the first, as the M-major A operand of the second.
//
// Roles.  16 worker warps dequantise a tile, take the softmax of S^T and at the
// end of a unit write O^T; one thread issues the MMAs; one warp looks one unit
// ahead (which tiles hold anything visible, which tokens and positions).  The
// tile is handed over in chunks of 64 dims: the first product follows the
// dequantisation chunk by chunk, and the next tile is dequantised into the
// chunks the second product has finished with.  Every wait is bounded (2 s of
// wall time, counted in psk_device_wait_timeouts).
//
// Softmax in one pass: a running reference m per column.  It follows the
// maximum lazily, only when a tile's maximum lies more than 2^8 above it, so
// that O^T is rescaled on few tiles and a weight is at most 2^8; the reference
// cancels in out and in lse.  Sums and weights are binary32; the weights are
// rounded to bf16 for the second product alone (the operands of one MMA share a
// type, and a row's bf16 values do not fit fp16's range), while l sums them
// unrounded, so that lse keeps binary32 accuracy and the roundings in out, being
// unbiased, average out.
#include <atomic>
#include <cmath>

#include "attention.h"
#include "psk_common.cuh"
#include "umma.cuh"

namespace psk {
namespace {

constexpr int kTile = 128;            // rows of a tile (M of the first product)
constexpr int kWorkers = 16;          // worker warps
constexpr int kMmaWarp = kWorkers;
constexpr int kPlanWarp = kWorkers + 1;
constexpr int kThreads = (kWorkers + 2) * kWarp;
constexpr int kMaxChunks = 8;         // 64-dim chunks of a row (head_dim 512)
constexpr int kChunkBytes = kTile * 128;
constexpr int kMaxCols = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;         // log2 units the maximum may run ahead of the reference
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ unsigned int g_attn_wait_timeouts = 0;

enum { kIndexed = 0, kOneToken = 1, kTokens = 2 };

// What a CTA does next: a set of tiles for a set of columns.
struct Unit {
    int32_t done;
    int32_t ntiles;
    int32_t first;        // the tiles are first, first + 1, ... where mask is 0
    int32_t part;         // which part of the split work (row of the workspace)
    uint64_t mask;        // index form with at most 64 tiles: those with a visible row
    int32_t lo, hi;       // position form: the positions of all columns
    int32_t req;
    int32_t pad;
    int32_t col_token[kMaxCols];  // -1: column not in use
    int32_t col_head[kMaxCols];
    int32_t col_lo[kMaxCols], col_hi[kMaxCols];  // kTokens: positions a column sees
};

struct Shared {
    Unit unit[2];
    uint64_t unit_full[2], unit_empty[2];
    uint64_t full[kMaxChunks];         // chunk c of the tile is dequantised
    uint64_t freed[kMaxChunks / 2];    // the second product is done with chunks 2j, 2j + 1
    uint64_t s_ready, p_ready, drain;
    uint64_t group_bar[4];
    uint32_t tmem;
    uint8_t row_ok[2][kTile];          // the row exists (and is visible where one token is at work)
    uint8_t row_bad[2][kTile];         // kTokens: it holds a NaN or an infinity
    alignas(16) float red[4][2][4][16];  // [group][exchange parity][lane quarter][column]
    alignas(16) float ref[kWorkers][16];
    alignas(16) float aux[kWorkers][16];
};

struct LaunchShape {
    int32_t heads_per_unit;  // heads of one token in a unit
    int32_t head_groups;     // ceil(num_heads / heads_per_unit)
    int32_t tokens_per_unit; // kTokens: neighbouring tokens in a unit
    int32_t splits;
    int64_t units;
    uint32_t tmem_cols;
    float scale_log2;
    float* part_o;           // [token][head][split][D]
    float* part_ml;          // [token][head][split][2]
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait_bounded(bar, parity, kWaitLimitNs);
    return __all_sync(0xFFFFFFFFu, ok);
}

// ---- the planning warp -------------------------------------------------------------

struct TokenRange {
    int32_t req, lo, hi;  // req < 0: a padding token; lo > hi: sees nothing
};

__device__ __forceinline__ TokenRange token_range(const AttnParams& p, int64_t t) {
    TokenRange x{-1, 0, -1};
    const int32_t r = p.t2r[t];
    if (r < 0 || r >= p.num_reqs || (p.valid && !p.valid[t])) return x;
    x.req = r;
    const int64_t q0 = p.qsl[r], q1 = p.qsl[r + 1];
    const int64_t pos = (int64_t)p.seq_lens[r] - (q1 - q0) + (t - q0);
    int64_t lo = p.window > 0 ? pos - p.window + 1 : 0;
    if (p.replay) lo = max(lo, (int64_t)p.replay[r]);
    // no further than the table reaches: positions outside it have no page
    const int64_t first = p.base_off ? (int64_t)p.base_off[r] * p.cache.block_size : 0;
    const int64_t last = first + (int64_t)p.bt_width * p.cache.block_size - 1;
    lo = max(lo, max(first, (int64_t)0));
    const int64_t hi = min(min(pos, last), (int64_t)INT32_MAX - kTile);
    if (lo <= hi) {
        x.lo = (int32_t)lo;
        x.hi = (int32_t)hi;
    }
    return x;
}

__device__ __forceinline__ bool slot_ok(const AttnParams& p, int32_t col, int32_t slot) {
    const AttnCache& c = col < p.split ? p.cache : p.extra;
    return slot >= 0 && slot < c.num_pages * c.block_size;
}

// Even share `part` of n tiles: [first, first + count).
__device__ __forceinline__ void share(int32_t n, int32_t part, int32_t parts, int32_t& first,
                                      int32_t& count) {
    first = (int32_t)((int64_t)n * part / parts);
    count = (int32_t)((int64_t)n * (part + 1) / parts) - first;
}

// Waits for the slot of unit `seq`, which two units before it have used.
__device__ __forceinline__ bool unit_slot(Shared& sh, int seq) {
    return seq < 2 || wait_all(&sh.unit_empty[seq & 1], ((seq >> 1) - 1) & 1);
}

__device__ __forceinline__ void unit_publish(Shared& sh, int seq, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.unit_full[seq & 1]);
}

template <int kSrc>
__device__ bool plan(const AttnParams& p, const LaunchShape& ls, Shared& sh) {
    const int lane = threadIdx.x % kWarp;
    int seq = 0;
    for (int64_t u = blockIdx.x; u < ls.units; u += gridDim.x) {
        const int32_t part = (int32_t)(u % ls.splits);
        const int64_t v = u / ls.splits;
        if (kSrc != kTokens) {
            const int64_t t = v / ls.head_groups;
            const int32_t h0 = (int32_t)(v % ls.head_groups) * ls.heads_per_unit;
            const int32_t heads = min(ls.heads_per_unit, p.num_heads - h0);
            uint64_t mask = 0;
            int32_t first = 0, count = 0;
            TokenRange x{0, 0, -1};
            if (kSrc == kIndexed) {
                const int32_t n = p.cols / kTile + (p.cols % kTile != 0);
                if (n <= 64) {
                    const int32_t* row = p.idx + t * p.idx_stride;
                    for (int32_t i = 0; i < n; ++i) {
                        bool any = false;
#pragma unroll
                        for (int j = 0; j < kTile / kWarp; ++j) {
                            const int32_t c = i * kTile + j * kWarp + lane;
                            if (c < p.cols) any |= slot_ok(p, c, row[c]);
                        }
                        if (__any_sync(0xFFFFFFFFu, any)) mask |= 1ull << i;
                    }
                    share(__popcll(mask), part, ls.splits, first, count);
                    for (int32_t k = 0; k < first; ++k) mask &= mask - 1;
                    uint64_t rest = mask;
                    for (int32_t k = 0; k < count; ++k) rest &= rest - 1;
                    mask ^= rest;
                } else {
                    share(n, part, ls.splits, first, count);
                }
            } else {
                x = token_range(p, t);
                const int32_t n = x.hi < x.lo ? 0 : (int32_t)(((int64_t)x.hi - x.lo) / kTile) + 1;
                share(n, part, ls.splits, first, count);
            }
            if (!unit_slot(sh, seq)) return false;
            Unit& un = sh.unit[seq & 1];
            if (lane == 0) {
                un.done = 0;
                un.ntiles = count;
                un.first = first;
                un.part = part;
                un.mask = mask;
                un.lo = x.lo;
                un.hi = x.hi;
                un.req = x.req;
            }
#pragma unroll
            for (int k = 0; k < kMaxCols / kWarp; ++k) {
                const int c = lane + k * kWarp;
                un.col_token[c] = c < heads ? (int32_t)t : -1;
                un.col_head[c] = h0 + c;
            }
            unit_publish(sh, seq, lane);
            ++seq;
        } else {
            // a run of neighbouring tokens of one request is a unit
            const int64_t t0 = v * ls.tokens_per_unit;
            const int32_t n = (int32_t)min((int64_t)ls.tokens_per_unit, p.num_tokens - t0);
            TokenRange x{-2, 0, -1};
            if (lane < n) x = token_range(p, t0 + lane);
            const int32_t before = __shfl_up_sync(0xFFFFFFFFu, x.req, 1);
            uint32_t starts = __ballot_sync(0xFFFFFFFFu, lane < n && (lane == 0 || x.req != before));
            while (starts) {
                const int32_t a = __ffs(starts) - 1;
                starts &= starts - 1;
                const int32_t b = starts ? __ffs(starts) - 1 : n;
                const bool in = lane >= a && lane < b && x.lo <= x.hi;
                const int32_t lo = __reduce_min_sync(0xFFFFFFFFu, in ? x.lo : INT32_MAX);
                const int32_t hi = __reduce_max_sync(0xFFFFFFFFu, in ? x.hi : -1);
                const int32_t tiles = hi < lo ? 0 : (int32_t)(((int64_t)hi - lo) / kTile) + 1;
                int32_t first, count;
                share(tiles, part, ls.splits, first, count);
                if (!unit_slot(sh, seq)) return false;
                Unit& un = sh.unit[seq & 1];
                const int32_t req = __shfl_sync(0xFFFFFFFFu, x.req, a);
                if (lane == 0) {
                    un.done = 0;
                    un.ntiles = count;
                    un.first = first;
                    un.part = part;
                    un.mask = 0;
                    un.lo = lo;
                    un.hi = hi;
                    un.req = req;
                }
#pragma unroll
                for (int k = 0; k < kMaxCols / kWarp; ++k) {
                    const int c = lane + k * kWarp;
                    const int tok = a + c / p.num_heads;
                    const bool used = tok < b;
                    const int32_t clo = __shfl_sync(0xFFFFFFFFu, x.lo, tok & 31);
                    const int32_t chi = __shfl_sync(0xFFFFFFFFu, x.hi, tok & 31);
                    un.col_token[c] = used ? (int32_t)(t0 + tok) : -1;
                    un.col_head[c] = c % p.num_heads;
                    un.col_lo[c] = used ? clo : 0;
                    un.col_hi[c] = used ? chi : -1;
                }
                unit_publish(sh, seq, lane);
                ++seq;
            }
        }
    }
    if (!unit_slot(sh, seq)) return false;
    if (lane == 0) sh.unit[seq & 1].done = 1;
    unit_publish(sh, seq, lane);
    return true;
}

// ---- the MMA thread ------------------------------------------------------------------

template <int N>
__device__ bool issue(const AttnParams& p, Shared& sh, uint32_t k_tile, uint32_t q_tile,
                      uint32_t p_tile, uint32_t tmem) {
    const int chunks = p.head_dim / 64, blocks = p.head_dim / 128;
    constexpr uint32_t kFirst = umma_idesc(kTile, N, false), kSecond = umma_idesc(128, N, true);
    uint32_t step = 0;
    for (int seq = 0;; ++seq) {
        if (!mbar_wait_bounded(&sh.unit_full[seq & 1], (seq >> 1) & 1, kWaitLimitNs)) return false;
        const Unit& un = sh.unit[seq & 1];
        const int32_t done = un.done, ntiles = un.ntiles;
        mbar_arrive(&sh.unit_empty[seq & 1]);
        if (done) return true;
        for (int32_t i = 0; i < ntiles; ++i, ++step) {
            for (int c = 0; c < chunks; ++c) {
                if (!mbar_wait_bounded(&sh.full[c], step & 1, kWaitLimitNs)) return false;
                tmem_fence_after();
                // K-major, 128-byte swizzle: 8-row groups 1024 bytes apart, 32 bytes a step
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_bf16(tmem, umma_desc(k_tile + c * kChunkBytes + k * 32, 16, 1024, kSwizzle128),
                              umma_desc(q_tile + c * (N * 128) + k * 32, 16, 1024, kSwizzle128), kFirst,
                              c > 0 || k > 0);
            }
            umma_commit(&sh.s_ready);
            if (!mbar_wait_bounded(&sh.p_ready, step & 1, kWaitLimitNs)) return false;
            tmem_fence_after();
            for (int j = 0; j < blocks; ++j) {
                // A: M-major, 128-byte swizzle: 64-dim chunks kChunkBytes apart, 8-row groups
                // 1024 bytes apart.  B: N-major, no swizzle: 8-column groups 2048 bytes
                // apart, 8-row groups 128 bytes apart.
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    umma_bf16(tmem + N + j * N,
                              umma_desc(k_tile + j * 2 * kChunkBytes + k * 2048, kChunkBytes, 1024,
                                        kSwizzle128),
                              umma_desc(p_tile + k * 256, 128, 2048, kSwizzleNone), kSecond,
                              i > 0 || k > 0);
                umma_commit(&sh.freed[j]);
            }
        }
    }
}

// ---- the worker warps ----------------------------------------------------------------

struct Row {
    const uint8_t* data;  // null: the row does not exist
    uint2 scales;
};

// The cache entry of tile row `row`: a slot (index form) or a page, -1 for none.
template <int kSrc>
__device__ __forceinline__ int32_t row_entry(const AttnParams& p, const Unit& un, int32_t tile, int row) {
    if (kSrc == kIndexed) {
        const int64_t c = (int64_t)tile * kTile + row;
        if (c >= p.cols) return -1;
        const int32_t s = p.idx[(int64_t)un.col_token[0] * p.idx_stride + c];
        return slot_ok(p, (int32_t)c, s) ? s : -1;
    }
    const int64_t pos = (int64_t)un.lo + (int64_t)tile * kTile + row;
    if (pos > un.hi) return -1;
    int32_t off;
    const int32_t logical = div_block32((int32_t)pos, p.cache.block_size, p.cache.shift, off) -
                            (p.base_off ? p.base_off[un.req] : 0);
    if (logical < 0 || logical >= p.bt_width) return -1;
    const int32_t page = p.bt[(int64_t)un.req * p.bt_stride + logical];
    return page >= 0 && page < p.cache.num_pages ? page : -1;
}

template <int kSrc>
__device__ __forceinline__ Row row_of(const AttnParams& p, const Unit& un, int32_t tile, int row,
                                      int32_t entry) {
    Row r{nullptr, make_uint2(0, 0)};
    if (entry < 0) return r;
    const AttnCache& c = kSrc == kIndexed && tile * kTile + row >= p.split ? p.extra : p.cache;
    int32_t page = entry, off;
    if (kSrc == kIndexed)
        page = div_block32(entry, c.block_size, c.shift, off);
    else
        div_block32((int32_t)((int64_t)un.lo + (int64_t)tile * kTile + row), c.block_size, c.shift, off);
    const int32_t token_stride = p.head_dim + p.rope_dim, nsc = p.head_dim / 64;
    const uint8_t* pg = c.base + (int64_t)page * c.page_stride;
    r.data = pg + (int64_t)off * token_stride;
    const uint8_t* sc = pg + (int64_t)c.block_size * token_stride + (int64_t)off * nsc;
    if (nsc == 8) {
        r.scales = ld_nc_v2(sc);
    } else if (nsc == 4) {
        r.scales.x = ld_nc_u32(sc);
    } else {
        r.scales.x = ld_nc_u8(sc) | (ld_nc_u8(sc + 1) << 8);
    }
    return r;
}

// The quarter (16 dims) of chunk c that a thread dequantises: 16 E4M3 bytes, or
// 32 bytes of bf16 where the chunk lies in the rope dims.
__device__ __forceinline__ void load_quarter(const AttnParams& p, const Row& r, int c, int quarter,
                                             uint4 (&raw)[2]) {
    raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
    if (r.data == nullptr) return;
    const int nope = p.head_dim - p.rope_dim;
    if (c * 64 < nope) {
        raw[0] = ld_stream_v4(r.data + c * 64 + quarter * 16);
    } else {
        const uint8_t* b = r.data + nope + (c * 64 - nope) * 2 + quarter * 32;
        raw[0] = ld_stream_v4(b);
        raw[1] = ld_stream_v4(b + 16);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(uint32_t bytes, uint64_t scale2) {
    return scale_f16x2_to_bf16x2(cvt_e4m3x2_to_f16x2(bytes), scale2);
}

// 16 dims as eight bf16 pairs, by the rule of the gather.
__device__ __forceinline__ void dequant_quarter(const AttnParams& p, const Row& r, int c,
                                                const uint4 (&raw)[2], uint32_t (&w)[8]) {
    if (c * 64 < p.head_dim - p.rope_dim) {
        const uint32_t b = ((c < 4 ? r.scales.x : r.scales.y) >> (8 * (c & 3))) & 0xFFu;
        const uint64_t s2 = splat_f32x2(r.data == nullptr ? 0.0f : ue8m0_scale(b));
        const uint32_t in[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = bf16_pair(in[i] & 0xFFFFu, s2);
            w[2 * i + 1] = bf16_pair(in[i] >> 16, s2);
        }
    } else {
        w[0] = raw[0].x; w[1] = raw[0].y; w[2] = raw[0].z; w[3] = raw[0].w;
        w[4] = raw[1].x; w[5] = raw[1].y; w[6] = raw[1].z; w[7] = raw[1].w;
    }
}

// Clears the non-finite values of w; true if there were any.
__device__ __forceinline__ bool clear_non_finite(uint32_t (&w)[8]) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool lo = (w[i] & 0x7F80u) == 0x7F80u, hi = (w[i] & 0x7F800000u) == 0x7F800000u;
        if (lo) w[i] &= 0xFFFF0000u;
        if (hi) w[i] &= 0x0000FFFFu;
        bad |= lo | hi;
    }
    return bad;
}

template <int N, int kSrc>
__device__ bool work(const AttnParams& p, const LaunchShape& ls, Shared& sh, uint8_t* k_tile,
                     uint8_t* q_tile, uint8_t* p_tile, uint32_t tmem) {
    constexpr int NC = N / 4;  // columns of a worker warp
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const int quad = warp % 4, group = warp / 4;
    const int row = tid / 4, quarter = tid % 4;        // dequantisation
    const int srow = quad * kWarp + lane;              // softmax: the tile row of this lane
    const int chunks = p.head_dim / 64, blocks = p.head_dim / 128;
    const uint32_t k_addr = smem_u32(k_tile) + row * 128;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * kWarp) << 16);
    uint32_t step = 0, exchange = 0;

    for (int seq = 0;; ++seq) {
        if (!wait_all(&sh.unit_full[seq & 1], (seq >> 1) & 1)) return false;
        const Unit& un = sh.unit[seq & 1];
        if (un.done) return true;
        const int32_t ntiles = un.ntiles;
        uint64_t mask = un.mask;
        const bool masked = mask != 0;

        float l[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) l[i] = 0.0f;
        float m_used = -INFINITY;  // of column `lane`, for lane < NC

        if (ntiles > 0) {
            // queries of the unit into the swizzled B tile; unused columns are zero
            for (int i = tid; i < N * chunks * 8; i += kWorkers * kWarp) {
                const int part = i % 8, c = (i / 8) % chunks, n = i / (8 * chunks);
                const uint32_t dst = smem_u32(q_tile) + c * (N * 128) + n * 128 + ((part ^ (n & 7)) * 16);
                const int32_t t = un.col_token[n];
                uint4 v = make_uint4(0, 0, 0, 0);
                if (t >= 0)
                    v = ld_nc_v4(p.q + (int64_t)t * p.q_stride_t + (int64_t)un.col_head[n] * p.q_stride_h +
                                 c * 64 + part * 8);
                sts_v4(dst, v.x, v.y, v.z, v.w);
            }
            int32_t tile = masked ? __ffsll(mask) - 1 : un.first;
            int32_t entry = row_entry<kSrc>(p, un, tile, row);
            for (int32_t i = 0; i < ntiles; ++i, ++step) {
                const int buf = step & 1;
                const Row r = row_of<kSrc>(p, un, tile, row, entry);
                if (quarter == 0) {
                    sh.row_ok[buf][row] = r.data != nullptr;
                    if (kSrc == kTokens) sh.row_bad[buf][row] = 0;
                }
                __syncwarp();
                uint4 raw[4][2];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c < chunks) load_quarter(p, r, c, quarter, raw[c]);
                const int32_t this_tile = tile;
                if (i + 1 < ntiles) {
                    mask &= mask - 1;
                    tile = masked ? __ffsll(mask) - 1 : tile + 1;
                    entry = row_entry<kSrc>(p, un, tile, row);
                }
#pragma unroll
                for (int c = 0; c < kMaxChunks; ++c) {
                    if (c >= chunks) break;
                    if (step > 0 && c % 2 == 0 && !wait_all(&sh.freed[c / 2], (step - 1) & 1)) return false;
                    uint32_t w[8];
                    dequant_quarter(p, r, c, raw[c % 4], w);
                    if (kSrc == kTokens && clear_non_finite(w)) sh.row_bad[buf][row] = 1;
                    const uint32_t dst = k_addr + c * kChunkBytes;
                    sts_v4(dst + (((2 * quarter) ^ (row & 7)) * 16), w[0], w[1], w[2], w[3]);
                    sts_v4(dst + (((2 * quarter + 1) ^ (row & 7)) * 16), w[4], w[5], w[6], w[7]);
                    if (c + 4 < chunks) load_quarter(p, r, c + 4, quarter, raw[c % 4]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.full[c]);
                }

                // softmax of the tile: this lane's row, NC columns
                if (!wait_all(&sh.full[chunks - 1], step & 1)) return false;  // row_ok, row_bad
                if (!wait_all(&sh.s_ready, step & 1)) return false;
                tmem_fence_after();
                float s[NC];
                tmem_ld<NC>(lane_base + group * NC, s);
                const bool ok = sh.row_ok[buf][srow];
                const int32_t pos = un.lo + this_tile * kTile + srow;
                const bool bad = kSrc == kTokens && sh.row_bad[buf][srow];
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    bool see = ok;
                    if (kSrc == kTokens)
                        see = see && pos >= un.col_lo[group * NC + k] && pos <= un.col_hi[group * NC + k];
                    s[k] = see ? (bad ? NAN : s[k] * ls.scale_log2) : -INFINITY;
                }
                float mine = -INFINITY;
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float x = warp_max(s[k]);
                    if (lane == k) mine = x;
                }
                float(&red)[4][16] = sh.red[group][exchange & 1];
                if (lane < NC) red[quad][lane] = mine;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.group_bar[group]);
                if (!wait_all(&sh.group_bar[group], exchange & 1)) return false;
                ++exchange;
                bool grow = false;
                if (lane < NC) {
                    const float top = fmaxf(fmaxf(red[0][lane], red[1][lane]), fmaxf(red[2][lane], red[3][lane]));
                    float alpha = 1.0f;
                    if (top > m_used + kLazy) {
                        alpha = m_used == -INFINITY ? 1.0f : ex2_approx(m_used - top);  // no sums before
                        grow = alpha != 1.0f;
                        m_used = top;
                    }
                    sh.ref[warp][lane] = m_used == -INFINITY ? 0.0f : m_used;
                    sh.aux[warp][lane] = alpha;
                }
                __syncwarp();
                if (__any_sync(0xFFFFFFFFu, grow)) {
                    // the previous tile's second product is done: s_ready came after it
                    float a[NC];
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        a[k] = sh.aux[warp][k];
                        l[k] *= a[k];
                    }
                    for (int j = 0; j < blocks; ++j) {
                        float o[NC];
                        tmem_ld<NC>(lane_base + N + j * N + group * NC, o);
#pragma unroll
                        for (int k = 0; k < NC; ++k) o[k] *= a[k];
                        tmem_st<NC>(lane_base + N + j * N + group * NC, o);
                    }
                    tmem_wait_st();
                }
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    s[k] = ex2_approx(s[k] - sh.ref[warp][k]);
                    l[k] += s[k];
                }
                // weights to the N-major B tile: 8 columns (16 bytes) of a row, rows side by side
                if constexpr (NC >= 8) {
#pragma unroll
                    for (int k = 0; k < NC; k += 8)
                        sts_v4(smem_u32(p_tile) + (group * NC + k) / 8 * (kTile * 16) + srow * 16,
                               pack_bf16x2(s[k], s[k + 1]), pack_bf16x2(s[k + 2], s[k + 3]),
                               pack_bf16x2(s[k + 4], s[k + 5]), pack_bf16x2(s[k + 6], s[k + 7]));
                } else {
                    sts_v2(smem_u32(p_tile) + (group / 2) * (kTile * 16) + srow * 16 + (group & 1) * 8,
                           pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
                }
                fence_async_smem();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready);
            }
        }

        // the unit's sums: over the lanes, then over the group's four warps
        float mine = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float x = l[k];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
            if (lane == k) mine = x;
        }
        float(&red)[4][16] = sh.red[group][exchange & 1];
        if (lane < NC) red[quad][lane] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.group_bar[group]);
        if (!wait_all(&sh.group_bar[group], exchange & 1)) return false;
        ++exchange;
        if (lane < NC) {
            const float total = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
            const int n = group * NC + lane;
            const int32_t t = un.col_token[n];
            float inv = 1.0f;
            if (t >= 0) {
                const int32_t h = un.col_head[n];
                if (ls.splits > 1) {
                    if (quad == 0) {
                        float* ml = ls.part_ml + (((int64_t)t * p.num_heads + h) * ls.splits + un.part) * 2;
                        ml[0] = m_used;
                        ml[1] = total;
                    }
                } else {
                    const float ref = m_used == -INFINITY ? 0.0f : m_used;
                    const float den = total + (p.sink ? ex2_approx(p.sink[h] * kLog2e - ref) : 0.0f);
                    inv = total == 0.0f ? 0.0f : 1.0f / den;
                    if (p.lse && quad == 0)
                        p.lse[(int64_t)t * p.lse_stride_t + h] =
                            total == 0.0f ? -INFINITY : (ref + log2f(total)) * kLn2;
                }
            }
            sh.aux[warp][lane] = inv;
        }
        __syncwarp();
        if (ntiles > 0) {
            if (!wait_all(&sh.freed[blocks - 1], (step - 1) & 1)) return false;
            tmem_fence_after();
        }
        for (int j = 0; j < blocks; ++j) {
            float o[NC];
            if (ntiles > 0) {
                tmem_ld<NC>(lane_base + N + j * N + group * NC, o);
            } else {
#pragma unroll
                for (int k = 0; k < NC; ++k) o[k] = 0.0f;
            }
            const int d = j * 128 + srow;
            if (ls.splits > 1) {
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const int32_t t = un.col_token[group * NC + k], h = un.col_head[group * NC + k];
                    if (t >= 0)
                        ls.part_o[(((int64_t)t * p.num_heads + h) * ls.splits + un.part) * p.head_dim + d] = o[k];
                }
            } else {
                // two dims a store: even lanes take column k, odd lanes column k + 1
#pragma unroll
                for (int k = 0; k < NC; k += 2) {
                    const float a = o[k] * sh.aux[warp][k], b = o[k + 1] * sh.aux[warp][k + 1];
                    const bool odd = lane & 1;
                    const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
                    const uint32_t w = odd ? pack_bf16x2(other, b) : pack_bf16x2(a, other);
                    const int n = group * NC + k + (odd ? 1 : 0);
                    const int32_t t = un.col_token[n];
                    if (t >= 0)
                        *reinterpret_cast<uint32_t*>(p.out + (int64_t)t * p.out_stride_t +
                                                     (int64_t)un.col_head[n] * p.out_stride_h + (d & ~1)) = w;
                }
            }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.unit_empty[seq & 1]);
    }
}

constexpr size_t kAlign = 1024;

size_t smem_bytes(int n, int head_dim) {
    return kAlign + (size_t)head_dim / 64 * kChunkBytes + (size_t)head_dim / 64 * n * 128 +
           (size_t)n / 8 * kTile * 16 + sizeof(Shared);
}

template <int N, int kSrc>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ LaunchShape ls) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((kAlign - (smem_u32(smem_raw) & (kAlign - 1))) & (kAlign - 1));
    const int chunks = p.head_dim / 64;
    uint8_t* k_tile = base;
    uint8_t* q_tile = k_tile + chunks * kChunkBytes;
    uint8_t* p_tile = q_tile + chunks * (N * 128);
    Shared& sh = *reinterpret_cast<Shared*>(p_tile + N / 8 * kTile * 16);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.unit_full[i], 1);
            mbar_init(&sh.unit_empty[i], kWorkers + 1);
        }
        for (int i = 0; i < kMaxChunks; ++i) mbar_init(&sh.full[i], kWorkers);
        for (int i = 0; i < kMaxChunks / 2; ++i) mbar_init(&sh.freed[i], 1);
        mbar_init(&sh.s_ready, 1);
        mbar_init(&sh.p_ready, kWorkers);
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&sh.group_bar[i], 4);
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&sh.tmem, ls.tmem_cols);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_wait();
    pdl_launch_dependents();

    bool ok = true;
    if (warp < kWorkers) {
        ok = work<N, kSrc>(p, ls, sh, k_tile, q_tile, p_tile, tmem);
    } else if (warp == kPlanWarp) {
        ok = plan<kSrc>(p, ls, sh);
    } else if (lane == 0) {
        ok = issue<N>(p, sh, smem_u32(k_tile), smem_u32(q_tile), smem_u32(p_tile), tmem);
        if (!ok) {  // wait for the MMAs in flight before the operands go
            umma_commit(&sh.drain);
            mbar_wait_bounded(&sh.drain, 0, kWaitLimitNs);
        }
    }
    if (!ok && lane == 0) atomicAdd(&g_attn_wait_timeouts, 1u);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, ls.tmem_cols);
}

// ---- joining the parts of a split row ----------------------------------------------------
//
// out = sum_i 2^(m_i - m) o_i / (sum_i 2^(m_i - m) l_i + 2^(sink' - m)), m = max m_i
// (log2 units).  One CTA per (token, head); a thread takes four dims, so the
// parts are read as whole rows.
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnParams p, const LaunchShape ls) {
    extern __shared__ float s_ml[];
    pdl_wait();
    const int64_t th = blockIdx.x;
    const int32_t h = (int32_t)(th % p.num_heads);
    const int64_t t = th / p.num_heads;
    const int S = ls.splits;
    for (int i = threadIdx.x; i < 2 * S; i += blockDim.x) s_ml[i] = ls.part_ml[th * 2 * S + i];
    __syncthreads();
    pdl_launch_dependents();
    float m = -INFINITY;
    for (int i = 0; i < S; ++i) m = fmaxf(m, s_ml[2 * i]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float total = 0.0f;
    for (int i = 0; i < S; ++i) total += ex2_approx(s_ml[2 * i] - ref) * s_ml[2 * i + 1];
    const int d = threadIdx.x * 4;
    if (d < p.head_dim) {
        float4 a = make_float4(0, 0, 0, 0);
        const float* o = ls.part_o + th * S * p.head_dim + d;
#pragma unroll 4
        for (int i = 0; i < S; ++i) {
            const float w = ex2_approx(s_ml[2 * i] - ref);
            const float4 v = *reinterpret_cast<const float4*>(o + (int64_t)i * p.head_dim);
            a.x += w * v.x;
            a.y += w * v.y;
            a.z += w * v.z;
            a.w += w * v.w;
        }
        const float den = total + (p.sink ? ex2_approx(p.sink[h] * kLog2e - ref) : 0.0f);
        const float inv = total == 0.0f ? 0.0f : 1.0f / den;
        st_v2(p.out + t * p.out_stride_t + (int64_t)h * p.out_stride_h + d,
              make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv)));
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[t * p.lse_stride_t + h] = total == 0.0f ? -INFINITY : (ref + log2f(total)) * kLn2;
}

// ---- host ------------------------------------------------------------------------------------

// How a call is cut into units; kSrc and N as the launch takes them.
struct Plan {
    int src, n;
    LaunchShape ls;
};

Plan make_plan(int64_t num_tokens, int32_t num_heads, int32_t head_dim, int64_t max_keys, bool indexed,
               int32_t num_reqs) {
    Plan pl{};
    LaunchShape& ls = pl.ls;
    ls.head_groups = (num_heads + kMaxCols - 1) / kMaxCols;
    ls.heads_per_unit = (num_heads + ls.head_groups - 1) / ls.head_groups;
    ls.tokens_per_unit = 1;
    pl.src = indexed ? kIndexed : kOneToken;
    int cols = ls.heads_per_unit;
    // Neighbouring tokens share a unit where most requests bring several: a unit
    // never crosses a request.
    if (!indexed && num_heads <= kMaxCols / 2 && num_tokens >= 4 * (int64_t)num_reqs) {
        ls.tokens_per_unit = kMaxCols / num_heads < kWarp ? kMaxCols / num_heads : kWarp;
        cols = ls.tokens_per_unit * num_heads;
        pl.src = kTokens;
    }
    pl.n = cols <= 16 ? 16 : cols <= 32 ? 32 : 64;
    const int64_t base = (num_tokens + ls.tokens_per_unit - 1) / ls.tokens_per_unit * ls.head_groups;
    // Few units: each is cut along its tiles until they fill the SMs.
    const int64_t tiles = (max_keys + kTile - 1) / kTile;
    int64_t splits = base < sm_count() ? sm_count() / base : 1;
    if (splits > tiles) splits = tiles;
    ls.splits = (int32_t)(splits < 1 ? 1 : splits);
    ls.units = base * ls.splits;
    const uint32_t need = (uint32_t)pl.n * (1 + head_dim / 128);
    ls.tmem_cols = 32;
    while (ls.tmem_cols < need) ls.tmem_cols *= 2;
    return pl;
}

int64_t part_bytes(int64_t num_tokens, int32_t num_heads, int32_t head_dim, int32_t splits) {
    return splits <= 1 ? 0 : num_tokens * num_heads * splits * (head_dim + 4) * (int64_t)sizeof(float);
}

template <int N, int kSrc>
cudaError_t launch(const AttnParams& p, const LaunchShape& ls, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_limit_per_device(attention_kernel<N, kSrc>, (int)smem_bytes(N, 512), done);
    if (e != cudaSuccess) return e;
    const int64_t grid = ls.units < sm_count() ? ls.units : sm_count();
    return launch_pdl(attention_kernel<N, kSrc>, dim3((unsigned)grid), dim3(kThreads), smem_bytes(N, p.head_dim),
                      stream, p, ls);
}

template <int kSrc>
cudaError_t launch_n(const AttnParams& p, const Plan& pl, cudaStream_t stream) {
    return pl.n == 16 ? launch<16, kSrc>(p, pl.ls, stream)
                      : pl.n == 32 ? launch<32, kSrc>(p, pl.ls, stream) : launch<64, kSrc>(p, pl.ls, stream);
}

cudaError_t run(AttnParams p, int64_t max_keys, bool indexed, cudaStream_t stream) {
    Plan pl = make_plan(p.num_tokens, p.num_heads, p.head_dim, max_keys, indexed, p.num_reqs);
    p.cache.shift = log2_if_pow2(p.cache.block_size);
    p.extra.shift = log2_if_pow2(p.extra.block_size);
    pl.ls.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
    pl.ls.part_o = static_cast<float*>(p.workspace);
    pl.ls.part_ml = pl.ls.part_o + p.num_tokens * p.num_heads * pl.ls.splits * p.head_dim;
    cudaError_t e = pl.src == kIndexed ? launch_n<kIndexed>(p, pl, stream)
                    : pl.src == kOneToken ? launch_n<kOneToken>(p, pl, stream)
                                          : launch_n<kTokens>(p, pl, stream);
    if (e != cudaSuccess || pl.ls.splits == 1) return e;
    return launch_pdl(attention_join_kernel, dim3((unsigned)(p.num_tokens * p.num_heads)), dim3(128),
                      (size_t)pl.ls.splits * 2 * sizeof(float), stream, p, pl.ls);
}

}  // namespace

int64_t attention_workspace_bytes(int64_t num_tokens, int32_t num_heads, int32_t head_dim, int64_t max_keys,
                                  bool indexed, int32_t num_reqs) {
    const Plan pl = make_plan(num_tokens, num_heads, head_dim, max_keys, indexed, num_reqs);
    return part_bytes(num_tokens, num_heads, head_dim, pl.ls.splits);
}

cudaError_t launch_attention_indexed(AttnParams p, cudaStream_t stream) {
    return run(p, p.cols, true, stream);
}

cudaError_t launch_attention_chunk(AttnParams p, cudaStream_t stream) {
    const int64_t all = (int64_t)p.bt_width * p.cache.block_size;
    return run(p, p.window > 0 && p.window < all ? p.window : all, false, stream);
}

cudaError_t read_attention_wait_timeouts(uint32_t* count) {
    return cudaMemcpyFromSymbol(count, g_attn_wait_timeouts, sizeof(uint32_t));
}

}  // namespace psk
