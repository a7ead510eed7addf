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
// Roles.  Worker warps dequantise a tile, take the softmax of S^T and at the end of a
// unit write O^T; one warp issues the MMAs; one plans ahead: it finds the tiles
// that hold anything visible and puts the addresses of their rows into a ring,
// across units.  The tile is handed over in blocks of 128 dims: the first product
// follows the dequantisation block by block, and the next tile is dequantised into
// the blocks the second product has finished with.  The first loads of a tile are in
// flight during the softmax of the one before.  Every wait is bounded (2 s of wall
// time, counted in psk_device_wait_timeouts).
//
// Softmax in one pass: a running reference m per column.  It follows the
// maximum lazily: the first tile sets it, and later ones raise it only where a
// weight would exceed 2^16, so that O^T is hardly ever rescaled and the maxima
// of most tiles are never formed; the reference cancels in out and in lse.  Sums
// and weights are binary32; the weights are rounded to bf16 for the second
// product alone (the operands of one MMA share a type, and a row's bf16 values do
// not fit fp16's range), while l sums them unrounded, so that lse keeps binary32
// accuracy and the roundings in out, being unbiased, average out.
//
// What bounds it.  The tensor cores read both operands from shared memory: an MMA of
// 128 rows and 64 columns moves 6 KB and takes the 48 cycles those need at 128 bytes a
// cycle, half again its arithmetic.  A tile (head_dim 512, 64 columns) is 64 of
// them, 3100 cycles; dequantising it writes 128 KB more, 1000 cycles, and the loads,
// barriers and weights share the port, which the counters have busy 68 % of the time.
// Measured 8100 cycles a tile, its share of writing O^T (6000 a unit) included: 4096
// tokens of 128 heads over 640 rows take 964 us, 568 TFLOP/s, against 288 us at the
// matrix rate and 490 at the port's.  The rest is the chain dequantise - scores - softmax -
// weights, which one 128 KB tile beside 64 KB of queries cannot overlap with itself.
// Other forms of it, measured on the 4096 tokens when this one took 1164 us:
//  * tiles of 64 rows, two in work: 1454 us; the first product drops to half rate and
//    each tile pays the waits of a whole one;
//  * separate warps for dequantisation and softmax on top of it: 1510;
//  * records copied into shared memory in bulk, one copy a row, by a copying warp:
//    2364 (a copy of 576 bytes takes some 130 cycles of the copy unit).
#include <atomic>
#include <cmath>

#include "attention.h"
#include "psk_common.cuh"
#include "umma.cuh"

namespace psk {
namespace {

constexpr int kTile = 128;            // rows of a tile (M of the first product)
constexpr int kMaxGroups = 4;
constexpr int kMaxBlocks = 4;         // 128-dim blocks of a row (head_dim 512)
constexpr int kChunkBytes = kTile * 128;
constexpr int kMaxCols = 64;
constexpr int kMostParts = 8;         // parts a cluster joins
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 16.0f;        // log2 units the maximum may run ahead of the reference
constexpr float kNone = -3.0e38f;     // reference of a column that has seen nothing
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ unsigned int g_attn_wait_timeouts = 0;

// What a row that does not exist (or is not visible) is read from: the longest
// record, all zero, so that the loads of a tile need no conditions.
__device__ const uint4 g_zero_row[64 + 2 * 448 / 16] = {};

enum { kIndexed = 0, kOneToken = 1, kTokens = 2 };

// 16 worker warps (64 heads: 64 tokens 23.8 us against 27.9 with 8; 32 heads: 19.1
// against 21.4), 8 where 16 would have fewer than 8 columns each.  16 columns as 32
// with 16 warps: 64 tokens of 16 heads 19.1 us against 18.7, one row of 8192 keys for
// each 122 against 114.
template <int N>
struct Roles {
    static constexpr int kWorkers = N == 16 ? 8 : 16;
    static constexpr int kGroups = kWorkers / 4;  // warps of a group share their columns, each with 32 rows
    static constexpr int kMmaWarp = kWorkers, kPlanWarp = kWorkers + 1;
    static constexpr int kThreads = (kWorkers + 2) * kWarp;
};

// A set of columns; its tiles follow one another in the stream of tiles.
struct Unit {
    int64_t part_row;              // a unit cut in parts: row of its column 0 among such columns; else -1
    int32_t part;                  // which part
    int32_t all_lo, all_hi;        // kTokens: positions that every column in use sees
    int32_t pad;
    int64_t col_q[kMaxCols];       // element offset of the column's query
    int64_t col_out[kMaxCols];     // and of its output row (of its part, where the work is split)
    float col_sink[kMaxCols];      // log2 units; -infinity without one
    int32_t col_token[kMaxCols];   // -1: column not in use
    int32_t col_head[kMaxCols];
    int32_t col_lo[kMaxCols], col_hi[kMaxCols];  // kTokens: positions the column sees
};

struct alignas(16) Row {
    const uint8_t* data;    // g_zero_row: the row does not exist or is not visible
    const uint8_t* scales;  // its UE8M0 bytes
};

constexpr int kFirst = 1, kLast = 2, kEmpty = 4, kDone = 8;

// One step of the stream: a tile's rows, and where it stands in its unit.
struct Tile {
    int32_t flags;
    int32_t unit;   // slot of its unit
    int32_t pos;    // position form: position of row 0
    int32_t pad;
    Row row[kTile];
};

constexpr int kTiles = 3;  // tiles the planning warp may be ahead, the current one included

struct Shared {
    Tile tile[kTiles];
    Unit unit[2];
    alignas(16) float red[2][4][kMaxCols];  // [parity of the group's exchange][quad][column]
    alignas(16) float ref[4 * kMaxCols];    // a copy per quad, by warps
    alignas(16) float aux[4 * kMaxCols];
    int32_t over[kMaxGroups][2][4];
    uint64_t tile_full[kTiles], tile_empty[kTiles];
    uint64_t unit_empty[2];
    uint64_t full[kMaxBlocks];     // 128 dims of the tile are dequantised
    uint64_t freed[kMaxBlocks];    // the second product is done with them
    uint64_t s_ready, p_ready, drain;
    uint64_t group_bar[kMaxGroups];
    uint32_t tmem;
    uint2 scales[2][kTile];        // UE8M0 bytes of the rows
    uint8_t row_bad[2][kTile];     // kTokens: the row holds a NaN or an infinity
    int32_t failed;                // a wait of this CTA expired
    float2 part_ml[kMaxCols];      // joined in a cluster: the columns' references and sums
};

struct LaunchShape {
    int32_t heads_per_unit;  // heads of one token in a unit
    int32_t head_groups;     // ceil(num_heads / heads_per_unit)
    int32_t tokens_per_unit; // kTokens: neighbouring tokens in a unit
    int32_t splits;
    int64_t units;           // with every part of a cut unit counted
    int64_t whole;           // units before this one are not cut
    int64_t part_rows;       // columns of the cut ones
    int32_t cluster;         // 1: a unit's parts are the CTAs of a cluster, which joins them
    uint32_t tmem_cols;
    float scale_log2;
    float* part_o;           // [row of a cut unit's column][split][D]
    float* part_ml;          // [row][split][2]
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_poll_bounded(bar, parity, kWaitLimitNs);
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

// Even share `part` of n tiles: [first, end).
__device__ __forceinline__ void share(int32_t n, int32_t part, int32_t parts, int32_t& first,
                                      int32_t& end) {
    first = (int32_t)((int64_t)n * part / parts);
    end = (int32_t)((int64_t)n * (part + 1) / parts);
}

// What the rows of a unit are looked up by.
struct Source {
    int64_t token;           // index form
    int32_t req, lo, hi;     // position form
    int32_t base;            // logical page of the table row's first entry
};

constexpr int kRowsPerLane = kTile / kWarp;

// What a tile's rows lane, lane + 32, ... are looked up in: slots (index form) or
// pages, -1 past the end.  The loads are left in flight.
template <int kSrc>
__device__ __forceinline__ void tile_lookup(const AttnParams& p, const Source& src, int32_t tile, int lane,
                                            int32_t (&x)[kRowsPerLane]) {
#pragma unroll
    for (int j = 0; j < kRowsPerLane; ++j) {
        x[j] = -1;
        const int64_t i = (int64_t)tile * kTile + j * kWarp + lane;
        if (kSrc == kIndexed) {
            if (i < p.cols) x[j] = p.idx[src.token * p.idx_stride + i];
        } else {
            const int64_t pos = src.lo + i;
            if (pos <= src.hi) {
                int32_t off;
                const int32_t logical =
                    div_block32((int32_t)pos, p.cache.block_size, p.cache.shift, off) - src.base;
                if (logical >= 0 && logical < p.bt_width) x[j] = p.bt[(int64_t)src.req * p.bt_stride + logical];
            }
        }
    }
}

// The entries among them that exist, the others -1.  True if any row has one.
template <int kSrc>
__device__ __forceinline__ bool tile_entries(const AttnParams& p, int32_t tile, int lane,
                                             int32_t (&x)[kRowsPerLane]) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < kRowsPerLane; ++j) {
        const int32_t c = tile * kTile + j * kWarp + lane;
        const AttnCache& k = kSrc == kIndexed && c >= p.split ? p.extra : p.cache;
        const int64_t limit = kSrc == kIndexed ? k.num_pages * k.block_size : k.num_pages;
        if (x[j] >= limit) x[j] = -1;
        any |= x[j] >= 0;
    }
    return __any_sync(0xFFFFFFFFu, any);
}

// Fills `rows` with the addresses of the entries' data and scales.
template <int kSrc>
__device__ __forceinline__ void tile_rows(const AttnParams& p, const Source& src, int32_t tile, int lane,
                                          const int32_t (&entry)[kRowsPerLane], Row* rows) {
    const int32_t token_stride = p.head_dim + p.rope_dim;
#pragma unroll
    for (int j = 0; j < kRowsPerLane; ++j) {
        const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
        Row r{zero, zero};
        if (entry[j] >= 0) {
            const int32_t i = tile * kTile + j * kWarp + lane;
            const AttnCache& c = kSrc == kIndexed && i >= p.split ? p.extra : p.cache;
            int32_t page = entry[j], off;
            if (kSrc == kIndexed)
                page = div_block32(entry[j], c.block_size, c.shift, off);
            else
                div_block32(src.lo + i, c.block_size, c.shift, off);
            const uint8_t* pg = c.base + (int64_t)page * c.page_stride;
            r.data = pg + (int64_t)off * token_stride;
            r.scales = pg + (int64_t)c.block_size * token_stride + (int64_t)off * (p.head_dim / 64);
        }
        rows[j * kWarp + lane] = r;
    }
}

struct Stream {
    int tiles = 0, units = 0;  // published so far
};

// Waits for the tile slot the next record takes.
__device__ __forceinline__ bool tile_slot(Shared& sh, const Stream& st) {
    return st.tiles < kTiles || wait_all(&sh.tile_empty[st.tiles % kTiles], (st.tiles / kTiles - 1) & 1);
}

__device__ __forceinline__ void publish(Shared& sh, Stream& st, int lane, int32_t flags, int32_t pos) {
    Tile& t = sh.tile[st.tiles % kTiles];
    if (lane == 0) {
        t.flags = flags;
        t.unit = st.units & 1;
        t.pos = pos;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.tile_full[st.tiles % kTiles]);
    ++st.tiles;
}

// The tiles [first, end) of a unit that hold anything.  Look-ups run two tiles
// ahead; a tile is published once it is known whether another one follows.
template <int kSrc>
__device__ __forceinline__ bool stream_unit(const AttnParams& p, Shared& sh, Stream& st, const Source& src,
                                            int32_t first, int32_t end, int lane) {
    int32_t cur[kRowsPerLane], ahead[2][kRowsPerLane];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (first + i < end) tile_lookup<kSrc>(p, src, first + i, lane, ahead[i]);
    int32_t flags = kFirst, pending = -1;  // the tile that waits to be published
    for (int32_t tile = first; tile < end; ++tile) {
        int32_t x[kRowsPerLane];
#pragma unroll
        for (int j = 0; j < kRowsPerLane; ++j) {
            x[j] = ahead[0][j];
            ahead[0][j] = ahead[1][j];
        }
        if (tile + 2 < end) tile_lookup<kSrc>(p, src, tile + 2, lane, ahead[1]);
        if (!tile_entries<kSrc>(p, tile, lane, x)) continue;
        if (pending >= 0) {
            if (!tile_slot(sh, st)) return false;
            tile_rows<kSrc>(p, src, pending, lane, cur, sh.tile[st.tiles % kTiles].row);
            publish(sh, st, lane, flags, kSrc == kIndexed ? 0 : src.lo + pending * kTile);
            flags = 0;
        }
        pending = tile;
#pragma unroll
        for (int j = 0; j < kRowsPerLane; ++j) cur[j] = x[j];
    }
    if (!tile_slot(sh, st)) return false;
    if (pending >= 0) {
        tile_rows<kSrc>(p, src, pending, lane, cur, sh.tile[st.tiles % kTiles].row);
        publish(sh, st, lane, flags | kLast, kSrc == kIndexed ? 0 : src.lo + pending * kTile);
    } else {
        publish(sh, st, lane, kFirst | kLast | kEmpty, 0);
    }
    ++st.units;
    return true;
}

// Waits for the slot of the next unit, which two units before it have used.
__device__ __forceinline__ bool unit_slot(Shared& sh, const Stream& st) {
    return st.units < 2 || wait_all(&sh.unit_empty[st.units & 1], ((st.units >> 1) - 1) & 1);
}

__device__ __forceinline__ void set_column(const AttnParams& p, const LaunchShape& ls, Unit& un, int c,
                                           int32_t part, int64_t part_row, int64_t t, int32_t h, bool used,
                                           int32_t lo, int32_t hi) {
    un.col_sink[c] = used && p.sink ? p.sink[h] * kLog2e : -INFINITY;
    un.col_token[c] = used ? (int32_t)t : -1;
    un.col_head[c] = h;
    un.col_q[c] = t * p.q_stride_t + h * p.q_stride_h;
    un.col_out[c] = part_row >= 0 ? ((part_row + c) * ls.splits + part) * p.head_dim
                                  : t * p.out_stride_t + h * p.out_stride_h;
    un.col_lo[c] = used ? lo : 0;
    un.col_hi[c] = used ? hi : -1;
}

template <int kSrc>
__device__ bool plan(const AttnParams& p, const LaunchShape& ls, Shared& sh) {
    const int lane = threadIdx.x % kWarp;
    Stream st;
    for (int64_t u = blockIdx.x; u < ls.units; u += gridDim.x) {
        const bool cut = u >= ls.whole;
        const int32_t parts = cut ? ls.splits : 1, part = cut ? (int32_t)((u - ls.whole) % parts) : 0;
        const int64_t v = cut ? ls.whole + (u - ls.whole) / parts : u;
        const int64_t part_row = cut ? (v - ls.whole) * ls.heads_per_unit * ls.tokens_per_unit : -1;
        if (kSrc != kTokens) {
            const int64_t t = v / ls.head_groups;
            const int32_t h0 = (int32_t)(v % ls.head_groups) * ls.heads_per_unit;
            const int32_t heads = min(ls.heads_per_unit, p.num_heads - h0);
            Source src{t, 0, 0, -1, 0};
            int32_t n, first, end;
            if (kSrc == kIndexed) {
                n = p.cols / kTile + (p.cols % kTile != 0);
            } else {
                const TokenRange x = token_range(p, t);
                src.req = x.req;
                src.lo = x.lo;
                src.hi = x.hi;
                if (p.base_off && x.req >= 0) src.base = p.base_off[x.req];
                n = x.hi < x.lo ? 0 : (x.hi - x.lo) / kTile + 1;
            }
            share(n, part, parts, first, end);
            if (!unit_slot(sh, st)) return false;
            Unit& un = sh.unit[st.units & 1];
            if (lane == 0) {
                un.part = part;
                un.part_row = part_row;
            }
#pragma unroll
            for (int c = lane; c < kMaxCols; c += kWarp)
                set_column(p, ls, un, c, part, part_row, t, h0 + c, c < heads, 0, 0);
            if (!stream_unit<kSrc>(p, sh, st, src, first, end, lane)) return false;
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
                Source src;
                src.token = 0;
                src.req = __shfl_sync(0xFFFFFFFFu, x.req, a);
                src.lo = __reduce_min_sync(0xFFFFFFFFu, in ? x.lo : INT32_MAX);
                src.hi = __reduce_max_sync(0xFFFFFFFFu, in ? x.hi : -1);
                src.base = p.base_off && src.req >= 0 ? p.base_off[src.req] : 0;
                const int32_t tiles = src.hi < src.lo ? 0 : (src.hi - src.lo) / kTile + 1;
                int32_t first, end;
                share(tiles, part, parts, first, end);
                const int64_t run_row = cut ? part_row + a * p.num_heads : -1;
                if (!unit_slot(sh, st)) return false;
                Unit& un = sh.unit[st.units & 1];
                const int32_t all_lo = __reduce_max_sync(0xFFFFFFFFu, lane >= a && lane < b ? x.lo : INT32_MIN);
                const int32_t all_hi = __reduce_min_sync(0xFFFFFFFFu, lane >= a && lane < b ? x.hi : INT32_MAX);
                if (lane == 0) {
                    un.part = part;
                    un.part_row = run_row;
                    un.all_lo = all_lo;
                    un.all_hi = all_hi;
                }
#pragma unroll
                for (int k = 0; k < kMaxCols / kWarp; ++k) {
                    const int c = lane + k * kWarp;
                    const int tok = a + c / p.num_heads;
                    const int32_t lo = __shfl_sync(0xFFFFFFFFu, x.lo, tok & 31);
                    const int32_t hi = __shfl_sync(0xFFFFFFFFu, x.hi, tok & 31);
                    set_column(p, ls, un, c, part, run_row, t0 + tok, c % p.num_heads, tok < b, lo, hi);
                }
                if (!stream_unit<kSrc>(p, sh, st, src, first, end, lane)) return false;
            }
        }
    }
    if (!tile_slot(sh, st)) return false;
    publish(sh, st, lane, kDone, 0);
    return true;
}

// ---- the MMA thread ------------------------------------------------------------------
//
// Both products take the 128-dim blocks in one order: first those without rope
// dims, from the last one down, then those with rope dims, whose copies take
// longest.  The second product frees them from the last block down, the order
// they are dequantised in.

// The whole warp walks the pipeline, so that descriptors stay in uniform
// registers; one elected lane issues.
template <int N, int D>
__device__ bool issue(Shared& sh, int rope_from, uint32_t k_tile, uint32_t q_tile, uint32_t p_tile,
                      uint32_t tmem) {
    constexpr int kBlocks = D / 128;
    constexpr uint32_t kS = umma_idesc(kTile, N, false), kO = umma_idesc(128, N, true);
    // K-major, 128-byte swizzle: 8-row groups 1024 bytes apart, 32 bytes a step of 16 dims
    const uint64_t k_desc = umma_desc(k_tile, 16, 1024, kSwizzle128);
    const uint64_t q_desc = umma_desc(q_tile, 16, 1024, kSwizzle128);
    // A of the second product: M-major, 128-byte swizzle: 64-dim chunks kChunkBytes apart,
    // 8-row groups 1024 bytes apart.  B: N-major, no swizzle: 8-column groups 2048 bytes
    // apart, 8-row groups 128 bytes apart.
    const uint64_t v_desc = umma_desc(k_tile, kChunkBytes, 1024, kSwizzle128);
    const uint64_t p_desc = umma_desc(p_tile, 128, 2048, kSwizzleNone);
    const uint32_t lead = elect_one();
    uint32_t step = 0;
    for (int seq = 0;; ++seq) {
        const int slot = seq % kTiles;
        if (!wait_all(&sh.tile_full[slot], (seq / kTiles) & 1)) return false;
        const int32_t flags = __shfl_sync(0xFFFFFFFFu, sh.tile[slot].flags, 0);
        if (lead) mbar_arrive(&sh.tile_empty[slot]);
        if (flags & kDone) return true;
        if (flags & kEmpty) continue;
        const auto first_product = [&](int j, bool first) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                umma_bf16(tmem, k_desc + ((j * 2 * kChunkBytes + (k / 4) * kChunkBytes + (k % 4) * 32) >> 4),
                          q_desc + ((j * 2 * (N * 128) + (k / 4) * (N * 128) + (k % 4) * 32) >> 4), kS,
                          !first || k > 0, lead);
        };
#pragma unroll
        for (int j = kBlocks - 1; j >= 0; --j) {  // blocks without rope dims
            if (j >= rope_from) continue;
            if (!wait_all(&sh.full[j], step & 1)) return false;
            tmem_fence_after();
            first_product(j, j == rope_from - 1);
        }
#pragma unroll
        for (int j = kBlocks - 1; j >= 0; --j) {
            if (j < rope_from) break;
            if (!wait_all(&sh.full[j], step & 1)) return false;
            tmem_fence_after();
            first_product(j, rope_from == 0 && j == kBlocks - 1);
        }
        umma_commit(&sh.s_ready, lead);
        if (!wait_all(&sh.p_ready, step & 1)) return false;
        tmem_fence_after();
        const bool first_tile = flags & kFirst;
#pragma unroll
        for (int j = kBlocks - 1; j >= 0; --j) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                umma_bf16(tmem + N + j * N, v_desc + ((j * 2 * kChunkBytes + k * 2048) >> 4),
                          p_desc + ((k * 256) >> 4), kO, !first_tile || k > 0, lead);
            umma_commit(&sh.freed[j], lead);
        }
        ++step;
    }
}

// ---- the worker warps ----------------------------------------------------------------

// 16 E4M3 bytes of UE8M0 scale byte b as eight bf16 pairs, by the rule of the
// gather (E4M3 -> fp16 exactly, binary32 product, rounded to bf16).  Per pair that
// is two conversions on the integer pipe and two on the fp16 one, 2 cycles of a
// scheduler each: placing the bits with shifts and masks and multiplying bf16
// pairs took 3 to 4 operations of the integer pipe per pair.
__device__ __forceinline__ void dequant16(uint4 raw, uint32_t b, uint32_t (&w)[8]) {
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    const uint64_t s2 = splat_f32x2(ue8m0_scale(b));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[2 * i] = scale_f16x2_to_bf16x2(cvt_e4m3x2_to_f16x2(in[i] & 0xFFFFu), s2);
        w[2 * i + 1] = scale_f16x2_to_bf16x2(cvt_e4m3x2_to_f16x2(in[i] >> 16), s2);
    }
}

// Whether any of eight bf16 values is an infinity or a NaN: all exponent bits set.
__device__ __forceinline__ bool any_non_finite(uint4 v) {
    const uint32_t ones = ((v.x & 0x7F807F80u) + 0x00800080u) | ((v.y & 0x7F807F80u) + 0x00800080u) |
                          ((v.z & 0x7F807F80u) + 0x00800080u) | ((v.w & 0x7F807F80u) + 0x00800080u);
    return (ones & 0x80008000u) != 0;
}

// Whether a row of the tile holds a value that is not finite; if so it is cleared, as
// a weight of 0 would not keep it from the columns that do not see the row.
// `flag` is set first, for the warps that look at the row when it is cleared.
template <int D>
__device__ __noinline__ bool clear_bad_row(uint32_t k_tile, int row, volatile uint8_t* flag) {
    bool bad = false;
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) bad |= any_non_finite(lds_v4(k_tile + i / 8 * kChunkBytes + row * 128 + i % 8 * 16));
    if (bad) {
        *flag = 1;
        __threadfence_block();
#pragma unroll 1
        for (int i = 0; i < D / 8; ++i) sts_v4(k_tile + i / 8 * kChunkBytes + row * 128 + i % 8 * 16, 0, 0, 0, 0);
    }
    __threadfence_block();
    return bad || *flag != 0;
}

// 16-byte copy global -> shared; `bytes` 0 writes zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Queries of a unit into the swizzled B tile of the first product; unused
// columns are zero.  Asynchronous.
template <int N, int D, int kWorkers>
__device__ __forceinline__ void load_queries(const AttnParams& p, const Unit& un, uint32_t q_tile, int tid) {
    const int part = tid & 7;
#pragma unroll
    for (int n0 = 0; n0 < N; n0 += kWorkers * kWarp / 8) {
        const int n = n0 + (tid >> 3);
        if (n >= N) break;
        const bool used = un.col_token[n] >= 0;
        const uint16_t* src = used ? p.q + un.col_q[n] + part * 8 : p.q;
        const uint32_t dst = q_tile + n * 128 + ((part ^ (n & 7)) * 16);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) copy16(dst + c * (N * 128), used ? src + c * 64 : src, used ? 16 : 0);
    }
}

// Sum of v[k] over the 32 lanes: lane i gets the sum of column i % K.  Halves the
// columns a lane holds at each exchange (K - 1 shuffles instead of 5 K).
template <int K>
__device__ __forceinline__ float column_sums(float (&v)[K], int lane) {
#pragma unroll
    for (int w = K / 2; w >= 1; w /= 2) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? v[i] : v[i + w];
            v[i] = (up ? v[i + w] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, send, w);
        }
    }
    float x = v[0];
#pragma unroll
    for (int o = K; o < kWarp; o *= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// Dequantisation: a worker warp owns 16 rows of the tile.  A 128-dim block without
// rope dims is read by 8 lanes per row, 16 bytes each, so that a load covers 4
// rows of 128 bytes (a load of 16 rows would take one pass through the L1 tags
// per row); the two 64-dim chunks and two rows are spread over the lanes so
// that every eight of them store to eight different 16-byte banks.
template <int N, int kSrc, int D>
__device__ bool work(const AttnParams& p, const LaunchShape& ls, Shared& sh, uint32_t k_tile,
                     uint32_t q_tile, uint32_t p_tile, uint32_t tmem) {
    constexpr int kWorkers = Roles<N>::kWorkers, kGroups = Roles<N>::kGroups;
    constexpr int NC = N / kGroups;  // columns of a worker warp
    constexpr int kChunks = D / 64, kBlocks = D / 128;
    constexpr int kOwn = kTile / kWorkers;             // rows of a warp
    static_assert(kOwn == 16 || kOwn == 8, "the lane maps below");
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const int quad = warp % 4, group = warp / 4;
    const int srow = quad * kWarp + lane;              // softmax: the tile row of this lane
    const int nope = D - p.rope_dim, fp8_chunks = nope / 64;
    const int rope_from = nope / 128;                  // blocks from here on hold rope dims
    const bool mixed = fp8_chunks % 2 != 0;            // and the first of them E4M3 dims too
    const int own = warp * kOwn;
    // block map: rows b_row + 4 i, 16 bytes at b_byte, in chunk b_chunk of the block
    const int b_row = own + (lane >> 4) * 2 + ((lane >> 2) & 1), b_chunk = (lane >> 3) & 1;
    const int b_byte = b_chunk * 64 + (lane & 3) * 16;
    const uint32_t b_dst = k_tile + b_chunk * kChunkBytes + b_row * 128 + (((2 * (lane & 3)) ^ (b_row & 7)) * 16);
    // chunk map: rows c_row + 8 i, 16 bytes at 16 (lane % 4)
    const int c_row = own + (lane >> 2);
    const uint32_t c_dst = k_tile + c_row * 128 + (((2 * (lane & 3)) ^ (c_row & 7)) * 16);
    // rope map: rows r_row + 4 i, 16 bytes at 16 (lane % 8)
    const int r_row = own + (lane >> 3);
    const uint32_t r_dst = k_tile + r_row * 128 + (((lane & 7) ^ (r_row & 7)) * 16);
    const uint32_t lane_base = tmem + ((uint32_t)(quad * kWarp) << 16) + group * NC;
    float* const aux = sh.aux + warp * NC;  // factors of the columns
    uint32_t step = 0, exchange = 0;

    float l[NC];
    float m_used = -INFINITY;  // of column `lane` of the group, for lane < NC
    constexpr int kFours = kOwn / 4, kEights = kOwn / 8;
    uint4 raw[2][kFours];      // blocks rope_from - 1, rope_from - 2, ... of a lane's rows
    uint4 raw_chunk[kEights];  // the E4M3 chunk of a mixed block
    uint2 scales = make_uint2(0, 0);  // of row own + lane % kOwn

    const auto load_block = [&](const Tile& t, uint4(&x)[kFours], int j) {
        const uint8_t* data[kFours];
#pragma unroll
        for (int i = 0; i < kFours; ++i) data[i] = t.row[b_row + 4 * i].data;
#pragma unroll
        for (int i = 0; i < kFours; ++i) x[i] = ld_nc_v4(data[i] + j * 128 + b_byte);
    };
    // Starts the first loads of a tile.  They are left to the L1, although no byte is read
    // twice: a line holds the ends of two blocks' pieces (304 tokens of 128 heads 152 us
    // against 172 with L1::no_allocate, 1901 ragged tokens 592 against 621, two of 131072
    // rows 103 against 100).
    const auto start = [&](const Tile& t) {
        const uint8_t* sc = t.row[own + lane % kOwn].scales;
        if (D == 512) {
            scales = ld_nc_v2(sc);
        } else if (D == 256) {
            scales.x = ld_nc_u32(sc);
        } else {
            scales.x = ld_nc_u8(sc) | (ld_nc_u8(sc + 1) << 8);
        }
        if (mixed) {
            const uint8_t* data[kEights];
#pragma unroll
            for (int i = 0; i < kEights; ++i) data[i] = t.row[c_row + 8 * i].data;
#pragma unroll
            for (int i = 0; i < kEights; ++i) raw_chunk[i] = ld_nc_v4(data[i] + (fp8_chunks - 1) * 64 + (lane & 3) * 16);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (b < rope_from) load_block(t, raw[b], rope_from - 1 - b);
    };

    if (!wait_all(&sh.tile_full[0], 0)) return false;
    int32_t flags = sh.tile[0].flags;
    if (!(flags & (kDone | kEmpty))) {
        load_queries<N, D, kWorkers>(p, sh.unit[sh.tile[0].unit], q_tile, tid);
        start(sh.tile[0]);
    }
    for (int seq = 0;; ++seq) {
        const int slot = seq % kTiles, nslot = (seq + 1) % kTiles;
        const Tile& tl = sh.tile[slot];
        const Unit& un = sh.unit[tl.unit];
        if (flags & kDone) return true;
        if (flags & kFirst) {
#pragma unroll
            for (int i = 0; i < NC; ++i) l[i] = 0.0f;
            m_used = -INFINITY;
        }
        if (!(flags & kEmpty)) {
            const int buf = step & 1;
            if (lane < kOwn) {
                sh.scales[buf][own + lane] = scales;
                if (kSrc == kTokens) sh.row_bad[buf][own + lane] = 0;
            }
            __syncwarp();
            uint2 row_scales[kFours];  // one 8-byte read per row instead of a byte per block
#pragma unroll
            for (int i = 0; i < kFours; ++i) row_scales[i] = sh.scales[buf][b_row + 4 * i];
            const uint8_t* sc = reinterpret_cast<const uint8_t*>(sh.scales[buf]);
            // ---- dequantisation, from the last dims down
            int block = kBlocks;  // blocks from here on are free
            const auto need = [&](int j) {
                if (j >= block) return true;
                block = j;
                return step == 0 || wait_all(&sh.freed[j], (step - 1) & 1);
            };
            const auto put = [&](uint4 x, uint32_t scale, uint32_t dst) {
                uint32_t w[8];
                dequant16(x, scale, w);
                sts_v4(dst, w[0], w[1], w[2], w[3]);
                sts_v4(dst ^ 16, w[4], w[5], w[6], w[7]);
            };
            if (fp8_chunks < kChunks) {
                const uint8_t* data[kFours];
#pragma unroll
                for (int i = 0; i < kFours; ++i) data[i] = tl.row[r_row + 4 * i].data;
                for (int c = kChunks - 1; c >= fp8_chunks; --c) {  // rope dims: bf16 as stored
                    if (!need(c / 2)) return false;
                    const int at = nope + (c * 64 - nope) * 2 + (lane & 7) * 16;
#pragma unroll
                    for (int i = 0; i < kFours; ++i) {
                        const uint32_t dst = (r_dst + c * kChunkBytes + i * 512) ^ ((i & 1) * 64);
                        copy16(dst, data[i] + at, 16);
                    }
                }
            }
            if (mixed) {
                const int c = fp8_chunks - 1;
                uint32_t scale[kEights];
#pragma unroll
                for (int i = 0; i < kEights; ++i) scale[i] = sc[(c_row + 8 * i) * 8 + c];
                if (!need(c / 2)) return false;
#pragma unroll
                for (int i = 0; i < kEights; ++i)  // 8 rows on, the swizzle is the same
                    put(raw_chunk[i], scale[i], c_dst + c * kChunkBytes + i * 1024);
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int j = rope_from - 1 - b;
                if (j < 0) break;
                uint32_t scale[kFours];
#pragma unroll
                for (int i = 0; i < kFours; ++i)
                    scale[i] = ((j < 2 ? row_scales[i].x : row_scales[i].y) >> (16 * (j & 1) + 8 * b_chunk)) & 0xFFu;
                if (!need(j)) return false;
#pragma unroll
                for (int i = 0; i < kFours; ++i)  // 4 rows on, bit 2 of the swizzle turns
                    put(raw[b % 2][i], scale[i], (b_dst + j * 2 * kChunkBytes + i * 512) ^ ((i & 1) * 64));
                if (j >= 2) load_block(tl, raw[b % 2], j - 2);
                if (b == 0 && (flags & kFirst)) copies_done();  // hands over the unit's queries too
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.full[j]);
            }
            if (rope_from < kBlocks) {
                copies_done();
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    for (int j = rope_from; j < kBlocks; ++j) mbar_arrive(&sh.full[j]);
            }
        }
        // ---- the next tile's loads, in flight during the softmax
        if (!wait_all(&sh.tile_full[nslot], ((seq + 1) / kTiles) & 1)) return false;
        const int32_t next_flags = sh.tile[nslot].flags;
        const bool next_rows = !(next_flags & (kDone | kEmpty));
        if (next_rows) start(sh.tile[nslot]);

        if (!(flags & kEmpty)) {
            // ---- softmax of the tile: this lane's row, NC columns
            const int buf = step & 1;
            if (!wait_all(&sh.s_ready, step & 1)) return false;
            tmem_fence_after();
            float s[NC];
            tmem_ld<NC>(lane_base, s);
            const bool ok = tl.row[srow].data != reinterpret_cast<const uint8_t*>(g_zero_row);
            if (kSrc == kTokens) {
                // A row with an infinity or a NaN gives none but such scores, whatever the query.
                float z = 0.0f;
#pragma unroll
                for (int k = 0; k < NC; ++k) z = fmaf(s[k], 0.0f, z);
                bool bad = false;
                if (__any_sync(0xFFFFFFFFu, z != 0.0f)) {
                    // every worker has handed over its share of the tile
                    if (!wait_all(&sh.full[0], step & 1)) return false;
                    if (rope_from < kBlocks && !wait_all(&sh.full[kBlocks - 1], step & 1)) return false;
                    if (z != 0.0f) bad = clear_bad_row<D>(k_tile, srow, &sh.row_bad[buf][srow]);
                    __syncwarp();
                }
                const int32_t pos = tl.pos + srow;
                if (!__all_sync(0xFFFFFFFFu, ok && !bad && pos >= un.all_lo && pos <= un.all_hi)) {
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        const bool see = ok && pos >= un.col_lo[group * NC + k] && pos <= un.col_hi[group * NC + k];
                        s[k] = see ? (bad ? NAN : s[k]) : -INFINITY;
                    }
                }
            } else if (!__all_sync(0xFFFFFFFFu, ok)) {
#pragma unroll
                for (int k = 0; k < NC; ++k) s[k] = ok ? s[k] : -INFINITY;
            }
            // The reference of a column only has to lie near its maximum: it is set by
            // the first tile and raised where a score lies far above it, which the
            // group's four warps have to agree on.
            bool raise = flags & kFirst;
            float* ref = sh.ref + warp * NC;
            if (!raise) {
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < NC; k += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(&ref[k]);
                    top = fmaxf(top, fmaf(s[k], ls.scale_log2, -m.x));
                    top = fmaxf(top, fmaf(s[k + 1], ls.scale_log2, -m.y));
                    top = fmaxf(top, fmaf(s[k + 2], ls.scale_log2, -m.z));
                    top = fmaxf(top, fmaf(s[k + 3], ls.scale_log2, -m.w));
                }
                const bool over = __any_sync(0xFFFFFFFFu, top > kLazy);
                int32_t(&flag)[4] = sh.over[group][exchange & 1];
                if (lane == 0) {
                    flag[quad] = over;
                    mbar_arrive(&sh.group_bar[group]);
                }
                if (!wait_all(&sh.group_bar[group], exchange & 1)) return false;
                ++exchange;
                raise = flag[0] | flag[1] | flag[2] | flag[3];
            }
            if (raise) {
                float* red = sh.red[exchange & 1][quad] + group * NC;
#pragma unroll
                for (int k = 0; k < NC; k += 4) {
                    const float x0 = warp_max(s[k]), x1 = warp_max(s[k + 1]);
                    const float x2 = warp_max(s[k + 2]), x3 = warp_max(s[k + 3]);
                    if (lane == 0) *reinterpret_cast<float4*>(&red[k]) = make_float4(x0, x1, x2, x3);
                }
                if (lane == 0) mbar_arrive(&sh.group_bar[group]);
                if (!wait_all(&sh.group_bar[group], exchange & 1)) return false;
                if (lane < NC) {
                    const float(&all)[4][kMaxCols] = sh.red[exchange & 1];
                    const int c = group * NC + lane;
                    const float top = ls.scale_log2 * fmaxf(fmaxf(all[0][c], all[1][c]), fmaxf(all[2][c], all[3][c]));
                    float alpha = 1.0f;
                    if (top > m_used) {
                        alpha = m_used == -INFINITY ? 1.0f : ex2_approx(m_used - top);  // no sums before
                        m_used = top;
                    }
                    // A score past binary32 makes the column NaN; fma(s, scale, -infinity) of a
                    // finite s would be -infinity, a weight of 0.
                    ref[lane] = m_used == -INFINITY ? kNone : m_used == INFINITY ? NAN : m_used;
                    aux[lane] = alpha;
                }
                ++exchange;
                __syncwarp();
                if (!(flags & kFirst)) {
                    // the previous tile's second product is done: s_ready came after it
#pragma unroll
                    for (int k = 0; k < NC; ++k) l[k] *= aux[k];
#pragma unroll 1  // rare: short code, few registers
                    for (int j = 0; j < kBlocks; ++j) {
#pragma unroll 1
                        for (int k0 = 0; k0 < NC; k0 += 8) {
                            float o[8];
                            tmem_ld<8>(lane_base + N + j * N + k0, o);
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] *= aux[k0 + k];
                            tmem_st8(lane_base + N + j * N + k0, o);
                        }
                    }
                    tmem_wait_st();
                }
            }
            // weights to the N-major B tile: 8 columns (16 bytes) of a row, rows side by side
#pragma unroll
            for (int k = 0; k < NC; k += 8) {
                const float4 m0 = *reinterpret_cast<const float4*>(&ref[k]);
                const float4 m1 = *reinterpret_cast<const float4*>(&ref[k + 4]);
                const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[k + i] = ex2_approx(fmaf(s[k + i], ls.scale_log2, -m[i]));
                    l[k + i] += s[k + i];
                }
                sts_v4(p_tile + (group * NC + k) / 8 * (kTile * 16) + srow * 16,
                       pack_bf16x2(s[k], s[k + 1]), pack_bf16x2(s[k + 2], s[k + 3]),
                       pack_bf16x2(s[k + 4], s[k + 5]), pack_bf16x2(s[k + 6], s[k + 7]));
            }
            fence_async_smem();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_ready);
            ++step;
        }
        if (flags & kLast) {
            // the first product of this unit is done with its queries
            if (next_rows) load_queries<N, D, kWorkers>(p, sh.unit[sh.tile[nslot].unit], q_tile, tid);
            // ---- the unit's sums: over the lanes, then over the group's four warps
            const float mine = column_sums(l, lane);
            float(&red)[4][kMaxCols] = sh.red[exchange & 1];
            if (lane < NC) red[quad][group * NC + lane] = mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.group_bar[group]);
            if (!wait_all(&sh.group_bar[group], exchange & 1)) return false;
            ++exchange;
            if (lane < NC) {
                const int n = group * NC + lane;
                const float total = (red[0][n] + red[1][n]) + (red[2][n] + red[3][n]);
                const int32_t t = un.col_token[n], h = un.col_head[n];
                float inv = 1.0f;
                if (t >= 0) {
                    if (un.part_row >= 0) {
                        if (kSrc != kTokens && ls.cluster) {
                            if (quad == 0) sh.part_ml[n] = make_float2(m_used, total);
                        } else if (quad == 0) {
                            float* ml = ls.part_ml + ((un.part_row + n) * ls.splits + un.part) * 2;
                            ml[0] = m_used;
                            ml[1] = total;
                        }
                    } else {
                        const float m = m_used == -INFINITY ? 0.0f : m_used;
                        const float den = total + ex2_approx(un.col_sink[n] - m);
                        inv = total == 0.0f ? 0.0f : 1.0f / den;
                        if (p.lse && quad == 0)
                            p.lse[(int64_t)t * p.lse_stride_t + h] =
                                total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2;
                    }
                }
                aux[lane] = inv;
            }
            __syncwarp();
            if (!(flags & kEmpty)) {
                if (!wait_all(&sh.freed[0], (step - 1) & 1)) return false;  // the last block
                tmem_fence_after();
            }
            if (kSrc != kTokens && ls.cluster) {
                // in place of the tile, which the products are done with: [column][dim]
                for (int j = 0; j < kBlocks; ++j) {
                    float o[NC];
#pragma unroll
                    for (int k = 0; k < NC; ++k) o[k] = 0.0f;
                    if (!(flags & kEmpty)) tmem_ld<NC>(lane_base + N + j * N, o);
#pragma unroll
                    for (int k = 0; k < NC; ++k)
                        sts_f32(k_tile + ((group * NC + k) * D + j * 128 + srow) * 4, o[k]);
                }
            } else if (un.part_row >= 0) {
                for (int j = 0; j < kBlocks; ++j) {
                    float o[NC];
#pragma unroll
                    for (int k = 0; k < NC; ++k) o[k] = 0.0f;
                    if (!(flags & kEmpty)) tmem_ld<NC>(lane_base + N + j * N, o);
                    const int d = j * 128 + srow;
#pragma unroll
                    for (int k0 = 0; k0 < NC; k0 += 8) {
                        int64_t at[8];
                        bool used[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            at[k] = un.col_out[group * NC + k0 + k] + d;
                            used[k] = un.col_token[group * NC + k0 + k] >= 0;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (used[k]) ls.part_o[at[k]] = o[k0 + k];
                    }
                }
            } else {
                // 4 x 4 exchanges among four lanes: each then holds four dims of the columns
                // k + lane % 4, where it stores them
                uint16_t* dst[NC / 4];
#pragma unroll
                for (int k = 0; k < NC / 4; ++k) {
                    const int n = group * NC + 4 * k + (lane & 3);
                    dst[k] = un.col_token[n] >= 0 ? p.out + un.col_out[n] + (srow & ~3) : nullptr;
                }
                // first the pairs of columns (with lane ^ 2), then the halves of the pairs
                const bool upper = lane & 2;
                const uint32_t low = upper ? 0x1054u : 0x5410u, high = upper ? 0x3276u : 0x7632u;
                const uint32_t keep = lane & 1 ? high : low, send = lane & 1 ? low : high;
                const uint32_t dims01 = lane & 1 ? 0x1054u : 0x5410u, dims23 = lane & 1 ? 0x3276u : 0x7632u;
                for (int j = 0; j < kBlocks; ++j) {
                    float o[NC];
#pragma unroll
                    for (int k = 0; k < NC; ++k) o[k] = 0.0f;
                    if (!(flags & kEmpty)) tmem_ld<NC>(lane_base + N + j * N, o);
#pragma unroll
                    for (int k = 0; k < NC / 4; ++k) {
                        const float4 inv = *reinterpret_cast<const float4*>(&aux[4 * k]);
                        const uint32_t w0 = pack_bf16x2(o[4 * k] * inv.x, o[4 * k + 1] * inv.y);
                        const uint32_t w1 = pack_bf16x2(o[4 * k + 2] * inv.z, o[4 * k + 3] * inv.w);
                        const uint32_t x = upper ? w1 : w0;
                        const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, upper ? w0 : w1, 2);
                        const uint32_t u = __byte_perm(x, y, keep);
                        const uint32_t v = __shfl_xor_sync(0xFFFFFFFFu, __byte_perm(x, y, send), 1);
                        if (dst[k] != nullptr)
                            st_v2(dst[k] + j * 128, make_uint2(__byte_perm(u, v, dims01), __byte_perm(u, v, dims23)));
                    }
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.unit_empty[tl.unit]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.tile_empty[slot]);
        flags = next_flags;
    }
}

// ---- joining the parts of a unit in a cluster -------------------------------------------
//
// The formula of attention_join_kernel, for few parts (kMostParts): their O^T stay in
// shared memory, and each CTA joins every splits-th column, a thread four dims of it.
// Bound by the latency of the other CTAs' shared memory, hence several columns at once.
template <int kCols, int D, int kWorking>
__device__ __forceinline__ void join_in_cluster(const AttnParams& p, const LaunchShape& ls, Shared& sh,
                                                uint32_t k_tile) {
    const Unit& un = sh.unit[0];
    const int S = ls.splits, rank = (int)(blockIdx.x % S);
    constexpr int kPer = D / 4, kAtOnce = kCols / 16;  // threads of a column; columns a thread has in work
    const int d = (int)threadIdx.x % kPer * 4, step = kWorking / kPer * S;
    for (int c0 = rank + (int)threadIdx.x / kPer * S; c0 < ls.heads_per_unit; c0 += kAtOnce * step) {
        float2 ml[kAtOnce][kMostParts];
        float ref[kAtOnce], total[kAtOnce];
        float4 a[kAtOnce];
#pragma unroll
        for (int i = 0; i < kMostParts; ++i)
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int c = min(c0 + u * step, kCols - 1);  // columns not in use are not stored
                ml[u][i] = make_float2(-INFINITY, 0.0f);
                if (i < S) ml[u][i] = ld_cluster_f32x2(smem_u32(&sh.part_ml[c]), i);
            }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < kMostParts; ++i) m = fmaxf(m, ml[u][i].x);
            ref[u] = m == -INFINITY ? 0.0f : m;
            total[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < kMostParts; ++i) {
                ml[u][i].x = ex2_approx(ml[u][i].x - ref[u]);
                total[u] += ml[u][i].x * ml[u][i].y;
            }
            a[u] = make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kMostParts; ++i) {
            if (i >= S) break;
            float4 v[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
                v[u] = ld_cluster_f32x4(k_tile + (min(c0 + u * step, kCols - 1) * D + d) * 4, i);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                a[u].x += ml[u][i].x * v[u].x;
                a[u].y += ml[u][i].x * v[u].y;
                a[u].z += ml[u][i].x * v[u].z;
                a[u].w += ml[u][i].x * v[u].w;
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int c = c0 + u * step;
            if (c >= ls.heads_per_unit || un.col_token[c] < 0) continue;
            const int64_t t = un.col_token[c], h = un.col_head[c];
            const float den = total[u] + ex2_approx(un.col_sink[c] - ref[u]);
            const float inv = total[u] == 0.0f ? 0.0f : 1.0f / den;
            st_v2(p.out + t * p.out_stride_t + h * p.out_stride_h + d,
                  make_uint2(pack_bf16x2(a[u].x * inv, a[u].y * inv), pack_bf16x2(a[u].z * inv, a[u].w * inv)));
            if (p.lse && d == 0)
                p.lse[t * p.lse_stride_t + h] = total[u] == 0.0f ? -INFINITY : (ref[u] + log2f(total[u])) * kLn2;
        }
    }
}

constexpr size_t kAlign = 1024;

size_t smem_bytes(int n, int head_dim) {
    return kAlign + (size_t)head_dim / 64 * kChunkBytes + (size_t)head_dim / 64 * n * 128 +
           (size_t)n / 8 * kTile * 16 + sizeof(Shared);
}

template <int N, int kSrc, int D>
__global__ void __launch_bounds__(Roles<N>::kThreads, 1)
    attention_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ LaunchShape ls) {
    constexpr int kWorkers = Roles<N>::kWorkers, kGroups = Roles<N>::kGroups;
    constexpr int kMmaWarp = Roles<N>::kMmaWarp, kPlanWarp = Roles<N>::kPlanWarp;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((kAlign - (smem_u32(smem_raw) & (kAlign - 1))) & (kAlign - 1));
    uint8_t* k_tile = base;
    uint8_t* q_tile = k_tile + D / 64 * kChunkBytes;
    uint8_t* p_tile = q_tile + D / 64 * (N * 128);
    Shared& sh = *reinterpret_cast<Shared*>(p_tile + N / 8 * kTile * 16);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.unit_empty[i], kWorkers);
        }
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&sh.tile_full[i], 1);
            mbar_init(&sh.tile_empty[i], kWorkers + 1);
        }
        for (int i = 0; i < kMaxBlocks; ++i) {
            mbar_init(&sh.full[i], kWorkers);
            mbar_init(&sh.freed[i], 1);
        }
        mbar_init(&sh.s_ready, 1);
        mbar_init(&sh.p_ready, kWorkers);
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < kGroups; ++i) mbar_init(&sh.group_bar[i], 4);
        sh.failed = 0;
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
        ok = work<N, kSrc, D>(p, ls, sh, smem_u32(k_tile), smem_u32(q_tile), smem_u32(p_tile), tmem);
    } else if (warp == kPlanWarp) {
        ok = plan<kSrc>(p, ls, sh);
    } else {
        ok = issue<N, D>(sh, (D - p.rope_dim) / 128, smem_u32(k_tile), smem_u32(q_tile), smem_u32(p_tile), tmem);
        if (!ok) {  // wait for the MMAs in flight before the operands go
            umma_commit(&sh.drain, elect_one());
            mbar_poll_bounded(&sh.drain, 0, kWaitLimitNs);
        }
    }
    if (!ok && lane == 0) atomicAdd(&g_attn_wait_timeouts, 1u);
    if (kSrc != kTokens && ls.cluster) {
        // every CTA comes to both barriers, also one whose waits expired
        if (!ok) sh.failed = 1;
        __syncwarp();
        cluster_sync();
        if (warp < kWorkers && !sh.failed) join_in_cluster<N, D, kWorkers * kWarp>(p, ls, sh, smem_u32(k_tile));
        cluster_sync();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, ls.tmem_cols);
}

// ---- joining the parts of a split row ----------------------------------------------------
//
// out = sum_i 2^(m_i - m) o_i / (sum_i 2^(m_i - m) l_i + 2^(sink' - m)), m = max m_i
// (log2 units).  One CTA per column of a cut unit; a thread takes four dims, so the
// parts are read as whole rows.  Bound by the bytes of the parts; two requests of 64
// heads in 76 parts each: 20 MB from L2.
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnParams p, const LaunchShape ls) {
    extern __shared__ float s_ml[];
    const int64_t th = blockIdx.x;
    int32_t h;
    int64_t t;
    if (ls.tokens_per_unit > 1) {
        t = ls.whole * ls.tokens_per_unit + th / p.num_heads;
        h = (int32_t)(th % p.num_heads);
    } else {
        const int64_t v = ls.whole + th / ls.heads_per_unit;
        t = v / ls.head_groups;
        h = (int32_t)(v % ls.head_groups) * ls.heads_per_unit + (int32_t)(th % ls.heads_per_unit);
    }
    if (t >= p.num_tokens || h >= p.num_heads) return;  // columns not in use
    pdl_wait();
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
    // Neighbouring tokens of a request share a unit, and with it the tiles, where few
    // heads leave room and requests bring enough tokens that units seldom end at their
    // boundaries.  64 requests, contexts up to 8192, 16 heads: 4 tokens a request 227 us
    // against 287 with one token a unit, 3 259 against 233; 32 heads, two tokens a unit:
    // 6 tokens a request 412 against 518, 4 354 against 325.  Not where windows are so
    // short that the shared tiles are no fewer (32 heads, a window of 128, 4096 tokens:
    // 184 us against 153).
    const auto tiles_of = [](int64_t keys) { return keys / kTile + (keys % kTile != 0); };
    const int64_t tiles = tiles_of(max_keys);
    if (!indexed && num_heads <= kMaxCols / 2) {
        const int32_t n = kMaxCols / num_heads < kWarp ? kMaxCols / num_heads : kWarp;
        if (num_tokens >= (n < 4 ? 6 : 4) * (int64_t)num_reqs && tiles_of(max_keys + n - 1) < n * tiles) {
            ls.tokens_per_unit = n;
            cols = n * num_heads;
            pl.src = kTokens;
        }
    }
    pl.n = cols <= 16 ? 16 : cols <= 32 ? 32 : 64;
    const int64_t base = (num_tokens + ls.tokens_per_unit - 1) / ls.tokens_per_unit * ls.head_groups;
    // Units are cut along their tiles to fill the SMs evenly.  In the index form all
    // are of one length: whole rounds of them stay whole, and the rest is cut until it
    // fills the SMs too (634 units of 9 tiles on 152 SMs: 191 us against 205 uncut).  In
    // the position form lengths differ from request to request: about four parts per SM
    // (32 requests of 8 tokens, contexts up to 8192: one per SM 253 us, two 238, four 196,
    // eight 195; 32 of 32 tokens 1013, 1012, 779, 823), of eight tiles or more; very few
    // units are cut into one part per SM (two requests of 131072 rows: 100 us, four per
    // SM 130).  The tiles are those the table has room for, the lengths being on the device:
    // parts behind a short context's tiles are empty, write zeros and are joined all the same
    // (figures of wide tables at chunk_mla_attention in psk.h).
    const int64_t sms = sm_count();
    int64_t rest = base, splits;
    if (indexed) {
        rest = base % sms;
        splits = rest > 0 ? sms / rest : 1;
    } else {
        splits = sms / base;
        if (base * 8 > sms) {
            const int64_t most = tiles / 8 > splits ? tiles / 8 : splits;
            splits = (4 * sms + base - 1) / base;
            if (splits > most) splits = most;
        }
    }
    if (splits > tiles) splits = tiles;
    if (splits <= 1) {
        splits = 1;
        rest = 0;
    }
    ls.whole = base - rest;
    ls.splits = (int32_t)splits;
    ls.units = ls.whole + rest * splits;
    ls.part_rows = rest * ls.heads_per_unit * ls.tokens_per_unit;
    // Few parts, one to a CTA, are joined in a cluster, which saves a launch and the
    // workspace (4 us of the host's time): pairs of parts (64 tokens of 64 heads 23.6 us
    // against 26.8 with the second kernel, 76 24.0 against 27.9), and up to eight parts of
    // 16 columns (one token of 16 heads 11.1 against 10.7 of device time).  Five parts of
    // 64 columns take 17.4 against 13.4, as each CTA then reads 130 KB from the others.  At
    // most 64 SMs in clusters of more than two: what a GPC has left over cannot take part
    // (30 units of 16 columns in 150 CTAs 22.0 us against 14.0).
    ls.cluster = pl.src != kTokens && ls.whole == 0 && splits > 1 && splits <= kMostParts && ls.units <= sms &&
                 (splits == 2 || (pl.n == 16 && ls.units <= 64));
    const uint32_t need = (uint32_t)pl.n * (1 + head_dim / 128);
    ls.tmem_cols = 32;
    while (ls.tmem_cols < need) ls.tmem_cols *= 2;
    return pl;
}

int64_t part_bytes(const LaunchShape& ls, int32_t head_dim) {
    return ls.cluster ? 0 : (ls.part_rows * ls.splits * (head_dim + 2) * (int64_t)sizeof(float) + 15) / 16 * 16;
}

template <int N, int kSrc, int D>
cudaError_t launch(const AttnParams& p, const LaunchShape& ls, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const int smem = (int)smem_bytes(N, D);
    const cudaError_t e = set_smem_limit_per_device(attention_kernel<N, kSrc, D>, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t grid = ls.units < sm_count() ? ls.units : sm_count();
    return launch_pdl_clusters(attention_kernel<N, kSrc, D>, ls.cluster ? ls.splits : 1, dim3((unsigned)grid),
                               dim3(Roles<N>::kThreads), smem, stream, p, ls);
}

template <int kSrc, int D>
cudaError_t launch_n(const AttnParams& p, const Plan& pl, cudaStream_t stream) {
    if constexpr (kSrc != kTokens) {  // several tokens fill more than 16 columns
        if (pl.n == 16) return launch<16, kSrc, D>(p, pl.ls, stream);
    }
    return pl.n == 32 ? launch<32, kSrc, D>(p, pl.ls, stream) : launch<64, kSrc, D>(p, pl.ls, stream);
}

template <int kSrc>
cudaError_t launch_d(const AttnParams& p, const Plan& pl, cudaStream_t stream) {
    return p.head_dim == 512 ? launch_n<kSrc, 512>(p, pl, stream)
                             : p.head_dim == 256 ? launch_n<kSrc, 256>(p, pl, stream) : launch_n<kSrc, 128>(p, pl, stream);
}

cudaError_t run(AttnParams p, int64_t max_keys, bool indexed, cudaStream_t stream) {
    Plan pl = make_plan(p.num_tokens, p.num_heads, p.head_dim, max_keys, indexed, p.num_reqs);
    p.cache.shift = log2_if_pow2(p.cache.block_size);
    p.extra.shift = log2_if_pow2(p.extra.block_size);
    pl.ls.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
    pl.ls.part_o = static_cast<float*>(p.workspace);
    pl.ls.part_ml = pl.ls.part_o + pl.ls.part_rows * pl.ls.splits * p.head_dim;
    cudaError_t e = pl.src == kIndexed ? launch_d<kIndexed>(p, pl, stream)
                    : pl.src == kOneToken ? launch_d<kOneToken>(p, pl, stream)
                                          : launch_d<kTokens>(p, pl, stream);
    if (e != cudaSuccess || pl.ls.splits == 1 || pl.ls.cluster) return e;
    return launch_pdl(attention_join_kernel, dim3((unsigned)pl.ls.part_rows), dim3(128),
                      (size_t)pl.ls.splits * 2 * sizeof(float), stream, p, pl.ls);
}

}  // namespace

int64_t attention_workspace_bytes(int64_t num_tokens, int32_t num_heads, int32_t head_dim, int64_t max_keys,
                                  bool indexed, int32_t num_reqs) {
    const Plan pl = make_plan(num_tokens, num_heads, head_dim, max_keys, indexed, num_reqs);
    return part_bytes(pl.ls, head_dim);
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
