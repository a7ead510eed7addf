// attn_weights.cu -- attention weights summed per cached row over new tokens and
// heads, on the 5th-generation tensor cores: what eviction ranks rows by.
//
//   sum_j = sum over tokens t that see row j, heads h, of exp(s_thj - L_th)
//   s = scale q.k_j,  L = log(exp(lse) + exp(sink)),  out_j = decay w_j + sum_j
//
// Layout.  A tile is 128 rows of a request, a column a (token, head) of it, and a
// column tile up to 128 columns: whole tokens of few heads, or a part of many heads.
//   S^T [128 rows x N columns] = K [128 x D] Q^T         (D/16 MMAs of M = 128)
// The logarithms are known, so a score becomes a weight by one fused multiply-add and
// one exp2, and a row's sum is a sum along a lane of tensor memory: nothing passes
// between threads until the tile ends.  K is dequantised into tensor memory (D/2 columns,
// two bf16 each) and is the MMAs' A operand from there, so that shared memory carries
// only the queries (a K tile there would be read again by every column tile: 128 bytes
// a cycle, all there is), and stays while the column tiles of its rows go by.  Scores
// have the other columns, two column tiles.
//
// Work.  Tiles and their column tiles stand in one sequence over all requests (a tile
// counts kTileCost column tiles besides, its dequantisation), which is cut into one
// equal range per CTA whatever the lengths are.  A tile cut between CTAs has its partial
// sums written to the workspace; a second kernel adds them up in order.  Tiles that no token sees
// rows of (before the windows, or of requests without tokens) go as runs to the warps that
// sum up, which fade their rows: 1048576 rows 9.3 us, where the planning warp took 77 and
// held the others up (for as long as a wait lasts from 75 GB of weights on).
//
// Roles.  One warp plans: it walks the CTA's range and puts tiles with the addresses of
// their rows into a ring.  Worker warps bring records into shared memory by
// asynchronous copies (32 rows and a part of the dims each, a copy of the next tile issued as
// soon as a block of 64 dims is read), dequantise them and write them to tensor memory; one
// warp fetches queries by TMA into a ring of 128-dim stages, one to four prepare the columns'
// logarithms and bounds; one issues the MMAs; others turn scores into sums.  Queries stay in
// the ring while the column tile does not change (a decode batch: one column tile per
// request).  Every wait is bounded (2 s of wall time, counted in psk_device_wait_timeouts).
//
// Pairs.  Where requests bring many columns, two CTAs share a tile of 256 rows (MMAs of M =
// 256, issued by the first): each has 128 of the rows in its own tensor memory and fetches half
// of each column tile's queries, which halves the bytes of queries per row and lets the
// ring hold two column tiles.
//
// What bounds it.  4096 tokens of 128 heads (1.1 TFLOP): 859 us, 1285 TFLOP/s; the tensor pipe is
// 71 % in use at the 1.6 GHz that the power limit leaves (cuBLAS: 1734 TFLOP/s sustained).  The
// rest is queries: 4.3 GB of them pass through L2 and 4.0 GB come from memory, at 4.7 TB/s, as
// CTAs are at different columns at a time.  203 tokens of 40 heads of 5 requests, over
// 11061 to 30023 rows: 166 us, 1350 TFLOP/s.  64 single tokens of 64 heads, over
// up to 8192 rows: 50 to 55 us from one machine to another for 177 MB, over 8192 rows each 75 us
// for 306 MB, 4.1 TB/s of the 6.7 measured.  A tile takes some 5000 cycles, of which
// dequantising it is 2000 issue slots of each scheduler; the first one's sums come after 30000:
// 17000 until the planning warp has found the range and published two tiles, mostly code that
// is not in the instruction cache yet, then all SMs' first records at once.  One token
// of 16 heads over 8192 rows: 9.6 us.
//
// Measured on the way, by cases as above (64 single tokens; last tokens; 4096 tokens):
//  * each role walking the sequence by itself, one warp for queries and columns: 76, 536, 1784;
//  * columns prepared by four warps: 103, 314, 1253; a planning warp: 67, 211, 1029;
//  * pairs, with a release of the cluster's scope on each hand-over: 69, 344, 1054, and
//    without: 69, 191, 935; stages of 128 dims instead of 64: 66, 186, 895;
//  * 16 dequantising warps instead of 8: 69 with the loops of the other roles unrolled,
//    as each passes its code once a tile and finds it gone from the instruction cache; 58 with
//    short loops and one barrier per block of all parts.
#include <cuda.h>

#include <atomic>
#include <cmath>

#include "attn_weights.h"
#include "psk_common.cuh"
#include "umma.cuh"

namespace psk {
namespace {

constexpr int kTile = 128;          // rows of a CTA's part of a tile
constexpr int kCols = 128;          // columns of a column tile, at most
// Warps by role.  A CTA of its own has few columns per row and many tiles: at head_dim 512 16
// warps dequantise and 4 sum up (64 single tokens of 64 heads over 8192 rows 81 us, 8 and 4 92,
// 16 and 8 91), at 256 8 and 4 (60 us, 16 and 4 68).  A pair has many columns: 8 and 8 (203 tokens
// of 40 heads of 5 requests 165 us, 16 and 8 184, 16 and 4 237).  Few warps for the columns leave
// the others registers: at head_dim 512 one instead of two or four 75, 76 and 79 us (up to 8192
// rows 55, 57 and 60), at 256 57, 53 and 53.
template <int kHeadDim, bool kTwo>
struct Roles {
    static constexpr int D = kHeadDim;
    static constexpr bool kPair = kTwo;
    static constexpr int kWorkers = !kPair && D == 512 ? 16 : 8, kParts = kWorkers / 4;  // each has D / kParts dims
    static constexpr int kSummers = kPair ? 8 : 4, kShares = kSummers / 4;              // of the columns
    static constexpr int kColumnWarps = kPair ? 4 : D == 512 ? 1 : 2;
    static constexpr int kColumnWarp = kWorkers + kSummers, kQueryWarp = kColumnWarp + kColumnWarps;
    static constexpr int kMmaWarp = kQueryWarp + 1, kPlanWarp = kMmaWarp + 1;
    static constexpr int kThreads = (kPlanWarp + 1) * kWarp;
};
constexpr int kMostParts = 4, kMostWarps = 32;
constexpr int kTileCost = 1;
constexpr int kMostStages = 12;
constexpr int kColSlots = 3;
constexpr int kTiles = 4;           // tiles the planning warp may be ahead
constexpr int kMostBlocks = 4;      // 64-dim blocks of a part
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ unsigned int g_weights_wait_timeouts = 0;

// What a row without a page is read from: the longest record, all zero.
__device__ const uint4 g_zero_row[(512 + 448) / 16] = {};

// A request's share of the call.
struct Request {
    int32_t tokens;   // new tokens, and the first of them
    int32_t token0;
    int32_t row0;     // row of its first new token (negative: before row 0)
    int32_t end;      // rows that have a weight
    int32_t replay;
    int32_t base;
};

// The parts of a cut tile: which tile a CTA starts in the middle of, and what it does there.
enum { kNone = 0, kMiddle = 1, kEnds = 2, kEmptyRange = 3 };
struct Record {
    int32_t kind, request, tile, pad;
};

struct Columns {
    float log[kCols];                 // log2 units
    int32_t lo[kCols], hi[kCols];     // rows a column sees
    // by 32 columns: rows that every one in use sees, and which are in use
    int4 all_lo, all_hi, all_used;
};

struct Row {
    const uint8_t* data;
    const uint8_t* scales;
};

// A step of the walk, as the planning warp publishes it.
struct Tile {
    int32_t request;          // -1: the end
    int32_t first_row, end;   // its first row; the rows of the request that have a weight
    int32_t first, total;     // first token group and number of its column tiles
    int32_t c0, c1;           // those of them that are this CTA's; both 0: rows first_row to end have none
    int32_t tokens, token0, row0, replay;  // of the request
    int32_t kept, keeps;      // the first column tile is at hand; the last one is the next tile's first
    uint32_t there[4];        // rows with a page
    Row row[kTile];
};

// Division of n in [0, 2^31) by a divisor fixed for the call: with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1 the quotient is (hi(n m) + n) >> s.
struct Divisor {
    uint32_t mul, shift;
};

__device__ __forceinline__ int32_t divide(int32_t n, Divisor d) {
    return (int32_t)(((uint64_t)__umulhi((uint32_t)n, d.mul) + (uint32_t)n) >> d.shift);
}

Divisor divisor(int32_t d) {
    Divisor x{0, 0};
    while ((1ll << x.shift) < d) ++x.shift;
    x.mul = (uint32_t)((((1ull << x.shift) - (uint64_t)d) << 32) / (uint64_t)d + 1);
    return x;
}

struct LaunchShape {
    int32_t ranks;                // CTAs that share a tile, 1 or 2
    int32_t row_shift;            // log2 of a tile's rows
    int32_t heads, tokens;        // of a column tile
    int32_t head_groups;
    Divisor by_tokens, by_groups; // of those two
    int32_t box_heads, box_tokens;  // of what a CTA fetches of it
    int32_t box_cols;             // columns of that, padded
    int32_t by_heads;             // two CTAs: they fetch the halves of the heads, else of the tokens
    int32_t staging_bytes;
    int32_t stages, stage_bytes;  // stages of two boxes of 64 dims
    int32_t keep_queries;         // the ring holds a whole column tile
    int32_t stride[kMostParts];   // bytes of a staged row, by part of the dims
    float scale_log2;
    float* parts;                 // [CTA][2][kTile]
    Record* records;              // [CTA]
};

struct Shared {
    Tile tile[kTiles];
    Columns columns[kColSlots];
    float half_sum[4][2][kWarp];  // second half of a quad's columns: sum and compensation
    uint64_t tile_full[kTiles], tile_free[kTiles];
    uint64_t k_full[kMostBlocks], k_free[kMostBlocks];  // by number of the block in its part
    uint64_t q_full[kMostStages], q_free[kMostStages];
    uint64_t col_full[kColSlots], col_free[kColSlots];
    uint64_t s_full[2], s_free[2];
    uint64_t half_full[4], half_free[4];
    uint64_t drain;
    int64_t scan[kMostWarps];
    int64_t first_at;             // where the CTA's range starts: prefix of that request
    int32_t first_request;
    uint32_t tmem;
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_poll_bounded(bar, parity, kWaitLimitNs);
    return __all_sync(0xFFFFFFFFu, ok);
}

// ---- the sequence of tiles --------------------------------------------------------------

__device__ __forceinline__ Request load_request(const WeightParams& p, int32_t r) {
    Request x;
    const int32_t rows = p.seq_lens[r];
    const int64_t q0 = p.qsl[r], q1 = p.qsl[r + 1];
    const int64_t first = q0 > 0 ? q0 : 0, last = q1 < p.num_tokens ? q1 : p.num_tokens;
    x.tokens = last > first ? (int32_t)(last - first) : 0;
    x.token0 = (int32_t)first;
    const int64_t row0 = (int64_t)rows - (q1 - q0) + (first - q0);
    x.row0 = (int32_t)(row0 < -(1 << 30) ? -(1 << 30) : row0 > INT32_MAX ? INT32_MAX : row0);
    x.end = rows < 0 ? 0 : rows < p.width ? rows : p.width;
    x.replay = p.replay ? p.replay[r] : 0;
    x.base = p.base_off ? p.base_off[r] : 0;
    return x;
}

// Column tiles of tile `k`: those of the token groups [first, first + groups).
__device__ __forceinline__ void column_tiles(const WeightParams& p, const LaunchShape& ls, const Request& q, int32_t k,
                                             int32_t& first, int32_t& groups) {
    // tokens i that see a row of the tile: row0 + i at or behind its first row, and (window)
    // row0 + i - window + 1 at or before its last
    const int64_t row = (int64_t)k << ls.row_shift, a = row - q.row0;
    const int32_t i0 = a <= 0 ? 0 : a >= q.tokens ? q.tokens : (int32_t)a;
    int32_t i1 = q.tokens;
    if (p.window > 0) {
        const int64_t b = row + (1 << ls.row_shift) - 1 + p.window - q.row0;
        if (b < i1) i1 = b > i0 ? (int32_t)b : i0;
    }
    first = divide(i0, ls.by_tokens);
    groups = i1 > i0 ? divide(i1 - 1, ls.by_tokens) + 1 - first : 0;
}

// Tiles of a request that cost the same: the first `blind`, which no token sees rows of, and
// those from `first` to `end`, which all column tiles see rows of, at even_cost each.  The others are
// few (rows of the new tokens, and where their windows begin) and are counted one by one: with
// all tiles of a windowed request one token over 1048576 rows took 1355 us, where 131 do.
struct Even {
    int32_t blind, first, end;
};

__device__ __forceinline__ int64_t even_cost(const LaunchShape& ls, const Request& q) {
    return kTileCost + (int64_t)(q.tokens > 0 ? divide(q.tokens - 1, ls.by_tokens) + 1 : 0) * ls.head_groups;
}

__device__ __forceinline__ Even even_tiles(const WeightParams& p, const LaunchShape& ls, const Request& q, int32_t tiles) {
    if (q.tokens == 0) return {tiles, tiles, tiles};
    const auto bounded = [](int64_t n, int32_t lo, int32_t hi) { return n < lo ? lo : n > hi ? hi : (int32_t)n; };
    Even e{0, 0, 0};
    if (p.window > 0) {
        e.blind = bounded(((int64_t)q.row0 - p.window + 1) >> ls.row_shift, 0, tiles);
        e.first = bounded(((int64_t)q.row0 + q.tokens - p.window) >> ls.row_shift, e.blind, tiles);
    }
    const int64_t last = (int64_t)q.row0 + min(ls.tokens, q.tokens) - 1;  // of the first token group
    e.end = bounded((last >> ls.row_shift) + 1, e.first, tiles);
    return e;
}

__device__ __forceinline__ int32_t tiles_of(const LaunchShape& ls, const Request& q) {
    return (int32_t)(((int64_t)q.end + (1 << ls.row_shift) - 1) >> ls.row_shift);
}

// Cost of the tiles of 32 requests, one a lane.
__device__ __forceinline__ int64_t request_costs(const WeightParams& p, const LaunchShape& ls, int32_t r) {
    const int lane = threadIdx.x % kWarp;
    Request q{};
    int32_t uneven = 0;
    Even e{};
    int64_t sum = 0;
    if (r < p.num_reqs) {
        q = load_request(p, r);
        const int32_t tiles = tiles_of(ls, q);
        e = even_tiles(p, ls, q, tiles);
        uneven = tiles - e.blind - (e.end - e.first);
        sum = (int64_t)kTileCost * e.blind + even_cost(ls, q) * (e.end - e.first);
    }
    // the uneven tiles of a request, 32 at a time
    for (uint32_t rest = __ballot_sync(0xFFFFFFFFu, uneven > 0); rest; rest &= rest - 1) {
        const int src = __ffs(rest) - 1;
        Request x{};
        x.tokens = __shfl_sync(0xFFFFFFFFu, q.tokens, src);
        x.row0 = __shfl_sync(0xFFFFFFFFu, q.row0, src);
        const int32_t blind = __shfl_sync(0xFFFFFFFFu, e.blind, src), n = __shfl_sync(0xFFFFFFFFu, uneven, src);
        const int32_t from = __shfl_sync(0xFFFFFFFFu, e.first, src), even = __shfl_sync(0xFFFFFFFFu, e.end, src) - from;
        int64_t mine = 0;
        for (int32_t i = lane; i < n; i += kWarp) {
            int32_t first, groups, k = blind + i;
            if (k >= from) k += even;
            column_tiles(p, ls, x, k, first, groups);
            mine += kTileCost + (int64_t)groups * ls.head_groups;
        }
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
        if (lane == src) sum += mine;
    }
    return sum;
}

// A walk over the tiles of a range of the sequence.  A step is a tile with columns, or a run
// of neighbouring ones that no token sees rows of.
struct Walk {
    int64_t ahead, left;     // from the current tile to the range's start and to its end
    int32_t r, k, tiles;     // request and tile; r < 0: past the end; tiles of the request
    int32_t count;           // tiles of this step
    int32_t first, total;    // its token groups start at `first`; its column tiles
    int32_t c0, c1;          // those of them in the range
    Request q;

    __device__ __forceinline__ bool done() const { return r < 0; }

    // Past the last tile of the run without columns that tile k is in: the first ones, before
    // every window, or the last ones, behind all tokens of the call.
    __device__ __forceinline__ int32_t run_end(const WeightParams& p, const LaunchShape& ls) const {
        if (((int64_t)k << ls.row_shift) >= (int64_t)q.row0 + q.tokens) return tiles;
        const int64_t n = ((int64_t)q.row0 - p.window + 1) >> ls.row_shift;
        return q.tokens == 0 || n > tiles ? tiles : (int32_t)n;
    }

    __device__ __forceinline__ void pass(int64_t cost) {
        ahead -= cost;
        left -= cost;
    }

    __device__ __forceinline__ void load(const WeightParams& p, const LaunchShape& ls) {
        q = load_request(p, r);
        tiles = tiles_of(ls, q);
        k = 0;
    }

    // Takes up the walk at the start of request r, in which the range starts, and passes over whole
    // tiles before it.
    __device__ __forceinline__ void start(const WeightParams& p, const LaunchShape& ls) {
        count = total = tiles = k = 0;
        if (left <= 0) return;
        load(p, ls);
        const Even e = even_tiles(p, ls, q, tiles);
        k = (int32_t)min(ahead / kTileCost, (int64_t)e.blind);
        pass((int64_t)kTileCost * k);
        if (k < e.blind) return;
#pragma unroll 1
        for (; k < e.first; ++k) {
            int32_t groups;
            column_tiles(p, ls, q, k, first, groups);
            const int32_t cost = kTileCost + groups * ls.head_groups;
            if (ahead < cost) return;
            pass(cost);
        }
        const int64_t cost = even_cost(ls, q);
        const int64_t skip = (ahead | cost) >> 32 == 0 ? (int64_t)((uint32_t)ahead / (uint32_t)cost) : ahead / cost;
        const int32_t n = (int32_t)min(skip, (int64_t)(e.end - e.first));
        k += n;
        pass(cost * n);
    }

    // Moves to the next step of which something lies in the range.
    __device__ __forceinline__ void next(const WeightParams& p, const LaunchShape& ls) {
        pass(kTileCost * count + total);
        k += count;
        for (;;) {
            if (left <= 0) {
                r = -1;
                return;
            }
            if (k >= tiles) {
                if (++r >= p.num_reqs) {
                    r = -1;
                    return;
                }
                load(p, ls);
                continue;
            }
            int32_t groups;
            column_tiles(p, ls, q, k, first, groups);
            total = groups * ls.head_groups;
            if (total == 0) {
                const int32_t n = run_end(p, ls) - k;
                const int32_t skip = ahead > 0 ? (int32_t)min(ahead, (int64_t)n) : 0;
                count = (int32_t)min(left, (int64_t)n) - skip;
                pass(skip);
                k += skip;
                c0 = c1 = 0;
                if (count > 0) return;
                continue;
            }
            count = 1;
            const int64_t a = ahead - kTileCost, b = left - kTileCost;
            c0 = a > 0 ? (int32_t)(a < total ? a : total) : 0;
            c1 = b > 0 ? (int32_t)(b < total ? b : total) : 0;
            if (c0 < c1) return;
            pass(kTileCost + total);
            ++k;
        }
    }
};

// Share i of n of a sequence.
__device__ __forceinline__ int64_t share(int64_t all, int64_t i, int64_t n) {
    return all >> 40 == 0 ? all * i / n : all / n * i + all % n * i / n;
}

// The CTA's range of the sequence and the request it starts in, by one warp.  The costs of up
// to four requests a lane stay in registers.
constexpr int kFewRequests = 4 * kWarp;

__device__ __forceinline__ void find_range_of_few(const WeightParams& p, const LaunchShape& ls, Walk& w) {
    const int lane = threadIdx.x % kWarp;
    int64_t cost[4], at[4], all = 0;  // request i * 32 + lane
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        int64_t c = 0;
        if (i * kWarp < p.num_reqs) c = request_costs(p, ls, i * kWarp + lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k == i) cost[k] = c;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int64_t sum = cost[i];
        if (i * kWarp < p.num_reqs) {
#pragma unroll
            for (int o = 1; o < kWarp; o *= 2) {
                const int64_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += x;
            }
        }
        at[i] = all + sum - cost[i];
        all = __shfl_sync(0xFFFFFFFFu, all + sum, kWarp - 1);
    }
    const int64_t b = blockIdx.x / ls.ranks, n = gridDim.x / ls.ranks;
    const int64_t from = share(all, b, n);
    w.r = 0;
    w.ahead = from;
    w.left = share(all, b + 1, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, at[i] <= from && from < at[i] + cost[i]);
        if (here) {
            const int src = __ffs(here) - 1;
            w.r = i * kWarp + src;
            w.pass(__shfl_sync(0xFFFFFFFFu, at[i], src));
        }
    }
}

// The same by the whole CTA, for the planning warp (sh.first_*).
template <int kThreads>
__device__ void find_range(const WeightParams& p, const LaunchShape& ls, Shared& sh, int64_t& from, int64_t& to) {
    constexpr int kWarps = kThreads / kWarp;
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    if (tid == 0) {
        sh.first_request = 0;
        sh.first_at = 0;
    }
    from = to = 0;
    int64_t cost = 0;
    // once for the sum of all costs, once for the places (one code: it is in the cache then)
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        int64_t before = 0;
#pragma unroll 1
        for (int32_t r0 = 0; r0 < p.num_reqs; r0 += kThreads) {
            if (pass == 0 || p.num_reqs > kThreads)
                cost = r0 + warp * kWarp < p.num_reqs ? request_costs(p, ls, r0 + tid) : 0;
            int64_t sum = cost;
#pragma unroll
            for (int o = 1; o < kWarp; o *= 2) {
                const int64_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += x;
            }
            __syncthreads();
            if (lane == kWarp - 1) sh.scan[warp] = sum;
            __syncthreads();
            int64_t below = lane < warp ? sh.scan[lane] : 0, all = lane < kWarps ? sh.scan[lane] : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
                all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
            }
            const int64_t at = before + below + sum - cost;
            if (pass == 1 && at <= from && from < at + cost) {
                sh.first_request = r0 + tid;
                sh.first_at = at;
            }
            before += all;
        }
        if (pass == 0) {
            const int64_t b = blockIdx.x / ls.ranks, n = gridDim.x / ls.ranks;
            from = share(before, b, n);
            to = share(before, b + 1, n);
        }
    }
    __syncthreads();
}

// What the block table has for row j, -1 where nothing is looked up.  Not looked at here, so
// that the load stays in flight.
__device__ __forceinline__ int32_t page_of(const WeightParams& p, int32_t r, const Request& q, int32_t j) {
    if (j >= q.end) return -1;
    int32_t off;
    const int64_t logical = (int64_t)div_block32(j, p.cache.block_size, p.cache.shift, off) - q.base;
    if (logical < 0 || logical >= p.bt_width) return -1;
    return p.bt[(int64_t)r * p.bt_stride + logical];
}

// ---- the planning warp ------------------------------------------------------------------------

__device__ bool plan(const WeightParams& p, const LaunchShape& ls, Shared& sh, Walk w) {
    constexpr int kPer = kTile / kWarp;
    const int lane = threadIdx.x % kWarp;
    const int64_t token_stride = p.head_dim + p.rope_dim;
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
    // row i * 32 + lane of this CTA's part of the tile
    const int32_t mine = (int32_t)(blockIdx.x % ls.ranks) * kTile + lane;
    const auto row_at = [&](const Walk& x, int i) { return (int32_t)min(((int64_t)x.k << ls.row_shift) + mine + i * kWarp, (int64_t)INT32_MAX); };
    w.start(p, ls);
    Walk x;  // the tile before the walk's, which is to be published
    x.r = -1;
    int32_t page[kPer];  // of x
    bool kept = false, started = false;
    const bool fades = p.decay != 1.0f || p.out != p.weights;  // else rows that no token sees stay as they are
    for (uint32_t n = 0;;) {
        // on to the next tile with columns
        for (;;) {
            w.next(p, ls);
            if (!started) {
                started = true;
                if (lane == 0) {
                    Record rec{w.ahead >= w.left ? kEmptyRange : kNone, 0, 0, 0};
                    if (!w.done() && w.c0 > 0) rec = {w.c1 == w.total ? kEnds : kMiddle, w.r, w.k, 0};
                    ls.records[blockIdx.x] = rec;
                }
            }
            if (w.done() || w.total > 0) break;
            if (!fades) continue;
            const uint32_t slot = n % kTiles;
            if (n >= kTiles && !wait_all(&sh.tile_free[slot], (n / kTiles - 1) & 1)) return false;
            if (lane == 0) {
                Tile& t = sh.tile[slot];
                // a pair halves the rows
                const int64_t from = (int64_t)w.k << ls.row_shift;
                const int64_t to = min((int64_t)w.q.end, from + ((int64_t)w.count << ls.row_shift));
                const int64_t half = (to - from + 1) / 2, rank = blockIdx.x % ls.ranks;
                t.request = w.r;
                t.first_row = (int32_t)(from + rank * half);
                t.end = (int32_t)(rank + 1 < ls.ranks ? from + half : to);
                t.c0 = t.c1 = t.kept = 0;
                mbar_arrive(&sh.tile_full[slot]);
            }
            ++n;
        }
        if (!x.done()) {
            const uint32_t slot = n % kTiles;
            if (n >= kTiles && !wait_all(&sh.tile_free[slot], (n / kTiles - 1) & 1)) return false;
            Tile& t = sh.tile[slot];
            // the first column tile of the walk's tile is the last of this one
            const bool keeps = ls.keep_queries && w.r == x.r &&
                               x.first * ls.head_groups + x.c1 - 1 == w.first * ls.head_groups + w.c0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                Row row{zero, zero};
                const bool there = page[i] >= 0 && page[i] < p.cache.num_pages;
                if (there) {
                    int32_t off;
                    div_block32(row_at(x, i), p.cache.block_size, p.cache.shift, off);
                    const uint8_t* pg = p.cache.base + (int64_t)page[i] * p.cache.page_stride;
                    row.data = pg + off * token_stride;
                    row.scales = pg + p.cache.block_size * token_stride + (int64_t)off * (p.head_dim / 64);
                }
                t.row[i * kWarp + lane] = row;
                const uint32_t rows = __ballot_sync(0xFFFFFFFFu, there);
                if (lane == 0) t.there[i] = rows;
            }
            if (lane == 0) {
                t.request = x.r;
                t.first_row = row_at(x, 0);  // lane 0's
                t.end = x.q.end;
                t.first = x.first;
                t.total = x.total;
                t.c0 = x.c0;
                t.c1 = x.c1;
                t.tokens = x.q.tokens;
                t.token0 = x.q.token0;
                t.row0 = x.q.row0;
                t.replay = x.q.replay;
                t.kept = kept;
                t.keeps = keeps;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.tile_full[slot]);
            kept = keeps;
            ++n;
        }
        if (w.done()) {
            const uint32_t slot = n % kTiles;
            if (n >= kTiles && !wait_all(&sh.tile_free[slot], (n / kTiles - 1) & 1)) return false;
            if (lane == 0) {
                sh.tile[slot].request = -1;
                mbar_arrive(&sh.tile_full[slot]);
            }
            return true;
        }
        x = w;
        // in flight until these rows are published
#pragma unroll
        for (int i = 0; i < kPer; ++i) page[i] = page_of(p, x.r, x.q, row_at(x, i));
    }
}

// Place of a role in the ring of tiles.
struct Tiles {
    uint32_t n = 0;
    __device__ __forceinline__ bool wait(Shared& sh) const { return wait_all(&sh.tile_full[n % kTiles], (n / kTiles) & 1); }
    __device__ __forceinline__ const Tile& at(const Shared& sh) const { return sh.tile[n % kTiles]; }
    // The next one with columns, or the end.
    __device__ __forceinline__ bool wait_columns(Shared& sh) {
        for (;;) {
            if (!wait(sh)) return false;
            if (at(sh).request < 0 || at(sh).c0 < at(sh).c1) return true;
            next(sh);
        }
    }
    // The tile has been read (by this warp).
    __device__ __forceinline__ void next(Shared& sh) {
        __syncwarp();
        if (threadIdx.x % kWarp == 0) mbar_arrive(&sh.tile_free[n % kTiles]);
        ++n;
    }
};

// ---- workers: records to tensor memory -----------------------------------------------------

// 16-byte copy global -> shared.  Records are read once: they leave L2 first, before the
// queries and the kernel's own code.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ uint64_t read_once() {
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 16 E4M3 bytes of UE8M0 scale byte b as eight bf16 pairs, by the rule of the gather.
__device__ __forceinline__ void dequant16(uint4 raw, uint32_t b, uint32_t* w) {
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    const uint64_t s2 = splat_f32x2(ue8m0_scale(b));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[2 * i] = scale_f16x2_to_bf16x2(cvt_e4m3x2_to_f16x2(in[i] & 0xFFFFu), s2);
        w[2 * i + 1] = scale_f16x2_to_bf16x2(cvt_e4m3x2_to_f16x2(in[i] >> 16), s2);
    }
}

// Lane i's row of tensor memory: 32 columns from `addr` on.
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
          "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
          "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
          "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(addr)
        : "memory");
}

// Arrives on a barrier of the CTA that issues the MMAs.  What it hands over stands in tensor
// memory, ordered by the tcgen05 fences, so that no cluster-wide release is needed (it
// would cost a step of the sums some 1000 cycles).
template <bool kPair>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    if constexpr (kPair)
        asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
 "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar)) : "memory");
    else
        mbar_arrive(bar);
}

// A worker warp has the rows 32 * quad ... of each tile and the dims of one part.  Records
// stand in its part of shared memory with a row stride that is an odd number of 16 bytes,
// so that lanes reading 16 bytes of their own rows hit different banks.
template <class R>
__device__ bool work(const WeightParams& p, const LaunchShape& ls, Shared& sh, uint32_t staging, uint32_t tmem_k) {
    constexpr int D = R::D, kBlocks = D / 64 / R::kParts;  // 64-dim blocks of a part
    constexpr bool kPair = R::kPair;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, quad = warp % 4, part = warp / 4;
    const int nope = D - p.rope_dim;
    const int d0 = part * (D / R::kParts);
    const auto byte_of = [&](int d) { return d <= nope ? d : nope + 2 * (d - nope); };
    const int stride = ls.stride[part], byte0 = byte_of(d0);
    uint32_t mine = staging + quad * kWarp * stride;
    for (int i = 0; i < part; ++i) mine += 4 * kWarp * ls.stride[i];
    const uint32_t own = mine + lane * stride;
    const uint64_t policy = read_once();

    const auto load_scales = [&](const uint8_t* at) {
        uint2 s = make_uint2(0, 0);
        if (D == 512) {
            s = ld_nc_v2(at);
        } else if (D == 256) {
            s.x = ld_nc_u32(at);
        } else {
            s.x = ld_nc_u8(at) | (ld_nc_u8(at + 1) << 8);
        }
        return s;
    };
    // Copies block b of a tile's rows: 4 or 8 lanes a row.
    const auto fetch = [&](const Tile& t, int b) {
        const int d = d0 + b * 64, at = byte_of(d);
        const Row* row = t.row + quad * kWarp;
        if (d >= nope) {
            const int first = lane / 8, piece = lane % 8 * 16;
            const uint32_t dst = mine + first * stride + (at - byte0) + piece;
#pragma unroll
            for (int i = 0; i < 8; ++i) copy16(dst + i * 4 * stride, row[first + i * 4].data + at + piece, policy);
        } else {
            const int first = lane / 4, piece = lane % 4 * 16;
            const uint32_t dst = mine + first * stride + (at - byte0) + piece;
#pragma unroll
            for (int i = 0; i < 4; ++i) copy16(dst + i * 8 * stride, row[first + i * 8].data + at + piece, policy);
        }
    };
    const auto hand_over = [&](int b) {
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader<kPair>(&sh.k_full[b]);
    };
    Tiles tiles;
    if (!tiles.wait_columns(sh)) return false;
    if (tiles.at(sh).request < 0) return true;
    for (int b = 0; b < kBlocks; ++b) {
        fetch(tiles.at(sh), b);
        copies_commit();
    }
    uint2 scales = load_scales(tiles.at(sh).row[quad * kWarp + lane].scales);
    tiles.next(sh);
    for (uint32_t step = 0;; ++step) {
        if (!tiles.wait_columns(sh)) return false;
        const bool more = tiles.at(sh).request >= 0;
        uint2 next_scales = make_uint2(0, 0);
        if (more) next_scales = load_scales(tiles.at(sh).row[quad * kWarp + lane].scales);
#pragma unroll 1
        for (int b = 0; b < kBlocks; ++b) {
            const int d = d0 + b * 64, block = part * kBlocks + b;
            const uint32_t at = own + byte_of(d) - byte0;
            copies_wait<kBlocks - 1>();
            __syncwarp();
            uint32_t w[32];
            if (d < nope) {
                uint4 raw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[i] = lds_v4(at + i * 16);
                __syncwarp();  // the block has been read: the next tile's copy may land there
                if (more) fetch(tiles.at(sh), b);
                copies_commit();
                const uint32_t sc = ((block < 4 ? scales.x : scales.y) >> (8 * (block & 3))) & 0xFFu;
#pragma unroll
                for (int i = 0; i < 4; ++i) dequant16(raw[i], sc, w + 8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = lds_v4(at + i * 16);
                    w[4 * i] = v.x;
                    w[4 * i + 1] = v.y;
                    w[4 * i + 2] = v.z;
                    w[4 * i + 3] = v.w;
                }
                __syncwarp();
                if (more) fetch(tiles.at(sh), b);
                copies_commit();
            }
            // the block before has had this one's time to be written
            if (b > 0) hand_over(b - 1);
            if (step > 0 && !wait_all(&sh.k_free[b], (step - 1) & 1)) return false;
            tmem_fence_after();
            tmem_st32(tmem_k + ((uint32_t)(quad * kWarp) << 16) + block * 32, w);
        }
        hand_over(kBlocks - 1);
        if (!more) return true;
        tiles.next(sh);
        scales = next_scales;
    }
}

// The block of 64 dims in half `half` of stage `i`: the parts' blocks in turn, as they come.
template <class R>
__device__ __forceinline__ constexpr int block_at(int i, int half) {
    const int n = 2 * i + half;
    return n % R::kParts * (R::D / 64 / R::kParts) + n / R::kParts;
}

// ---- queries and columns ---------------------------------------------------------------------

// kPair: the bytes are counted by the first CTA's barrier.
template <bool kPair>
__device__ __forceinline__ void tma_queries(uint32_t dst, const CUtensorMap& map, int32_t d, int32_t h, int32_t t, uint64_t* bar) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %5, 0;\n\t"
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [a];\n\t}"
            ::"r"(dst), "l"(reinterpret_cast<uint64_t>(&map)), "r"(d), "r"(h), "r"(t), "r"(smem_u32(bar)) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(dst), "l"(reinterpret_cast<uint64_t>(&map)), "r"(d), "r"(h), "r"(t), "r"(smem_u32(bar)) : "memory");
}

// Four lanes fetch the queries: a box each, of two stages.
template <class R>
__device__ bool fetch_queries(const WeightParams& p, const LaunchShape& ls, const CUtensorMap& map, Shared& sh, uint32_t ring) {
    constexpr bool kPair = R::kPair;
    constexpr int kStages = R::D / 128, kAtOnce = kStages > 1 ? 2 : 1;  // of a column tile; at a time
    constexpr uint32_t kLanes = (1u << (2 * kAtOnce)) - 1;
    const int lane = threadIdx.x % kWarp, half = lane & 1;
    if (lane >= 2 * kAtOnce) return true;
    const uint32_t bytes = (uint32_t)(ls.box_heads * ls.box_tokens * 128) * (kPair ? 4 : 2);
    const int rank = kPair ? (int)(blockIdx.x & 1) : 0;
    const int32_t from_t = ls.by_heads ? 0 : rank * ls.box_tokens, from_h = ls.by_heads ? rank * ls.box_heads : 0;
    uint32_t stage = lane / 2, round = 0, issued = lane / 2;  // this lane's next stage of all
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kTiles;
        ok = __all_sync(kLanes, mbar_poll_bounded(&sh.tile_full[slot], (n / kTiles) & 1, kWaitLimitNs));
        if (!ok) break;
        const Tile& tile = sh.tile[slot];
        const bool end = tile.request < 0;
        const int32_t c1 = tile.c1, token0 = tile.token0 + tile.first * ls.tokens;
        int32_t c = tile.c0 + tile.kept;
        __syncwarp(kLanes);
        if (end) return true;
        if (lane == 0) mbar_arrive(&sh.tile_free[slot]);
        int32_t group = divide(c, ls.by_groups), part = c - group * ls.head_groups;
        for (; ok && c < c1; ++c) {
            const int32_t t = token0 + group * ls.tokens + from_t, h = part * ls.heads + from_h;
#pragma unroll 1
            for (int i = 0; i < kStages; i += kAtOnce) {
                const bool free = round == 0 || mbar_poll_bounded(&sh.q_free[stage], (round - 1) & 1, kWaitLimitNs);
                ok = __all_sync(kLanes, free);
                if (!ok) break;
                if (half == 0 && rank == 0) mbar_arrive_expect_tx(&sh.q_full[stage], bytes);
                tma_queries<kPair>(ring + stage * ls.stage_bytes + half * (ls.stage_bytes / 2), map,
                                   block_at<R>(i + lane / 2, half) * 64, h, t, &sh.q_full[stage]);
                issued += kAtOnce;
                stage += kAtOnce;
                if (stage >= (uint32_t)ls.stages) {
                    stage -= ls.stages;
                    ++round;
                }
            }
            if (++part == ls.head_groups) {
                part = 0;
                ++group;
            }
        }
    }
    // a wait expired: copies in flight land before the CTA ends (the first CTA of a pair waits for
    // both, and they end together)
    for (int i = 0; i < ls.stages && rank == 0; i += kAtOnce) {
        if (issued < (uint32_t)(i + kAtOnce)) break;
        const uint32_t x = issued - kAtOnce - i;
        mbar_poll_bounded(&sh.q_full[x % ls.stages], (x / ls.stages) & 1, kWaitLimitNs / 8);
    }
    return false;
}

// The logarithms and bounds of the columns, one or two a thread.  The next column tile's lse is in
// flight while this one's is worked on.
template <class R>
__device__ bool columns(const WeightParams& p, const LaunchShape& ls, Shared& sh) {
    constexpr int kPer = kCols / kWarp / R::kColumnWarps;  // columns of a thread
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp - R::kColumnWarp;
    int32_t token[kPer], head[kPer];  // in the column tile; token -1: not in the box
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int col = (u * R::kColumnWarps + warp) * kWarp + lane, rank = col / ls.box_cols, at = col - rank * ls.box_cols;
        const bool in_box = at < ls.box_heads * ls.box_tokens && rank < ls.ranks;
        token[u] = in_box ? at / ls.box_heads + (ls.by_heads ? 0 : rank * ls.box_tokens) : -1;
        head[u] = at % ls.box_heads + (ls.by_heads ? rank * ls.box_heads : 0);
    }
    struct Column {
        bool used;
        int32_t pos, rows_from;
        float lse, sink;
    };
    Tiles tiles;
    int32_t c = 0, c1 = 0, group = 0, part = 0, tokens = 0, token0 = 0, row0 = 0, replay = 0;
    bool end = false;
    // this thread's columns of the column tile at hand
    Column next[kPer];
    const auto load = [&]() {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            Column x{false, 0, replay, 0.0f, -INFINITY};
            const int32_t i = group * ls.tokens + token[u], h = part * ls.heads + head[u];
            if (token[u] >= 0 && i < tokens && h < p.num_heads) {
                const int64_t t = (int64_t)token0 + i;
                x.used = p.valid == nullptr || p.valid[t] != 0;
                x.pos = row0 + i;
                x.lse = p.lse[t * p.lse_stride_t + h];
                if (p.sink) x.sink = p.sink[h];
            }
            next[u] = x;
        }
    };
    // moves on to the first column tile of a later tile
    const auto next_tile = [&]() {
        for (;;) {
            if (!tiles.wait(sh)) return false;
            const Tile& t = tiles.at(sh);
            if (t.request < 0) {
                end = true;
                return true;
            }
            c = t.c0 + t.kept;
            c1 = t.c1;
            tokens = t.tokens;
            token0 = t.token0;
            row0 = t.row0;
            replay = t.replay;
            group = divide(c, ls.by_groups);
            part = c - group * ls.head_groups;
            group += t.first;
            tiles.next(sh);
            if (c < c1) return true;
        }
    };
    if (!next_tile()) return false;
    if (!end) load();
    for (uint32_t seq = 0; !end; ++seq) {
        Column now[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) now[u] = next[u];
        // the next column tile is read ahead where that waits for no other role, which may be
        // waiting for this one
        const bool ahead = ++c < c1;
        if (ahead) {
            if (++part == ls.head_groups) {
                part = 0;
                ++group;
            }
            load();
        }
        const uint32_t slot = seq % kColSlots;
        if (seq >= kColSlots && !wait_all(&sh.col_free[slot], (seq / kColSlots - 1) & 1)) return false;
        Columns& co = sh.columns[slot];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const Column& x = now[u];
            const int group32 = u * R::kColumnWarps + warp, col = group32 * kWarp + lane;
            const float a = x.lse * kLog2e, b = x.sink * kLog2e, top = fmaxf(a, b);
            const float log = a != a || b != b ? NAN : isinf(top) ? top : top + log2f(1.0f + exp2f(-fabsf(a - b)));
            const bool used = x.used && log != -INFINITY;  // else a token that saw nothing
            const int32_t lo = max(p.window > 0 && x.pos >= p.window ? x.pos - p.window + 1 : 0, x.rows_from);
            const int32_t all_lo = __reduce_max_sync(0xFFFFFFFFu, used ? lo : INT32_MIN);
            const int32_t all_hi = __reduce_min_sync(0xFFFFFFFFu, used ? x.pos : INT32_MAX);
            const uint32_t in_use = __ballot_sync(0xFFFFFFFFu, used);
            co.log[col] = used ? log : 0.0f;
            co.lo[col] = used ? lo : INT32_MAX;
            co.hi[col] = used ? x.pos : -1;
            if (lane == 0) {
                (&co.all_lo.x)[group32] = all_lo;
                (&co.all_hi.x)[group32] = all_hi;
                (&co.all_used.x)[group32] = (int32_t)in_use;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.col_full[slot]);
        if (!ahead) {
            if (!next_tile()) return false;
            if (!end) load();
        }
    }
    return true;
}

// ---- the MMA warp ------------------------------------------------------------------------------

// Four steps of 16 dims, A from tensor memory; issued by the lane whose `lead` is 1.
template <bool kPair>
__device__ __forceinline__ void umma_bf16_ts4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool accumulate,
                                              uint32_t lead) {
#define PSK_TS4(GROUP)                                                                  \
    asm volatile(                                                                       \
        "{\n\t.reg .pred p, q, one;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"               \
        "setp.ne.u32 p, %4, 0;\n\t"                                                     \
        "setp.ne.u32 q, %5, 0;\n\t"                                                     \
        "setp.eq.u32 one, 0, 0;\n\t"                                                    \
        "@q tcgen05.mma." GROUP ".kind::f16 [%0], [%1], %2, %3, p;\n\t"                 \
        "add.u32 a, %1, 8;\n\tadd.u64 b, %2, 2;\n\t"                                    \
        "@q tcgen05.mma." GROUP ".kind::f16 [%0], [a], b, %3, one;\n\t"                 \
        "add.u32 a, %1, 16;\n\tadd.u64 b, %2, 4;\n\t"                                   \
        "@q tcgen05.mma." GROUP ".kind::f16 [%0], [a], b, %3, one;\n\t"                 \
        "add.u32 a, %1, 24;\n\tadd.u64 b, %2, 6;\n\t"                                   \
        "@q tcgen05.mma." GROUP ".kind::f16 [%0], [a], b, %3, one;\n\t}"                \
        ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead) \
        : "memory")
    if constexpr (kPair) {
        PSK_TS4("cta_group::2");
    } else {
        PSK_TS4("cta_group::1");
    }
#undef PSK_TS4
}

// The barrier (in both CTAs of a pair) completes one arrival when all MMAs issued by this
// thread (the lead lane) are done.
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t lead) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.u32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}"
            ::"r"(smem_u32(bar)), "r"(lead), "h"((uint16_t)3) : "memory");
    else
        umma_commit(bar, lead);
}

// Columns of a column tile of token group `group`, padded to what an MMA takes.
template <bool kPair>
__device__ __forceinline__ int32_t width_of(const LaunchShape& ls, int32_t tokens, int32_t group) {
    return kPair ? 2 * ls.box_cols : (min(ls.tokens, tokens - group * ls.tokens) * ls.heads + 15) / 16 * 16;
}

template <class R>
__device__ bool issue(const LaunchShape& ls, Shared& sh, uint32_t ring, uint32_t tmem_k, uint32_t tmem_s) {
    constexpr bool kPair = R::kPair;
    constexpr int kStages = R::D / 128;
    const uint32_t lead = elect_one();
    const uint64_t q_desc = umma_desc(ring, 16, 1024, kSwizzle128);
    const uint32_t stage_step = (uint32_t)ls.stage_bytes >> 4;
    uint32_t stage = 0, round = 0, step = 0, tile = 0;
    Tiles tiles;
    for (;;) {
        if (!tiles.wait_columns(sh)) return false;
        const Tile& t = tiles.at(sh);
        if (t.request < 0) return true;
        const int32_t c0 = t.c0, c1 = t.c1, first = t.first, tokens = t.tokens;
        const bool keeps = t.keeps;
        tiles.next(sh);
        if (kPair && (blockIdx.x & 1)) continue;  // the first CTA of a pair issues
        int32_t group = divide(c0, ls.by_groups), part = c0 - group * ls.head_groups;
        for (int32_t c = c0; c < c1; ++c, ++step) {
            const bool last = c == c1 - 1, keep = last && keeps;
            const uint32_t idesc = umma_idesc(kTile * (kPair ? 2 : 1), width_of<kPair>(ls, tokens, first + group), false), d = tmem_s + (step & 1) * kCols;
            if (step >= 2 && !wait_all(&sh.s_free[step & 1], (step / 2 - 1) & 1)) return false;
            uint32_t st = stage, rd = round;
            // not unrolled: in a batch of single tokens each warp passes its code once a tile,
            // and what is long has left the instruction cache by then
#pragma unroll 1
            for (int i = 0; i < kStages; ++i) {
                const int b = 2 * i / R::kParts;  // which blocks of the parts
                if (c == c0 && 2 * i % R::kParts == 0 && !wait_all(&sh.k_full[b], tile & 1)) return false;
                if (!wait_all(&sh.q_full[st], rd & 1)) return false;
                tmem_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    umma_bf16_ts4<kPair>(d, tmem_k + block_at<R>(i, half) * 32, q_desc + st * stage_step + half * (stage_step / 2),
                                         idesc, i > 0 || half > 0, lead);
                if (last && (2 * i + 2) % R::kParts == 0) commit<kPair>(&sh.k_free[b], lead);
                if (!keep) commit<kPair>(&sh.q_free[st], lead);
                if (++st == (uint32_t)ls.stages) {
                    st = 0;
                    ++rd;
                }
            }
            commit<kPair>(&sh.s_full[step & 1], lead);
            if (!keep) {
                stage = st;
                round = rd;
            }
            if (++part == ls.head_groups) {
                part = 0;
                ++group;
            }
        }
        ++tile;
    }
}

// ---- scores to sums --------------------------------------------------------------------------

struct Sum {
    float hi = 0.0f, lo = 0.0f;  // compensated by Kahan's rule
    __device__ __forceinline__ void add(float x) {
        const float y = x - lo, z = hi + y;
        lo = isfinite(z) ? (z - hi) - y : 0.0f;
        hi = z;
    }
};

// Rows [j, end) of a request that no token of the call sees: every `step`-th is this thread's.
__device__ __forceinline__ void fade(const WeightParams& p, int32_t request, int64_t j, int32_t end, int32_t step) {
    constexpr int kAtOnce = 4;
    const float* from = p.weights + (int64_t)request * p.w_stride;
    float* to = p.out + (int64_t)request * p.out_stride;
#pragma unroll 1
    for (; j < end; j += kAtOnce * step) {
        float v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) v[i] = p.decay != 0.0f && j + i * step < end ? p.decay * from[j + i * step] : 0.0f;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (j + i * step < end) to[j + i * step] = v[i];
    }
}

template <class R>
__device__ bool summarise(const WeightParams& p, const LaunchShape& ls, Shared& sh, uint32_t tmem_s) {
    constexpr bool kPair = R::kPair;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp - R::kWorkers, quad = warp % 4, half = warp / 4;
    const uint32_t lane_base = tmem_s + ((uint32_t)(quad * kWarp) << 16);
    uint32_t step = 0, seq = 0, tile = 0;
    bool loaded = false;
    Tiles tiles;
    for (;;) {
        if (!tiles.wait(sh)) return false;
        const Tile& t = tiles.at(sh);
        const int32_t request = t.request;
        if (request < 0) return true;
        if (t.c0 == t.c1) {
            const int32_t first_row = t.first_row, end = t.end;
            tiles.next(sh);
            fade(p, request, (int64_t)first_row + warp * kWarp + lane, end, R::kSummers * kWarp);
            continue;
        }
        const int32_t c0 = t.c0, c1 = t.c1, first = t.first, tokens = t.tokens;
        const bool ok = t.there[quad] >> lane & 1, whole = c0 == 0 && c1 == t.total, keeps = t.keeps;
        const int32_t j = t.first_row + quad * kWarp + lane;
        const bool in = j < t.end;
        tiles.next(sh);
        const int64_t out_at = (int64_t)request * p.out_stride + j;
        float old = 0.0f;
        if (p.decay != 0.0f && in && half == 0 && whole) old = p.weights[(int64_t)request * p.w_stride + j];
        Sum sum;
        int32_t group = divide(c0, ls.by_groups), part_of = c0 - group * ls.head_groups;
        for (int32_t c = c0; c < c1; ++c, ++step) {
            const int32_t n = width_of<kPair>(ls, tokens, first + group);
            if (loaded) {
                --seq;  // the columns are those of the step before
                loaded = false;
            } else if (!wait_all(&sh.col_full[seq % kColSlots], (seq / kColSlots) & 1)) {
                return false;
            }
            const Columns& co = sh.columns[seq % kColSlots];
            const int4 lo4 = co.all_lo, hi4 = co.all_hi, used4 = co.all_used;
            const bool rows = __all_sync(0xFFFFFFFFu, ok && j >= max(max(lo4.x, lo4.y), max(lo4.z, lo4.w)) &&
                                                          j <= min(min(hi4.x, hi4.y), min(hi4.z, hi4.w)));
            if (!wait_all(&sh.s_full[step & 1], (step / 2) & 1)) return false;
            tmem_fence_after();
            const uint32_t s_at = lane_base + (step & 1) * kCols;
            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int32_t n0 = half * 16; n0 < n; n0 += 16 * R::kShares) {
                float s[16];
                tmem_ld<16>(s_at + n0, s);
                const int32_t word = n0 < 32 ? used4.x : n0 < 64 ? used4.y : n0 < 96 ? used4.z : used4.w;
                const uint32_t used = ((uint32_t)word >> (n0 & 16)) & 0xFFFFu;
                if (rows && used == 0xFFFFu) {
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(&co.log[n0 + k]);
                        part[0] += ex2_approx(fmaf(s[k], ls.scale_log2, -x.x));
                        part[1] += ex2_approx(fmaf(s[k + 1], ls.scale_log2, -x.y));
                        part[2] += ex2_approx(fmaf(s[k + 2], ls.scale_log2, -x.z));
                        part[3] += ex2_approx(fmaf(s[k + 3], ls.scale_log2, -x.w));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(&co.log[n0 + k]);
                        const int4 lo = *reinterpret_cast<const int4*>(&co.lo[n0 + k]);
                        const int4 hi = *reinterpret_cast<const int4*>(&co.hi[n0 + k]);
                        part[0] += ok && j >= lo.x && j <= hi.x ? ex2_approx(fmaf(s[k], ls.scale_log2, -x.x)) : 0.0f;
                        part[1] += ok && j >= lo.y && j <= hi.y ? ex2_approx(fmaf(s[k + 1], ls.scale_log2, -x.y)) : 0.0f;
                        part[2] += ok && j >= lo.z && j <= hi.z ? ex2_approx(fmaf(s[k + 2], ls.scale_log2, -x.z)) : 0.0f;
                        part[3] += ok && j >= lo.w && j <= hi.w ? ex2_approx(fmaf(s[k + 3], ls.scale_log2, -x.w)) : 0.0f;
                    }
                }
            }
            sum.add((part[0] + part[1]) + (part[2] + part[3]));
            tmem_fence_before();
            __syncwarp();
            const bool keep = c == c1 - 1 && keeps;
            if (lane == 0) {
                arrive_leader<kPair>(&sh.s_free[step & 1]);
                if (!keep) mbar_arrive(&sh.col_free[seq % kColSlots]);
            }
            loaded = keep;
            ++seq;
            if (++part_of == ls.head_groups) {
                part_of = 0;
                ++group;
            }
        }
        // the halves of the columns
        if (half == 1) {
            if (tile > 0 && !wait_all(&sh.half_free[quad], (tile - 1) & 1)) return false;
            sh.half_sum[quad][0][lane] = sum.hi;
            sh.half_sum[quad][1][lane] = sum.lo;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.half_full[quad]);
        } else {
            if constexpr (R::kShares == 2) {
                if (!wait_all(&sh.half_full[quad], tile & 1)) return false;
                sum.add(sh.half_sum[quad][0][lane]);
                sum.add(-sh.half_sum[quad][1][lane]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.half_free[quad]);
            }
            const float total = sum.hi - sum.lo;
            if (whole) {
                if (in) p.out[out_at] = p.decay == 0.0f ? total : fmaf(p.decay, old, total);
            } else {
                ls.parts[((int64_t)blockIdx.x * 2 + (c0 > 0 ? 0 : 1)) * kTile + quad * kWarp + lane] = total;
            }
        }
        ++tile;
    }
}

constexpr size_t kAlign = 1024;

template <bool kPair>
__device__ __forceinline__ void alloc_tmem(uint32_t* dst) {
    if constexpr (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        tmem_alloc(dst, 512);
    }
}

template <bool kPair>
__device__ __forceinline__ void free_tmem(uint32_t addr) {
    if constexpr (kPair)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(addr));
    else
        tmem_dealloc(addr, 512);
}

template <class R>
__global__ void __launch_bounds__(R::kThreads, 1)
    attn_weights_kernel(const __grid_constant__ WeightParams p, const __grid_constant__ LaunchShape ls,
                        const __grid_constant__ CUtensorMap map) {
    constexpr bool kPair = R::kPair;
    constexpr int kWorkers = R::kWorkers, kColumnWarp = R::kColumnWarp, kQueryWarp = R::kQueryWarp, kPlanWarp = R::kPlanWarp;
    constexpr int kMmaWarp = R::kMmaWarp;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((kAlign - (smem_u32(smem_raw) & (kAlign - 1))) & (kAlign - 1));
    uint8_t* staging = ring + ls.stages * ls.stage_bytes;
    Shared& sh = *reinterpret_cast<Shared*>(staging + ls.staging_bytes);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&sh.tile_full[i], 1);
            mbar_init(&sh.tile_free[i], kPlanWarp);  // every other warp
        }
        for (int i = 0; i < kMostBlocks; ++i) {
            mbar_init(&sh.k_full[i], (kPair ? 2 : 1) * kWorkers);
            mbar_init(&sh.k_free[i], 1);
        }
        for (int i = 0; i < kMostStages; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_free[i], 1);
        }
        for (int i = 0; i < kColSlots; ++i) {
            mbar_init(&sh.col_full[i], R::kColumnWarps);
            mbar_init(&sh.col_free[i], R::kSummers);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], kPair ? 2 * R::kSummers : R::kSummers);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.half_full[i], 1);
            mbar_init(&sh.half_free[i], 1);
        }
        mbar_init(&sh.drain, 1);
        mbar_fence_init();
    }
    __syncwarp();
    if (kPair) cluster_sync();  // the other CTA's barriers are there too
    if (warp == kMmaWarp) alloc_tmem<kPair>(&sh.tmem);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem_s = sh.tmem, tmem_k = tmem_s + 2 * kCols;
    pdl_wait();
    pdl_launch_dependents();
    Walk walk{};
    if (p.num_reqs > kFewRequests) {
        find_range<R::kThreads>(p, ls, sh, walk.ahead, walk.left);
        walk.r = sh.first_request;
        walk.pass(sh.first_at);
    } else if (warp == kPlanWarp) {
        find_range_of_few(p, ls, walk);
    }

    bool ok = true;
    if (warp < kWorkers) {
        ok = work<R>(p, ls, sh, smem_u32(staging), tmem_k);
        if (!ok) copies_wait<0>();
    } else if (warp < kColumnWarp) {
        ok = summarise<R>(p, ls, sh, tmem_s);
    } else if (warp < kQueryWarp) {
        ok = columns<R>(p, ls, sh);
    } else if (warp == kQueryWarp) {
        ok = fetch_queries<R>(p, ls, map, sh, smem_u32(ring));
        __syncwarp();
    } else if (warp == kPlanWarp) {
        ok = plan(p, ls, sh, walk);
    } else {
        ok = issue<R>(ls, sh, smem_u32(ring), tmem_k, tmem_s);
        if (!ok && (!kPair || (blockIdx.x & 1) == 0)) {  // wait for the MMAs in flight before the operands go
            commit<kPair>(&sh.drain, elect_one());
            mbar_poll_bounded(&sh.drain, 0, kWaitLimitNs);
        }
    }
    __syncwarp();
    if (!ok && lane == 0) atomicAdd(&g_weights_wait_timeouts, 1u);
    tmem_fence_before();
    if (kPair) cluster_sync(); else __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) free_tmem<kPair>(sh.tmem);
    if (kPair) cluster_sync();
}

// ---- joining the parts of cut tiles ------------------------------------------------------------
//
// The CTA a tile ends in adds up its parts, from its own back to the one it starts in.
__global__ void __launch_bounds__(kTile) join_kernel(const WeightParams p, const LaunchShape ls) {
    pdl_wait();
    pdl_launch_dependents();
    const Record rec = ls.records[blockIdx.x];
    if (rec.kind != kEnds) return;
    const int i = threadIdx.x;
    double sum = ls.parts[(int64_t)blockIdx.x * 2 * kTile + i];
    for (int c = (int)blockIdx.x - ls.ranks; c >= 0; c -= ls.ranks) {
        const int kind = ls.records[c].kind;
        if (kind == kEmptyRange) continue;
        if (kind == kMiddle) {
            sum += ls.parts[(int64_t)c * 2 * kTile + i];
        } else {
            sum += ls.parts[((int64_t)c * 2 + 1) * kTile + i];
            break;
        }
    }
    const int32_t rows = p.seq_lens[rec.request];
    const int64_t j = ((int64_t)rec.tile << ls.row_shift) + blockIdx.x % ls.ranks * kTile + i;
    if (j >= rows || j >= p.width) return;
    float* out = p.out + (int64_t)rec.request * p.out_stride + j;
    const float total = (float)sum;
    *out = p.decay == 0.0f ? total : fmaf(p.decay, p.weights[(int64_t)rec.request * p.w_stride + j], total);
}

// ---- host ----------------------------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void*> cached{nullptr};
    void* fn = cached.load(std::memory_order_acquire);
    if (fn == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(fn, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(fn);
}

// Queries as [token][head][dim], read in boxes of 64 dims of a column tile.
bool query_map(const WeightParams& p, const LaunchShape& ls, CUtensorMap& map) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.num_heads, (cuuint64_t)p.num_tokens};
    // a dim of size 1 may carry any stride
    const cuuint64_t row = (cuuint64_t)p.head_dim * 2;
    const cuuint64_t strides[2] = {p.num_heads > 1 ? (cuuint64_t)p.q_stride_h * 2 : row,
                                   p.num_tokens > 1 ? (cuuint64_t)p.q_stride_t * 2 : row * (cuuint64_t)p.num_heads};
    const cuuint32_t box[3] = {64, (cuuint32_t)ls.box_heads, (cuuint32_t)ls.box_tokens}, ones[3] = {1, 1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMostShared = 227 * 1024;

// Pairs from this many columns a request on.  64 requests of 8192 rows, pairs against single
// CTAs: 64 columns 92 us against 78 (a pair has half the dequantising warps), 128 89 against 96
// (head_dim 256: 64 against 69), 256 120 against 147, 512 194 against 241.
constexpr int64_t kPairColumns = 128;

LaunchShape make_shape(const WeightParams& p) {
    LaunchShape ls{};
    const int H = p.num_heads;
    const int64_t T = p.num_tokens > 0 ? p.num_tokens : 1;
    const int64_t each = (T + p.num_reqs - 1) / p.num_reqs;  // tokens of a request, on average
    ls.ranks = T * H >= kPairColumns * p.num_reqs && sm_count() % 2 == 0 ? 2 : 1;
    ls.row_shift = ls.ranks == 2 ? 8 : 7;
    if (ls.ranks == 1) {
        ls.head_groups = (H + kCols - 1) / kCols;
        ls.heads = (H + ls.head_groups - 1) / ls.head_groups;
        ls.tokens = ls.head_groups > 1 ? 1 : kCols / ls.heads;
        if (ls.tokens > each) ls.tokens = (int32_t)each;
        ls.box_heads = ls.heads;
        ls.box_tokens = ls.tokens;
        ls.box_cols = kCols;
    } else {
        // the cut of heads and tokens that leaves the fewest columns unused
        double best = 0.0;
        const int half = kCols / 2;
        for (int groups = 1; groups <= (H + half - 1) / half + 3 && groups <= H; ++groups)
            for (int by_heads = 0; by_heads < 2; ++by_heads) {
                const int heads = (H + groups - 1) / groups, box = by_heads ? (heads + 1) / 2 : heads;
                if (box > half) continue;
                int tokens = half / box;
                const int64_t most = by_heads ? each : (each + 1) / 2;
                if (tokens > most) tokens = (int)most;
                const int64_t filled = by_heads ? tokens : 2 * tokens < each ? 2 * tokens : each;
                const double used = (double)H / groups * (double)filled;
                if (used <= best) continue;
                best = used;
                ls.by_heads = by_heads;
                ls.heads = by_heads ? 2 * box : heads;
                ls.head_groups = (H + ls.heads - 1) / ls.heads;
                ls.tokens = by_heads ? tokens : 2 * tokens;
                ls.box_heads = box;
                ls.box_tokens = tokens;
            }
        ls.box_cols = (ls.box_heads * ls.box_tokens + 15) / 16 * 16;
    }
    ls.by_tokens = divisor(ls.tokens);
    ls.by_groups = divisor(ls.head_groups);
    const int nope = p.head_dim - p.rope_dim, parts = ls.ranks == 1 && p.head_dim == 512 ? 4 : 2;
    const auto byte_of = [&](int d) { return d <= nope ? d : nope + 2 * (d - nope); };
    for (int i = 0; i < parts; ++i) {
        ls.stride[i] = byte_of((i + 1) * p.head_dim / parts) - byte_of(i * p.head_dim / parts) + 16;
        ls.staging_bytes += 4 * kWarp * ls.stride[i];
    }
    ls.stage_bytes = (ls.box_heads * ls.box_tokens + 15) / 16 * 16 * 128 * 2;
    const int room = kMostShared - (int)kAlign - ls.staging_bytes - (int)sizeof(Shared);
    ls.stages = room / ls.stage_bytes;
    if (ls.stages > kMostStages) ls.stages = kMostStages;
    const int most = p.head_dim == 128 ? 4 : 3 * p.head_dim / 128;
    if (ls.stages > most) ls.stages = most;
    ls.keep_queries = ls.stages >= p.head_dim / 128;
    return ls;
}

template <class R>
cudaError_t launch(const WeightParams& p, const LaunchShape& ls, const CUtensorMap& map, int ctas, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_limit_per_device(attn_weights_kernel<R>, kMostShared, done);
    if (e != cudaSuccess) return e;
    const size_t smem = kAlign + (size_t)ls.stages * ls.stage_bytes + ls.staging_bytes + sizeof(Shared);
    return launch_pdl_clusters(attn_weights_kernel<R>, ls.ranks, dim3((unsigned)ctas), dim3(R::kThreads), smem, stream, p, ls, map);
}

template <int D>
cudaError_t launch_ranks(const WeightParams& p, const LaunchShape& ls, const CUtensorMap& map, int ctas, cudaStream_t stream) {
    return ls.ranks == 2 ? launch<Roles<D, true>>(p, ls, map, ctas, stream) : launch<Roles<D, false>>(p, ls, map, ctas, stream);
}

}  // namespace

int64_t attn_weights_workspace_bytes() {
    return (int64_t)sm_count() * (2 * kTile * (int64_t)sizeof(float) + (int64_t)sizeof(Record));
}

cudaError_t launch_attn_weights(WeightParams p, cudaStream_t stream) {
    p.cache.shift = log2_if_pow2(p.cache.block_size);
    LaunchShape ls = make_shape(p);
    const int ctas = sm_count();
    ls.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
    ls.parts = static_cast<float*>(p.workspace);
    ls.records = reinterpret_cast<Record*>(ls.parts + (int64_t)ctas * 2 * kTile);
    CUtensorMap map{};
    if (p.num_tokens > 0 && !query_map(p, ls, map)) return cudaErrorNotSupported;
    const cudaError_t e = p.head_dim == 512   ? launch_ranks<512>(p, ls, map, ctas, stream)
                          : p.head_dim == 256 ? launch_ranks<256>(p, ls, map, ctas, stream)
                                              : launch_ranks<128>(p, ls, map, ctas, stream);
    // a request of one column tile at most is never cut
    const int64_t most = (p.num_tokens + ls.tokens - 1) / ls.tokens * ls.head_groups;
    if (e != cudaSuccess || most <= 1) return e;
    return launch_pdl(join_kernel, dim3((unsigned)ctas), dim3(kTile), 0, stream, p, ls);
}

cudaError_t read_attn_weights_wait_timeouts(uint32_t* count) {
    return cudaMemcpyFromSymbol(count, g_weights_wait_timeouts, sizeof(uint32_t));
}

}  // namespace psk
