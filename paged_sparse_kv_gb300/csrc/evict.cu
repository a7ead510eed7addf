// evict.cu -- eviction from a paged cache by accumulated attention weight: which
// rows of a request stay, and the records moved to where the others were.
#include "evict.h"
#include "psk_common.cuh"
#include "umma.cuh"

namespace psk {
namespace {

// ---- which rows stay -------------------------------------------------------------------
//
// Of the n rows of a request the m = min(n, keep) of the greatest weight stay; a protected
// row (an early or a recent position) counts as greater than any weight, and of equal ones
// the lower row stays.  Rows below m that stay do not move; the i-th of those from m on
// moves into the i-th row below m that goes, so nothing is read where something is written.
//
// Weights are mapped to unsigned keys of their order.  The m-th greatest key is found by
// radix selection over digits of 11, 11 and 10 bits: a histogram of the first digit of all
// keys, then of the next digit of those that share the digits found so far.  Ranks of
// rows in order come from counts per warp, each of which owns a run of neighbouring rows.
// A cluster of CTAs shares a long request; they add up histograms and counts through
// distributed shared memory.
//
// Latency bounds it: two reads of the rows, three histograms with their sums and three passes
// in order follow one another, each behind barriers of 1024 threads (and of the cluster).
// 64 requests of 2049 rows 8.8 us, 16 of up to 32768 rows in clusters of four 24.4 us, 3 of
// 131071 rows in clusters of eight 38.7 us, where bytes alone would take 0.3, 1 and 0.5.
constexpr int kThreads = 1024, kWarps = kThreads / kWarp;
constexpr int kBins = 2048;  // of the first two digits; the third has half as many
constexpr int kMostCtas = 8;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

struct SelectShared {
    alignas(8) uint32_t bins[3][kBins];
    uint32_t warp[kWarps];
    uint32_t ties[kWarps], holes[kWarps], movers[kWarps];  // of the rows of a warp
    uint32_t total[3];   // of this CTA: ties, holes, movers
    uint32_t found[3];   // the digit, how many of its keys stay, and how many it has
    int32_t newest;      // of this CTA
};

// Greater weights have greater keys; -0 as 0; NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0;
    const uint32_t b = __float_as_uint(w + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the warps below this one; `all` is the sum over all.  One barrier each side.
__device__ __forceinline__ uint32_t below_warp(const uint32_t (&x)[kWarps], uint32_t& all) {
    uint32_t v = x[threadIdx.x % kWarp], sum = v;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
#pragma unroll
    for (int o = 1; o < kWarp; o *= 2) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += u;
    }
    all = __shfl_sync(0xFFFFFFFFu, sum, kWarp - 1);
    const uint32_t before = __shfl_sync(0xFFFFFFFFu, sum - v, warp);
    return before;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* at, int rank) {
    uint32_t v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.u32 %0, [a];\n\t}"
                 : "=r"(v) : "r"(smem_u32(at)), "r"(rank) : "memory");
    return v;
}

__device__ __forceinline__ uint2 ld_cluster_u32x2(const uint32_t* at, int rank) {
    uint2 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
                 "ld.shared::cluster.v2.u32 {%0, %1}, [a];\n\t}"
                 : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(at)), "r"(rank) : "memory");
    return v;
}

// What stands at `at` in each CTA; all reads are in flight at once (one after the other took
// a microsecond each).
template <typename F>
__device__ __forceinline__ void for_ctas(const uint32_t* at, int ctas, F use) {
    uint32_t v[kMostCtas];
#pragma unroll
    for (int c = 0; c < kMostCtas; ++c) v[c] = c < ctas ? ld_cluster_u32(at, c) : 0;
#pragma unroll
    for (int c = 0; c < kMostCtas; ++c)
        if (c < ctas) use(c, v[c]);
}

__device__ __forceinline__ void sync_all(int ctas) {
    if (ctas > 1) cluster_sync(); else __syncthreads();
}

// kCached: the keys of a CTA's rows fit in shared memory.
template <bool kCached>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const SelectParams p, const int ctas) {
    extern __shared__ uint32_t s_keys[];
    __shared__ SelectShared sh;
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const int32_t r = (int32_t)blockIdx.x / ctas;
    const int rank = (int)blockIdx.x % ctas;
    for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.bins[0][0])[i] = 0;
    pdl_wait();
    const int32_t seq = p.seq_lens[r], keep = p.keep_lens[r];
    const bool wide = seq > p.width;  // rows without weights: nothing is evicted
    const int32_t n = wide ? 0 : max(seq, 0);
    const int32_t m = min(n, max(keep, 0));
    const float* w = p.weights + (int64_t)r * p.w_stride;
    const int32_t* pos = p.positions ? p.positions + (int64_t)r * p.pos_stride : nullptr;
    const bool select = m > 0 && m < n;
    // rows of a warp: a run of whole groups of 32
    const int32_t groups = (n + kWarp - 1) / kWarp, warps = ctas * kWarps;
    const int32_t per = (groups + warps - 1) / warps;
    const int64_t first64 = (int64_t)(rank * kWarps + warp) * per * kWarp;
    const int32_t first = (int32_t)min((int64_t)n, first64), end = (int32_t)min((int64_t)n, first64 + (int64_t)per * kWarp);
    uint32_t* cached = s_keys + warp * per * kWarp;

    int64_t newest = (int64_t)n - 1;
    if (select && pos && p.num_recent > 0) {  // the same in all CTAs of the request
        int32_t top = INT32_MIN;
#pragma unroll 8
        for (int32_t j = first + lane; j < end; j += kWarp) top = max(top, pos[j]);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0) sh.warp[warp] = (uint32_t)top;
        __syncthreads();
        if (warp == 0) {
            top = __reduce_max_sync(0xFFFFFFFFu, (int32_t)sh.warp[lane]);
            if (lane == 0) sh.newest = top;
        }
        sync_all(ctas);
        top = sh.newest;
        if (ctas > 1)
            for_ctas(reinterpret_cast<const uint32_t*>(&sh.newest), ctas, [&](int, uint32_t v) { top = max(top, (int32_t)v); });
        newest = top;
    }
    const int64_t recent = p.num_recent > 0 ? newest - p.num_recent : INT64_MAX;
    const auto key_of = [&](int32_t j) {
        const int64_t at = pos ? pos[j] : j;
        return at < p.num_first || at > recent ? kProtected : weight_key(w[j]);
    };
    const auto key_at = [&](int32_t j) { return kCached ? cached[j - first] : key_of(j); };

    uint32_t threshold = 0, left = (uint32_t)m;  // keys equal to the threshold of which `left` stay
    if (select) {
        if (kCached) {
#pragma unroll 8
            for (int32_t j = first + lane; j < end; j += kWarp) cached[j - first] = key_of(j);
        }
        __syncthreads();
        // ---- radix selection
        for (int digit = 0; digit < 3; ++digit) {
            const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
            const uint32_t bins = digit == 2 ? kBins / 2 : kBins;
#pragma unroll 4
            for (int32_t j0 = first; j0 < end; j0 += kWarp) {
                const int32_t j = j0 + lane;
                uint32_t key = 0;
                bool in = j < end;
                if (in) {
                    key = key_at(j);
                    in = digit == 0 || (digit == 1 ? key >> 21 == threshold >> 21 : key >> 10 == threshold >> 10);
                }
                const uint32_t bin = in ? (key >> shift) & (bins - 1) : ~0u;
                int same;
                __match_all_sync(0xFFFFFFFFu, bin, &same);
                if (same) {
                    if (in && lane == 0) atomicAdd(&sh.bins[digit][bin], (uint32_t)kWarp);
                } else if (in) {
                    atomicAdd(&sh.bins[digit][bin], 1u);
                }
            }
            sync_all(ctas);
            // thread i has the bins 2i and 2i + 1 counted from the top
            uint32_t x[2] = {0, 0};
            const int lower = (int)bins - 2 - 2 * tid;
            if (lower >= 0) {
                const uint32_t* at = &sh.bins[digit][lower];
                if (ctas == 1) {
                    x[0] = at[1];
                    x[1] = at[0];
                } else {
                    uint2 v[kMostCtas];
#pragma unroll
                    for (int c = 0; c < kMostCtas; ++c) v[c] = c < ctas ? ld_cluster_u32x2(at, c) : make_uint2(0, 0);
#pragma unroll
                    for (int c = 0; c < kMostCtas; ++c) {
                        x[0] += v[c].y;
                        x[1] += v[c].x;
                    }
                }
            }
            uint32_t sum = x[0] + x[1];
            const uint32_t mine = sum;
#pragma unroll
            for (int o = 1; o < kWarp; o *= 2) {
                const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += u;
            }
            if (lane == kWarp - 1) sh.warp[warp] = sum;
            __syncthreads();
            uint32_t all;
            const uint32_t above = below_warp(sh.warp, all) + sum - mine;
            // the bin that holds the left-th key from the top
            if (above < left && left <= above + mine) {
                const bool second = left > above + x[0];
                sh.found[0] = bins - 1 - (2 * tid + (second ? 1 : 0));
                sh.found[1] = left - above - (second ? x[0] : 0);
                sh.found[2] = second ? x[1] : x[0];
            }
            __syncthreads();
            threshold |= sh.found[0] << shift;
            left = sh.found[1];
        }
        // ---- of the keys equal to it the lowest rows stay (mostly all do, and need no ranks)
        uint32_t tied = 0;
        if (left < sh.found[2]) {  // the same in all CTAs
            uint32_t count = 0, all;
#pragma unroll 4
            for (int32_t j0 = first; j0 < end; j0 += kWarp) {
                const int32_t j = j0 + lane;
                count += __popc(__ballot_sync(0xFFFFFFFFu, j < end && key_at(j) == threshold));
            }
            if (lane == 0) sh.ties[warp] = count;
            __syncthreads();
            tied = below_warp(sh.ties, all);
            if (tid == 0) sh.total[0] = all;
            sync_all(ctas);
            if (ctas > 1)
                for_ctas(&sh.total[0], ctas, [&](int c, uint32_t v) { tied += c < rank ? v : 0; });
        }

        // ---- holes and movers: counts first, then their places
        uint32_t seen = tied, holes = 0, movers = 0;
        const auto group = [&](int32_t j0, uint32_t& ties, bool& stays) {
            const int32_t j = j0 + lane;
            const uint32_t key = j < end ? key_at(j) : 0;
            const bool tie = j < end && key == threshold;
            const uint32_t t = __ballot_sync(0xFFFFFFFFu, tie);
            stays = j < end && (key > threshold || (tie && ties + __popc(t & ((1u << lane) - 1)) < left));
            ties += __popc(t);
            return j;
        };
#pragma unroll 4
        for (int32_t j0 = first; j0 < end; j0 += kWarp) {
            bool stays;
            const int32_t j = group(j0, seen, stays);
            holes += __popc(__ballot_sync(0xFFFFFFFFu, j < end && j < m && !stays));
            movers += __popc(__ballot_sync(0xFFFFFFFFu, j >= m && stays));
        }
        if (lane == 0) {
            sh.holes[warp] = holes;
            sh.movers[warp] = movers;
        }
        __syncthreads();
        uint32_t all_holes, all_movers;
        uint32_t hole = below_warp(sh.holes, all_holes), mover = below_warp(sh.movers, all_movers);
        if (tid == 0) {
            sh.total[1] = all_holes;
            sh.total[2] = all_movers;
        }
        sync_all(ctas);
        uint32_t moves = all_holes;
        if (ctas > 1) {
            moves = 0;
            for_ctas(&sh.total[1], ctas, [&](int c, uint32_t v) {
                moves += v;
                hole += c < rank ? v : 0;
            });
            for_ctas(&sh.total[2], ctas, [&](int c, uint32_t v) { mover += c < rank ? v : 0; });
        }
        int2* list = p.moves + (int64_t)r * p.moves_stride;
        const bool copy_w = p.weights_out && p.weights_out != p.weights;
        const bool copy_p = p.positions_out && p.positions_out != p.positions;
        seen = tied;
#pragma unroll 4
        for (int32_t j0 = first; j0 < end; j0 += kWarp) {
            bool stays;
            const int32_t j = group(j0, seen, stays);
            const bool is_hole = j < end && j < m && !stays, is_mover = j >= m && stays;
            const uint32_t h = __ballot_sync(0xFFFFFFFFu, is_hole), v = __ballot_sync(0xFFFFFFFFu, is_mover);
            const uint32_t under = (1u << lane) - 1;
            if (is_hole) list[hole + __popc(h & under)].y = j;
            if (is_mover) list[mover + __popc(v & under)].x = j;
            hole += __popc(h);
            mover += __popc(v);
            if (stays && j < m) {
                if (copy_w) p.weights_out[(int64_t)r * p.wo_stride + j] = w[j];
                if (copy_p) p.positions_out[(int64_t)r * p.po_stride + j] = pos ? pos[j] : j;
            }
        }
        sync_all(ctas);  // the list is whole, and every weight has been read
#pragma unroll 2
        for (uint32_t i = rank * kThreads + tid; i < moves; i += ctas * kThreads) {
            const int2 move = list[i];
            if (p.weights_out) p.weights_out[(int64_t)r * p.wo_stride + move.y] = w[move.x];
            if (p.positions_out) p.positions_out[(int64_t)r * p.po_stride + move.y] = pos ? pos[move.x] : move.x;
        }
        if (rank == 0 && tid == 0) p.num_moves[r] = (int32_t)moves;
    } else {
        for (int32_t j = first + lane; j < min(end, m); j += kWarp) {  // all rows stay, or none
            if (p.weights_out && p.weights_out != p.weights) p.weights_out[(int64_t)r * p.wo_stride + j] = w[j];
            if (p.positions_out && p.positions_out != p.positions)
                p.positions_out[(int64_t)r * p.po_stride + j] = pos ? pos[j] : j;
        }
        if (rank == 0 && tid == 0) p.num_moves[r] = 0;
        sync_all(ctas);  // every CTA has read the length
    }
    pdl_launch_dependents();
    if (rank == 0 && tid == 0) {
        p.seq_lens_out[r] = wide ? seq : m;
        if (wide && p.err) atomicAdd(p.err, 1);
    }
    if (ctas > 1) cluster_sync();  // nothing of this CTA is read any more
}

// ---- moving the records ---------------------------------------------------------------
//
// A CTA takes kMoves moves of a request at a time: their addresses are looked up side by
// side, then all threads copy 16-byte pieces of data (and the scales) of all of them.
// 53500 records of 584 bytes: 14.8 us, 4.2 TB/s read and written, of the 6.7 measured; a
// chain of three reads (count, move, table entry) precedes each tile's copies, and only three
// CTAs an SM cover it (70 to 80 registers a thread, for the five accesses in flight; the grid has
// eight an SM).  57600 MXFP4 records of 68 bytes: 9.9 us; a tile of them has 160 pieces for 256
// threads.  One record in each of 64 requests: 2.9 us.
constexpr int kMoves = 32, kMoveThreads = 256;

// Of a request; max_moves may be all 31 bits.
__host__ __device__ __forceinline__ int32_t move_tiles(const MoveParams& p) {
    return p.max_moves / kMoves + (p.max_moves % kMoves != 0);
}

template <typename Unit>  // of the scales
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
    __shared__ int64_t s_at[kMoves][4];  // data from, data to, scales from, scales to; -1: no page
    pdl_wait();
    const int32_t pieces = p.data_bytes / 16, scales = p.scale_bytes / (int32_t)sizeof(Unit);
    const int32_t per = pieces + scales;
    const int32_t tiles = move_tiles(p);
    // the first tiles of all requests come first: the filled ones spread evenly over the CTAs
    for (int64_t id = blockIdx.x; id < (int64_t)tiles * p.num_reqs; id += gridDim.x) {
        const int32_t r = (int32_t)(id % p.num_reqs), first = (int32_t)(id / p.num_reqs) * kMoves;
        const int32_t count = min(min(max(p.num_moves[r], 0), p.max_moves) - first, kMoves);
        if (count <= 0) continue;
        __syncthreads();  // the last tile's addresses have been read
        if (threadIdx.x < 2 * count) {
            const int i = threadIdx.x / 2, to = threadIdx.x % 2;
            const int2 move = p.moves[(int64_t)r * p.moves_stride + first + i];
            const int32_t row = to ? move.y : move.x;
            int64_t data = -1, scale = -1;
            if (row >= 0) {
                int32_t off;
                const int64_t logical = (int64_t)div_block32(row, p.block_size, p.shift, off) - (p.base ? p.base[r] : 0);
                if (logical >= 0 && logical < p.bt_width) {
                    const int32_t page = p.bt[(int64_t)r * p.bt_stride + logical];
                    if (page >= 0 && page < p.num_pages) {
                        data = page * p.page_stride + (int64_t)off * p.data_bytes;
                        scale = page * p.page_stride + (int64_t)p.block_size * p.data_bytes + (int64_t)off * p.scale_bytes;
                    }
                }
            }
            s_at[i][to] = data;
            s_at[i][2 + to] = scale;
        }
        __syncthreads();
        if (p.err && threadIdx.x < count && (s_at[threadIdx.x][0] < 0 || s_at[threadIdx.x][1] < 0)) atomicAdd(p.err, 1);
        constexpr int kAtOnce = 5;
        for (int32_t c0 = threadIdx.x; c0 < count * per; c0 += kAtOnce * kMoveThreads) {
            uint4 v[kAtOnce];
            Unit u[kAtOnce];
            uint8_t* to[kAtOnce];
            bool data[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int32_t c = c0 + k * kMoveThreads;
                to[k] = nullptr;
                if (c >= count * per) continue;
                const int32_t i = c / per, piece = c - i * per;
                data[k] = piece < pieces;
                if (s_at[i][0] < 0 || s_at[i][1] < 0) continue;
                const int64_t off = data[k] ? (int64_t)piece * 16 : (int64_t)(piece - pieces) * (int64_t)sizeof(Unit);
                const uint8_t* from = p.cache + s_at[i][data[k] ? 0 : 2] + off;
                to[k] = p.cache + s_at[i][data[k] ? 1 : 3] + off;
                if (data[k])
                    v[k] = *reinterpret_cast<const uint4*>(from);
                else
                    u[k] = *reinterpret_cast<const Unit*>(from);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (to[k] == nullptr) continue;
                if (data[k])
                    *reinterpret_cast<uint4*>(to[k]) = v[k];
                else
                    *reinterpret_cast<Unit*>(to[k]) = u[k];
            }
        }
    }
    pdl_launch_dependents();
}

constexpr int kMostKeys = 48 * 1024;  // of a CTA's rows in shared memory

}  // namespace

cudaError_t launch_select_evictions(const SelectParams& p, cudaStream_t stream) {
    // 4096 rows or more a CTA, and clusters that run at the same time: a CTA fills an SM, and what a
    // GPC has left over cannot take part.  us at 32768 rows a request in clusters of 1, 2, 4 and 8:
    // 8 requests 39.8, 27.1, 18.8, 18.7; 12 39.8, 27.1, 18.9, 19.3; 16 39.8, 27.1, 18.9, 35.7;
    // 25 40.0, 27.1, 19.4, 38.3; 32 40.0, 27.2, 19.5, 54.5; 40 40.0, 27.3, 37.5, 56.9; 64 40.2,
    // 27.3, 38.5, 91.3; 100 40.3, 53.7, 57.4, 130.  The rule takes the best up to 25 requests and
    // is careful past that: 26 to 38 requests could have clusters of four, 51 to 76 of two.
    int ctas = 1;
    while (ctas < kMostCtas && (int64_t)ctas * 4096 < p.width && 3 * ctas * (int64_t)p.num_reqs <= sm_count()) ctas *= 2;
    const int32_t groups = (p.width + kWarp - 1) / kWarp, warps = ctas * kWarps;
    const int64_t keys = (int64_t)((groups + warps - 1) / warps) * kThreads;
    const bool cached = keys <= kMostKeys;
    const size_t smem = cached ? (size_t)keys * 4 : 0;
    auto* k = cached ? select_kernel<true> : select_kernel<false>;
    if (cached) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = set_smem_limit_per_device(k, kMostKeys * 4, done);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl_clusters(k, ctas, dim3((unsigned)(p.num_reqs * (int64_t)ctas)), dim3(kThreads), smem, stream, p, ctas);
}

cudaError_t launch_move_rows(MoveParams p, cudaStream_t stream) {
    p.shift = log2_if_pow2(p.block_size);
    const int64_t tiles = (int64_t)move_tiles(p) * p.num_reqs, most = (int64_t)sm_count() * 8;
    const dim3 grid((unsigned)(tiles < most ? tiles : most));
    auto* k = p.scale_bytes >= 16  ? move_kernel<uint4>
              : p.scale_bytes == 8 ? move_kernel<uint2>
              : p.scale_bytes == 4 ? move_kernel<uint32_t>
              : p.scale_bytes == 2 ? move_kernel<uint16_t>
                                   : move_kernel<uint8_t>;
    return launch_pdl(k, grid, dim3(kMoveThreads), 0, stream, p);
}

}  // namespace psk
