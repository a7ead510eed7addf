// batch_meta.cu -- batch metadata built on the device: positions, the
// token-to-request map and cache slots from request lengths, and block tables
// grown from request lengths and a list of unused pages.
#include "batch_meta.h"
#include "psk_common.cuh"

namespace psk {
namespace {

constexpr int kThreads = 256;

// ---- slot maps -------------------------------------------------------------------
//
// Token t of request r (qsl[r] <= t < qsl[r + 1]) sits at
//   pos = seq_lens[r] - (qsl[r + 1] - qsl[r]) + (t - qsl[r]),
// its slot is table[r][pos / bs - base[r]] * bs + pos % bs.  The request is found
// by binary search; up to kStageReqs boundaries are staged in shared memory by
// one coalesced read, so that the search costs no chain of L2 reads.
//
// With few tokens the time is the launch and a chain of four dependent reads (boundary,
// length, table, store): 256 tokens 2.7 us.  With many it is 2.3 times that of the 28 bytes
// written per token (1000003 tokens of 37 requests 9.6 us, 2.9 TB/s of the 6.8 measured),
// with 55 % of the issue slots in use.  No unit is full; the chain of a search and three
// reads, in 2.6 waves of CTAs, is the likely rest.  Two tokens a thread halve the searches
// and make every store of a warp 512 contiguous bytes (one takes 11.2 us; four, whose
// 16-byte stores leave gaps, 11.9), which pays once the SMs are full: 300000 tokens 4.37 us
// against 4.64 with one, 100000 3.55 against 2.90.  Staging the boundaries: 256 requests 2.76 us against 3.24 from L2, 4000
// requests of 250 tokens 13.3 against 13.9, 8000 of 125 15.0 against 14.4.
constexpr int kStageReqs = 4096;

__device__ __forceinline__ int64_t map_slot(const SlotMapTable& m, int32_t r, int64_t entry) {
    if (entry < 0) return -1;
    int64_t off;
    const int64_t logical = div_block(entry, m.block_size, m.shift, off) -
                            (m.base ? (int64_t)m.base[r] : 0);
    if (logical < 0 || logical >= m.width) return -1;
    const int32_t page = m.bt[(int64_t)r * m.stride + logical];
    return page < 0 ? -1 : (int64_t)page * m.block_size + off;
}

// V consecutive tokens per thread; kStage: the boundaries are staged.
template <int V, bool kStage>
__global__ void __launch_bounds__(kThreads) slot_map_kernel(const SlotMapParams p) {
    extern __shared__ int32_t s_qsl[];
    pdl_wait();
    const int32_t R = p.num_reqs;
    const int32_t* qsl = p.qsl;
    if (kStage) {
        for (int i = threadIdx.x; i <= R; i += kThreads) s_qsl[i] = p.qsl[i];
        __syncthreads();
        qsl = s_qsl;
    }
    const int64_t t0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V;
    if (t0 >= p.num_tokens) {
        pdl_launch_dependents();
        return;
    }
    // the last r in [0, R) with qsl[r] <= t0 (0 if there is none)
    int32_t lo = 0, hi = R;
    while (hi - lo > 1) {
        const int32_t mid = lo + ((hi - lo) >> 1);
        if (qsl[mid] <= t0) lo = mid; else hi = mid;
    }
    int32_t r = lo, at = -1;
    int32_t q0 = 0, q1 = 0, seq = 0;
    int64_t pos[V], slot[V], comp[V];
    int32_t req[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t t = t0 + v;
        while (r + 1 < R && qsl[r + 1] <= t) ++r;
        if (at != r) {
            q0 = qsl[r];
            q1 = qsl[r + 1];
            seq = p.seq_lens[r];
            at = r;
        }
        const bool in = t >= q0 && t < q1;  // else the token is padding
        req[v] = in ? r : -1;
        pos[v] = in ? (int64_t)seq - ((int64_t)q1 - q0) + (t - q0) : -1;
        slot[v] = p.slots && in ? map_slot(p.main, r, pos[v]) : -1;
        comp[v] = -1;
        if (p.comp_slots && in && pos[v] >= 0) {
            int64_t rem;
            const int64_t e = div_block(pos[v] + 1, p.compress_ratio, p.ratio_shift, rem);
            if (rem == 0) comp[v] = map_slot(p.comp, r, e - 1);
        }
    }
    pdl_launch_dependents();
    if constexpr (V == 2) {
        if (t0 + V <= p.num_tokens) {  // 16-byte stores: the launcher checked the alignment
            const auto put = [&](int64_t* dst, const int64_t* x) {
                if (dst) *reinterpret_cast<longlong2*>(dst + t0) = make_longlong2(x[0], x[1]);
            };
            put(p.positions, pos);
            put(p.slots, slot);
            put(p.comp_slots, comp);
            if (p.token_to_req)
                *reinterpret_cast<int2*>(p.token_to_req + t0) = make_int2(req[0], req[1]);
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t t = t0 + v;
        if (t >= p.num_tokens) break;
        if (p.positions) p.positions[t] = pos[v];
        if (p.token_to_req) p.token_to_req[t] = req[v];
        if (p.slots) p.slots[t] = slot[v];
        if (p.comp_slots) p.comp_slots[t] = comp[v];
    }
}

// ---- block tables ------------------------------------------------------------------
//
// Row r holds have = page_counts[r] pages and needs ceil((seq / ratio) / bs); the
// missing ones are pool[start_r ...], start_r = head + the demand of all earlier
// rows.  Every CTA works out the demand before its first row by itself (two reads
// per earlier row, from L2), so rows are filled in parallel by one launch that
// keeps no counters; the CTA whose rows hold the last served one writes the head.
//
// Bound by the table written and the pages read, and by the chain before them
// (counts and lengths of all earlier rows, the head, the pages): 2048 rows of 2048
// columns 8.7 us, 3.0 TB/s of the 6.8 measured; 256 rows of 128 2.4 us.  Measured before
// powers of two were divided by shifts, when this form took 11.1: the tails of the rows
// filled before the demand is known 12.5, one row a CTA 13.0, 512 threads a CTA 13.6.

struct Demand {
    int32_t have, more;
    bool wide;  // needs more columns than the table has
};

__device__ __forceinline__ Demand demand_of(const ExtendParams& p, int32_t r) {
    Demand d;
    const int32_t seq = max(p.seq_lens[r], 0);
    int32_t rem;
    const int32_t entries = div_block32(seq, p.compress_ratio, p.ratio_shift, rem);
    const int32_t whole = div_block32(entries, p.block_size, p.block_shift, rem);
    const int32_t need = whole + (rem != 0 ? 1 : 0);
    d.have = p.page_counts ? min(max(p.page_counts[r], 0), p.bt_width) : 0;
    d.wide = need > p.bt_width;
    d.more = d.wide ? 0 : max(need - d.have, 0);
    return d;
}

__global__ void __launch_bounds__(kThreads) extend_tables_kernel(const ExtendParams p) {
    __shared__ int64_t s_part[kThreads / kWarp];
    __shared__ int64_t s_before;
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const int32_t R = p.num_reqs;
    const int32_t r0 = (int32_t)blockIdx.x * p.rows_per_cta;
    const int32_t r1 = min(R, r0 + p.rows_per_cta);

    int64_t sum = 0;
#pragma unroll 4
    for (int32_t r = tid; r < r0; r += kThreads) sum += demand_of(p, r).more;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) s_part[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        int64_t all = p.pool_head ? max(*p.pool_head, 0) : 0;
        for (int w = 0; w < kThreads / kWarp; ++w) all += s_part[w];
        s_before = all;
    }
    __syncthreads();

    int64_t start = s_before;
    int64_t head = start;  // end of the last served range so far
    const bool own_head = start <= p.pool_size || blockIdx.x == 0;
    for (int32_t r = r0; r < r1; ++r) {
        const Demand d = demand_of(p, r);
        const bool served = d.more == 0 || start + d.more <= p.pool_size;
        const int32_t got = served ? d.more : 0;
        int32_t* row = p.bt + (int64_t)r * p.bt_stride;
        const int32_t count = d.have + got;
        for (int32_t c = d.have + tid; c < count; c += kThreads)
            row[c] = p.pool[start + (c - d.have)];
        // -1 past the row's pages: 16 bytes a thread between the unaligned ends
        const int32_t lead = (int32_t)((16 - (reinterpret_cast<uintptr_t>(row + count) & 15)) & 15) / 4;
        const int32_t a = min(p.bt_width, count + lead);
        const int32_t b = a + (p.bt_width - a) / 4 * 4;
        for (int32_t c = count + tid; c < a; c += kThreads) row[c] = -1;
        for (int32_t c = a + 4 * tid; c < b; c += 4 * kThreads)
            *reinterpret_cast<int4*>(row + c) = make_int4(-1, -1, -1, -1);
        for (int32_t c = b + tid; c < p.bt_width; c += kThreads) row[c] = -1;
        if (tid == 0) {
            p.page_counts_out[r] = count;
            if (p.err_count && (d.wide || !served)) atomicAdd(p.err_count, 1);
        }
        start += d.more;
        if (served && d.more > 0) head = start;
    }
    pdl_launch_dependents();
    // Exactly one CTA has a start within the pool and an end past it (or is the
    // last one); a head past the pool leaves nothing to serve and CTA 0 keeps it.
    if (tid == 0 && own_head) {
        const bool past = blockIdx.x == 0 && s_before > p.pool_size;
        if (past || start > p.pool_size || r1 == R) *p.pool_head_out = (int32_t)head;
    }
}

}  // namespace

cudaError_t launch_slot_mappings(SlotMapParams p, cudaStream_t stream) {
    p.main.shift = log2_if_pow2(p.main.block_size);
    p.comp.shift = log2_if_pow2(p.comp.block_size);
    p.ratio_shift = log2_if_pow2(p.compress_ratio);
    const uintptr_t all = reinterpret_cast<uintptr_t>(p.positions) |
                          reinterpret_cast<uintptr_t>(p.token_to_req) |
                          reinterpret_cast<uintptr_t>(p.slots) |
                          reinterpret_cast<uintptr_t>(p.comp_slots);
    const bool two = all % 16 == 0 && p.num_tokens >= (int64_t)sm_count() * kThreads * 6;
    const bool stage = p.num_reqs < kStageReqs;
    const int V = two ? 2 : 1;
    const int64_t ctas = (p.num_tokens + (int64_t)kThreads * V - 1) / ((int64_t)kThreads * V);
    const size_t smem = stage ? (size_t)(p.num_reqs + 1) * 4 : 0;
    auto* k = two ? (stage ? slot_map_kernel<2, true> : slot_map_kernel<2, false>)
                   : (stage ? slot_map_kernel<1, true> : slot_map_kernel<1, false>);
    return launch_pdl(k, dim3((unsigned)ctas), dim3(kThreads), smem, stream, p);
}

cudaError_t launch_extend_block_tables(ExtendParams p, cudaStream_t stream) {
    p.ratio_shift = log2_if_pow2(p.compress_ratio);
    p.block_shift = log2_if_pow2(p.block_size);
    const int64_t most = (int64_t)sm_count() * 8;  // eight CTAs of 256 threads fill an SM
    p.rows_per_cta = (int32_t)((p.num_reqs + most - 1) / most);
    const int32_t ctas = (p.num_reqs + p.rows_per_cta - 1) / p.rows_per_cta;
    return launch_pdl(extend_tables_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, stream, p);
}

}  // namespace psk
