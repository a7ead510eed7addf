// abi.cu -- the extern "C" entry points of libpsk (declared in include/psk.h).
//
// Each entry point validates its arguments on the host, returns
// PSK_ERR_INVALID_ARGUMENT before touching the GPU when they are wrong,
// returns PSK_OK without a launch when there is no work, and otherwise
// launches one kernel (the attention calls and the accumulation of their weights one or two)
// on the caller's stream.  Nothing here allocates, synchronises or keeps state beyond the
// per-thread error text.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>
#include <utility>

#include "attention.h"
#include "attn_weights.h"
#include "batch_meta.h"
#include "compressor.h"
#include "evict.h"
#include "gather.h"
#include "index_build.h"
#include "insert.h"
#include "launch.h"
#include "psk.h"
#include "psk_common.cuh"
#include "rotary.h"

namespace {

thread_local std::string g_last_error;

psk_status fail(psk_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

psk_status ok() {
    g_last_error.clear();
    return PSK_OK;
}

psk_status cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return ok();
    return fail(PSK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define CHECK(cond, ...)                                                \
    do {                                                                \
        if (!(cond)) return fail(PSK_ERR_INVALID_ARGUMENT, __VA_ARGS__); \
    } while (0)

bool fp8_head_dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256 || d == 512 || d == 1024; }
bool mxfp4_head_dim_ok(int32_t d) {
    return d == 32 || d == 64 || d == 128 || d == 256 || d == 512 || d == 1024;
}

int64_t fp8_record_bytes(int32_t head_dim, int32_t rope_dim, int32_t ue8m0) {
    return (int64_t)(head_dim - rope_dim) + 2 * (int64_t)rope_dim +
           (int64_t)(head_dim / 64) * (ue8m0 ? 1 : 4);
}

psk_status check_cache(const uint8_t* cache, int64_t num_pages, int64_t page_stride,
                       int32_t block_size, int64_t record_bytes) {
    CHECK(cache != nullptr, "cache is null");
    CHECK(num_pages >= 1, "num_pages must be >= 1 (got %lld)", (long long)num_pages);
    CHECK(block_size >= 1, "block_size must be >= 1 (got %d)", block_size);
    CHECK(page_stride >= (int64_t)block_size * record_bytes,
          "page_stride %lld is smaller than block_size * record bytes = %lld",
          (long long)page_stride, (long long)block_size * record_bytes);
    CHECK(page_stride % 16 == 0, "page_stride must be a multiple of 16 bytes");
    CHECK(aligned(cache, 16), "cache must be 16-byte aligned");
    CHECK(num_pages <= INT64_MAX / page_stride, "cache size overflows int64");
    return PSK_OK;
}

bool attn_head_dim_ok(int32_t d) { return d == 128 || d == 256 || d == 512; }

// The arguments both attention entry points share.  `work` = false where the
// call has no tokens: pointers are not looked at.
psk_status check_attention(const psk::AttnParams& p, bool work, int64_t workspace_need,
                           int64_t workspace_bytes) {
    CHECK(p.num_heads >= 1, "num_heads must be >= 1");
    CHECK(std::isnormal(p.scale) && p.scale > 0.0f && p.scale <= 1e38f,
          "softmax_scale must be a normal number in (0, 1e38]");
    CHECK(p.q_stride_t >= 0 && p.q_stride_h >= 0 && p.q_stride_t % 8 == 0 &&
              p.q_stride_h % 8 == 0,
          "query strides must be non-negative multiples of 8 elements");
    CHECK(p.out_stride_t % 8 == 0 && p.out_stride_h % 8 == 0 &&
              (p.num_tokens <= 1 || p.out_stride_t >= p.head_dim) &&
              (p.num_heads <= 1 || p.out_stride_h >= p.head_dim) && p.out_stride_t >= 0 &&
              p.out_stride_h >= 0,
          "output strides must be multiples of 8 elements and at least head_dim");
    CHECK(p.lse == nullptr || p.num_tokens <= 1 || p.lse_stride_t >= p.num_heads,
          "lse_stride_t must be >= num_heads");
    if (!work) return PSK_OK;
    CHECK(p.num_tokens <= (int64_t)INT32_MAX, "num_tokens must fit in int32");
    CHECK(p.q != nullptr && p.out != nullptr, "q and out must be non-null");
    CHECK(aligned(p.q, 16) && aligned(p.out, 16), "q and out must be 16-byte aligned");
    CHECK(aligned(p.sink, 4) && aligned(p.lse, 4), "sink and lse must be 4-byte aligned");
    CHECK(workspace_bytes >= workspace_need, "workspace must hold %lld bytes (got %lld)",
          (long long)workspace_need, (long long)workspace_bytes);
    CHECK(workspace_need == 0 || (p.workspace != nullptr && aligned(p.workspace, 16)),
          "workspace must be non-null and 16-byte aligned");
    return PSK_OK;
}

// Whether rows of `dim` elements share memory, `rows` of them t apart in each of `heads` groups that are h
// apart; both at least dim.
bool rows_overlap(int64_t rows, int64_t t, int64_t heads, int64_t h, int64_t dim) {
    if (rows <= 1 || heads <= 1 || t >= (heads - 1) * h + dim || h >= (rows - 1) * t + dim) return false;
    if (rows < heads) {
        std::swap(rows, heads);
        std::swap(t, h);
    }
    for (int64_t b = 1; b < heads; ++b) {  // b groups on, the nearest rows: a and a + 1
        const int64_t a = b * h / t, rest = b * h % t;
        if (a >= rows) break;
        if ((a >= 1 && rest < dim) || (a + 1 < rows && t - rest < dim)) return true;
    }
    return false;
}

// The strides of one of apply_rotary_embedding's tensors, in elements of `size` bytes.
psk_status check_rotary(const void* in, int64_t it, int64_t ih, const void* out, int64_t ot, int64_t oh,
                        int32_t heads, int64_t num_tokens, int32_t head_dim, int32_t size, const char* name) {
    CHECK(heads >= 1, "the number of heads of %s must be >= 1", name);
    CHECK(in != nullptr && out != nullptr, "%s and its output must be non-null", name);
    CHECK(aligned(in, size) && aligned(out, size), "%s and its output must be aligned to their elements", name);
    CHECK(it >= 0 && ih >= 0 && ot >= 0 && oh >= 0, "strides of %s must not be negative", name);
    const int64_t most = INT64_MAX / 8;
    const int64_t most_t = num_tokens > 1 ? most / (num_tokens - 1) : most, most_h = heads > 1 ? most / (heads - 1) : most;
    CHECK(it <= most_t && ih <= most_h && ot <= most_t && oh <= most_h, "strides of %s overflow", name);
    CHECK((num_tokens <= 1 || ot >= head_dim) && (heads <= 1 || oh >= head_dim),
          "output strides of %s must be at least head_dim", name);
    CHECK(!rows_overlap(num_tokens, ot, heads, oh, head_dim), "output rows of %s must not overlap", name);
    CHECK(in != out || ((num_tokens <= 1 || it == ot) && (heads <= 1 || ih == oh)),
          "%s in place needs equal strides", name);
    return PSK_OK;
}

// A number as the unevaluated sum of two doubles, |lo| <= ulp(hi) / 2: 106 bits (Dekker's sums, Knuth's
// error of a sum, the error of a product by a fused multiply-add).
struct Wide {
    double hi, lo;
};

Wide normal(double a, double b) {
    const double s = a + b;
    return {s, b - (s - a)};
}

Wide operator+(Wide a, Wide b) {
    const double s = a.hi + b.hi, v = s - a.hi;
    return normal(s, ((a.hi - (s - v)) + (b.hi - v)) + (a.lo + b.lo));
}

Wide operator*(Wide a, Wide b) {
    const double p = a.hi * b.hi;
    return normal(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}

Wide operator/(Wide a, double b) {
    const double q = a.hi / b;
    return normal(q, (std::fma(-q, b, a.hi) + a.lo) / b);
}

// theta^(-1/n), n <= 256: Newton's step from the nearest double.  The powers are of a number in [1/2, 1),
// with the exponents of two apart, so that none underflows.
Wide inverse_root(double theta, int32_t n) {
    int e0, e1;
    const double x = std::frexp(std::pow(theta, -1.0 / n), &e0), t = std::frexp(theta, &e1);
    Wide power = {t, 0.0}, square = {x, 0.0};
    for (int32_t bits = n; bits != 0; bits /= 2, square = square * square)
        if (bits % 2 != 0) power = power * square;
    const int e = e0 * n + e1;
    power = {std::ldexp(power.hi, e), std::ldexp(power.lo, e)};  // x^n theta, nearly 1
    const double off = (power.hi - 1.0) + power.lo;
    const Wide root = normal(x, -x * off / n);
    return {std::ldexp(root.hi, e0), std::ldexp(root.lo, e0)};
}

// 2^64 w, rounded; 0 <= w < 1.
uint64_t fraction64(Wide w) {
    const double a = std::ldexp(w.hi, 64), whole = std::floor(a);
    return (uint64_t)whole + (uint64_t)(int64_t)std::floor((a - whole) + std::ldexp(w.lo, 64) + 0.5);
}

// The largest number of positions a token of a call can see.
int64_t chunk_max_keys(int32_t bt_width, int32_t block_size, int32_t window) {
    const int64_t all = (int64_t)bt_width * block_size;
    return window > 0 && window < all ? window : all;
}

}  // namespace

extern "C" {

const char* psk_last_error(void) { return g_last_error.c_str(); }

int32_t psk_abi_version(void) { return 7; }

psk_status psk_device_wait_timeouts(uint32_t* count) {
    CHECK(count != nullptr, "count must be non-null");
    uint32_t gather = 0, index = 0, compress = 0, attention = 0, weights = 0;
    psk_status st = cuda_status(psk::read_wait_timeouts(&gather), "reading the wait-timeout counter");
    if (st != PSK_OK) return st;
    st = cuda_status(psk::read_index_wait_timeouts(&index), "reading the wait-timeout counter");
    if (st != PSK_OK) return st;
    st = cuda_status(psk::read_compress_wait_timeouts(&compress), "reading the wait-timeout counter");
    if (st != PSK_OK) return st;
    st = cuda_status(psk::read_attention_wait_timeouts(&attention),
                     "reading the wait-timeout counter");
    if (st != PSK_OK) return st;
    st = cuda_status(psk::read_attn_weights_wait_timeouts(&weights), "reading the wait-timeout counter");
    if (st != PSK_OK) return st;
    *count = gather + index + compress + attention + weights;
    return PSK_OK;
}

psk_status psk_device_wait_selftest(uint64_t limit_ns, psk_stream_t stream) {
    CHECK(limit_ns >= 1000 && limit_ns <= 1000000000ull, "limit_ns must be in [1e3, 1e9]");
    return cuda_status(psk::launch_wait_selftest(limit_ns, reinterpret_cast<cudaStream_t>(stream)),
                       "psk_device_wait_selftest launch");
}

psk_status quantize_and_insert_k_cache(const void* k, int64_t k_row_stride,
                                       const int64_t* slot_mapping, int64_t num_tokens,
                                       uint8_t* k_cache, int64_t num_pages, int64_t page_stride,
                                       int32_t block_size, int32_t head_dim, int32_t rope_dim,
                                       int32_t is_ue8m0, int32_t* err_count,
                                       psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(is_ue8m0 == 0 || is_ue8m0 == 1, "is_ue8m0 must be 0 or 1");
    CHECK(fp8_head_dim_ok(head_dim), "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)",
          head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    psk_status st = check_cache(k_cache, num_pages, page_stride, block_size,
                                fp8_record_bytes(head_dim, rope_dim, is_ue8m0));
    if (st != PSK_OK) return st;
    if (num_tokens == 0) return ok();
    CHECK(k != nullptr && slot_mapping != nullptr, "k and slot_mapping must be non-null");
    CHECK(aligned(k, 16), "k must be 16-byte aligned");
    CHECK(k_row_stride >= head_dim && k_row_stride % 8 == 0,
          "k_row_stride must be >= head_dim and a multiple of 8 elements");
    CHECK(aligned(slot_mapping, 8), "slot_mapping must be 8-byte aligned");
    CHECK(err_count == nullptr || aligned(err_count, 4), "err_count must be 4-byte aligned");
    psk::InsertParams p{k, k_row_stride, slot_mapping, num_tokens, k_cache, num_pages,
                        page_stride, block_size, head_dim, rope_dim, is_ue8m0, err_count};
    return cuda_status(psk::launch_fp8_insert(p, reinterpret_cast<cudaStream_t>(stream)),
                       "quantize_and_insert_k_cache launch");
}

psk_status write_indexer_mxfp4_cache(const void* index_k, int64_t k_row_stride,
                                     const int64_t* slot_mapping, int64_t num_tokens,
                                     uint8_t* cache, int64_t num_pages, int64_t page_stride,
                                     int32_t block_size, int32_t head_dim, int32_t* err_count,
                                     psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(mxfp4_head_dim_ok(head_dim),
          "head_dim must be one of 32, 64, 128, 256, 512, 1024 (got %d)", head_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size,
                                head_dim / 2 + head_dim / 32);
    if (st != PSK_OK) return st;
    if (num_tokens == 0) return ok();
    CHECK(index_k != nullptr && slot_mapping != nullptr,
          "index_k and slot_mapping must be non-null");
    CHECK(aligned(index_k, 16), "index_k must be 16-byte aligned");
    CHECK(k_row_stride >= head_dim && k_row_stride % 8 == 0,
          "k_row_stride must be >= head_dim and a multiple of 8 elements");
    CHECK(aligned(slot_mapping, 8), "slot_mapping must be 8-byte aligned");
    CHECK(err_count == nullptr || aligned(err_count, 4), "err_count must be 4-byte aligned");
    psk::InsertParams p{index_k, k_row_stride, slot_mapping, num_tokens, cache, num_pages,
                        page_stride, block_size, head_dim, 0, 1, err_count};
    return cuda_status(psk::launch_mxfp4_insert(p, reinterpret_cast<cudaStream_t>(stream)),
                       "write_indexer_mxfp4_cache launch");
}

psk_status compute_global_topk_indices_and_lens(
    const int32_t* topk_local, int64_t topk_stride, int64_t num_tokens, int32_t topk,
    const int32_t* token_to_req, const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    int32_t num_reqs, int32_t block_size, const int32_t* base_offsets,
    const uint8_t* is_valid_token, int32_t* out_indices, int64_t out_stride, int32_t* out_lens,
    psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(topk >= 0, "topk must be >= 0");
    CHECK(block_size >= 1, "block_size must be >= 1");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    CHECK(topk_stride >= topk && out_stride >= topk, "row strides must be >= topk");
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(token_to_req && out_lens, "token_to_req and out_lens must be non-null");
    CHECK(topk == 0 || (topk_local && out_indices), "topk_local and out_indices must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(topk_local, 4) && aligned(out_indices, 4) && aligned(token_to_req, 4) &&
              aligned(block_table, 4) && aligned(base_offsets, 4) && aligned(out_lens, 4),
          "int32 arrays must be 4-byte aligned");
    psk::IndexParams p{};
    p.t2r = token_to_req;
    p.num_reqs = num_reqs;
    p.num_tokens = num_tokens;
    p.comp_bt = block_table;
    p.comp_stride = bt_stride;
    p.comp_width = bt_width;
    p.comp_base = base_offsets;
    p.comp_bs = block_size;
    p.comp_shift = psk::log2_if_pow2(block_size);
    p.window = 0;
    p.topk = topk;
    p.out_cols = topk;
    p.topk_local = topk_local;
    p.topk_stride = topk_stride;
    p.valid = is_valid_token;
    p.out = out_indices;
    p.out_stride = out_stride;
    p.lens = out_lens;
    return cuda_status(psk::launch_index_build(p, false, reinterpret_cast<cudaStream_t>(stream)),
                       "compute_global_topk_indices_and_lens launch");
}

psk_status combine_topk_swa_indices(
    const int32_t* query_start_loc, const int32_t* seq_lens, const int32_t* token_to_req,
    const int32_t* replay_start, int32_t num_reqs, int64_t num_tokens,
    const int32_t* swa_block_table, int64_t swa_bt_stride, int32_t swa_bt_width,
    const int32_t* swa_base_offsets, int32_t swa_block_size, const int32_t* comp_block_table,
    int64_t comp_bt_stride, int32_t comp_bt_width, const int32_t* comp_base_offsets,
    int32_t comp_block_size, int32_t window, int32_t compress_ratio, const int32_t* topk_local,
    int64_t topk_stride, int32_t topk, const uint8_t* is_valid_token, int32_t* sparse_indices,
    int64_t out_stride, int32_t* lens, psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(window >= 0 && topk >= 0, "window and topk must be >= 0");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(swa_block_size >= 1 && comp_block_size >= 1, "block sizes must be >= 1");
    CHECK(swa_bt_width >= 0 && swa_bt_stride >= swa_bt_width,
          "need 0 <= swa_bt_width <= swa_bt_stride");
    if (comp_block_table != nullptr) {
        CHECK(comp_bt_width >= 0 && comp_bt_stride >= comp_bt_width,
              "need 0 <= comp_bt_width <= comp_bt_stride");
    }
    const int64_t padded = ((int64_t)topk + 3) / 4 * 4;
    const int64_t cols = (int64_t)window + padded;
    CHECK(cols <= INT32_MAX, "window + padded topk overflows int32");
    CHECK(topk_stride >= topk, "topk_stride must be >= topk");
    CHECK(out_stride >= cols, "out_stride must be >= window + roundup(topk, 4)");
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(query_start_loc && seq_lens && token_to_req && sparse_indices && lens,
          "query_start_loc, seq_lens, token_to_req, sparse_indices and lens must be non-null");
    CHECK(topk == 0 || topk_local, "topk_local must be non-null");
    CHECK(swa_bt_width == 0 || swa_block_table, "swa_block_table must be non-null");
    CHECK(aligned(query_start_loc, 4) && aligned(seq_lens, 4) && aligned(token_to_req, 4) &&
              aligned(replay_start, 4) && aligned(swa_block_table, 4) &&
              aligned(swa_base_offsets, 4) && aligned(comp_block_table, 4) &&
              aligned(comp_base_offsets, 4) && aligned(topk_local, 4) &&
              aligned(sparse_indices, 4) && aligned(lens, 4),
          "int32 arrays must be 4-byte aligned");
    psk::IndexParams p{};
    p.qsl = query_start_loc;
    p.seq_lens = seq_lens;
    p.t2r = token_to_req;
    p.replay = replay_start;
    p.num_reqs = num_reqs;
    p.num_tokens = num_tokens;
    p.swa_bt = swa_block_table;
    p.swa_stride = swa_bt_stride;
    p.swa_width = swa_bt_width;
    p.swa_base = swa_base_offsets;
    p.swa_bs = swa_block_size;
    p.swa_shift = psk::log2_if_pow2(swa_block_size);
    if (comp_block_table == nullptr) {
        p.comp_bt = swa_block_table;
        p.comp_stride = swa_bt_stride;
        p.comp_width = swa_bt_width;
    } else {
        p.comp_bt = comp_block_table;
        p.comp_stride = comp_bt_stride;
        p.comp_width = comp_bt_width;
    }
    p.comp_base = comp_base_offsets;
    p.comp_bs = comp_block_size;
    p.comp_shift = psk::log2_if_pow2(comp_block_size);
    p.window = window;
    p.topk = topk;
    p.out_cols = (int32_t)cols;
    p.topk_local = topk_local;
    p.topk_stride = topk_stride;
    p.valid = is_valid_token;
    p.out = sparse_indices;
    p.out_stride = out_stride;
    p.lens = lens;
    return cuda_status(psk::launch_index_build(p, true, reinterpret_cast<cudaStream_t>(stream)),
                       "combine_topk_swa_indices launch");
}

psk_status dequantize_and_gather_k_cache(void* out, int64_t out_stride_t, int64_t out_stride_j,
                                         const uint8_t* cache, int64_t num_pages,
                                         int64_t page_stride, int32_t block_size,
                                         psk_record record, int32_t head_dim, int32_t rope_dim,
                                         int32_t is_ue8m0, const int32_t* indices,
                                         int64_t idx_stride, int64_t rows, int32_t cols,
                                         psk_stream_t stream) {
    CHECK(rows >= 0 && cols >= 0, "rows and cols must be >= 0");
    CHECK(record == PSK_REC_FP8_DS_MLA || record == PSK_REC_MXFP4 ||
              record == PSK_REC_FP8_INDEXER,
          "unknown record %d", (int)record);
    int64_t rec_bytes;
    if (record == PSK_REC_FP8_INDEXER) {
        CHECK(mxfp4_head_dim_ok(head_dim),
              "head_dim must be one of 32, 64, 128, 256, 512, 1024 (got %d)", head_dim);
        CHECK(rope_dim == 0, "rope_dim must be 0 for the FP8 indexer record");
        rec_bytes = head_dim + 4;
    } else if (record == PSK_REC_FP8_DS_MLA) {
        CHECK(is_ue8m0 == 0 || is_ue8m0 == 1, "is_ue8m0 must be 0 or 1");
        CHECK(fp8_head_dim_ok(head_dim),
              "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)", head_dim);
        CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
              "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
        rec_bytes = fp8_record_bytes(head_dim, rope_dim, is_ue8m0);
    } else {
        CHECK(mxfp4_head_dim_ok(head_dim),
              "head_dim must be one of 32, 64, 128, 256, 512, 1024 (got %d)", head_dim);
        CHECK(rope_dim == 0, "rope_dim must be 0 for the MXFP4 record");
        rec_bytes = head_dim / 2 + head_dim / 32;
    }
    psk_status st = check_cache(cache, num_pages, page_stride, block_size, rec_bytes);
    if (st != PSK_OK) return st;
    CHECK(idx_stride >= cols, "idx_stride must be >= cols");
    if (rows == 0 || cols == 0) return ok();
    CHECK(out != nullptr && indices != nullptr, "out and indices must be non-null");
    CHECK(aligned(out, 16), "out must be 16-byte aligned");
    CHECK(out_stride_t >= 0 && out_stride_j >= 0 && out_stride_t % 8 == 0 &&
              out_stride_j % 8 == 0,
          "output strides must be non-negative multiples of 8 elements");
    CHECK(aligned(indices, 4), "indices must be 4-byte aligned");
    CHECK(rows <= INT64_MAX / (cols > 0 ? cols : 1), "rows * cols overflows");
    psk::GatherParams p{static_cast<uint16_t*>(out), out_stride_t, out_stride_j, cache,
                        num_pages, page_stride, block_size, (int32_t)record, head_dim,
                        rope_dim, is_ue8m0, indices, idx_stride, rows, cols};
    return cuda_status(psk::launch_gather(p, reinterpret_cast<cudaStream_t>(stream)),
                       "dequantize_and_gather_k_cache launch");
}

psk_status dequantize_and_gather_k_cache_ranges(
    void* out, int64_t out_stride_r, int64_t out_stride_i, int64_t out_rows, const uint8_t* cache,
    int64_t num_pages, int64_t page_stride, int32_t block_size, psk_record record,
    int32_t head_dim, int32_t rope_dim, int32_t is_ue8m0, const int32_t* seq_lens,
    const int32_t* gather_lens, const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    const int32_t* base_offsets, int32_t num_reqs, int64_t offset, psk_stream_t stream) {
    if (record != PSK_REC_FP8_DS_MLA)
        return fail(PSK_ERR_UNSUPPORTED, "the range form gathers fp8_ds_mla records only");
    CHECK(is_ue8m0 == 0 || is_ue8m0 == 1, "is_ue8m0 must be 0 or 1");
    CHECK(fp8_head_dim_ok(head_dim), "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)",
          head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size,
                                fp8_record_bytes(head_dim, rope_dim, is_ue8m0));
    if (st != PSK_OK) return st;
    CHECK(num_reqs >= 0, "num_reqs must be >= 0");
    CHECK(offset >= 0 && out_rows >= offset, "need 0 <= offset <= out_rows");
    CHECK(out_rows - offset <= INT32_MAX, "out_rows - offset must fit in int32");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    if (num_reqs == 0 || out_rows == offset) return ok();
    CHECK(out && seq_lens, "out and seq_lens must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(out, 16), "out must be 16-byte aligned");
    CHECK(out_stride_r >= 0 && out_stride_i >= 0 && out_stride_r % 8 == 0 && out_stride_i % 8 == 0,
          "output strides must be non-negative multiples of 8 elements");
    CHECK(aligned(seq_lens, 4) && aligned(gather_lens, 4) && aligned(block_table, 4) &&
              aligned(base_offsets, 4),
          "int32 arrays must be 4-byte aligned");
    psk::RangeParams p{static_cast<uint16_t*>(out), out_stride_r, out_stride_i, out_rows, offset,
                       cache, num_pages, page_stride, block_size, head_dim, rope_dim, is_ue8m0,
                       seq_lens, gather_lens, block_table, bt_stride, bt_width, base_offsets,
                       num_reqs};
    return cuda_status(psk::launch_gather_ranges(p, reinterpret_cast<cudaStream_t>(stream)),
                       "dequantize_and_gather_k_cache_ranges launch");
}

psk_status combine_topk_swa_workspace_indices(
    const int32_t* query_start_loc, const int32_t* seq_lens, const int32_t* gather_lens,
    const int32_t* token_to_req, int32_t num_reqs, int64_t num_tokens, int32_t window,
    int32_t compress_ratio, const int32_t* topk_local, int64_t topk_stride, int32_t topk,
    int64_t workspace_width, int64_t compressed_base, const uint8_t* is_valid_token,
    int32_t* indices, int64_t out_stride, int32_t* lens, psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(window >= 0 && topk >= 0, "window and topk must be >= 0");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(workspace_width >= 0 && compressed_base >= 0,
          "workspace_width and compressed_base must be >= 0");
    const int64_t cols = (int64_t)window + ((int64_t)topk + 3) / 4 * 4;
    CHECK(cols <= INT32_MAX, "window + padded topk overflows int32");
    CHECK(topk_stride >= topk, "topk_stride must be >= topk");
    CHECK(out_stride >= cols, "out_stride must be >= window + roundup(topk, 4)");
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(query_start_loc && seq_lens && gather_lens && token_to_req && indices && lens,
          "query_start_loc, seq_lens, gather_lens, token_to_req, indices and lens must be non-null");
    CHECK(topk == 0 || topk_local, "topk_local must be non-null");
    CHECK(aligned(query_start_loc, 4) && aligned(seq_lens, 4) && aligned(gather_lens, 4) &&
              aligned(token_to_req, 4) && aligned(topk_local, 4) && aligned(indices, 4) &&
              aligned(lens, 4),
          "int32 arrays must be 4-byte aligned");
    psk::WorkspaceIndexParams p{query_start_loc, seq_lens, gather_lens, token_to_req, num_reqs,
                                num_tokens, window, compress_ratio, topk_local, topk_stride,
                                topk, workspace_width, compressed_base, is_valid_token, indices,
                                out_stride, lens, nullptr};
    return cuda_status(psk::launch_workspace_indices(p, reinterpret_cast<cudaStream_t>(stream)),
                       "combine_topk_swa_workspace_indices launch");
}

psk_status indexer_mxfp4_paged_gather(uint8_t* values_out, uint8_t* scales_out,
                                      const uint8_t* cache, int64_t num_pages,
                                      int64_t page_stride, int32_t block_size, int32_t head_dim,
                                      const int32_t* block_table, int64_t bt_stride,
                                      int32_t bt_width, const int32_t* cu_seq_lens,
                                      int32_t num_reqs, int64_t total_rows,
                                      psk_stream_t stream) {
    CHECK(mxfp4_head_dim_ok(head_dim),
          "head_dim must be one of 32, 64, 128, 256, 512, 1024 (got %d)", head_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size,
                                head_dim / 2 + head_dim / 32);
    if (st != PSK_OK) return st;
    CHECK(total_rows >= 0 && num_reqs >= 0, "total_rows and num_reqs must be >= 0");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    if (total_rows == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1 when total_rows > 0");
    CHECK(values_out && scales_out && cu_seq_lens, "outputs and cu_seq_lens must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(values_out, 4) && aligned(scales_out, 4) && aligned(cu_seq_lens, 4) &&
              aligned(block_table, 4),
          "values_out, scales_out and int32 arrays must be 4-byte aligned");
    psk::RawGatherParams p{values_out, scales_out, cache, num_pages, page_stride, block_size,
                           head_dim, block_table, bt_stride, bt_width, cu_seq_lens, num_reqs,
                           total_rows};
    return cuda_status(psk::launch_mxfp4_raw_gather(p, reinterpret_cast<cudaStream_t>(stream)),
                       "indexer_mxfp4_paged_gather launch");
}

psk_status decode_swa_indices_and_lens(
    const int32_t* query_start_loc, const int32_t* seq_lens, const int32_t* token_to_req,
    int32_t num_reqs, int64_t num_tokens, const int32_t* block_table, int64_t bt_stride,
    int32_t bt_width, const int32_t* base_offsets, int32_t block_size, int32_t window,
    const uint8_t* is_valid_token, int32_t* out_indices, int64_t out_stride, int32_t* out_lens,
    psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(window >= 0, "window must be >= 0");
    CHECK(block_size >= 1, "block_size must be >= 1");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    CHECK(out_stride >= window, "out_stride must be >= window");
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(query_start_loc && seq_lens && token_to_req && out_indices && out_lens,
          "query_start_loc, seq_lens, token_to_req, out_indices and out_lens must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(query_start_loc, 4) && aligned(seq_lens, 4) && aligned(token_to_req, 4) &&
              aligned(block_table, 4) && aligned(base_offsets, 4) && aligned(out_indices, 4) &&
              aligned(out_lens, 4),
          "int32 arrays must be 4-byte aligned");
    psk::IndexParams p{};
    p.qsl = query_start_loc;
    p.seq_lens = seq_lens;
    p.t2r = token_to_req;
    p.replay = nullptr;
    p.num_reqs = num_reqs;
    p.num_tokens = num_tokens;
    p.swa_bt = p.comp_bt = block_table;
    p.swa_stride = p.comp_stride = bt_stride;
    p.swa_width = p.comp_width = bt_width;
    p.swa_base = p.comp_base = base_offsets;
    p.swa_bs = p.comp_bs = block_size;
    p.swa_shift = p.comp_shift = psk::log2_if_pow2(block_size);
    p.window = window;
    p.topk = 0;
    p.out_cols = window;
    p.topk_local = nullptr;
    p.topk_stride = 0;
    p.valid = is_valid_token;
    p.out = out_indices;
    p.out_stride = out_stride;
    p.lens = out_lens;
    return cuda_status(psk::launch_index_build(p, true, reinterpret_cast<cudaStream_t>(stream)),
                       "decode_swa_indices_and_lens launch");
}

psk_status compute_dense_compressed_indices_and_lens(
    const int64_t* positions, int64_t num_tokens, const int32_t* token_to_req, int32_t num_reqs,
    const int32_t* block_table, int64_t bt_stride, int32_t bt_width, const int32_t* base_offsets,
    int32_t block_size, int32_t compress_ratio, int32_t width, const uint8_t* is_valid_token,
    int32_t* out_indices, int64_t out_stride, int32_t* out_lens, psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(width >= 0, "width must be >= 0");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(block_size >= 1, "block_size must be >= 1");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    CHECK(out_stride >= width, "out_stride must be >= width");
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(positions && token_to_req && out_lens,
          "positions, token_to_req and out_lens must be non-null");
    CHECK(width == 0 || out_indices, "out_indices must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(positions, 8), "positions must be 8-byte aligned");
    CHECK(aligned(token_to_req, 4) && aligned(block_table, 4) && aligned(base_offsets, 4) &&
              aligned(out_indices, 4) && aligned(out_lens, 4),
          "int32 arrays must be 4-byte aligned");
    CHECK(num_tokens <= ((int64_t)INT32_MAX * 256) / (width > 0 ? width : 1),
          "num_tokens x width is too large");
    psk::DenseParams p{positions, num_tokens, token_to_req, num_reqs, block_table, bt_stride,
                       bt_width, base_offsets, block_size, compress_ratio, width, is_valid_token,
                       out_indices, out_stride, out_lens};
    return cuda_status(psk::launch_dense_indices(p, true, reinterpret_cast<cudaStream_t>(stream)),
                       "compute_dense_compressed_indices_and_lens launch");
}

psk_status build_dense_prefill_local_compressed_indices(const int64_t* positions,
                                                        int64_t num_tokens,
                                                        int32_t compress_ratio, int32_t width,
                                                        int32_t* out, int64_t out_stride,
                                                        psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(width >= 0, "width must be >= 0");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(out_stride >= width, "out_stride must be >= width");
    if (num_tokens == 0 || width == 0) return ok();
    CHECK(positions && out, "positions and out must be non-null");
    CHECK(aligned(positions, 8), "positions must be 8-byte aligned");
    CHECK(aligned(out, 4), "out must be 4-byte aligned");
    CHECK(num_tokens <= ((int64_t)INT32_MAX * 256) / width, "num_tokens x width is too large");
    psk::DenseParams p{};
    p.positions = positions;
    p.num_tokens = num_tokens;
    p.ratio = compress_ratio;
    p.width = width;
    p.bs = 1;
    p.out = out;
    p.out_stride = out_stride;
    return cuda_status(psk::launch_dense_indices(p, false, reinterpret_cast<cudaStream_t>(stream)),
                       "build_dense_prefill_local_compressed_indices launch");
}

psk_status combine_dense_swa_indices(const int64_t* positions, const int32_t* token_to_req,
                                     const int32_t* seq_lens, const int32_t* gather_lens,
                                     int32_t num_reqs, int64_t num_tokens, int32_t window,
                                     int64_t workspace_width, int64_t compressed_base,
                                     int32_t* indices, int64_t out_stride, int32_t* lens,
                                     psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(window >= 0, "window must be >= 0");
    CHECK(workspace_width >= 0 && compressed_base >= 0,
          "workspace_width and compressed_base must be >= 0");
    CHECK(out_stride >= window, "out_stride must be >= window");
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(positions && token_to_req && seq_lens && gather_lens && indices && lens,
          "positions, token_to_req, seq_lens, gather_lens, indices and lens must be non-null");
    CHECK(aligned(positions, 8), "positions must be 8-byte aligned");
    CHECK(aligned(token_to_req, 4) && aligned(seq_lens, 4) && aligned(gather_lens, 4) &&
              aligned(indices, 4) && aligned(lens, 4),
          "int32 arrays must be 4-byte aligned");
    psk::WorkspaceIndexParams p{nullptr, seq_lens, gather_lens, token_to_req, num_reqs,
                                num_tokens, window, 1, nullptr, 0, 0, workspace_width,
                                compressed_base, nullptr, indices, out_stride, lens, positions};
    return cuda_status(psk::launch_workspace_indices(p, reinterpret_cast<cudaStream_t>(stream)),
                       "combine_dense_swa_indices launch");
}

psk_status write_indexer_fp8_cache(const void* index_k, int64_t k_row_stride,
                                   const int64_t* slot_mapping, int64_t num_tokens,
                                   uint8_t* cache, int64_t num_pages, int64_t page_stride,
                                   int32_t block_size, int32_t head_dim, int32_t* err_count,
                                   psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(mxfp4_head_dim_ok(head_dim),
          "head_dim must be one of 32, 64, 128, 256, 512, 1024 (got %d)", head_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size, head_dim + 4);
    if (st != PSK_OK) return st;
    if (num_tokens == 0) return ok();
    CHECK(index_k != nullptr && slot_mapping != nullptr,
          "index_k and slot_mapping must be non-null");
    CHECK(aligned(index_k, 16), "index_k must be 16-byte aligned");
    CHECK(k_row_stride >= head_dim && k_row_stride % 8 == 0,
          "k_row_stride must be >= head_dim and a multiple of 8 elements");
    CHECK(aligned(slot_mapping, 8), "slot_mapping must be 8-byte aligned");
    CHECK(err_count == nullptr || aligned(err_count, 4), "err_count must be 4-byte aligned");
    psk::InsertParams p{index_k, k_row_stride, slot_mapping, num_tokens, cache, num_pages,
                        page_stride, block_size, head_dim, 0, 1, err_count};
    return cuda_status(psk::launch_fp8_indexer_insert(p, reinterpret_cast<cudaStream_t>(stream)),
                       "write_indexer_fp8_cache launch");
}

psk_status indexer_k_norm_rope_store(const void* k_pre, int64_t k_row_stride,
                                     const int64_t* positions, const float* cos_sin_cache,
                                     int64_t cs_stride, int64_t max_pos,
                                     const float* rms_norm_weight, float rms_norm_eps,
                                     const int64_t* kv_slot_mapping, int64_t num_tokens,
                                     int32_t compress_ratio, psk_record record,
                                     uint8_t* k_cache, int64_t num_pages, int64_t page_stride,
                                     int32_t block_size, int32_t* err_count,
                                     psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(record == PSK_REC_MXFP4 || record == PSK_REC_FP8_INDEXER,
          "record must be PSK_REC_MXFP4 or PSK_REC_FP8_INDEXER (got %d)", (int)record);
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(max_pos >= 0 && cs_stride >= 64, "need max_pos >= 0 and cs_stride >= 64");
    psk_status st = check_cache(k_cache, num_pages, page_stride, block_size,
                                record == PSK_REC_MXFP4 ? 68 : 132);
    if (st != PSK_OK) return st;
    if (num_tokens == 0) return ok();
    CHECK(k_pre && positions && cos_sin_cache && rms_norm_weight && kv_slot_mapping,
          "k_pre, positions, cos_sin_cache, rms_norm_weight and kv_slot_mapping must be non-null");
    CHECK(aligned(k_pre, 16) && k_row_stride >= 128 && k_row_stride % 8 == 0,
          "k_pre must be 16-byte aligned with a row stride >= 128 and a multiple of 8 elements");
    CHECK(aligned(positions, 8) && aligned(kv_slot_mapping, 8),
          "positions and kv_slot_mapping must be 8-byte aligned");
    CHECK(aligned(cos_sin_cache, 4), "cos_sin_cache must be 4-byte aligned");
    CHECK(aligned(rms_norm_weight, 16), "rms_norm_weight must be 16-byte aligned");
    CHECK(err_count == nullptr || aligned(err_count, 4), "err_count must be 4-byte aligned");
    CHECK(num_tokens <= INT64_MAX / 32, "num_tokens is too large");
    psk::NormRopeParams p{static_cast<const uint16_t*>(k_pre), k_row_stride, positions,
                          cos_sin_cache, cs_stride, max_pos, rms_norm_weight, rms_norm_eps,
                          kv_slot_mapping, num_tokens, compress_ratio, (int32_t)record, k_cache,
                          num_pages, page_stride, block_size, err_count};
    return cuda_status(psk::launch_norm_rope_store(p, reinterpret_cast<cudaStream_t>(stream)),
                       "indexer_k_norm_rope_store launch");
}

psk_status save_compressor_state(const float* kv, const float* score, int64_t in_stride,
                                 const float* ape, int32_t state_width,
                                 const int64_t* slot_mapping, const int64_t* positions,
                                 int64_t num_tokens, int32_t compress_ratio, float* state_cache,
                                 int64_t num_pages, int32_t block_size, int32_t* err_count,
                                 psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(state_width > 0 && state_width % 4 == 0, "state_width must be a positive multiple of 4");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(num_pages >= 1 && block_size >= 1, "num_pages and block_size must be >= 1");
    CHECK(state_cache != nullptr && aligned(state_cache, 16), "state_cache must be 16-byte aligned");
    if (num_tokens == 0) return ok();
    CHECK(kv && score && ape && slot_mapping && positions,
          "kv, score, ape, slot_mapping and positions must be non-null");
    CHECK(in_stride >= state_width && in_stride % 4 == 0,
          "in_stride must be >= state_width and a multiple of 4");
    CHECK(aligned(kv, 16) && aligned(score, 16) && aligned(ape, 16),
          "kv, score and ape must be 16-byte aligned");
    CHECK(aligned(slot_mapping, 8) && aligned(positions, 8),
          "slot_mapping and positions must be 8-byte aligned");
    CHECK(err_count == nullptr || aligned(err_count, 4), "err_count must be 4-byte aligned");
    CHECK(num_tokens <= INT64_MAX / 32, "num_tokens is too large");
    psk::SaveStateParams p{kv, score, in_stride, ape, state_width, slot_mapping, positions,
                           num_tokens, compress_ratio, state_cache, num_pages, block_size,
                           err_count};
    return cuda_status(psk::launch_save_compressor_state(p, reinterpret_cast<cudaStream_t>(stream)),
                       "save_compressor_state launch");
}

psk_status compress_kv_cache_insert(
    const float* state_cache, int64_t state_num_pages, int32_t state_block_size,
    int32_t state_width, const int32_t* token_to_req, const int64_t* positions,
    const int64_t* state_slot_mapping, const int32_t* block_table, int64_t bt_stride,
    int32_t bt_width, const int32_t* base_offsets, int32_t num_reqs, int64_t num_tokens,
    int32_t compress_ratio, int32_t overlap, const float* rms_norm_weight, float rms_norm_eps,
    const float* cos_sin_cache, int64_t cs_stride, int64_t max_pos, uint8_t* kv_cache,
    int64_t kv_num_pages, int64_t kv_page_stride, int32_t kv_block_size,
    const int64_t* kv_slot_mapping, int32_t* err_count, psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(overlap == 0 || overlap == 1, "overlap must be 0 or 1");
    CHECK(compress_ratio >= 1 && (overlap ? 2 : 1) * (int64_t)compress_ratio <= 256,
          "the window ((overlap ? 2 : 1) * compress_ratio) must be in [1, 256]");
    CHECK(state_width == (overlap ? 2 : 1) * 512,
          "state_width must be 512 (1024 with overlap) for 512-dim keys");
    CHECK(state_num_pages >= 1 && state_block_size >= 1, "state pages and block size must be >= 1");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    CHECK(max_pos >= 0 && cs_stride >= 64, "need max_pos >= 0 and cs_stride >= 64");
    psk_status st = check_cache(kv_cache, kv_num_pages, kv_page_stride, kv_block_size,
                                fp8_record_bytes(512, 64, 1));
    if (st != PSK_OK) return st;
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(state_cache && token_to_req && positions && state_slot_mapping && rms_norm_weight &&
              cos_sin_cache && kv_slot_mapping,
          "state_cache, token_to_req, positions, state_slot_mapping, rms_norm_weight, "
          "cos_sin_cache and kv_slot_mapping must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(state_cache, 16) && aligned(rms_norm_weight, 16),
          "state_cache and rms_norm_weight must be 16-byte aligned");
    CHECK(aligned(positions, 8) && aligned(state_slot_mapping, 8) && aligned(kv_slot_mapping, 8),
          "positions and slot mappings must be 8-byte aligned");
    CHECK(aligned(token_to_req, 4) && aligned(block_table, 4) && aligned(base_offsets, 4) &&
              aligned(cos_sin_cache, 4),
          "int32 arrays and cos_sin_cache must be 4-byte aligned");
    CHECK(err_count == nullptr || aligned(err_count, 4), "err_count must be 4-byte aligned");
    CHECK(num_tokens <= 0x7FFFFFFFll, "num_tokens must fit a grid");
    psk::CompressParams p{state_cache, state_num_pages, state_block_size, state_width,
                          token_to_req, positions, state_slot_mapping, block_table, bt_stride,
                          bt_width, base_offsets, num_reqs, num_tokens, compress_ratio, overlap,
                          rms_norm_weight, rms_norm_eps, cos_sin_cache, cs_stride, max_pos,
                          kv_cache, kv_num_pages, kv_page_stride, kv_block_size, kv_slot_mapping,
                          err_count};
    return cuda_status(psk::launch_compress_kv_insert(p, reinterpret_cast<cudaStream_t>(stream)),
                       "compress_kv_cache_insert launch");
}

psk_status dequantize_and_gather_k_cache_topk(
    void* out, int64_t out_stride_t, int64_t out_stride_j, const uint8_t* cache,
    int64_t num_pages, int64_t page_stride, int32_t block_size, psk_record record,
    int32_t head_dim, int32_t rope_dim, const int32_t* topk_local, int64_t topk_stride,
    int64_t num_tokens, int32_t topk, const int32_t* token_to_req, const int32_t* block_table,
    int64_t bt_stride, int32_t bt_width, int32_t num_reqs, const int32_t* base_offsets,
    const uint8_t* is_valid_token, psk_stream_t stream) {
    CHECK(num_tokens >= 0 && topk >= 0, "num_tokens and topk must be >= 0");
    CHECK(record == PSK_REC_FP8_DS_MLA || record == PSK_REC_MXFP4 ||
              record == PSK_REC_FP8_INDEXER,
          "unknown record %d", (int)record);
    int64_t rec_bytes;
    if (record == PSK_REC_FP8_DS_MLA) {
        CHECK(fp8_head_dim_ok(head_dim),
              "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)", head_dim);
        CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
              "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
        rec_bytes = fp8_record_bytes(head_dim, rope_dim, 1);
    } else {
        CHECK(mxfp4_head_dim_ok(head_dim),
              "head_dim must be one of 32, 64, 128, 256, 512, 1024 (got %d)", head_dim);
        CHECK(rope_dim == 0, "rope_dim must be 0 for this record");
        rec_bytes = record == PSK_REC_MXFP4 ? head_dim / 2 + head_dim / 32 : head_dim + 4;
    }
    psk_status st = check_cache(cache, num_pages, page_stride, block_size, rec_bytes);
    if (st != PSK_OK) return st;
    CHECK(topk_stride >= topk, "topk_stride must be >= topk");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    if (num_tokens == 0 || topk == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(out && topk_local && token_to_req, "out, topk_local and token_to_req must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(out, 16), "out must be 16-byte aligned");
    CHECK(out_stride_t >= 0 && out_stride_j >= 0 && out_stride_t % 8 == 0 && out_stride_j % 8 == 0,
          "output strides must be non-negative multiples of 8 elements");
    CHECK(aligned(topk_local, 4) && aligned(token_to_req, 4) && aligned(block_table, 4) &&
              aligned(base_offsets, 4),
          "int32 arrays must be 4-byte aligned");
    psk::GatherParams p{static_cast<uint16_t*>(out), out_stride_t, out_stride_j, cache,
                        num_pages, page_stride, block_size, (int32_t)record, head_dim,
                        rope_dim, 1, nullptr, 0, num_tokens, topk};
    psk::TopkSource tk{topk_local, topk_stride, token_to_req, is_valid_token, num_reqs,
                       block_table, bt_stride, bt_width, base_offsets};
    return cuda_status(psk::launch_gather_topk(p, tk, reinterpret_cast<cudaStream_t>(stream)),
                       "dequantize_and_gather_k_cache_topk launch");
}

psk_status dequantize_and_gather_k_cache_window(
    void* out, int64_t out_stride_t, int64_t out_stride_j, const uint8_t* cache,
    int64_t num_pages, int64_t page_stride, int32_t block_size, int32_t head_dim,
    int32_t rope_dim, const int32_t* query_start_loc, const int32_t* seq_lens,
    const int32_t* token_to_req, const int32_t* replay_start, int32_t num_reqs,
    int64_t num_tokens, const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    const int32_t* base_offsets, int32_t window, const uint8_t* is_valid_token,
    psk_stream_t stream) {
    CHECK(num_tokens >= 0 && window >= 0, "num_tokens and window must be >= 0");
    CHECK(fp8_head_dim_ok(head_dim),
          "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)", head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size,
                                fp8_record_bytes(head_dim, rope_dim, 1));
    if (st != PSK_OK) return st;
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    if (num_tokens == 0 || window == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(out && query_start_loc && seq_lens && token_to_req,
          "out, query_start_loc, seq_lens and token_to_req must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(out, 16), "out must be 16-byte aligned");
    CHECK(out_stride_t >= 0 && out_stride_j >= 0 && out_stride_t % 8 == 0 && out_stride_j % 8 == 0,
          "output strides must be non-negative multiples of 8 elements");
    CHECK(aligned(query_start_loc, 4) && aligned(seq_lens, 4) && aligned(token_to_req, 4) &&
              aligned(replay_start, 4) && aligned(block_table, 4) && aligned(base_offsets, 4),
          "int32 arrays must be 4-byte aligned");
    psk::GatherParams p{static_cast<uint16_t*>(out), out_stride_t, out_stride_j, cache,
                        num_pages, page_stride, block_size, 0, head_dim, rope_dim, 1, nullptr, 0,
                        num_tokens, window};
    psk::WindowSource wn{query_start_loc, seq_lens, token_to_req, replay_start, is_valid_token,
                         num_reqs, block_table, bt_stride, bt_width, base_offsets};
    return cuda_status(psk::launch_gather_window(p, wn, reinterpret_cast<cudaStream_t>(stream)),
                       "dequantize_and_gather_k_cache_window launch");
}

psk_status dequantize_and_gather_k_cache_pair(
    void* out, int64_t out_stride_t, int64_t out_stride_j, const uint8_t* cache_a,
    int64_t num_pages_a, int64_t page_stride_a, int32_t block_size_a, const uint8_t* cache_b,
    int64_t num_pages_b, int64_t page_stride_b, int32_t block_size_b, int32_t head_dim,
    int32_t rope_dim, const int32_t* indices, int64_t idx_stride, int64_t rows, int32_t cols,
    int32_t split, psk_stream_t stream) {
    CHECK(rows >= 0 && cols >= 0, "rows and cols must be >= 0");
    CHECK(split >= 0 && split <= cols, "need 0 <= split <= cols");
    CHECK(fp8_head_dim_ok(head_dim),
          "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)", head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    const int64_t rec_bytes = fp8_record_bytes(head_dim, rope_dim, 1);
    psk_status st = check_cache(cache_a, num_pages_a, page_stride_a, block_size_a, rec_bytes);
    if (st != PSK_OK) return st;
    st = check_cache(cache_b, num_pages_b, page_stride_b, block_size_b, rec_bytes);
    if (st != PSK_OK) return st;
    CHECK(idx_stride >= cols, "idx_stride must be >= cols");
    if (rows == 0 || cols == 0) return ok();
    CHECK(out != nullptr && indices != nullptr, "out and indices must be non-null");
    CHECK(aligned(out, 16), "out must be 16-byte aligned");
    CHECK(out_stride_t >= 0 && out_stride_j >= 0 && out_stride_t % 8 == 0 &&
              out_stride_j % 8 == 0,
          "output strides must be non-negative multiples of 8 elements");
    CHECK(aligned(indices, 4), "indices must be 4-byte aligned");
    CHECK(rows <= INT64_MAX / cols, "rows * cols overflows");
    psk::GatherParams p{static_cast<uint16_t*>(out), out_stride_t, out_stride_j, cache_a,
                        num_pages_a, page_stride_a, block_size_a, 0, head_dim, rope_dim, 1,
                        indices, idx_stride, rows, cols};
    psk::PairSource pr{cache_b, num_pages_b, page_stride_b, block_size_b, -1, split};
    return cuda_status(psk::launch_gather_pair(p, pr, reinterpret_cast<cudaStream_t>(stream)),
                       "dequantize_and_gather_k_cache_pair launch");
}

psk_status dequantize_and_gather_k_cache_dense(
    void* out, int64_t out_stride_t, int64_t out_stride_j, const uint8_t* cache,
    int64_t num_pages, int64_t page_stride, int32_t block_size, int32_t head_dim,
    int32_t rope_dim, const int64_t* positions, int64_t num_tokens, const int32_t* token_to_req,
    int32_t num_reqs, const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    const int32_t* base_offsets, int32_t compress_ratio, int32_t width,
    const uint8_t* is_valid_token, psk_stream_t stream) {
    CHECK(num_tokens >= 0 && width >= 0, "num_tokens and width must be >= 0");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(fp8_head_dim_ok(head_dim),
          "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)", head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size,
                                fp8_record_bytes(head_dim, rope_dim, 1));
    if (st != PSK_OK) return st;
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    if (num_tokens == 0 || width == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(out && positions && token_to_req, "out, positions and token_to_req must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(out, 16), "out must be 16-byte aligned");
    CHECK(out_stride_t >= 0 && out_stride_j >= 0 && out_stride_t % 8 == 0 && out_stride_j % 8 == 0,
          "output strides must be non-negative multiples of 8 elements");
    CHECK(aligned(positions, 8), "positions must be 8-byte aligned");
    CHECK(aligned(token_to_req, 4) && aligned(block_table, 4) && aligned(base_offsets, 4),
          "int32 arrays must be 4-byte aligned");
    CHECK(num_tokens <= INT64_MAX / width, "num_tokens * width overflows");
    psk::GatherParams p{static_cast<uint16_t*>(out), out_stride_t, out_stride_j, cache,
                        num_pages, page_stride, block_size, 0, head_dim, rope_dim, 1, nullptr, 0,
                        num_tokens, width};
    psk::DenseSource ds{positions, token_to_req, is_valid_token, num_reqs, block_table, bt_stride,
                        bt_width, base_offsets, compress_ratio};
    return cuda_status(psk::launch_gather_dense(p, ds, reinterpret_cast<cudaStream_t>(stream)),
                       "dequantize_and_gather_k_cache_dense launch");
}

psk_status compute_slot_mappings(
    const int32_t* query_start_loc, const int32_t* seq_lens, int32_t num_reqs,
    int64_t num_tokens, const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    const int32_t* base_offsets, int32_t block_size, const int32_t* comp_block_table,
    int64_t comp_bt_stride, int32_t comp_bt_width, const int32_t* comp_base_offsets,
    int32_t comp_block_size, int32_t compress_ratio, int64_t* positions, int32_t* token_to_req,
    int64_t* slot_mapping, int64_t* comp_slot_mapping, psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(block_size >= 1 && comp_block_size >= 1, "block sizes must be >= 1");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    if (comp_block_table != nullptr) {
        CHECK(comp_bt_width >= 0 && comp_bt_stride >= comp_bt_width,
              "need 0 <= comp_bt_width <= comp_bt_stride");
    }
    if (num_tokens == 0 || !(positions || token_to_req || slot_mapping || comp_slot_mapping))
        return ok();
    CHECK(num_tokens <= (int64_t)INT32_MAX, "num_tokens must fit in int32 (query_start_loc is)");
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(query_start_loc && seq_lens, "query_start_loc and seq_lens must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(query_start_loc, 4) && aligned(seq_lens, 4) && aligned(block_table, 4) &&
              aligned(base_offsets, 4) && aligned(comp_block_table, 4) &&
              aligned(comp_base_offsets, 4) && aligned(token_to_req, 4),
          "int32 arrays must be 4-byte aligned");
    CHECK(aligned(positions, 8) && aligned(slot_mapping, 8) && aligned(comp_slot_mapping, 8),
          "int64 arrays must be 8-byte aligned");
    psk::SlotMapParams p{};
    p.qsl = query_start_loc;
    p.seq_lens = seq_lens;
    p.num_reqs = num_reqs;
    p.num_tokens = num_tokens;
    p.main = {block_table, bt_stride, bt_width, base_offsets, block_size, -1};
    p.comp = comp_block_table == nullptr
                 ? psk::SlotMapTable{block_table, bt_stride, bt_width, comp_base_offsets,
                                     comp_block_size, -1}
                 : psk::SlotMapTable{comp_block_table, comp_bt_stride, comp_bt_width,
                                     comp_base_offsets, comp_block_size, -1};
    p.compress_ratio = compress_ratio;
    p.positions = positions;
    p.token_to_req = token_to_req;
    p.slots = slot_mapping;
    p.comp_slots = comp_slot_mapping;
    return cuda_status(psk::launch_slot_mappings(p, reinterpret_cast<cudaStream_t>(stream)),
                       "compute_slot_mappings launch");
}

psk_status extend_block_tables(
    const int32_t* seq_lens, int32_t num_reqs, int32_t block_size, int32_t compress_ratio,
    const int32_t* page_counts, const int32_t* page_pool, int64_t pool_size,
    const int32_t* pool_head, int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    int32_t* page_counts_out, int32_t* pool_head_out, int32_t* err_count, psk_stream_t stream) {
    CHECK(num_reqs >= 0, "num_reqs must be >= 0");
    CHECK(block_size >= 1, "block_size must be >= 1");
    CHECK(compress_ratio >= 1, "compress_ratio must be >= 1");
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    CHECK(pool_size >= 0 && pool_size <= (int64_t)INT32_MAX,
          "pool_size must be in [0, INT32_MAX]");
    if (num_reqs == 0) return ok();
    CHECK(seq_lens && page_counts_out && pool_head_out,
          "seq_lens, page_counts_out and pool_head_out must be non-null");
    CHECK(pool_size == 0 || page_pool, "page_pool must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(seq_lens, 4) && aligned(page_counts, 4) && aligned(page_pool, 4) &&
              aligned(pool_head, 4) && aligned(block_table, 4) && aligned(page_counts_out, 4) &&
              aligned(pool_head_out, 4) && aligned(err_count, 4),
          "int32 arrays must be 4-byte aligned");
    // every CTA reads all counts and the head: they are not updated in place
    const auto overlap = [](const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
        return a != nullptr && b != nullptr && a < b + m && b < a + n;
    };
    CHECK(!overlap(page_counts, num_reqs, page_counts_out, num_reqs) &&
              !overlap(pool_head, 1, pool_head_out, 1) &&
              !overlap(page_counts, num_reqs, pool_head_out, 1) &&
              !overlap(pool_head, 1, page_counts_out, num_reqs) &&
              !overlap(page_counts_out, num_reqs, pool_head_out, 1) &&
              !overlap(seq_lens, num_reqs, page_counts_out, num_reqs) &&
              !overlap(seq_lens, num_reqs, pool_head_out, 1),
          "page_counts_out and pool_head_out must not overlap the inputs or each other");
    psk::ExtendParams p{seq_lens, num_reqs, block_size, compress_ratio, page_counts, page_pool,
                        pool_size, pool_head, block_table, bt_stride, bt_width, page_counts_out,
                        pool_head_out, err_count, 0};
    return cuda_status(psk::launch_extend_block_tables(p, reinterpret_cast<cudaStream_t>(stream)),
                       "extend_block_tables launch");
}

int64_t sparse_mla_attention_workspace_bytes(int64_t num_tokens, int32_t num_heads,
                                             int32_t head_dim, int32_t cols) {
    if (num_tokens < 1 || num_heads < 1 || !attn_head_dim_ok(head_dim) || cols < 1) return 0;
    return psk::attention_workspace_bytes(num_tokens, num_heads, head_dim, cols, true, 0);
}

psk_status sparse_mla_attention(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t num_tokens,
    int32_t num_heads, const uint8_t* cache, int64_t num_pages, int64_t page_stride,
    int32_t block_size, const uint8_t* extra_cache, int64_t extra_num_pages,
    int64_t extra_page_stride, int32_t extra_block_size, int32_t head_dim, int32_t rope_dim,
    const int32_t* indices, int64_t idx_stride, int32_t cols, int32_t split,
    float softmax_scale, const float* sink, void* out, int64_t out_stride_t,
    int64_t out_stride_h, float* lse, int64_t lse_stride_t, void* workspace,
    int64_t workspace_bytes, psk_stream_t stream) {
    CHECK(num_tokens >= 0 && cols >= 0 && cols <= (1 << 30),
          "num_tokens must be >= 0 and cols in [0, 2^30]");
    CHECK(split >= 0 && split <= cols, "need 0 <= split <= cols");
    CHECK(attn_head_dim_ok(head_dim), "head_dim must be one of 128, 256, 512 (got %d)", head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    const int64_t rec = fp8_record_bytes(head_dim, rope_dim, 1);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size, rec);
    if (st != PSK_OK) return st;
    if (split < cols || extra_cache != nullptr) {
        st = check_cache(extra_cache, extra_num_pages, extra_page_stride, extra_block_size, rec);
        if (st != PSK_OK) return st;
    }
    CHECK(idx_stride >= cols, "idx_stride must be >= cols");
    psk::AttnParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride_t = q_stride_t;
    p.q_stride_h = q_stride_h;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.head_dim = head_dim;
    p.rope_dim = rope_dim;
    p.cache = {cache, num_pages, page_stride, block_size, -1};
    p.scale = softmax_scale;
    p.sink = sink;
    p.out = static_cast<uint16_t*>(out);
    p.out_stride_t = out_stride_t;
    p.out_stride_h = out_stride_h;
    p.lse = lse;
    p.lse_stride_t = lse_stride_t;
    p.workspace = workspace;
    p.extra = extra_cache == nullptr
                  ? p.cache
                  : psk::AttnCache{extra_cache, extra_num_pages, extra_page_stride,
                                   extra_block_size, -1};
    p.idx = indices;
    p.idx_stride = idx_stride;
    p.cols = cols;
    p.split = split;
    st = check_attention(
        p, num_tokens > 0,
        sparse_mla_attention_workspace_bytes(num_tokens, num_heads, head_dim, cols),
        workspace_bytes);
    if (st != PSK_OK) return st;
    if (num_tokens == 0) return ok();
    CHECK(cols == 0 || indices != nullptr, "indices must be non-null");
    CHECK(aligned(indices, 4), "indices must be 4-byte aligned");
    return cuda_status(psk::launch_attention_indexed(p, reinterpret_cast<cudaStream_t>(stream)),
                       "sparse_mla_attention launch");
}

int64_t chunk_mla_attention_workspace_bytes(int64_t num_tokens, int32_t num_reqs,
                                            int32_t num_heads, int32_t head_dim,
                                            int32_t bt_width, int32_t block_size,
                                            int32_t window) {
    if (num_tokens < 1 || num_reqs < 1 || num_heads < 1 || !attn_head_dim_ok(head_dim) || bt_width < 1 ||
        block_size < 1 || window < 0)
        return 0;
    return psk::attention_workspace_bytes(num_tokens, num_heads, head_dim,
                                          chunk_max_keys(bt_width, block_size, window), false,
                                          num_reqs);
}

psk_status chunk_mla_attention(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t num_tokens,
    int32_t num_heads, const uint8_t* cache, int64_t num_pages, int64_t page_stride,
    int32_t block_size, int32_t head_dim, int32_t rope_dim, const int32_t* query_start_loc,
    const int32_t* seq_lens, const int32_t* token_to_req, const int32_t* replay_start,
    int32_t num_reqs, const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    const int32_t* base_offsets, int32_t window, const uint8_t* is_valid_token,
    float softmax_scale, const float* sink, void* out, int64_t out_stride_t,
    int64_t out_stride_h, float* lse, int64_t lse_stride_t, void* workspace,
    int64_t workspace_bytes, psk_stream_t stream) {
    CHECK(num_tokens >= 0, "num_tokens must be >= 0");
    CHECK(window >= 0, "window must be >= 0");
    CHECK(attn_head_dim_ok(head_dim), "head_dim must be one of 128, 256, 512 (got %d)", head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size,
                                fp8_record_bytes(head_dim, rope_dim, 1));
    if (st != PSK_OK) return st;
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    psk::AttnParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride_t = q_stride_t;
    p.q_stride_h = q_stride_h;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.head_dim = head_dim;
    p.rope_dim = rope_dim;
    p.cache = {cache, num_pages, page_stride, block_size, -1};
    p.scale = softmax_scale;
    p.sink = sink;
    p.out = static_cast<uint16_t*>(out);
    p.out_stride_t = out_stride_t;
    p.out_stride_h = out_stride_h;
    p.lse = lse;
    p.lse_stride_t = lse_stride_t;
    p.workspace = workspace;
    p.extra = p.cache;
    p.qsl = query_start_loc;
    p.seq_lens = seq_lens;
    p.t2r = token_to_req;
    p.replay = replay_start;
    p.valid = is_valid_token;
    p.num_reqs = num_reqs;
    p.bt = block_table;
    p.bt_stride = bt_stride;
    p.bt_width = bt_width;
    p.base_off = base_offsets;
    p.window = window;
    st = check_attention(p, num_tokens > 0,
                         chunk_mla_attention_workspace_bytes(num_tokens, num_reqs, num_heads, head_dim,
                                                             bt_width, block_size, window),
                         workspace_bytes);
    if (st != PSK_OK) return st;
    if (num_tokens == 0) return ok();
    CHECK(num_reqs >= 1, "num_reqs must be >= 1");
    CHECK(query_start_loc && seq_lens && token_to_req,
          "query_start_loc, seq_lens and token_to_req must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(query_start_loc, 4) && aligned(seq_lens, 4) && aligned(token_to_req, 4) &&
              aligned(replay_start, 4) && aligned(block_table, 4) && aligned(base_offsets, 4),
          "int32 arrays must be 4-byte aligned");
    return cuda_status(psk::launch_attention_chunk(p, reinterpret_cast<cudaStream_t>(stream)),
                       "chunk_mla_attention launch");
}

psk_status build_rope_cos_sin_cache(float* cos_sin_cache, int64_t cs_stride, int64_t first_pos,
                                    int64_t num_pos, int32_t rope_dim, double theta,
                                    psk_rope_scaling scaling, double factor,
                                    int64_t original_max_pos, double beta_fast, double beta_slow,
                                    double attention_factor, psk_stream_t stream) {
    CHECK(num_pos >= 0 && first_pos >= 0 && first_pos <= (1ll << 31) && num_pos <= (1ll << 31) - first_pos,
          "need 0 <= first_pos and first_pos + num_pos <= 2^31");
    CHECK(rope_dim >= 2 && rope_dim % 2 == 0 && rope_dim <= 2 * psk::kMaxTablePairs,
          "rope_dim must be even and in [2, %d] (got %d)", 2 * psk::kMaxTablePairs, rope_dim);
    CHECK(std::isfinite(theta) && theta > 1.0, "theta must be finite and > 1");
    CHECK(scaling == PSK_ROPE_UNSCALED || scaling == PSK_ROPE_LINEAR || scaling == PSK_ROPE_YARN,
          "unknown scaling %d", (int)scaling);
    CHECK(scaling == PSK_ROPE_UNSCALED || (std::isfinite(factor) && factor >= 1.0),
          "factor must be finite and >= 1");
    CHECK(scaling != PSK_ROPE_YARN ||
              (original_max_pos >= 1 && beta_slow > 0.0 && beta_fast >= beta_slow && std::isfinite(beta_fast)),
          "need original_max_pos >= 1 and beta_fast >= beta_slow > 0");
    const float m = (float)attention_factor;
    CHECK(std::isfinite(m) && m > 0.0f, "attention_factor must be finite and > 0");
    CHECK(cs_stride >= rope_dim, "cs_stride must be >= rope_dim");
    CHECK(cs_stride <= (INT64_MAX >> 34), "cs_stride overflows");
    if (num_pos == 0) return ok();
    CHECK(cos_sin_cache != nullptr && aligned(cos_sin_cache, 4), "cos_sin_cache must be non-null and 4-byte aligned");
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    // 1 / (2 pi): the double next to it, and what that leaves
    const Wide per_radian = {0.15915494309189535, -9.8393383375912430e-18};
    psk::RopeTableParams p{};
    p.out = cos_sin_cache;
    p.stride = cs_stride;
    p.first_pos = first_pos;
    p.num_pos = num_pos;
    p.pairs = rope_dim / 2;
    p.factor = m;
    const auto pair_of = [&](double turns) {
        return rope_dim * std::log((double)original_max_pos / (kTwoPi * turns)) / (2.0 * std::log(theta));
    };
    double lo = 0.0, span = 1.0;
    if (scaling == PSK_ROPE_YARN) {
        lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
        span = std::fmax(std::fmin(std::ceil(pair_of(beta_slow)), rope_dim - 1.0) - lo, 0.001);
    }
    // A position of 2^31 turns by the error of a frequency 2^31 times over: in doubles that came to
    // 3.1e-7 of an angle, more than binary32 gives away.
    const Wide ratio = inverse_root(theta, p.pairs);
    Wide f = {1.0, 0.0};  // theta^(-2 i / rope_dim)
    for (int32_t i = 0; i < p.pairs; ++i, f = f * ratio) {
        Wide scaled = f;
        if (scaling == PSK_ROPE_LINEAR || (scaling == PSK_ROPE_YARN && i - lo >= span)) {
            scaled = f / factor;
        } else if (scaling == PSK_ROPE_YARN && i > lo) {
            const Wide g = Wide{i - lo, 0.0} / span, rest = Wide{1.0, 0.0} + Wide{-g.hi, -g.lo};
            scaled = f * (rest + g / factor);
        }
        p.turn[i] = fraction64(scaled * per_radian);
    }
    return cuda_status(psk::launch_rope_table(p, reinterpret_cast<cudaStream_t>(stream)),
                       "build_rope_cos_sin_cache launch");
}

psk_status apply_rotary_embedding(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, int32_t num_heads, const void* k,
    int64_t k_stride_t, int64_t k_stride_h, int32_t num_k_heads, int64_t num_tokens,
    psk_dtype dtype, int32_t head_dim, int32_t rope_offset, int32_t rope_dim,
    int32_t interleaved, int32_t inverse, const int64_t* positions, const float* cos_sin_cache,
    int64_t cs_stride, int64_t max_pos, void* q_out, int64_t q_out_stride_t,
    int64_t q_out_stride_h, void* k_out, int64_t k_out_stride_t, int64_t k_out_stride_h,
    int32_t* err_count, psk_stream_t stream) {
    CHECK(num_tokens >= 0 && num_tokens <= (int64_t)INT32_MAX, "num_tokens must be in [0, INT32_MAX]");
    CHECK(dtype == PSK_DTYPE_BF16 || dtype == PSK_DTYPE_FP16 || dtype == PSK_DTYPE_FP32, "unknown dtype %d",
          (int)dtype);
    CHECK(head_dim >= 2 && head_dim <= (1 << 16), "head_dim must be in [2, 65536] (got %d)", head_dim);
    CHECK(rope_dim >= 2 && rope_dim % 2 == 0, "rope_dim must be even and >= 2 (got %d)", rope_dim);
    CHECK(rope_offset >= 0 && rope_offset <= head_dim - rope_dim, "need 0 <= rope_offset <= head_dim - rope_dim");
    CHECK(interleaved == 0 || interleaved == 1, "interleaved must be 0 or 1");
    CHECK(inverse == 0 || inverse == 1, "inverse must be 0 or 1");
    CHECK(max_pos >= 0 && cs_stride >= rope_dim, "need max_pos >= 0 and cs_stride >= rope_dim");
    CHECK(num_heads >= 1 && (k == nullptr || num_k_heads >= 1), "numbers of heads must be >= 1");
    // 32 bits hold a row index and a step of the whole grid
    CHECK((int64_t)num_heads + (k == nullptr ? 0 : num_k_heads) <= psk::kMostRotaryHeads, "too many heads");
    if (num_tokens == 0) return ok();
    const int32_t size = dtype == PSK_DTYPE_FP32 ? 4 : 2;
    psk_status st = check_rotary(q, q_stride_t, q_stride_h, q_out, q_out_stride_t, q_out_stride_h, num_heads,
                                 num_tokens, head_dim, size, "q");
    if (st != PSK_OK) return st;
    if (k != nullptr) {
        st = check_rotary(k, k_stride_t, k_stride_h, k_out, k_out_stride_t, k_out_stride_h, num_k_heads,
                          num_tokens, head_dim, size, "k");
        if (st != PSK_OK) return st;
    }
    CHECK(positions != nullptr && aligned(positions, 8), "positions must be non-null and 8-byte aligned");
    CHECK((max_pos == 0 || cos_sin_cache != nullptr) && aligned(cos_sin_cache, 4),
          "cos_sin_cache must be non-null and 4-byte aligned");
    CHECK(aligned(err_count, 4), "err_count must be 4-byte aligned");
    psk::RotaryParams p{};
    p.q = {static_cast<const uint8_t*>(q), static_cast<uint8_t*>(q_out), q_stride_t * size, q_stride_h * size,
           q_out_stride_t * size, q_out_stride_h * size};
    p.heads = p.all_heads = num_heads;
    p.copy_q = q != q_out;
    if (k != nullptr) {
        p.k = {static_cast<const uint8_t*>(k), static_cast<uint8_t*>(k_out), k_stride_t * size,
               k_stride_h * size, k_out_stride_t * size, k_out_stride_h * size};
        p.all_heads += num_k_heads;
        p.copy_k = k != k_out;
    }
    p.num_tokens = num_tokens;
    p.dtype = dtype;
    p.head_dim = head_dim;
    p.offset = rope_offset;
    p.rope_dim = rope_dim;
    p.half = !interleaved;
    p.inverse = inverse;
    p.positions = positions;
    p.cos_sin = cos_sin_cache;
    p.cs_stride = cs_stride;
    p.max_pos = max_pos;
    p.err = err_count;
    return cuda_status(psk::launch_rotary(p, reinterpret_cast<cudaStream_t>(stream)),
                       "apply_rotary_embedding launch");
}

int64_t accumulate_attention_weights_workspace_bytes(void) {
    return psk::attn_weights_workspace_bytes();
}

psk_status accumulate_attention_weights(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t num_tokens,
    int32_t num_heads, const float* lse, int64_t lse_stride_t, const uint8_t* cache,
    int64_t num_pages, int64_t page_stride, int32_t block_size, int32_t head_dim,
    int32_t rope_dim, const int32_t* query_start_loc, const int32_t* seq_lens,
    const int32_t* replay_start, int32_t num_reqs, const int32_t* block_table,
    int64_t bt_stride, int32_t bt_width, const int32_t* base_offsets, int32_t window,
    const uint8_t* is_valid_token, float softmax_scale, const float* sink,
    const float* weights, int64_t w_stride, int32_t width, float decay, float* out,
    int64_t out_stride, void* workspace, int64_t workspace_bytes, psk_stream_t stream) {
    CHECK(num_tokens >= 0 && num_tokens <= (int64_t)INT32_MAX, "num_tokens must be in [0, INT32_MAX]");
    CHECK(num_reqs >= 0 && num_reqs <= (1 << 27), "num_reqs must be in [0, 2^27]");
    CHECK(num_heads >= 1 && num_heads <= (1 << 20), "num_heads must be in [1, 2^20]");
    CHECK(window >= 0, "window must be >= 0");
    CHECK(attn_head_dim_ok(head_dim), "head_dim must be one of 128, 256, 512 (got %d)", head_dim);
    CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
          "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
    psk_status st = check_cache(cache, num_pages, page_stride, block_size,
                                fp8_record_bytes(head_dim, rope_dim, 1));
    if (st != PSK_OK) return st;
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    CHECK(std::isnormal(softmax_scale) && softmax_scale > 0.0f && softmax_scale <= 1e38f,
          "softmax_scale must be a normal number in (0, 1e38]");
    CHECK(std::isfinite(decay) && decay >= 0.0f, "decay must be finite and >= 0");
    CHECK(width >= 0 && width <= (1 << 30), "width must be in [0, 2^30]");
    CHECK(out_stride >= width && (decay == 0.0f || w_stride >= width), "strides of weights and out must be >= width");
    CHECK(q_stride_t % 8 == 0 && q_stride_h % 8 == 0 && (num_tokens <= 1 || q_stride_t >= head_dim) &&
              (num_heads <= 1 || q_stride_h >= head_dim),
          "query strides must be multiples of 8 elements and at least head_dim");
    CHECK(q_stride_t <= (1ll << 38) && q_stride_h <= (1ll << 38), "query strides must be at most 2^38");
    CHECK(num_tokens <= 1 || lse_stride_t >= num_heads, "lse_stride_t must be >= num_heads");
    if (num_reqs == 0 || width == 0) return ok();
    CHECK(seq_lens && query_start_loc, "query_start_loc and seq_lens must be non-null");
    CHECK(num_tokens == 0 || (q != nullptr && lse != nullptr), "q and lse must be non-null");
    CHECK(aligned(q, 16), "q must be 16-byte aligned");
    CHECK(out != nullptr && (decay == 0.0f || weights != nullptr), "weights and out must be non-null");
    CHECK(out != weights || out_stride == w_stride, "weights in place need equal strides");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(query_start_loc, 4) && aligned(seq_lens, 4) && aligned(replay_start, 4) &&
              aligned(block_table, 4) && aligned(base_offsets, 4) && aligned(lse, 4) && aligned(sink, 4) &&
              aligned(weights, 4) && aligned(out, 4),
          "int32 and binary32 arrays must be 4-byte aligned");
    const int64_t need = psk::attn_weights_workspace_bytes();
    CHECK(workspace_bytes >= need, "workspace must hold %lld bytes (got %lld)", (long long)need,
          (long long)workspace_bytes);
    CHECK(need == 0 || (workspace != nullptr && aligned(workspace, 16)),
          "workspace must be non-null and 16-byte aligned");
    psk::WeightParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride_t = q_stride_t;
    p.q_stride_h = q_stride_h;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.head_dim = head_dim;
    p.rope_dim = rope_dim;
    p.lse = lse;
    p.lse_stride_t = lse_stride_t;
    p.sink = sink;
    p.scale = softmax_scale;
    p.cache = {cache, num_pages, page_stride, block_size, -1};
    p.qsl = query_start_loc;
    p.seq_lens = seq_lens;
    p.replay = replay_start;
    p.valid = is_valid_token;
    p.num_reqs = num_reqs;
    p.bt = block_table;
    p.bt_stride = bt_stride;
    p.bt_width = bt_width;
    p.base_off = base_offsets;
    p.window = window;
    p.weights = weights;
    p.w_stride = w_stride;
    p.width = width;
    p.decay = decay;
    p.out = out;
    p.out_stride = out_stride;
    p.workspace = workspace;
    return cuda_status(psk::launch_attn_weights(p, reinterpret_cast<cudaStream_t>(stream)),
                       "accumulate_attention_weights launch");
}

psk_status select_cache_evictions(
    const float* weights, int64_t w_stride, const int32_t* seq_lens, const int32_t* keep_lens,
    int32_t num_reqs, int32_t width, const int32_t* row_positions, int64_t pos_stride,
    int32_t num_first, int32_t num_recent, float* weights_out, int64_t wo_stride,
    int32_t* positions_out, int64_t po_stride, int32_t* moves, int64_t moves_stride,
    int32_t* num_moves, int32_t* seq_lens_out, int32_t* err_count, psk_stream_t stream) {
    CHECK(num_reqs >= 0 && num_reqs <= (1 << 27), "num_reqs must be in [0, 2^27]");
    CHECK(width >= 0 && width <= (1 << 30), "width must be in [0, 2^30]");
    CHECK(num_first >= 0 && num_recent >= 0, "num_first and num_recent must be >= 0");
    CHECK(w_stride >= width && (row_positions == nullptr || pos_stride >= width),
          "strides of the inputs must be >= width");
    CHECK((weights_out == nullptr || wo_stride >= width) && (positions_out == nullptr || po_stride >= width),
          "strides of the outputs must be >= width");
    CHECK(moves_stride >= width / 2 * 2 && moves_stride % 2 == 0,
          "moves_stride must be even and hold width / 2 pairs");
    if (num_reqs == 0) return ok();
    CHECK(seq_lens && keep_lens && num_moves && seq_lens_out,
          "seq_lens, keep_lens, num_moves and seq_lens_out must be non-null");
    CHECK(width == 0 || weights != nullptr, "weights must be non-null");
    CHECK(width < 2 || moves != nullptr, "moves must be non-null");
    CHECK(aligned(moves, 8), "moves must be 8-byte aligned");
    CHECK(aligned(weights, 4) && aligned(seq_lens, 4) && aligned(keep_lens, 4) && aligned(row_positions, 4) &&
              aligned(weights_out, 4) && aligned(positions_out, 4) && aligned(num_moves, 4) &&
              aligned(seq_lens_out, 4) && aligned(err_count, 4),
          "arrays must be 4-byte aligned");
    CHECK(weights_out != weights || weights == nullptr || wo_stride == w_stride,
          "weights in place need equal strides");
    CHECK(positions_out != row_positions || row_positions == nullptr || po_stride == pos_stride,
          "positions in place need equal strides");
    const auto overlap = [&](const int32_t* a, const int32_t* b) { return a < b + num_reqs && b < a + num_reqs; };
    CHECK(!overlap(num_moves, seq_lens_out) && !overlap(num_moves, seq_lens) && !overlap(num_moves, keep_lens) &&
              !overlap(seq_lens_out, keep_lens) && (seq_lens_out == seq_lens || !overlap(seq_lens_out, seq_lens)),
          "num_moves and seq_lens_out must not overlap the inputs or each other");
    psk::SelectParams p{weights, w_stride, seq_lens, keep_lens, num_reqs, width, row_positions, pos_stride,
                        num_first, num_recent, weights_out, wo_stride, positions_out, po_stride,
                        reinterpret_cast<int2*>(moves), moves_stride / 2, num_moves, seq_lens_out, err_count};
    return cuda_status(psk::launch_select_evictions(p, reinterpret_cast<cudaStream_t>(stream)),
                       "select_cache_evictions launch");
}

psk_status move_cache_rows(
    uint8_t* cache, int64_t num_pages, int64_t page_stride, int32_t block_size,
    psk_record record, int32_t head_dim, int32_t rope_dim, int32_t is_ue8m0,
    const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
    const int32_t* base_offsets, int32_t num_reqs, const int32_t* moves, int64_t moves_stride,
    int32_t max_moves, const int32_t* num_moves, int32_t* err_count, psk_stream_t stream) {
    CHECK(num_reqs >= 0 && max_moves >= 0, "num_reqs and max_moves must be >= 0");
    CHECK(record == PSK_REC_FP8_DS_MLA || record == PSK_REC_MXFP4 || record == PSK_REC_FP8_INDEXER,
          "unknown record kind %d", (int)record);
    CHECK(is_ue8m0 == 0 || is_ue8m0 == 1, "is_ue8m0 must be 0 or 1");
    psk::MoveParams p{};
    if (record == PSK_REC_FP8_DS_MLA) {
        CHECK(fp8_head_dim_ok(head_dim), "head_dim must be one of 64, 128, 256, 512, 1024 (got %d)", head_dim);
        CHECK(rope_dim >= 0 && rope_dim < head_dim && rope_dim % 64 == 0,
              "rope_dim must be a multiple of 64 in [0, head_dim) (got %d)", rope_dim);
        p.data_bytes = head_dim + rope_dim;
        p.scale_bytes = head_dim / 64 * (is_ue8m0 ? 1 : 4);
    } else {
        CHECK(mxfp4_head_dim_ok(head_dim), "head_dim must be one of 32, 64, 128, 256, 512, 1024 (got %d)", head_dim);
        CHECK(rope_dim == 0, "rope_dim must be 0 for this record (got %d)", rope_dim);
        p.data_bytes = record == PSK_REC_MXFP4 ? head_dim / 2 : head_dim;
        p.scale_bytes = record == PSK_REC_MXFP4 ? head_dim / 32 : 4;
    }
    psk_status st = check_cache(cache, num_pages, page_stride, block_size, p.data_bytes + p.scale_bytes);
    if (st != PSK_OK) return st;
    CHECK(bt_width >= 0 && bt_stride >= bt_width, "need 0 <= bt_width <= bt_stride");
    CHECK(moves_stride >= 2 * (int64_t)max_moves && moves_stride % 2 == 0,
          "moves_stride must be even and hold max_moves pairs");
    if (num_reqs == 0 || max_moves == 0) return ok();
    CHECK(moves && num_moves, "moves and num_moves must be non-null");
    CHECK(bt_width == 0 || block_table, "block_table must be non-null");
    CHECK(aligned(moves, 8), "moves must be 8-byte aligned");
    CHECK(aligned(num_moves, 4) && aligned(block_table, 4) && aligned(base_offsets, 4) && aligned(err_count, 4),
          "int32 arrays must be 4-byte aligned");
    p.cache = cache;
    p.num_pages = num_pages;
    p.page_stride = page_stride;
    p.block_size = block_size;
    p.bt = block_table;
    p.bt_stride = bt_stride;
    p.bt_width = bt_width;
    p.base = base_offsets;
    p.num_reqs = num_reqs;
    p.moves = reinterpret_cast<const int2*>(moves);
    p.moves_stride = moves_stride / 2;
    p.max_moves = max_moves;
    p.num_moves = num_moves;
    p.err = err_count;
    return cuda_status(psk::launch_move_rows(p, reinterpret_cast<cudaStream_t>(stream)),
                       "move_cache_rows launch");
}

}  // extern "C"

namespace psk {

int sm_count() {
    static std::atomic<int> cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
    if (dev < 64) {
        const int c = cached[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 148;
    if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace psk
