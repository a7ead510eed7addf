// rotary.cu -- rotary positions: the table of cosines and sines, and the
// rotation of a part of each head.
#include "psk.h"
#include "psk_common.cuh"
#include "rotary.h"

namespace psk {
namespace {

constexpr int kThreads = 256;

// ---- the table ---------------------------------------------------------------------
//
// Row p holds cos and sin of (first + p) f_i.  The angle is kept as a fraction of a turn
// in 64 bits, turn_i = f_i / (2 pi) 2^64: a product modulo 2^64 drops whole turns exactly,
// so a far position costs no accuracy and no binary64 arithmetic (of which this part does
// little).  An eighth of a turn to either side of the nearest quarter is left for the
// series of sine and cosine.
//
// 1048576 positions of 64 dims (268 MB written) take 47.4 us, 5.7 TB/s of the 6.7 measured; the
// issue slots are 81 % in use, so the arithmetic weighs as much as the stores.  One pair a
// thread with its own product took 234 us; stores of 512 contiguous bytes by exchange between
// threads 57.7, as without (the conversion below held both up).

// sin and cos of a fraction of a turn: quarters off, then Taylor's series on
// [-pi/4, pi/4], whose first dropped terms (x^11/11!, x^12/12!) are below 2^-28.
// Three roundings and the constant put x off by 3.5 2^-24 of itself, which moves a value by at
// most 1.95 2^-24 (x cos x and x sin x stay below 0.556); the series' own roundings add 1.1 2^-24
// and the product with the factor 0.71 2^-24 there: below m 2^-22 in all.
__device__ __forceinline__ void sincos_turn(uint64_t u, float& s, float& c) {
    const uint32_t quarter = (uint32_t)((u + (1ull << 61)) >> 62);
    constexpr float kRadians = (float)(6.283185307179586 / 18446744073709551616.0);  // 2 pi / 2^64
    const uint64_t rest = u - ((uint64_t)quarter << 62);
    // in two halves: with one conversion of 64 bits the table above took 57.4 us
    const float x = fmaf(__int2float_rn((int32_t)(rest >> 32)), 4294967296.0f, __uint2float_rn((uint32_t)rest)) * kRadians;
    const float y = x * x;
    float a = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
    a = fmaf(a, y, 8.3333333e-3f);
    a = fmaf(a, y, -0.16666667f);
    const float sn = fmaf(a * y, x, x);
    float b = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);
    b = fmaf(b, y, -1.3888889e-3f);
    b = fmaf(b, y, 4.1666667e-2f);
    b = fmaf(b, y, -0.5f);
    const float cs = fmaf(b, y, 1.0f);
    s = quarter & 1 ? cs : sn;
    c = quarter & 1 ? sn : cs;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
}

// A thread keeps V neighbouring pairs and walks over rows, so that an angle is one 64-bit
// addition from the last; with V = 4 a warp stores whole lines of 128 bytes.
template <int V>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeTableParams p, const int32_t rows_per_cta) {
    const int32_t groups = p.pairs / V, at_once = max(kThreads / groups, 1);
    const int32_t group = (int32_t)threadIdx.x % groups, row0 = (int32_t)threadIdx.x / groups;
    pdl_wait();
    const int64_t first = (int64_t)blockIdx.x * rows_per_cta, end = min(first + rows_per_cta, p.num_pos);
    if (row0 < at_once) {
        uint64_t at[V], step[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t turn = p.turn[group * V + i];
            at[i] = (uint64_t)(p.first_pos + first + row0) * turn;
            step[i] = (uint64_t)at_once * turn;
        }
        float* out = p.out + (first + row0) * p.stride + group * V;
#pragma unroll 2
        for (int64_t row = first + row0; row < end; row += at_once) {
            float s[V], c[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sincos_turn(at[i], s[i], c[i]);
                s[i] *= p.factor;
                c[i] *= p.factor;
                at[i] += step[i];
            }
            if constexpr (V == 4) {
                *reinterpret_cast<float4*>(out) = make_float4(c[0], c[1], c[2], c[3]);
                *reinterpret_cast<float4*>(out + p.pairs) = make_float4(s[0], s[1], s[2], s[3]);
            } else {
                out[0] = c[0];
                out[p.pairs] = s[0];
            }
            out += at_once * p.stride;
        }
    }
    pdl_launch_dependents();
}

// ---- the rotation -------------------------------------------------------------------
//
// (a, b) -> (a c - b s, b c + a s) for the pairs (2i, 2i + 1) or (i, i + rope_dim / 2) of
// the rotated dims; products and sums in binary32, one rounding to the tensor's type.
// A unit is what one thread takes of a row at a time: 16 bytes that hold whole pairs, or
// two times 16 bytes of the half layout, or 16 bytes to copy; single pairs and elements
// where sizes, strides or addresses allow no 16-byte accesses.  A thread keeps its unit
// for all the heads it visits, so a token's cosines and sines are read once per CTA.
//
// Bound by memory where it is large: 4096 tokens, the 64 rope dims of 128 heads of 512 in
// bf16 (134 MB in pieces of 128 bytes): 27.5 us, 4.9 TB/s of the 6.7 measured, with eight CTAs
// an SM (five: 30.3).  The half layout holds two packs and spills with eight: 1901 tokens of
// 36 heads of 256 dims (70 MB, in part from L2) 14 to 15.4 us with five, 20.6 with eight.  Several
// heads in flight a thread cost more CTAs than they gain (two 33.7, four 46 us against 30.3).
// These limits are bf16's.  The fp16 forms spill 8 bytes a thread at them, which does not show:
// in place on the last 64 of 512 dims, 4096 tokens of 129 heads, data in L2 (67.6 MB), 21.0 us in
// either type, half layout 22.6; binary32 (135 MB) 47.6 and 63.4.  Whole heads out of place, 1.08
// GB, 174 us.  64 tokens of 64 heads take 1.9 us: launch and two dependent reads.

template <int kType> struct Elem;
template <> struct Elem<PSK_DTYPE_BF16> {
    using Raw = uint16_t;
    static __device__ __forceinline__ float get(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ __forceinline__ uint16_t put(float x) { return (uint16_t)pack_bf16x2(x, 0.0f); }
};
template <> struct Elem<PSK_DTYPE_FP16> {
    using Raw = uint16_t;
    static __device__ __forceinline__ float get(uint16_t x) {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(x));
        return f;
    }
    static __device__ __forceinline__ uint16_t put(float x) {
        uint16_t r;
        asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(x));
        return r;
    }
};
template <> struct Elem<PSK_DTYPE_FP32> {
    using Raw = float;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};

// Elements a thread moves at once.
template <int kType, bool kWide>
constexpr int per_access() { return kWide ? 16 / (int)sizeof(typename Elem<kType>::Raw) : 1; }

template <typename Raw, int V>
struct alignas(sizeof(Raw) * V) Pack {
    Raw v[V];
};

// (a, b) of packs that hold pairs side by side, or of one pack with interleaved pairs.
template <int kType, int V>
__device__ __forceinline__ void turn(typename Elem<kType>::Raw& a, typename Elem<kType>::Raw& b, float c, float s) {
    using E = Elem<kType>;
    const float x = E::get(a), y = E::get(b);
    a = E::put(fmaf(x, c, -(y * s)));
    b = E::put(fmaf(y, c, x * s));
}

struct RotaryShape {
    int32_t units, rope_units;  // of a row; those that rotate come first
    int32_t rows_at_once;       // rows a CTA works on at a time
    int32_t tokens;             // tokens of a CTA (where all rows of several fit at once)
};

template <int kType, bool kHalf, bool kWide>
__global__ void __launch_bounds__(kThreads, kHalf ? 5 : 8) rotary_kernel(const RotaryParams p, const RotaryShape sh) {
    using Raw = typename Elem<kType>::Raw;
    constexpr int V = per_access<kType, kWide>();
    // pairs of a unit; interleaved single elements make no pair, so two are taken
    constexpr int kPairs = kHalf ? V : V > 1 ? V / 2 : 1;
    using P = Pack<Raw, V>;
    pdl_wait();
    const int slot = (int)threadIdx.x / min(sh.units, kThreads);
    const int unit0 = (int)threadIdx.x % min(sh.units, kThreads);
    int row0 = slot + (int)blockIdx.y * sh.rows_at_once, row_step = sh.rows_at_once * (int)gridDim.y;
    int64_t t = (int64_t)blockIdx.x * sh.tokens;
    bool in = slot < sh.rows_at_once;
    if (sh.tokens > 1) {
        t += slot / p.all_heads;
        row0 = slot % p.all_heads;
        row_step = p.all_heads;
        in = slot < sh.tokens * p.all_heads;
    }
    if (!in || t >= p.num_tokens) return;
    const int64_t pos = p.positions[t];
    const bool known = pos >= 0 && pos < p.max_pos;  // else the rows stay as they are
    if (p.err && pos >= p.max_pos && unit0 == 0 && row0 == 0) atomicAdd(p.err, 1);
    const int n = p.rope_dim / 2;
    for (int unit = unit0; unit < sh.units; unit += kThreads) {
        const bool rotates = unit < sh.rope_units;
        // first element of the unit, and of its second pack
        int at, second = 0;
        float c[kPairs], s[kPairs];
        if (rotates) {
            const int pair = unit * kPairs;
            at = p.offset + (kHalf ? pair : 2 * pair);
            second = kHalf ? n : 1;
            if (known) {
                const float* cs = p.cos_sin + pos * p.cs_stride + pair;
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    c[i] = cs[i];
                    s[i] = p.inverse ? -cs[n + i] : cs[n + i];
                }
            }
        } else {
            at = (unit - sh.rope_units) * V;
            if (at >= p.offset) at += p.rope_dim;
        }
        for (int row = row0; row < p.all_heads; row += row_step) {
            const bool is_k = row >= p.heads;
            const RotaryTensor& x = is_k ? p.k : p.q;
            const int h = is_k ? row - p.heads : row;
            const bool copy = is_k ? p.copy_k : p.copy_q;
            const uint8_t* src = x.in + t * x.in_stride_t + h * x.in_stride_h + (int64_t)at * sizeof(Raw);
            uint8_t* dst = x.out + t * x.out_stride_t + h * x.out_stride_h + (int64_t)at * sizeof(Raw);
            if (!copy && (!rotates || !known)) continue;
            P a = *reinterpret_cast<const P*>(src);
            if (!rotates) {
                *reinterpret_cast<P*>(dst) = a;
            } else if constexpr (kHalf || V == 1) {
                P b = *reinterpret_cast<const P*>(src + second * sizeof(Raw));
                if (known) {
#pragma unroll
                    for (int i = 0; i < V; ++i) turn<kType, V>(a.v[i], b.v[i], c[i], s[i]);
                }
                *reinterpret_cast<P*>(dst) = a;
                *reinterpret_cast<P*>(dst + second * sizeof(Raw)) = b;
            } else {
                if (known) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) turn<kType, V>(a.v[2 * i], a.v[2 * i + 1], c[i], s[i]);
                }
                *reinterpret_cast<P*>(dst) = a;
            }
        }
    }
    pdl_launch_dependents();
}

template <int kType, bool kHalf, bool kWide>
cudaError_t launch(const RotaryParams& p, cudaStream_t stream) {
    constexpr int V = per_access<kType, kWide>();
    RotaryShape sh{};
    sh.rope_units = kHalf ? p.rope_dim / 2 / V : V > 1 ? p.rope_dim / V : p.rope_dim / 2;
    sh.units = sh.rope_units + (p.copy_q || p.copy_k ? (p.head_dim - p.rope_dim) / V : 0);
    sh.rows_at_once = sh.units >= kThreads ? 1 : kThreads / sh.units;
    sh.tokens = p.all_heads < sh.rows_at_once ? sh.rows_at_once / p.all_heads : 1;
    if (sh.tokens > p.num_tokens) sh.tokens = (int32_t)p.num_tokens;
    if (sh.tokens == 1 && sh.rows_at_once > p.all_heads) sh.rows_at_once = p.all_heads;
    const int64_t x = (p.num_tokens + sh.tokens - 1) / sh.tokens;
    // few tokens: their rows are spread over CTAs until there are two per SM
    int64_t y = (2 * (int64_t)sm_count() + x - 1) / x;
    if (y * sh.rows_at_once > (1 << 20)) y = (1 << 20) / sh.rows_at_once;  // kMostRotaryHeads counts on that
    const int64_t most = sh.tokens > 1 ? 1 : (p.all_heads + sh.rows_at_once - 1) / sh.rows_at_once;
    if (y > most) y = most;
    return launch_pdl(rotary_kernel<kType, kHalf, kWide>, dim3((unsigned)x, (unsigned)y), dim3(kThreads), 0, stream, p, sh);
}

template <int kType>
cudaError_t launch_type(const RotaryParams& p, cudaStream_t stream) {
    constexpr int kSize = sizeof(typename Elem<kType>::Raw), V = 16 / kSize;
    const auto even = [](const RotaryTensor& x) {
        return ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out) | (uintptr_t)x.in_stride_t |
                 (uintptr_t)x.in_stride_h | (uintptr_t)x.out_stride_t | (uintptr_t)x.out_stride_h) & 15) == 0;
    };
    const bool wide = even(p.q) && (p.all_heads == p.heads || even(p.k)) && p.offset % V == 0 &&
                      p.rope_dim % (p.half ? 2 * V : V) == 0 && p.head_dim % V == 0;
    if (p.half) return wide ? launch<kType, true, true>(p, stream) : launch<kType, true, false>(p, stream);
    return wide ? launch<kType, false, true>(p, stream) : launch<kType, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream) {
    const bool wide = p.pairs % 4 == 0 && p.stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
    const int32_t groups = p.pairs / (wide ? 4 : 1), at_once = groups < kThreads ? kThreads / groups : 1;
    // a grid of eight CTAs an SM (three run at a time), each with whole turns of its threads
    const int64_t turns = (p.num_pos + at_once - 1) / at_once, most = (int64_t)sm_count() * 8;
    const int64_t rows = (turns + most - 1) / most * at_once, ctas = (p.num_pos + rows - 1) / rows;
    return launch_pdl(wide ? rope_table_kernel<4> : rope_table_kernel<1>, dim3((unsigned)ctas), dim3(kThreads), 0, stream, p,
                      (int32_t)rows);
}

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
    return p.dtype == PSK_DTYPE_BF16   ? launch_type<PSK_DTYPE_BF16>(p, stream)
           : p.dtype == PSK_DTYPE_FP16 ? launch_type<PSK_DTYPE_FP16>(p, stream)
                                       : launch_type<PSK_DTYPE_FP32>(p, stream);
}

}  // namespace psk
