// Shared by the attention half's kernels: element types, the layout of a page
// of the 4-bit key/value cache, and the map from a launch's work units to
// sequences.
//
// A page of one (layer, head) is page_tokens * (head_dim + 8) bytes:
//   key codes    [token][head_dim / 2 bytes]
//   value codes  [token / 8][head_dim] 32-bit words
//   key scales   fp32 [token], value scales fp32 [token]
// so a head's keys, values and scales of a page are one contiguous stretch.
// The codes stand in the order in which the matrix instructions take them.
// v_mfma_f32_16x16x32_f16 gives lane l row l % 16 and the K-values 8*(l/16) ..
// +7, and the conversion of a word to fp16 makes pairs of the nibbles i and
// i + 4.  Therefore
//   a key row's word g*(head_dim/32) + s holds columns 32*s + 8*g .. +7 (one
//   16-byte load per lane is the operand of head_dim/32 consecutive MFMAs), and
//   a value word holds one column of 8 consecutive tokens (the product with the
//   probabilities contracts over tokens, so no transpose is needed);
// in both, nibble i is element 2i of the eight and nibble i + 4 element 2i + 1.
#pragma once

#include <hip/hip_bfloat16.h>
#include <hip/hip_fp16.h>

#include "moedec_attn.h"
#include "persist.h"

namespace moedec {
namespace attn {

using mfma::floatx4;
using mfma::half2v;
using mfma::half8;
using mfma::u32x4;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

// ------------------------------------------------------------- element types

struct F32 {
    typedef float type;
    static constexpr int bytes = 4;
    __device__ static float get(float v) { return v; }
    __device__ static float put(float v) { return v; }
};
struct F16 {
    typedef _Float16 type;
    static constexpr int bytes = 2;
    __device__ static float get(_Float16 v) { return (float)v; }
    __device__ static _Float16 put(float v) { return (_Float16)v; }
};
struct BF16 {
    typedef uint16_t type;
    static constexpr int bytes = 2;
    __device__ static float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    // round to nearest even; a NaN stays a NaN (quiet)
    __device__ static uint16_t put(float v) {
        const uint32_t u = __float_as_uint(v);
        if (v != v) return (uint16_t)((u >> 16) | 0x40u);
        return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
    }
};

// Eight consecutive elements (16-byte aligned) as floats.
template <typename T>
__device__ __forceinline__ void load8(const typename T::type* p, float* o) {
    if constexpr (T::bytes == 4) {
        const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = a[i];
            o[4 + i] = b[i];
        }
    } else {
        const u16x8 a = *reinterpret_cast<const u16x8*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = T::get(__builtin_bit_cast(typename T::type, (uint16_t)a[i]));
    }
}

template <typename T>
__device__ __forceinline__ void store8(typename T::type* p, const float* v) {
    if constexpr (T::bytes == 4) {
        reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
        reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        u16x8 a;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = __builtin_bit_cast(uint16_t, T::put(v[i]));
        *reinterpret_cast<u16x8*>(p) = a;
    }
}

template <typename T>
__device__ __forceinline__ void store4(typename T::type* p, const float* v) {
    if constexpr (T::bytes == 4) {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
        typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
        u16x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = __builtin_bit_cast(uint16_t, T::put(v[i]));
        *reinterpret_cast<u16x4*>(p) = a;
    }
}

// ----------------------------------------------------------- 4-bit codes

// Bit position of element e (0..7) in a word of codes.
__device__ __forceinline__ constexpr int nibble_shift(int e) { return 4 * ((e >> 1) + 4 * (e & 1)); }

// The eight codes of a word as exact fp16 integers, in element order: the code
// with its sign bit flipped, placed in the mantissa of 1024, less 1032; a code
// four bits higher in the mantissa counts 16 times and comes down by an exact
// fused multiply.  Nine instructions a word.
__device__ __forceinline__ half8 codes_f16(uint32_t w) {
    const half2v bias = __builtin_bit_cast(half2v, 0x64086408u);            // 1032
    const half2v sixteenth = __builtin_bit_cast(half2v, 0x2C002C00u);       // 1 / 16
    const half2v seventy2 = __builtin_bit_cast(half2v, 0xD480D480u);        // -72
    const uint32_t h = w >> 8;
    const half2v a = __builtin_bit_cast(half2v, (w & 0x000F000Fu) ^ 0x64086408u) - bias;
    const half2v b = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (w & 0x00F000F0u) ^ 0x64806480u), sixteenth,
                                               seventy2);
    const half2v c = __builtin_bit_cast(half2v, (h & 0x000F000Fu) ^ 0x64086408u) - bias;
    const half2v d = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (h & 0x00F000F0u) ^ 0x64806480u), sixteenth,
                                               seventy2);
    return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ int code_of(uint32_t w, int e) {
    return (int)(w << (28 - nibble_shift(e))) >> 28;
}

// ------------------------------------------------------------------ pages

struct Cache {
    uint8_t* data;
    int32_t* table;
    int32_t* len;
    int32_t* ref;
    int layers, n_pages, kv_heads, n_seqs, max_pages;
    int pt_log2;                                    // page_tokens = 1 << pt_log2
    int head_dim;

    __host__ __device__ int page_tokens() const { return 1 << pt_log2; }
    __host__ __device__ int64_t unit_bytes() const { return (int64_t)(head_dim + 8) << pt_log2; }
    __host__ __device__ int64_t page_bytes() const { return unit_bytes() * kv_heads; }
    // tokens of sequence s that its table row can describe
    __device__ int held(int s) const {
        const int n = len[s], cap = max_pages << pt_log2;
        return n < 0 ? 0 : n > cap ? cap : n;
    }
    __device__ uint8_t* unit(int layer, int page, int head) const {
        return data + (((int64_t)layer * n_pages + page) * kv_heads + head) * unit_bytes();
    }
    __device__ bool good(int page) const { return (unsigned)page < (unsigned)n_pages; }
};

// Rows of sequence s: [q0, q1) clamped to the call's rows.
struct Span {
    int q0, q1;
};
__device__ __forceinline__ Span span_of(const int32_t* q_start, int s, int rows) {
    int a = q_start[s], b = q_start[s + 1];
    a = a < 0 ? 0 : a > rows ? rows : a;
    b = b < a ? a : b > rows ? rows : b;
    return {a, b};
}

// Work units of a launch are numbered so that sequence s owns the slots base(s)
// .. base(s+1)-1 with base(s) = floor(q_start[s] * mul / per) + extra * s: at
// least as many as it can need, computed without a prefix sum.  The wave finds
// the sequence of a slot by a 64-way search (two rounds at most for 1024
// sequences; base ascends).
__device__ __forceinline__ int slot_base(const int32_t* q_start, int s, int rows, int mul, int per, int extra) {
    int a = q_start[s];
    a = a < 0 ? 0 : a > rows ? rows : a;
    return (int)((int64_t)a * mul / per) + extra * s;
}
__device__ __forceinline__ int seq_of_slot(const int32_t* q_start, int n_seqs, int rows, int mul, int per, int extra,
                                           int slot) {
    const int lane = threadIdx.x & (kWave - 1);
    int lo = 0, n = n_seqs;                          // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave;
        const int s = lo + lane * step;
        const bool le = lane * step < n && slot_base(q_start, s, rows, mul, per, extra) <= slot;
        const int c = __popcll(__ballot(le));
        const int k = c > 0 ? c - 1 : 0;
        const int left = n - k * step;
        lo += k * step;
        n = left < step ? left : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// --------------------------------------------------------------- launches

hipError_t launch_append(const Cache& c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
                         int rows, const int32_t* q_start, const int32_t* granted, hipStream_t st);
hipError_t launch_read(const Cache& c, int layer, const int32_t* first, const int32_t* q_start, int rows, void* k,
                       int64_t ldk, void* v, int64_t ldv, int dtype, hipStream_t st);

struct AttnArgs {
    const void* q;
    void* out;
    float* lse;
    const int32_t* q_start;
    const int32_t* granted;
    void* workspace;
    int64_t ldq, ldo;
    int layer, rows, heads, window;
    float scale;
    int64_t max_len;
};
int64_t attention_grid(const Cache& c, int rows, int heads, int64_t max_len);   // workgroups of the launch
int64_t attention_workspace(const Cache& c, int rows, int heads, int64_t max_len);
hipError_t launch_attention(const Cache& c, const AttnArgs& a, int dtype, hipStream_t st);

hipError_t launch_reserve(const Cache& c, const int32_t* n_new, int32_t* granted, int32_t* ws, hipStream_t st);
hipError_t launch_fork(const Cache& c, int n, const int32_t* src, const int32_t* dst, const int32_t* n_tokens,
                       int32_t* ok, hipStream_t st);
hipError_t launch_truncate(const Cache& c, const int32_t* new_len, hipStream_t st);
hipError_t launch_compact(const Cache& c, int32_t* remap, int32_t* n_live, int32_t* ws, hipStream_t st);

struct LinearArgs {
    const void* x;
    const uint8_t* w;
    const float* scale;
    const float* bias;
    const void* residual;
    void* y;
    void* workspace;
    int64_t ldx, ldr, ldy;
    int T, K, N, act;
};
int64_t linear_grid(const LinearArgs& a);       // workgroups of the largest launch at most
int64_t linear_workspace(int bits, int dtype, int64_t T, int64_t K, int64_t N);
hipError_t launch_linear(int bits, int dtype, const LinearArgs& a, hipStream_t st);

}  // namespace attn
}  // namespace moedec
