// Writing rows of keys and values into the 4-bit cache and reading them back.
//
// A row (one token of one head) is quantised by the rule of the weights' row
// quantiser: s = absmax / 7, code = rint(x / s) (both divisions IEEE fp32, ties
// to even, clamped to the field), a zero row gets s = 0 and codes 0, a row with
// a NaN or an infinity s = NaN and codes 0.
//
// HBM- or latency-bound: 2 * head_dim elements read and head_dim + 8 bytes
// written per row (5601 bf16 tokens of 8 heads of 128: 16.5 us written, 1.8 TB/s, and
// 13 read back; 42 tokens 3.9 us and 3.7, a launch and three memory latencies).  One wave owns the rows of an aligned block of 8 tokens, so
// that every word of value codes (8 tokens of one column) is written whole by
// one lane; a block that the call covers in part is read first and merged.
// Blocks at a sequence's ends are the only ones written in part, and a page that
// is written belongs to one sequence, so no two waves share a word.
#include "attn.h"

namespace moedec {
namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr float kFltMax = 3.402823466e38f;
constexpr float kInf = __builtin_inff();

// Lanes that hold a row of keys, eight columns each: a power of two.
constexpr int key_lanes(int D) { return D == 64 ? 8 : D == 128 ? 16 : 32; }

struct Rows {
    const int32_t* q_start;
    const int32_t* granted;      // append
    const int32_t* first;        // read
    int rows, slots;
};

// The unit of a wave: block `blk` of 8 positions of sequence s; its tokens
// [t0, t1) of the block are rows row0 + (t - t0).
struct Block {
    int s, page_index, slot0;    // slot0: the block's first position inside its page
    int t0, t1, row0;
    bool any;
};

// `slots` work slots hold all blocks: a sequence of n rows spans at most
// (n - 1) / 8 + 2 blocks and owns at least n / 8 + 2 slots.
__device__ __forceinline__ Block find_block(const Cache& c, const Rows& r, int slot, bool read) {
    Block b;
    b.s = seq_of_slot(r.q_start, c.n_seqs, r.rows, 1, 8, 2, slot);
    const Span q = span_of(r.q_start, b.s, r.rows);
    int m = q.q1 - q.q0;
    if (r.granted) m = min(m, max(r.granted[b.s], 0));
    const int64_t p0 = read ? (int64_t)r.first[b.s] : (int64_t)c.held(b.s) - m;
    const int64_t blk = (p0 >> 3) + (slot - slot_base(r.q_start, b.s, r.rows, 1, 8, 2));
    const int64_t lo = blk * 8 > p0 ? blk * 8 : p0, hi = min(blk * 8 + 8, p0 + m);
    b.any = m > 0 && slot < r.slots && lo < hi;
    b.t0 = (int)(lo - blk * 8);
    b.t1 = (int)(hi - blk * 8);
    b.row0 = q.q0 + (int)(lo - p0);
    const int64_t cap = (int64_t)c.max_pages << c.pt_log2;
    b.page_index = blk < 0 || blk * 8 >= cap ? -1 : (int)(blk * 8 >> c.pt_log2);
    b.slot0 = (int)(blk * 8) & (c.page_tokens() - 1);
    return b;
}

// The row scale of an absolute maximum (NaN if the row held a NaN or infinity).
__device__ __forceinline__ float scale_of(float amax, bool bad) {
    return bad ? __uint_as_float(0x7FC00000u) : amax / 7.0f;
}

// How a row is divided by its scale s.  With r = 1/s correctly rounded, q0 = x*r
// and e = x - q0*s (one fma, exact), fma(e, r, q0) is the correctly rounded
// quotient (Markstein 1990) as long as nothing under- or overflows; scales far
// from 1 take the division itself.
struct Divisor {
    float s, r;
    bool plain, live;
};
__device__ __forceinline__ Divisor divisor(float s) {
    return {s, 1.0f / s, s > 0x1p-90f && s < 0x1p90f, s > 0.f};
}
__device__ __forceinline__ float quotient(float x, const Divisor& d) {
    const float q = x * d.r;
    return fmaf(fmaf(-q, d.s, x), d.r, q);
}
__device__ __forceinline__ uint32_t code(float q) {
    return (uint32_t)(int)fminf(fmaxf(rintf(q), -8.f), 7.f) & 15u;
}
// Hands the codes of N values of a row to put(i, code); a row whose scale is 0 or
// NaN has none (its codes stay 0).
template <int N, typename F>
__device__ __forceinline__ void add_codes(const float* x, const Divisor& d, F&& put) {
    if (d.plain) {
#pragma unroll
        for (int i = 0; i < N; ++i) put(i, code(quotient(x[i], d)));
    } else if (d.live) {
#pragma unroll
        for (int i = 0; i < N; ++i) put(i, code(x[i] / d.s));
    }
}

// Columns of the values: lane l holds pairs (2l, 2l + 1) of every whole 128 and,
// where 64 are left over, column l of those.
template <int D>
__device__ __forceinline__ constexpr int value_col(int j, int lane) {
    return j < D / 128 * 2 ? j / 2 * 128 + 2 * lane + (j & 1) : D / 128 * 128 + lane;
}
template <typename T, int D>
__device__ __forceinline__ void load_values(const typename T::type* row, int lane, float* x) {
    typedef typename T::type pair __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int j = 0; j < D / 128 * 2; j += 2) {
        const pair p = *reinterpret_cast<const pair*>(row + value_col<D>(j, lane));
        x[j] = T::get(p[0]);
        x[j + 1] = T::get(p[1]);
    }
    if constexpr (D % 128 != 0) x[D / 64 - 1] = T::get(row[value_col<D>(D / 64 - 1, lane)]);
}
template <typename T, int D>
__device__ __forceinline__ void store_values(typename T::type* row, int lane, const float* x) {
    typedef typename T::type pair __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int j = 0; j < D / 128 * 2; j += 2)
        *reinterpret_cast<pair*>(row + value_col<D>(j, lane)) = pair{T::put(x[j]), T::put(x[j + 1])};
    if constexpr (D % 128 != 0) row[value_col<D>(D / 64 - 1, lane)] = T::put(x[D / 64 - 1]);
}
template <int D>
__device__ __forceinline__ void load_value_words(const uint32_t* p, int lane, uint32_t* w) {
#pragma unroll
    for (int j = 0; j < D / 128 * 2; j += 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p + value_col<D>(j, lane));
        w[j] = v.x;
        w[j + 1] = v.y;
    }
    if constexpr (D % 128 != 0) w[D / 64 - 1] = p[value_col<D>(D / 64 - 1, lane)];
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Cache c, Rows r, int layer,
                                                              const typename T::type* __restrict__ k, int64_t ldk,
                                                              const typename T::type* __restrict__ v, int64_t ldv) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t u = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int head = (int)((u >> 1) % c.kv_heads), slot = (int)((u >> 1) / c.kv_heads);
    const Block b = find_block(c, r, slot, false);
    if (!b.any || b.page_index < 0) return;
    const int page = c.table[(int64_t)b.s * c.max_pages + b.page_index];
    if (!c.good(page)) return;
    const int pt = c.page_tokens();
    uint8_t* unit = c.unit(layer, page, head);
    if ((u & 1) == 0) {
        // keys: kLanes lanes a row, 8 columns (one word) a lane, kAtOnce rows together
        constexpr int kLanes = key_lanes(D), kAtOnce = kWave / kLanes, kPasses = 8 / kAtOnce;
        const int l = lane % kLanes, sub = lane / kLanes;
        const bool mine = l < D / 8;
        const int g = l & 3, s = l >> 2;                     // columns 32*s + 8*g
        float x[kPasses][8];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int t = i * kAtOnce + sub;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
            if (mine && t >= b.t0 && t < b.t1)
                load8<T>(k + (int64_t)(b.row0 + t - b.t0) * ldk + (int64_t)head * D + 8 * l, x[i]);
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int t = i * kAtOnce + sub;
            float a = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = fabsf(x[i][e]);
                a = f <= kFltMax ? fmaxf(a, f) : kInf;       // a NaN or an infinity: bad, and stays so
            }
            a = fmaxf(a, dpp_f<0xB1>(a));
            a = fmaxf(a, dpp_f<0x4E>(a));
            a = fmaxf(a, dpp_f<0x141>(a));
            if constexpr (kLanes >= 16) a = fmaxf(a, dpp_f<0x140>(a));
            if constexpr (kLanes >= 32) a = fmaxf(a, __shfl_xor(a, 16, kWave));
            const float sc = scale_of(a, a > kFltMax);
            if (mine && t >= b.t0 && t < b.t1) {
                uint32_t w = 0;
                add_codes<8>(x[i], divisor(sc), [&](int e, uint32_t q) { w |= q << nibble_shift(e); });
                const int tok = b.slot0 + t;
                reinterpret_cast<uint32_t*>(unit)[tok * (D / 8) + g * (D / 32) + s] = w;
                if (l == 0) reinterpret_cast<float*>(unit + (int64_t)pt * D)[tok] = sc;
            }
        }
        return;
    }
    // values: a lane holds its columns of all 8 tokens and packs them
    constexpr int J = D / 64;
    float x[8][J];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int j = 0; j < J; ++j) x[t][j] = 0.f;
        if (t >= b.t0 && t < b.t1)
            load_values<T, D>(v + (int64_t)(b.row0 + t - b.t0) * ldv + (int64_t)head * D, lane, x[t]);
    }
    uint32_t* words = reinterpret_cast<uint32_t*>(unit + (int64_t)pt * (D / 2)) + (int64_t)(b.slot0 >> 3) * D;
    uint32_t w[J], keep = 0xFFFFFFFFu;
#pragma unroll
    for (int t = 0; t < 8; ++t)
        if (t >= b.t0 && t < b.t1) keep &= ~(15u << nibble_shift(t));
    if (keep) load_value_words<D>(words, lane, w);       // a block written in part
#pragma unroll
    for (int j = 0; j < J; ++j) w[j] = keep ? w[j] & keep : 0u;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if (t < b.t0 || t >= b.t1) continue;
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float f = fabsf(x[t][j]);
            a = f <= kFltMax ? fmaxf(a, f) : kInf;
        }
        a = wave_max(a);
        const float sc = scale_of(a, a > kFltMax);
        add_codes<J>(x[t], divisor(sc), [&](int j, uint32_t q) { w[j] |= q << nibble_shift(t); });
        if (lane == 0) reinterpret_cast<float*>(unit + (int64_t)pt * (D + 4))[b.slot0 + t] = sc;
    }
#pragma unroll
    for (int j = 0; j < D / 128 * 2; j += 2)
        *reinterpret_cast<uint2*>(words + value_col<D>(j, lane)) = uint2{w[j], w[j + 1]};
    if constexpr (D % 128 != 0) words[value_col<D>(J - 1, lane)] = w[J - 1];
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Cache c, Rows r, int layer,
                                                            typename T::type* __restrict__ k, int64_t ldk,
                                                            typename T::type* __restrict__ v, int64_t ldv) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t u = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int head = (int)((u >> 1) % c.kv_heads), slot = (int)((u >> 1) / c.kv_heads);
    const Block b = find_block(c, r, slot, true);
    if (!b.any) return;
    const int page = b.page_index < 0 ? -1 : c.table[(int64_t)b.s * c.max_pages + b.page_index];
    // tokens of the block that are there: a sequence's positions, in a good page
    const int end = c.good(page) ? c.held(b.s) - (b.page_index << c.pt_log2) - b.slot0 : 0;
    const int pt = c.page_tokens();
    const uint8_t* unit = c.unit(layer, c.good(page) ? page : 0, head);
    if ((u & 1) == 0) {
        constexpr int kLanes = key_lanes(D), kAtOnce = kWave / kLanes;
        const int l = lane % kLanes, g = l & 3, s = l >> 2;
        if (l >= D / 8) return;
#pragma unroll
        for (int i = 0; i < 8 / kAtOnce; ++i) {
            const int t = i * kAtOnce + lane / kLanes;
            if (t < b.t0 || t >= b.t1) continue;
            float o[8] = {};
            if (t < end) {
                const int tok = b.slot0 + t;
                const uint32_t w = reinterpret_cast<const uint32_t*>(unit)[tok * (D / 8) + g * (D / 32) + s];
                const float sc = reinterpret_cast<const float*>(unit + (int64_t)pt * D)[tok];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = (float)code_of(w, e) * sc;
            }
            store8<T>(k + (int64_t)(b.row0 + t - b.t0) * ldk + (int64_t)head * D + 8 * l, o);
        }
        return;
    }
    const uint32_t* words = reinterpret_cast<const uint32_t*>(unit + (int64_t)pt * (D / 2)) + (int64_t)(b.slot0 >> 3) * D;
    const float* scales = reinterpret_cast<const float*>(unit + (int64_t)pt * (D + 4)) + b.slot0;
    constexpr int J = D / 64;
    uint32_t w[J] = {};
    if (end > 0) load_value_words<D>(words, lane, w);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if (t < b.t0 || t >= b.t1) continue;
        const float sc = t < end ? scales[t] : 0.f;
        float x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) x[j] = t < end ? (float)code_of(w[j], t) * sc : 0.f;
        store_values<T, D>(v + (int64_t)(b.row0 + t - b.t0) * ldv + (int64_t)head * D, lane, x);
    }
}

template <typename T, int D>
void rows_launch(const Cache& c, const Rows& r, int layer, void* k, int64_t ldk, void* v, int64_t ldv, bool read,
                 hipStream_t st) {
    typedef typename T::type E;
    const int64_t units = (int64_t)r.slots * c.kv_heads * 2;
    const dim3 grid((unsigned)((units + kWaves - 1) / kWaves));
    if (read)
        hipLaunchKernelGGL((kv4_read_kernel<T, D>), grid, dim3(kThreads), 0, st, c, r, layer, (E*)k, ldk, (E*)v, ldv);
    else
        hipLaunchKernelGGL((kv4_append_kernel<T, D>), grid, dim3(kThreads), 0, st, c, r, layer, (const E*)k, ldk,
                           (const E*)v, ldv);
}

template <typename T>
hipError_t rows_dim(const Cache& c, const Rows& r, int layer, void* k, int64_t ldk, void* v, int64_t ldv, bool read,
                    hipStream_t st) {
    switch (c.head_dim) {
        case 64: rows_launch<T, 64>(c, r, layer, k, ldk, v, ldv, read, st); break;
        case 128: rows_launch<T, 128>(c, r, layer, k, ldk, v, ldv, read, st); break;
        case 192: rows_launch<T, 192>(c, r, layer, k, ldk, v, ldv, read, st); break;
        case 256: rows_launch<T, 256>(c, r, layer, k, ldk, v, ldv, read, st); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t rows_any(const Cache& c, const Rows& r, int layer, void* k, int64_t ldk, void* v, int64_t ldv, int dtype,
                    bool read, hipStream_t st) {
    if (r.rows == 0) return hipSuccess;
    switch (dtype) {
        case MOEDEC_F32: return rows_dim<F32>(c, r, layer, k, ldk, v, ldv, read, st);
        case MOEDEC_F16: return rows_dim<F16>(c, r, layer, k, ldk, v, ldv, read, st);
        case MOEDEC_BF16: return rows_dim<BF16>(c, r, layer, k, ldk, v, ldv, read, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_append(const Cache& c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
                         int rows, const int32_t* q_start, const int32_t* granted, hipStream_t st) {
    const Rows r{q_start, granted, nullptr, rows, rows / 8 + 2 * c.n_seqs};
    return rows_any(c, r, layer, const_cast<void*>(k), ldk, const_cast<void*>(v), ldv, dtype, false, st);
}

hipError_t launch_read(const Cache& c, int layer, const int32_t* first, const int32_t* q_start, int rows, void* k,
                       int64_t ldk, void* v, int64_t ldv, int dtype, hipStream_t st) {
    const Rows r{q_start, nullptr, first, rows, rows / 8 + 2 * c.n_seqs};
    return rows_any(c, r, layer, k, ldk, v, ldv, dtype, true, st);
}

}  // namespace attn
}  // namespace moedec
