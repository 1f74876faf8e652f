// Writing rows of keys and values into the 4-bit cache and reading them back.
//
// A row (one token of one head) is quantised by the rule of the weights' row
// quantiser: s = absmax / 7, code = rint(x / s) (both divisions IEEE fp32, ties
// to even, clamped to the field), a zero row gets s = 0 and codes 0, a row with
// a NaN or an infinity s = NaN and codes 0.
//
// HBM- or latency-bound: 2 * head_dim elements read and head_dim + 8 bytes
// written per row.  One wave owns the rows of an aligned block of 8 tokens, so
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
__device__ __forceinline__ uint32_t code(float x, float s) {
    if (!(s > 0.f)) return 0;
    return (uint32_t)(int)fminf(fmaxf(rintf(x / s), -8.f), 7.f) & 15u;
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Cache c, Rows r, int layer,
                                                              const typename T::type* __restrict__ k, int64_t ldk,
                                                              const typename T::type* __restrict__ v, int64_t ldv) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t u = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    const int head = (int)((u >> 1) % c.kv_heads), slot = (int)((u >> 1) / c.kv_heads);
    const Block b = find_block(c, r, slot, false);
    if (!b.any || b.page_index < 0) return;
    const int page = c.table[(int64_t)b.s * c.max_pages + b.page_index];
    if (!c.good(page)) return;
    uint8_t* unit = c.unit(layer, page, head);
    const int pt = c.page_tokens();
    if ((u & 1) == 0) {
        // keys: 32 lanes a row, 8 columns (one word) a lane, two rows at once
        const int l = lane & 31;
        const bool mine = l < D / 8;
        const int g = l & 3, s = l >> 2;                     // columns 32*s + 8*g
        float x[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 2 * i + (lane >> 5);
            const bool on = mine && t >= b.t0 && t < b.t1;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
            if (on) load8<T>(k + (int64_t)(b.row0 + t - b.t0) * ldk + (int64_t)head * D + 8 * l, x[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 2 * i + (lane >> 5);
            const bool on = mine && t >= b.t0 && t < b.t1;
            float a = 0.f;
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = fabsf(x[i][e]);
                bad = bad || !(f <= kFltMax);
                a = fmaxf(a, f);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) a = fmaxf(a, __shfl_xor(a, o, kWave));
            const uint64_t bm = __ballot(bad);
            const float sc = scale_of(a, (lane < 32 ? (uint32_t)bm : (uint32_t)(bm >> 32)) != 0);
            if (on) {
                uint32_t w = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) w |= code(x[i][e], sc) << nibble_shift(e);
                const int tok = b.slot0 + t;
                reinterpret_cast<uint32_t*>(unit)[tok * (D / 8) + g * (D / 32) + s] = w;
                if (l == 0) reinterpret_cast<float*>(unit + (int64_t)pt * D)[tok] = sc;
            }
        }
        return;
    }
    // values: a lane holds column lane + 64*j of all 8 tokens and packs them
    constexpr int J = D / 64;
    float x[8][J];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int j = 0; j < J; ++j)
            x[t][j] = t >= b.t0 && t < b.t1
                          ? T::get(v[(int64_t)(b.row0 + t - b.t0) * ldv + (int64_t)head * D + lane + 64 * j])
                          : 0.f;
    uint32_t w[J] = {}, keep = 0xFFFFFFFFu;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        float a = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float f = fabsf(x[t][j]);
            bad = bad || !(f <= kFltMax);
            a = fmaxf(a, f);
        }
        a = wave_max(a);
        const float sc = scale_of(a, __ballot(bad) != 0);
        if (t >= b.t0 && t < b.t1) {
            keep &= ~(15u << nibble_shift(t));
#pragma unroll
            for (int j = 0; j < J; ++j) w[j] |= code(x[t][j], sc) << nibble_shift(t);
            if (lane == 0) reinterpret_cast<float*>(unit + (int64_t)pt * (D + 4))[b.slot0 + t] = sc;
        }
    }
    uint32_t* words = reinterpret_cast<uint32_t*>(unit + (int64_t)pt * (D / 2)) + (int64_t)(b.slot0 >> 3) * D;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (keep) w[j] |= words[lane + 64 * j] & keep;
        words[lane + 64 * j] = w[j];
    }
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Cache c, Rows r, int layer,
                                                            typename T::type* __restrict__ k, int64_t ldk,
                                                            typename T::type* __restrict__ v, int64_t ldv) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t u = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    const int head = (int)((u >> 1) % c.kv_heads), slot = (int)((u >> 1) / c.kv_heads);
    const Block b = find_block(c, r, slot, true);
    if (!b.any) return;
    const int page = b.page_index < 0 ? -1 : c.table[(int64_t)b.s * c.max_pages + b.page_index];
    // tokens of the block that are there: a sequence's positions, in a good page
    const int end = c.good(page) ? c.held(b.s) - (b.page_index << c.pt_log2) - b.slot0 : 0;
    const uint8_t* unit = c.unit(layer, c.good(page) ? page : 0, head);
    const int pt = c.page_tokens();
    if ((u & 1) == 0) {
        const int l = lane & 31;
        if (l >= D / 8) return;
        const int g = l & 3, s = l >> 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 2 * i + (lane >> 5);
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
    uint32_t w[J];
#pragma unroll
    for (int j = 0; j < J; ++j) w[j] = end > 0 ? words[lane + 64 * j] : 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if (t < b.t0 || t >= b.t1) continue;
        const float sc = t < end ? scales[t] : 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j)
            v[(int64_t)(b.row0 + t - b.t0) * ldv + (int64_t)head * D + lane + 64 * j] =
                T::put(t < end ? (float)code_of(w[j], t) * sc : 0.f);
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
