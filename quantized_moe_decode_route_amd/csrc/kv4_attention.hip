// Attention over the paged 4-bit cache.
//
//   S[j][m] = q_m . k_j = s_k[j] * sum_c code_k[j][c] * q_m[c]
//   p = exp2(S * scale * log2 e - M_m),  O[m] = sum_j (p * s_v[j]) * code_v[j] / sum_j p
//
// The row scales factor out of both products, so the matrix cores work on the
// codes themselves, which are exact in fp16.  With 16-bit queries the keys' codes
// enter as unsigned fields in fp16 subnormals, 5 instructions a word instead of 9
// (u = code + 8 at bit 0 or 4 of its half is u * 2^-24 or u * 2^-20; the 2^4 is
// taken out of the query element that meets it, the offset out of the start of the
// sum, which is -8 times the sum of the row's queries and as such the product's
// free addend); the matrix core loses the subnormals' leading zeros below the
// largest product, 1e-5 of a sum's rms, far below the rounding of a 16-bit
// result, and fp32 queries meet signed codes.  A row m is one query head of one
// token; 16 rows that share a key/value head are the N side of the products
// (B operand), 32 keys at a time the M side of S^T = K Q^T and the K side of
// O^T = V^T P^T.  In S^T a lane holds one row (lane % 16) and, with the tokens
// of a 32-key step given to the two 16-key MFMAs as 8*(r/4) + 4*t + r%4, keys
// 8*(lane/16) .. +7: exactly the K-values its B operand of the second product
// needs.  So probabilities never leave their lane, and the running maximum, the
// sum and the rescaling of the accumulators are per-lane scalars.
//
// A workgroup owns NT * 16 rows and a stretch of keys, its four waves take every
// fourth 32-key step, so a code is converted once per workgroup however many rows
// it serves: NT = 1 for single tokens, 2 and 3 for drafts and prompts.  Bound by
// HBM for few rows (each step's 32 * (head_dim + 8) bytes are loaded one step
// ahead), by the vector ALUs for many (about 150 instructions a step for the
// codes, fewer beside 16-bit queries, and 75 a row tile for the softmax, against 16
// MFMAs of 16 cycles a row tile at head_dim 128).  At head_dim 128, 8 heads of keys
// and 48 of queries: 64 sequences of up to 8192 keys, one bf16 query each, 80 + 5
// us for 315 MB, 3.9 TB/s; 3 fp32 queries each of two sequences, up to 131,072 keys,
// 101 + 7 us for 245 MB; 2813 bf16 queries of two sequences of up to 6000 keys 530
// us, 636 TF/s.
//
// Queries enter as fp16 under one power of two per row: exact for fp16 and bf16,
// as a hi/lo pair (22 bits) for fp32.  The probabilities times their value scale
// enter the second product as fp16 (fp32: again as a pair) under one power of two
// per wave that follows the largest value scale seen.  For 16-bit activations the
// rounding of a probability to fp16 (2^-12 relative) is below that of the output.
// Scores, maxima, sums and accumulators are fp32.  The maximum is a reference,
// moved (with a rescaling) only when a score passes it by a factor of 2^8.
#include "attn.h"

namespace moedec {
namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kKeys = 32;                 // keys of a wave's step
constexpr int kRound = kKeys * kWaves;    // keys of a round of the workgroup
constexpr int kMinChunk = 256;            // keys of a split at least
constexpr int kMaxSplits = 256;
constexpr int kNoSplit = 768;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kFltMax = 3.402823466e38f;
constexpr float kSlack = 8.f;             // log2 by which a score may pass the reference

__device__ __forceinline__ floatx4 mfma16(const half8& a, const half8& b, const floatx4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The largest of three, ignoring NaN: one instruction (fmaxf adds one per operand
// whose bits come from memory, to quiet signalling NaNs).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float max8(const float* v) {
    return max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), max3(v[6], v[7], v[7]));
}

// 2^k as a float, k in [-126, 127].
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// Exponent k with m * 2^k in [2^14, 2^15) (0 for zero and non-finite m).
__device__ __forceinline__ int row_exponent(float m) {
    if (!(m > 0.f) || !(m <= kFltMax)) return 0;
    const int e = (int)(__float_as_uint(m) >> 23) - 127;        // -127 for subnormals
    const int k = 14 - e;
    return k > 120 ? 120 : k;
}

template <int N>
struct Words {
    uint32_t w[N];
};
// N consecutive words, in 16- or 8-byte loads (N even, p aligned to them).
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint32_t* p) {
    Words<N> o;
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) o.w[4 * i + k] = v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint2 v = reinterpret_cast<const uint2*>(p)[i];
            o.w[2 * i] = v.x;
            o.w[2 * i + 1] = v.y;
        }
    }
    return o;
}

// A row tile: rows [r0, r0 + rt) of sequence s's m * group rows (row = token *
// group + head of the group), and the keys [lo, hi) that any of them sees.
struct Tile {
    int s, q0, n, m, len, r0, lo, hi, per;
    int full0, full1;                    // keys [full0, full1) are seen by every row of the tile
    bool any;
};

__device__ __forceinline__ Tile find_tile(const Cache& c, const AttnArgs& a, int slot, int splits, int rt) {
    Tile t;
    const int group = a.heads / c.kv_heads;
    t.s = seq_of_slot(a.q_start, c.n_seqs, a.rows, group, rt, 1, slot);
    const Span q = span_of(a.q_start, t.s, a.rows);
    t.q0 = q.q0;
    t.n = q.q1 - q.q0;
    t.m = a.granted ? min(t.n, max(a.granted[t.s], 0)) : t.n;
    t.len = c.held(t.s);
    t.r0 = (slot - slot_base(a.q_start, t.s, a.rows, group, rt, 1)) * rt;
    t.any = t.r0 >= 0 && t.r0 < t.n * group;                                 // slots before the first sequence: none
    const int first = t.len - t.m + t.r0 / group;                            // position of the first row
    const int last = t.len - t.m + min(t.r0 + rt - 1, t.m * group - 1) / group;
    t.hi = t.r0 < t.m * group ? max(last + 1, 0) : 0;
    t.lo = a.window > 0 ? max(first - a.window + 1, 0) & ~(kKeys - 1) : 0;
    if (t.hi < t.lo) t.hi = t.lo;
    t.full1 = first + 1;
    t.full0 = a.window > 0 ? last - a.window + 1 : 0;
    const int each = (t.hi - t.lo + splits - 1) / splits;
    t.per = max(kMinChunk, (each + kRound - 1) / kRound * kRound);
    return t;
}

// The eight codes of a word as unsigned fields: element e is (code + 8) *
// 2^(field_bit(e) - 24).
__device__ __forceinline__ half8 codes_unsigned(uint32_t w) {
    const uint32_t h = w >> 8;
    return __builtin_bit_cast(half8, u32x4{(w & 0x000F000Fu) ^ 0x00080008u, (w & 0x00F000F0u) ^ 0x00800080u,
                                           (h & 0x000F000Fu) ^ 0x00080008u, (h & 0x00F000F0u) ^ 0x00800080u});
}
__device__ __forceinline__ constexpr int field_bit(int e) { return e & 2 ? 4 : 0; }

// Waves a SIMD is to hold (the register budget): as many as the accumulators allow
// without spilling.
constexpr int waves_per_simd(int D, int NT, bool pair) {
    return D <= 128 && NT == 1 ? 4 : D == 64 ? (pair ? 4 : 3) : 2;
}

// One split of one tile of one key/value head.
template <typename T, int D, int NT>
__global__ __launch_bounds__(kThreads, waves_per_simd(D, NT, T::bytes == 4)) void kv4_attention_kernel(Cache c, AttnArgs a, int splits) {
    constexpr bool kPair = T::bytes == 4, kOffset = !kPair;
    constexpr int kP = kPair ? 2 : 1;
    constexpr int kS = D / 32;            // MFMAs of a score, K side
    constexpr int kH = D / 64;            // 64-column parts of the output
    constexpr int kRT = 16 * NT;
    constexpr int kLd = D + 4;
    __shared__ half8 qs[NT][kS][kP][kWave];
    __shared__ float so[kRT][kLd];
    __shared__ float scm[kRT], sstart[kRT], sm[kWaves][kRT], sl[kWaves][kRT];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane & 15, g = lane >> 4;
    const int head = blockIdx.x % c.kv_heads, sp = blockIdx.x / c.kv_heads % splits;
    const int slots = gridDim.x / c.kv_heads / splits;
    const int slot = slots - 1 - (int)(blockIdx.x / c.kv_heads / splits);    // the longest tiles of a prompt first
    const int group = a.heads / c.kv_heads;
    const Tile t = find_tile(c, a, slot, splits, kRT);
    if (!t.any) return;
    const int k0 = t.lo + sp * t.per, k1 = min(t.hi, k0 + t.per);
    if (sp > 0 && k0 >= t.hi) return;
    const int rows = t.m * group;          // rows that count

    const int width = a.window > 0 ? a.window : 0x7FFFFFFF;     // see1 - width stays in range: see1 >= 0
    const int pt = c.page_tokens();
    const int32_t* row_pages = c.table + (int64_t)t.s * c.max_pages;
    const int first = k0 + wave * kKeys;
    const int steps = first < k1 ? (k1 - first + kRound - 1) / kRound : 0;
    // lane i: the page of step 64*k + i
    auto load_pages = [&](int step) {
        const int j = first + (step + lane) * kRound;
        return step + lane < steps ? row_pages[j >> c.pt_log2] : -1;
    };
    const uint8_t* base = c.data + (int64_t)a.layer * c.n_pages * c.page_bytes() + head * c.unit_bytes();
    auto unit_of = [&](int page) { return base + (int64_t)page * c.page_bytes(); };
    Words<kS> kw[2];                       // codes and scales of a step's keys: loaded a step ahead
    Words<8> ks;
    auto load_keys = [&](int page, int step) {
        const uint8_t* unit = unit_of(page);
        const int at = (first + step * kRound) & (pt - 1);
#pragma unroll
        for (int tl = 0; tl < 2; ++tl) {
            const int kt = at + 8 * (n >> 2) + 4 * tl + (n & 3);
            kw[tl] = load_words<kS>(reinterpret_cast<const uint32_t*>(unit) + kt * (D / 8) + g * kS);
        }
        ks = load_words<8>(reinterpret_cast<const uint32_t*>(unit + pt * D) + at + 8 * g);
    };

    int pages = load_pages(0);
    int page = steps > 0 ? __builtin_amdgcn_readlane(pages, 0) : -1;
    if (c.good(page)) load_keys(page, 0);
    // The queries, one 16-row block a wave, to LDS in operand order; cm turns a
    // score of codes and fp16 queries into log2 units (its sign is the queries').
    for (int nt = wave; nt < NT; nt += kWaves) {
        const int row = t.r0 + 16 * nt + n;
        const bool on = row < rows;
        const typename T::type* src = reinterpret_cast<const typename T::type*>(a.q) +
                                      (int64_t)(t.q0 + (on ? row / group : 0)) * a.ldq +
                                      (int64_t)(head * group + (on ? row % group : 0)) * D + 8 * g;
        float x[kS][8], m = 0.f;
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            load8<T>(src + 32 * s, x[s]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!on) x[s][e] = 0.f;
                m = fmaxf(m, fabsf(x[s][e]));
            }
        }
        m = fmaxf(m, __shfl_xor(m, 16, kWave));
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        const int k = row_exponent(m);
        const float f = a.scale < 0.f ? -pow2(k) : pow2(k);
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            half8 h, l;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = x[s][e] * (kOffset && field_bit(e) ? f * 0.0625f : f);
                if (kPair) asm volatile("" : "+v"(v));          // one rounding for both halves
                const _Float16 hv = (_Float16)v;
                h[e] = hv;
                sum += (float)hv * (float)(1 << field_bit(e));
                l[e] = (_Float16)(v - (float)hv);
            }
            qs[nt][s][0][lane] = h;
            if (kPair) qs[nt][s][kP - 1][lane] = l;
        }
        // never 0: the score of an unseen key is -inf times cm
        // (kOffset: half of the sums' 2^24, the other half goes to the keys' scales)
        if (g == 0) scm[16 * nt + n] = fmaxf(pow2(-k) * fabsf(a.scale) * kLog2e * (kOffset ? 0x1p12f : 1.f), 0x1p-126f);
        if (kOffset) {
            sum += __shfl_xor(sum, 16, kWave);
            sum += __shfl_xor(sum, 32, kWave);
            if (g == 0) sstart[16 * nt + n] = sum * (-8.f * 0x1p-24f);
        }
    }

    __syncthreads();                       // queries staged
    float cm[NT], M[NT], L[NT];            // M: reference score, L: this lane's part of the sum
    int see1[NT];                          // keys [see1 - window, see1) are seen
    floatx4 acc[NT][kH][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int row = t.r0 + 16 * i + n, pos = t.len - t.m + row / group;
        cm[i] = scm[16 * i + n];
        M[i] = kNegInf;
        L[i] = 0.f;
        see1[i] = row < rows ? max(pos + 1, 0) : 0;
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][h][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    floatx4 start[NT];                     // the first product's addend, held in registers
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const float v = kOffset ? sstart[16 * i + n] : 0.f;
        start[i] = floatx4{v, v, v, v};
        asm volatile("" : "+v"(start[i]));
    }
    float vref = 0x1p-100f, vinv = 0x1p105f;       // value scales enter as s_v * vinv <= 2^5, vinv = 2^5 / vref

    for (int step = 0; step < steps; ++step) {
        int next = -1;
        if (step + 1 < steps) {
            if (((step + 1) & (kWave - 1)) == 0) pages = load_pages(step + 1);
            next = __builtin_amdgcn_readlane(pages, (step + 1) & (kWave - 1));
        }
        if (!c.good(page)) {                       // positions that are not there
            page = next;
            if (c.good(page)) load_keys(page, step + 1);
            continue;
        }
        const int j0 = first + step * kRound;
        Words<4> vw[kH];                           // this step's values: needed after the softmax
        Words<8> vsw;
        {
            const uint8_t* unit = unit_of(page);
            const int at = j0 & (pt - 1);
            const uint32_t* vp = reinterpret_cast<const uint32_t*>(unit + pt * (D / 2)) + ((at >> 3) + g) * D + 4 * n;
#pragma unroll
            for (int h = 0; h < kH; ++h) vw[h] = load_words<4>(vp + 64 * h);
            vsw = load_words<8>(reinterpret_cast<const uint32_t*>(unit + pt * (D + 4)) + at + 8 * g);
        }

        const bool edge = j0 < t.full0 || j0 + kKeys > t.full1;    // some row does not see some key

    // scores: z[i][e] = s_k * (codes . q) of key j0 + 8*g + e, before cm
        floatx4 sc[NT][2];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const half8 kf0 = kOffset ? codes_unsigned(kw[0].w[s]) : codes_f16(kw[0].w[s]);
            const half8 kf1 = kOffset ? codes_unsigned(kw[1].w[s]) : codes_f16(kw[1].w[s]);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const half8 q = qs[i][s][p][lane];
                    sc[i][0] = mfma16(kf0, q, s == 0 && p == 0 ? start[i] : sc[i][0]);
                    sc[i][1] = mfma16(kf1, q, s == 0 && p == 0 ? start[i] : sc[i][1]);
                }
        }
        bool move = false;
        float z[NT][8], mx[NT], kscale[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) kscale[e] = __uint_as_float(ks.w[e]) * (kOffset ? 0x1p12f : 1.f);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z[i][e] = sc[i][e >> 2][e & 3] * kscale[e];
            if (edge) {
                asm volatile("");                  // a branch, not selects in every step
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int key = j0 + 8 * g + e;
                    z[i][e] = key < see1[i] && key >= see1[i] - width ? z[i][e] : kNegInf;
                }
            }
            mx[i] = max8(z[i]);
            move = move || (mx[i] - M[i]) * cm[i] > kSlack || (M[i] == kNegInf && mx[i] > kNegInf);
        }
        page = next;
        if (c.good(page)) load_keys(page, step + 1);
        float vs[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) vs[e] = __uint_as_float(vsw.w[e]);
        if (edge) {                                // positions past the last key may hold anything
#pragma unroll
            for (int e = 0; e < 8; ++e) vs[e] = j0 + 8 * g + e < t.hi ? vs[e] : 0.f;
        }
        const float vmx = max8(vs);
        move = move || (vmx > vref && vmx <= kFltMax);
        if (__ballot(move)) {
            float vm = fmaxf(vmx, __shfl_xor(vmx, 16, kWave));
            vm = fmaxf(vm, __shfl_xor(vm, 32, kWave));
            float down = 1.f;
            if (vm > vref && vm <= kFltMax) {      // a power of two above every scale so far
                const float nr = pow2(min((int)(__float_as_uint(vm) >> 23) - 126, 126));
                down = vref / nr;
                vref = nr;
                vinv = 0x1p5f / nr;
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float m = fmaxf(mx[i], __shfl_xor(mx[i], 16, kWave));
                m = fmaxf(m, __shfl_xor(m, 32, kWave));
                const float Mn = fmaxf(M[i], m);
                const float f = M[i] == kNegInf ? 0.f : exp2f((M[i] - Mn) * cm[i]);
                L[i] *= f;
                M[i] = Mn;
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][h][j] = acc[i][h][j] * (f * down);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) vs[e] *= vinv;
        half8 ph[NT], pl[kPair ? NT : 1];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const float ref = M[i] == kNegInf ? 0.f : M[i] * cm[i];
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = __builtin_amdgcn_exp2f(fmaf(z[i][e], cm[i], -ref));
                L[i] += p;
                v[e] = p * vs[e];
            }
            if (edge) {                            // an unseen key's scale may be NaN
                asm volatile("");
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = z[i][e] == kNegInf ? 0.f : v[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (kPair) asm volatile("" : "+v"(v[e]));
                const _Float16 hv = (_Float16)v[e];
                ph[i][e] = hv;
                if (kPair) pl[i][e] = (_Float16)(v[e] - (float)hv);
            }
        }
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const half8 vf = codes_f16(vw[h].w[j]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[i][h][j] = mfma16(vf, ph[i], acc[i][h][j]);
                    if (kPair) acc[i][h][j] = mfma16(vf, pl[i], acc[i][h][j]);
                }
            }
    }

    // The four waves' parts under the common maximum, added in their order.
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        L[i] += __shfl_xor(L[i], 16, kWave);
        L[i] += __shfl_xor(L[i], 32, kWave);
        M[i] = M[i] == kNegInf ? kNegInf : M[i] * cm[i];
        if (L[i] != L[i]) M[i] = 0.f;              // NaN scores only: not an empty row
        if (g == 0) {
            sm[wave][16 * i + n] = M[i];
            sl[wave][16 * i + n] = L[i];
        }
    }
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
        if (wave == w) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float Mx = kNegInf;
#pragma unroll
                for (int k = 0; k < kWaves; ++k) Mx = fmaxf(Mx, sm[k][16 * i + n]);
                const float f = M[i] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(M[i] - Mx) * (vref * 0x1p-5f);
                // register r of the MFMA row 4*g + r is column 64*h + 4*(4*g + r) + j
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        f32x4* o = reinterpret_cast<f32x4*>(&so[16 * i + n][64 * h + 16 * g + 4 * r]);
                        f32x4 v = {acc[i][h][0][r] * f, acc[i][h][1][r] * f, acc[i][h][2][r] * f, acc[i][h][3][r] * f};
                        if (w > 0) v += *o;
                        *o = v;
                    }
            }
        }
        __syncthreads();
    }
    constexpr int kQ = D / 4;              // float4 columns
    for (int i = threadIdx.x; i < kRT * kQ; i += kThreads) {
        const int m = i / kQ, col = i % kQ * 4, row = t.r0 + m;
        if (row >= (splits > 1 ? rows : t.n * group)) break;
        float mm = kNegInf, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm[w][m]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            l += sm[w][m] == kNegInf ? 0.f : sl[w][m] * __builtin_amdgcn_exp2f(sm[w][m] - mm);
        f32x4 o = *reinterpret_cast<const f32x4*>(&so[m][col]);
        if (splits > 1) {
            float* part = reinterpret_cast<float*>(a.workspace) +
                          (((int64_t)slot * c.kv_heads + head) * splits + sp) * (kRT * (D + 2));
            *reinterpret_cast<f32x4*>(part + m * D + col) = o;
            if (col == 0) {
                part[kRT * D + m] = mm;
                part[kRT * D + kRT + m] = l;
            }
            continue;
        }
        // one split: the answer.  Rows outside the granted count give zeros.
        const bool empty = mm == kNegInf || row >= rows;
        const float inv = empty ? 0.f : 1.0f / l;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = empty ? 0.f : o[k] * inv;
        const int64_t at = (int64_t)(t.q0 + row / group);
        const int oh = head * group + row % group;
        store4<T>(reinterpret_cast<typename T::type*>(a.out) + at * a.ldo + (int64_t)oh * D + col, v);
        if (a.lse && col == 0) a.lse[at * a.heads + oh] = empty ? kNegInf : (mm + log2f(l)) * kLn2;
    }
}

// Joins the splits of a tile's rows: sum_s 2^(M_s - M) O_s.  A thread holds four
// columns.  With up to kFewSplits parts the workgroup's kG thread groups take a
// row each and all of its parts; with more they share a row, every kG-th part
// each, and LDS adds their sums in a fixed order.  `per` workgroups a tile.  All
// loads of a thread go out together: the launch is a few latencies long.
constexpr int kFewSplits = 8;

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_attention_join(Cache c, AttnArgs a, int splits, int rt, int per) {
    constexpr int kQ = D / 4, kG = kThreads / kQ;          // float4 columns, groups
    __shared__ f32x4 so[kG][kQ];
    __shared__ float sl[kG], sm[kG];
    const int j = blockIdx.x % per, head = blockIdx.x / per % c.kv_heads, slot = blockIdx.x / per / c.kv_heads;
    const int group = a.heads / c.kv_heads;
    const Tile t = find_tile(c, a, slot, splits, rt);
    if (!t.any) return;
    const int used = max((t.hi - t.lo + t.per - 1) / t.per, 1);
    const int64_t stride = (int64_t)rt * (D + 2);
    const float* parts = reinterpret_cast<const float*>(a.workspace) +
                         ((int64_t)slot * c.kv_heads + head) * splits * stride;
    const int q = threadIdx.x % kQ, k = threadIdx.x / kQ;
    const int end = min(rt, t.n * group - t.r0), live = t.m * group - t.r0;      // rows to write, rows that count
    auto put = [&](int m, const f32x4& o, float mm, float l) {
        const int row = t.r0 + m;
        const bool empty = m >= live || mm == kNegInf;
        const float inv = empty ? 0.f : 1.0f / l;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = empty ? 0.f : o[i] * inv;
        const int64_t at = (int64_t)(t.q0 + row / group);
        const int oh = head * group + row % group;
        store4<T>(reinterpret_cast<typename T::type*>(a.out) + at * a.ldo + (int64_t)oh * D + 4 * q, v);
        if (a.lse && q == 0) a.lse[at * a.heads + oh] = empty ? kNegInf : (mm + log2f(l)) * kLn2;
    };
    // up to kFewSplits parts first, first + step, ... of row m: their sum under their
    // own maximum mm (a part without a key has M = -inf, L = 0, O = 0)
    auto gather = [&](int m, int first, int step, f32x4& o, float& l, float& mm) {
        float ms[kFewSplits], ls[kFewSplits];
        f32x4 v[kFewSplits];
#pragma unroll
        for (int i = 0; i < kFewSplits; ++i) {
            const float* p = parts + min(first + i * step, used - 1) * stride;
            ms[i] = p[rt * D + m];
            ls[i] = p[rt * D + rt + m];
            v[i] = *reinterpret_cast<const f32x4*>(p + m * D + 4 * q);
        }
        float top = mm;
#pragma unroll
        for (int i = 0; i < kFewSplits; ++i) top = first + i * step < used ? fmaxf(top, ms[i]) : top;
        const float ref = top == kNegInf ? 0.f : top, f0 = mm == kNegInf ? 0.f : __builtin_amdgcn_exp2f(mm - ref);
        o = o * f0;
        l *= f0;
#pragma unroll
        for (int i = 0; i < kFewSplits; ++i) {
            if (first + i * step >= used) break;
            const float f = __builtin_amdgcn_exp2f(ms[i] - ref);
            l += ls[i] * f;
            o += v[i] * f;
        }
        mm = top;
    };
    if (used <= kFewSplits) {
        if (k >= kG) return;
        for (int m = j * kG + k; m < end; m += per * kG) {
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
            float l = 0.f, mm = kNegInf;
            if (m < live) gather(m, 0, 1, o, l, mm);
            put(m, o, mm, l);
        }
        return;
    }
    for (int m = j; m < end; m += per) {                   // the whole workgroup, row by row
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        float l = 0.f, mm = kNegInf;
        if (m < live && k < kG)
            for (int s = k; s < used; s += kG * kFewSplits) gather(m, s, kG, o, l, mm);
        __syncthreads();                                   // the last row's sums are read
        if (k < kG) {
            so[k][q] = o;
            if (q == 0) {
                sl[k] = l;
                sm[k] = mm;
            }
        }
        __syncthreads();
        if (threadIdx.x < kQ) {
            float top = kNegInf;
#pragma unroll
            for (int i = 0; i < kG; ++i) top = fmaxf(top, sm[i]);
            o = f32x4{0.f, 0.f, 0.f, 0.f};
            l = 0.f;
            const float ref = top == kNegInf ? 0.f : top;
#pragma unroll
            for (int i = 0; i < kG; ++i) {
                const float f = __builtin_amdgcn_exp2f(sm[i] - ref);
                o += so[i][q] * f;
                l += sl[i] * f;
            }
            put(m, o, top, l);
        }
    }
}

// How a call is cut: 16-row blocks of a workgroup by the rows a sequence has on
// average (prompts: three at head_dim 128, where four spilled registers, 614
// against 587 us for 2813 queries of 48 heads over up to 6000 keys, now 530, and two
// elsewhere: at 64 two took 64 us for 3 x 1000 queries of 8 heads over 3000 keys,
// three 70), and splits of the keys: enough workgroups for four
// on every compute unit if the splits keep kMinChunk keys, and four times as many,
// which evens out ragged lengths, if they keep eight times that.  Up to kNoSplit keys
// the second launch would cost more than it saves.
struct Cut {
    int nt, splits, joins;
    int64_t slots;
};
Cut cut_of(const Cache& c, int rows, int heads, int64_t max_len) {
    Cut k;
    const int64_t group = heads / c.kv_heads, total = rows * group;
    const int64_t mean = total / c.n_seqs;
    k.nt = mean <= 16 ? 1 : mean <= 32 || c.head_dim != 128 ? 2 : 3;
    const int rt = 16 * k.nt;
    k.slots = total / rt + c.n_seqs;                       // a sequence of n rows owns at least ceil(n / rt)
    const int64_t busy = (total + rt - 1) / rt;
    const int64_t tiles = busy > c.n_seqs ? busy : rows < c.n_seqs ? rows : c.n_seqs;
    const int64_t base = (tiles < 1 ? 1 : tiles) * c.kv_heads;
    auto pieces = [&](int64_t want, int64_t chunk) {
        const int64_t s = (want + base - 1) / base, most = (max_len + chunk - 1) / chunk;
        return s < most ? s : most;
    };
    int64_t s = max_len <= kNoSplit ? 1 : pieces(1024, kMinChunk);
    const int64_t fine = pieces(4096, 8 * kMinChunk);
    if (fine > s && mean <= 32) s = fine;
    k.splits = (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
    // a workgroup a row where it shares the row's many parts, else one a few rows
    k.joins = k.splits > kFewSplits ? rt : k.nt;
    return k;
}

template <typename T, int D, int NT>
void launch_tile(const Cache& c, const AttnArgs& a, const Cut& k, hipStream_t st) {
    hipLaunchKernelGGL((kv4_attention_kernel<T, D, NT>), dim3((unsigned)(k.slots * c.kv_heads * k.splits)),
                       dim3(kThreads), 0, st, c, a, k.splits);
}

template <typename T, int D>
hipError_t launch_dim(const Cache& c, const AttnArgs& a, hipStream_t st) {
    const Cut k = cut_of(c, a.rows, a.heads, a.max_len);
    if (k.nt == 1) launch_tile<T, D, 1>(c, a, k, st);
    else if (k.nt == 2) launch_tile<T, D, 2>(c, a, k, st);
    else if constexpr (D == 128) launch_tile<T, D, 3>(c, a, k, st);
    if (k.splits > 1)
        hipLaunchKernelGGL((kv4_attention_join<T, D>), dim3((unsigned)(k.slots * c.kv_heads * k.joins)), dim3(kThreads),
                           0, st, c, a, k.splits, 16 * k.nt, k.joins);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_type(const Cache& c, const AttnArgs& a, hipStream_t st) {
    switch (c.head_dim) {
        case 64: return launch_dim<T, 64>(c, a, st);
        case 128: return launch_dim<T, 128>(c, a, st);
        case 192: return launch_dim<T, 192>(c, a, st);
        case 256: return launch_dim<T, 256>(c, a, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

int64_t attention_workspace(const Cache& c, int rows, int heads, int64_t max_len) {
    const Cut k = cut_of(c, rows, heads, max_len);
    if (k.splits == 1 || rows == 0) return 0;
    return k.slots * c.kv_heads * k.splits * (16 * k.nt) * (c.head_dim + 2) * 4;
}

int64_t attention_grid(const Cache& c, int rows, int heads, int64_t max_len) {
    const Cut k = cut_of(c, rows, heads, max_len);
    return k.slots * c.kv_heads * (k.splits > k.joins ? k.splits : k.joins);
}

hipError_t launch_attention(const Cache& c, const AttnArgs& a, int dtype, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    switch (dtype) {
        case MOEDEC_F32: return launch_type<F32>(c, a, st);
        case MOEDEC_F16: return launch_type<F16>(c, a, st);
        case MOEDEC_BF16: return launch_type<BF16>(c, a, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace attn
}  // namespace moedec
