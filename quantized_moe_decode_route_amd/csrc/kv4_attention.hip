// Attention over the paged 4-bit cache.
//
//   S[j][m] = q_m . k_j = s_k[j] * sum_c code_k[j][c] * q_m[c]
//   p = exp2(S * scale * log2 e - M_m),  O[m] = sum_j (p * s_v[j]) * code_v[j] / sum_j p
//
// The row scales factor out of both products, so the matrix cores work on the
// codes themselves, which are exact in fp16.  A row m is one query head of one
// token; 16 rows that share a key/value head are the N side of the products
// (B operand), 32 keys at a time the M side of S^T = K Q^T and the K side of
// O^T = V^T P^T.  In S^T a lane holds one row (lane % 16) and, with the tokens
// of a 32-key tile given to the two 16-key MFMAs as 8*(r/4) + 4*t + r%4, keys
// 8*(lane/16) .. +7: exactly the K-values its B operand of the second product
// needs.  So probabilities never leave their lane, and the running maximum, the
// sum and the rescaling of the accumulators are per-lane scalars.
//
// Queries enter as fp16 under one power of two per row: exact for fp16 and bf16,
// as a hi/lo pair (22 bits) for fp32.  The probabilities times their value scale
// enter the second product as fp16 (fp32: again as a pair) under one power of two
// per wave that follows the largest value scale seen.  For 16-bit activations the
// rounding of a probability to fp16 (2^-12 relative) is below that of the output.
// Scores, maxima, sums and accumulators are fp32.
#include "attn.h"

namespace moedec {
namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kRows = 16;                 // rows (query heads of tokens) of a tile
constexpr int kKeys = 32;                 // keys of a wave's step
constexpr int kMinChunk = 256;            // keys of a split at least
constexpr int kMaxSplits = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ floatx4 mfma16(const half8& a, const half8& b, const floatx4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 2^k as a float, k in [-126, 127].
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// Exponent k with m * 2^k in [2^14, 2^15) (0 for zero and non-finite m).
__device__ __forceinline__ int row_exponent(float m) {
    if (!(m > 0.f) || !(m <= 3.402823466e38f)) return 0;
    const int e = (int)(__float_as_uint(m) >> 23) - 127;        // -127 for subnormals
    const int k = 14 - e;
    return k > 120 ? 120 : k;
}

// A row tile: rows [r0, r0 + 16) of sequence s's m * group rows (row = token *
// group + head of the group), and the keys [lo, hi) that any of them sees.
struct Tile {
    int s, q0, m, len, r0, lo, hi, per;
    bool any;
};

__device__ __forceinline__ Tile find_tile(const Cache& c, const AttnArgs& a, int slot, int splits) {
    Tile t;
    const int group = a.heads / c.kv_heads;
    t.s = seq_of_slot(a.q_start, c.n_seqs, a.rows, group, kRows, 1, slot);
    const Span q = span_of(a.q_start, t.s, a.rows);
    t.q0 = q.q0;
    const int n = q.q1 - q.q0;
    t.m = a.granted ? min(n, max(a.granted[t.s], 0)) : n;
    t.len = c.held(t.s);
    t.r0 = (slot - slot_base(a.q_start, t.s, a.rows, group, kRows, 1)) * kRows;
    t.any = t.r0 < n * group;
    const int first = t.len - t.m + t.r0 / group;                            // position of the first row
    const int last = t.len - t.m + min(t.r0 + kRows - 1, t.m * group - 1) / group;
    t.hi = t.r0 < t.m * group ? max(last + 1, 0) : 0;
    t.lo = a.window > 0 ? max(first - a.window + 1, 0) & ~(kKeys - 1) : 0;
    if (t.hi < t.lo) t.hi = t.lo;
    const int each = (t.hi - t.lo + splits - 1) / splits;
    t.per = max(kMinChunk, (each + kKeys * kWaves - 1) / (kKeys * kWaves) * (kKeys * kWaves));
    return t;
}

// One split of one tile of one key/value head.
template <typename T, int D, bool kPair>
__global__ __launch_bounds__(kThreads) void kv4_attention_kernel(Cache c, AttnArgs a, int splits) {
    constexpr int kS = D / 32;            // MFMAs of a score, K side
    constexpr int kH = D / 64;            // 64-column parts of the output
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, g = lane >> 4;
    const int sp = blockIdx.x % splits, head = (blockIdx.x / splits) % c.kv_heads;
    const int slot = blockIdx.x / splits / c.kv_heads;
    const int group = a.heads / c.kv_heads;
    const Tile t = find_tile(c, a, slot, splits);
    if (!t.any) return;
    const int k0 = t.lo + sp * t.per, k1 = min(t.hi, k0 + t.per);
    if (sp > 0 && k0 >= t.hi) return;

    // this lane's row, its position and the keys it sees
    const int row = t.r0 + n, tok = row / group;
    const bool on = row < t.m * group;
    const int pos = t.len - t.m + tok;
    const int see1 = on ? pos + 1 : 0, see0 = a.window > 0 ? pos - a.window + 1 : 0;
    const int64_t r_at = (int64_t)(t.q0 + tok);
    const int qh = head * group + row % group;

    half8 qhi[kS], qlo[kPair ? kS : 1];
    float cm;                              // score (codes times q in fp16) -> log2 domain
    {
        float x[kS][8];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[s][e] = 0.f;
            if (on)
                load8<T>(reinterpret_cast<const typename T::type*>(a.q) + r_at * a.ldq + (int64_t)qh * D + 32 * s + 8 * g,
                         x[s]);
        }
        float m = 0.f;
#pragma unroll
        for (int s = 0; s < kS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[s][e]));
        m = fmaxf(m, __shfl_xor(m, 16, kWave));
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        const int k = row_exponent(m);
        const float f = pow2(k);
#pragma unroll
        for (int s = 0; s < kS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = x[s][e] * f;
                asm volatile("" : "+v"(v));
                const _Float16 h = (_Float16)v;
                qhi[s][e] = h;
                if (kPair) qlo[s][e] = (_Float16)(v - (float)h);
            }
        cm = pow2(-k) * a.scale * kLog2e;
    }

    floatx4 acc[kH][4];
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[h][i] = floatx4{0.f, 0.f, 0.f, 0.f};
    float M = kNegInf, L = 0.f;
    float vref = 0x1p-100f, vinv = 0x1p105f;       // value scales enter as s_v * vinv <= 2^6, vinv = 2^5 / vref

    const int pt = c.page_tokens();
    const int32_t* row_pages = c.table + (int64_t)t.s * c.max_pages;
    for (int j0 = k0 + wave * kKeys; j0 < k1; j0 += kWaves * kKeys) {
        const int page = row_pages[j0 >> c.pt_log2];
        if (!c.good(page)) continue;
        const uint8_t* unit = c.unit(a.layer, page, head);
        const int at = j0 & (pt - 1);
        uint32_t kw[2][kS], vw[kH][4];
        float ks[8], vs[8];
#pragma unroll
        for (int tl = 0; tl < 2; ++tl) {
            const int kt = at + 8 * (n >> 2) + 4 * tl + (n & 3);
            const uint32_t* p = reinterpret_cast<const uint32_t*>(unit) + kt * (D / 8) + g * kS;
#pragma unroll
            for (int s = 0; s < kS; ++s) kw[tl][s] = p[s];
        }
        const uint32_t* vp = reinterpret_cast<const uint32_t*>(unit + (int64_t)pt * (D / 2)) + ((at >> 3) + g) * D + 4 * n;
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) vw[h][i] = vp[64 * h + i];
        const float* ksp = reinterpret_cast<const float*>(unit + (int64_t)pt * D) + at + 8 * g;
        const float* vsp = ksp + pt;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ks[e] = ksp[e];
            vs[e] = vsp[e];
        }

        floatx4 sc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                const half8 kf = codes_f16(kw[tl][s]);
                sc[tl] = mfma16(kf, qhi[s], sc[tl]);
                if (kPair) sc[tl] = mfma16(kf, qlo[s], sc[tl]);
            }
        // scores of keys j0 + 8*g + e in the log2 domain; unseen keys are -inf
        float z[8], mx = kNegInf, vmx = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int key = j0 + 8 * g + e;
            const bool seen = key < see1 && key >= see0;
            z[e] = seen ? sc[e >> 2][e & 3] * ks[e] * cm : kNegInf;
            mx = fmaxf(mx, z[e]);
            if (key < t.hi) vmx = fmaxf(vmx, vs[e]);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
        mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
        vmx = fmaxf(vmx, __shfl_xor(vmx, 16, kWave));
        vmx = fmaxf(vmx, __shfl_xor(vmx, 32, kWave));
        const float Mn = fmaxf(M, mx);
        const float base = Mn == kNegInf ? 0.f : Mn;
        float f = M == kNegInf ? 0.f : exp2f(M - base);
        L *= f;
        if (vmx > vref && vmx <= 3.402823466e38f) {       // a power of two at least as large as every scale so far
            const float nr = pow2(min((int)(__float_as_uint(vmx) >> 23) - 126, 126));
            f *= vref / nr;
            vref = nr;
            vinv = 0x1p5f / nr;
        }
        M = Mn;
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][i] = acc[h][i] * f;
        half8 phi, plo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float p = exp2f(z[e] - base);
            L += p;
            float v = p > 0.f || p != p ? p * (vs[e] * vinv) : 0.f;     // an unseen key's scale may be anything
            asm volatile("" : "+v"(v));
            const _Float16 hv = (_Float16)v;
            phi[e] = hv;
            if (kPair) plo[e] = (_Float16)(v - (float)hv);
        }
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const half8 vf = codes_f16(vw[h][i]);
                acc[h][i] = mfma16(vf, phi, acc[h][i]);
                if (kPair) acc[h][i] = mfma16(vf, plo, acc[h][i]);
            }
    }
    L += __shfl_xor(L, 16, kWave);
    L += __shfl_xor(L, 32, kWave);
    if (L != L) M = 0.f;                   // NaN scores only: not an empty row

    // The four waves' parts under the common maximum: each wave's sum of the
    // output lands in LDS, wave 0 .. 3 added in that order.
    __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];
    __shared__ float so[kWaves][kRows][D + 4];
    if (g == 0) {
        sm[wave][n] = M;
        sl[wave][n] = L;
    }
    __syncthreads();
    float Mx = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) Mx = fmaxf(Mx, sm[w][n]);
    const float f = M == kNegInf ? 0.f : exp2f(M - Mx) * (vref * 0x1p-5f);
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // register i of the MFMA's row 4*g + i' is column 64*h + 4*(4*g + i') + i
#pragma unroll
            for (int r = 0; r < 4; ++r) so[wave][n][64 * h + 16 * g + 4 * r + i] = acc[h][i][r] * f;
        }
    __syncthreads();
    float* wsf = reinterpret_cast<float*>(a.workspace);
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
        const int m = i / (D / 4), col = i % (D / 4) * 4;
        const int mrow = t.r0 + m;
        if (splits > 1 && mrow >= t.m * group) continue;
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        float mm = kNegInf, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm[w][m]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            l += sm[w][m] == kNegInf ? 0.f : sl[w][m] * exp2f(sm[w][m] - mm);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] += so[w][m][col + k];
        }
        if (splits > 1) {
            const int64_t part = ((int64_t)slot * c.kv_heads + head) * splits + sp;
            float* base = wsf + part * (kRows * (D + 2));
#pragma unroll
            for (int k = 0; k < 4; ++k) base[m * D + col + k] = o[k];
            if (col == 0) {
                base[kRows * D + m] = mm;
                base[kRows * D + kRows + m] = l;
            }
            continue;
        }
        // one split: the answer.  Rows outside the granted count give zeros.
        const Span q = span_of(a.q_start, t.s, a.rows);
        const int tk = mrow / group;
        if (tk >= q.q1 - q.q0) continue;
        const float inv = mm == kNegInf || mrow >= t.m * group ? 0.f : 1.0f / l;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = inv == 0.f ? 0.f : o[k] * inv;
        const int64_t at = (int64_t)(t.q0 + tk);
        const int oh = head * group + mrow % group;
        store4<T>(reinterpret_cast<typename T::type*>(a.out) + at * a.ldo + (int64_t)oh * D + col, o);
        if (a.lse && col == 0) a.lse[at * a.heads + oh] = inv == 0.f ? kNegInf : mm * kLn2 + logf(l);
    }
}

// Joins the splits of one tile of one key/value head: sum_s 2^(M_s - M) O_s.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_attention_join(Cache c, AttnArgs a, int splits) {
    const int head = blockIdx.x % c.kv_heads, slot = blockIdx.x / c.kv_heads;
    const int group = a.heads / c.kv_heads;
    const Tile t = find_tile(c, a, slot, splits);
    if (!t.any) return;
    const Span q = span_of(a.q_start, t.s, a.rows);
    const int used = max((t.hi - t.lo + t.per - 1) / t.per, 1);
    const float* parts = reinterpret_cast<const float*>(a.workspace) +
                         ((int64_t)slot * c.kv_heads + head) * splits * (kRows * (D + 2));
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
        const int m = i / (D / 4), col = i % (D / 4) * 4, mrow = t.r0 + m, tk = mrow / group;
        if (tk >= q.q1 - q.q0) continue;
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        float mm = kNegInf, l = 0.f;
        const bool on = mrow < t.m * group;
        if (on) {
            for (int s = 0; s < used; ++s) mm = fmaxf(mm, parts[(int64_t)s * kRows * (D + 2) + kRows * D + m]);
            for (int s = 0; s < used; ++s) {
                const float* p = parts + (int64_t)s * kRows * (D + 2);
                const float ms = p[kRows * D + m];
                const float f = ms == kNegInf ? 0.f : exp2f(ms - mm);
                l += ms == kNegInf ? 0.f : p[kRows * D + kRows + m] * f;
                const f32x4 v = *reinterpret_cast<const f32x4*>(p + m * D + col);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] += ms == kNegInf ? 0.f : v[k] * f;
            }
        }
        const bool empty = !on || mm == kNegInf;
        const float inv = empty ? 0.f : 1.0f / l;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = empty ? 0.f : o[k] * inv;
        const int64_t at = (int64_t)(t.q0 + tk);
        const int oh = head * group + mrow % group;
        store4<T>(reinterpret_cast<typename T::type*>(a.out) + at * a.ldo + (int64_t)oh * D + col, o);
        if (a.lse && col == 0) a.lse[at * a.heads + oh] = empty ? kNegInf : mm * kLn2 + logf(l);
    }
}

// Row tiles of a launch at most: a sequence of n rows owns floor-difference + 1 slots.
int64_t tile_slots(const Cache& c, int rows, int heads) {
    return (int64_t)rows * (heads / c.kv_heads) / kRows + c.n_seqs;
}

// Splits of the keys: enough workgroups for two on every compute unit, none
// shorter than kMinChunk keys.
int split_count(const Cache& c, int rows, int heads, int64_t max_len) {
    const int64_t base = (int64_t)rows * (heads / c.kv_heads) / kRows * c.kv_heads + c.kv_heads;
    int64_t s = (4 * 256 + base - 1) / base;
    const int64_t most = (max_len + kMinChunk - 1) / kMinChunk;
    if (s > most) s = most;
    return (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

template <typename T, int D>
hipError_t launch_dim(const Cache& c, const AttnArgs& a, hipStream_t st) {
    const int splits = split_count(c, a.rows, a.heads, a.max_len);
    const int64_t tiles = tile_slots(c, a.rows, a.heads) * c.kv_heads;
    hipLaunchKernelGGL((kv4_attention_kernel<T, D, T::bytes == 4>), dim3((unsigned)(tiles * splits)), dim3(kThreads), 0,
                       st, c, a, splits);
    if (splits > 1)
        hipLaunchKernelGGL((kv4_attention_join<T, D>), dim3((unsigned)tiles), dim3(kThreads), 0, st, c, a, splits);
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
    const int splits = split_count(c, rows, heads, max_len);
    if (splits == 1 || rows == 0) return 0;
    return tile_slots(c, rows, heads) * c.kv_heads * splits * kRows * (c.head_dim + 2) * 4;
}

int64_t attention_grid(const Cache& c, int rows, int heads, int64_t max_len) {
    return tile_slots(c, rows, heads) * c.kv_heads * split_count(c, rows, heads, max_len);
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
