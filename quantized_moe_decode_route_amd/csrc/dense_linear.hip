// y = act(scale * (x . codes) + bias) + residual on packed row-scaled weights.
//
// Codes.  Beside 16-bit activations a code q of b bits enters as the unsigned u =
// q + 2^(b-1), isolated with its sign bit flipped by one bit operation and left
// where it stands in the low byte of its 16-bit half (2 bits: 3 bits higher): read
// as fp16 that is u * 2^j * 2^-24, j its bit position, exactly, subnormal or just
// above.  The 2^j is taken out of the activation that meets it, 2^24 out of the
// sum, and the offset out of the start of the sum,
//   sum x q = -2^(b-1) sum x + sum x u,
// with sum x over the activations as they enter.  Converting 8 codes of 4 bits then
// costs 5 vector instructions instead of 9, of 8 bits 6 instead of 10, of 2 bits
// 5 instead of 12.  (int4, bf16, 6144 -> 8192: 1024 tokens 136 us, 146 with signed
// codes, 4096 tokens 426 / 449.)  It costs bits of the sum: the matrix core aligns
// products by their operands' exponent fields, so a subnormal's leading zeros are
// lost below the largest product.  Measured against 64 bits, relative to the
// result's rms: 1e-5 for 4 bits at K = 6144, where an fp16 result rounds by 2e-4 and
// a bf16 one by 1.7e-3 (2 bits left in place: 3.3e-5, hence the 3 bits), but an
// fp32 result by 2.5e-8.  fp32 keeps signed codes, whose sums are within 2e-7.
//
// Activations.  Every fp16 or bf16 activation is exact in fp16, up to the exponent
// range, once its row is scaled by a power of two that brings the largest
// magnitude to [2^14, 2^15): the products on v_mfma_f32_16x16x32_f16 are then
// exact and only the fp32 sums round.  fp32 activations enter as a hi/lo pair of
// fp16 (about 22 bits), two MFMAs instead of one.  The power of two, the row scale,
// bias, activation and residual are applied once, in fp32, to the sums.
//
// Weight rows are the M side (A operand: lane l holds row l % 16), tokens the N
// side.  A wave turns the packed codes into fp16 in its own registers: at 2 to 8
// bits they are a small fraction of the bytes, so they go from global memory
// straight to the lanes and only the activations pass through LDS.
#include "attn.h"
#include "mfma.h"

namespace moedec {
namespace attn {

namespace {

using mfma::MfmaCodec;

// Codes of a 32-bit word as unsigned fields of fp16 patterns (see above): the
// fields `mask` selects of both halves, their sign bits `flip` inverted.
__device__ __forceinline__ uint32_t fields(uint32_t w, uint32_t mask, uint32_t flip) { return (w & mask) ^ flip; }

// Whether codes enter as unsigned fields, for elements of that many bytes.
constexpr bool offset_codes(int bytes) { return bytes == 2; }
// The lowest bit position of a field in its half.
constexpr int field_base(int bits) { return bits == 2 ? 3 : 0; }

// Operand of call c of a 16-byte group of codes, in the element order of
// MfmaCodec: element e holds u * 2^(field_base + field_bit(e)) * 2^-24 (kOffset)
// or q.
template <int BITS, bool kOffset>
__device__ __forceinline__ half8 a_operand(const uint4& q, int c) {
    if constexpr (!kOffset) {
        if constexpr (BITS == 4) return codes_f16(mfma::dword(q, c));
        else return mfma::a_operand<BITS>(q, c);
    }
    u32x4 p;
    if constexpr (BITS == 4) {
        const uint32_t w = mfma::dword(q, c), h = w >> 8;
        p = u32x4{fields(w, 0x000F000Fu, 0x00080008u), fields(w, 0x00F000F0u, 0x00800080u),
                  fields(h, 0x000F000Fu, 0x00080008u), fields(h, 0x00F000F0u, 0x00800080u)};
    } else if constexpr (BITS == 8) {
        const uint32_t w0 = mfma::dword(q, 2 * c), w1 = mfma::dword(q, 2 * c + 1);
        p = u32x4{fields(w0, 0x00FF00FFu, 0x00800080u), fields(w0 >> 8, 0x00FF00FFu, 0x00800080u),
                  fields(w1, 0x00FF00FFu, 0x00800080u), fields(w1 >> 8, 0x00FF00FFu, 0x00800080u)};
    } else {
        const uint32_t d = mfma::dword(q, c >> 1), w = c & 1 ? d >> 5 : d << 3;
        p = u32x4{fields(w, 0x00180018u, 0x00100010u), fields(w, 0x00600060u, 0x00400040u),
                  fields(w, 0x01800180u, 0x01000100u), fields(w, 0x06000600u, 0x04000400u)};
    }
    return __builtin_bit_cast(half8, p);
}
// Bit position of element e's field above the lowest.
template <int BITS, bool kOffset>
__device__ __forceinline__ constexpr int field_bit(int e) {
    return !kOffset ? 0 : BITS == 4 ? 4 * ((e >> 1) & 1) : BITS == 2 ? 2 * (e >> 1) : 0;
}
// The offset as an operand: u = -2^(BITS-1) in every element.
template <int BITS>
__device__ __forceinline__ half8 minus_offset() {
    constexpr uint32_t sign = 0x80008000u;
    u32x4 p;
    if constexpr (BITS == 4) p = u32x4{0x00080008u | sign, 0x00800080u | sign, 0x00080008u | sign, 0x00800080u | sign};
    else if constexpr (BITS == 8)
        p = u32x4{0x00800080u | sign, 0x00800080u | sign, 0x00800080u | sign, 0x00800080u | sign};
    else p = u32x4{0x00100010u | sign, 0x00400040u | sign, 0x01000100u | sign, 0x04000400u | sign};
    return __builtin_bit_cast(half8, p);
}

constexpr int kPrepThreads = 256;
constexpr int kStage = 4;                 // MFMA calls (of 32 columns) of a staged step
constexpr float kFltMax = 3.402823466e38f;

__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// Exponent k with m * 2^k in [2^14, 2^15) (0 for zero and non-finite m).
__device__ __forceinline__ int row_exponent(float m) {
    if (!(m > 0.f) || !(m <= kFltMax)) return 0;
    const int k = 14 - ((int)(__float_as_uint(m) >> 23) - 127);
    return k > 120 ? 120 : k;
}

// Columns a plane's row is padded to: whole 64-byte chunks of codes (4 groups of
// 16 bytes, one per lane of a row) and whole staged steps.
__host__ __device__ constexpr int pad_of(int bits) { return bits == 2 ? 256 : 128; }
__host__ __device__ inline int64_t padded(int64_t K, int bits) {
    return (K + pad_of(bits) - 1) / pad_of(bits) * pad_of(bits);
}
__host__ __device__ inline int64_t blocks16(int64_t T) { return (T + 15) / 16; }

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case MOEDEC_ACT_SILU: return v / (1.0f + expf(-v));
        case MOEDEC_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
        case MOEDEC_ACT_RELU: return v < 0.f ? 0.f : v;
        default: return v;
    }
}

// Row scale and bias of four consecutive rows r .. r+3, loaded ahead of the sums.
struct Params {
    float scale[4], bias[4];
};
__device__ __forceinline__ Params load_params(const LinearArgs& a, int r) {
    Params p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = min(r + i, a.N - 1);
        p.scale[i] = a.scale[n];
        p.bias[i] = a.bias ? a.bias[n] : 0.f;
    }
    return p;
}

// Four consecutive elements at any element's alignment (one load or store: the
// memory system takes them from any address).
template <typename T>
struct Four {
    typedef typename T::type type __attribute__((ext_vector_type(4), aligned(T::bytes)));
};

// The epilogue of rows r .. r+3 of token t.
template <typename T, int BITS>
__device__ __forceinline__ void finish4(const LinearArgs& a, int t, int r, float inv, const floatx4& sum,
                                        const Params& p) {
    if (r >= a.N) return;
    constexpr bool kOffset = offset_codes(T::bytes);
    constexpr float unit = (float)(1 << (24 - field_base(BITS)));
    typedef typename Four<T>::type four;
    typename T::type* y = reinterpret_cast<typename T::type*>(a.y) + (int64_t)t * a.ldy + r;
    const typename T::type* res = reinterpret_cast<const typename T::type*>(a.residual) + (int64_t)t * a.ldr + r;
    const bool whole = r + 3 < a.N;
    four old = {};
    if (a.residual && whole) old = *reinterpret_cast<const four*>(res);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = sum[i] * (kOffset ? unit : 1.f) * inv * p.scale[i] + p.bias[i];
    if (a.act != MOEDEC_ACT_NONE) {                // uniform
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(v[i], a.act);
    }
    if (whole) {
        four o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = T::put(a.residual ? v[i] + T::get(old[i]) : v[i]);
        *reinterpret_cast<four*>(y) = o;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (r + i >= a.N) break;
        if (a.residual) v[i] += T::get(res[i]);
        y[i] = T::put(v[i]);
    }
}

// ---------------------------------------------------------- units of a row
//
// A unit is the 8 columns that one lane group (0 .. 3) supplies to one call: two
// pieces of 4 consecutive columns, interleaved as a_operand orders the codes.

template <typename T>
__device__ __forceinline__ void load4(const typename T::type* p, float* o) {
    if constexpr (T::bytes == 4) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a[i];
    } else {
        typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
        const u16x4 a = *reinterpret_cast<const u16x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = T::get(__builtin_bit_cast(typename T::type, (uint16_t)a[i]));
    }
}

// First columns of the two pieces of unit u = call * 4 + group.  K is a multiple
// of a 16-byte group's columns, so a unit lies inside the row or past its end.
template <int BITS>
__device__ __forceinline__ void unit_cols(int u, int& c0, int& c1) {
    using M = MfmaCodec<BITS>;
    const int q = u >> 2, c = q % M::NCALL, col0 = (q / M::NCALL * 4 + (u & 3)) * (128 / BITS);
    c0 = col0 + M::col(c, 0);
    c1 = c0 + (BITS == 2 ? 8 : 4);
}
template <typename T, int BITS>
__device__ __forceinline__ void load_unit(const typename T::type* row, int K, int u, float* v) {
    int c0, c1;
    unit_cols<BITS>(u, c0, c1);
    if (c0 < K) {
        load4<T>(row + c0, v);
        load4<T>(row + c1, v + 4);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
}
// Piece element of operand element e.
template <int BITS>
__device__ __forceinline__ constexpr int unit_element(int e) {
    return BITS == 8 ? 4 * (e >> 2) + ((e >> 1) & 1) + 2 * (e & 1) : (e >> 1) + 4 * (e & 1);
}
// The unit's operands: element e times f * 2^-field_bit(e), as a pair.
template <int BITS, bool kOffset>
__device__ __forceinline__ void split_unit(const float* v, float f, half8& hi, half8& lo) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const mfma::F16Pair p = mfma::split_f16(v[unit_element<BITS>(e)], f * (1.0f / (1 << field_bit<BITS, kOffset>(e))));
        hi[e] = p.hi;
        lo[e] = p.lo;
    }
}
// The sum of a unit's operands, their field positions taken out.
template <int BITS, bool kPair>
__device__ __forceinline__ float unit_sum(const half8& hi, const half8& lo) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += ((float)hi[e] + (kPair ? (float)lo[e] : 0.f)) * (float)(1 << field_bit<BITS, true>(e));
    return s;
}

__device__ __forceinline__ float max8(const float* v, float m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
    return m;
}

// ------------------------------------------------------- activations as planes

// A plane holds fp16 activations in the order the B operand of the MFMAs takes
// them: [16 tokens][call of 32 columns][lane][8], 1 KB a call, so every later
// load of it is linear.  Call q of chunk c multiplies the columns that a_operand
// gives for call q of a 16-byte group of codes.
//
// WPT waves a token.  Rows of up to 512 * WPT * NU columns stay in registers
// between the pass for the largest magnitude and the conversion (NU = 0: read
// twice).  HBM-bound for many tokens (x read once, the planes written once; the 16
// bytes a lane stores meet those of the block's other tokens in the L2 of one
// XCD), a few microseconds of latency for few: those take four waves a token.
struct Row {
    float inv;                           // 1 / the row's power of two
    float start;                         // of the sum: -2^(BITS-1) * 2^(field_base-24) times the sum of the row, or 0
};

template <typename T, int BITS, int NU, int WPT>
__global__ __launch_bounds__(kPrepThreads) void linear_prepare(const typename T::type* __restrict__ x, int64_t ldx,
                                                               int T_, int K, int calls, half8* __restrict__ hi,
                                                               half8* __restrict__ lo, Row* __restrict__ info) {
    constexpr int kPer = kPrepThreads / kWave / WPT;       // tokens of a workgroup
    constexpr int kParts = 16 / kPer;                      // workgroups of a block of 16 tokens: all on one XCD
    constexpr int kLanes = WPT * kWave;
    constexpr bool kOffset = offset_codes(T::bytes);
    __shared__ float red[kPrepThreads / kWave];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), j = threadIdx.x % kLanes;
    const int xcd = blockIdx.x % 8, i8 = blockIdx.x / 8;
    const int64_t block = (int64_t)(i8 / kParts) * 8 + xcd;
    const int n = i8 % kParts * kPer + wave / WPT;
    const int64_t t = block * 16 + n;
    if (block * 16 >= T_) return;
    const bool on = t < T_;
    const typename T::type* row = x + (on ? t : 0) * ldx;
    const int units = calls * 4, cols = on ? K : 0;
    float sum = 0.f;
    auto put = [&](int u, const float* v, float f) {
        half8 h, l;
        split_unit<BITS, kOffset>(v, f, h, l);
        if (kOffset) sum += unit_sum<BITS, T::bytes == 4>(h, l);
        const int64_t at = (block * calls + (u >> 2)) * kWave + (u & 3) * 16 + n;
        hi[at] = h;
        if (T::bytes == 4) lo[at] = l;
    };
    auto row_max = [&](float m) {
        m = wave_max(m);
        if constexpr (WPT == 1) return m;
        if ((threadIdx.x & (kWave - 1)) == 0) red[wave] = m;
        __syncthreads();
        return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    };
    float m = 0.f;
    if constexpr (NU > 0) {
        float v[NU][8];
#pragma unroll
        for (int i = 0; i < NU; ++i) load_unit<T, BITS>(row, j + i * kLanes < units ? cols : 0, j + i * kLanes, v[i]);
#pragma unroll
        for (int i = 0; i < NU; ++i) m = max8(v[i], m);
        m = row_max(m);
        const float f = pow2(row_exponent(m));
#pragma unroll
        for (int i = 0; i < NU; ++i)
            if (j + i * kLanes < units) put(j + i * kLanes, v[i], f);
    } else {
        float v[8];
        for (int u = j; u < units; u += kLanes) {
            load_unit<T, BITS>(row, cols, u, v);
            m = max8(v, m);
        }
        m = row_max(m);
        const float f = pow2(row_exponent(m));
        for (int u = j; u < units; u += kLanes) {
            load_unit<T, BITS>(row, cols, u, v);
            put(u, v, f);
        }
    }
    if (kOffset) sum = group_sum<kWave>(sum);
    if constexpr (WPT > 1 && kOffset) {
        __syncthreads();                                   // the maxima are read
        if ((threadIdx.x & (kWave - 1)) == 0) red[wave] = sum;
        __syncthreads();
        sum = (red[0] + red[1]) + (red[2] + red[3]);
    }
    if (j == 0) {
        Row r;
        r.inv = pow2(-row_exponent(m));
        r.start = kOffset ? sum * (-(float)(1 << (BITS - 1)) / (1 << (24 - field_base(BITS)))) : 0.f;
        info[t] = r;
    }
}

// ------------------------------------------------------------- many tokens

typedef __attribute__((address_space(1))) const void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

// A packed step of one 16-row block: the words of kStage consecutive calls.
template <int BITS>
struct Packed {
    uint32_t w[BITS];                    // 4 calls * 8 codes * BITS / 32 words
};
template <int BITS>
__device__ __forceinline__ Packed<BITS> load_packed(const uint8_t* tile, uint32_t row, int groups, int s, int g) {
    Packed<BITS> p;
    auto at = [&](int gr) { return tile + (row + (uint32_t)min(gr, groups - 1) * 16u); };
    if constexpr (BITS == 4) {
        const uint4 q = ld16(at(4 * s + g));
        p.w[0] = q.x, p.w[1] = q.y, p.w[2] = q.z, p.w[3] = q.w;
    } else if constexpr (BITS == 8) {
        const uint4 q = ld16(at(8 * s + g));
        const uint4 r = ld16(at(8 * s + 4 + g));
        p.w[0] = q.x, p.w[1] = q.y, p.w[2] = q.z, p.w[3] = q.w;
        p.w[4] = r.x, p.w[5] = r.y, p.w[6] = r.z, p.w[7] = r.w;
    } else {
        const uint2 q = *reinterpret_cast<const uint2*>(at(4 * (s >> 1) + g) + 8 * (s & 1));
        p.w[0] = q.x, p.w[1] = q.y;
    }
    return p;
}
// The A operand of call c (0 .. 3) of a packed step.
template <int BITS, bool kOffset>
__device__ __forceinline__ half8 step_operand(const Packed<BITS>& p, int c) {
    if constexpr (BITS == 4) return a_operand<4, kOffset>(uint4{p.w[0], p.w[1], p.w[2], p.w[3]}, c);
    else if constexpr (BITS == 8)
        return a_operand<8, kOffset>(uint4{p.w[4 * (c >> 1)], p.w[4 * (c >> 1) + 1], p.w[4 * (c >> 1) + 2],
                                  p.w[4 * (c >> 1) + 3]}, c & 1);
    else return a_operand<2, kOffset>(uint4{p.w[0], p.w[1], 0, 0}, c);
}

// Workgroup tile: WN * NB * 16 weight rows by WT * TB * 16 tokens, WN x WT waves,
// over the steps of one of `splits` equal parts of K.  A step is 128 columns (fp32:
// 64 columns of both planes, each converted code used twice).  The activations of
// a step (WT * TB * 4 KB) go to one of D LDS buffers by direct loads, the packed
// codes to registers, D - 1 steps ahead; one barrier a step.  With one part the
// tile is finished here, else its fp32 sums go to `part` [split][token][row].
//
// Bound by the matrix cores where tokens are many: a wave's step is 4 * NB * TB
// MFMAs of 16 cycles against 4 * NB conversions of 5 or 6 vector instructions.
// 4096 tokens of 6144 -> 8192 in int4, bf16: 409 us, 1008 TF/s, of 1129 that a large
// bf16 library product of 8192^3 reaches; 777 fp32 tokens of 2048 -> 6145 in int2: 70
// us, 560 TF/s of the pair's products.
// Workgroups are dealt to the eight XCDs in contiguous runs of tiles, four token
// tiles by the weight tiles, so that an XCD's L2 serves each activation tile to
// several workgroups.
template <int N>
__device__ __forceinline__ void wait_loads_and_barrier() {
    // all but the last N loads of this wave have landed; then the workgroup meets
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename T, int BITS, int NB, int TB, int WN, int WT, int D>
__global__ __launch_bounds__(WN * WT * kWave) void linear_gemm(LinearArgs a, const half8* __restrict__ hi,
                                                               const half8* __restrict__ lo,
                                                               const Row* __restrict__ info, float* __restrict__ part,
                                                               int calls, int splits) {
    constexpr int kPlanes = T::bytes == 4 ? 2 : 1;
    constexpr int kW = WN * WT;
    constexpr int kLoads = WT * TB * kStage / kW;          // 1 KB direct loads a wave makes per step
    static_assert(WT * TB * kStage % kW == 0, "direct loads divide over the waves");
    __shared__ half8 buf[D][WT * TB * kStage * kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane & 15, g = lane >> 4, wn = wave % WN, wt = wave / WN;
    const int tiles_n = (a.N + WN * NB * 16 - 1) / (WN * NB * 16), tiles_t = (a.T + WT * TB * 16 - 1) / (WT * TB * 16);
    const int total = tiles_n * tiles_t * splits, per = (total + 7) / 8;
    const int unit = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || unit >= total) return;
    const int id = unit / splits, split = unit % splits;
    const int band = id / (4 * tiles_n), in = id % (4 * tiles_n), high = min(tiles_t - 4 * band, 4);
    const int tile_t = 4 * band + in % high, tile_n = in / high;
    const int r0 = (tile_n * WN + wn) * NB * 16, tb0 = tile_t * WT * TB, last_tb = (int)blocks16(a.T) - 1;
    const int groups = a.K / (128 / BITS);
    const int packs = calls / kStage, p0 = (int)((int64_t)packs * split / splits),
              p1 = (int)((int64_t)packs * (split + 1) / splits), steps = (p1 - p0) * kPlanes;
    // the tile's rows by 32-bit offsets (at most 256 rows of 64 KB)
    const int tr0 = tile_n * WN * NB * 16;
    const uint8_t* wtile = a.w + (int64_t)tr0 * groups * 16;
    uint32_t wrow[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wrow[b] = (uint32_t)(min(r0 + 16 * b + n, a.N - 1) - tr0) * (uint32_t)(groups * 16);

    // LDS unit k (0 .. 3) of a token block: call k, or (fp32) plane k / 2 of call k % 2
    auto stage = [&](int s, half8* to) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int u = wave * kLoads + i;                               // (token block, call)
            const int tb = min(tb0 + u / kStage, last_tb);
            const int k = u % kStage;
            const half8* src = (kPlanes == 2 && k >= 2 ? lo : hi) +
                               ((int64_t)tb * calls + (kPlanes == 2 ? 2 * s + (k & 1) : kStage * s + k)) * kWave + lane;
            __builtin_amdgcn_global_load_lds((gptr_t)src, (lptr_t)(to + u * kWave), 16, 0, 0);
        }
    };

    floatx4 acc[NB][TB];
    // tokens past the end belong to the last block's padding or repeat it: any start will do
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const float s = split == 0 ? info[min((tb0 + wt * TB + t), last_tb) * 16 + n].start : 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b][t] = floatx4{s, s, s, s};
    }
    // Packed steps held.  One plane: the ring follows the buffers (with one step
    // ahead the loop is not unrolled and the next codes move over: unrolled by two
    // it spilled registers).  Two planes: a packed step lasts two steps, the next
    // one is loaded at the first of them into the other slot.
    constexpr bool kMove = D == 2 && kPlanes == 1;
    constexpr int kUnroll = kMove ? 1 : 4;
    constexpr int kPackRing = kMove || kPlanes == 2 ? 2 : D;
    static_assert(kMove || D == 4 || (D == 2 && kPlanes == 2), "static buffer turns");
    Packed<BITS> pk[kPackRing][NB];
    auto codes = [&](Packed<BITS>* to, int p) {
#pragma unroll
        for (int b = 0; b < NB; ++b) to[b] = load_packed<BITS>(wtile, wrow[b], groups, p0 + p, g);
    };
    const int first = p0 * kPlanes;
    if (kMove) codes(pk[1], 0);
    if (kPlanes == 2) codes(pk[0], 0);
#pragma unroll
    for (int j = 0; j < D - 1; ++j) {
        if (j >= steps) break;
        if (kPlanes == 1 && !kMove) codes(pk[j % kPackRing], j);
        stage(first + j, buf[j]);
    }
    for (int s0 = 0; s0 < steps; s0 += kUnroll) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int s = s0 + j;
            if (s >= steps) break;
            // step s has landed once only the loads of the steps after it are left: at least
            // (D - 2) * kLoads direct loads (fewer steps remain at the end: then all)
            if (D > 2 && s + D - 1 <= steps) wait_loads_and_barrier<(D > 2 ? (D - 2) * kLoads : 0)>();
            else wait_loads_and_barrier<0>();
            const int nx = s + D - 1;
            if (kMove) {
#pragma unroll
                for (int b = 0; b < NB; ++b) pk[0][b] = pk[1][b];
            }
            if (kPlanes == 2 && j % 2 == 0 && s + 2 < steps) codes(pk[(j / 2 + 1) % 2], s / 2 + 1);
            if (nx < steps) {
                if (kPlanes == 1) codes(pk[kMove ? 1 : (j + D - 1) % kPackRing], nx);
                stage(first + nx, buf[kMove ? nx & 1 : (j + D - 1) % D]);
            }
            const half8* x = buf[kMove ? s & 1 : j % D] + wt * TB * kStage * kWave + lane;
#pragma unroll
            for (int c = 0; c < kStage / kPlanes; ++c) {
                half8 w[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    w[b] = step_operand<BITS, offset_codes(T::bytes)>(pk[kMove ? 0 : kPlanes == 2 ? j / 2 : j % kPackRing][b], kPlanes == 2 ? 2 * (j % 2) + c : c);
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int k = c; k < kStage; k += kStage / kPlanes) {
                        const half8 v = x[(t * kStage + k) * kWave];
#pragma unroll
                        for (int b = 0; b < NB; ++b) acc[b][t] = mfma::mfma(w[b], v, acc[b][t]);
                    }
            }
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int r = r0 + 16 * b + 4 * g;
        if (splits > 1) {
            if (r >= a.N) continue;
            const int64_t ldp = (a.N + 3) / 4 * 4;
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const int tok = (tb0 + wt * TB + t) * 16 + n;
                if (tok < a.T) *reinterpret_cast<floatx4*>(part + ((int64_t)split * a.T + tok) * ldp + r) = acc[b][t];
            }
            continue;
        }
        const Params par = load_params(a, r);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const int tok = (tb0 + wt * TB + t) * 16 + n;
            if (tok < a.T) finish4<T, BITS>(a, tok, r, info[tok].inv, acc[b][t], par);
        }
    }
}

// The sum of the parts of K in their order, and the epilogue: four rows a thread.
constexpr int kJoinThreads = 256;
template <typename T, int BITS>
__global__ __launch_bounds__(kJoinThreads) void linear_join(LinearArgs a, const Row* __restrict__ info,
                                                            const float* __restrict__ part, int splits) {
    const int quads = (a.N + 3) / 4, blocks = (quads + kJoinThreads - 1) / kJoinThreads;
    const int t = blockIdx.x / blocks, r = (blockIdx.x % blocks * kJoinThreads + threadIdx.x) * 4;
    if (r >= a.N) return;
    const Params par = load_params(a, r);
    const floatx4* p = reinterpret_cast<const floatx4*>(part) + (int64_t)t * quads + r / 4;
    floatx4 v = p[0];
#pragma unroll 4
    for (int s = 1; s < splits; ++s) v += p[(int64_t)s * a.T * quads];
    finish4<T, BITS>(a, t, r, info[t].inv, v, par);
}

// ------------------------------------------------------------- some tokens
//
// Up to TB * 16 tokens (64, 32 in fp32): bound by the weights' bytes and the planes'
// L2 reads.  A workgroup owns NB * 16 weight rows and all tokens; its waves split K
// by chunks of 64 bytes of a row, all loads linear, kRowFlight chunks of codes in
// flight, and meet in LDS in a fixed order.  37 bf16 tokens of 2048 -> 6144 in int8:
// 8.5 us after 2.5 us of planes.
constexpr int kRowWaves = 8;
constexpr int kRowFlight = 4;               // even: the operands' two buffers alternate with it

template <typename T, int BITS, int TB, int NB>
__global__ __launch_bounds__(kRowWaves * kWave) void linear_rows(LinearArgs a, const half8* __restrict__ hi,
                                                                 const half8* __restrict__ lo,
                                                                 const Row* __restrict__ info, int calls) {
    using M = MfmaCodec<BITS>;
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane & 15, g = lane >> 4;
    const int r0 = blockIdx.x * 16 * NB, last_tb = (int)blocks16(a.T) - 1;
    const int groups = a.K / (128 / BITS), chunks = (groups + 3) / 4;
    const uint8_t* wrow[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wrow[b] = a.w + (int64_t)min(r0 + 16 * b + n, a.N - 1) * groups * 16;
    auto codes = [&](int b, int ch) { return ld16(wrow[b] + (int64_t)min(4 * ch + g, groups - 1) * 16); };
    uint4 q[kRowFlight][NB];
#pragma unroll
    for (int i = 0; i < kRowFlight; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) q[i][b] = codes(b, wave + i * kRowWaves);
    constexpr int kFinish = TB * NB;                       // 16 x 16 blocks to finish, one a wave
    const int ft = wave % TB, fb = wave / TB % NB;
    Params par;
    if (wave < kFinish) par = load_params(a, r0 + 16 * fb + 4 * g);
    floatx4 acc[TB][NB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const float s = wave == 0 ? info[min(t, last_tb) * 16 + n].start : 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[t][b] = floatx4{s, s, s, s};
    }
    // the planes' operands of a chunk, one chunk ahead where they fit the registers
    constexpr int kPlanes = T::bytes == 4 ? 2 : 1;
    constexpr bool kAhead = M::NCALL * TB * kPlanes <= 16;
    half8 xv[kAhead ? 2 : 1][kAhead ? M::NCALL : 1][TB][kPlanes];
    auto call = [&](half8 (*to)[kPlanes], int ch, int c) {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const int64_t at = ((int64_t)min(t, last_tb) * calls + ch * M::NCALL + c) * kWave + lane;
            to[t][0] = hi[at];
            if (kPlanes == 2) to[t][kPlanes - 1] = lo[at];
        }
    };
    auto acts = [&](int to, int ch) {
#pragma unroll
        for (int c = 0; c < M::NCALL; ++c) call(xv[to][c], ch, c);
    };
    if constexpr (kAhead) {
        if (wave < chunks) acts(0, wave);
    }
    for (int c0 = wave; c0 < chunks; c0 += kRowFlight * kRowWaves) {
#pragma unroll
        for (int i = 0; i < kRowFlight; ++i) {
            const int ch = c0 + i * kRowWaves;
            if (ch >= chunks) break;
            if constexpr (kAhead) {
                if (ch + kRowWaves < chunks) acts((i + 1) & 1, ch + kRowWaves);
            }
#pragma unroll
            for (int c = 0; c < M::NCALL; ++c) {
                half8(*x)[kPlanes] = xv[kAhead ? i & 1 : 0][kAhead ? c : 0];
                if constexpr (!kAhead) call(x, ch, c);
                half8 w[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) w[b] = a_operand<BITS, offset_codes(T::bytes)>(q[i][b], c);
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int k = 0; k < kPlanes; ++k)
#pragma unroll
                        for (int b = 0; b < NB; ++b) acc[t][b] = mfma::mfma(w[b], x[t][k], acc[t][b]);
            }
            const int nx = ch + kRowFlight * kRowWaves;
            if (nx < chunks) {
#pragma unroll
                for (int b = 0; b < NB; ++b) q[i][b] = codes(b, nx);
            }
        }
    }
    __shared__ floatx4 part[kRowWaves][kFinish][kWave];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) part[wave][b * TB + t][lane] = acc[t][b];
    __syncthreads();
    if (wave >= kFinish) return;
    floatx4 v = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) v += part[w][wave][lane];
    const int tok = ft * 16 + n;
    if (tok < a.T) finish4<T, BITS>(a, tok, r0 + 16 * fb + 4 * g, info[tok].inv, v, par);
}

// -------------------------------------------------------------- few tokens
//
// Up to kFewTokens tokens of kFewValues values together, in one launch: every
// workgroup converts the activations itself while its first weight loads are in
// flight.  With one to eight tokens the 16 MFMA columns hold the hi parts (0 ..
// 7) and, for fp32, the lo parts (8 .. 15) side by side, so a pair costs no
// second MFMA; columns without a token repeat one and are dropped.  One fp32 token
// of 6144 -> 8192 in int4: 10.6 us, 2.4 TB/s of weights, of which the launch and the
// first memory latencies are about half.
constexpr int kFewTokens = 8;
constexpr int kFewValues = 16384;         // tokens times padded columns at most
constexpr int kFewFlight = 8;             // chunks a wave has in flight
constexpr int kFewUnits = kFewValues / 8 / (kRowWaves * kWave);   // units a thread converts at most

template <typename T, int BITS>
__global__ __launch_bounds__(kRowWaves * kWave) void linear_few(LinearArgs a, int calls) {
    using M = MfmaCodec<BITS>;
    constexpr int CW = 128 / BITS;
    constexpr int kThreads = kRowWaves * kWave;
    constexpr int kPlanes = T::bytes == 4 ? 2 : 1;
    constexpr bool kOffset = offset_codes(T::bytes);
    extern __shared__ half8 xs[];                          // [token][plane][call][lane group]
    __shared__ unsigned top[kFewTokens];                   // largest magnitudes as bits (they are not negative)
    __shared__ floatx4 part[kRowWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane & 15, g = lane >> 4;
    const int r0 = blockIdx.x * 16, units = calls * 4, total = a.T * units;
    const int groups = a.K / CW, chunks = (groups + 3) / 4;
    const uint8_t* wrow = a.w + (int64_t)min(r0 + n, a.N - 1) * groups * 16;
    if (threadIdx.x < kFewTokens) top[threadIdx.x] = 0;

    // the activations first: what waits for them need not wait for the weights
    const typename T::type* x = reinterpret_cast<const typename T::type*>(a.x);
    float v[kFewUnits][8];
#pragma unroll
    for (int i = 0; i < kFewUnits; ++i) {
        const int k = threadIdx.x + i * kThreads;
        if (i * kThreads < total) {
            const int t = min(k, total - 1) / units;
            load_unit<T, BITS>(x + t * a.ldx, k < total ? a.K : 0, k - t * units, v[i]);
        }
    }
    uint4 q[kFewFlight];
#pragma unroll
    for (int i = 0; i < kFewFlight; ++i)
        if (i == 0 || i * kRowWaves < chunks)
            q[i] = ld16(wrow + (int64_t)min(4 * (wave + i * kRowWaves) + g, groups - 1) * 16);
    Params par;
    if (wave == 0) par = load_params(a, r0 + 4 * g);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewUnits; ++i) {
        const int k = threadIdx.x + i * kThreads;
        if (i * kThreads < total) {
            // 16 consecutive units belong to one token (units is a multiple of 16)
            float m = max8(v[i], 0.f);
            m = fmaxf(m, dpp_f<0xB1>(m));
            m = fmaxf(m, dpp_f<0x4E>(m));
            m = fmaxf(m, dpp_f<0x141>(m));
            m = fmaxf(m, dpp_f<0x140>(m));
            if ((lane & 15) == 0 && k < total) atomicMax(&top[k / units], __float_as_uint(m));
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewUnits; ++i) {
        const int k = threadIdx.x + i * kThreads;
        if (k < total) {
            const int t = k / units;
            half8 h, l;
            split_unit<BITS, kOffset>(v[i], pow2(row_exponent(__uint_as_float(top[t]))), h, l);
            xs[kPlanes * t * units + k - t * units] = h;
            if (kPlanes == 2) xs[(2 * t + 1) * units + k - t * units] = l;
        }
    }
    __syncthreads();

    const int tok = kPlanes == 2 ? n & 7 : n;
    const half8* mine = xs + (kPlanes * min(tok, a.T - 1) + (kPlanes == 2 ? n >> 3 : 0)) * units + g;
    const half8 offset = minus_offset<BITS>();
    floatx4 acc2[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int c0 = wave; c0 < chunks; c0 += kFewFlight * kRowWaves) {
#pragma unroll
        for (int i = 0; i < kFewFlight; ++i) {
            const int ch = c0 + i * kRowWaves;
            if (ch < chunks) {
#pragma unroll
                for (int c = 0; c < M::NCALL; ++c) {
                    const half8 xv = mine[(ch * M::NCALL + c) * 4];
                    if (kOffset) {
                        acc2[0] = mfma::mfma(a_operand<BITS, kOffset>(q[i], c), xv, acc2[0]);
                        acc2[1] = mfma::mfma(offset, xv, acc2[1]);     // the offset's part of the sum
                    } else {
                        acc2[c & 1] = mfma::mfma(a_operand<BITS, kOffset>(q[i], c), xv, acc2[c & 1]);
                    }
                }
            }
            const int nx = ch + kFewFlight * kRowWaves;
            if (nx < chunks) q[i] = ld16(wrow + (int64_t)min(4 * nx + g, groups - 1) * 16);
        }
    }
    part[wave][lane] = acc2[0] + acc2[1];
    __syncthreads();
    if (wave != 0) return;
    floatx4 sum = part[0][lane];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) sum += part[w][lane];
    if (kPlanes == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += __shfl_xor(sum[i], 8, kWave);
    }
    if (tok >= a.T || (kPlanes == 2 && n >= 8)) return;
    finish4<T, BITS>(a, tok, r0 + 4 * g, pow2(-row_exponent(__uint_as_float(top[tok]))), sum, par);
}

// ------------------------------------------------------------------- launches

// linear_rows up to here: as many blocks of 16 tokens as keep a chunk's operands in
// registers, twice (64 bf16 tokens of 6144 -> 8192 in int4: 20 us, 25 by linear_gemm).
constexpr int rows_tokens(int bytes) { return bytes == 4 ? 32 : 64; }
constexpr int kCus = 256;

// The one-launch form: every workgroup converts all activations, so it pays while
// they are few (int4, bf16, 4096 -> 4096, 4 tokens: 7.6 us against 8.6 by way of
// planes; 6144 -> 8192, 4 tokens: 14.2 against 12.6).
bool few(int64_t T, int64_t K, int bits) { return T <= kFewTokens && T * padded(K, bits) <= kFewValues; }

// The tile of linear_gemm and the parts of K.  Two tiles: 128 weight rows by 64
// tokens, of which a compute unit holds two (sixteen waves hide the loads of short
// runs), and 256 by 256, one a compute unit, 1.3 times as fast per output where
// there are enough of them.  Up to 512 small tiles K is split until the compute
// units have one or two each (at least 512 columns a part); beyond that the two
// are priced by the rounds they take, 2.8 fs for an output's column in a small
// tile's round, and the joining of the parts at 5 TB/s.  Measured at 6144 -> 8192
// in int4, bf16: 64 tokens 24 us small against 47 large, 256: 50 / 59, 512: 79 /
// 84, 1024: 160 / 149, 4096: - / 449 (before the unsigned codes, 409 with them).
struct Tiling {
    bool large;
    int splits;
};
Tiling tiling(int64_t T, int64_t K, int64_t N, int bits, int bytes) {
    auto count = [&](int r, int t) { return ((N + r - 1) / r) * ((T + t - 1) / t); };
    const int64_t small = count(128, 64), most = padded(K, bits) / 512;
    auto parts = [&](int64_t tiles, int64_t want) {
        int64_t s = (want + tiles / 2) / tiles;
        if (s > most) s = most;
        return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
    };
    if (small <= 2 * kCus) return {false, parts(small, small < kCus / 2 ? kCus : 2 * kCus)};
    const int64_t large = count(256, 256);
    const int s = parts(large, kCus);
    const double unit = 2.8e-9 * (double)K * (bytes == 4 ? 2 : 1);                          // us an output
    const double t_small = unit * 128 * 64 * 2 * kCus * ((small + 2 * kCus - 1) / (2 * kCus));
    const double t_large = unit * 256 * 256 * kCus / (1.3 * s) * ((large * s + kCus - 1) / kCus) +
                           (s > 1 ? 3.0 + 1.6e-6 * s * (double)T * N : 0.0);
    if (t_small <= t_large) return {false, 1};
    return {true, s};
}

template <typename T, int BITS, int NB, int TB, int WN, int WT, int D>
void launch_gemm(const LinearArgs& a, const half8* hi, const half8* lo, const Row* info, float* part, int calls,
                 int splits, hipStream_t st) {
    const int64_t tiles = (int64_t)((a.N + WN * NB * 16 - 1) / (WN * NB * 16)) *
                          ((a.T + WT * TB * 16 - 1) / (WT * TB * 16)) * splits;
    hipLaunchKernelGGL((linear_gemm<T, BITS, NB, TB, WN, WT, D>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                       dim3(WN * WT * kWave), 0, st, a, hi, lo, info, part, calls, splits);
    if (splits > 1) {
        const int64_t blocks = ((a.N + 3) / 4 + kJoinThreads - 1) / kJoinThreads;
        hipLaunchKernelGGL((linear_join<T, BITS>), dim3((unsigned)(blocks * a.T)), dim3(kJoinThreads), 0, st, a, info, part,
                           splits);
    }
}

template <typename T, int BITS, int NU, int WPT>
void launch_units(const LinearArgs& a, half8* hi, half8* lo, Row* info, int calls, hipStream_t st) {
    const int64_t grid = (blocks16(a.T) + 7) / 8 * 8 * (16 / (kPrepThreads / kWave / WPT));
    hipLaunchKernelGGL((linear_prepare<T, BITS, NU, WPT>), dim3((unsigned)grid), dim3(kPrepThreads), 0, st,
                       reinterpret_cast<const typename T::type*>(a.x), a.ldx, a.T, a.K, calls, hi, lo, info);
}

// Four waves a token while that fills the compute units no more than a few times
// over (4 us instead of 8 for 16 tokens of 6144 columns), else one.
template <typename T, int BITS>
void launch_prepare(const LinearArgs& a, half8* hi, half8* lo, Row* info, int calls, hipStream_t st) {
    const int units = calls * 4;
    if (a.T <= 1024) {
        if (units <= 256) launch_units<T, BITS, 1, 4>(a, hi, lo, info, calls, st);
        else if (units <= 1024) launch_units<T, BITS, 4, 4>(a, hi, lo, info, calls, st);
        else launch_units<T, BITS, 0, 4>(a, hi, lo, info, calls, st);
    } else {
        if (units <= 256) launch_units<T, BITS, 4, 1>(a, hi, lo, info, calls, st);
        else if (units <= 1024) launch_units<T, BITS, 16, 1>(a, hi, lo, info, calls, st);
        else launch_units<T, BITS, 0, 4>(a, hi, lo, info, calls, st);
    }
}

template <typename T, int BITS, int TB>
void launch_rows(const LinearArgs& a, const half8* hi, const half8* lo, const Row* info, int calls, hipStream_t st) {
    // two row blocks a workgroup where that still gives every compute unit one
    if (a.N >= kCus * 32)
        hipLaunchKernelGGL((linear_rows<T, BITS, TB, 2>), dim3((a.N + 31) / 32), dim3(kRowWaves * kWave), 0, st, a, hi,
                           lo, info, calls);
    else
        hipLaunchKernelGGL((linear_rows<T, BITS, TB, 1>), dim3((a.N + 15) / 16), dim3(kRowWaves * kWave), 0, st, a, hi,
                           lo, info, calls);
}

template <typename T, int BITS>
hipError_t launch_bits(const LinearArgs& a, hipStream_t st) {
    const int64_t Kp = padded(a.K, BITS);
    const int calls = (int)(Kp / 32);
    if (few(a.T, a.K, BITS)) {
        const size_t lds = (size_t)a.T * Kp * (T::bytes == 4 ? 4 : 2);
        hipLaunchKernelGGL((linear_few<T, BITS>), dim3((a.N + 15) / 16), dim3(kRowWaves * kWave), lds, st, a, calls);
        return hipGetLastError();
    }
    const int64_t blocks = blocks16(a.T);
    half8* hi = reinterpret_cast<half8*>(a.workspace);
    half8* lo = hi + (T::bytes == 4 ? blocks * calls * kWave : 0);
    Row* info = reinterpret_cast<Row*>(lo + blocks * calls * kWave);
    float* part = reinterpret_cast<float*>(info + blocks * 16);
    launch_prepare<T, BITS>(a, hi, lo, info, calls, st);
    if (a.T <= 16) {
        launch_rows<T, BITS, 1>(a, hi, lo, info, calls, st);
    } else if (a.T <= 32) {
        launch_rows<T, BITS, 2>(a, hi, lo, info, calls, st);
    } else if (a.T <= rows_tokens(T::bytes)) {
        if constexpr (rows_tokens(T::bytes) > 32) {
            if (a.T <= 48) launch_rows<T, BITS, 3>(a, hi, lo, info, calls, st);
            else launch_rows<T, BITS, 4>(a, hi, lo, info, calls, st);
        }
    } else {
        const Tiling k = tiling(a.T, a.K, a.N, BITS, T::bytes);
        if (k.large) launch_gemm<T, BITS, 4, 8, 4, 2, 2>(a, hi, lo, info, part, calls, k.splits, st);
        else launch_gemm<T, BITS, 1, 4, 8, 1, 4>(a, hi, lo, info, part, calls, k.splits, st);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_type(int bits, const LinearArgs& a, hipStream_t st) {
    switch (bits) {
        case 4: return launch_bits<T, 4>(a, st);
        case 8: return launch_bits<T, 8>(a, st);
        case 2: return launch_bits<T, 2>(a, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

int64_t linear_workspace(int bits, int dtype, int64_t T, int64_t K, int64_t N) {
    const int bytes = dtype == MOEDEC_F32 ? 4 : 2;
    if (T == 0 || few(T, K, bits)) return 0;
    int64_t n = blocks16(T) * 16 * (padded(K, bits) * bytes + (int64_t)sizeof(Row));
    if (T > rows_tokens(bytes)) {
        const int splits = tiling(T, K, N, bits, bytes).splits;
        if (splits > 1) n += splits * T * ((N + 3) / 4 * 16);
    }
    return n;
}

int64_t linear_grid(const LinearArgs& a) {
    return (int64_t)((a.N + 127) / 128) * ((a.T + 63) / 64) * 16 + (int64_t)a.T * ((a.N + 1023) / 1024) + 8;
}

hipError_t launch_linear(int bits, int dtype, const LinearArgs& a, hipStream_t st) {
    if (a.T == 0) return hipSuccess;
    switch (dtype) {
        case MOEDEC_F32: return launch_type<F32>(bits, a, st);
        case MOEDEC_F16: return launch_type<F16>(bits, a, st);
        case MOEDEC_BF16: return launch_type<BF16>(bits, a, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace attn
}  // namespace moedec
