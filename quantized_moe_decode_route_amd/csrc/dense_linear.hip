// y = act(scale * (x . codes) + bias) + residual on packed row-scaled weights.
//
// The codes are exact in fp16 and so, up to the exponent range, is every fp16 or
// bf16 activation once its row is scaled by a power of two that brings the
// largest magnitude to [2^14, 2^15): the products on v_mfma_f32_16x16x32_f16 are
// then exact and only the fp32 sums round.  fp32 activations enter as a hi/lo
// pair of fp16 (about 22 bits), two MFMAs instead of one.  The power of two, the
// row scale, bias, activation and residual are applied once, in fp32, to the
// sums.
#include "attn.h"
#include "mfma.h"

namespace moedec {
namespace attn {

namespace {

using mfma::a_operand;
using mfma::MfmaCodec;

constexpr int kPad = 256;                 // columns a plane's row is padded to (a chunk of 2-bit codes)
constexpr int kPrepThreads = 256;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// Exponent k with m * 2^k in [2^14, 2^15) (0 for zero and non-finite m).
__device__ __forceinline__ int row_exponent(float m) {
    if (!(m > 0.f) || !(m <= 3.402823466e38f)) return 0;
    const int k = 14 - ((int)(__float_as_uint(m) >> 23) - 127);
    return k > 120 ? 120 : k;
}

__host__ __device__ inline int64_t padded(int64_t K) { return (K + kPad - 1) / kPad * kPad; }

// A row of x as fp16 planes (hi, and lo for fp32), its columns in the order the
// codes of a 16-byte group enter the MFMAs, zero past K; inv = 2^-k of the row.
template <typename T, int BITS>
__global__ __launch_bounds__(kPrepThreads) void linear_prepare(const typename T::type* __restrict__ x, int64_t ldx,
                                                               int K, int Kp, _Float16* __restrict__ hi,
                                                               _Float16* __restrict__ lo, float* __restrict__ inv) {
    using M = MfmaCodec<BITS>;
    constexpr int CW = 128 / BITS;
    const int64_t t = blockIdx.x;
    const typename T::type* row = x + t * ldx;
    __shared__ float red[kPrepThreads / kWave];
    float m = 0.f;
    for (int c = threadIdx.x * 8; c < K; c += kPrepThreads * 8) {
        float v[8];
        load8<T>(row + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
    }
    m = wave_max(m);
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const int k = row_exponent(m);
    const float f = pow2(k);
    if (threadIdx.x == 0) inv[t] = pow2(-k);
    for (int c = threadIdx.x * 8; c < Kp; c += kPrepThreads * 8) {
        half8 h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = c / CW * CW + M::col(c % CW / 8, e);
            const float v = col < K ? T::get(row[col]) : 0.f;
            const mfma::F16Pair p = mfma::split_f16(v, f);
            h[e] = p.hi;
            l[e] = p.lo;
        }
        *reinterpret_cast<half8*>(hi + t * Kp + c) = h;
        if (T::bytes == 4) *reinterpret_cast<half8*>(lo + t * Kp + c) = l;
    }
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case MOEDEC_ACT_SILU: return v / (1.0f + expf(-v));
        case MOEDEC_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
        case MOEDEC_ACT_RELU: return v < 0.f ? 0.f : v;
        default: return v;
    }
}

// 16 weight rows by 16 tokens a workgroup, its waves splitting K.
template <typename T, int BITS>
__global__ __launch_bounds__(kThreads) void linear_simple(LinearArgs a, int Kp, const _Float16* __restrict__ hi,
                                                          const _Float16* __restrict__ lo,
                                                          const float* __restrict__ inv) {
    using M = MfmaCodec<BITS>;
    constexpr int CW = 128 / BITS;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, g = lane >> 4;
    const int tiles = (a.N + 15) / 16, r0 = blockIdx.x % tiles * 16, t0 = blockIdx.x / tiles * 16;
    const int groups = a.K / CW, chunks = (groups + 3) / 4;
    const uint8_t* wrow = a.w + (int64_t)min(r0 + n, a.N - 1) * groups * 16;
    const int64_t xrow = (int64_t)min(t0 + n, a.T - 1) * Kp;
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int ch = wave; ch < chunks; ch += kWaves) {
        const int gr = ch * 4 + g;
        uint4 q = {0, 0, 0, 0};
        if (gr < groups) q = ld16(wrow + (int64_t)gr * 16);
#pragma unroll
        for (int c = 0; c < M::NCALL; ++c) {
            const half8 w = a_operand<BITS>(q, c);
            acc = mfma::mfma(w, *reinterpret_cast<const half8*>(hi + xrow + (int64_t)gr * CW + 8 * c), acc);
            if (T::bytes == 4)
                acc = mfma::mfma(w, *reinterpret_cast<const half8*>(lo + xrow + (int64_t)gr * CW + 8 * c), acc);
        }
    }
    __shared__ floatx4 part[kWaves][kWave];
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    const int t = t0 + n;
    if (t >= a.T) return;
    typename T::type* y = reinterpret_cast<typename T::type*>(a.y) + (int64_t)t * a.ldy;
    const typename T::type* res = reinterpret_cast<const typename T::type*>(a.residual) + (int64_t)t * a.ldr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * g + i;
        if (r >= a.N) break;
        float v = (part[0][lane][i] + part[1][lane][i]) + (part[2][lane][i] + part[3][lane][i]);
        v = v * inv[t] * a.scale[r];
        if (a.bias) v += a.bias[r];
        v = activate(v, a.act);
        if (a.residual) v += T::get(res[r]);
        y[r] = T::put(v);
    }
}

template <typename T, int BITS>
hipError_t launch_bits(const LinearArgs& a, hipStream_t st) {
    const int64_t Kp = padded(a.K);
    _Float16* hi = reinterpret_cast<_Float16*>(a.workspace);
    _Float16* lo = hi + (T::bytes == 4 ? (int64_t)a.T * Kp : 0);
    float* inv = reinterpret_cast<float*>(lo + (int64_t)a.T * Kp);
    hipLaunchKernelGGL((linear_prepare<T, BITS>), dim3(a.T), dim3(kPrepThreads), 0, st,
                       reinterpret_cast<const typename T::type*>(a.x), a.ldx, a.K, (int)Kp, hi, lo, inv);
    hipLaunchKernelGGL((linear_simple<T, BITS>), dim3((unsigned)linear_grid(a)), dim3(kThreads), 0, st, a,
                       (int)Kp, hi, lo, inv);
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

int64_t linear_workspace(int dtype, int64_t T, int64_t K) {
    if (T == 0) return 0;
    return T * padded(K) * (dtype == MOEDEC_F32 ? 4 : 2) + (T * 4 + 15) / 16 * 16;
}

int64_t linear_grid(const LinearArgs& a) { return (int64_t)((a.N + 15) / 16) * ((a.T + 15) / 16); }

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
