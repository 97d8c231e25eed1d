// quantize.hip -- dynamic quantisation of tokens to 8-bit integers.
//
//   m = max_c |x|,  scale = m / 127,  q = round_half_even(127 x / m)
//
// The rounding is that of the exact quotient.  t = x * (127 / m) in fp32 is off by
// less than 1.6e-5 (|t| <= 127, two roundings), so it decides unless it lies within
// 1e-4 of a half; those few go to 64 bits.  With x = X 2^a, m = M 2^b (X, M of 24 bits) the quotient
// differs from a half (2k+1)/2 by (254 X 2^(a-b) - (2k+1) M) / 2M: it is one, which a double holds
// and the division gives without error, or at least 2^(a-b) / 2^25 away.  A quotient next to a half
// is about 1/2 or more, so x / m is at least about 1/254 and a - b >= -8: 2^-33, far more than the
// double's error of 2^-46.
//
// Memory bound (8192 x 4096 bf16: 19.7 us, 5.1 TB/s).  Tokens first: a token's values stay in registers between the
// maximum and the rounding, so x is read once.  Channel-major: a tile of 32 tokens
// is read twice (the second time mostly from the last-level cache) and turned in LDS.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int kThreads = 256;
typedef signed char i8x8 __attribute__((ext_vector_type(8)));

// |v| as the bits of a non-negative float (infinities and NaN compare above every number).
DEVI uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
DEVI uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
constexpr uint32_t kInfBits = 0x7f800000u;

DEVI float token_scale(uint32_t m) {
    return m >= kInfBits ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / 127.0f;
}

struct Rounding {
    uint32_t m;
    float inv;      // 0 where the quotient is taken in 64 bits throughout
};

DEVI Rounding rounding(uint32_t m) {
    // below 2^-100, 127 / m could overflow
    return {m, m >= 0x0d800000u && m < kInfBits ? 127.0f / __uint_as_float(m) : 0.0f};
}

DEVI signed char quant1(float x, const Rounding &r) {
    const float t = x * r.inv, n = __builtin_rintf(t), off = __builtin_fabsf(t - n);
    if (r.inv != 0.0f && off < 0.4999f) return (signed char)(int)n;
    if (r.m == 0 || r.m >= kInfBits) return 0;
    return (signed char)(int)__builtin_rint((double)x * 127.0 / (double)__uint_as_float(r.m));
}

DEVI i8x8 quant8(const float (&v)[8], const Rounding &r) {
    i8x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = quant1(v[i], r);
    return o;
}

DEVI uint32_t max8(const float (&v)[8], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, abs_bits(v[i]));
    return m;
}

// TPT threads per token, NV vectors of eight channels per thread held in registers;
// channels past NV * 8 * TPT are read again.
template <int DT, int TPT, int NV>
__global__ __launch_bounds__(kThreads) void quantize_kernel(int L, int C, int C_pad, long long tokens,
                                                            const typename Elem<DT>::T *x, long long sb, long long sl,
                                                            signed char *q, float *scale, uint32_t first) {
    __shared__ uint32_t red[kThreads / 64];
    const int sub = threadIdx.x % TPT;
    const long long tok = (long long)(first + blockIdx.x) * (kThreads / TPT) + threadIdx.x / TPT;
    if (TPT == 64 && tok >= tokens) return;     // one wave: no barrier ahead
    const int b = (int)(tok / L), l = (int)(tok - (long long)b * L);
    const typename Elem<DT>::T *row = x + b * sb + l * sl;
    float v[NV][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load8<DT>(row, (i * TPT + sub) * 8, C, v[i]);
        m = max8(v[i], m);
    }
    for (int c = (NV * TPT + sub) * 8; c < C; c += TPT * 8) {
        float w[8];
        load8<DT>(row, c, C, w);
        m = max8(w, m);
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) m = umax(m, __shfl_xor(m, k));
    if constexpr (TPT > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) m = umax(m, red[i]);
    }
    const Rounding r = rounding(m);
    signed char *out = q + tok * C_pad;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPT + sub) * 8;
        if (c < C_pad) *(i8x8 *)(out + c) = quant8(v[i], r);     // zeros past C
    }
    for (int c = (NV * TPT + sub) * 8; c < C_pad; c += TPT * 8) {
        float w[8];
        load8<DT>(row, c, C, w);
        *(i8x8 *)(out + c) = quant8(w, r);
    }
    if (sub == 0) scale[tok] = token_scale(m);
}

// 32 time steps of one sequence per work-group: a thread holds eight steps of one of
// 64 channels at a time.
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_cm_kernel(int L, int C, int C_pad, int tiles,
                                                               const typename Elem<DT>::T *x, long long sb, long long sc,
                                                               signed char *q, float *scale, uint32_t first) {
    __shared__ uint32_t red[64][33];
    __shared__ __attribute__((aligned(16))) signed char turn[32][72];
    const uint32_t tile = first + blockIdx.x;
    const int b = tile / tiles, l0 = (tile - b * tiles) * 32;
    const int part = threadIdx.x & 3, ch = threadIdx.x >> 2, l = l0 + part * 8;
    const typename Elem<DT>::T *base = x + b * sb;
    uint32_t m[8] = {};
    for (int c = ch; c < C; c += 64) {
        float v[8];
        load8<DT>(base + c * sc, l, L, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = umax(m[i], abs_bits(v[i]));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[ch][part * 8 + i] = m[i];
    __syncthreads();
    for (int h = 32; h > 0; h >>= 1) {
        if (ch < h)
#pragma unroll
            for (int i = 0; i < 8; ++i) red[ch][part * 8 + i] = umax(red[ch][part * 8 + i], red[ch + h][part * 8 + i]);
        __syncthreads();
    }
    Rounding r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = rounding(red[0][part * 8 + i]);
    if (threadIdx.x < 32 && l0 + (int)threadIdx.x < L)
        scale[(long long)b * L + l0 + threadIdx.x] = token_scale(red[0][threadIdx.x]);
    const int tok = threadIdx.x >> 3, piece = (threadIdx.x & 7) * 8;
    for (int c0 = 0; c0 < C_pad; c0 += 64) {
        float v[8] = {};
        if (c0 + ch < C) load8<DT>(base + (c0 + ch) * sc, l, L, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) turn[part * 8 + i][ch] = quant1(v[i], r[i]);
        __syncthreads();
        if (l0 + tok < L) *(i8x8 *)(q + ((long long)b * L + l0 + tok) * C_pad + c0 + piece) = *(const i8x8 *)&turn[tok][piece];
        __syncthreads();
    }
}

template <int DT>
int quantize(int B, int L, int C, const void *xp, long long sb, long long sl, long long sc, signed char *q,
             float *scale, hipStream_t st) {
    typedef typename Elem<DT>::T T;
    const T *x = (const T *)xp;
    const int C_pad = (C + MICONV_I8_PAD - 1) / MICONV_I8_PAD * MICONV_I8_PAD;
    const long long tokens = (long long)B * L;
    if (sc != 1 && C > 1) {
        const int tiles = (L + 31) / 32;
        return launch_groups((long long)B * tiles, kThreads, [&](unsigned n, unsigned first) {
            hipLaunchKernelGGL(quantize_cm_kernel<DT>, dim3(n), dim3(kThreads), 0, st, L, C, C_pad, tiles, x, sb, sc, q, scale,
                               first);
        });
    }
    // up to 2048 channels a wave per token: no barrier (8192 tokens of 1000: 7.9 us against 13.8 with a
    // work-group per token, of 2048 13.4 against 15.2, of 4096 26.2 against 19.7)
    const auto kern = C <= 1024   ? quantize_kernel<DT, 64, 2>
                      : C <= 2048 ? quantize_kernel<DT, 64, 4>
                      : C <= 4096 ? quantize_kernel<DT, 256, 2>
                                  : quantize_kernel<DT, 256, 4>;
    return launch_groups(C <= 2048 ? (tokens + 3) / 4 : tokens, kThreads, [&](unsigned n, unsigned first) {
        hipLaunchKernelGGL(kern, dim3(n), dim3(kThreads), 0, st, L, C, C_pad, tokens, x, sb, sl, q, scale, first);
    });
}

}  // namespace

int launch_quantize(int B, int L, int C, int dtype, const void *x, long long sb, long long sl, long long sc,
                    signed char *q, float *scale, hipStream_t st) {
    return dtype ? quantize<1>(B, L, C, x, sb, sl, sc, q, scale, st)
                 : quantize<0>(B, L, C, x, sb, sl, sc, q, scale, st);
}

}  // namespace miconv
