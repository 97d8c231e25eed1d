// quantize.hip -- dynamic quantisation of tokens to 8-bit integers.
//
//   m = max_c |x|,  scale = m / 127,  q = round_half_even(127 x / m)
//
// The quotient is rounded in 64 bits, which decides as the exact quotient would:
// x and m have at most 24 significant bits, so 127 x / m is a half exactly or at
// least 2^-25 away from one, and a half is held without error.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int kThreads = 256;

// Largest |v| of a token as the bits of a non-negative float (infinities and NaN
// compare above every number).
DEVI uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

DEVI uint32_t block_max(uint32_t m, uint32_t *red) {
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) {
        const uint32_t o = __shfl_xor(m, k);
        m = o > m ? o : m;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int i = 0; i < kThreads / 64; ++i) m = red[i] > m ? red[i] : m;
    return m;
}

DEVI int quant1(float x, uint32_t mbits) {
    if (mbits == 0 || mbits >= kInfBits) return 0;
    return (int)__builtin_rint((double)x * 127.0 / (double)__uint_as_float(mbits));
}

// One work-group per token.
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(int L, int C, int C_pad, const typename Elem<DT>::T *x,
                                                            long long sb, long long sl, long long sc,
                                                            signed char *q, float *scale) {
    __shared__ uint32_t red[kThreads / 64];
    const long long tok = blockIdx.x;
    const int b = (int)(tok / L), l = (int)(tok - (long long)b * L);
    const typename Elem<DT>::T *row = x + b * sb + l * sl;
    uint32_t m = 0;
    for (int c = threadIdx.x; c < C; c += kThreads) {
        const uint32_t a = abs_bits(Elem<DT>::get(row[c * sc]));
        m = a > m ? a : m;
    }
    m = block_max(m, red);
    signed char *out = q + tok * C_pad;
    for (int c = threadIdx.x; c < C_pad; c += kThreads)
        out[c] = c < C ? (signed char)quant1(Elem<DT>::get(row[c * sc]), m) : (signed char)0;
    if (threadIdx.x == 0) scale[tok] = m >= kInfBits ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / 127.0f;
}

}  // namespace

int launch_quantize(int B, int L, int C, int dtype, const void *x, long long sb, long long sl, long long sc,
                    signed char *q, float *scale, hipStream_t st) {
    const int C_pad = (C + MICONV_I8_PAD - 1) / MICONV_I8_PAD * MICONV_I8_PAD;
    const dim3 grid((unsigned)((long long)B * L));
    if (dtype)
        hipLaunchKernelGGL(quantize_kernel<1>, grid, dim3(kThreads), 0, st, L, C, C_pad, (const __bf16 *)x, sb, sl, sc, q,
                           scale);
    else
        hipLaunchKernelGGL(quantize_kernel<0>, grid, dim3(kThreads), 0, st, L, C, C_pad, (const float *)x, sb, sl, sc, q,
                           scale);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

}  // namespace miconv
