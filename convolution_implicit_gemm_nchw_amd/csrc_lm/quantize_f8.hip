// quantize_f8.hip -- quantisation to 8-bit floating point (e4m3) with a power of two for each token and block of
// 128 channels:
//   scale = the least 2^e, e >= -127, with max|x| <= 448 * 2^e,   q = x / scale rounded to nearest, ties to even.
// With a power of two the quotient is exact, so q is rounded once, and the product's MFMAs apply the scales by
// themselves.  A block that holds an infinity or a NaN gets the scale's NaN (255) and q = NaN.
//
// Memory bound.  Tokens first: 16 lanes hold a block between the maximum and the rounding.  Channel-major: a
// work-group holds 64 tokens' block and turns it in LDS.  8192 tokens of 4096 channels, bf16, tokens first: 19 us, 101 MB
// at 5.3 TB/s.
#include "f8.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr uint32_t kInfinite = 0x7f800000u;

DEVI uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale's exponent plus 127, of a block whose largest magnitude has these bits: 448 = 1.75 * 2^8.
DEVI uint32_t scale_code(uint32_t top) {
    if (top >= kInfinite) return 255u;
    const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)((e < -127 ? -127 : e) + 127);
}

// 1 / scale: 2^(127 - code), a normal number for every finite code (at most 247).
DEVI float scale_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }

// Eight values to eight bytes.
DEVI u32x2 pack8(const float (&v)[8], uint32_t code) {
    if (code == 255u) return u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
    const float r = scale_inverse(code);
    u32x2 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * r, v[4 * i + 1] * r, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * r, v[4 * i + 3] * r, w, true);
        o[i] = (uint32_t)w;
    }
    return o;
}

DEVI uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The maximum over 16 lanes of a row.
DEVI uint32_t max16(uint32_t v) {
    v = larger(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));
    v = larger(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));
    v = larger(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));
    return larger(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));
}

// A work-group takes 16 tokens and NB blocks.
template <int DT, int NB>
__global__ __launch_bounds__(256) void f8_tokens_kernel(const void *x, long long sb, long long sl, int L, FDiv by_length,
                                                        uint32_t tokens, int C, int blocks, unsigned char *q,
                                                        unsigned char *scale, int parts, uint32_t first) {
    typedef typename Elem<DT>::T T;
    const uint32_t id = first + blockIdx.x;
    const int part = id % parts, in = threadIdx.x & 15;
    const uint32_t token = id / parts * 16 + (threadIdx.x >> 4);
    if (token >= tokens) return;
    const int b = (int)fdiv(token, by_length), l = (int)token - b * L;
    const T *row = (const T *)x + (long long)b * sb + (long long)l * sl;
    float v[NB][8];
#pragma unroll
    for (int i = 0; i < NB; ++i) load8<DT>(row, (part * NB + i) * 128 + in * 8, C, v[i]);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int block = part * NB + i;
        if (block >= blocks) break;
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = larger(top, magnitude(v[i][e]));
        const uint32_t code = scale_code(max16(top));
        *(u32x2 *)(q + (size_t)token * blocks * 128 + block * 128 + in * 8) = pack8(v[i], code);
        if (in == 0) scale[(size_t)block * tokens + token] = (unsigned char)code;
    }
}

// A work-group takes 64 steps of one sequence and one block of channels: eight lanes of eight steps, 32 row groups of
// four channels.
template <int DT>
__global__ __launch_bounds__(256) void f8_rows_kernel(const void *x, long long sb, long long sc, int L, int tiles, int C,
                                                      int blocks, uint32_t tokens, unsigned char *q, unsigned char *scale,
                                                      uint32_t first) {
    typedef typename Elem<DT>::T T;
    __shared__ uint32_t red[32][64 + 1], code[64];
    __shared__ __attribute__((aligned(16))) unsigned char turned[64][128 + 16];
    const uint32_t id = first + blockIdx.x;
    const int tile = id % tiles, rest = id / tiles, block = rest % blocks, b = rest / blocks;
    const int g = threadIdx.x >> 3, t0 = tile * 64, tl = (threadIdx.x & 7) * 8;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = block * 128 + g * 4 + i;
        load8<DT>((const T *)x + (long long)b * sb + (long long)(c < C ? c : 0) * sc, t0 + tl, c < C ? L : 0, v[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = larger(top, magnitude(v[i][e]));
        red[g][tl + e] = top;
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = larger(top, red[i][threadIdx.x]);
        const uint32_t k = scale_code(top);
        code[threadIdx.x] = k;
        const int t = t0 + threadIdx.x;
        if (t < L) scale[(size_t)block * tokens + (size_t)b * L + t] = (unsigned char)k;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t k = code[tl + e];
        uint32_t w = 0x7f7f7f7fu;
        if (k != 255u) {
            const float r = scale_inverse(k);
            int two = __builtin_amdgcn_cvt_pk_fp8_f32(v[0][e] * r, v[1][e] * r, 0, false);
            w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2][e] * r, v[3][e] * r, two, true);
        }
        *(uint32_t *)&turned[tl + e][g * 4] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = i * 256 + threadIdx.x, t = at >> 3, piece = (at & 7) * 16;
        if (t0 + t < L)
            *(u32x4 *)(q + ((size_t)b * L + t0 + t) * blocks * 128 + block * 128 + piece) = *(const u32x4 *)&turned[t][piece];
    }
}

template <int DT>
int quantize(int B, int L, int C, const void *x, long long sb, long long sl, long long sc, unsigned char *q,
             unsigned char *scale, hipStream_t st) {
    const int blocks = (C + 127) / 128;
    const uint32_t tokens = (uint32_t)B * L;
    if (sc == 1 || C == 1) {
        constexpr int NB = 4;
        const int parts = (blocks + NB - 1) / NB;
        return launch_groups(((long long)tokens + 15) / 16 * parts, 256, [&](unsigned n, unsigned first) {
            hipLaunchKernelGGL((f8_tokens_kernel<DT, NB>), dim3(n), dim3(256), 0, st, x, sb, sl, L, make_fdiv((uint32_t)L),
                               tokens, C, blocks, q, scale, parts, first);
        });
    }
    const int tiles = (L + 63) / 64;
    return launch_groups((long long)B * tiles * blocks, 256, [&](unsigned n, unsigned first) {
        hipLaunchKernelGGL(f8_rows_kernel<DT>, dim3(n), dim3(256), 0, st, x, sb, sc, L, tiles, C, blocks, tokens, q, scale,
                           first);
    });
}

}  // namespace

int launch_quantize_f8(int B, int L, int C, int dtype, const void *x, long long sb, long long sl, long long sc,
                       unsigned char *q, unsigned char *scale, hipStream_t st) {
    return dtype == MICONV_BF16 ? quantize<1>(B, L, C, x, sb, sl, sc, q, scale, st)
                                : quantize<0>(B, L, C, x, sb, sl, sc, q, scale, st);
}

}  // namespace miconv
