// delta_device.h -- device helpers of the gated delta rule: fp32 values as sums of bf16 planes, products of
// planes on 16x16x32 MFMAs.
#pragma once
#include "delta.h"
#include "ssm_device.h"

namespace miconv {

// Splits into planes are exact: a plane takes the eight leading bits of what the planes before it left (by
// truncation, so that nothing rounds up to infinity), and three hold all 24 bits of an fp32 value.  bf16
// operands are one plane.  The products of planes i and j with i + j <= ORDER are summed: for ORDER 2 what is left
// out is below 2^-24 of the product, so three bf16 planes stand for fp32 at 3 (one operand bf16) or 6 MFMAs, where
// the fp32 MFMA takes the time of 16.

constexpr int in_planes(int DT) { return DT == 1 ? 1 : 3; }

// Outputs of bf16 type (y, and the gradients of q, k and v) rest on sums to order 1: what is left out there, below
// 2^-16, is far under the half step of their type, 2^-8.
constexpr int out_order(int DT) { return DT == 1 ? 1 : 2; }

DEVI uint32_t upper_pair(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

DEVI float upper(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

// v[0..4) as planes; plane p's four values are out[p].
template <int N>
DEVI void split4(const float (&v)[4], u32x2 (&out)[N]) {
    float r[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int p = 0; p < N; ++p) {
        out[p] = u32x2{upper_pair(r[0], r[1]), upper_pair(r[2], r[3])};
        if (p + 1 < N) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] -= upper(r[i]);
        }
    }
}

template <int N>
DEVI void split8(const float (&v)[8], u32x4 (&out)[N]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
    for (int p = 0; p < N; ++p) {
        out[p] = u32x4{upper_pair(r[0], r[1]), upper_pair(r[2], r[3]), upper_pair(r[4], r[5]), upper_pair(r[6], r[7])};
        if (p + 1 < N) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] -= upper(r[i]);
        }
    }
}

// Planes of four values of a lane, and a lane's eight of a column or row operand, in LDS.
template <int N>
DEVI void put_planes(uint16_t *to, int plane, const float (&v)[4]) {
    u32x2 s[N];
    split4<N>(v, s);
#pragma unroll
    for (int p = 0; p < N; ++p) *(u32x2 *)(to + p * plane) = s[p];
}

template <int N>
DEVI void get_planes(const uint16_t *from, int plane, u32x4 (&v)[N]) {
#pragma unroll
    for (int p = 0; p < N; ++p) v[p] = *(const u32x4 *)(from + p * plane);
}

// acc += sum of a[i] b[j] over i + j <= ORDER, 32 deep.
template <int NA, int NB, int ORDER>
DEVI void multiply(const u32x4 (&a)[NA], const u32x4 (&b)[NB], f32x4 &acc) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j <= ORDER)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[i]),
                                                              __builtin_bit_cast(bf16x8, b[j]), acc, 0, 0, 0);
}

// A lane's 16 bytes of every plane of fragment `frag`; planes are `plane` bytes apart.
template <int N>
DEVI void fragment(const char *at, int frag, int plane, u32x4 (&v)[N]) {
#pragma unroll
    for (int p = 0; p < N; ++p) v[p] = *(const u32x4 *)(at + p * plane + frag * 1024 + (threadIdx.x & 63) * 16);
}

// Four consecutive elements of a row, zeros from `end` on (not loaded).
template <int DT>
DEVI void load4_until(const typename Elem<DT>::T *row, int t, int end, float (&v)[4]) {
    if (__builtin_expect(t + 4 <= end, 1)) {
        load4<DT>(row + t, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = t + i < end ? Elem<DT>::get(row[t + i]) : 0.0f;
    }
}

// row[t + i] = v[i] for t + i < end.
template <int DT>
DEVI void store4_until(typename Elem<DT>::T *row, int t, int end, const float (&v)[4]) {
    if (__builtin_expect(t + 4 <= end, 1)) {
        if constexpr (DT == 1) {
            u32x2 r;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                const bf16x2 p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
                r[i] = __builtin_bit_cast(uint32_t, p);
            }
            *(u32x2_row *)(row + t) = r;
        } else {
            u32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
            *(u32x4_row *)(row + t) = r;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i < end) row[t + i] = Elem<DT>::put(v[i]);
    }
}

template <int DT>
DEVI typename Elem<DT>::T *row_of(const miconv_rows_t &r, int b, int d) {
    return (typename Elem<DT>::T *)r.data + (long long)b * r.stride_b + (long long)d * r.stride_d;
}

// exp for arguments of either sign; the products' rounding is put right for negative ones.
DEVI float exp_any(float v) { return v <= 0.0f ? exp_neg(v) : exp2_hw(v * kLog2e); }

}  // namespace miconv
