// delta_device.h -- device helpers of the gated delta rule: fp32 values as sums of bf16 planes, products of
// planes on 16x16x32 MFMAs.
#pragma once
#include "delta.h"
#include "ssm_device.h"

namespace miconv {

// Splits into planes are exact: a plane takes eight bits of what the planes before it left, and three hold all 24 of
// an fp32 value.  The first is cut, so that nothing rounds up to infinity, the second rounded to nearest, so that what
// the products leave out has either sign (cut, it is of one, 2^-25 of every product on average).  bf16 operands are one plane.  The products of planes i and j with i + j <= ORDER are summed: for ORDER 2 what is left
// out is below 2^-24 of the product, so three bf16 planes stand for fp32 at 3 (one operand bf16) or 6 MFMAs, where
// the fp32 MFMA takes the time of 16.

constexpr int in_planes(int DT) { return DT == 1 ? 1 : 3; }

DEVI uint32_t upper_pair(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

DEVI float upper(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

// Plane p of N of two values, which keep what is left of them.
template <int N>
DEVI uint32_t take_plane(int p, float &lo, float &hi) {
    if (p == 0 || p + 1 == N) {
        const uint32_t o = upper_pair(lo, hi);
        lo -= upper(lo);
        hi -= upper(hi);
        return o;
    }
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 near = {(__bf16)lo, (__bf16)hi};
    const uint32_t o = __builtin_bit_cast(uint32_t, near);
    lo -= __uint_as_float(o << 16);
    hi -= __uint_as_float(o & 0xffff0000u);
    return o;
}

// v[0..4) as planes; plane p's four values are out[p].
template <int N>
DEVI void split4(const float (&v)[4], u32x2 (&out)[N]) {
    float r[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int p = 0; p < N; ++p) out[p] = u32x2{take_plane<N>(p, r[0], r[1]), take_plane<N>(p, r[2], r[3])};
}

template <int N>
DEVI void split8(const float (&v)[8], u32x4 (&out)[N]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
    for (int p = 0; p < N; ++p)
        out[p] = u32x4{take_plane<N>(p, r[0], r[1]), take_plane<N>(p, r[2], r[3]), take_plane<N>(p, r[4], r[5]),
                       take_plane<N>(p, r[6], r[7])};
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

// The same with a sum for each order, for a few products that the next step waits for: an MFMA's sum is ready only
// several issues later, and the orders' chains run side by side.
template <int ORDER>
struct Sums {
    f32x4 s[ORDER + 1];
    DEVI Sums() {
#pragma unroll
        for (int i = 0; i <= ORDER; ++i) s[i] = f32x4{0, 0, 0, 0};
    }
    template <int NA, int NB>
    DEVI void add(const u32x4 (&a)[NA], const u32x4 (&b)[NB]) {
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (i + j <= ORDER)
                    s[i + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[i]),
                                                                       __builtin_bit_cast(bf16x8, b[j]), s[i + j], 0, 0, 0);
    }
    // Read here, not where the total is used.  In the scans no branch lies between the products and this, and the compiler
    // counts the states in between right; where one does, settle(s) goes first.
    DEVI f32x4 total() const {
        f32x4 t = s[ORDER];
#pragma unroll
        for (int i = ORDER - 1; i >= 0; --i) t += s[i];
        asm volatile("" : "+v"(t));
        return t;
    }
};

template <bool W>
struct Whole {
    static constexpr bool value = W;
};

// Consecutive steps of one row as they stand, zeros from `end` on.  `whole` says for the whole wave that none lies
// there: a branch per lane would wait for its load before the other side could run.
template <int DT>
DEVI Raw8<DT> steps8(const typename Elem<DT>::T *row, bool whole, int t, int end) {
    if (!whole) return fetch8<DT>(row, t, end);
    Raw8<DT> o;
    o.r[0] = *(const u32x4_row *)(row + t);
    if constexpr (DT == 0) o.r[1] = *(const u32x4_row *)(row + t + 4);
    return o;
}

template <int DT>
struct Raw4 {
    uint32_t r[DT == 1 ? 2 : 4];
};
template <int DT>
DEVI Raw4<DT> steps4(const typename Elem<DT>::T *row, bool whole, int t, int end) {
    Raw4<DT> o;
    if (whole) {
        if constexpr (DT == 1) {
            const u32x2 v = *(const u32x2_row *)(row + t);
            o.r[0] = v[0];
            o.r[1] = v[1];
        } else {
            const u32x4 v = *(const u32x4_row *)(row + t);
#pragma unroll
            for (int i = 0; i < 4; ++i) o.r[i] = v[i];
        }
        return o;
    }
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = 0;
        if (t + i < end) {
            if constexpr (DT == 1)
                v[i] = ((const uint16_t *)row)[t + i];
            else
                v[i] = ((const uint32_t *)row)[t + i];
        }
    }
    if constexpr (DT == 1) {
        o.r[0] = v[0] | v[1] << 16;
        o.r[1] = v[2] | v[3] << 16;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o.r[i] = v[i];
    }
    return o;
}
// Their values, or zeros where `in` is false: of a row that stands for one past the tensor's.
template <int DT>
DEVI void widen4(const Raw4<DT> &o, bool in, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = DT == 0 ? o.r[i & (DT == 0 ? 3 : 1)] : (i & 1 ? o.r[i >> 1] & 0xffff0000u : o.r[i >> 1] << 16);
        v[i] = in ? __uint_as_float(u) : 0.0f;
    }
}
template <int DT>
DEVI Raw8<DT> only(const Raw8<DT> &o, bool in) {
    Raw8<DT> r;
#pragma unroll
    for (int h = 0; h < (DT == 1 ? 1 : 2); ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) r.r[h][i] = in ? o.r[h][i] : 0u;
    return r;
}
template <int DT>
DEVI void planes_of(const Raw8<DT> &r, u32x4 (&v)[in_planes(DT)]) {
    if constexpr (DT == 1) {
        v[0] = r.r[0];
    } else {
        float f[8];
        widen8<DT>(r, f);
        split8<3>(f, v);
    }
}

// A lane's 16 bytes of every plane of fragment `frag`; planes are `plane` bytes apart.
template <int N>
DEVI void fragment(const char *at, int frag, int plane, u32x4 (&v)[N]) {
#pragma unroll
    for (int p = 0; p < N; ++p) v[p] = *(const u32x4 *)(at + p * plane + frag * 1024 + (threadIdx.x & 63) * 16);
}

// row[t + i] = v[i] for t + i < end; `whole` as for steps8.
template <int DT>
DEVI void store4_until(typename Elem<DT>::T *row, bool whole, int t, int end, const float (&v)[4]) {
    if (whole) {
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
