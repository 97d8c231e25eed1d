// ssm_device.h -- device helpers of the state-space operators: loads and stores
// of eight consecutive time steps, exp / softplus / logistic in fp32.
#pragma once
#include "device.h"

namespace miconv {

// Rows start at any element, so vectors are aligned to the element only.
typedef uint32_t u32x4_row __attribute__((ext_vector_type(4), aligned(2)));

template <int DT>
struct Elem;
template <>
struct Elem<0> {
    typedef float T;
    static DEVI float get(float v) { return v; }
    static DEVI float put(float v) { return v; }
};
template <>
struct Elem<1> {
    typedef __bf16 T;
    static DEVI float get(__bf16 v) { return (float)v; }
    static DEVI __bf16 put(float v) { return (__bf16)v; }   // to nearest, ties to even
};

// v[i] = row[t + i] for t + i < end, 0 from end on (not loaded).  t >= 0.
template <int DT>
DEVI void load8(const typename Elem<DT>::T *row, int t, int end, float (&v)[8]) {
    if (__builtin_expect(t + 8 <= end, 1)) {
        if constexpr (DT == 1) {
            const u32x4 r = *(const u32x4_row *)(row + t);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(r[i] << 16);
                v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
            }
        } else {
            const u32x4 r0 = *(const u32x4_row *)(row + t), r1 = *(const u32x4_row *)(row + t + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(r0[i]);
                v[4 + i] = __uint_as_float(r1[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = t + i < end ? Elem<DT>::get(row[t + i]) : 0.0f;
    }
}

typedef uint32_t u32x2_row __attribute__((ext_vector_type(2), aligned(2)));

template <int DT>
DEVI void load4(const typename Elem<DT>::T *p, float (&v)[4]) {
    if constexpr (DT == 1) {
        const u32x2 r = *(const u32x2_row *)p;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    } else {
        const u32x4 r = *(const u32x4_row *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
    }
}

// The same as load8 in two steps: fetch8 issues the loads, widen8 takes their values later.
template <int DT>
struct Raw8 {
    u32x4 r[DT == 1 ? 1 : 2];
};

template <int DT>
DEVI Raw8<DT> fetch8(const typename Elem<DT>::T *row, int t, int end) {
    Raw8<DT> o;
    if (__builtin_expect(t + 8 <= end, 1)) {
        o.r[0] = *(const u32x4_row *)(row + t);
        if constexpr (DT == 0) o.r[1] = *(const u32x4_row *)(row + t + 4);
    } else {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0;
            if (t + i < end) {
                if constexpr (DT == 1)
                    v[i] = ((const uint16_t *)row)[t + i];
                else
                    v[i] = ((const uint32_t *)row)[t + i];
            }
        }
        if constexpr (DT == 1) {
            o.r[0] = pack<2>(v);
        } else {
            o.r[0] = pack<4>(v);
            o.r[1] = pack<4>(v + 4);
        }
    }
    return o;
}

template <int DT>
DEVI void widen8(const Raw8<DT> &o, float (&v)[8]) {
    if constexpr (DT == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(o.r[0][i] << 16);
            v[2 * i + 1] = __uint_as_float(o.r[0][i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(o.r[0][i]);
            v[4 + i] = __uint_as_float(o.r[DT == 0][i]);
        }
    }
}

template <bool STREAM>
DEVI void put_vec(u32x4 v, u32x4_row *to) {
    if constexpr (STREAM)
        __builtin_nontemporal_store(v, to);
    else
        *to = v;
}

// row[t + i] = v[i] for t + i < end.  STREAM: past the caches, see streams().
template <int DT, bool STREAM = false>
DEVI void store8(typename Elem<DT>::T *row, int t, int end, const float (&v)[8]) {
    if (__builtin_expect(t + 8 <= end, 1)) {
        if constexpr (DT == 1) {
            u32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                const bf16x2 p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
                r[i] = __builtin_bit_cast(uint32_t, p);
            }
            put_vec<STREAM>(r, (u32x4_row *)(row + t));
        } else {
            u32x4 r0, r1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r0[i] = __float_as_uint(v[i]);
                r1[i] = __float_as_uint(v[4 + i]);
            }
            put_vec<STREAM>(r0, (u32x4_row *)(row + t));
            put_vec<STREAM>(r1, (u32x4_row *)(row + t + 4));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + i < end) row[t + i] = Elem<DT>::put(v[i]);
    }
}

DEVI float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }
DEVI float rcp_hw(float v) { return __builtin_amdgcn_rcpf(v); }

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = 1.92596299112661746887e-8f;   // log2(e) - kLog2e
constexpr float kLn2 = 0.69314718055994530942f;

// exp(v) for v <= 0 with the rounding of v*log2(e) put right: the plain product
// is off by |v| 2^-24 relative.
DEVI float exp_neg(float v) {
    const float t = v * kLog2e;
    const float r = __builtin_fmaf(v, kLog2eLow, __builtin_fmaf(v, kLog2e, -t));
    const float e = exp2_hw(t);
    return v < -100.0f ? 0.0f : __builtin_fmaf(e, r * kLn2, e);
}

// 1 / (1 + exp(-v)), from exp(-|v|) so that neither end overflows.
DEVI float logistic(float v) {
    const float e = exp_neg(-__builtin_fabsf(v));
    const float r = rcp_hw(1.0f + e);
    return v < 0.0f ? e * r : r;
}

// The logistic function of gates and slopes, for operands of DT's type.  With bf16 operands
// the plain exponential serves, at a third of the instructions: its relative error |v| 2^-23
// stays far below the operands' own half step, 2^-9 (and that of a bf16 result).  exp(-v) = inf
// gives 0.
template <int DT>
DEVI float logistic_for(float v) {
    if constexpr (DT == 1)
        return rcp_hw(1.0f + exp2_hw(v * -kLog2e));
    else
        return logistic(v);
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], with
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3: s times a polynomial in s^2 whose relative
// error's extremes are equal, 2^-27 (the series itself would need three terms more).  No
// cancellation at either end.  The rounding of |v| log2(e) stays in: it is worth |v| 2^-24 of e,
// as much as half a step of v itself.  Found to be within 4 + |v| half steps of the result.
DEVI float softplus(float v) {
    const float e = exp2_hw(__builtin_fabsf(v) * -kLog2e);
    const float s = e * rcp_hw(2.0f + e), q = s * s;
    float p = 0.28178334f;
    p = __builtin_fmaf(p, q, 0.27960601f);
    p = __builtin_fmaf(p, q, 0.40024909f);
    p = __builtin_fmaf(p, q, 0.66666317f);
    p = __builtin_fmaf(p, q, 2.0f);
    const int bits = __float_as_int(v);        // its maximum with 0 is max(v, 0), in one instruction
    return __builtin_fmaf(s, p, __int_as_float(bits > 0 ? bits : 0));
}

// A log2(e), held to what fp32 has: a step of size 0 then decays by exp2(0 * that) = 1 rather
// than by exp2(0 * -inf), as the definition does for every finite A.
DEVI float log2_decay(float A) {
    const float a = A * kLog2e;
    return a < -__FLT_MAX__ ? -__FLT_MAX__ : a;
}

// Lane crossings of a wave of 64 in four rows of 16.
constexpr int kRowShr = 0x110;      // + n: lane i reads lane i - n of its row
constexpr int kRowShl = 0x100;      // + n: lane i reads lane i + n of its row
constexpr int kWaveShl1 = 0x130, kWaveShr1 = 0x138;
constexpr int kRowBcast15 = 0x142;  // rows 1..3 read the last lane of the row before
constexpr int kRowBcast31 = 0x143;  // rows 2, 3 read lane 31

// The crossing's source lane, or 0 where there is none.
template <int CTRL, int ROWS = 0xf>
DEVI float cross(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, ROWS == 0xf));
}
// The crossing's source lane, or `other` where there is none.
template <int CTRL>
DEVI float cross_or(float other, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(v), CTRL, 0xf, 0xf, false));
}
DEVI float lane_of(float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); }

// Sums of v over the lanes up to each one.
DEVI float prefix_sum(float v) {
    v += cross<kRowShr + 1>(v);
    v += cross<kRowShr + 2>(v);
    v += cross<kRowShr + 4>(v);
    v += cross<kRowShr + 8>(v);
    v += cross<kRowBcast15, 0xa>(v);
    return v + cross<kRowBcast31, 0xc>(v);
}

// Scans of the lanes' maps v -> p v + h (the product of a lane's decays, its state from zero):
// h becomes the state after the lane's steps, from the first lane's h on, which includes
// what entered it.  A step adds p times the source lane's h and multiplies p by its p; a lane
// without a source stays as it is.  Written as instructions, because the compiler takes two
// for the crossing and the fma where one does both.  A crossing may read a
// register that a vector instruction wrote only after two wait states, which the compiler does not
// count in here: between dependent instructions stand two others or an s_nop.
//
// Along each row of 16, h upwards and g downwards, both by p:
DEVI void scan_rows(float &h, float &g, float p) {
    float q = p;
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %0, %2 row_shr:1 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %1, %3 row_shl:1 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %2, %2, %2 row_shr:1 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %3, %3, %3 row_shl:1 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %0, %2 row_shr:2 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %1, %3 row_shl:2 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %2, %2, %2 row_shr:2 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %3, %3, %3 row_shl:2 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %0, %2 row_shr:4 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %1, %3 row_shl:4 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %2, %2, %2 row_shr:4 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %3, %3, %3 row_shl:4 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %0, %2 row_shr:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %1, %3 row_shl:8 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1"
        : "+v"(h), "+v"(g), "+v"(p), "+v"(q));
}

// Upwards, along each row of 16 or the whole wave:
template <int LANES>
DEVI float scan_lanes(float h, float p) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %0, %1 row_shr:1 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %1, %1, %1 row_shr:1 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 0\n\t"
        "v_fmac_f32_dpp %0, %0, %1 row_shr:2 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %1, %1, %1 row_shr:2 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 0\n\t"
        "v_fmac_f32_dpp %0, %0, %1 row_shr:4 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %1, %1, %1 row_shr:4 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 0\n\t"
        "v_fmac_f32_dpp %0, %0, %1 row_shr:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %1, %1, %1 row_shr:8 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 0"
        : "+v"(h), "+v"(p));
    if constexpr (LANES == 64)
        asm("s_nop 0\n\t"
            "v_fmac_f32_dpp %0, %0, %1 row_bcast:15 row_mask:0xa bank_mask:0xf\n\t"
            "v_mul_f32_dpp %1, %1, %1 row_bcast:15 row_mask:0xa bank_mask:0xf\n\t"
            "s_nop 0\n\t"
            "v_fmac_f32_dpp %0, %0, %1 row_bcast:31 row_mask:0xc bank_mask:0xf\n\t"
            "s_nop 1"
            : "+v"(h), "+v"(p));
    return h;
}

// `held` with lane n's value replaced by lane 63's of v.  (The lane is read ahead of the choice:
// inside it only lane n would run, and v need not be computed in lane 63.)
DEVI float keep(float held, float v, int n) {
    const float last = lane_of(v, 63);
    return (int)(threadIdx.x & 63) == n ? last : held;
}

// v, of which the compiler does not know that it is: addresses made from it are made where
// they are used rather than held in registers through the turns.
DEVI int again(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Orders this wave's LDS accesses: what a lane wrote before is read by the others after.
DEVI void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// dt of n consecutive steps from t on, in place of delta; 0 (no decay) from `end` on, which only a
// chunk that reaches past it has to look at.
template <int N>
DEVI void step_sizes(float (&dt)[N], float bias, int use_softplus, int t, int chunk_end, int end) {
#pragma unroll
    for (int i = 0; i < N; ++i) dt[i] += bias;
    if (use_softplus) {
#pragma unroll
        for (int i = 0; i < N; ++i) dt[i] = softplus(dt[i]);
    }
    if (chunk_end > end) {
#pragma unroll
        for (int i = 0; i < N; ++i) dt[i] = t + i < end ? dt[i] : 0.0f;
    }
}

// Valid steps of sequence b among L from `first` on.
DEVI int valid_steps(const int *lengths, int b, int L, int first = 0) {
    if (!lengths) return L;
    const int n = (lengths[b] < 0 ? 0 : lengths[b]) - first;
    return n < 0 ? 0 : (n > L ? L : n);
}

}  // namespace miconv
