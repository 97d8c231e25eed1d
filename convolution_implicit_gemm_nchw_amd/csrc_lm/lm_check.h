// lm_check.h -- what the entry points of the language-model operators check before anything is
// enqueued: sizes, strides, alignment, and operands that share memory.
#pragma once
#include <stdint.h>

#include "../../include/miconv.h"

namespace miconv {

constexpr long long kMaxSize = 1ll << 30;
// No tensor spans this many elements: products of sizes and strides cannot overflow.
constexpr __int128 kMaxSpan = (__int128)1 << 46;

inline bool bad_size(long long v) { return v < 1 || v > kMaxSize; }

// A strided tensor's place in memory: nb x nd rows of L elements.
struct Span {
    uintptr_t at;
    long long nb, sb, nd, sd, L;
    size_t es;
    size_t bytes() const { return (size_t)((nb - 1) * sb + (nd - 1) * sd + L) * es; }
};

inline Span flat(const void *p, size_t n, size_t es) { return {(uintptr_t)p, 1, 0, 1, 0, (long long)n, es}; }

inline int check_span(const Span &s) {
    if (s.sb < 0 || s.sd < 0) return MICONV_ERR_BAD_DIM;
    const __int128 n = (__int128)(s.nb - 1) * s.sb + (__int128)(s.nd - 1) * s.sd + s.L;
    if (n > kMaxSpan) return MICONV_ERR_TOO_LARGE;
    return s.at % s.es ? MICONV_ERR_ALIGN : MICONV_OK;
}

// Rows of an output must not overlap each other (either axis may be the outer one).
inline int check_out_rows(const Span &s) {
    const __int128 in_b = (__int128)(s.nd - 1) * s.sd + s.L, in_d = (__int128)(s.nb - 1) * s.sb + s.L;
    const bool b_outer = (s.nd == 1 || s.sd >= s.L) && (s.nb == 1 || s.sb >= in_b);
    const bool d_outer = (s.nb == 1 || s.sb >= s.L) && (s.nd == 1 || s.sd >= in_d);
    return b_outer || d_outer ? MICONV_OK : MICONV_ERR_BAD_DIM;
}

// The bytes that a tensor's rows cover modulo `period`, from its first on: an axis whose stride
// is a multiple of it adds none.
inline long long window(const Span &s, long long period) {
    const long long es = (long long)s.es, b = (s.nb - 1) * s.sb * es, d = (s.nd - 1) * s.sd * es;
    return s.L * es + (s.sb * es % period ? b : 0) + (s.sd * es % period ? d : 0);
}

// Whether two tensors share memory.  Ranges that interleave are told apart where one of their strides
// repeats both, each in a part of its own: halves of one projection, or slices along time of one buffer.
inline bool share(const Span &a, const Span &b) {
    if (!a.at || !b.at) return false;
    const size_t an = a.bytes(), bn = b.bytes();
    if (a.at + an <= b.at || b.at + bn <= a.at) return false;
    const long long es_a = (long long)a.es, es_b = (long long)b.es;
    for (const long long period : {a.sb * es_a, a.sd * es_a, b.sb * es_b, b.sd * es_b}) {
        if (period <= 0) continue;
        long long off = (long long)(b.at - a.at) % period;
        if (off < 0) off += period;
        if (off >= window(a, period) && off + window(b, period) <= period) return false;
    }
    return true;
}

inline Span rows_span(const miconv_rows_t &r, int B, int D, int L, size_t es) {
    return {(uintptr_t)r.data, B, r.stride_b, D, r.stride_d, L, es};
}

struct Checker {
    Span in[24], out[16];
    int ni = 0, no = 0, status = MICONV_OK;
    void fail(int s) {
        if (status == MICONV_OK) status = s;
    }
    void input(const Span &s, bool required) {
        if (!s.at) {
            if (required) fail(MICONV_ERR_NULL);
            return;
        }
        fail(check_span(s));
        in[ni++] = s;
    }
    void output(const Span &s, bool required) {
        if (!s.at) {
            if (required) fail(MICONV_ERR_NULL);
            return;
        }
        fail(check_span(s));
        if (status == MICONV_OK) fail(check_out_rows(s));
        out[no++] = s;
    }
    int done() {
        if (status != MICONV_OK) return status;
        for (int i = 0; i < no; ++i) {
            for (int j = 0; j < ni; ++j)
                if (share(out[i], in[j])) return MICONV_ERR_ALIAS;
            for (int j = 0; j < i; ++j)
                if (share(out[i], out[j])) return MICONV_ERR_ALIAS;
        }
        return MICONV_OK;
    }
};

inline bool bad_dtype(int d) { return d != MICONV_F32 && d != MICONV_BF16; }
inline size_t elem_size(int d) { return d == MICONV_BF16 ? 2 : 4; }

}  // namespace miconv
