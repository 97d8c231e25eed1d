// tile_store.h -- where a product's tile puts its values: token-major rows, or channel-major lines of L tokens.
#pragma once
#include "ssm_device.h"

namespace miconv {

// Eight consecutive values of row r of y [NR][NC] from c0 on: at y[r * row + c], or with len > 0
// at y[((c / len) * NR + r) * len + c % len].
template <int OD, bool STREAM>
DEVI void store_row8(void *out, long long row, int len, const FDiv &fd_len, int NC, int NR, int r, int c0,
                     const float (&v)[8]) {
    typedef typename Elem<OD>::T T;
    T *y = (T *)out;
    if (len == 0) {
        store8<OD, STREAM>(y + (long long)r * row, c0, NC, v);
        return;
    }
    const int b = (int)fdiv((uint32_t)c0, fd_len), l = c0 - b * len;
    T *line = y + ((long long)b * NR + r) * len;
    if (l + 8 <= len) {
        store8<OD, STREAM>(line, l, len, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = c0 + i;
        if (c >= NC) break;
        const int bi = (int)fdiv((uint32_t)c, fd_len);
        y[((long long)bi * NR + r) * len + (c - bi * len)] = Elem<OD>::put(v[i]);
    }
}

}  // namespace miconv
