// causal_conv.hip -- short causal depthwise convolution on [B][D][L] with bias
// and SiLU: forward, backward and one-token step.
//
//   u[t] = bias + sum_k w[k] x~[t-K+1+k],  y = u * sigmoid(u)
//
// Memory bound: an element is read and written once (backward: x and dy read, dx
// written) for 2K multiply-adds.  4 x 4096 x 2048, K 4, bf16: forward 31 us (4.3 TB/s), backward
// 46 us (4.3 TB/s).  A thread takes eight consecutive time steps of
// one row, so one 16-byte load (bf16) brings its own steps and a second, which
// the neighbouring lane has loaded too, the K-1 before them; taps and bias stay
// in registers.  K is a template argument: the tap loops unroll.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int kThreads = 256;

// The eight steps before t (x~ at t < 0 from the initial state).  t is a multiple of 8.
template <int DT, int K>
DEVI void load_before(const typename Elem<DT>::T *row, const typename Elem<DT>::T *init, int t, int end,
                      float (&v)[8]) {
    if (t > 0) {
        load8<DT>(row, t - 8, end, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (init && i >= 9 - K) ? Elem<DT>::get(init[i - (9 - K)]) : 0.0f;
    }
}

// x~ with the initial state in front: full[f], f = 0 .. n + K - 2.
template <int DT, int K>
DEVI float full_at(const typename Elem<DT>::T *row, const typename Elem<DT>::T *init, int f) {
    if (f >= K - 1) return Elem<DT>::get(row[f - (K - 1)]);
    return init ? Elem<DT>::get(init[f]) : 0.0f;
}

// 2^lg_tpr threads per row.  WAVE: a row takes whole waves, so that what belongs to it
// (addresses, taps, bias) is scalar.
template <int DT, int K, bool WAVE, bool STREAM>
__global__ __launch_bounds__(kThreads) void causal_fwd_kernel(miconv_causal_conv_t c, int lg_tpr, FDiv fd_D, uint32_t first) {
    typedef typename Elem<DT>::T T;
    const int sub = threadIdx.x & ((1 << lg_tpr) - 1);
    const int rib = WAVE ? uniform(threadIdx.x >> lg_tpr) : threadIdx.x >> lg_tpr;
    const long long row64 = (long long)(first + blockIdx.x) * (kThreads >> lg_tpr) + rib;
    if (row64 >= (long long)c.B * c.D) return;
    const int row = (int)row64, b = WAVE ? uniform((int)fdiv(row, fd_D)) : (int)fdiv(row, fd_D), d = row - b * c.D;
    const int len = valid_steps(c.lengths, b, c.L);
    const T *x = (const T *)c.x.data + b * c.x.stride_b + d * c.x.stride_d;
    const T *init = c.initial_state ? (const T *)c.initial_state + (long long)row * (K - 1) : nullptr;
    T *y = (T *)c.y.data + b * c.y.stride_b + d * c.y.stride_d;
    float w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = Elem<DT>::get(((const T *)c.w)[(long long)d * K + k]);
    const float bias = c.bias ? c.bias[d] : 0.0f;
    for (long long t64 = (((long long)blockIdx.y << lg_tpr) + sub) * 8; t64 < c.L;
         t64 += ((long long)gridDim.y << lg_tpr) * 8) {
        const int t = (int)t64;
        float out[8] = {};
        if (t < len) {
            float v[16];
            float (&before)[8] = *(float (*)[8])v, (&own)[8] = *(float (*)[8])(v + 8);
            load8<DT>(x, t, len, own);
            load_before<DT, K>(x, init, t, len, before);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float u = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) u = __builtin_fmaf(w[k], v[8 + i - (K - 1) + k], u);
                out[i] = t + i < len ? (c.silu ? u * logistic_for<DT>(u) : u) : 0.0f;
            }
        }
        store8<DT, STREAM>(y, t, c.L, out);
        if (t == 0 && c.final_state) {
            T *fs = (T *)c.final_state + (long long)row * (K - 1);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) fs[j] = Elem<DT>::put(full_at<DT, K>(x, init, len + j));
        }
    }
}

// One work-group: channel d, items [split * per, ...) of the B * tiles eight-step tiles.
// dx needs du of the K-1 steps after its own, which the next lane has: a wave takes 63
// consecutive tiles, and its last lane only computes du for the one before.  (Computing
// those steps again instead takes two more loads and (K-1)/8 more gates per step: 16 x 2048
// x 1024, K 4, bf16: 60 us.)  A thread keeps its part of dw and dbias; the parts are added
// in a fixed tree and written to part[split][d][K+1] (or dw, dbias).
// A step past the end (du = 0) stands before values of its window that belong to the sequence: without
// SILU it is left out of dw, so that an infinity among them stays in its own tap.  With SILU such a
// value has made du of its last step NaN, and with it all taps (selects there cost 8 %: 3 x 1001 x 1533).
template <int DT, int K, bool SILU>
__global__ __launch_bounds__(kThreads) void causal_bwd_kernel(miconv_causal_conv_t c, int tiles, long long per, int splits,
                                                        float *part, uint32_t first_channel) {
    typedef typename Elem<DT>::T T;
    __shared__ float red[kThreads / 64][K + 1];
    const int waves = blockDim.x >> 6, step = waves * 63, d = first_channel + blockIdx.x, split = blockIdx.y;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const long long items = (long long)c.B * tiles;
    const long long first = split * per, last = first + per < items ? first + per : items;
    float w[K], dw[K], db = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        w[k] = Elem<DT>::get(((const T *)c.w)[(long long)d * K + k]);
        dw[k] = 0.0f;
    }
    const float bias = c.bias ? c.bias[d] : 0.0f;
    const long long mine = first + wave * 63 + lane;
    int b = (int)(mine / tiles), tile = (int)(mine - (long long)b * tiles);
    const int step_b = step / tiles, step_t = step - step_b * tiles;
    for (long long base = first + wave * 63; base < last; base += step) {
        const long long it = base + lane;
        const bool there = it < items, counts = lane < 63 && it < last;
        const int t = tile * 8, bb = there ? b : 0;
        const int len = there ? valid_steps(c.lengths, bb, c.L) : 0;
        const long long row = (long long)bb * c.D + d;
        const T *init = c.initial_state ? (const T *)c.initial_state + row * (K - 1) : nullptr;
        float v[16], g[8 + K];                 // x~ of the eight steps before and of these; du
        if (t < len) {
            const T *x = (const T *)c.x.data + bb * c.x.stride_b + d * c.x.stride_d;
            const T *dy = (const T *)c.dy.data + bb * c.dy.stride_b + d * c.dy.stride_d;
            load_before<DT, K>(x, init, t, len, *(float (*)[8])v);
            load8<DT>(x, t, len, *(float (*)[8])(v + 8));
            load8<DT>(dy, t, len, *(float (*)[8])g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!SILU) continue;
                float u = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) u = __builtin_fmaf(w[k], v[8 + i - (K - 1) + k], u);
                const float sg = logistic_for<DT>(u);
                // a step past the end has du = 0 whatever u is there
                g[i] = t + i < len ? g[i] * (sg * __builtin_fmaf(u, 1.0f - sg, 1.0f)) : 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = v[i] = v[8 + i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const float next = cross<kWaveShl1>(g[i]);
            g[8 + i] = tile + 1 < tiles ? next : 0.0f;
        }
        if (counts) {
            const T *dfs = c.d_final_state ? (const T *)c.d_final_state + row * (K - 1) : nullptr;
            float out[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    s = __builtin_fmaf(w[k], g[i + K - 1 - k], s);
                    if (SILU) dw[k] = __builtin_fmaf(g[i], v[8 + i - (K - 1) + k], dw[k]);
                }
                db += g[i];
                const int j = t + i - len + K - 1;   // final_state[j] is x[t + i]
                if (dfs && j >= 0 && t + i < len) s += Elem<DT>::get(dfs[j]);
                out[i] = t + i < len ? s : 0.0f;
            }
            if constexpr (!SILU) {
                const int own = len - t;
                if (own >= 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k] = __builtin_fmaf(g[i], v[8 + i - (K - 1) + k], dw[k]);
                } else {
#pragma unroll
                    for (int i = 0; i < 7; ++i)
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            dw[k] = i < own ? __builtin_fmaf(g[i], v[8 + i - (K - 1) + k], dw[k]) : dw[k];
                }
            }
            if (c.dx.data) store8<DT>((T *)c.dx.data + bb * c.dx.stride_b + d * c.dx.stride_d, t, c.L, out);
            if (t == 0 && c.d_initial_state) {
                T *di = (T *)c.d_initial_state + row * (K - 1);
#pragma unroll
                for (int f = 0; f < K - 1; ++f) {
                    float s = 0.0f;
#pragma unroll
                    for (int u = 0; u <= f; ++u) s = __builtin_fmaf(w[f - u], g[u], s);
                    if (dfs && f >= len) s += Elem<DT>::get(dfs[f - len]);
                    di[f] = Elem<DT>::put(s);
                }
            }
        }
        b += step_b;
        tile += step_t;
        if (tile >= tiles) {
            tile -= tiles;
            ++b;
        }
    }
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        float s = k < K ? dw[k < K ? k : 0] : db;
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
        if (lane == 0) red[wave][k] = s;
    }
    __syncthreads();
    if (threadIdx.x <= K) {
        float s = 0.0f;
        for (int i = 0; i < waves; ++i) s += red[i][threadIdx.x];
        if (splits > 1) {
            part[((long long)split * c.D + d) * (K + 1) + threadIdx.x] = s;
        } else if (threadIdx.x < K) {
            if (c.dw) c.dw[(long long)d * K + threadIdx.x] = s;
        } else if (c.dbias) {
            c.dbias[d] = s;
        }
    }
}

__global__ __launch_bounds__(kThreads) void causal_bwd_reduce(const float *part, float *dw, float *dbias, int D, int K,
                                                              int splits) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x, n = (long long)D * (K + 1);
    if (i >= n) return;
    float s = 0.0f;
    for (int z = 0; z < splits; ++z) s += part[z * n + i];
    const int d = (int)(i / (K + 1)), k = (int)(i - (long long)d * (K + 1));
    if (k < K) {
        if (dw) dw[(long long)d * K + k] = s;
    } else if (dbias) {
        dbias[d] = s;
    }
}

// One thread per (sequence, channel): all reads of a state come before its writes,
// so state_out may be state.
template <int DT, int K>
__global__ __launch_bounds__(kThreads) void causal_step_kernel(int B, int D, int silu, miconv_rows_t x,
                                                               const typename Elem<DT>::T *state, int slots,
                                                               const int *slot_of, const typename Elem<DT>::T *w,
                                                               const float *bias, typename Elem<DT>::T *state_out,
                                                               miconv_rows_t y, FDiv fd_D) {
    typedef typename Elem<DT>::T T;
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;                   // rows are at most 2^30
    if (i >= (uint32_t)B * (uint32_t)D) return;
    const int b = (int)fdiv(i, fd_D), d = (int)i - b * D;
    const int slot = slot_of ? slot_of[b] : b;
    T *yo = (T *)y.data + b * y.stride_b + d * y.stride_d;
    if (slot < 0 || slot >= slots) {
        *yo = Elem<DT>::put(0.0f);
        return;
    }
    const long long so = ((long long)slot * D + d) * (K - 1);
    float v[K], u = bias ? bias[d] : 0.0f;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) v[k] = Elem<DT>::get(state[so + k]);
    v[K - 1] = Elem<DT>::get(((const T *)x.data)[b * x.stride_b + d * x.stride_d]);
#pragma unroll
    for (int k = 0; k < K; ++k) u = __builtin_fmaf(w[(long long)d * K + k] , v[k], u);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) state_out[so + k] = Elem<DT>::put(v[k + 1]);
    *yo = Elem<DT>::put(silu ? u * logistic_for<DT>(u) : u);
}

int lg2_up(long long v, int most) {
    int l = 0;
    while (l < most && (1ll << l) < v) ++l;
    return l;
}

template <int DT, int K>
int fwd_k(const miconv_causal_conv_t &c, hipStream_t st) {
    const long long tiles = (c.L + 7) / 8;
    const int lg = lg2_up(tiles, 8);
    const long long rpb = kThreads >> lg, row_blocks = ((long long)c.B * c.D + rpb - 1) / rpb;
    const long long along = (tiles + (1ll << lg) - 1) >> lg;
    const FDiv fd = make_fdiv((uint32_t)c.D);
    const auto kern = lg < 6 ? causal_fwd_kernel<DT, K, false, false>
                             : (streams(DT, (size_t)c.B * c.D * c.L) ? causal_fwd_kernel<DT, K, true, DT == 1>
                                                                     : causal_fwd_kernel<DT, K, true, false>);
    return launch_groups(row_blocks, kThreads, [&](unsigned n, unsigned first) {
        hipLaunchKernelGGL(kern, dim3(n, (unsigned)(along < 65535 ? along : 65535)), dim3(kThreads), 0, st, c, lg, fd, first);
    });
}

template <int DT, int K>
int bwd_k(const miconv_causal_conv_t &c, int splits, float *ws, hipStream_t st) {
    const int tiles = (c.L + 7) / 8;
    const long long items = (long long)c.B * tiles, per = (items + splits - 1) / splits;
    // up to four waves; fewer only where they hold all of a channel's tiles at once
    const int waves = per >= 4 * 63 ? 4 : (int)((per + 62) / 63);
    const auto kern = c.silu ? causal_bwd_kernel<DT, K, true> : causal_bwd_kernel<DT, K, false>;
    const int bad = launch_groups(c.D, waves * 64, [&](unsigned n, unsigned first) {
        hipLaunchKernelGGL(kern, dim3(n, splits), dim3(waves * 64), 0, st, c, tiles, per, splits, ws,
                           first);
    });
    if (bad != MICONV_OK) return bad;
    if (splits > 1 && (c.dw || c.dbias)) {
        const long long n = (long long)c.D * (K + 1);
        hipLaunchKernelGGL(causal_bwd_reduce, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                           ws, c.dw, c.dbias, c.D, K, splits);
        if (hipGetLastError() != hipSuccess) return MICONV_ERR_HIP;
    }
    return MICONV_OK;
}

template <int DT, int K>
int step_k(int B, int D, int silu, miconv_rows_t x, const void *state, int slots, const int *slot_of, const void *w,
           const float *bias, void *state_out, miconv_rows_t y, hipStream_t st) {
    typedef typename Elem<DT>::T T;
    const long long n = (long long)B * D;
    hipLaunchKernelGGL((causal_step_kernel<DT, K>), dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       st, B, D, silu, x, (const T *)state, slots, slot_of, (const T *)w, bias, (T *)state_out, y,
                       make_fdiv((uint32_t)D));
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

}  // namespace

// Enough work-groups per channel to fill 256 CUs four deep, each with at least
// 256 tiles of eight steps; fewer where the partial sums do not fit the budget.  (16 x 64 rows of
// 8192, bf16: 23 us split 16 ways, 122 whole; 8 x 512 of 2048: 20.6 in two, 23.4 whole.)
int causal_bwd_splits(const miconv_causal_conv_t &c, size_t budget) {
    const long long items = (long long)c.B * ((c.L + 7) / 8), one = (long long)c.D * (c.K + 1) * 4;
    long long s = 1024 / c.D;
    if (s > items / 256) s = items / 256;
    if (s > 64) s = 64;
    if (s > (long long)(budget / (size_t)one)) s = (long long)(budget / (size_t)one);
    return s < 1 ? 1 : (int)s;
}

#define MICONV_BY_TAPS(F, ...)                                      \
    switch (K) {                                                    \
        case 1: return dtype ? F<1, 1>(__VA_ARGS__) : F<0, 1>(__VA_ARGS__); \
        case 2: return dtype ? F<1, 2>(__VA_ARGS__) : F<0, 2>(__VA_ARGS__); \
        case 3: return dtype ? F<1, 3>(__VA_ARGS__) : F<0, 3>(__VA_ARGS__); \
        case 4: return dtype ? F<1, 4>(__VA_ARGS__) : F<0, 4>(__VA_ARGS__); \
        case 5: return dtype ? F<1, 5>(__VA_ARGS__) : F<0, 5>(__VA_ARGS__); \
        case 6: return dtype ? F<1, 6>(__VA_ARGS__) : F<0, 6>(__VA_ARGS__); \
        case 7: return dtype ? F<1, 7>(__VA_ARGS__) : F<0, 7>(__VA_ARGS__); \
        case 8: return dtype ? F<1, 8>(__VA_ARGS__) : F<0, 8>(__VA_ARGS__); \
        default: return MICONV_ERR_BAD_DIM;                         \
    }

int launch_causal_fwd(const miconv_causal_conv_t &c, int dtype, hipStream_t st) {
    const int K = c.K;
    MICONV_BY_TAPS(fwd_k, c, st)
}

int launch_causal_bwd(const miconv_causal_conv_t &c, int dtype, int splits, float *ws, hipStream_t st) {
    const int K = c.K;
    MICONV_BY_TAPS(bwd_k, c, splits, ws, st)
}

int launch_causal_step(int B, int D, int K, int silu, int dtype, miconv_rows_t x, const void *state, int slots,
                       const int *slot_of, const void *w, const float *bias, void *state_out, miconv_rows_t y,
                       hipStream_t st) {
    MICONV_BY_TAPS(step_k, B, D, silu, x, state, slots, slot_of, w, bias, state_out, y, st)
}

}  // namespace miconv
