// layer_norm.hip -- layer normalisation over the channels of each token, y = (x - m) r w + b with
// r = 1 / sqrt(var + eps), and its gradients: with h = dy w and n = (x - m) r,
//   dx = r (h - mean(h) - n mean(h n)),   dw = sum over tokens of dy n,   db = sum over tokens of dy.
// Memory bound: x (and dy) are read once, held in registers between the sums and the result.  8192 tokens of 4096 channels
// in bf16, tokens first, forward: 24.5 us, 134 MB at 5.5 TB/s.  8192 tokens of 2048, channel-major: forward 19.5 us, 67 MB at
// 3.4 TB/s, backward 31 us, 101 MB at 3.3: one or two work-groups a CU read all of theirs, then write all.
//
// The variance is the mean square of the differences from the mean, in a second run over the registers: no
// cancellation however large the mean.
#include "norm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

template <int DT>
DEVI typename Elem<DT>::T *token_of(const miconv_tokens_t &v, int b, int l) {
    return (typename Elem<DT>::T *)v.data + (long long)b * v.stride_b + (long long)l * v.stride_l;
}

// v[i] = p[c + i], `fill` where p is absent or past the channels.
DEVI void param8(const float *p, int c, int C, float fill, float (&v)[8]) {
    if (p) {
        load8<0>(p, c, C, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fill;
    }
}

// ------------------------------------------------------------------ tokens first
//
// A token's channels over the 64 lanes of a wave (ROW 64) or the threads of a work-group, eight neighbours each, VPT times.
template <int ROW>
struct Row {
    static constexpr int kThreads = ROW < 256 ? 256 : ROW, kTokens = kThreads / ROW, kWaves = ROW / 64;
};

// Sums over the threads of a token, in the same order for every call.
template <int ROW, int N>
DEVI void row_sum(float (&s)[N], float (*red)[2]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 32; o; o /= 2) s[i] += __shfl_xor(s[i], o);
    }
    if constexpr (ROW > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();                       // what was read before
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[wave][i] = s[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < ROW / 64; ++w) t += red[w][i];
            s[i] = t;
        }
    }
}

template <int DT, int ROW, int VPT>
__global__ __launch_bounds__(Row<ROW>::kThreads) void norm_fwd_kernel(miconv_layer_norm_t a, FDiv by_length, uint32_t first) {
    typedef Row<ROW> X;
    typedef typename Elem<DT>::T T;
    __shared__ float red[X::kWaves][2];
    const int in = threadIdx.x % ROW;
    const uint32_t token = (first + blockIdx.x) * X::kTokens + threadIdx.x / ROW;
    if (token >= (uint32_t)a.B * a.L) return;  // whole waves, and with one token per work-group none
    const int b = (int)fdiv(token, by_length), l = (int)token - b * a.L;
    T *const y = token_of<DT>(a.y, b, l);
    const bool valid = l < valid_steps(a.lengths, b, a.L);
    const T *const x = token_of<DT>(a.x, b, l);
    float v[VPT][8], s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        load8<DT>(x, (i * ROW + in) * 8, valid ? a.C : 0, v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[i][e];
    }
    row_sum<ROW, 1>(s, red);
    const float mean = s[0] / (float)a.C;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * ROW + in) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] = c + e < a.C ? v[i][e] - mean : 0.0f;
            s[0] = __builtin_fmaf(v[i][e], v[i][e], s[0]);
        }
    }
    row_sum<ROW, 1>(s, red);
    const float r = 1.0f / __builtin_sqrtf(s[0] / (float)a.C + a.eps);
    if (a.stats && in == 0) {
        a.stats[token] = mean;
        a.stats[(size_t)a.B * a.L + token] = r;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * ROW + in) * 8;
        if (c >= a.C) break;
        float w[8], g[8];
        param8(a.weight, c, a.C, 1.0f, w);
        param8(a.bias, c, a.C, 0.0f, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = valid ? __builtin_fmaf(v[i][e] * r, w[e], g[e]) : 0.0f;
        store8<DT>(y, c, a.C, v[i]);
    }
}

// Work-group p takes tokens p, p + parts, ... (ROW 64: four at a time, one a wave), its channels' sums of dw and db
// in registers; the four waves' sums are joined in LDS, which leaves a quarter of the rows to write and read again.
template <int DT, int ROW, int VPT>
__global__ __launch_bounds__(Row<ROW>::kThreads) void norm_bwd_kernel(miconv_layer_norm_t a, FDiv by_length, int parts,
                                                                      float *part) {
    typedef Row<ROW> X;
    typedef typename Elem<DT>::T T;
    __shared__ float red[X::kWaves][2];
    const int in = threadIdx.x % ROW, p = blockIdx.x * X::kTokens + threadIdx.x / ROW, step = parts * X::kTokens;
    float dw[VPT][8] = {}, db[VPT][8] = {};
    const uint32_t tokens = (uint32_t)a.B * a.L;
    for (uint32_t token = p; token < tokens; token += step) {
        const int b = (int)fdiv(token, by_length), l = (int)token - b * a.L;
        T *const dx = token_of<DT>(a.dx, b, l);
        const bool valid = l < valid_steps(a.lengths, b, a.L);
        if (!valid) {
            const float zeros[8] = {};
#pragma unroll
            for (int i = 0; i < VPT; ++i) store8<DT>(dx, (i * ROW + in) * 8, a.C, zeros);
            continue;
        }
        const T *const x = token_of<DT>(a.x, b, l), *const dy = token_of<DT>(a.dy, b, l);
        const float mean = a.stats[token], r = a.stats[(size_t)tokens + token];
        float n[VPT][8], h[VPT][8], s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * ROW + in) * 8;
            float w[8];
            load8<DT>(x, c, a.C, n[i]);
            load8<DT>(dy, c, a.C, h[i]);
            param8(a.weight, c, a.C, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[i][e] = c + e < a.C ? (n[i][e] - mean) * r : 0.0f;
                dw[i][e] = __builtin_fmaf(h[i][e], n[i][e], dw[i][e]);
                db[i][e] += h[i][e];
                h[i][e] *= w[e];
                s[0] += h[i][e];
                s[1] = __builtin_fmaf(h[i][e], n[i][e], s[1]);
            }
        }
        row_sum<ROW, 2>(s, red);
        s[0] /= (float)a.C;
        s[1] /= (float)a.C;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = r * (h[i][e] - s[0] - n[i][e] * s[1]);
            store8<DT>(dx, (i * ROW + in) * 8, a.C, h[i]);
        }
    }
    float *const mine = part + (size_t)blockIdx.x * 2 * a.C;
    if constexpr (X::kTokens > 1) {
        __shared__ float joined[X::kTokens][2][VPT * 64][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            *(f32x4 *)&joined[threadIdx.x / ROW][0][i * ROW + in][0] = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
            *(f32x4 *)&joined[threadIdx.x / ROW][0][i * ROW + in][4] = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
            *(f32x4 *)&joined[threadIdx.x / ROW][1][i * ROW + in][0] = f32x4{db[i][0], db[i][1], db[i][2], db[i][3]};
            *(f32x4 *)&joined[threadIdx.x / ROW][1][i * ROW + in][4] = f32x4{db[i][4], db[i][5], db[i][6], db[i][7]};
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.C; c += X::kThreads)
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                float t = 0.0f;
#pragma unroll
                for (int w = 0; w < X::kTokens; ++w) t += joined[w][which][c / 8][c % 8];
                mine[which * a.C + c] = t;
            }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        store8<0>(mine, (i * ROW + in) * 8, a.C, dw[i]);
        store8<0>(mine + a.C, (i * ROW + in) * 8, a.C, db[i]);
    }
}

// Tokens of more channels than registers hold: x is read again, from the caches, for each of the sums.
template <int DT>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(miconv_layer_norm_t a, FDiv by_length, uint32_t first) {
    typedef typename Elem<DT>::T T;
    __shared__ float red[16][2];
    const uint32_t token = first + blockIdx.x;
    const int b = (int)fdiv(token, by_length), l = (int)token - b * a.L;
    T *const y = token_of<DT>(a.y, b, l);
    const bool valid = l < valid_steps(a.lengths, b, a.L);
    const T *const x = token_of<DT>(a.x, b, l);
    const int end = valid ? a.C : 0;
    float v[8], s[1] = {0.0f};
    for (int c = threadIdx.x * 8; c < end; c += 8192) {
        load8<DT>(x, c, end, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e];
    }
    row_sum<1024, 1>(s, red);
    const float mean = s[0] / (float)a.C;
    s[0] = 0.0f;
    for (int c = threadIdx.x * 8; c < end; c += 8192) {
        load8<DT>(x, c, end, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = c + e < end ? v[e] - mean : 0.0f;
            s[0] = __builtin_fmaf(d, d, s[0]);
        }
    }
    row_sum<1024, 1>(s, red);
    const float r = 1.0f / __builtin_sqrtf(s[0] / (float)a.C + a.eps);
    if (a.stats && threadIdx.x == 0) {
        a.stats[token] = mean;
        a.stats[(size_t)a.B * a.L + token] = r;
    }
    for (int c = threadIdx.x * 8; c < a.C; c += 8192) {
        float w[8], g[8];
        load8<DT>(x, c, end, v);
        param8(a.weight, c, a.C, 1.0f, w);
        param8(a.bias, c, a.C, 0.0f, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = valid ? __builtin_fmaf((v[e] - mean) * r, w[e], g[e]) : 0.0f;
        store8<DT>(y, c, a.C, v);
    }
}

template <int DT>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(miconv_layer_norm_t a, FDiv by_length, int parts, float *part) {
    typedef typename Elem<DT>::T T;
    __shared__ float red[16][2];
    float *const mine = part + (size_t)blockIdx.x * 2 * a.C;      // each thread's own channels
    const uint32_t tokens = (uint32_t)a.B * a.L;
    bool begun = false;
    for (uint32_t token = blockIdx.x; token < tokens; token += parts) {
        const int b = (int)fdiv(token, by_length), l = (int)token - b * a.L;
        T *const dx = token_of<DT>(a.dx, b, l);
        const bool valid = l < valid_steps(a.lengths, b, a.L);
        const T *const x = token_of<DT>(a.x, b, l), *const dy = token_of<DT>(a.dy, b, l);
        const float mean = a.stats[token], r = a.stats[(size_t)tokens + token];
        float n[8], h[8], w[8], s[2] = {0.0f, 0.0f};
        for (int c = threadIdx.x * 8; valid && c < a.C; c += 8192) {
            float dw[8] = {}, db[8] = {};
            load8<DT>(x, c, a.C, n);
            load8<DT>(dy, c, a.C, h);
            param8(a.weight, c, a.C, 1.0f, w);
            if (begun) {
                load8<0>(mine, c, a.C, dw);
                load8<0>(mine + a.C, c, a.C, db);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float one = c + e < a.C ? (n[e] - mean) * r : 0.0f;
                dw[e] = __builtin_fmaf(h[e], one, dw[e]);
                db[e] += h[e];
                s[0] = __builtin_fmaf(h[e], w[e], s[0]);
                s[1] = __builtin_fmaf(h[e] * w[e], one, s[1]);
            }
            store8<0>(mine, c, a.C, dw);
            store8<0>(mine + a.C, c, a.C, db);
        }
        begun = begun || valid;
        row_sum<1024, 2>(s, red);
        s[0] /= (float)a.C;
        s[1] /= (float)a.C;
        for (int c = threadIdx.x * 8; c < a.C; c += 8192) {
            float out[8] = {};
            if (valid) {
                load8<DT>(x, c, a.C, n);
                load8<DT>(dy, c, a.C, h);
                param8(a.weight, c, a.C, 1.0f, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = r * (h[e] * w[e] - s[0] - (n[e] - mean) * r * s[1]);
            }
            store8<DT>(dx, c, a.C, out);
        }
    }
    if (!begun) {
        const float zeros[8] = {};
        for (int c = threadIdx.x * 8; c < a.C; c += 8192) {
            store8<0>(mine, c, a.C, zeros);
            store8<0>(mine + a.C, c, a.C, zeros);
        }
    }
}

// ------------------------------------------------------------------ channels first
//
// A work-group takes TL * 8 neighbouring time steps and all channels: TL lanes of eight steps along a row, the
// others on other rows, R of them each (channel g, g + groups, ...), held as they were read.  More channels than
// that (LOOP) are read again from the caches.
template <int TL>
DEVI void steps_sum(float (&s)[8], float (*red)[64]) {
    const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = 32; o >= TL; o /= 2) s[i] += __shfl_xor(s[i], o);
    }
    __syncthreads();
    if (lane < TL) {
#pragma unroll
        for (int i = 0; i < 8; ++i) red[wave][lane * 8 + i] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    for (int w = 0; w < waves; ++w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += red[w][(lane % TL) * 8 + i];
    }
}

// Eight steps of channel c from t on as they stand, zeros from `end` on and past the channels.  Threads whose steps
// are all inside take no branch per row.
template <int DT, int R>
DEVI void fetch_rows(const typename Elem<DT>::T *x, long long stride, int C, int c, int groups, int t, int end,
                     Raw8<DT> (&held)[R]) {
    if (__builtin_expect(t + 8 <= end, 1)) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int at = c + i * groups;
            const typename Elem<DT>::T *from = x + (long long)(at < C ? at : C - 1) * stride + t;
            held[i].r[0] = *(const u32x4_row *)from;
            if constexpr (DT == 0) held[i].r[1] = *(const u32x4_row *)(from + 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int at = c + i * groups;
            held[i] = fetch8<DT>(x + (long long)(at < C ? at : C - 1) * stride, t, end);
        }
    }
}

// v as read, of which the compiler does not know that it is what it widened before: it would hold that instead.
template <int DT>
DEVI Raw8<DT> unseen(Raw8<DT> v) {
    asm volatile("" : "+v"(v.r[0]));
    if constexpr (DT == 0) asm volatile("" : "+v"(v.r[1]));
    return v;
}

template <int DT, int TL, int R, bool LOOP>
__global__ __launch_bounds__(1024) void norm_rows_fwd_kernel(miconv_layer_norm_t a, int tiles, uint32_t first) {
    typedef typename Elem<DT>::T T;
    __shared__ float red[16][64];
    const int id = xcd_remap(blockIdx.x, gridDim.x) + first;     // neighbours share lines: on one XCD
    const int b = id / tiles, t0 = (id - b * tiles) * TL * 8, tl = threadIdx.x % TL, g = threadIdx.x / TL;
    const int groups = blockDim.x / TL, t = t0 + tl * 8, end = valid_steps(a.lengths, b, a.L);
    const T *const x = (const T *)a.x.data + (long long)b * a.x.stride_b;
    T *const y = (T *)a.y.data + (long long)b * a.y.stride_b;
    Raw8<DT> held[LOOP ? 1 : R];
    float s[8] = {}, mean[8], r[8], v[8];
    const auto row = [&](int i, int c) {
        if constexpr (LOOP)
            load8<DT>(x + (long long)c * a.x.stride_c, t, end, v);
        else
            widen8<DT>(unseen<DT>(held[i]), v);
    };
    constexpr int U = LOOP ? 1 : R;
    const int rows = LOOP ? (a.C + groups - 1) / groups : R;
    if constexpr (!LOOP) fetch_rows<DT, R>(x, a.x.stride_c, a.C, g, groups, t, end, held);
#pragma unroll U
    for (int i = 0; i < rows; ++i) {
        const int c = i * groups + g;
        if (c >= a.C) break;
        row(i, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
    steps_sum<TL>(s, red);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        mean[e] = s[e] / (float)a.C;
        s[e] = 0.0f;
    }
#pragma unroll U
    for (int i = 0; i < rows; ++i) {
        const int c = i * groups + g;
        if (c >= a.C) break;
        row(i, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(v[e] - mean[e], v[e] - mean[e], s[e]);
    }
    steps_sum<TL>(s, red);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = 1.0f / __builtin_sqrtf(s[e] / (float)a.C + a.eps);
    if (a.stats && g == 0) {
        store8<0>(a.stats + (size_t)b * a.L, t, a.L, mean);
        store8<0>(a.stats + ((size_t)a.B + b) * a.L, t, a.L, r);
    }
    // Four rows' parameters are loaded ahead of the stores before them: loads behind stores would wait for those.
    constexpr int kAhead = LOOP ? 1 : 4;
    float w[2][kAhead], o[2][kAhead];
    const auto params = [&](int i, int set) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int c = (i + k) * groups + g, at = c < a.C ? c : a.C - 1;
            w[set][k] = a.weight ? a.weight[at] : 1.0f;
            o[set][k] = a.bias ? a.bias[at] : 0.0f;
        }
    };
    params(0, 0);
    constexpr int UA = LOOP ? 2 : R / kAhead;
#pragma unroll UA
    for (int j = 0; j < (LOOP ? rows : R / kAhead); ++j) {
        if (LOOP || j + 1 < R / kAhead) params((j + 1) * kAhead, (j + 1) % 2);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = j * kAhead + k, c = i * groups + g;
            if (c >= a.C) return;
            row(i, c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = t + e < end ? __builtin_fmaf((v[e] - mean[e]) * r[e], w[j % 2][k], o[j % 2][k]) : 0.0f;
            store8<DT>(y + (long long)c * a.y.stride_c, t, a.L, v);
        }
    }
}

// Work-group p takes tiles p, p + parts, ...; a thread's sums of dw and db stay in registers over them (LOOP: in
// its row of the workspace).
template <int DT, int TL, int R, bool LOOP>
__global__ __launch_bounds__(512) void norm_rows_bwd_kernel(miconv_layer_norm_t a, int tiles, int parts, float *part) {
    typedef typename Elem<DT>::T T;
    __shared__ float red[16][64];
    constexpr int U = LOOP ? 1 : R;
    const int p = xcd_remap(blockIdx.x, gridDim.x), tl = threadIdx.x % TL, groups = blockDim.x / TL;
    const int rows = LOOP ? (a.C + groups - 1) / groups : R;
    float *const mine = part + (size_t)p * 2 * a.C;
    float dw[LOOP ? 1 : R] = {}, db[LOOP ? 1 : R] = {}, held_w[LOOP ? 1 : R];
    if constexpr (!LOOP) {                     // held: loads behind the stores of dx would wait for those
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = i * groups + threadIdx.x / TL;
            held_w[i] = a.weight ? a.weight[c < a.C ? c : a.C - 1] : 1.0f;
        }
    }
    const auto weight = [&](int i, int c) {
        if constexpr (LOOP)
            return a.weight ? a.weight[c] : 1.0f;
        else
            return held_w[i];
    };
    bool begun = false;
    for (long long id = p; id < (long long)a.B * tiles; id += parts) {
        const int g = again(threadIdx.x / TL);  // the rows' addresses are not held from tile to tile
        const int b = (int)(id / tiles), t = (int)(id - (long long)b * tiles) * TL * 8 + tl * 8;
        const int end = valid_steps(a.lengths, b, a.L);
        const T *const x = (const T *)a.x.data + (long long)b * a.x.stride_b;
        const T *const dy = (const T *)a.dy.data + (long long)b * a.dy.stride_b;
        T *const dx = (T *)a.dx.data + (long long)b * a.dx.stride_b;
        Raw8<DT> hx[LOOP ? 1 : R], hy[LOOP ? 1 : R];
        if constexpr (!LOOP) {
            fetch_rows<DT, R>(x, a.x.stride_c, a.C, g, groups, t, end, hx);
            fetch_rows<DT, R>(dy, a.dy.stride_c, a.C, g, groups, t, end, hy);
        }
        float mean[8], r[8], n[8], h[8], s[8] = {}, q[8] = {};
        load8<0>(a.stats + (size_t)b * a.L, t, end, mean);
        load8<0>(a.stats + ((size_t)a.B + b) * a.L, t, end, r);      // 0 past the end: so is n there
        const auto row = [&](int i, int c) {   // normalised x and dy; zeros past the sequence's end
            if constexpr (LOOP) {
                load8<DT>(x + (long long)c * a.x.stride_c, t, end, n);
                load8<DT>(dy + (long long)c * a.dy.stride_c, t, end, h);
            } else {
                widen8<DT>(unseen<DT>(hx[i]), n);
                widen8<DT>(unseen<DT>(hy[i]), h);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = (n[e] - mean[e]) * r[e];
        };
#pragma unroll U
        for (int i = 0; i < rows; ++i) {
            const int c = i * groups + g;
            if (c >= a.C) break;
            row(i, c);
            const float w = weight(i, c);
            float sw = 0.0f, sb = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sw = __builtin_fmaf(h[e], n[e], sw);
                sb += h[e];
                s[e] = __builtin_fmaf(h[e], w, s[e]);
                q[e] = __builtin_fmaf(h[e] * w, n[e], q[e]);
            }
            if constexpr (LOOP) {
#pragma unroll
                for (int o = 1; o < TL; o *= 2) {
                    sw += __shfl_xor(sw, o);
                    sb += __shfl_xor(sb, o);
                }
                if (tl == 0) {
                    mine[c] = (begun ? mine[c] : 0.0f) + sw;
                    mine[a.C + c] = (begun ? mine[a.C + c] : 0.0f) + sb;
                }
            } else {
                dw[i] += sw;
                db[i] += sb;
                // here, not after the last row, with every row's values in registers till then
                asm volatile("" : "+v"(dw[i]), "+v"(db[i]));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(s[e]), "+v"(q[e]));
        }
        begun = true;
        steps_sum<TL>(s, red);
        steps_sum<TL>(q, red);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] /= (float)a.C;
            q[e] /= (float)a.C;
        }
#pragma unroll U
        for (int i = 0; i < rows; ++i) {
            const int c = i * groups + g;
            if (c >= a.C) break;
            row(i, c);
            const float w = weight(i, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = t + e < end ? r[e] * (h[e] * w - s[e] - n[e] * q[e]) : 0.0f;
            store8<DT>(dx + (long long)c * a.dx.stride_c, t, a.L, h);
        }
    }
    if constexpr (!LOOP) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = i * groups + threadIdx.x / TL;
            if (c >= a.C) break;
#pragma unroll
            for (int o = 1; o < TL; o *= 2) {
                dw[i] += __shfl_xor(dw[i], o);
                db[i] += __shfl_xor(db[i], o);
            }
            if (tl == 0) {
                mine[c] = dw[i];
                mine[a.C + c] = db[i];
            }
        }
    }
}

// The sums of dw and db over the parts, in their order: 64 columns per work-group, every 16th part per wave.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float *part, int parts, int C, float *dw, float *db) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long column = (long long)blockIdx.x * 64 + lane, columns = 2ll * C;
    float s = 0.0f;
    if (column < columns) {
        int p = wave;
        for (; p + 112 < parts; p += 128) {      // eight loads in flight: their latency bounds this kernel
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = part[(p + i * 16) * columns + column];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; p < parts; p += 16) s += part[p * columns + column];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave || column >= columns) return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    if (column < C) {
        if (dw) dw[column] = s;
    } else if (db) {
        db[column - C] = s;
    }
}

// ------------------------------------------------------------------ which kernel

bool contiguous(const miconv_tokens_t &v, int C) { return v.stride_c == 1 || C == 1; }

template <int DT>
int tokens_fwd(const miconv_layer_norm_t &n, hipStream_t st) {
    const FDiv f = make_fdiv((uint32_t)n.L);
    const long long tokens = (long long)n.B * n.L;
#define MICONV_NORM(ROW, VPT)                                                                                         \
    launch_groups((tokens + Row<ROW>::kTokens - 1) / Row<ROW>::kTokens, Row<ROW>::kThreads, [&](unsigned g, unsigned first) { \
        hipLaunchKernelGGL((norm_fwd_kernel<DT, ROW, VPT>), dim3(g), dim3(Row<ROW>::kThreads), 0, st, n, f, first);   \
    })
    const TokensForm t = tokens_form(n.C);
    if (t.threads == 64) return t.times == 1 ? MICONV_NORM(64, 1) : MICONV_NORM(64, 2);
    switch (t.times) {
        case 1: return MICONV_NORM(256, 1);
        case 2: return MICONV_NORM(256, 2);
        case 4: return MICONV_NORM(256, 4);
    }
#undef MICONV_NORM
    return launch_groups(tokens, 1024, [&](unsigned g, unsigned first) {
        hipLaunchKernelGGL(norm_fwd_long_kernel<DT>, dim3(g), dim3(1024), 0, st, n, f, first);
    });
}

template <int DT>
int tokens_bwd(const miconv_layer_norm_t &n, int parts, float *part, hipStream_t st) {
    const FDiv f = make_fdiv((uint32_t)n.L);
#define MICONV_NORM(ROW, VPT)                                                                                       \
    hipLaunchKernelGGL((norm_bwd_kernel<DT, ROW, VPT>), dim3(parts), dim3(Row<ROW>::kThreads), 0, st, n, f, parts, part)
    const TokensForm t = tokens_form(n.C);
    if (t.threads == 64 && t.times == 1)
        MICONV_NORM(64, 1);
    else if (t.threads == 64)
        MICONV_NORM(64, 2);
    else if (t.times == 1)
        MICONV_NORM(256, 1);
    else if (t.times == 2)
        MICONV_NORM(256, 2);
    else if (t.times == 4)
        MICONV_NORM(256, 4);
    else
        hipLaunchKernelGGL(norm_bwd_long_kernel<DT>, dim3(parts), dim3(1024), 0, st, n, f, parts, part);
#undef MICONV_NORM
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

template <int DT>
int rows_fwd(const miconv_layer_norm_t &n, hipStream_t st) {
    const RowsForm f = rows_form(n, DT, false);
    const int tiles = (n.L + f.lanes * 8 - 1) / (f.lanes * 8);
    constexpr int R = DT == 1 ? 16 : 8;
    return launch_groups((long long)n.B * tiles, 1024, [&](unsigned g, unsigned first) {
#define MICONV_NORM(TL, LOOP) \
    hipLaunchKernelGGL((norm_rows_fwd_kernel<DT, TL, R, LOOP>), dim3(g), dim3(f.threads), 0, st, n, tiles, first)
        switch (f.loop ? 0 : f.lanes) {
            case 8: MICONV_NORM(8, false); break;
            case 4: MICONV_NORM(4, false); break;
            case 2: MICONV_NORM(2, false); break;
            case 1: MICONV_NORM(1, false); break;
            default: MICONV_NORM(8, true);
        }
#undef MICONV_NORM
    });
}

template <int DT>
int rows_bwd(const miconv_layer_norm_t &n, int parts, float *part, hipStream_t st) {
    const RowsForm f = rows_form(n, DT, true);
    const int tiles = (n.L + f.lanes * 8 - 1) / (f.lanes * 8);
    constexpr int R = DT == 1 ? 16 : 8;
#define MICONV_NORM(TL, LOOP) \
    hipLaunchKernelGGL((norm_rows_bwd_kernel<DT, TL, R, LOOP>), dim3(parts), dim3(f.threads), 0, st, n, tiles, parts, part)
    switch (f.loop ? 0 : f.lanes) {
        case 8: MICONV_NORM(8, false); break;
        case 4: MICONV_NORM(4, false); break;
        case 2: MICONV_NORM(2, false); break;
        case 1: MICONV_NORM(1, false); break;
        default: MICONV_NORM(8, true);
    }
#undef MICONV_NORM
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

}  // namespace

// Up to 1024 channels a wave, up to 8192 a work-group of 256 holds a token in registers (at 8192 the backward pass has 256
// registers of them; another step would not fit).
TokensForm tokens_form(int C) {
    if (C <= 1024) return {64, C <= 512 ? 1 : 2};
    if (C <= 8192) return {256, C <= 2048 ? 1 : C <= 4096 ? 2 : 4};
    return {1024, 0};
}

// Time lanes of the channel-major kernels: as many as leave most CUs a tile, forward two tiles.
// 4 x 2048 tokens of 2048 channels in bf16 take, with 256 tiles of 4 lanes and 512 of 2, forward 22.2 and 22.1 us
// (fp32, a larger one: 43.8 and 37), backward 32 and 46, as its 256 work-groups then take two tiles each.
RowsForm rows_form(const miconv_layer_norm_t &n, int dtype, bool backward) {
    const int held = dtype == MICONV_BF16 ? 16 : 8, most = backward ? 512 : 1024;
    int lanes = 8;
    while (lanes > 1 && (most / lanes * held < n.C || (long long)n.B * ((n.L + lanes * 8 - 1) / (lanes * 8)) < (backward ? 200 : 400))) lanes /= 2;
    if (most / lanes * held < n.C) return {8, most, true};
    int threads = 256;
    while (threads < most && threads / lanes * held < n.C) threads *= 2;
    return {lanes, threads, false};
}

bool norm_tokens_first(const miconv_layer_norm_t &n, bool backward) {
    if (!contiguous(n.x, n.C)) return false;
    return backward ? contiguous(n.dy, n.C) && contiguous(n.dx, n.C) : contiguous(n.y, n.C);
}

// Work-groups of the backward pass, a row of partial sums each.  Tokens first, up to four a CU hide each other's loads, but long
// rows of sums cost more than that gains: 8192 tokens take, with 256 / 512 / 1024 / 2048 work-groups, 54 / 35 / 29 / 35 us at 2048
// channels and 83 / 55 / 60 / 62 at 4096 (bf16); 2048 tokens of 8192 channels 43 / 49 / 63 / 96 (fp32).  Channel-major a
// work-group mostly fills a CU: 7 x 1626 tokens of 1382 channels in fp32 take 58 us with 256 and 73 with 512, 8 x 4096 of 256 in
// bf16 24 and 20, others differ little.
int norm_parts(const miconv_layer_norm_t &n, int dtype, size_t budget) {
    long long most;
    if (norm_tokens_first(n, true)) {
        const int at_once = n.C <= 1024 ? Row<64>::kTokens : 1;
        most = ((long long)n.B * n.L + at_once - 1) / at_once;
        const int rows = n.C <= 2048 ? 1024 : n.C <= 4096 ? 512 : 256;
        if (most > rows) most = rows;
    } else {
        const int steps = rows_form(n, dtype, true).lanes * 8;
        most = (long long)n.B * ((n.L + steps - 1) / steps);
        if (most > 256) most = 256;
    }
    const long long fit = (long long)(budget / ((size_t)n.C * 8));
    if (most > fit) most = fit;
    return most < 1 ? 1 : (int)most;
}

int launch_norm_fwd(const miconv_layer_norm_t &n, int dtype, hipStream_t st) {
    if (norm_tokens_first(n, false)) return dtype == MICONV_BF16 ? tokens_fwd<1>(n, st) : tokens_fwd<0>(n, st);
    return dtype == MICONV_BF16 ? rows_fwd<1>(n, st) : rows_fwd<0>(n, st);
}

int launch_norm_bwd(const miconv_layer_norm_t &n, int dtype, int parts, float *ws, hipStream_t st) {
    const int status = norm_tokens_first(n, true)
                           ? (dtype == MICONV_BF16 ? tokens_bwd<1>(n, parts, ws, st) : tokens_bwd<0>(n, parts, ws, st))
                           : (dtype == MICONV_BF16 ? rows_bwd<1>(n, parts, ws, st) : rows_bwd<0>(n, parts, ws, st));
    if (status != MICONV_OK || (!n.dw && !n.db)) return status;
    hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((2ll * n.C + 63) / 64)), dim3(1024), 0, st, ws, parts, n.C, n.dw,
                       n.db);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

}  // namespace miconv
