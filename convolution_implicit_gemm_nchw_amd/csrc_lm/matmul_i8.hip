// matmul_i8.hip -- y[m][n] = qs[m] ws[n] sum_k q[m][k] wq[n][k] (+ bias[n]), the
// sum exact in 32-bit integers on the integer MFMAs.
//
// Both operands hold k contiguously, so either can be an MFMA's row operand.  The
// one along whose axis y is contiguous (channels for token-major y, tokens for
// channel-major y) takes the rows, called axis C below, because a lane's
// accumulators run along the rows; the other is axis R.
//
// Many tokens are bound by the MFMAs under the power limit (8192 tokens, 4096 -> 8192: 233 us,
// 2.36 POP/s with the output; on zeros 172 us, 3.2 POP/s), few by the weight's bytes (8 tokens:
// 7.3 us, 4.6 TB/s).
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

struct I8Args {
    const signed char *c, *r;       // [NC][K], [NR][K]
    const float *c_scale, *r_scale; // per row of c, of r
    const float *c_bias, *r_bias;   // one of them, or none
    int c_first;                    // order of the two scales: the tokens' first
    void *y;
    int NC, NR, K;
    // y[r * row + c], or channel-major y[((c / len) * NR + r) * len + c % len]
    long long row;
    int len;                        // 0: the first form
    FDiv fd_len;
    int tiles_c, tiles_r;
    int *part;                      // split sums [split][NR][NC], or null
    int k_split;                    // bytes of k per split
};

DEVI float scaled(const I8Args &a, int sum, float cs, float rs) {
    const float s = (float)sum;
    return a.c_first ? s * cs * rs : s * rs * cs;
}

// Eight consecutive values of one row of y from c0 on.
template <int OD, bool STREAM>
DEVI void put8(const I8Args &a, int r, int c0, const float (&v)[8]) {
    typedef typename Elem<OD>::T T;
    T *y = (T *)a.y;
    if (a.len == 0) {
        store8<OD, STREAM>(y + (long long)r * a.row, c0, a.NC, v);
        return;
    }
    const int b = (int)fdiv((uint32_t)c0, a.fd_len), l = c0 - b * a.len;
    T *line = y + ((long long)b * a.NR + r) * a.len;
    if (l + 8 <= a.len) {
        store8<OD, STREAM>(line, l, a.len, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = c0 + i;
        if (c >= a.NC) break;
        const int bi = (int)fdiv((uint32_t)c, a.fd_len);
        y[((long long)bi * a.NR + r) * a.len + (c - bi * a.len)] = Elem<OD>::put(v[i]);
    }
}

// Scales and biases of eight columns.
DEVI void columns(const I8Args &a, int c, float (&cs)[8], float (&cb)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int at = c + e < a.NC ? c + e : a.NC - 1;
        cs[e] = a.c_scale[at];
        cb[e] = a.c_bias ? a.c_bias[at] : 0.0f;
    }
}

// The sums of eight columns of row r, stored as they are (split) or finished.
template <int OD, bool STREAM = false>
DEVI void finish8(const I8Args &a, int split, int r, int c, const int (&sum)[8], const float (&cs)[8],
                  const float (&cb)[8], float rs, float rb) {
    if (a.part && split >= 0) {
        int *dst = a.part + ((long long)split * a.NR + r) * a.NC + c;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < a.NC) dst[e] = sum[e];
        return;
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = scaled(a, sum[e], cs[e], rs) + (cb[e] + rb);
    put8<OD, STREAM>(a, r, c, v);
}

// ------------------------------------------------------------------ tiles
//
// A work-group of WC x WR waves computes a (WC*FC*32) x (WR*FR*32) tile, a wave
// FC x FR blocks of 32 x 32.  128 bytes of k of every row of the tile are brought
// into LDS at a time, straight from memory (no registers in between), ST stages in
// turn: the next ones load while this one is multiplied.  A row's eight
// 16-byte pieces are stored at piece ^ (row / 2 & 7): two rows span the 64 banks, so the
// 16 rows that a part of an MFMA operand's read covers take 16 different places (with row & 7
// a fifth of the time went to bank conflicts); since the load writes LDS in lane
// order, the lanes fetch the pieces in that order instead.
template <int WC, int WR, int FC, int FR, int ST>
struct Tile {
    static constexpr int kWaves = WC * WR, kThreads = 64 * kWaves;
    static constexpr int C = WC * FC * 32, R = WR * FR * 32;
    static constexpr int kBytes = (C + R) * 128;
    // Waves of eight blocks read LDS as long as they multiply, and gain from reading ahead
    // (8192 tokens, 8192 -> 8192: 456 -> 431 us); smaller ones lose (2048 tokens, 4096 -> 2048,
    // in tiles of 128: 26.3 -> 27.2).
    static constexpr bool kAhead = FC * FR >= 8;
    static constexpr int kRowsPerLoad = kWaves * 8, kLoads = (C + R) / kRowsPerLoad;   // per wave and stage

    struct Src {
        rsrc_t rc, rr;
        uint32_t oc[C / kRowsPerLoad], orr[R / kRowsPerLoad];
    };

    static DEVI void source(const I8Args &a, int c0, int r0, Src &s) {
        const int row = threadIdx.x >> 3, piece = (threadIdx.x & 7) ^ (row >> 1 & 7);
        s.rc = make_rsrc(a.c + (long long)c0 * a.K, 0x7fffffffu);
        s.rr = make_rsrc(a.r + (long long)r0 * a.K, 0x7fffffffu);
        // rows past the end read the last row; their results are not stored
#pragma unroll
        for (int i = 0; i < C / kRowsPerLoad; ++i) {
            const int at = i * kRowsPerLoad + row;
            s.oc[i] = (uint32_t)(c0 + at < a.NC ? at : a.NC - 1 - c0) * a.K + piece * 16;
        }
#pragma unroll
        for (int i = 0; i < R / kRowsPerLoad; ++i) {
            const int at = i * kRowsPerLoad + row;
            s.orr[i] = (uint32_t)(r0 + at < a.NR ? at : a.NR - 1 - r0) * a.K + piece * 16;
        }
    }

    // Part 0 of a stage's loads is axis C's, part 1 axis R's.
    static DEVI void load_axis(const Src &s, char *lds, int k, int part) {
        const int wave = uniform(threadIdx.x >> 6);
        if (part == 0) {
#pragma unroll
            for (int i = 0; i < C / kRowsPerLoad; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rc, (lds_void *)(lds + (i * kWaves + wave) * 1024), 16,
                                                         s.oc[i], k, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < R / kRowsPerLoad; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rr, (lds_void *)(lds + C * 128 + (i * kWaves + wave) * 1024),
                                                         16, s.orr[i], k, 0, 0);
        }
    }

    static DEVI void load(const Src &s, char *lds, int k) {
        load_axis(s, lds, k, 0);
        load_axis(s, lds, k, 1);
    }

    // The operands of 32 steps of k: a lane's 16 bytes of each block.
    struct Frag {
        i32x4 c[FC], r[FR];
    };

    static DEVI void fetch(const char *lds, int kk, Frag &f) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int wc = wave % WC, wr = wave / WC, row = lane & 31, half = lane >> 5;
        const char *pc = lds + (wc * FC * 32 + row) * 128, *pr = lds + C * 128 + (wr * FR * 32 + row) * 128;
        const int piece = ((kk * 2 + half) ^ (row >> 1 & 7)) * 16;
#pragma unroll
        for (int j = 0; j < FR; ++j) f.r[j] = *(const i32x4 *)(pr + j * 32 * 128 + piece);
#pragma unroll
        for (int i = 0; i < FC; ++i) f.c[i] = *(const i32x4 *)(pc + i * 32 * 128 + piece);
    }

    static DEVI void multiply(const Frag &f, i32x16 (&acc)[FC][FR]) {
#pragma unroll
        for (int i = 0; i < FC; ++i)
#pragma unroll
            for (int j = 0; j < FR; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.c[i], f.r[j], acc[i][j], 0, 0, 0);
    }

    // A read of LDS after each product, of those since the last call; by itself the compiler
    // puts the reads first.
    static DEVI void interleave() {
#pragma unroll
        for (int i = 0; i < FC + FR; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, FC * FR, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
};

template <int OD, int WC, int WR, int FC, int FR, int ST, bool STREAM>
__global__ __launch_bounds__(64 * WC * WR) void i8_tile_kernel(I8Args a) {
    typedef Tile<WC, WR, FC, FR, ST> X;
    __shared__ __attribute__((aligned(1024))) char stages[ST * X::kBytes];
    // each XCD a contiguous range of tiles, in columns of eight C tiles: the tiles that
    // run on it together share their operands in its L2
    const int per_split = a.tiles_c * a.tiles_r, split = blockIdx.x / per_split;
    const int t = xcd_remap(blockIdx.x - split * per_split, per_split);
    const int band = t / (8 * a.tiles_r), in = t - band * 8 * a.tiles_r;
    const int wide = a.tiles_c - band * 8 < 8 ? a.tiles_c - band * 8 : 8;
    const int c0 = (band * 8 + in % wide) * X::C, r0 = (in / wide) * X::R;
    typename X::Src src;
    X::source(a, c0, r0, src);
    i32x16 acc[FC][FR];
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
        for (int j = 0; j < FR; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
    const int first = split * a.k_split, end = first + a.k_split < a.K ? first + a.k_split : a.K;
#pragma unroll
    for (int i = 0; i < ST - 1; ++i)
        if (first + i * 128 < end) X::load(src, stages + i * X::kBytes, first + i * 128);
    // what the epilogue needs from memory: a lane's columns' and one row's scale and bias
    constexpr int kW = FC * 32, kMine = 32 * kW, kMix = kW >= 64 ? 15 : 7;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wc = wave % WC, wr = wave / WC;
    constexpr int kLanes = kW / 8;             // lanes per row, eight columns each
    const int col = (lane % kLanes) * 8, c = c0 + wc * kW + col;
    float cs[8], cb[8];
    columns(a, c, cs, cb);
    static_assert(FR <= 2, "one row's scale per lane");
    const int rl = r0 + wr * FR * 32 + lane, rc = rl < a.NR ? rl : a.NR - 1;
    const float rs = a.r_scale[rc], rb = a.r_bias ? a.r_bias[rc] : 0.0f;
    typename X::Frag f0, f1;
    if constexpr (X::kAhead) {
        // Operands are read one fragment ahead of the products, over the end of the stage: after
        // its third fragment's products the next stage must have arrived and every wave have
        // read this one, whose place the stage after next takes.  One half of its loads is
        // issued there, the other a fragment later.
        char *in = stages, *to = stages + X::kBytes;
        const auto arrived = [] {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __syncthreads();
        };
        if (first + 128 < end) X::load_axis(src, to, first + 128, 0);
        arrived();
        X::fetch(in, 0, f0);
        for (int k = first + 128; k < end; k += 128) {
            X::load_axis(src, to, k, 1);
            __builtin_amdgcn_sched_barrier(0);
            X::fetch(in, 1, f1);
            X::multiply(f0, acc);
            X::interleave();
            X::fetch(in, 2, f0);
            X::multiply(f1, acc);
            X::interleave();
            X::fetch(in, 3, f1);
            X::multiply(f0, acc);
            X::interleave();
            arrived();
            if (k + 128 < end) X::load_axis(src, in, k + 128, 0);
            X::fetch(to, 0, f0);
            X::multiply(f1, acc);
            X::interleave();
            char *const was = in;
            in = to;
            to = was;
        }
        X::fetch(in, 1, f1);
        X::multiply(f0, acc);
        X::fetch(in, 2, f0);
        X::multiply(f1, acc);
        X::fetch(in, 3, f1);
        X::multiply(f0, acc);
        X::multiply(f1, acc);
    } else {
        int now = 0, next = ST - 1;
        for (int k = first; k < end; k += 128) {
            // this stage has arrived (each wave waits for its own loads, of which those of the
            // ST - 2 stages after it may be in flight; the compiler does not always tie an LDS
            // load to the reads behind the barrier), and the stage before has been read
            if (ST > 2 && k + (ST - 2) * 128 < end)
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"((ST - 2) * X::kLoads) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (k + (ST - 1) * 128 < end) X::load(src, stages + next * X::kBytes, k + (ST - 1) * 128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                X::fetch(stages + now * X::kBytes, kk, f0);
                X::multiply(f0, acc);
            }
            now = now + 1 < ST ? now + 1 : 0;
            next = next + 1 < ST ? next + 1 : 0;
        }
    }
    __syncthreads();
    // Through LDS, 32 rows of the wave's FC*32 columns at a time, so that y is written
    // in 16-byte pieces of consecutive lanes; a row's pieces are permuted as above.
    static_assert(X::kWaves * kMine * 4 <= ST * X::kBytes, "the exchange fits the stages");
    int *mine = (int *)stages + wave * kMine;
#pragma unroll
    for (int j = 0; j < FR; ++j) {
        const int rw = r0 + (wr * FR + j) * 32;
#pragma unroll
        for (int i = 0; i < FC; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                i32x4 four;
#pragma unroll
                for (int e = 0; e < 4; ++e) four[e] = acc[i][j][g * 4 + e];
                const int row = lane & 31, piece = (i * 8 + g * 2 + (lane >> 5)) ^ (row & kMix);
                *(i32x4 *)(mine + row * kW + piece * 4) = four;
            }
        wave_lds_sync();
#pragma unroll 2
        for (int p = 0; p < 32 * kLanes / 64; ++p) {
            const int row = p * (64 / kLanes) + lane / kLanes, r = rw + row;
            const float rsr = __shfl(rs, j * 32 + row), rbr = __shfl(rb, j * 32 + row);
            if (r >= a.NR || c >= a.NC) continue;
            const i32x4 lo = *(const i32x4 *)(mine + row * kW + ((col >> 2) ^ (row & kMix)) * 4);
            const i32x4 hi = *(const i32x4 *)(mine + row * kW + (((col >> 2) + 1) ^ (row & kMix)) * 4);
            int sum[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[e] = lo[e];
                sum[4 + e] = hi[e];
            }
            finish8<OD, STREAM>(a, split, r, c, sum, cs, cb, rsr, rbr);
        }
        wave_lds_sync();
    }
}

// Adds the splits' sums and finishes them.
template <int OD>
__global__ __launch_bounds__(256) void i8_join_kernel(I8Args a, int splits) {
    const int per_row = (a.NC + 7) / 8;
    const long long n = (long long)a.NR * per_row;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const int r = (int)(i / per_row), c = (int)(i - (long long)r * per_row) * 8;
        int sum[8] = {};
        for (int z = 0; z < splits; ++z) {
            const int *p = a.part + ((long long)z * a.NR + r) * a.NC + c;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < a.NC) sum[e] += p[e];
        }
        float cs[8], cb[8];
        columns(a, c, cs, cb);
        finish8<OD>(a, -1, r, c, sum, cs, cb, a.r_scale[r], a.r_bias ? a.r_bias[r] : 0.0f);
    }
}

// ------------------------------------------------------------------ few tokens
//
// With few tokens the weight's bytes count: each is read once, straight into
// registers, as the row operand of 16x16x64 MFMAs.  A work-group takes 32 channels,
// its eight waves an eighth of k each (pieces of 256 bytes in turn), and adds the
// waves' sums in LDS.  FT blocks of 16 tokens.
template <int OD, int FT>
__global__ __launch_bounds__(512) void i8_few_kernel(const signed char *q, const signed char *wq, const float *qs,
                                                     const float *ws, const float *bias, int T, int O, int K, int L,
                                                     int channel_major, void *y, uint32_t first) {
    __shared__ int red[8][32][FT * 16 + 1];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), row = lane & 15, kq = (lane >> 4) * 16;
    const int n0 = (int)(first + blockIdx.x) * 32;
    const signed char *pw[2], *pq[FT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = n0 + i * 16 + row;
        pw[i] = wq + (long long)(n < O ? n : O - 1) * K + kq;
    }
#pragma unroll
    for (int i = 0; i < FT; ++i) {
        const int m = i * 16 + row;
        pq[i] = q + (long long)(m < T ? m : T - 1) * K + kq;
    }
    i32x4 acc[2][FT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // the next 128 bytes of k load while these are multiplied
    i32x4 a[2][2], b[2][FT];
    auto fetch = [&](int k) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < 2; ++i) a[s][i] = *(const i32x4 *)(pw[i] + k + s * 64);
#pragma unroll
            for (int j = 0; j < FT; ++j) b[s][j] = *(const i32x4 *)(pq[j] + k + s * 64);
        }
    };
    if (wave * 128 < K) fetch(wave * 128);
    for (int k = wave * 128; k < K; k += 8 * 128) {
        i32x4 a0[2][2], b0[2][FT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < 2; ++i) a0[s][i] = a[s][i];
#pragma unroll
            for (int j = 0; j < FT; ++j) b0[s][j] = b[s][j];
        }
        if (k + 8 * 128 < K) fetch(k + 8 * 128);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0[s][i], b0[s][j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[wave][i * 16 + (lane >> 4) * 4 + e][j * 16 + row] = acc[i][j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * FT * 16; i += 512) {
        // token-major: consecutive lanes on consecutive channels
        const int n = channel_major ? i / (FT * 16) : i & 31, m = channel_major ? i % (FT * 16) : i >> 5;
        if (n0 + n >= O || m >= T) continue;
        int sum = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += red[w][n][m];
        float v = (float)sum * qs[m] * ws[n0 + n];
        if (bias) v += bias[n0 + n];
        const int b = m / L;
        const long long at = channel_major ? ((long long)b * O + n0 + n) * L + (m - b * L) : (long long)m * O + n0 + n;
        ((typename Elem<OD>::T *)y)[at] = Elem<OD>::put(v);
    }
}

template <int OD, int FT>
int few(int T, int O, int K, int L, const signed char *q, const float *qs, const signed char *wq, const float *ws,
         const float *bias, int channel_major, void *y, hipStream_t st) {
    return launch_groups(((long long)O + 31) / 32, 512, [&](unsigned n, unsigned first) {
        hipLaunchKernelGGL((i8_few_kernel<OD, FT>), dim3(n), dim3(512), 0, st, q, wq, qs, ws, bias, T, O, K, L, channel_major,
                           y, first);
    });
}

template <int OD, int WC, int WR, int FC, int FR, int ST, bool STREAM = false>
int tiled(I8Args a, int splits, hipStream_t st) {
    typedef Tile<WC, WR, FC, FR, ST> X;
    a.tiles_c = (a.NC + X::C - 1) / X::C;
    a.tiles_r = (a.NR + X::R - 1) / X::R;
    if (splits == 1) a.part = nullptr;
    a.k_split = ((a.K / 128 + splits - 1) / splits) * 128;
    hipLaunchKernelGGL((i8_tile_kernel<OD, WC, WR, FC, FR, ST, STREAM>), dim3((unsigned)((long long)a.tiles_c * a.tiles_r * splits)),
                       dim3(X::kThreads), 0, st, a);
    if (hipGetLastError() != hipSuccess) return MICONV_ERR_HIP;
    if (splits > 1) {
        long long blocks = ((long long)a.NR * ((a.NC + 7) / 8) + 255) / 256;
        hipLaunchKernelGGL(i8_join_kernel<OD>, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, a,
                           splits);
        if (hipGetLastError() != hipSuccess) return MICONV_ERR_HIP;
    }
    return MICONV_OK;
}

// Up to here one 16-token block after the other costs less than a 64-row tile (4096 -> 8192:
// 16 tokens 8.0 against 14.3 us, 64 tokens 14.0 against 16.6).
constexpr int kFewTokens = 64;

long long tile_count(long long T, long long O, int side) {
    return ((T + side - 1) / side) * ((O + side - 1) / side);
}

// Side of the square tile: the largest that gives most of the 256 CUs a tile.  In us: 128 tiles of
// 256, 4096 deep, 52.6 against 41.7 with side 128; 144 tiles 52.6 against 58.9 (1024 deep 23.4 against
// 22.1); 128 tiles of 128, 4096 deep, 23.2 against 17.1 with side 64; 144 tiles, 2048 deep, 12.7
// against 15.9.
int tile_side(int T, int O) {
    if (tile_count(T, O, 256) >= 140) return 256;
    if (tile_count(T, O, 128) >= 140) return 128;
    return 64;
}

}  // namespace

// Splits of k: a step of 128 bytes takes 0.3 us, joining the sums 4 to 5 us, so only products
// 8192 deep or more with few tiles gain (100 tokens, 8192 -> 512: 21.0 us whole, 16.3 in four;
// 128 tokens, 4096 -> 2048: 12.1 whole, 14.8 in two), each split at least 2048 deep.
int i8_splits(int T, int O, int K, size_t budget) {
    if (T <= kFewTokens || K < 8192) return 1;
    const long long tiles = tile_count(T, O, tile_side(T, O));
    long long s = 160 / tiles;
    if (s > K / 2048) s = K / 2048;
    if (s > 16) s = 16;
    const size_t one = (size_t)T * O * 4;
    if (s > (long long)(budget / one)) s = (long long)(budget / one);
    if (s < 2) return 1;
    const int steps = K / 128, per = (int)((steps + s - 1) / s);
    return (steps + per - 1) / per;            // no empty split
}

I8Form i8_form(int T, int O, int K, int splits) {
    if (T <= kFewTokens) return {T <= 16 ? 1 : (T <= 32 ? 2 : 4), 0, 0};
    const int side = tile_side(T, O);
    // small tiles leave LDS room for four stages, which tall and narrow products (few tiles,
    // long k) need: 65 tokens, 4096 -> 8192: 17.4 us with two, 12.8 with four.  Of the 128-tiles two
    // stages let two work-groups share a CU; where each has its own and k is long, four hide
    // more (2048 tokens, 4096 -> 2048: 27.0 -> 25.1 us; 2048 deep 14.6 -> 15.1)
    const bool four = side == 64 || (side == 128 && tile_count(T, O, 128) * splits <= 256 && K >= 4096);
    return {0, side, four ? 4 : 2};
}

template <int OD>
static int i8_by_form(const I8Args &a, const I8Form &f, bool stream, int splits, hipStream_t st) {
    switch (f.side) {
        case 256:
            if (stream) return tiled<OD, 2, 4, 4, 2, 2, OD == 1>(a, splits, st);
            return tiled<OD, 2, 4, 4, 2, 2>(a, splits, st);
        // eight waves of a block pair each rather than four of four (1300 tokens, 2048 -> 2048: 15.0 ->
        // 12.8 us)
        case 128:
            if (f.stages == 4) return tiled<OD, 4, 2, 1, 2, 4>(a, splits, st);
            return tiled<OD, 4, 2, 1, 2, 2>(a, splits, st);
        default: return tiled<OD, 2, 2, 1, 1, 4>(a, splits, st);
    }
}

int launch_matmul_i8(int B, int L, int O, int K, const signed char *q, const float *qs, const signed char *wq,
                     const float *ws, const float *bias, int channel_major, int out_dtype, void *y, int splits,
                     int *part, hipStream_t st) {
    const int T = B * L;
    const I8Form f = i8_form(T, O, K, splits);
    if (f.few) {
#define MICONV_FEW(FT)                                                                            \
    (out_dtype ? few<1, FT>(T, O, K, L, q, qs, wq, ws, bias, channel_major, y, st)                \
               : few<0, FT>(T, O, K, L, q, qs, wq, ws, bias, channel_major, y, st))
        return f.few == 1 ? MICONV_FEW(1) : (f.few == 2 ? MICONV_FEW(2) : MICONV_FEW(4));
    }
    I8Args a = {};
    a.K = K;
    a.y = y;
    a.part = part;
    if (channel_major) {
        a.c = q; a.c_scale = qs; a.NC = T; a.c_first = 1;
        a.r = wq; a.r_scale = ws; a.NR = O; a.r_bias = bias;
        a.row = T;
        a.len = B > 1 ? L : 0;
        a.fd_len = make_fdiv((uint32_t)L);
    } else {
        a.c = wq; a.c_scale = ws; a.NC = O; a.c_bias = bias;
        a.r = q; a.r_scale = qs; a.NR = T;
        a.row = O;
    }
    const bool stream = streams(out_dtype, (size_t)T * O);
    return out_dtype ? i8_by_form<1>(a, f, stream, splits, st) : i8_by_form<0>(a, f, stream, splits, st);
}

}  // namespace miconv
