// scan_bwd.hip -- selective scan, backward.
//
// With e_t the gradient of v_t (dy_t silu(z_t), or dy_t) and G_t = exp(dt_t A) g_t the
// gradient that step t hands to the state before it:
//   g_t[n] = C_t[n] e_t + G_{t+1}[n]
//   dC_t[n] = sum_d e_t h_t[n]         dB_t[n] = sum_d g_t[n] dt_t x_t
//   dx_t = dt_t sum_n g_t[n] B_t[n] + D e_t
//   d(dt)_t = sum_n (A[n] g_t[n] a_t h_{t-1}[n]) + x_t sum_n g_t[n] B_t[n]
//   dA[n] = sum_{b,t} dt_t g_t[n] a_t h_{t-1}[n]
// h is rebuilt chunk by chunk from the states that the forward pass saved; G runs
// through the chunks from the last to the first.  Both are scans of first-order
// maps, as in the forward pass.
//
// Bound by the vector ALUs: a (step, state) pair costs 18 slots of four cycles and its
// share of the two scans.  The split keeps everything else off that path:
//   - a row of 16 lanes takes one channel, eight steps a lane, so the scans stay inside
//     DPP rows (half the cost of a scan over the wave) and a wave holds four channels;
//   - a work-group takes 16 channels (four such groups) of one sequence; its four waves
//     have NS states each, for all 16 channels, so that the sums over channels of dB and
//     dC are kept in registers and leave them once per chunk;
//   - what belongs to a step (softplus, gate, their derivatives) is computed once, by
//     the wave that owns the group, and shared through LDS;
//   - the sums over states meet in LDS: in turn i wave w works on group (i + w) mod 4, so
//     every group has one wave at a time adding to it, in a fixed order.
// The 16-channel sums of dB and dC go to the workspace and are added in order by a
// second kernel.  More than 16 states are taken 16 per launch, the sums over the states
// of the earlier launches waiting in the workspace, or, where a launch leaves CUs without a
// work-group, by work-groups side by side, whose sums another kernel adds and finishes.
//
// 2 x 4096 rows of 2048, N 16, bf16: 260 us, 22 of them the second kernel's; 27 instructions per
// pair (17 in the states' loop), the ALUs busy 81 % of the time.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int kStates = 16, kT = kScanChunk, kCh = kScanBwdChannels;
static_assert(kT == 128 && kCh == 16, "16 lanes x 8 steps, 4 waves x 4 rows");

struct BwdOut {
    float *dB, *dC;           // [parts][B][G][N][L]
    float *dA, *dD, *db;      // [segs][B][D][N], [segs][B][D], [segs][B][D]
    const float *G;           // [B][D][chunks][N] G of the step after each chunk, or null: one segment
    int segs, seg_chunks;     // time segments (a work-group each), chunks of one
    float *sums;              // [3][B][D][L] sums over the states of earlier launches, or null; side by side
                              // [blocks of 16 states] of them
    int parts;
    int n_first, n_end, last; // states of this launch (side by side: 16 per blockIdx.y); whether it finishes
    int t_first, chunks;      // a slice of the time steps: its first one; saved states per row
};

// Per-step values of the 16 channels: [group][half][64 lanes][4 steps].
struct Steps {
    float v[4][2][64][4];
};

DEVI void put_steps(Steps &s, int group, int lane, const float (&v)[8]) {
    *(f32x4 *)s.v[group][0][lane] = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4 *)s.v[group][1][lane] = f32x4{v[4], v[5], v[6], v[7]};
}
DEVI void get_steps(const Steps &s, int group, int lane, float (&v)[8]) {
    const f32x4 lo = *(const f32x4 *)s.v[group][0][lane], hi = *(const f32x4 *)s.v[group][1][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = lo[i];
        v[4 + i] = hi[i];
    }
}

// Where the rows of a work-group's channels and states start, kept in LDS: made from bases and
// strides in every chunk they cost a tenth of the kernel's instructions, and held in registers
// they spill.
enum { kX, kDelta, kDy, kZ, kDx, kDdelta, kDz, kB, kC, kDB, kDC, kTable };

struct Lds {
    Steps dt, dtx, e;                       // shared by the waves
    Steps sdt, sgB, sv;                     // sums over states: A g a h, g B, C h
    Steps zslope;                           // dy silu'(z)
    float bc[kStates][2][2][16][4];         // B and C of the chunk: [state][B, C][half][lane of a row][4]
    float a2[kCh][kStates];                 // A log2(e)
    float carry[kCh][kStates];              // G of the step after the chunk
    float none[kStates];                    // zeros: what the other lanes read in its place
    float dA[4][4][4][16];                  // [wave][turn][state][4 lanes of each row]
    unsigned long long rows[kTable][16];    // addresses, see below
};

// Sums over the four rows of the wave: of u in rows 0, 1 and of v in rows 2, 3 (rows of a
// pair hold what the next step adds).
DEVI float join_halves(float u, float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(u), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
DEVI float join_rows(float u, float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(u), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

DEVI float row_sum(float v) {          // in the last lane of each row
    v += cross<kRowShr + 1>(v);
    v += cross<kRowShr + 2>(v);
    v += cross<kRowShr + 4>(v);
    return v + cross<kRowShr + 8>(v);
}

// e = dy silu(z) in place of dy, and dy silu'(z).
template <int DT>
DEVI void gate(float (&e)[8], const float (&z)[8], float (&zslope)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float sg = logistic_for<DT>(z[i]);
        zslope[i] = e[i] * (sg * __builtin_fmaf(z[i], 1.0f - sg, 1.0f));
        e[i] *= z[i] * sg;
    }
}

// The derivative of the step size in place of delta, 0 past the end.
template <int DT>
DEVI void slopes(float (&v)[8], float bias, int use_softplus, int t, int chunk_end, int len) {
    if (use_softplus) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = logistic_for<DT>(v[i] + bias);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    }
    if (chunk_end > len) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = t + i < len ? v[i] : 0.0f;
    }
}

// From the sums over the states (that of A g a h was taken with A log2(e)) to d(delta) and
// dx, and the sums over time of the bias's and D's gradients.
DEVI void finish_steps(const float (&x)[8], const float (&slope)[8], const float (&dt)[8], const float (&e)[8], float skip,
                       float (&sdt)[8], float (&sgB)[8], float &sb, float &sD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sdt[i] = __builtin_fmaf(x[i], sgB[i], sdt[i] * kLn2) * slope[i];
        sb += sdt[i];
        sD = __builtin_fmaf(e[i], x[i], sD);
        sgB[i] = __builtin_fmaf(dt[i], sgB[i], skip * e[i]);
    }
}

// Zeros from max(t, end) to t + 8, as far as the row goes.
template <int DT>
DEVI void zero_past(typename Elem<DT>::T *row, int t, int end, int L) {
    const float zero[8] = {};
    store8<DT>(row, t < end ? end : t, t + 8 < L ? t + 8 : L, zero);
}

template <typename P>
DEVI P *at_row(const miconv_rows_t &r, int b, int d) {
    return (P *)r.data + b * r.stride_b + d * r.stride_d;
}

// An address of the table, which is known to be one of global memory.
template <typename P>
DEVI P *row_at(const Lds &m, int what, int i) {
    return (P *)(__attribute__((address_space(1))) P *)m.rows[what][i];
}

template <int DT, int NS>
__global__ __launch_bounds__(256, 2) void scan_bwd_kernel(miconv_scan_t s, BwdOut o, uint32_t first_group) {
    typedef typename Elem<DT>::T T;
    __shared__ __attribute__((aligned(16))) Lds m;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), row = lane >> 4, sub = lane & 15;
    const int per_group = s.D / s.G;
    const uint32_t id = first_group + blockIdx.x;
    const int part = id % o.parts, bg = id / o.parts % (s.B * s.G), seg = id / (o.parts * s.B * s.G);
    const int g = bg % s.G, b = bg / s.G;
    const int first = g * per_group + part * kCh;                        // the work-group's first channel
    const int channels = per_group - part * kCh < kCh ? per_group - part * kCh : kCh;
    const int n_first = o.n_first + blockIdx.y * kStates;                // states of the work-group, of the wave
    const int nn = o.n_end - n_first < kStates ? o.n_end - n_first : kStates, j0 = wave * NS;
    const int len = valid_steps(s.lengths, b, s.L, o.t_first);
    const int chunks = (s.L + kT - 1) / kT;
    const int c_first = seg * o.seg_chunks, c_end = c_first + o.seg_chunks < chunks ? c_first + o.seg_chunks : chunks;
    // the channel that this lane owns between the turns
    const int own = wave * 4 + row;
    const bool live = own < channels;
    const int d = first + (live ? own : 0);
    const float bias = s.delta_bias ? s.delta_bias[d] : 0.0f, skip = s.D_skip ? s.D_skip[d] : 0.0f;
    const bool gated = s.z.data != nullptr;
    for (int i = threadIdx.x; i < kCh * kStates; i += 256) {
        const int c = i / kStates, j = i % kStates;
        const bool used = c < channels && j < nn;
        const long long at = ((long long)b * s.D + first + c) * s.N + n_first + j;
        m.a2[c][j] = used ? log2_decay(s.A[(long long)(first + c) * s.N + n_first + j]) : 0.0f;
        const float *G = c_end < chunks ? o.G + (((long long)b * s.D + first + c) * chunks + c_end - 1) * s.N + n_first + j
                                        : (s.d_final_state ? s.d_final_state + at : nullptr);
        m.carry[c][j] = used && G ? *G : 0.0f;
    }
    for (int i = threadIdx.x; i < 4 * 4 * 4 * 16; i += 256) (&m.dA[0][0][0][0])[i] = 0.0f;
    if (threadIdx.x < kStates) m.none[threadIdx.x] = 0.0f;
    if (threadIdx.x < 16) {
        const int k = threadIdx.x, dk = first + (k < channels ? k : 0), n = n_first + (k < nn ? k : 0);
        m.rows[kX][k] = (unsigned long long)at_row<const T>(s.x, b, dk);
        m.rows[kDelta][k] = (unsigned long long)at_row<const T>(s.delta, b, dk);
        m.rows[kDy][k] = (unsigned long long)at_row<const T>(s.dy, b, dk);
        m.rows[kZ][k] = (unsigned long long)at_row<const T>(s.z.data ? s.z : s.x, b, dk);
        m.rows[kDx][k] = (unsigned long long)at_row<T>(s.dx, b, dk);
        m.rows[kDdelta][k] = (unsigned long long)at_row<T>(s.ddelta, b, dk);
        m.rows[kDz][k] = s.z.data ? (unsigned long long)at_row<T>(s.dz, b, dk) : 0;
        m.rows[kB][k] = (unsigned long long)((const T *)s.Bm.data + b * s.Bm.stride_b + g * s.Bm.stride_g + n * s.Bm.stride_n);
        m.rows[kC][k] = (unsigned long long)((const T *)s.Cm.data + b * s.Cm.stride_b + g * s.Cm.stride_g + n * s.Cm.stride_n);
        const long long at = ((((long long)part * s.B + b) * s.G + g) * s.N + n) * s.L;
        m.rows[kDB][k] = (unsigned long long)(o.dB + at);
        m.rows[kDC][k] = (unsigned long long)(o.dC + at);
    }
    __syncthreads();
    float sD = 0.0f, sb = 0.0f;
    const int end = live ? len : 0;
    // What lies past the sequence's end is zeros, and not computed: states and parameters that are
    // not finite would make padding NaN.
    int c = c_end - 1;
    for (; c >= c_first; --c) {
        const int t = c * kT + sub * 8;
        if (len >= s.L || len >= (c + 1) * kT) break;
        if (live && o.last) {
            zero_past<DT>(row_at<T>(m, kDx, own), t, len, s.L);
            zero_past<DT>(row_at<T>(m, kDdelta, own), t, len, s.L);
            if (gated) zero_past<DT>(row_at<T>(m, kDz, own), t, len, s.L);
        }
        for (int i = wave * 4 + row; i < 2 * nn; i += 16)
            zero_past<0>(row_at<float>(m, i & 1 ? kDC : kDB, i >> 1), t, len, s.L);
        if (c * kT < len) break;
    }
    // What a chunk reads of its rows, fetched while the chunk before is finished.
    Raw8<DT> rx, rd, ry, rz, rbc[2];
    auto fetch = [&](int c) {
        const int t = c * kT + sub * 8;
        rx = fetch8<DT>(row_at<const T>(m, kX, own), t, end);
        rd = fetch8<DT>(row_at<const T>(m, kDelta, own), t, end);
        ry = fetch8<DT>(row_at<const T>(m, kDy, own), t, end);
        rz = fetch8<DT>(row_at<const T>(m, kZ, own), t, end);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = threadIdx.x + k * 256, which = (i < nn * 32 ? i : 0) >> 4;
            rbc[k] = fetch8<DT>(row_at<const T>(m, which & 1 ? kC : kB, which >> 1), t, len);
        }
    };
    if (c >= c_first) fetch(c);
    // Of the two work-groups that share a CU's ALUs the older one would be served first and leave
    // the other to end alone, at half the ALUs' rate.  The one with more work left goes first, to
    // a chunk's precision at the end (L 2048: 291 -> 263 us).
    __builtin_amdgcn_s_setprio(3);
    const int todo = c - c_first + 1;
    for (; c >= c_first; --c) {
        const int left = c - c_first;
        if (left == 0) __builtin_amdgcn_s_setprio(0);
        else if (left * 8 <= todo) __builtin_amdgcn_s_setprio(1);
        else if (left * 8 <= todo * 3) __builtin_amdgcn_s_setprio(2);
        const int t0 = c * kT, t = t0 + sub * 8;
        float dB[NS][8], dC[NS][8];
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) dB[j][i] = dC[j][i] = 0.0f;
        {
            // B and C of the chunk, and what belongs to the steps of the wave's own group
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = threadIdx.x + k * 256, which = i >> 4;
                if (i >= nn * 32) break;
                float w[8];
                widen8<DT>(rbc[k], w);
                *(f32x4 *)m.bc[which >> 1][which & 1][0][sub] = f32x4{w[0], w[1], w[2], w[3]};
                *(f32x4 *)m.bc[which >> 1][which & 1][1][sub] = f32x4{w[4], w[5], w[6], w[7]};
            }
            {
                float dt[8], e[8], dtx[8];
                widen8<DT>(rx, dtx);
                widen8<DT>(rd, dt);
                widen8<DT>(ry, e);
                if (gated) {
                    float zv[8], zslope[8];
                    widen8<DT>(rz, zv);
                    gate<DT>(e, zv, zslope);
                    put_steps(m.zslope, wave, lane, zslope);
                }
                step_sizes(dt, bias, s.softplus, t, live ? t0 + kT : len + 1, end);
#pragma unroll
                for (int i = 0; i < 8; ++i) dtx[i] *= dt[i];
                put_steps(m.dt, wave, lane, dt);
                put_steps(m.dtx, wave, lane, dtx);
                put_steps(m.e, wave, lane, e);
            }
            __syncthreads();
#pragma unroll 1
            for (int turn = 0; turn < 4; ++turn) {
                const int group = (turn + wave) & 3, ch = group * 4 + row;
                if (j0 < nn || turn == 0) {          // a wave without states adds zeros, as the first
                    float dt[8], dtx[8], e[8], sdt[8], sgB[8], sv[8];
                    get_steps(m.dt, group, lane, dt);
                    get_steps(m.dtx, group, lane, dtx);
                    get_steps(m.e, group, lane, e);
                    if (turn == 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) sdt[i] = sgB[i] = sv[i] = 0.0f;
                    } else {
                        get_steps(m.sdt, group, lane, sdt);
                        get_steps(m.sgB, group, lane, sgB);
                        get_steps(m.sv, group, lane, sv);
                    }
                    float h0s[NS];
                    const bool there = ch < channels && sub == 0;
                    const float *entry = s.states + (((long long)b * s.D + first + (there ? ch : 0)) * o.chunks + c) * s.N + n_first;
#pragma unroll
                    for (int j = 0; j < NS; ++j) h0s[j] = there && j0 + j < nn ? entry[j0 + j] : 0.0f;
                    float all = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) all += dt[i];
                    const float *const entry_G = sub == 15 ? &m.carry[ch][j0] : m.none;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        const int n = j0 + j;
                        if (n >= nn) break;
                        const float a2 = m.a2[ch][n], G0 = entry_G[j], h0 = h0s[j];       // of the row's end, else 0
                        float bv[8], cv[8], a[8], u[8], h = h0, G = G0;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const f32x4 fb = *(const f32x4 *)m.bc[n][0][q][sub], fc = *(const f32x4 *)m.bc[n][1][q][sub];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                bv[q * 4 + i] = fb[i];
                                cv[q * 4 + i] = fc[i];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            a[i] = exp2_hw(dt[i] * a2);
                            u[i] = dtx[i] * bv[i];
                            h = __builtin_fmaf(a[i], h, u[i]);
                        }
#pragma unroll
                        for (int i = 7; i >= 0; --i) G = a[i] * __builtin_fmaf(cv[i], e[i], G);
                        scan_rows(h, G, exp2_hw(all * a2));
                        if (sub == 0) m.carry[ch][n] = G;
                        h = cross_or<kRowShr + 1>(h0, h);
                        G = cross_or<kRowShl + 1>(G0, G);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float ah = a[i] * h;
                            h = ah + u[i];
                            u[i] = ah;
                            sv[i] = __builtin_fmaf(cv[i], h, sv[i]);
                            dC[j][i] = __builtin_fmaf(e[i], h, dC[j][i]);
                        }
                        float sA = 0.0f;
#pragma unroll
                        for (int i = 7; i >= 0; --i) {
                            const float gt = __builtin_fmaf(cv[i], e[i], G), w = gt * u[i];
                            G = a[i] * gt;
                            sdt[i] = __builtin_fmaf(a2, w, sdt[i]);
                            sA = __builtin_fmaf(dt[i], w, sA);
                            sgB[i] = __builtin_fmaf(gt, bv[i], sgB[i]);
                            dB[j][i] = __builtin_fmaf(gt, dtx[i], dB[j][i]);
                        }
                        sA += cross<kRowShr + 8>(sA);
                        sA += cross<kRowShr + 4>(sA);
                        // (one lane adds to each place: the order is the program's)
                        if (sub >= 12)
                            __hip_atomic_fetch_add(&m.dA[wave][turn][j][row * 4 + (sub & 3)], sA, __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_WORKGROUP);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    put_steps(m.sdt, group, lane, sdt);
                    put_steps(m.sgB, group, lane, sgB);
                    put_steps(m.sv, group, lane, sv);
                }
                __syncthreads();
            }
        }
        // this chunk's x and delta once more, and the next chunk's rows, while dB and dC leave
        Raw8<DT> ox, od;
        {
            ox = fetch8<DT>(row_at<const T>(m, kX, own), t, end);
            od = fetch8<DT>(row_at<const T>(m, kDelta, own), t, end);
        }
        fetch(c > c_first ? c - 1 : c);              // (without a condition: else the old values stay live)
        __builtin_amdgcn_sched_barrier(0);
        // dB and dC summed over the wave's four rows: rows 0, 1 end up with dB, 2, 3 with dC, of
        // the first and the second half of the wave's states
        constexpr int NH = NS > 1 ? NS / 2 : 1;
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            const int j2 = NS > 1 ? j + NH : j;
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = join_rows(join_halves(dB[j][i], dC[j][i]), join_halves(dB[j2][i], dC[j2][i]));
            const int n = j0 + (row & 1 ? j2 : j);
            if (n < nn && t < len && !(NS == 1 && (row & 1)))
                store8<0>(row_at<float>(m, row & 2 ? kDC : kDB, n), t, len, w);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (live) {
            float sdt[8], sgB[8], sv[8], dt[8], e[8], xv[8];
            get_steps(m.sdt, wave, lane, sdt);
            get_steps(m.sgB, wave, lane, sgB);
            get_steps(m.sv, wave, lane, sv);
            if (o.sums) {
                const long long one = (long long)s.B * s.D * s.L;
                float *past = o.sums + 3 * one * blockIdx.y + ((long long)b * s.D + again(d)) * s.L;
                if (o.n_first) {
                    float w[8];
                    load8<0>(past, t, len, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sdt[i] += w[i];
                    load8<0>(past + one, t, len, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sgB[i] += w[i];
                    load8<0>(past + 2 * one, t, len, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sv[i] += w[i];
                }
                if (!o.last) {
                    store8<0>(past, t, s.L, sdt);
                    store8<0>(past + one, t, s.L, sgB);
                    store8<0>(past + 2 * one, t, s.L, sv);
                }
            }
            if (o.last) {
                float slope[8];
                widen8<DT>(od, slope);
                slopes<DT>(slope, bias, s.softplus, t, t0 + kT, len);
                get_steps(m.dt, wave, lane, dt);
                get_steps(m.e, wave, lane, e);
                widen8<DT>(ox, xv);
                if (gated) {
                    float zslope[8];
                    get_steps(m.zslope, wave, lane, zslope);
#pragma unroll
                    for (int i = 0; i < 8; ++i) zslope[i] *= __builtin_fmaf(skip, xv[i], sv[i]);
                    store8<DT>(row_at<T>(m, kDz, own), t, len, zslope);
                }
                finish_steps(xv, slope, dt, e, skip, sdt, sgB, sb, sD);
                store8<DT>(row_at<T>(m, kDdelta, own), t, len, sdt);
                store8<DT>(row_at<T>(m, kDx, own), t, len, sgB);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kCh * kStates; i += 256) {
        const int c = i / kStates, j = i % kStates;
        if (c >= channels || j >= nn) continue;
        const int w = j / NS, turn = (c / 4 - w) & 3;
        const float *v = m.dA[w][turn][j % NS] + (c & 3) * 4;
        const long long at = ((long long)b * s.D + first + c) * s.N + n_first + j;
        o.dA[(long long)seg * s.B * s.D * s.N + at] = (v[0] + v[1]) + (v[2] + v[3]);
        if (s.d_initial_state && seg == 0) s.d_initial_state[at] = m.carry[c][j];
    }
    sD = row_sum(sD);
    sb = row_sum(sb);
    if (o.last && live && sub == 15) {
        const long long at = ((long long)seg * s.B + b) * s.D + d;
        o.dD[at] = sD;
        o.db[at] = sb;
    }
}

// Side by side: the blocks' sums added in order, then what the last of successive launches does.
// A wave per row, eight steps a lane.
template <int DT>
__global__ __launch_bounds__(256) void scan_bwd_finish_kernel(miconv_scan_t s, BwdOut o, int blocks) {
    typedef typename Elem<DT>::T T;
    const int lane = threadIdx.x & 63;
    const long long row = (long long)blockIdx.x * 4 + uniform(threadIdx.x >> 6), rows = (long long)s.B * s.D;
    if (row >= rows) return;
    const int b = (int)(row / s.D), d = (int)(row - (long long)b * s.D);
    const int len = valid_steps(s.lengths, b, s.L, o.t_first);
    const float bias = s.delta_bias ? s.delta_bias[d] : 0.0f, skip = s.D_skip ? s.D_skip[d] : 0.0f;
    float sD = 0.0f, sb = 0.0f;
    for (int t = lane * 8; t < s.L; t += 512) {
        float sum[3][8] = {}, x[8], dt[8], e[8], slope[8];
        for (int k = 0; k < blocks; ++k)
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                float w[8];
                load8<0>(o.sums + ((k * 3 + j) * rows + row) * s.L, t, len, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[j][i] += w[i];
            }
        load8<DT>(at_row<const T>(s.x, b, d), t, len, x);
        load8<DT>(at_row<const T>(s.delta, b, d), t, len, dt);
        load8<DT>(at_row<const T>(s.dy, b, d), t, len, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) slope[i] = dt[i];
        slopes<DT>(slope, bias, s.softplus, t, t + 8, len);
        step_sizes(dt, bias, s.softplus, t, t + 8, len);
        if (s.z.data) {
            float z[8], zslope[8];
            load8<DT>(at_row<const T>(s.z, b, d), t, len, z);
            gate<DT>(e, z, zslope);
#pragma unroll
            for (int i = 0; i < 8; ++i) zslope[i] *= __builtin_fmaf(skip, x[i], sum[2][i]);
            store8<DT>(at_row<T>(s.dz, b, d), t, len, zslope);
            if (len < s.L && t + 8 > len) zero_past<DT>(at_row<T>(s.dz, b, d), t, len, s.L);
        }
        finish_steps(x, slope, dt, e, skip, sum[0], sum[1], sb, sD);
        store8<DT>(at_row<T>(s.ddelta, b, d), t, len, sum[0]);
        store8<DT>(at_row<T>(s.dx, b, d), t, len, sum[1]);
        if (len < s.L && t + 8 > len) {
            zero_past<DT>(at_row<T>(s.ddelta, b, d), t, len, s.L);
            zero_past<DT>(at_row<T>(s.dx, b, d), t, len, s.L);
        }
    }
    sD = prefix_sum(sD);
    sb = prefix_sum(sb);
    if (lane == 63) {
        o.dD[row] = sD;
        o.db[row] = sb;
    }
}

// G at the end of every chunk, for a backward pass whose time segments run side by side:
// the forward kernel's scan with the lanes in reversed order of time, and no outputs but
// the values between chunks.  A wave per row, 64 lanes x 16 steps, the work-group's rows
// sharing C in LDS.  Few rows split this pass too: a wave per row and segment then starts
// from zero, notes the G that leaves its segment and the sums of dt, and a second kernel
// adds what comes from the segments after it.
struct Carry {
    float *G;                 // [B][D][chunks][N]
    float *ends, *after;      // [B][D][segs][N + 1] G and sum of dt; [B][D][chunks] dt up to the segment's end
    int segs, steps, t_first;
};

constexpr int kCarryWaves = 8, kCarryItems = 16, kCarryT = 64 * kCarryItems;

template <int DT>
__global__ __launch_bounds__(64 * kCarryWaves, 4) void scan_bwd_carry_kernel(miconv_scan_t s, Carry out, int blocks_g) {
    typedef typename Elem<DT>::T T;
    constexpr int kStage = 16, kEvery = kT / kCarryItems;
    __shared__ __attribute__((aligned(16))) float cs[kStage][kCarryT];     // [ITEMS / 4][lane][4]
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int per_group = s.D / s.G;
    const int blk = blockIdx.x % blocks_g, bg = blockIdx.x / blocks_g % (s.B * s.G), g = bg % s.G, b = bg / s.G;
    const int seg = blockIdx.x / (blocks_g * s.B * s.G), start = seg * out.steps;
    const int stop = out.segs == 1 || s.L - start < out.steps ? s.L : start + out.steps;
    const int in_group = blk * kCarryWaves + wave;
    const bool live = in_group < per_group;
    const int d = g * per_group + (live ? in_group : 0);
    const long long row = (long long)b * s.D + d;
    const int len = valid_steps(s.lengths, b, s.L, out.t_first), chunks = (s.L + kT - 1) / kT;
    const T *dl = at_row<const T>(s.delta, b, d), *dy = at_row<const T>(s.dy, b, d);
    const T *z = s.z.data ? at_row<const T>(s.z, b, d) : nullptr;
    const T *Cm = (const T *)s.Cm.data + b * s.Cm.stride_b + g * s.Cm.stride_g;
    const float bias = s.delta_bias ? s.delta_bias[d] : 0.0f;
    float carried = 0.0f, a_lane = 0.0f;               // lane n: state n
    if (lane < s.N) {
        if (s.d_final_state && out.segs == 1) carried = s.d_final_state[row * s.N + lane];
        a_lane = log2_decay(s.A[(long long)d * s.N + lane]);
    }
    float later = 0.0f;                                // dt from the chunk's end to the segment's
    for (int t0 = start + (stop - 1 - start) / kCarryT * kCarryT; t0 >= start; t0 -= kCarryT) {
        const int t = t0 + (63 - lane) * kCarryItems;
        float dt[kCarryItems], e[kCarryItems], sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kCarryItems; q += 8) {
            load8<DT>(dl, t + q, len, *(float (*)[8])(dt + q));
            load8<DT>(dy, t + q, len, *(float (*)[8])(e + q));
            if (z) {
                float zv[8];
                load8<DT>(z, t + q, len, zv);
#pragma unroll
                for (int i = 0; i < 8; ++i) e[q + i] *= zv[i] * logistic(zv[i]);
            }
        }
        step_sizes(dt, bias, s.softplus, t, t0 + kCarryT, len);
#pragma unroll
        for (int i = 0; i < kCarryItems; ++i) sum += dt[i];
        const int ends_here = t0 / kT + (64 - lane) / kEvery - 1;      // the chunk that ends where this lane begins
        const bool saves = live && lane % kEvery == 0 && ends_here * kT < stop;
        const float sums = prefix_sum(sum);
        if (out.segs > 1 && saves) out.after[row * chunks + ends_here] = later + (sums - sum);
        later += lane_of(sums, 63);
        for (int n0 = 0; n0 < s.N; n0 += kStage) {
            const int nn = s.N - n0 < kStage ? s.N - n0 : kStage;
            __syncthreads();
            for (int i = threadIdx.x; i < nn * (kCarryT / 8); i += 64 * kCarryWaves) {
                const int at = i % (kCarryT / 8) * 8, k = i / (kCarryT / 8);
                float w[8];
                load8<DT>(Cm + (n0 + k) * s.Cm.stride_n, t0 + at, len, w);
                float *to = cs[k] + (at % kCarryItems / 4) * 256 + (63 - at / kCarryItems) * 4;
                *(f32x4 *)to = f32x4{w[0], w[1], w[2], w[3]};
                *(f32x4 *)(to + 256) = f32x4{w[4], w[5], w[6], w[7]};
            }
            __syncthreads();
            for (int k = 0; k < nn; ++k) {
                const int n = n0 + k;
                const float a2 = lane_of(a_lane, n), G0 = lane_of(carried, n);
                float G = lane == 0 ? G0 : 0.0f;
#pragma unroll
                for (int i = kCarryItems - 4; i >= 0; i -= 4) {
                    const f32x4 c = *(const f32x4 *)(cs[k] + i * 64 + lane * 4);
#pragma unroll
                    for (int j = 3; j >= 0; --j) G = exp2_hw(dt[i + j] * a2) * __builtin_fmaf(c[j], e[i + j], G);
                }
                G = scan_lanes<64>(G, exp2_hw(a2 * sum));
                carried = keep(carried, G, n);
                G = cross_or<kWaveShr1>(G0, G);
                if (saves) out.G[(row * chunks + ends_here) * s.N + n] = G;
            }
        }
    }
    if (out.segs > 1 && live) {
        float *to = out.ends + (row * out.segs + seg) * (s.N + 1);
        if (lane < s.N) to[lane] = carried;
        if (lane == 0) to[s.N] = later;
    }
}

// G at every chunk's end: what the segment found plus what enters it from the right.  A
// thread per row and state, from the last segment to the first.
__global__ __launch_bounds__(256) void scan_bwd_chain_kernel(miconv_scan_t s, Carry out) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)s.B * s.D * s.N) return;
    const long long row = i / s.N;
    const int n = (int)(i - row * s.N), d = (int)(row % s.D), chunks = (s.L + kT - 1) / kT, per = out.steps / kT;
    const float a2 = log2_decay(s.A[(long long)d * s.N + n]);
    float G = s.d_final_state ? s.d_final_state[i] : 0.0f;
    for (int seg = out.segs - 1; seg >= 0; --seg) {
        const int last = (seg + 1) * per < chunks ? (seg + 1) * per : chunks;
        for (int c = seg * per; c < last; ++c) {
            float *at = out.G + (row * chunks + c) * s.N + n;
            *at = __builtin_fmaf(exp2_hw(a2 * out.after[row * chunks + c]), G, *at);
        }
        const float *end = out.ends + (row * out.segs + seg) * (s.N + 1);
        G = __builtin_fmaf(exp2_hw(a2 * end[s.N]), G, end[n]);
    }
}


// out[i] = sum over p of part[p][i] for several arrays: a work-group takes 256 consecutive i,
// a wave a share of the parts (four i per lane, so every load is 16 bytes next to its
// neighbours'); the waves' sums are added in order.  16 waves, because a short array has no other
// work to hide its loads behind (256 parts of 32 floats: with 4 waves 10.9 us, with 16 4.2).
constexpr int kSumWaves = 16;

struct SumJob {
    const float *part;
    float *out;
    long long n;
    int parts, add;           // add: to what out holds
    int row, row_out;         // out's rows of `row` are row_out apart, where that is more
};
struct SumJobs {
    SumJob j[5];
    long long first[6];       // first work-group of each array
    int count;
};

__global__ __launch_bounds__(64 * kSumWaves) void scan_bwd_sum(SumJobs jobs, uint32_t first_group) {
    __shared__ f32x4 share[kSumWaves][64];
    int k = 0;
    const long long group = (long long)first_group + blockIdx.x;
    while (k + 1 < jobs.count && group >= jobs.first[k + 1]) ++k;
    const SumJob j = jobs.j[k];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long i = (group - jobs.first[k]) * 256 + lane * 4;
    const int per = (j.parts + kSumWaves - 1) / kSumWaves, p0 = wave * per, p1 = p0 + per < j.parts ? p0 + per : j.parts;
    f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i + 4 <= j.n) {
        const float *src = j.part + i;
#pragma unroll 8
        for (int p = p0; p < p1; ++p) {
            const u32x4 v = *(const u32x4_row *)(src + p * j.n);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] += __uint_as_float(v[e]);
        }
    } else if (i < j.n) {
        // the array's last lane: what lies past the end repeats the last value and is not stored
#pragma unroll 4
        for (int p = p0; p < p1; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] += j.part[p * j.n + (i + e < j.n ? i + e : j.n - 1)];
    }
    share[wave][lane] = a;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < kSumWaves; ++w) a += share[w][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < j.n) {
                long long at = i + e;
                if (j.row < j.row_out) at += at / j.row * (j.row_out - j.row);
                j.out[at] = j.add ? j.out[at] + a[e] : a[e];
            }
    }
}

}  // namespace

// Where the groups of 16 channels give the 256 CUs (two work-groups each) half of what they hold or less,
// the time axis can be split too, at the price of a pass that finds G between the segments.
// It is where the estimate for N = 16, bf16 gains: a chunk takes 11 us of a work-group alone on its CU and 14 of
// two, 1024 steps of the pass between 12 and 20 (4096 rows of 512: 60 us whole, 68 in two; of 1024: 105 and
// 95; 1024 rows of 256: 32 and 35; of 512: 54 and 37).  `whole` takes neither segments nor blocks of states
// side by side: the least workspace.
static ScanBwdPlan plan_rows(const miconv_scan_t &s, bool whole) {
    ScanBwdPlan p;
    p.parts = (s.D / s.G + kCh - 1) / kCh;
    const long long groups = (long long)s.B * s.G * p.parts;
    const int chunks = scan_chunks(s.L);
    p.segs = 1;
    p.seg_chunks = chunks;
    p.carry_segs = 1;
    p.carry_steps = 0;
    if (groups * 2 <= 512 && chunks > 1 && !whole) {
        const long long segs = 512 / groups < chunks ? 512 / groups : chunks;
        const int seg_chunks = (int)((chunks + segs - 1) / segs);
        // the pass between the segments is split as the forward scan is
        const long long rows_groups = (long long)s.B * s.G * ((s.D / s.G + kCarryWaves - 1) / kCarryWaves);
        const int long_chunks = (s.L + kCarryT - 1) / kCarryT;
        int per = long_chunks;
        if (rows_groups <= 128 && long_chunks >= 3) {
            const long long n = 512 / rows_groups < long_chunks ? 512 / rows_groups : long_chunks;
            per = (int)((long_chunks + n - 1) / n);
        }
        const double between = 3 + per * (rows_groups <= 256 ? 12.0 : rows_groups <= 512 ? 20.0 : 20.0 * rows_groups / 512);
        if (seg_chunks * (groups * segs <= 256 ? 11.0 : 14.0) + between < chunks * 11.0) {
            p.seg_chunks = seg_chunks;
            p.segs = (chunks + seg_chunks - 1) / seg_chunks;
            p.carry_segs = (long_chunks + per - 1) / per;
            p.carry_steps = per < long_chunks ? per * kCarryT : 0;
        }
    }
    // blocks of 16 states side by side where one of them leaves CUs without a second work-group (64
    // states, bf16: 1024 rows of 300 170 -> 64 us, 4096 of 128 81 -> 62, 4 x 100 of 2, with the
    // forward pass, 106 -> 58; a block of one state costs: 17 states, 4096 rows of 100 45 -> 48)
    p.beside = s.N > kStates && groups * p.segs <= 256 && !whole ? (s.N + kStates - 1) / kStates : 1;
    const size_t bc = (size_t)p.parts * s.B * s.G * s.N * s.L, bd = (size_t)s.B * s.D;
    p.off_dB = 0;
    p.off_dC = bc;
    p.off_dA = 2 * bc;
    p.off_dD = p.off_dA + bd * s.N * p.segs;
    p.off_db = p.off_dD + bd * p.segs;
    p.off_G = p.off_db + bd * p.segs;
    p.off_ends = p.off_G + (p.segs > 1 ? bd * chunks * s.N : 0);
    p.off_after = p.off_ends + (p.carry_segs > 1 ? bd * p.carry_segs * (s.N + 1) : 0);
    p.off_sums = p.off_after + (p.carry_segs > 1 ? bd * chunks : 0);
    p.bytes = (p.off_sums + (s.N > kStates ? 3 * bd * s.L * p.beside : 0)) * 4;
    return p;
}

ScanBwdPlan plan_scan_bwd(const miconv_scan_t &s, size_t budget) {
    const ScanBwdPlan p = plan_rows(s, false);
    return p.bytes <= budget ? p : plan_rows(s, true);
}

// Of `sequences` sequences from b on, the channels from `first` on in groups from g on, and the steps from t on.
// More than one sequence goes with all groups and channels, more than one group with all channels.
static miconv_scan_t slice_of(const miconv_scan_t &s, size_t es, int b, int sequences, int g, int groups, size_t first,
                              int channels, int t, int steps) {
    miconv_scan_t r = s;
    const size_t row = (size_t)b * s.D + first;
    r.B = sequences;
    r.G = groups;
    r.D = groups * channels;
    r.L = steps;
    for (miconv_rows_t *v : {&r.x, &r.delta, &r.z, &r.dy, &r.dx, &r.ddelta, &r.dz})
        if (v->data) v->data = (char *)v->data + ((size_t)b * v->stride_b + first * v->stride_d + t) * es;
    for (miconv_scan_in_t *v : {&r.Bm, &r.Cm}) v->data = (char *)v->data + ((size_t)b * v->stride_b + (size_t)g * v->stride_g + t) * es;
    if (s.lengths) r.lengths = s.lengths + b;
    r.A = s.A + first * s.N;
    if (s.D_skip) r.D_skip = s.D_skip + first;
    if (s.delta_bias) r.delta_bias = s.delta_bias + first;
    r.states = s.states + (row * scan_chunks(s.L) + t / kScanChunk) * s.N;
    if (s.d_final_state) r.d_final_state = s.d_final_state + row * s.N;
    if (s.d_initial_state) r.d_initial_state = s.d_initial_state + row * s.N;
    r.dA = s.dA + first * s.N;
    if (s.dD) r.dD = s.dD + first;
    if (s.ddelta_bias) r.ddelta_bias = s.ddelta_bias + first;
    const size_t bc = ((size_t)b * s.G + g) * s.N * s.L + t;
    r.dB = s.dB + bc;
    r.dC = s.dC + bc;
    return r;
}

// The most of `n`, in equal shares of whole `unit`s, whose bytes(share) fit the budget; one unit if none do.
template <typename F>
static int share_within(int n, int unit, size_t budget, F bytes) {
    if (n <= unit || bytes(n) <= budget) return n;
    int fits = 1, over = (n + unit - 1) / unit;                   // units
    while (over - fits > 1) {
        const int mid = fits + (over - fits) / 2;
        (bytes(mid * unit) <= budget ? fits : over) = mid;
    }
    const int most = fits * unit, shares = (n + most - 1) / most, even = (n + shares - 1) / shares;
    return (even + unit - 1) / unit * unit;
}

// Slices cost least where each still gives the CUs their two work-groups each (512): so sequences are
// sliced down to that, then the time axis, which only adds launches, then the rows left.
// (In 10^9 bytes and in what they take whole, bf16: 8 x 8192 rows of 8192, N 16: 8.4 ms in 8 slices, 7.9 whole in
// 4.3 GB; 1 x 8192 of 65536: 8.3 in 5, 8.1 in 4.3 GB; 2 x 8192 of 8192, N 64: 9.2 in 8, 8.7 in 5.9 GB.)
ScanBwdSlice slice_scan_bwd(const miconv_scan_t &s, size_t budget) {
    const int per_group = s.D / s.G, chunks = scan_chunks(s.L);
    ScanBwdSlice r = {s.B, s.G, per_group, s.L, 0, 0};
    const auto size = [&](bool whole) {
        miconv_scan_t one = s;
        one.B = r.sequences;
        one.G = r.groups;
        one.D = r.groups * r.channels;
        one.L = r.steps;
        r.carry = r.steps < s.L ? 2 * (size_t)one.B * one.D * s.N : 0;
        r.bytes = r.carry * 4 + plan_rows(one, whole).bytes;
        return r.bytes;
    };
    if (size(false) <= budget) return r;
    const long long per_sequence = (long long)s.G * ((per_group + kCh - 1) / kCh);
    const int filling = (int)(per_sequence >= 512 ? 1 : (512 + per_sequence - 1) / per_sequence);
    if (s.B > filling) {
        r.sequences = share_within(s.B, 1, budget, [&](int n) { r.sequences = n; return size(false); });
        if (r.sequences < filling) r.sequences = filling;
    }
    const auto sliced = [&](int n) {
        r.steps = n < chunks ? n * kT : s.L;
        return size(false);
    };
    if (size(false) > budget) sliced(share_within(chunks, 1, budget, sliced));
    if (r.bytes > budget && r.sequences > 1) {
        r.sequences = share_within(r.sequences, 1, budget, [&](int n) { r.sequences = n; return size(false); });
        size(false);
    }
    if (r.bytes > budget && r.groups > 1) {
        r.groups = share_within(s.G, 1, budget, [&](int n) { r.groups = n; return size(false); });
        size(false);
    }
    if (r.bytes > budget) {
        r.channels = share_within(per_group, kCh, budget, [&](int n) { r.channels = n; return size(false); });
        size(false);
    }
    if (r.bytes > budget) size(true);
    return r;
}

// What one slice does about the others.
struct BwdPlace {
    int add_bc, add_rest;     // dB and dC, the other sums over sequences hold those of earlier slices
    int t, L;                 // its first step, all steps
};

static int launch_slice(const miconv_scan_t &s, int dtype, size_t budget, const BwdPlace &place, float *ws, hipStream_t st) {
    const ScanBwdPlan p = plan_scan_bwd(s, budget);
    BwdOut o;
    o.dB = ws + p.off_dB;
    o.dC = ws + p.off_dC;
    o.dA = ws + p.off_dA;
    o.dD = ws + p.off_dD;
    o.db = ws + p.off_db;
    o.G = p.segs > 1 ? ws + p.off_G : nullptr;
    o.sums = s.N > kStates ? ws + p.off_sums : nullptr;
    o.parts = p.parts;
    o.segs = p.segs;
    o.seg_chunks = p.seg_chunks;
    o.t_first = place.t;
    o.chunks = scan_chunks(place.L);
    if (p.segs > 1) {
        const int blocks_g = (s.D / s.G + kCarryWaves - 1) / kCarryWaves;
        const Carry out = {ws + p.off_G, ws + p.off_ends, ws + p.off_after, p.carry_segs, p.carry_steps, place.t};
        const dim3 cgrid((unsigned)((long long)s.B * s.G * blocks_g * p.carry_segs)), cblock(64 * kCarryWaves);
        if (dtype)
            hipLaunchKernelGGL(scan_bwd_carry_kernel<1>, cgrid, cblock, 0, st, s, out, blocks_g);
        else
            hipLaunchKernelGGL(scan_bwd_carry_kernel<0>, cgrid, cblock, 0, st, s, out, blocks_g);
        if (p.carry_segs > 1)
            hipLaunchKernelGGL(scan_bwd_chain_kernel, dim3((unsigned)(((long long)s.B * s.D * s.N + 255) / 256)), dim3(256),
                               0, st, s, out);
        if (hipGetLastError() != hipSuccess) return MICONV_ERR_HIP;
    }
    const int per_launch = kStates * p.beside;
    for (int n = 0; n < s.N; n += per_launch) {
        o.n_first = n;
        o.n_end = s.N < n + per_launch ? s.N : n + per_launch;
        o.last = p.beside == 1 && o.n_end == s.N;
        const int nn = o.n_end - n;
        // as few states per wave as give each of the four waves some
        const void *kern = nn <= 4   ? (dtype ? (const void *)scan_bwd_kernel<1, 1> : (const void *)scan_bwd_kernel<0, 1>)
                           : nn <= 8 ? (dtype ? (const void *)scan_bwd_kernel<1, 2> : (const void *)scan_bwd_kernel<0, 2>)
                                     : (dtype ? (const void *)scan_bwd_kernel<1, 4> : (const void *)scan_bwd_kernel<0, 4>);
        const int bad = launch_groups((long long)s.B * s.G * p.parts * p.segs, 256, [&](unsigned groups, unsigned first) {
            miconv_scan_t a = s;
            void *args[] = {(void *)&a, (void *)&o, (void *)&first};
            (void)hipLaunchKernel(kern, dim3(groups, (unsigned)p.beside), dim3(256), args, 0, st);
        });
        if (bad != MICONV_OK) return bad;
    }
    const int time_parts = p.beside > 1 ? 1 : p.segs;     // of dD and the bias's gradient
    if (p.beside > 1) {
        const dim3 rows((unsigned)(((long long)s.B * s.D + 3) / 4));
        if (dtype)
            hipLaunchKernelGGL(scan_bwd_finish_kernel<1>, rows, dim3(256), 0, st, s, o, p.beside);
        else
            hipLaunchKernelGGL(scan_bwd_finish_kernel<0>, rows, dim3(256), 0, st, s, o, p.beside);
        if (hipGetLastError() != hipSuccess) return MICONV_ERR_HIP;
    }
    SumJobs jobs = {};
    const long long bc = (long long)s.B * s.G * s.N * s.L;
    jobs.j[jobs.count++] = {o.dB, s.dB, bc, p.parts, place.add_bc, s.L, place.L};
    jobs.j[jobs.count++] = {o.dC, s.dC, bc, p.parts, place.add_bc, s.L, place.L};
    jobs.j[jobs.count++] = {o.dA, s.dA, (long long)s.D * s.N, s.B * p.segs, place.add_rest, 0, 0};
    if (s.dD) jobs.j[jobs.count++] = {o.dD, s.dD, s.D, s.B * time_parts, place.add_rest, 0, 0};
    if (s.ddelta_bias) jobs.j[jobs.count++] = {o.db, s.ddelta_bias, s.D, s.B * time_parts, place.add_rest, 0, 0};
    for (int k = 0; k < jobs.count; ++k) jobs.first[k + 1] = jobs.first[k] + (jobs.j[k].n + 255) / 256;
    return launch_groups(jobs.first[jobs.count], 64 * kSumWaves, [&](unsigned groups, unsigned first) {
        hipLaunchKernelGGL(scan_bwd_sum, dim3(groups), dim3(64 * kSumWaves), 0, st, jobs, first);
    });
}

int launch_scan_bwd(const miconv_scan_t &s, int dtype, const ScanBwdSlice &slice, float *ws, hipStream_t st) {
    const int per_group = s.D / s.G, last = (s.L - 1) / slice.steps;
    const size_t budget = slice.bytes - slice.carry * 4;
    float *const carry[2] = {ws, ws + slice.carry / 2};
    const auto left = [](long long n, int most) { return (int)(n < most ? n : most); };
    for (long long b = 0; b < s.B; b += slice.sequences)
        for (long long g = 0; g < s.G; g += slice.groups)
            for (long long d = 0; d < per_group; d += slice.channels)
                for (int k = last; k >= 0; --k) {
                    const BwdPlace place = {d > 0, b > 0 || k < last, k * slice.steps, s.L};
                    miconv_scan_t part = slice_of(s, dtype ? 2 : 4, (int)b, left(s.B - b, slice.sequences), (int)g,
                                                  left(s.G - g, slice.groups), (size_t)g * per_group + d,
                                                  left(per_group - d, slice.channels), place.t, left(s.L - place.t, slice.steps));
                    if (k < last) part.d_final_state = carry[(k + 1) & 1];
                    if (k > 0) part.d_initial_state = carry[k & 1];
                    const int bad = launch_slice(part, dtype, budget, place, ws + slice.carry, st);
                    if (bad != MICONV_OK) return bad;
                }
    return MICONV_OK;
}

}  // namespace miconv
