// scan_fwd.hip -- selective scan, forward, and its one-token step.
//
//   h_t[n] = exp(dt_t A[n]) h_{t-1}[n] + dt_t x_t B_t[n],  v_t = sum_n C_t[n] h_t[n] + D x_t
//
// The map h -> a h + b composes: (a1, b1) then (a2, b2) is (a1 a2, a2 b1 + b2).  A row
// (sequence, channel) is taken by LANES lanes x ITEMS time steps at a time: each lane
// runs its steps from a zero state, the lanes' maps are combined by a prefix scan, and
// each lane runs its steps again from its true entry state.
//
// Bound by the vector ALUs, not by memory: a (step, state) pair costs seven slots of
// four cycles -- argument, exponential (two), input, and a multiply-add each for the two
// runs and for C h -- against 8 bytes per step for N = 16 pairs of them (bf16).  So
//   - a lane crossing of the scan is part of its fma (DPP), and what enters the chunk is
//     the first lane's start: the scan costs 26 slots;
//   - 16 steps per lane where the row is long enough to share it;
//   - B and C are widened to fp32 once per work-group, in LDS, for its channels.
// 1 x 4096 rows of 4096, N 16, bf16: 90 us, 3.0 T pairs/s; 10.5 instructions per pair with the
// per-step work (softplus, gate, conversions, staging), the ALUs busy 90 % of the time.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int kThreads = 256;

// Work-groups of 8 waves; 64 lanes x 16 or 8 steps per row, or four rows of 16 lanes x 8 steps per
// wave.  SHARE: the waves take the same four rows and an eighth of the states each, their parts of
// v meeting in LDS: few short rows then wait for N / 8 states rather than N.
constexpr int kScanWaves = 8;

template <int DT, int LANES, int ITEMS, bool SHARE = false>
__global__ __launch_bounds__(64 * kScanWaves, 4) void scan_fwd_kernel(miconv_scan_t s, int blocks_g, ScanSplit split,
                                                                        uint32_t first_group) {
    typedef typename Elem<DT>::T T;
    constexpr int kT = LANES * ITEMS, kRows = 64 / LANES, kEvery = kScanChunk / ITEMS, kPairs = kT * 2 * 4;   // bytes of B and C per state
    constexpr int kStage = SHARE ? 32 : 65536 / kPairs < 16 ? 65536 / kPairs : 16;            // states staged at a time
    // [state][B, C][ITEMS / 4][LANES][4]: a lane reads four steps as 16 bytes next to its neighbours'
    __shared__ __attribute__((aligned(16))) float bc[kStage * 2 * kT];
    // 16 lanes per row: A[n] log2(e) and the state n between chunks, of each row
    constexpr int kHeld = LANES == 64 ? 1 : SHARE ? kRows : kScanWaves * kRows;
    __shared__ float a_rows[kHeld][MICONV_SCAN_MAX_STATES], h_rows[kHeld][MICONV_SCAN_MAX_STATES];
    // SHARE: the waves' parts of v, [wave][row][step]
    __shared__ __attribute__((aligned(16))) float parts[SHARE ? kScanWaves * kRows * kT : 1];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), sub = lane % LANES;
    const int per_group = s.D / s.G;
    const uint32_t group = first_group + blockIdx.x;
    const int blk = group % blocks_g, bg = group / blocks_g % (s.B * s.G), g = bg % s.G, b = bg / s.G;
    const int seg = group / (blocks_g * s.B * s.G), start = seg * split.steps;
    const int stop = split.segs == 1 || s.L - start < split.steps ? s.L : start + split.steps;
    const int in_group = (SHARE ? blk : blk * kScanWaves + wave) * kRows + lane / LANES;
    const bool live = in_group < per_group;              // the last work-group's other rows only help to stage
    const int d = g * per_group + (live ? in_group : 0);
    const long long row = (long long)b * s.D + d;
    const int len = valid_steps(s.lengths, b, s.L);
    const T *x = (const T *)s.x.data + b * s.x.stride_b + d * s.x.stride_d;
    const T *dl = (const T *)s.delta.data + b * s.delta.stride_b + d * s.delta.stride_d;
    const T *z = s.z.data ? (const T *)s.z.data + b * s.z.stride_b + d * s.z.stride_d : nullptr;
    T *y = (T *)s.y.data + b * s.y.stride_b + d * s.y.stride_d;
    const T *Bm = (const T *)s.Bm.data + b * s.Bm.stride_b + g * s.Bm.stride_g;
    const T *Cm = (const T *)s.Cm.data + b * s.Cm.stride_b + g * s.Cm.stride_g;
    const float skip = s.D_skip ? s.D_skip[d] : 0.0f, bias = s.delta_bias ? s.delta_bias[d] : 0.0f;
    const int saved = scan_chunks(s.L);
    // 64 lanes per row: lane n holds them for state n
    const int my = LANES == 64 ? 0 : (SHARE ? 0 : wave * kRows) + lane / LANES;
    // SHARE: wave w has the states w, w + 8, ...
    constexpr int kStride = SHARE ? kScanWaves : 1;
    const int n_mine = SHARE ? wave : 0;
    float carried = 0.0f, a_lane = 0.0f;
    if constexpr (LANES == 64) {
        if (lane < s.N) {
            if (split.segs > 1)
                carried = split.entry[(row * split.segs + seg) * s.N + lane];
            else if (s.initial_state)
                carried = s.initial_state[row * s.N + lane];
            a_lane = log2_decay(s.A[(long long)d * s.N + lane]);
        }
    } else {
        for (int n = n_mine + sub * kStride; n < s.N; n += LANES * kStride) {
            h_rows[my][n] = s.initial_state ? s.initial_state[row * s.N + n] : 0.0f;
            a_rows[my][n] = log2_decay(s.A[(long long)d * s.N + n]);
        }
        wave_lds_sync();
    }
    // Work-groups that share a CU: the older one would be served first and the last one end alone,
    // at a part of the ALUs' rate.  The one with more stages left goes first (2 x 4096 rows of 2048:
    // 98 -> 90 us, of 4096: 178 -> 163; 3 x 1536 of 1000, fp32, whose last work-groups start as the first
    // end: 43 -> 45).
    __builtin_amdgcn_s_setprio(3);
    const int stages = ((len < stop ? len : stop) - start + kT - 1) / kT * ((s.N + kStage - 1) / kStage);
    int left = stages;
    int t0 = start;
    for (; t0 < len && t0 < stop; t0 += kT) {
        const int c = t0 / kScanChunk, t = t0 + sub * ITEMS;
        float xv[ITEMS], dt[ITEMS], v[ITEMS], sum = 0.0f;
#pragma unroll
        for (int q = 0; q < ITEMS; q += 8) {
            load8<DT>(x, t + q, len, *(float (*)[8])(xv + q));
            load8<DT>(dl, t + q, len, *(float (*)[8])(dt + q));
        }
        step_sizes(dt, bias, s.softplus, t, t0 + kT, len);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            sum += dt[i];
            v[i] = !SHARE || wave == 0 ? skip * xv[i] : 0.0f;
            xv[i] *= dt[i];
        }
        for (int n0 = 0; n0 < s.N; n0 += kStage) {
            const int nn = s.N - n0 < kStage ? s.N - n0 : kStage;
            --left;
            if (left == 0) __builtin_amdgcn_s_setprio(0);
            else if (left * 4 <= stages) __builtin_amdgcn_s_setprio(1);
            else if (left * 2 <= stages) __builtin_amdgcn_s_setprio(2);
            __syncthreads();
            // where this thread's eight steps of a staged row are, and go to
            const int tid = again(threadIdx.x), at = tid % (kT / 8) * 8;
            float *const to = bc + (at % ITEMS / 4) * LANES * 4 + at / ITEMS * 4;
            for (int which = tid / (kT / 8); which < 2 * nn; which += 64 * kScanWaves / (kT / 8)) {
                const int n = n0 + (which >> 1);
                float w[8];
                load8<DT>(which & 1 ? Cm + n * s.Cm.stride_n : Bm + n * s.Bm.stride_n, t0 + at, len, w);
                *(f32x4 *)(to + which * kT) = f32x4{w[0], w[1], w[2], w[3]};
                *(f32x4 *)(to + which * kT + LANES * 4) = f32x4{w[4], w[5], w[6], w[7]};
            }
            __syncthreads();
            for (int k = n_mine; k < nn; k += kStride) {
                const int n = n0 + k;
                float a2, h0;
                if constexpr (LANES == 64) {
                    a2 = lane_of(a_lane, n);
                    h0 = lane_of(carried, n);
                } else {
                    a2 = a_rows[my][n];
                    h0 = h_rows[my][n];
                }
                const float *pb = bc + k * 2 * kT + sub * 4, *pc = pb + kT;
                float a[ITEMS], bv[ITEMS], h = sub == 0 ? h0 : 0.0f;
#pragma unroll
                for (int i = 0; i < ITEMS; i += 4) {
                    const f32x4 q = *(const f32x4 *)(pb + i * LANES);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a[i + e] = exp2_hw(dt[i + e] * a2);
                        bv[i + e] = q[e] * xv[i + e];
                        h = __builtin_fmaf(a[i + e], h, bv[i + e]);
                    }
                }
                h = scan_lanes<LANES>(h, exp2_hw(a2 * sum));
                if constexpr (LANES == 64) {
                    carried = keep(carried, h, n);
                    h = cross_or<kWaveShr1>(h0, h);
                } else {
                    if (sub == LANES - 1) h_rows[my][n] = h;
                    h = cross_or<kRowShr + 1>(h0, h);
                }
                // lanes at the start of a saved chunk hold its entry state
                if (s.states && live && sub % kEvery == 0 && c + sub / kEvery < saved)
                    s.states[(row * saved + c + sub / kEvery) * s.N + n] = h;
#pragma unroll
                for (int i = 0; i < ITEMS; i += 4) {
                    const f32x4 q = *(const f32x4 *)(pc + i * LANES);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h = __builtin_fmaf(a[i + e], h, bv[i + e]);
                        v[i + e] = __builtin_fmaf(q[e], h, v[i + e]);
                    }
                }
            }
        }
        if constexpr (SHARE) {
            float *const to = parts + (wave * kRows + lane / LANES) * kT + sub * ITEMS;
#pragma unroll
            for (int i = 0; i < ITEMS; i += 4) *(f32x4 *)(to + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
            __syncthreads();
            static_assert(kRows * kT == 64 * kScanWaves, "a step of a row per thread");
            const int r = threadIdx.x / kT, step = threadIdx.x % kT, at = t0 + step, dr = blk * kRows + r;
            if (dr < per_group && at < s.L) {
                const int dd = g * per_group + dr;
                float out = 0.0f;
#pragma unroll
                for (int w = 0; w < kScanWaves; ++w) out += parts[(w * kRows + r) * kT + step];
                if (s.z.data && at < len) {
                    const float zv = Elem<DT>::get(((const T *)s.z.data + b * s.z.stride_b + dd * s.z.stride_d)[at]);
                    out *= zv * logistic_for<DT>(zv);
                }
                ((T *)s.y.data + b * s.y.stride_b + dd * s.y.stride_d)[at] = Elem<DT>::put(at < len ? out : 0.0f);
            }
        } else if (live) {
#pragma unroll
            for (int q = 0; q < ITEMS; q += 8) {
                float (&out)[8] = *(float (*)[8])(v + q);
                if (t + q >= len) break;
                if (z) {
                    float zv[8];
                    load8<DT>(z, t + q, len, zv);
#pragma unroll
                    for (int i = 0; i < 8; ++i) out[i] *= zv[i] * logistic_for<DT>(zv[i]);
                }
                store8<DT>(y, t + q, len, out);
            }
        }
    }
    if (!live) return;
    if constexpr (LANES == 16) wave_lds_sync();
    for (int n = n_mine + sub * kStride; n < s.N; n += LANES * kStride) {
        const float h = LANES == 64 ? carried : h_rows[my][n];
        if (s.final_state && stop == s.L) s.final_state[row * s.N + n] = h;
        // chunks past the end: the state stays
        if (s.states)
            for (int c = t0 / kScanChunk; c * kScanChunk < stop; ++c) s.states[(row * saved + c) * s.N + n] = h;
    }
    if (SHARE && wave) return;
    // what lies past the end is not computed (an infinite state would make padding NaN)
    const int past = SHARE ? t0 : (len < start ? start : len);
    for (int t = past + sub * 8; t < stop; t += LANES * 8) {
        const float zero[8] = {};
        store8<DT>(y, t, stop, zero);
    }
}

// Few rows and a long time axis: the state that each segment would end with from zero, and
// its sum of dt.  A wave per row and segment of split.steps (a multiple of 1024).
template <int DT>
__global__ __launch_bounds__(64 * kScanWaves, 4) void scan_local_kernel(miconv_scan_t s, int blocks_g, ScanSplit split) {
    typedef typename Elem<DT>::T T;
    constexpr int ITEMS = 16, kT = 64 * ITEMS, kStage = 16;
    __shared__ __attribute__((aligned(16))) float bs[kStage][kT];       // [ITEMS / 4][lane][4]
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int per_group = s.D / s.G;
    const int blk = blockIdx.x % blocks_g, bg = blockIdx.x / blocks_g % (s.B * s.G), g = bg % s.G, b = bg / s.G;
    const int seg = blockIdx.x / (blocks_g * s.B * s.G), start = seg * split.steps;
    const int stop = s.L - start < split.steps ? s.L : start + split.steps;
    const int in_group = blk * kScanWaves + wave;
    const bool live = in_group < per_group;
    const int d = g * per_group + (live ? in_group : 0);
    const long long row = (long long)b * s.D + d;
    const int len = valid_steps(s.lengths, b, s.L);
    const T *x = (const T *)s.x.data + b * s.x.stride_b + d * s.x.stride_d;
    const T *dl = (const T *)s.delta.data + b * s.delta.stride_b + d * s.delta.stride_d;
    const T *Bm = (const T *)s.Bm.data + b * s.Bm.stride_b + g * s.Bm.stride_g;
    const float bias = s.delta_bias ? s.delta_bias[d] : 0.0f;
    const float a_lane = lane < s.N ? log2_decay(s.A[(long long)d * s.N + lane]) : 0.0f;
    float carried = 0.0f, total = 0.0f;
    for (int t0 = start; t0 < len && t0 < stop; t0 += kT) {
        const int t = t0 + lane * ITEMS;
        float xv[ITEMS], dt[ITEMS], sum = 0.0f;
#pragma unroll
        for (int q = 0; q < ITEMS; q += 8) {
            load8<DT>(x, t + q, len, *(float (*)[8])(xv + q));
            load8<DT>(dl, t + q, len, *(float (*)[8])(dt + q));
        }
        step_sizes(dt, bias, s.softplus, t, t0 + kT, len);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            sum += dt[i];
            xv[i] *= dt[i];
        }
        total += lane_of(prefix_sum(sum), 63);
        for (int n0 = 0; n0 < s.N; n0 += kStage) {
            const int nn = s.N - n0 < kStage ? s.N - n0 : kStage;
            __syncthreads();
            for (int i = threadIdx.x; i < nn * (kT / 8); i += 64 * kScanWaves) {
                const int at = i % (kT / 8) * 8, k = i / (kT / 8);
                float w[8];
                load8<DT>(Bm + (n0 + k) * s.Bm.stride_n, t0 + at, len, w);
                float *to = bs[k] + (at % ITEMS / 4) * 256 + at / ITEMS * 4;
                *(f32x4 *)to = f32x4{w[0], w[1], w[2], w[3]};
                *(f32x4 *)(to + 256) = f32x4{w[4], w[5], w[6], w[7]};
            }
            __syncthreads();
            for (int k = 0; k < nn; ++k) {
                const int n = n0 + k;
                const float a2 = lane_of(a_lane, n);
                const float h0 = lane_of(carried, n);
                float h = lane == 0 ? h0 : 0.0f;
#pragma unroll
                for (int i = 0; i < ITEMS; i += 4) {
                    const f32x4 q = *(const f32x4 *)(bs[k] + i * 64 + lane * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h = __builtin_fmaf(exp2_hw(dt[i + e] * a2), h, q[e] * xv[i + e]);
                }
                h = scan_lanes<64>(h, exp2_hw(a2 * sum));
                carried = keep(carried, h, n);
            }
        }
    }
    if (!live) return;
    if (lane < s.N) split.entry[(row * split.segs + seg) * s.N + lane] = carried;
    if (lane == 0) split.sums[row * split.segs + seg] = total;
}

// The state before each segment, in place of its local end.  A thread per row and state.
__global__ __launch_bounds__(kThreads) void scan_chain_kernel(miconv_scan_t s, ScanSplit split) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)s.B * s.D * s.N) return;
    const long long row = i / s.N;
    const int n = (int)(i - row * s.N), d = (int)(row % s.D);
    const float a2 = log2_decay(s.A[(long long)d * s.N + n]);
    float h = s.initial_state ? s.initial_state[i] : 0.0f;
    for (int seg = 0; seg < split.segs; ++seg) {
        float *at = split.entry + (row * split.segs + seg) * s.N + n;
        const float local = *at;
        *at = h;
        h = __builtin_fmaf(exp2_hw(a2 * split.sums[row * split.segs + seg]), h, local);
    }
}

// One time step.  Memory bound: 8 bytes per state, read and written once.  PER lanes per
// (sequence, channel), four states each, so that consecutive lanes read consecutive 16
// bytes of the states; their products with C are added across the lanes.  VEC: N is a
// multiple of 4, the states are 16-byte aligned, B and C have their states next to each other.  All reads of a state come before its
// writes, so state_out may be state.  Such states pass by the caches: those of a model's layers
// together do not fit them from one token to the next (32 layers in turn, bf16, N 16, a step of 2.1 MB of states
// 3.98 -> 3.59 us, of 16.8 MB 11.4 -> 9.8, of 67 MB 33.3 -> 31.5; one layer's alone, read again at once, 3.3 us
// either way, 9.4 -> 9.1 and 28.3 -> 31.2).
template <int DT, int PER, bool VEC>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(miconv_scan_t s, const float *state, int slots,
                                                             const int *slot_of, float *state_out, FDiv fd_D,
                                                             FDiv fd_group, uint32_t first_group) {
    typedef typename Elem<DT>::T T;
    const int sub = threadIdx.x % PER, n0 = sub * 4;
    const uint32_t i = (first_group + blockIdx.x) * (kThreads / PER) + threadIdx.x / PER;     // rows are at most 2^30
    if (i >= (uint32_t)s.B * (uint32_t)s.D) return;
    const int b = (int)fdiv(i, fd_D), d = (int)i - b * s.D, g = (int)fdiv(d, fd_group);
    const int slot = slot_of ? slot_of[b] : b;
    T *yo = (T *)s.y.data + b * s.y.stride_b + d * s.y.stride_d;
    if (slot < 0 || slot >= slots) {
        if (sub == 0) *yo = Elem<DT>::put(0.0f);
        return;
    }
    const long long so = ((long long)slot * s.D + d) * s.N + n0;
    const T *Bm = (const T *)s.Bm.data + b * s.Bm.stride_b + g * s.Bm.stride_g;
    const T *Cm = (const T *)s.Cm.data + b * s.Cm.stride_b + g * s.Cm.stride_g;
    const float *A = s.A + (long long)d * s.N + n0;
    float h[4], a[4], bv[4], cv[4];
    if (VEC && n0 < s.N) {
        const f32x4 hv = __builtin_nontemporal_load((const f32x4 *)(state + so));
        const u32x4 av = *(const u32x4_row *)A;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[e] = hv[e];
            a[e] = __uint_as_float(av[e]);
        }
        load4<DT>(Bm + n0, bv);
        load4<DT>(Cm + n0, cv);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool in = n0 + e < s.N;
        if (!VEC || n0 >= s.N) {
            h[e] = in ? state[so + e] : 0.0f;
            a[e] = in ? A[e] : 0.0f;
            bv[e] = in ? Elem<DT>::get(Bm[(n0 + e) * s.Bm.stride_n]) : 0.0f;
            cv[e] = in ? Elem<DT>::get(Cm[(n0 + e) * s.Cm.stride_n]) : 0.0f;
        }
    }
    const float x = Elem<DT>::get(((const T *)s.x.data)[b * s.x.stride_b + d * s.x.stride_d]);
    const float raw = Elem<DT>::get(((const T *)s.delta.data)[b * s.delta.stride_b + d * s.delta.stride_d]) +
                      (s.delta_bias ? s.delta_bias[d] : 0.0f);
    const float z = s.z.data ? Elem<DT>::get(((const T *)s.z.data)[b * s.z.stride_b + d * s.z.stride_d]) : 0.0f;
    const float dt = s.softplus ? softplus(raw) : raw, dtx = dt * x;
    float v = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = __builtin_fmaf(exp2_hw(dt * log2_decay(a[e])), h[e], dtx * bv[e]);
        v = __builtin_fmaf(cv[e], h[e], v);
    }
    if (VEC && n0 < s.N) {
        const f32x4 hv = {h[0], h[1], h[2], h[3]};
        __builtin_nontemporal_store(hv, (f32x4 *)(state_out + so));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + e < s.N) state_out[so + e] = h[e];
    }
#pragma unroll
    for (int m = 1; m < PER; m <<= 1) v += __shfl_xor(v, m);
    if (sub == 0) {
        v = s.D_skip ? __builtin_fmaf(s.D_skip[d], x, v) : v;
        *yo = Elem<DT>::put(s.z.data ? v * (z * logistic_for<DT>(z)) : v);
    }
}

}  // namespace

template <int DT, int LANES, int ITEMS, bool SHARE = false>
static int scan_fwd(const miconv_scan_t &s, const ScanSplit &split, hipStream_t st) {
    const int rows = (SHARE ? 1 : kScanWaves) * (64 / LANES), blocks_g = (s.D / s.G + rows - 1) / rows;
    return launch_groups((long long)s.B * s.G * blocks_g * split.segs, 64 * kScanWaves, [&](unsigned n, unsigned first) {
        hipLaunchKernelGGL((scan_fwd_kernel<DT, LANES, ITEMS, SHARE>), dim3(n), dim3(64 * kScanWaves), 0, st, s, blocks_g,
                           split, first);
    });
}

namespace {

// Which form of the kernel takes a problem: the one with the least work on the longest CU.
// A work-group's time per chunk, N = 16 bf16, alone on its CU and where two share it, in us:
// 64 lanes x 16 steps 14 and 20.3, 64 x 8 8.4 and 11.7, four rows of 16 x 8 7.2 and 9.9, the same with
// the eight waves sharing four rows' states 2.5 and 3.5 (5 where more than two wait for a CU).
// So many long rows take 64 x 16 (2 x 4096 rows of 2048: 81 against 91 and 117 us), lengths
// just past its chunk 64 x 8 (of 1536: 71 against 81 and 89), a length just past a chunk or
// many short rows 16 x 8 (of 129: 16 against 46 and 29; of 300: 24 against 48 and 31), few rows of
// a few hundred 64 x 8 (1024 rows of 500: 12.6 against 19.7, 30 and 13.5), few short rows the
// shared form (1024 rows of 2: 5.7 against 10, of 256: 7.9 against 11.3; 64 states, of 128: 8.2
// against 25, of 1000: 47 against 52).
double form_cost(const miconv_scan_t &s, int rows, int steps, double alone, double shared) {
    const double groups = (double)s.B * s.G * ((s.D / s.G + rows - 1) / rows), chunks = (s.L + steps - 1) / steps;
    return chunks * (groups <= 256 ? alone : shared * (groups < 512 ? 1.0 : groups / 512));
}

ScanForm cheapest_form(const miconv_scan_t &s) {
    const double per_state = 0.2 + 0.05 * s.N;                       // of the times at N = 16
    const double a = per_state * form_cost(s, kScanWaves, 1024, 14.0, 20.3),
                 b = per_state * form_cost(s, kScanWaves, 512, 8.4, 11.7),
                 c = per_state * form_cost(s, 4 * kScanWaves, 128, 7.2, 9.9);
    const double groups = (double)s.B * s.G * ((s.D / s.G + 3) / 4), chunks = (s.L + 127) / 128;
    const double d = (0.64 + 0.0225 * s.N) * chunks * (groups <= 256 ? 2.5 : groups <= 512 ? 3.5 : groups / 512 * 5.0);
    if (d < a && d < b && d < c) return kShared;
    return a <= b && a <= c ? kLong : (b <= c ? kMiddle : kRows);
}

}  // namespace

// (time segments are whole chunks of 64 x 16)
ScanForm scan_form(const miconv_scan_t &s, const ScanSplit &split) { return split.segs > 1 ? kLong : cheapest_form(s); }

// The time axis is split where the rows alone leave half of the CUs without work and a row
// has at least three chunks of 1024: each segment costs its local state's pass (two thirds of
// the scan) besides, but runs beside the others.
ScanSplit plan_scan_fwd(const miconv_scan_t &s, size_t budget) {
    ScanSplit p = {1, 0, nullptr, nullptr, 0};
    const long long groups = (long long)s.B * s.G * ((s.D / s.G + kScanWaves - 1) / kScanWaves);
    const int chunks = (s.L + 1023) / 1024;
    if (groups > 128 || chunks < 3) return p;
    long long segs = 512 / groups < chunks ? 512 / groups : chunks;
    const int per = (int)((chunks + segs - 1) / segs);
    segs = (chunks + per - 1) / per;
    const size_t rows = (size_t)s.B * s.D, bytes = rows * segs * (s.N + 1) * 4;
    if (bytes > budget) return p;
    p.segs = (int)segs;
    p.steps = per * 1024;
    p.bytes = bytes;
    return p;
}

int launch_scan_fwd(const miconv_scan_t &s, int dtype, ScanSplit split, float *ws, hipStream_t st) {
    if (split.segs > 1) {
        const long long rows = (long long)s.B * s.D;
        split.entry = ws;
        split.sums = ws + rows * split.segs * s.N;
        const int blocks_g = (s.D / s.G + kScanWaves - 1) / kScanWaves;
        const dim3 grid((unsigned)((long long)s.B * s.G * blocks_g * split.segs)), block(64 * kScanWaves);
        if (dtype)
            hipLaunchKernelGGL(scan_local_kernel<1>, grid, block, 0, st, s, blocks_g, split);
        else
            hipLaunchKernelGGL(scan_local_kernel<0>, grid, block, 0, st, s, blocks_g, split);
        hipLaunchKernelGGL(scan_chain_kernel, dim3((unsigned)((rows * s.N + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                           st, s, split);
        if (hipGetLastError() != hipSuccess) return MICONV_ERR_HIP;
    }
    switch (scan_form(s, split)) {
        case kLong: return dtype ? scan_fwd<1, 64, 16>(s, split, st) : scan_fwd<0, 64, 16>(s, split, st);
        case kMiddle: return dtype ? scan_fwd<1, 64, 8>(s, split, st) : scan_fwd<0, 64, 8>(s, split, st);
        case kShared: return dtype ? scan_fwd<1, 16, 8, true>(s, split, st) : scan_fwd<0, 16, 8, true>(s, split, st);
        default: return dtype ? scan_fwd<1, 16, 8>(s, split, st) : scan_fwd<0, 16, 8>(s, split, st);
    }
}

template <int DT, int PER>
static int scan_step(const miconv_scan_t &s, const float *state, int slots, const int *slot_of, float *state_out,
                     hipStream_t st) {
    const long long rows = (long long)s.B * s.D;
    const FDiv fd_D = make_fdiv((uint32_t)s.D), fd_group = make_fdiv((uint32_t)(s.D / s.G));
    const bool together = s.N == 1 || (s.Bm.stride_n == 1 && s.Cm.stride_n == 1);
    const bool vec = s.N % 4 == 0 && together && ((uintptr_t)state | (uintptr_t)state_out) % 16 == 0;
    const auto kern = vec ? scan_step_kernel<DT, PER, true> : scan_step_kernel<DT, PER, false>;
    return launch_groups((rows + kThreads / PER - 1) / (kThreads / PER), kThreads, [&](unsigned n, unsigned first) {
        hipLaunchKernelGGL(kern, dim3(n), dim3(kThreads), 0, st, s, state, slots, slot_of, state_out, fd_D, fd_group, first);
    });
}

int launch_scan_step(const miconv_scan_t &s, int dtype, const float *state, int slots, const int *slot_of,
                     float *state_out, hipStream_t st) {
#define MICONV_STEP(PER)                                                        \
    return dtype ? scan_step<1, PER>(s, state, slots, slot_of, state_out, st)   \
                 : scan_step<0, PER>(s, state, slots, slot_of, state_out, st)
    if (s.N <= 4) MICONV_STEP(1);
    if (s.N <= 8) MICONV_STEP(2);
    if (s.N <= 16) MICONV_STEP(4);
    if (s.N <= 32) MICONV_STEP(8);
    MICONV_STEP(16);
#undef MICONV_STEP
}

}  // namespace miconv
