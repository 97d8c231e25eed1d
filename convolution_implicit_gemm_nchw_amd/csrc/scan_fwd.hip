// scan_fwd.hip -- selective scan, forward, and its one-token step.
//
//   h_t[n] = exp(dt_t A[n]) h_{t-1}[n] + dt_t x_t B_t[n],  v_t = sum_n C_t[n] h_t[n] + D x_t
//
// The map h -> a h + b composes: (a1, b1) then (a2, b2) is (a1 a2, a2 b1 + b2).  A
// wave takes one row (sequence, channel) and 64 lanes x 8 time steps of it at a
// time: each lane runs its eight steps from a zero state, the lanes' maps are
// combined by a prefix scan over the wave, and each lane runs its steps again
// from its true entry state.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int kThreads = 256;

template <int DT>
__global__ __launch_bounds__(kThreads) void scan_fwd_kernel(miconv_scan_t s) {
    typedef typename Elem<DT>::T T;
    __shared__ float carry[kThreads / 64][MICONV_SCAN_MAX_STATES];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const long long row = (long long)blockIdx.x * (kThreads / 64) + wave;
    if (row >= (long long)s.B * s.D) return;
    const int b = (int)(row / s.D), d = (int)(row - (long long)b * s.D), g = d / (s.D / s.G);
    const int len = valid_steps(s.lengths, b, s.L);
    const T *x = (const T *)s.x.data + b * s.x.stride_b + d * s.x.stride_d;
    const T *dl = (const T *)s.delta.data + b * s.delta.stride_b + d * s.delta.stride_d;
    const T *z = s.z.data ? (const T *)s.z.data + b * s.z.stride_b + d * s.z.stride_d : nullptr;
    T *y = (T *)s.y.data + b * s.y.stride_b + d * s.y.stride_d;
    const T *Bm = (const T *)s.Bm.data + b * s.Bm.stride_b + g * s.Bm.stride_g;
    const T *Cm = (const T *)s.Cm.data + b * s.Cm.stride_b + g * s.Cm.stride_g;
    const float *A = s.A + (long long)d * s.N;
    const float skip = s.D_skip ? s.D_skip[d] : 0.0f, bias = s.delta_bias ? s.delta_bias[d] : 0.0f;
    float *carried = carry[wave];
    const int chunks = (s.L + kScanChunk - 1) / kScanChunk;
    if (lane < s.N) carried[lane] = s.initial_state ? s.initial_state[row * s.N + lane] : 0.0f;
    for (int c = 0; c < chunks; ++c) {
        wave_lds_sync();
        if (s.states && lane < s.N) s.states[(row * chunks + c) * s.N + lane] = carried[lane];
        const int t = c * kScanChunk + lane * 8;
        float xv[8], dt[8], v[8], sum = 0.0f;
        load8<DT>(x, t, len, xv);
        load8<DT>(dl, t, len, dt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float raw = dt[i] + bias;
            dt[i] = t + i < len ? (s.softplus ? softplus(raw) : raw) : 0.0f;   // no decay past the end
            sum += dt[i];
            v[i] = skip * xv[i];
            xv[i] *= dt[i];
        }
        for (int n = 0; n < s.N; ++n) {
            const float a2 = A[n] * kLog2e;
            float bv[8], cv[8], a[8], h = 0.0f;
            load8<DT>(Bm + n * s.Bm.stride_n, t, len, bv);
            load8<DT>(Cm + n * s.Cm.stride_n, t, len, cv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] = exp2_hw(dt[i] * a2);
                bv[i] *= xv[i];
                h = __builtin_fmaf(a[i], h, bv[i]);
            }
            float p = exp2_hw(sum * a2);
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const float hp = __shfl_up(h, m), pp = __shfl_up(p, m);
                if (lane >= m) {
                    h = __builtin_fmaf(p, hp, h);
                    p *= pp;
                }
            }
            const float h0 = carried[n];
            const float end = __builtin_fmaf(p, h0, h);
            h = __shfl_up(end, 1);
            if (lane == 0) h = h0;
            if (lane == 63) carried[n] = end;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h = __builtin_fmaf(a[i], h, bv[i]);
                v[i] = __builtin_fmaf(cv[i], h, v[i]);
            }
        }
        if (z) {
            float zv[8];
            load8<DT>(z, t, len, zv);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= zv[i] * logistic(zv[i]);
        }
        if (t < s.L) store8<DT>(y, t, s.L, v);
    }
    wave_lds_sync();
    if (s.final_state && lane < s.N) s.final_state[row * s.N + lane] = carried[lane];
}

// One thread per (sequence, channel); its N states are contiguous.
template <int DT>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(miconv_scan_t s, const float *state, int slots,
                                                             const int *slot_of, float *state_out) {
    typedef typename Elem<DT>::T T;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)s.B * s.D) return;
    const int b = (int)(i / s.D), d = (int)(i - (long long)b * s.D), g = d / (s.D / s.G);
    const int slot = slot_of ? slot_of[b] : b;
    T *yo = (T *)s.y.data + b * s.y.stride_b + d * s.y.stride_d;
    if (slot < 0 || slot >= slots) {
        *yo = Elem<DT>::put(0.0f);
        return;
    }
    const float x = Elem<DT>::get(((const T *)s.x.data)[b * s.x.stride_b + d * s.x.stride_d]);
    const float raw = Elem<DT>::get(((const T *)s.delta.data)[b * s.delta.stride_b + d * s.delta.stride_d]) +
                      (s.delta_bias ? s.delta_bias[d] : 0.0f);
    const float dt = s.softplus ? softplus(raw) : raw, dtx = dt * x;
    const T *Bm = (const T *)s.Bm.data + b * s.Bm.stride_b + g * s.Bm.stride_g;
    const T *Cm = (const T *)s.Cm.data + b * s.Cm.stride_b + g * s.Cm.stride_g;
    const long long so = ((long long)slot * s.D + d) * s.N;
    float v = s.D_skip ? s.D_skip[d] * x : 0.0f;
    for (int n = 0; n < s.N; ++n) {
        const float a = exp2_hw(dt * (s.A[(long long)d * s.N + n] * kLog2e));
        const float h = __builtin_fmaf(a, state[so + n], dtx * Elem<DT>::get(Bm[n * s.Bm.stride_n]));
        state_out[so + n] = h;
        v = __builtin_fmaf(Elem<DT>::get(Cm[n * s.Cm.stride_n]), h, v);
    }
    if (s.z.data) {
        const float z = Elem<DT>::get(((const T *)s.z.data)[b * s.z.stride_b + d * s.z.stride_d]);
        v *= z * logistic(z);
    }
    *yo = Elem<DT>::put(v);
}

}  // namespace

int launch_scan_fwd(const miconv_scan_t &s, int dtype, hipStream_t st) {
    const long long rows = (long long)s.B * s.D, per = kThreads / 64;
    const dim3 grid((unsigned)((rows + per - 1) / per));
    if (dtype)
        hipLaunchKernelGGL(scan_fwd_kernel<1>, grid, dim3(kThreads), 0, st, s);
    else
        hipLaunchKernelGGL(scan_fwd_kernel<0>, grid, dim3(kThreads), 0, st, s);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

int launch_scan_step(const miconv_scan_t &s, int dtype, const float *state, int slots, const int *slot_of,
                     float *state_out, hipStream_t st) {
    const long long rows = (long long)s.B * s.D;
    const dim3 grid((unsigned)((rows + kThreads - 1) / kThreads));
    if (dtype)
        hipLaunchKernelGGL(scan_step_kernel<1>, grid, dim3(kThreads), 0, st, s, state, slots, slot_of, state_out);
    else
        hipLaunchKernelGGL(scan_step_kernel<0>, grid, dim3(kThreads), 0, st, s, state, slots, slot_of, state_out);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

}  // namespace miconv
