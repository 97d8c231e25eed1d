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
// maps, over the lanes of a wave as in the forward pass.
//
// A work-group takes R channels of one sequence and group, a wave NS = 4 of the N
// states for all of them, so that the sums over channels of dB and dC are kept in
// its registers; the sums over states (d(dt), g B, v) meet in LDS.  The R-channel
// sums go to the workspace and are added in order by a second kernel.  More than
// 32 states are taken 32 at a time (a wave's sums would not fit its registers);
// the sums over states of the earlier launches wait in the workspace.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int NS = 4, kStates = 32;

// Sum over the wave, in every lane.
DEVI float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

struct BwdOut {
    float *dB, *dC;           // [parts][B][G][N][L]
    float *dA, *dD, *db;      // [B][D][N], [B][D], [B][D]
    float *sums;              // [3][B][D][L] sums over the states of earlier launches, or null
    int R, parts;
    int n_first, n_end, last; // states of this launch; whether it is the last one
};

template <int DT, int TH>
__global__ __launch_bounds__(TH) void scan_bwd_kernel(miconv_scan_t s, BwdOut o) {
    typedef typename Elem<DT>::T T;
    extern __shared__ float lds[];
    const int waves = blockDim.x >> 6, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int per_group = s.D / s.G;
    const int part = blockIdx.x % o.parts, g = (blockIdx.x / o.parts) % s.G, b = blockIdx.x / (o.parts * s.G);
    const int d0 = g * per_group + part * o.R;
    const int R = per_group - part * o.R < o.R ? per_group - part * o.R : o.R;
    const int n0 = o.n_first + wave * NS;
    float *sums = lds;                                    // [waves][3][kScanChunk]
    // [R][N] G of the step after the chunk; only this launch's states are used
    float *carry = lds + waves * 3 * kScanChunk;
    float *dA = carry + o.R * s.N;                        // [R][N]
    float *dD = dA + o.R * s.N, *db = dD + o.R;           // [R]
    const int len = valid_steps(s.lengths, b, s.L);
    const int chunks = (s.L + kScanChunk - 1) / kScanChunk;
    for (int i = threadIdx.x; i < R * s.N; i += blockDim.x) {
        const long long at = ((long long)b * s.D + d0) * s.N + i;
        carry[i] = s.d_final_state ? s.d_final_state[at] : 0.0f;
        dA[i] = 0.0f;
    }
    for (int i = threadIdx.x; i < R; i += blockDim.x) dD[i] = db[i] = 0.0f;
    __syncthreads();
    const T *Bm = (const T *)s.Bm.data + b * s.Bm.stride_b + g * s.Bm.stride_g;
    const T *Cm = (const T *)s.Cm.data + b * s.Cm.stride_b + g * s.Cm.stride_g;
    for (int c = chunks - 1; c >= 0; --c) {
        const int t = c * kScanChunk + lane * 8;
        float dBv[NS][8], dCv[NS][8];
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) dBv[j][i] = dCv[j][i] = 0.0f;
        for (int r = 0; r < R; ++r) {
            const int d = d0 + r;
            const long long row = (long long)b * s.D + d;
            const T *x = (const T *)s.x.data + b * s.x.stride_b + d * s.x.stride_d;
            const T *dl = (const T *)s.delta.data + b * s.delta.stride_b + d * s.delta.stride_d;
            const T *dy = (const T *)s.dy.data + b * s.dy.stride_b + d * s.dy.stride_d;
            const T *z = s.z.data ? (const T *)s.z.data + b * s.z.stride_b + d * s.z.stride_d : nullptr;
            const float bias = s.delta_bias ? s.delta_bias[d] : 0.0f;
            float xv[8], dt[8], e[8], total = 0.0f, ddt[8], gB[8], v[8];
            load8<DT>(x, t, len, xv);
            load8<DT>(dl, t, len, dt);
            load8<DT>(dy, t, len, e);
            if (z) {
                float zv[8];
                load8<DT>(z, t, len, zv);
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] *= zv[i] * logistic(zv[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float raw = dt[i] + bias;
                dt[i] = t + i < len ? (s.softplus ? softplus(raw) : raw) : 0.0f;
                total += dt[i];
                xv[i] *= dt[i];
                ddt[i] = gB[i] = v[i] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const int n = n0 + j;
                if (n >= o.n_end) break;
                const float A = s.A[(long long)d * s.N + n], a2 = A * kLog2e;
                float bv[8], cv[8], a[8], h = 0.0f, G = 0.0f;
                load8<DT>(Bm + n * s.Bm.stride_n, t, len, bv);
                load8<DT>(Cm + n * s.Cm.stride_n, t, len, cv);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] = exp2_hw(dt[i] * a2);
                    h = __builtin_fmaf(a[i], h, xv[i] * bv[i]);
                }
#pragma unroll
                for (int i = 7; i >= 0; --i) G = a[i] * __builtin_fmaf(cv[i], e[i], G);
                float p = exp2_hw(total * a2), q = p;
#pragma unroll
                for (int m = 1; m < 64; m <<= 1) {
                    const float hp = __shfl_up(h, m), pp = __shfl_up(p, m);
                    const float Gq = __shfl_down(G, m), qq = __shfl_down(q, m);
                    if (lane >= m) {
                        h = __builtin_fmaf(p, hp, h);
                        p *= pp;
                    }
                    if (lane + m < 64) {
                        G = __builtin_fmaf(q, Gq, G);
                        q *= qq;
                    }
                }
                const float h0 = s.states[(row * chunks + c) * s.N + n], G0 = carry[r * s.N + n];
                h = __shfl_up(__builtin_fmaf(p, h0, h), 1);
                if (lane == 0) h = h0;
                const float Gend = __builtin_fmaf(q, G0, G);
                G = __shfl_down(Gend, 1);
                if (lane == 63) G = G0;
                if (lane == 0) carry[r * s.N + n] = Gend;
                float hh[8], ah[8], sA = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ah[i] = a[i] * h;
                    h = __builtin_fmaf(xv[i], bv[i], ah[i]);
                    hh[i] = h;
                }
#pragma unroll
                for (int i = 7; i >= 0; --i) {
                    const float gt = __builtin_fmaf(cv[i], e[i], G);
                    G = a[i] * gt;
                    const float w = gt * ah[i];
                    ddt[i] = __builtin_fmaf(A, w, ddt[i]);
                    sA = __builtin_fmaf(dt[i], w, sA);
                    gB[i] = __builtin_fmaf(gt, bv[i], gB[i]);
                    v[i] = __builtin_fmaf(cv[i], hh[i], v[i]);
                    dBv[j][i] = __builtin_fmaf(gt, xv[i], dBv[j][i]);
                    dCv[j][i] = __builtin_fmaf(e[i], hh[i], dCv[j][i]);
                }
                sA = wave_sum(sA);
                if (lane == 0) dA[r * s.N + n] += sA;
                // one state's loads at a time: the unrolled states' together do not fit the registers
                __builtin_amdgcn_sched_barrier(0);
            }
            float *mine = sums + wave * 3 * kScanChunk + lane * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mine[i] = ddt[i];
                mine[kScanChunk + i] = gB[i];
                mine[2 * kScanChunk + i] = v[i];
            }
            __syncthreads();
            const float skip = s.D_skip ? s.D_skip[d] : 0.0f;
            float sD = 0.0f, sb = 0.0f;
            T *dx = (T *)s.dx.data + b * s.dx.stride_b + d * s.dx.stride_d;
            T *dd = (T *)s.ddelta.data + b * s.ddelta.stride_b + d * s.ddelta.stride_d;
            T *dz = s.dz.data ? (T *)s.dz.data + b * s.dz.stride_b + d * s.dz.stride_d : nullptr;
            for (int i = threadIdx.x; i < kScanChunk; i += blockDim.x) {
                const int tt = c * kScanChunk + i;
                if (tt >= s.L) break;
                if (tt >= len) {
                    dx[tt] = dd[tt] = Elem<DT>::put(0.0f);
                    if (dz) dz[tt] = Elem<DT>::put(0.0f);
                    continue;
                }
                float sdt = 0.0f, sgB = 0.0f, sv = 0.0f;
                for (int w = 0; w < waves; ++w) {
                    sdt += sums[w * 3 * kScanChunk + i];
                    sgB += sums[w * 3 * kScanChunk + kScanChunk + i];
                    sv += sums[w * 3 * kScanChunk + 2 * kScanChunk + i];
                }
                if (o.sums) {
                    float *past = o.sums + row * s.L + tt;
                    const long long one = (long long)s.B * s.D * s.L;
                    if (o.n_first) {
                        sdt += past[0];
                        sgB += past[one];
                        sv += past[2 * one];
                    }
                    if (!o.last) {
                        past[0] = sdt;
                        past[one] = sgB;
                        past[2 * one] = sv;
                        continue;
                    }
                }
                const float xt = Elem<DT>::get(x[tt]), dyt = Elem<DT>::get(dy[tt]);
                const float raw = Elem<DT>::get(dl[tt]) + bias;
                float et = dyt;
                if (z) {
                    const float zt = Elem<DT>::get(z[tt]), sg = logistic(zt);
                    et *= zt * sg;
                    if (dz) dz[tt] = Elem<DT>::put(dyt * __builtin_fmaf(skip, xt, sv) * (sg * __builtin_fmaf(zt, 1.0f - sg, 1.0f)));
                }
                dx[tt] = Elem<DT>::put(__builtin_fmaf(s.softplus ? softplus(raw) : raw, sgB, skip * et));
                sdt = __builtin_fmaf(xt, sgB, sdt);
                if (s.softplus) sdt *= logistic(raw);
                dd[tt] = Elem<DT>::put(sdt);
                sD = __builtin_fmaf(et, xt, sD);
                sb += sdt;
            }
            // the waves' parts of dD and dbias, in order
            sD = wave_sum(sD);
            sb = wave_sum(sb);
            __syncthreads();
            if (lane == 0) {
                sums[2 * wave] = sD;
                sums[2 * wave + 1] = sb;
            }
            __syncthreads();
            if (threadIdx.x == 0)
                for (int w = 0; w < waves; ++w) {
                    dD[r] += sums[2 * w];
                    db[r] += sums[2 * w + 1];
                }
            __syncthreads();
        }
        if (t < s.L) {
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const int n = n0 + j;
                if (n >= o.n_end) break;
                const long long at = ((((long long)part * s.B + b) * s.G + g) * s.N + n) * s.L;
                store8<0>(o.dB + at, t, s.L, dBv[j]);
                store8<0>(o.dC + at, t, s.L, dCv[j]);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < R * s.N; i += blockDim.x) {
        const int n = i % s.N;
        if (n < o.n_first || n >= o.n_end) continue;
        const long long at = ((long long)b * s.D + d0) * s.N + i;
        o.dA[at] = dA[i];
        if (s.d_initial_state) s.d_initial_state[at] = carry[i];
    }
    if (!o.last) return;
    for (int i = threadIdx.x; i < R; i += blockDim.x) {
        o.dD[(long long)b * s.D + d0 + i] = dD[i];
        o.db[(long long)b * s.D + d0 + i] = db[i];
    }
}

// out[i] = sum over p of part[p][i], p in order, for up to three arrays.
struct SumJob {
    const float *part;
    float *out;
    long long n;
    int parts;
};
struct SumJobs {
    SumJob j[5];
    int count;
};

__global__ __launch_bounds__(256) void scan_bwd_sum(SumJobs jobs) {
    for (int k = 0; k < jobs.count; ++k) {
        const SumJob j = jobs.j[k];
        for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < j.n; i += (long long)gridDim.x * 256) {
            float a = 0.0f;
            for (int p = 0; p < j.parts; ++p) a += j.part[p * j.n + i];
            j.out[i] = a;
        }
    }
}

}  // namespace

ScanBwdPlan plan_scan_bwd(const miconv_scan_t &s) {
    ScanBwdPlan p;
    const int per_group = s.D / s.G;
    p.R = per_group < 16 ? per_group : 16;
    p.parts = (per_group + p.R - 1) / p.R;
    const size_t bc = (size_t)p.parts * s.B * s.G * s.N * s.L, bd = (size_t)s.B * s.D;
    p.off_dB = 0;
    p.off_dC = bc;
    p.off_dA = 2 * bc;
    p.off_dD = p.off_dA + bd * s.N;
    p.off_db = p.off_dD + bd;
    p.off_sums = p.off_db + bd;
    p.bytes = (p.off_sums + (s.N > kStates ? 3 * bd * s.L : 0)) * 4;
    return p;
}

int launch_scan_bwd(const miconv_scan_t &s, int dtype, float *ws, hipStream_t st) {
    const ScanBwdPlan p = plan_scan_bwd(s);
    BwdOut o;
    o.dB = ws + p.off_dB;
    o.dC = ws + p.off_dC;
    o.dA = ws + p.off_dA;
    o.dD = ws + p.off_dD;
    o.db = ws + p.off_db;
    o.sums = s.N > kStates ? ws + p.off_sums : nullptr;
    o.R = p.R;
    o.parts = p.parts;
    const dim3 grid((unsigned)((long long)s.B * s.G * p.parts));
    for (int n = 0; n < s.N; n += kStates) {
        o.n_first = n;
        o.n_end = s.N < n + kStates ? s.N : n + kStates;
        o.last = o.n_end == s.N;
        const int waves = (o.n_end - n + NS - 1) / NS;
        const size_t lds = ((size_t)waves * 3 * kScanChunk + 2 * (size_t)p.R * s.N + 2 * p.R) * 4;
        const void *kern;
        if (waves <= 4)
            kern = dtype ? (const void *)scan_bwd_kernel<1, 256> : (const void *)scan_bwd_kernel<0, 256>;
        else
            kern = dtype ? (const void *)scan_bwd_kernel<1, 512> : (const void *)scan_bwd_kernel<0, 512>;
        if (lds > 64 * 1024 &&
            hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
            return MICONV_ERR_HIP;
        miconv_scan_t a = s;
        void *args[] = {(void *)&a, (void *)&o};
        if (hipLaunchKernel(kern, grid, dim3(waves * 64), args, lds, st) != hipSuccess) return MICONV_ERR_HIP;
    }
    SumJobs jobs = {};
    const long long bc = (long long)s.B * s.G * s.N * s.L;
    jobs.j[jobs.count++] = {o.dB, s.dB, bc, p.parts};
    jobs.j[jobs.count++] = {o.dC, s.dC, bc, p.parts};
    jobs.j[jobs.count++] = {o.dA, s.dA, (long long)s.D * s.N, s.B};
    if (s.dD) jobs.j[jobs.count++] = {o.dD, s.dD, s.D, s.B};
    if (s.ddelta_bias) jobs.j[jobs.count++] = {o.db, s.ddelta_bias, s.D, s.B};
    long long blocks = (bc + 255) / 256;
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(scan_bwd_sum, dim3((unsigned)blocks), dim3(256), 0, st, jobs);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

}  // namespace miconv
