// matmul_i8.hip -- y[m][n] = qs[m] ws[n] sum_k q[m][k] wq[n][k] (+ bias[n]).
//
// A wave computes a 16 x 16 tile with 16x16x64 integer MFMAs: a lane holds 16
// consecutive k of one row of each operand.
#include "device.h"
#include "ssm.h"
#include "ssm_device.h"

namespace miconv {

namespace {

constexpr int kThreads = 256;
typedef int i32x4 __attribute__((ext_vector_type(4)));

struct I8Out {
    const float *qs, *ws, *bias;
    void *y;
    int T, O, L, channel_major;
};

template <int OD>
DEVI void put_y(const I8Out &o, int m, int n, int sum) {
    if (m >= o.T || n >= o.O) return;
    float v = (float)sum * o.qs[m] * o.ws[n];
    if (o.bias) v += o.bias[n];
    long long at;
    if (o.channel_major) {
        const int b = m / o.L, l = m - b * o.L;
        at = ((long long)b * o.O + n) * o.L + l;
    } else {
        at = (long long)m * o.O + n;
    }
    ((typename Elem<OD>::T *)o.y)[at] = Elem<OD>::put(v);
}

template <int OD>
__global__ __launch_bounds__(kThreads) void matmul_i8_kernel(const signed char *q, const signed char *wq, int K,
                                                             long long tiles_n, long long tiles, I8Out o) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long tile = (long long)blockIdx.x * (kThreads / 64) + wave;
    if (tile >= tiles) return;
    const int m0 = (int)(tile / tiles_n) * 16, n0 = (int)(tile % tiles_n) * 16;
    const int r = lane & 15, kq = lane >> 4;
    const int ma = m0 + r < o.T ? m0 + r : o.T - 1, nb = n0 + r < o.O ? n0 + r : o.O - 1;
    const i32x4 *a = (const i32x4 *)(q + (long long)ma * K) + kq, *b = (const i32x4 *)(wq + (long long)nb * K) + kq;
    i32x4 acc = {0, 0, 0, 0};
    for (int k = 0; k < K / 16; k += 4) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[k], b[k], acc, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) put_y<OD>(o, m0 + kq * 4 + i, n0 + r, acc[i]);
}

}  // namespace

int i8_splits(int, int, int, size_t) { return 1; }

int launch_matmul_i8(int B, int L, int O, int K, const signed char *q, const float *qs, const signed char *wq,
                     const float *ws, const float *bias, int channel_major, int out_dtype, void *y, int, int *,
                     hipStream_t st) {
    I8Out o = {qs, ws, bias, y, B * L, O, L, channel_major};
    const long long tn = (O + 15) / 16, tiles = tn * ((o.T + 15) / 16);
    const dim3 grid((unsigned)((tiles + 3) / 4));
    if (out_dtype)
        hipLaunchKernelGGL(matmul_i8_kernel<1>, grid, dim3(kThreads), 0, st, q, wq, K, tn, tiles, o);
    else
        hipLaunchKernelGGL(matmul_i8_kernel<0>, grid, dim3(kThreads), 0, st, q, wq, K, tn, tiles, o);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

}  // namespace miconv
