// f8_abi.cpp -- the C entry points of the 8-bit floating-point products: validation (before anything is
// enqueued), workspace, launches.
#include <hip/hip_runtime_api.h>
#include <stdio.h>

#include "f8.h"
#include "lm_check.h"

using namespace miconv;

namespace {

constexpr int kMaxDepth = 131072;

int check_product(int B, int L, int O, int C_pad) {
    if (bad_size(B) || bad_size(L) || bad_size(O) || C_pad < MICONV_I8_PAD || C_pad > kMaxDepth || C_pad % MICONV_I8_PAD)
        return MICONV_ERR_BAD_DIM;
    if ((long long)B * L > kMaxSize) return MICONV_ERR_TOO_LARGE;
    // 16 x 16 tiles are counted in a 32-bit grid
    if ((((long long)B * L + 15) / 16) * (((long long)O + 15) / 16) > kMaxSize) return MICONV_ERR_TOO_LARGE;
    return MICONV_OK;
}

}  // namespace

extern "C" {

int quantize_f8(int B, int L, int C, int dtype, const void *x, long long stride_b, long long stride_l,
                long long stride_c, unsigned char *q, unsigned char *scale, void *stream) {
    if (bad_size(B) || bad_size(L) || C < 1 || C > kMaxDepth) return MICONV_ERR_BAD_DIM;
    if ((long long)B * L > kMaxSize) return MICONV_ERR_TOO_LARGE;
    if (bad_dtype(dtype)) return MICONV_ERR_DTYPE;
    if (stride_c != 1 && C > 1 && stride_l != 1 && L > 1) return MICONV_ERR_BAD_DIM;
    if (stride_b < 0 || stride_l < 0 || stride_c < 0) return MICONV_ERR_BAD_DIM;
    const size_t es = elem_size(dtype), blocks = ((size_t)C + MICONV_I8_PAD - 1) / MICONV_I8_PAD, tokens = (size_t)B * L;
    if (tokens * blocks > 0x7fffffff) return MICONV_ERR_TOO_LARGE;      // the kernels number them in 31 bits
    const __int128 one = (__int128)(L - 1) * stride_l + (__int128)(C - 1) * stride_c + 1;
    if (one > kMaxSpan) return MICONV_ERR_TOO_LARGE;
    Checker k;
    k.input({(uintptr_t)x, B, stride_b, 1, 0, (long long)one, es}, true);
    k.output(flat(q, tokens * blocks * MICONV_I8_PAD, 1), true);
    k.output(flat(scale, tokens * blocks, 1), true);
    if ((uintptr_t)q % 16) k.fail(MICONV_ERR_ALIGN);
    const int bad = k.done();
    if (bad != MICONV_OK) return bad;
    return launch_quantize_f8(B, L, C, dtype, x, stride_b, stride_l, stride_c, q, scale, (hipStream_t)stream);
}

int matmul_f8_workspace_size(int B, int L, int O, int C_pad, size_t workspace_limit, size_t *bytes_out) {
    if (!bytes_out) return MICONV_ERR_NULL;
    const int st = check_product(B, L, O, C_pad);
    if (st != MICONV_OK) return st;
    const size_t cap = MICONV_MAX_WORKSPACE_BYTES;
    const int s = f8_splits(B * L, O, C_pad, workspace_limit < cap ? workspace_limit : cap);
    *bytes_out = s > 1 ? (size_t)s * B * L * O * 4 : 0;
    return MICONV_OK;
}

int matmul_f8_describe(int B, int L, int O, int C_pad, size_t workspace_bytes, char *buf, size_t buflen) {
    if (!buf || buflen == 0) return MICONV_ERR_NULL;
    buf[0] = 0;
    const int st = check_product(B, L, O, C_pad);
    if (st != MICONV_OK) return st;
    const size_t cap = MICONV_MAX_WORKSPACE_BYTES;
    const int splits = f8_splits(B * L, O, C_pad, workspace_bytes < cap ? workspace_bytes : cap);
    const F8Form f = f8_form(B * L, O);
    if (f.few)
        snprintf(buf, buflen, "algo=f8_few tokens=%d", f.few * 16);
    else
        snprintf(buf, buflen, "algo=f8_tile tile=%d stages=%d splits=%d", f.side, f.stages, splits);
    return MICONV_OK;
}

int matmul_f8(int B, int L, int O, int C_pad, const unsigned char *q, const unsigned char *qscale,
              const unsigned char *wq, const unsigned char *wscale, const float *bias, int channel_major, int out_dtype,
              void *y, void *workspace, size_t workspace_bytes, void *stream) {
    const int st = check_product(B, L, O, C_pad);
    if (st != MICONV_OK) return st;
    if (bad_dtype(out_dtype)) return MICONV_ERR_DTYPE;
    if (!workspace && workspace_bytes) return MICONV_ERR_NULL;
    const size_t T = (size_t)B * L, es = elem_size(out_dtype), blocks = C_pad / MICONV_I8_PAD, cap = MICONV_MAX_WORKSPACE_BYTES;
    Checker k;
    k.input(flat(q, T * C_pad, 1), true);
    k.input(flat(qscale, T * blocks, 1), true);
    k.input(flat(wq, (size_t)O * C_pad, 1), true);
    k.input(flat(wscale, (size_t)O * blocks, 1), true);
    k.input(flat(bias, O, 4), false);
    k.output(flat(y, T * O, es), true);
    if ((uintptr_t)q % 16 || (uintptr_t)wq % 16) k.fail(MICONV_ERR_ALIGN);
    const int splits = f8_splits((int)T, O, C_pad, !workspace ? 0 : (workspace_bytes < cap ? workspace_bytes : cap));
    if (splits > 1) k.output(flat(workspace, (size_t)splits * T * O, 4), true);
    const int bad = k.done();
    if (bad != MICONV_OK) return bad;
    return launch_matmul_f8(B, L, O, C_pad, q, qscale, wq, wscale, bias, channel_major != 0, out_dtype, y, splits,
                            (float *)workspace, (hipStream_t)stream);
}

}  // extern "C"
