// f8.h -- host entries into the 8-bit floating-point products; arguments are already validated.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>

#include "../../include/miconv.h"
#include "ssm.h"

namespace miconv {

int launch_quantize_f8(int B, int L, int C, int dtype, const void *x, long long sb, long long sl, long long sc,
                       unsigned char *q, unsigned char *scale, hipStream_t st);
// Splits of the summed axis matmul_f8 takes under `budget` bytes of workspace.
int f8_splits(int T, int O, int K, size_t budget);
// The kernel it takes: blocks of 16 tokens for few (0: tiles), else the tile's side and LDS stages.
struct F8Form {
    int few, side, stages;
};
F8Form f8_form(int T, int O);
int launch_matmul_f8(int B, int L, int O, int K, const unsigned char *q, const unsigned char *qs, const unsigned char *wq,
                     const unsigned char *ws, const float *bias, int channel_major, int out_dtype, void *y, int splits,
                     float *part, hipStream_t st);

}  // namespace miconv
