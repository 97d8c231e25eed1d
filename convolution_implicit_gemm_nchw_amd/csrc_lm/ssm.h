// ssm.h -- host entries into the kernels of the state-space operators.  The
// arguments are already validated; structures go to the kernels by value.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>

#include "../../include/miconv.h"

namespace miconv {

// Time steps between two saved scan states.
constexpr int kScanChunk = 128;
// Channels that one work-group of the scan's backward pass sums dB and dC over.
constexpr int kScanBwdChannels = 16;

constexpr int scan_chunks(int L) { return (L + kScanChunk - 1) / kScanChunk; }

// A launch counts its work-items along an axis modulo 2^32, without an error: more work-groups than
// that go in several launches.  launch(n, first) launches n of them from the first on.
template <typename F>
int launch_groups(long long groups, int threads, F launch) {
    const long long most = 0xffffffffll / threads;
    for (long long first = 0; first < groups; first += most) {
        const long long n = groups - first < most ? groups - first : most;
        launch((unsigned)n, (unsigned)first);
        if (hipGetLastError() != hipSuccess) return MICONV_ERR_HIP;
    }
    return MICONV_OK;
}

// Whether an output is written past the caches: in bf16 from half of the 256 MB last-level cache
// on, where the next reader would not find it there.  (Causal forward followed by a read of
// its output: 128 MB 121 -> 106 us; 64 MB 50 -> 55 us, though the call alone falls from 31 to 25.)
// Not in fp32, where a lane's eight values are two stores that the caches have to join
// (8192 x 8192 from 8-bit products 128 deep: 74 -> 101 us).
constexpr bool streams(int dtype, size_t count) { return dtype == MICONV_BF16 && count * 2 >= (128u << 20); }

// Time segments of the scan's forward pass that run side by side (1: none), their length,
// and in the workspace the state before each segment [B][D][segs][N] and its sum of dt.
struct ScanSplit {
    int segs, steps;
    float *entry, *sums;
    size_t bytes;
};
ScanSplit plan_scan_fwd(const miconv_scan_t &s, size_t budget);
// The forms of the scan's forward kernel: lanes x steps per row; shared: a row's states over the waves.
enum ScanForm { kLong, kMiddle, kRows, kShared };
ScanForm scan_form(const miconv_scan_t &s, const ScanSplit &split);

// Workspace of the scan's backward pass: partial sums per group of channels, time segments
// that run side by side, and offsets.
struct ScanBwdPlan {
    int parts, segs, seg_chunks;
    int beside;                         // blocks of 16 states in one launch (1: one after the other)
    int carry_segs, carry_steps;        // time segments of the pass that finds G between them
    size_t off_G, off_ends, off_after, off_dB, off_dC, off_dA, off_dD, off_db, off_sums, bytes;   // floats, except bytes
};
// The fastest plan within the budget, or the smallest one where none is.
ScanBwdPlan plan_scan_bwd(const miconv_scan_t &s, size_t budget);

// The backward pass goes through its problem slice by slice where the workspace asks for it: sequences,
// groups of one sequence, channels of one group (a multiple of kScanBwdChannels), and of each the time
// steps (a multiple of kScanChunk) from the last on.
struct ScanBwdSlice {
    int sequences, groups, channels, steps;
    size_t carry, bytes;                // floats that pass from one time slice to the next; workspace of the largest
};
// The largest slice within the budget, or the smallest there is.
ScanBwdSlice slice_scan_bwd(const miconv_scan_t &s, size_t budget);

// Work-groups per channel of the convolution's backward pass.
int causal_bwd_splits(const miconv_causal_conv_t &c, size_t budget);

int launch_causal_fwd(const miconv_causal_conv_t &c, int dtype, hipStream_t st);
int launch_causal_bwd(const miconv_causal_conv_t &c, int dtype, int splits, float *ws, hipStream_t st);
int launch_causal_step(int B, int D, int K, int silu, int dtype, miconv_rows_t x, const void *state, int slots,
                       const int *slot_of, const void *w, const float *bias, void *state_out, miconv_rows_t y,
                       hipStream_t st);

int launch_scan_fwd(const miconv_scan_t &s, int dtype, ScanSplit split, float *ws, hipStream_t st);
int launch_scan_bwd(const miconv_scan_t &s, int dtype, const ScanBwdSlice &slice, float *ws, hipStream_t st);
int launch_scan_step(const miconv_scan_t &s, int dtype, const float *state, int slots, const int *slot_of,
                     float *state_out, hipStream_t st);

int launch_quantize(int B, int L, int C, int dtype, const void *x, long long sb, long long sl, long long sc,
                    signed char *q, float *scale, hipStream_t st);
// Splits of the summed axis matmul_i8 takes under `budget` bytes of workspace.
int i8_splits(int T, int O, int K, size_t budget);
// The kernel it takes: blocks of 16 tokens for few (0: tiles), else the tile's side and LDS stages.
struct I8Form {
    int few, side, stages;
};
I8Form i8_form(int T, int O, int K, int splits);
int launch_matmul_i8(int B, int L, int O, int K, const signed char *q, const float *qs, const signed char *wq,
                     const float *ws_, const float *bias, int channel_major, int out_dtype, void *y, int splits,
                     int *part, hipStream_t st);

}  // namespace miconv
