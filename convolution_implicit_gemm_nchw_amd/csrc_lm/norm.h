// norm.h -- host entries into layer norm's kernels; arguments are already validated.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>

#include "../../include/miconv.h"
#include "ssm.h"

namespace miconv {

// Whether channels are contiguous in every operand (tokens first), else time steps are.
bool norm_tokens_first(const miconv_layer_norm_t &n, bool backward);
// Work-groups of the backward pass, each with a row of partial sums of dw and db in the workspace.
int norm_parts(const miconv_layer_norm_t &n, int dtype, size_t budget);

// Tokens first: threads of a token, and how often each takes eight channels (0: a loop over them).
struct TokensForm {
    int threads, times;
};
TokensForm tokens_form(int C);
// Channel-major: time lanes of a work-group, eight steps each, its threads, and whether it loops over the channels.
struct RowsForm {
    int lanes, threads;
    bool loop;
};
RowsForm rows_form(const miconv_layer_norm_t &n, int dtype, bool backward);

int launch_norm_fwd(const miconv_layer_norm_t &n, int dtype, hipStream_t st);
int launch_norm_bwd(const miconv_layer_norm_t &n, int dtype, int parts, float *ws, hipStream_t st);

}  // namespace miconv
