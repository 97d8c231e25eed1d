// norm_abi.cpp -- the C entry points of layer norm: validation (before anything is enqueued),
// workspace, launches.
#include <float.h>
#include <hip/hip_runtime_api.h>
#include <stdio.h>

#include "lm_check.h"
#include "norm.h"

using namespace miconv;

namespace {

int check_sizes(const miconv_layer_norm_t &n, int dtype) {
    if (bad_size(n.B) || bad_size(n.L) || n.C < 1 || n.C > MICONV_NORM_MAX_CHANNELS) return MICONV_ERR_BAD_DIM;
    if ((long long)n.B * n.L > kMaxSize) return MICONV_ERR_TOO_LARGE;
    return bad_dtype(dtype) ? MICONV_ERR_DTYPE : MICONV_OK;
}

// An operand as rows of its contiguous axis.
Span span(const miconv_layer_norm_t &n, const miconv_tokens_t &v, bool tokens_first, size_t es) {
    if (tokens_first) return {(uintptr_t)v.data, n.B, v.stride_b, n.L, v.stride_l, n.C, es};
    return {(uintptr_t)v.data, n.B, v.stride_b, n.C, v.stride_c, n.L, es};
}

bool rows_of_steps(const miconv_layer_norm_t &n, const miconv_tokens_t &v) { return v.stride_l == 1 || n.L == 1; }

size_t parts_bytes(const miconv_layer_norm_t &n, int parts) { return (size_t)parts * n.C * 8; }

}  // namespace

extern "C" {

int layer_norm_fwd(const miconv_layer_norm_t *n, int dtype, void *stream) {
    if (!n) return MICONV_ERR_NULL;
    const int bad_sizes = check_sizes(*n, dtype);
    if (bad_sizes != MICONV_OK) return bad_sizes;
    if (!(n->eps >= 0.0f && n->eps <= FLT_MAX)) return MICONV_ERR_BAD_DIM;
    const bool first = norm_tokens_first(*n, false);
    if (!first && !(rows_of_steps(*n, n->x) && rows_of_steps(*n, n->y))) return MICONV_ERR_BAD_DIM;
    const size_t es = elem_size(dtype);
    Checker k;
    k.input(span(*n, n->x, first, es), true);
    k.input(flat(n->weight, n->C, 4), false);
    k.input(flat(n->bias, n->C, 4), false);
    k.input(flat(n->lengths, n->B, 4), false);
    k.output(span(*n, n->y, first, es), true);
    k.output(flat(n->stats, (size_t)n->B * n->L * 2, 4), false);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : launch_norm_fwd(*n, dtype, (hipStream_t)stream);
}

int layer_norm_bwd_workspace_size(const miconv_layer_norm_t *n, int dtype, size_t workspace_limit, size_t *bytes_out) {
    if (!n || !bytes_out) return MICONV_ERR_NULL;
    const int bad_sizes = check_sizes(*n, dtype);
    if (bad_sizes != MICONV_OK) return bad_sizes;
    const size_t cap = MICONV_MAX_WORKSPACE_BYTES;
    *bytes_out = parts_bytes(*n, norm_parts(*n, dtype, workspace_limit < cap ? workspace_limit : cap));
    return MICONV_OK;
}

int layer_norm_describe(const miconv_layer_norm_t *n, int dtype, int backward, size_t workspace_bytes, char *buf,
                        size_t buflen) {
    if (!buf || buflen == 0) return MICONV_ERR_NULL;
    buf[0] = 0;
    if (!n) return MICONV_ERR_NULL;
    const int bad = check_sizes(*n, dtype);
    if (bad != MICONV_OK) return bad;
    char parts[32] = "";
    if (backward) {
        const size_t cap = MICONV_MAX_WORKSPACE_BYTES;
        const int p = norm_parts(*n, dtype, workspace_bytes < cap ? workspace_bytes : cap);
        if (parts_bytes(*n, p) > workspace_bytes) return MICONV_ERR_WORKSPACE;
        snprintf(parts, sizeof parts, " parts=%d", p);
    }
    if (norm_tokens_first(*n, backward != 0)) {
        const TokensForm f = tokens_form(n->C);
        snprintf(buf, buflen, "algo=norm_tokens threads=%d times=%d%s", f.threads, f.times, parts);
    } else {
        const RowsForm f = rows_form(*n, dtype, backward != 0);
        snprintf(buf, buflen, "algo=%s lanes=%d threads=%d%s", f.loop ? "norm_rows_loop" : "norm_rows", f.lanes, f.threads,
                 parts);
    }
    return MICONV_OK;
}

int layer_norm_bwd(const miconv_layer_norm_t *n, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!n) return MICONV_ERR_NULL;
    const int bad_sizes = check_sizes(*n, dtype);
    if (bad_sizes != MICONV_OK) return bad_sizes;
    if (!workspace) return MICONV_ERR_NULL;
    const bool first = norm_tokens_first(*n, true);
    if (!first && !(rows_of_steps(*n, n->x) && rows_of_steps(*n, n->dy) && rows_of_steps(*n, n->dx)))
        return MICONV_ERR_BAD_DIM;
    const size_t es = elem_size(dtype), cap = MICONV_MAX_WORKSPACE_BYTES;
    const int parts = norm_parts(*n, dtype, workspace_bytes < cap ? workspace_bytes : cap);
    if (parts_bytes(*n, parts) > workspace_bytes) return MICONV_ERR_WORKSPACE;
    Checker k;
    k.input(span(*n, n->x, first, es), true);
    k.input(span(*n, n->dy, first, es), true);
    k.input(flat(n->weight, n->C, 4), false);
    k.input(flat(n->lengths, n->B, 4), false);
    k.input(flat(n->stats, (size_t)n->B * n->L * 2, 4), true);
    k.output(span(*n, n->dx, first, es), true);
    k.output(flat(n->dw, n->C, 4), false);
    k.output(flat(n->db, n->C, 4), false);
    k.output(flat(workspace, parts_bytes(*n, parts) / 4, 4), true);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : launch_norm_bwd(*n, dtype, parts, (float *)workspace, (hipStream_t)stream);
}

}  // extern "C"
