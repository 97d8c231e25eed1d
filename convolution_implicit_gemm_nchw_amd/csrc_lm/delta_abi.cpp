// delta_abi.cpp -- the C entry points of the gated delta rule: validation (before anything is
// enqueued), slices and workspace, launches.
#include <hip/hip_runtime_api.h>
#include <stdio.h>

#include "delta.h"
#include "lm_check.h"

namespace miconv {

DeltaWork delta_work(const miconv_gated_delta_t &d, int dtype, const DeltaSlice &s, bool backward) {
    DeltaWork w = {};
    size_t at = 0;
    const auto take = [&](size_t *place, size_t bytes) {
        *place = at;
        at += (bytes + 255) / 256 * 256;
    };
    const size_t chunks = (size_t)s.nb * s.nc, heads = chunks * d.Hv, DK = delta_key_pad(d.P), Vp = delta_value_pad(d.V);
    const size_t operand = chunks * d.Hk * (dtype == MICONV_BF16 ? 1 : 3) * kDeltaChunk * DK * 2;
    take(&w.k, operand);
    if (!backward) take(&w.q, operand);
    take(&w.inv, heads * 3 * kDeltaSquare);
    take(&w.attn, heads * 3 * kDeltaSquare);
    take(&w.steps, heads * sizeof(DeltaSteps));
    if (backward) {
        take(&w.F, heads * Vp * kDeltaChunk * 4);
        take(&w.after, heads * DK * Vp * 4);
        if (DK == 256 && d.Hv > d.Hk) take(&w.sums, chunks * d.Hk * 2 * kDeltaChunk * DK * 4);
    }
    if (s.nc < delta_chunks(d.L)) take(&w.state, (size_t)s.nb * d.Hv * DK * Vp * 4);
    w.bytes = at;
    return w;
}

// Whole sequences as long as they fit, fewer chunks of time then, fewer sequences where one chunk of all is too
// much.  A pass over a slice of time ends with a state that the next one takes up, so time slices cost launches and
// that state's bytes only.
DeltaSlice delta_slice(const miconv_gated_delta_t &d, int dtype, size_t budget, bool backward) {
    const int chunks = delta_chunks(d.L);
    // a launch of the scans counts its work-groups in 32 bits of work-items
    const long long most = ((1ll << 32) / 512 - 1) / ((long long)d.Hv * (delta_value_pad(d.V) / kDeltaSlice));
    const int nb = d.B < most ? d.B : (int)(most > 1 ? most : 1);
    const auto fits = [&](int b, int c) {
        return delta_work(d, dtype, {0, b, 0, c}, backward).bytes <= budget && (long long)b * c * d.Hv < (1ll << 30);
    };
    const auto largest = [&](int top, auto ok) {              // the largest n in 1..top with ok(n), or 1
        int lo = 1, hi = top;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (ok(mid))
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    };
    if (fits(nb, chunks)) return {0, nb, 0, chunks};
    if (fits(nb, 1)) return {0, nb, 0, largest(chunks, [&](int c) { return fits(nb, c); })};
    return {0, largest(nb, [&](int b) { return fits(b, 1); }), 0, 1};
}

}  // namespace miconv

using namespace miconv;

namespace {

int check_sizes(const miconv_gated_delta_t &d, int dtype) {
    if (bad_size(d.B) || bad_size(d.L) || d.Hk < 1 || d.Hv < 1 || d.P < 1 || d.P > MICONV_DELTA_MAX_KEY || d.V < 1 ||
        d.V > MICONV_DELTA_MAX_VALUE || d.Hv > 65536)
        return MICONV_ERR_BAD_DIM;
    if (d.Hv % d.Hk) return MICONV_ERR_BAD_DIM;
    if ((long long)d.B * d.Hv > kMaxSize) return MICONV_ERR_TOO_LARGE;
    return bad_dtype(dtype) ? MICONV_ERR_DTYPE : MICONV_OK;
}

void inputs(const miconv_gated_delta_t &d, size_t es, Checker *k) {
    k->input(rows_span(d.q, d.B, d.Hk * d.P, d.L, es), true);
    k->input(rows_span(d.k, d.B, d.Hk * d.P, d.L, es), true);
    k->input(rows_span(d.v, d.B, d.Hv * d.V, d.L, es), true);
    k->input(rows_span(d.g, d.B, d.Hv, d.L, 4), true);
    k->input(rows_span(d.beta, d.B, d.Hv, d.L, 4), true);
}

// Counts of values.  Sizes that pass on their own can have products past 64 bits: from kMaxSpan + 1 on a count stands
// for all larger ones, and no tensor is that large.
size_t count(__int128 n) { return (size_t)(n > kMaxSpan ? kMaxSpan + 1 : n); }
size_t state_count(const miconv_gated_delta_t &d, int states) { return count((__int128)states * d.Hv * d.P * d.V); }
size_t saved_count(const miconv_gated_delta_t &d) {
    return count((__int128)d.B * d.Hv * delta_chunks(d.L) * delta_saved(d.P, d.V));
}

size_t capped(size_t bytes) { return bytes < MICONV_MAX_WORKSPACE_BYTES ? bytes : MICONV_MAX_WORKSPACE_BYTES; }

// The kernels of a pass, slice by slice.
int run(const miconv_gated_delta_t &d, int dtype, const DeltaSlice &slice, char *ws, bool backward, hipStream_t st) {
    DeltaArgs a = {};
    a.d = d;
    a.rep = d.Hv / d.Hk;
    a.chunks = delta_chunks(d.L);
    a.Vp = delta_value_pad(d.V);
    a.ws = ws;
    a.w = delta_work(d, dtype, slice, backward);
    const int parts = (a.chunks + slice.nc - 1) / slice.nc;
    for (int b0 = 0; b0 < d.B; b0 += slice.nb)
        for (int i = 0; i < parts; ++i) {
            const int part = backward ? parts - 1 - i : i, c0 = part * slice.nc;
            a.s = {b0, d.B - b0 < slice.nb ? d.B - b0 : slice.nb, c0,
                   a.chunks - c0 < slice.nc ? a.chunks - c0 : slice.nc};
            a.first = part == 0;
            a.last = part == parts - 1;
            int status = launch_delta_prepare(a, dtype, backward, st);
            if (status == MICONV_OK)
                status = backward ? launch_delta_bwd(a, dtype, st) : launch_delta_fwd(a, dtype, st);
            if (status == MICONV_OK && backward) status = launch_delta_grads(a, dtype, st);
            if (status != MICONV_OK) return status;
        }
    return MICONV_OK;
}

}  // namespace

extern "C" {

int gated_delta_states_size(int B, int Hv, int P, int V, int L, size_t *bytes_out) {
    if (!bytes_out) return MICONV_ERR_NULL;
    miconv_gated_delta_t d = {};
    d.B = B, d.Hk = 1, d.Hv = Hv, d.P = P, d.V = V, d.L = L;
    const int bad = check_sizes(d, MICONV_F32);
    if (bad != MICONV_OK) return bad;
    const size_t n = saved_count(d);
    if (n > kMaxSpan) return MICONV_ERR_TOO_LARGE;
    *bytes_out = n * 4;
    return MICONV_OK;
}

int gated_delta_workspace_size(const miconv_gated_delta_t *d, int dtype, int backward, size_t workspace_limit,
                               size_t *bytes_out) {
    if (!d || !bytes_out) return MICONV_ERR_NULL;
    const int bad = check_sizes(*d, dtype);
    if (bad != MICONV_OK) return bad;
    *bytes_out = delta_work(*d, dtype, delta_slice(*d, dtype, capped(workspace_limit), backward != 0), backward != 0).bytes;
    return MICONV_OK;
}

int gated_delta_describe(const miconv_gated_delta_t *d, int dtype, int backward, size_t workspace_bytes, char *buf,
                         size_t buflen) {
    if (!buf || buflen == 0) return MICONV_ERR_NULL;
    buf[0] = 0;
    if (!d) return MICONV_ERR_NULL;
    const int bad = check_sizes(*d, dtype);
    if (bad != MICONV_OK) return bad;
    const DeltaSlice s = delta_slice(*d, dtype, capped(workspace_bytes), backward != 0);
    const size_t need = delta_work(*d, dtype, s, backward != 0).bytes;
    if (need > capped(workspace_bytes)) return MICONV_ERR_WORKSPACE;
    snprintf(buf, buflen, "algo=gated_delta_%s slice=%dx%d ws=%zu", backward ? "bwd" : "fwd", s.nb, s.nc, need);
    return MICONV_OK;
}

int gated_delta_fwd(const miconv_gated_delta_t *d, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!d) return MICONV_ERR_NULL;
    const int bad_sizes = check_sizes(*d, dtype);
    if (bad_sizes != MICONV_OK) return bad_sizes;
    if (!workspace) return MICONV_ERR_NULL;
    const DeltaSlice s = delta_slice(*d, dtype, capped(workspace_bytes), false);
    const size_t es = elem_size(dtype), need = delta_work(*d, dtype, s, false).bytes;
    if (need > capped(workspace_bytes)) return MICONV_ERR_WORKSPACE;
    Checker k;
    inputs(*d, es, &k);
    k.input(flat(d->initial_state, state_count(*d, d->B), 4), false);
    k.input(flat(d->lengths, d->B, 4), false);
    k.output(rows_span(d->y, d->B, d->Hv * d->V, d->L, es), true);
    k.output(flat(d->final_state, state_count(*d, d->B), 4), false);
    k.output(flat(d->states, saved_count(*d), 4), false);
    k.output(flat(workspace, need / 4, 4), true);
    if ((uintptr_t)workspace % 16 || (uintptr_t)d->states % 16) k.fail(MICONV_ERR_ALIGN);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : run(*d, dtype, s, (char *)workspace, false, (hipStream_t)stream);
}

int gated_delta_bwd(const miconv_gated_delta_t *d, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!d) return MICONV_ERR_NULL;
    const int bad_sizes = check_sizes(*d, dtype);
    if (bad_sizes != MICONV_OK) return bad_sizes;
    if (!workspace) return MICONV_ERR_NULL;
    const DeltaSlice s = delta_slice(*d, dtype, capped(workspace_bytes), true);
    const size_t es = elem_size(dtype), need = delta_work(*d, dtype, s, true).bytes, steps = (size_t)d->B * d->Hv * d->L;
    if (need > capped(workspace_bytes)) return MICONV_ERR_WORKSPACE;
    Checker k;
    inputs(*d, es, &k);
    k.input(flat(d->lengths, d->B, 4), false);
    k.input(flat(d->states, saved_count(*d), 4), true);
    k.input(rows_span(d->dy, d->B, d->Hv * d->V, d->L, es), true);
    k.input(flat(d->d_final_state, state_count(*d, d->B), 4), false);
    k.output(rows_span(d->dq, d->B, d->Hk * d->P, d->L, es), true);
    k.output(rows_span(d->dk, d->B, d->Hk * d->P, d->L, es), true);
    k.output(rows_span(d->dv, d->B, d->Hv * d->V, d->L, es), true);
    k.output(flat(d->dg, steps, 4), true);
    k.output(flat(d->dbeta, steps, 4), true);
    k.output(flat(d->d_initial_state, state_count(*d, d->B), 4), false);
    k.output(flat(workspace, need / 4, 4), true);
    if ((uintptr_t)workspace % 16 || (uintptr_t)d->states % 16) k.fail(MICONV_ERR_ALIGN);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : run(*d, dtype, s, (char *)workspace, true, (hipStream_t)stream);
}

int gated_delta_step(const miconv_gated_delta_t *d, int dtype, const float *state, int slots, const int *slot_of,
                     float *state_out, void *stream) {
    if (!d) return MICONV_ERR_NULL;
    const int bad_sizes = check_sizes(*d, dtype);
    if (bad_sizes != MICONV_OK) return bad_sizes;
    if (d->L != 1 || bad_size(slots) || (!slot_of && slots != d->B)) return MICONV_ERR_BAD_DIM;
    // the kernel numbers its work-groups in 31 bits
    if ((long long)d->B * d->Hv * ((d->V + kDeltaStepValues - 1) / kDeltaStepValues) > 0x7fffffff) return MICONV_ERR_TOO_LARGE;
    const size_t es = elem_size(dtype), ns = state_count(*d, slots);
    Checker k;
    inputs(*d, es, &k);
    k.input(flat(slot_of, d->B, 4), false);
    k.output(rows_span(d->y, d->B, d->Hv * d->V, 1, es), true);
    k.output(flat(state_out, ns, 4), true);
    if (state != state_out) k.input(flat(state, ns, 4), true);
    const int bad = k.done();
    return bad != MICONV_OK ? bad
                            : launch_delta_step(*d, dtype, state, slots, slot_of, state_out, (hipStream_t)stream);
}

}  // extern "C"
