// ssm_abi.cpp -- the C entry points of the state-space operators: argument
// validation (before anything is enqueued), workspace sizing, launch.
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/miconv.h"
#include "ssm.h"

using namespace miconv;

namespace {

constexpr long long kMaxSize = 1ll << 30;
// No tensor spans this many elements: products of sizes and strides cannot overflow.
constexpr __int128 kMaxSpan = (__int128)1 << 46;

bool bad_size(long long v) { return v < 1 || v > kMaxSize; }

// A strided tensor's place in memory: nb x nd rows of L elements.
struct Span {
    uintptr_t at;
    long long nb, sb, nd, sd, L;
    size_t es;
    size_t bytes() const { return (size_t)((nb - 1) * sb + (nd - 1) * sd + L) * es; }
};

Span flat(const void *p, size_t n, size_t es) { return {(uintptr_t)p, 1, 0, 1, 0, (long long)n, es}; }

int check_span(const Span &s) {
    if (s.sb < 0 || s.sd < 0) return MICONV_ERR_BAD_DIM;
    const __int128 n = (__int128)(s.nb - 1) * s.sb + (__int128)(s.nd - 1) * s.sd + s.L;
    if (n > kMaxSpan) return MICONV_ERR_TOO_LARGE;
    return s.at % s.es ? MICONV_ERR_ALIGN : MICONV_OK;
}

// Rows of an output must not overlap each other (either axis may be the outer one).
int check_out_rows(const Span &s) {
    const __int128 in_b = (__int128)(s.nd - 1) * s.sd + s.L, in_d = (__int128)(s.nb - 1) * s.sb + s.L;
    const bool b_outer = (s.nd == 1 || s.sd >= s.L) && (s.nb == 1 || s.sb >= in_b);
    const bool d_outer = (s.nb == 1 || s.sb >= s.L) && (s.nd == 1 || s.sd >= in_d);
    return b_outer || d_outer ? MICONV_OK : MICONV_ERR_BAD_DIM;
}

// The bytes that a tensor's rows cover modulo `period`, from its first on: an axis whose stride
// is a multiple of it adds none.
long long window(const Span &s, long long period) {
    const long long es = (long long)s.es, b = (s.nb - 1) * s.sb * es, d = (s.nd - 1) * s.sd * es;
    return s.L * es + (s.sb * es % period ? b : 0) + (s.sd * es % period ? d : 0);
}

// Whether two tensors share memory.  Ranges that interleave are told apart where one of their strides
// repeats both, each in a part of its own: halves of one projection, or slices along time of one buffer.
bool share(const Span &a, const Span &b) {
    if (!a.at || !b.at) return false;
    const size_t an = a.bytes(), bn = b.bytes();
    if (a.at + an <= b.at || b.at + bn <= a.at) return false;
    const long long es_a = (long long)a.es, es_b = (long long)b.es;
    for (const long long period : {a.sb * es_a, a.sd * es_a, b.sb * es_b, b.sd * es_b}) {
        if (period <= 0) continue;
        long long off = (long long)(b.at - a.at) % period;
        if (off < 0) off += period;
        if (off >= window(a, period) && off + window(b, period) <= period) return false;
    }
    return true;
}

Span rows_span(const miconv_rows_t &r, int B, int D, int L, size_t es) {
    return {(uintptr_t)r.data, B, r.stride_b, D, r.stride_d, L, es};
}

struct Checker {
    Span in[24], out[16];
    int ni = 0, no = 0, status = MICONV_OK;
    void fail(int s) {
        if (status == MICONV_OK) status = s;
    }
    void input(const Span &s, bool required) {
        if (!s.at) {
            if (required) fail(MICONV_ERR_NULL);
            return;
        }
        fail(check_span(s));
        in[ni++] = s;
    }
    void output(const Span &s, bool required) {
        if (!s.at) {
            if (required) fail(MICONV_ERR_NULL);
            return;
        }
        fail(check_span(s));
        if (status == MICONV_OK) fail(check_out_rows(s));
        out[no++] = s;
    }
    int done() {
        if (status != MICONV_OK) return status;
        for (int i = 0; i < no; ++i) {
            for (int j = 0; j < ni; ++j)
                if (share(out[i], in[j])) return MICONV_ERR_ALIAS;
            for (int j = 0; j < i; ++j)
                if (share(out[i], out[j])) return MICONV_ERR_ALIAS;
        }
        return MICONV_OK;
    }
};

bool bad_dtype(int d) { return d != MICONV_F32 && d != MICONV_BF16; }
size_t elem_size(int d) { return d == MICONV_BF16 ? 2 : 4; }

int check_conv_sizes(int B, int D, int L, int K, int dtype) {
    if (bad_size(B) || bad_size(D) || bad_size(L) || K < 1 || K > MICONV_CAUSAL_MAX_TAPS) return MICONV_ERR_BAD_DIM;
    if ((long long)B * D > kMaxSize) return MICONV_ERR_TOO_LARGE;
    return bad_dtype(dtype) ? MICONV_ERR_DTYPE : MICONV_OK;
}

void conv_inputs(const miconv_causal_conv_t &c, size_t es, Checker *k) {
    const size_t rows = (size_t)c.B * c.D;
    k->input(rows_span(c.x, c.B, c.D, c.L, es), true);
    k->input(flat(c.w, (size_t)c.D * c.K, es), true);
    k->input(flat(c.bias, c.D, 4), false);
    // one tap has no state: pointers are ignored
    if (c.K > 1) k->input(flat(c.initial_state, rows * (c.K - 1), es), false);
    k->input(flat(c.lengths, c.B, 4), false);
}

int check_scan_sizes(const miconv_scan_t &s, int dtype) {
    if (bad_size(s.B) || bad_size(s.D) || bad_size(s.L) || bad_size(s.G) || s.N < 1 || s.N > MICONV_SCAN_MAX_STATES)
        return MICONV_ERR_BAD_DIM;
    if (s.D % s.G) return MICONV_ERR_BAD_DIM;
    if ((long long)s.B * s.D > kMaxSize || (long long)s.B * s.G * s.N > kMaxSize) return MICONV_ERR_TOO_LARGE;
    return bad_dtype(dtype) ? MICONV_ERR_DTYPE : MICONV_OK;
}

// Bm or Cm as (B) x (G*N as one axis when its strides allow) rows: for the overlap
// test the whole extent is enough.
void scan_bc(const miconv_scan_t &s, const miconv_scan_in_t &v, size_t es, Checker *k) {
    if (!v.data) return k->fail(MICONV_ERR_NULL);
    if (v.stride_b < 0 || v.stride_g < 0 || v.stride_n < 0) return k->fail(MICONV_ERR_BAD_DIM);
    const __int128 one = (__int128)(s.G - 1) * v.stride_g + (__int128)(s.N - 1) * v.stride_n + s.L;
    if (one > kMaxSpan) return k->fail(MICONV_ERR_TOO_LARGE);
    k->input({(uintptr_t)v.data, s.B, v.stride_b, 1, 0, (long long)one, es}, true);
}

void scan_inputs(const miconv_scan_t &s, size_t es, Checker *k) {
    k->input(rows_span(s.x, s.B, s.D, s.L, es), true);
    k->input(rows_span(s.delta, s.B, s.D, s.L, es), true);
    k->input(rows_span(s.z, s.B, s.D, s.L, es), false);
    k->input(flat(s.A, (size_t)s.D * s.N, 4), true);
    scan_bc(s, s.Bm, es, k);
    scan_bc(s, s.Cm, es, k);
    k->input(flat(s.D_skip, s.D, 4), false);
    k->input(flat(s.delta_bias, s.D, 4), false);
}

size_t state_count(const miconv_scan_t &s) { return (size_t)s.B * s.D * s.N; }

}  // namespace

extern "C" {

int causal_conv1d_fwd(const miconv_causal_conv_t *c, int dtype, void *stream) {
    if (!c) return MICONV_ERR_NULL;
    const int st = check_conv_sizes(c->B, c->D, c->L, c->K, dtype);
    if (st != MICONV_OK) return st;
    const size_t es = elem_size(dtype), ns = (size_t)c->B * c->D * (c->K - 1);
    Checker k;
    conv_inputs(*c, es, &k);
    k.output(rows_span(c->y, c->B, c->D, c->L, es), true);
    if (c->K > 1) k.output(flat(c->final_state, ns, es), false);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : launch_causal_fwd(*c, dtype, (hipStream_t)stream);
}

int causal_conv1d_bwd_workspace_size(const miconv_causal_conv_t *c, int dtype, size_t workspace_limit,
                                     size_t *bytes_out) {
    if (!c || !bytes_out) return MICONV_ERR_NULL;
    const int st = check_conv_sizes(c->B, c->D, c->L, c->K, dtype);
    if (st != MICONV_OK) return st;
    const int s = causal_bwd_splits(*c, workspace_limit);
    *bytes_out = s > 1 ? (size_t)s * c->D * (c->K + 1) * 4 : 0;
    return MICONV_OK;
}

int causal_conv1d_bwd(const miconv_causal_conv_t *c, int dtype, void *workspace, size_t workspace_bytes,
                      void *stream) {
    if (!c) return MICONV_ERR_NULL;
    const int st = check_conv_sizes(c->B, c->D, c->L, c->K, dtype);
    if (st != MICONV_OK) return st;
    if (!workspace && workspace_bytes) return MICONV_ERR_NULL;
    const size_t es = elem_size(dtype), ns = (size_t)c->B * c->D * (c->K - 1);
    Checker k;
    conv_inputs(*c, es, &k);
    k.input(rows_span(c->dy, c->B, c->D, c->L, es), true);
    if (c->K > 1) k.input(flat(c->d_final_state, ns, es), false);
    k.output(rows_span(c->dx, c->B, c->D, c->L, es), false);
    k.output(flat(c->dw, (size_t)c->D * c->K, 4), false);
    k.output(flat(c->dbias, c->D, 4), false);
    if (c->K > 1) k.output(flat(c->d_initial_state, ns, es), false);
    const int splits = causal_bwd_splits(*c, workspace ? workspace_bytes : 0);
    if (splits > 1) k.output(flat(workspace, (size_t)splits * c->D * (c->K + 1), 4), true);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : launch_causal_bwd(*c, dtype, splits, (float *)workspace, (hipStream_t)stream);
}

int causal_conv1d_step(int B, int D, int K, int silu, int dtype, miconv_rows_t x, const void *state, int slots,
                       const int *slot_of, const void *w, const float *bias, void *state_out, miconv_rows_t y,
                       void *stream) {
    const int st = check_conv_sizes(B, D, 1, K, dtype);
    if (st != MICONV_OK) return st;
    if (bad_size(slots) || (!slot_of && slots != B)) return MICONV_ERR_BAD_DIM;
    const size_t es = elem_size(dtype), ns = (size_t)slots * D * (K - 1);
    Checker k;
    k.input(rows_span(x, B, D, 1, es), true);
    k.input(flat(w, (size_t)D * K, es), true);
    k.input(flat(bias, D, 4), false);
    k.input(flat(slot_of, B, 4), false);
    k.output(rows_span(y, B, D, 1, es), true);
    if (K > 1) {
        k.output(flat(state_out, ns, es), true);
        if (state != state_out) k.input(flat(state, ns, es), true);
    }
    const int bad = k.done();
    if (bad != MICONV_OK) return bad;
    return launch_causal_step(B, D, K, silu, dtype, x, state, slots, slot_of, w, bias, state_out, y,
                              (hipStream_t)stream);
}

int selective_scan_states_size(int B, int D, int L, int N, size_t *bytes_out) {
    if (!bytes_out) return MICONV_ERR_NULL;
    if (bad_size(B) || bad_size(D) || bad_size(L) || N < 1 || N > MICONV_SCAN_MAX_STATES) return MICONV_ERR_BAD_DIM;
    if ((long long)B * D > kMaxSize) return MICONV_ERR_TOO_LARGE;
    *bytes_out = (size_t)B * D * scan_chunks(L) * N * 4;
    return MICONV_OK;
}

int selective_scan_fwd_workspace_size(const miconv_scan_t *s, int dtype, size_t workspace_limit, size_t *bytes_out) {
    if (!s || !bytes_out) return MICONV_ERR_NULL;
    const int st = check_scan_sizes(*s, dtype);
    if (st != MICONV_OK) return st;
    *bytes_out = plan_scan_fwd(*s, workspace_limit).bytes;
    return MICONV_OK;
}

int selective_scan_fwd(const miconv_scan_t *s, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!s) return MICONV_ERR_NULL;
    const int st = check_scan_sizes(*s, dtype);
    if (st != MICONV_OK) return st;
    if (!workspace && workspace_bytes) return MICONV_ERR_NULL;
    const ScanSplit split = plan_scan_fwd(*s, workspace ? workspace_bytes : 0);
    const size_t es = elem_size(dtype), ns = state_count(*s);
    Checker k;
    scan_inputs(*s, es, &k);
    k.input(flat(s->initial_state, ns, 4), false);
    k.input(flat(s->lengths, s->B, 4), false);
    k.output(rows_span(s->y, s->B, s->D, s->L, es), true);
    k.output(flat(s->final_state, ns, 4), false);
    k.output(flat(s->states, ns * scan_chunks(s->L), 4), false);
    if (split.bytes) k.output(flat(workspace, split.bytes / 4, 4), true);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : launch_scan_fwd(*s, dtype, split, (float *)workspace, (hipStream_t)stream);
}

int selective_scan_fwd_describe(const miconv_scan_t *s, int dtype, size_t workspace_bytes, char *buf, size_t buflen) {
    if (!buf || buflen == 0) return MICONV_ERR_NULL;
    buf[0] = 0;
    if (!s) return MICONV_ERR_NULL;
    const int st = check_scan_sizes(*s, dtype);
    if (st != MICONV_OK) return st;
    const ScanSplit p = plan_scan_fwd(*s, workspace_bytes);
    static const char *const names[] = {"64x16", "64x8", "16x8", "16x8shared"};
    snprintf(buf, buflen, "algo=scan_fwd form=%s segments=%d ws=%zu", names[scan_form(*s, p)], p.segs, p.bytes);
    return MICONV_OK;
}

// The slices of a backward pass with this workspace, of which it uses the cap at most.
static ScanBwdSlice bwd_slice(const miconv_scan_t &s, size_t workspace_bytes) {
    const size_t cap = MICONV_MAX_WORKSPACE_BYTES;
    return slice_scan_bwd(s, workspace_bytes < cap ? workspace_bytes : cap);
}

int selective_scan_bwd_workspace_size_ex(const miconv_scan_t *s, int dtype, size_t workspace_limit,
                                         size_t *bytes_out) {
    if (!s || !bytes_out) return MICONV_ERR_NULL;
    const int st = check_scan_sizes(*s, dtype);
    if (st != MICONV_OK) return st;
    *bytes_out = bwd_slice(*s, workspace_limit).bytes;
    return MICONV_OK;
}

int selective_scan_bwd_workspace_size(const miconv_scan_t *s, int dtype, size_t *bytes_out) {
    return selective_scan_bwd_workspace_size_ex(s, dtype, MICONV_MAX_WORKSPACE_BYTES, bytes_out);
}

int selective_scan_bwd(const miconv_scan_t *s, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!s) return MICONV_ERR_NULL;
    const int st = check_scan_sizes(*s, dtype);
    if (st != MICONV_OK) return st;
    if (!workspace) return MICONV_ERR_NULL;
    const ScanBwdSlice p = bwd_slice(*s, workspace_bytes);
    const size_t es = elem_size(dtype), ns = state_count(*s), nbc = (size_t)s->B * s->G * s->N * s->L;
    if (workspace_bytes < p.bytes) return MICONV_ERR_WORKSPACE;
    if ((s->z.data != nullptr) != (s->dz.data != nullptr)) return MICONV_ERR_NULL;
    Checker k;
    scan_inputs(*s, es, &k);
    k.input(flat(s->lengths, s->B, 4), false);
    k.input(flat(s->states, ns * scan_chunks(s->L), 4), true);
    k.input(rows_span(s->dy, s->B, s->D, s->L, es), true);
    k.input(flat(s->d_final_state, ns, 4), false);
    k.output(rows_span(s->dx, s->B, s->D, s->L, es), true);
    k.output(rows_span(s->ddelta, s->B, s->D, s->L, es), true);
    k.output(rows_span(s->dz, s->B, s->D, s->L, es), false);
    k.output(flat(s->dA, (size_t)s->D * s->N, 4), true);
    k.output(flat(s->dB, nbc, 4), true);
    k.output(flat(s->dC, nbc, 4), true);
    k.output(flat(s->dD, s->D, 4), false);
    k.output(flat(s->ddelta_bias, s->D, 4), false);
    k.output(flat(s->d_initial_state, ns, 4), false);
    k.output(flat(workspace, p.bytes / 4, 4), true);
    const int bad = k.done();
    return bad != MICONV_OK ? bad : launch_scan_bwd(*s, dtype, p, (float *)workspace, (hipStream_t)stream);
}

int selective_scan_bwd_describe(const miconv_scan_t *s, int dtype, size_t workspace_bytes, char *buf, size_t buflen) {
    if (!buf || buflen == 0) return MICONV_ERR_NULL;
    buf[0] = 0;
    if (!s) return MICONV_ERR_NULL;
    const int st = check_scan_sizes(*s, dtype);
    if (st != MICONV_OK) return st;
    const ScanBwdSlice r = bwd_slice(*s, workspace_bytes);
    if (workspace_bytes < r.bytes) return MICONV_ERR_WORKSPACE;
    miconv_scan_t one = *s;
    one.B = r.sequences;
    one.G = r.groups;
    one.D = r.groups * r.channels;
    one.L = r.steps;
    const ScanBwdPlan p = plan_scan_bwd(one, r.bytes - r.carry * 4);
    snprintf(buf, buflen, "algo=scan_bwd segments=%d carry_segments=%d beside=%d slice=%dx%dx%dx%d ws=%zu", p.segs,
             p.carry_segs, p.beside, r.sequences, r.groups, r.channels, r.steps, r.bytes);
    return MICONV_OK;
}

int selective_scan_step(const miconv_scan_t *s, int dtype, const float *state, int slots, const int *slot_of,
                        float *state_out, void *stream) {
    if (!s) return MICONV_ERR_NULL;
    const int st = check_scan_sizes(*s, dtype);
    if (st != MICONV_OK) return st;
    if (s->L != 1 || bad_size(slots) || (!slot_of && slots != s->B)) return MICONV_ERR_BAD_DIM;
    const size_t es = elem_size(dtype), ns = (size_t)slots * s->D * s->N;
    Checker k;
    scan_inputs(*s, es, &k);
    k.input(flat(slot_of, s->B, 4), false);
    k.output(rows_span(s->y, s->B, s->D, 1, es), true);
    k.output(flat(state_out, ns, 4), true);
    if (state != state_out) k.input(flat(state, ns, 4), true);
    const int bad = k.done();
    if (bad != MICONV_OK) return bad;
    return launch_scan_step(*s, dtype, state, slots, slot_of, state_out, (hipStream_t)stream);
}

int quantize_tokens(int B, int L, int C, int dtype, const void *x, long long stride_b, long long stride_l,
                    long long stride_c, signed char *q, float *scale, void *stream) {
    if (bad_size(B) || bad_size(L) || C < 1 || C > 131072) return MICONV_ERR_BAD_DIM;
    if ((long long)B * L > kMaxSize) return MICONV_ERR_TOO_LARGE;
    if (bad_dtype(dtype)) return MICONV_ERR_DTYPE;
    if (stride_c != 1 && stride_l != 1) return MICONV_ERR_BAD_DIM;
    if (stride_b < 0 || stride_l < 0 || stride_c < 0) return MICONV_ERR_BAD_DIM;
    const size_t es = elem_size(dtype);
    const int pad = (C + MICONV_I8_PAD - 1) / MICONV_I8_PAD * MICONV_I8_PAD;
    const __int128 one = (__int128)(L - 1) * stride_l + (__int128)(C - 1) * stride_c + 1;
    if (one > kMaxSpan) return MICONV_ERR_TOO_LARGE;
    Checker k;
    k.input({(uintptr_t)x, B, stride_b, 1, 0, (long long)one, es}, true);
    k.output(flat(q, (size_t)B * L * pad, 1), true);
    k.output(flat(scale, (size_t)B * L, 4), true);
    if ((uintptr_t)q % 16) k.fail(MICONV_ERR_ALIGN);
    const int bad = k.done();
    if (bad != MICONV_OK) return bad;
    return launch_quantize(B, L, C, dtype, x, stride_b, stride_l, stride_c, q, scale, (hipStream_t)stream);
}

static int check_i8_sizes(int B, int L, int O, int C_pad) {
    if (bad_size(B) || bad_size(L) || bad_size(O) || C_pad < MICONV_I8_PAD || C_pad > 131072 ||
        C_pad % MICONV_I8_PAD)
        return MICONV_ERR_BAD_DIM;
    if ((long long)B * L > kMaxSize) return MICONV_ERR_TOO_LARGE;
    // 16 x 16 tiles are counted in a 32-bit grid
    if ((((long long)B * L + 15) / 16) * ((O + 15) / 16) > kMaxSize) return MICONV_ERR_TOO_LARGE;
    return MICONV_OK;
}

int matmul_i8_workspace_size(int B, int L, int O, int C_pad, size_t workspace_limit, size_t *bytes_out) {
    if (!bytes_out) return MICONV_ERR_NULL;
    const int st = check_i8_sizes(B, L, O, C_pad);
    if (st != MICONV_OK) return st;
    const int s = i8_splits(B * L, O, C_pad, workspace_limit);
    *bytes_out = s > 1 ? (size_t)s * B * L * O * 4 : 0;
    return MICONV_OK;
}

int matmul_i8_describe(int B, int L, int O, int C_pad, size_t workspace_bytes, char *buf, size_t buflen) {
    if (!buf || buflen == 0) return MICONV_ERR_NULL;
    buf[0] = 0;
    const int st = check_i8_sizes(B, L, O, C_pad);
    if (st != MICONV_OK) return st;
    const int splits = i8_splits(B * L, O, C_pad, workspace_bytes);
    const I8Form f = i8_form(B * L, O, C_pad, splits);
    if (f.few)
        snprintf(buf, buflen, "algo=i8_few tokens=%d", f.few * 16);
    else
        snprintf(buf, buflen, "algo=i8_tile tile=%d stages=%d splits=%d", f.side, f.stages, splits);
    return MICONV_OK;
}

int matmul_i8(int B, int L, int O, int C_pad, const signed char *q, const float *qscale, const signed char *wq,
              const float *wscale, const float *bias, int channel_major, int out_dtype, void *y, void *workspace,
              size_t workspace_bytes, void *stream) {
    const int st = check_i8_sizes(B, L, O, C_pad);
    if (st != MICONV_OK) return st;
    if (bad_dtype(out_dtype)) return MICONV_ERR_DTYPE;
    if (!workspace && workspace_bytes) return MICONV_ERR_NULL;
    const size_t T = (size_t)B * L, es = elem_size(out_dtype);
    Checker k;
    k.input(flat(q, T * C_pad, 1), true);
    k.input(flat(qscale, T, 4), true);
    k.input(flat(wq, (size_t)O * C_pad, 1), true);
    k.input(flat(wscale, O, 4), true);
    k.input(flat(bias, O, 4), false);
    k.output(flat(y, T * O, es), true);
    if ((uintptr_t)q % 16 || (uintptr_t)wq % 16) k.fail(MICONV_ERR_ALIGN);
    const int splits = i8_splits((int)T, O, C_pad, workspace ? workspace_bytes : 0);
    if (splits > 1) k.output(flat(workspace, (size_t)splits * T * O, 4), true);
    const int bad = k.done();
    if (bad != MICONV_OK) return bad;
    return launch_matmul_i8(B, L, O, C_pad, q, qscale, wq, wscale, bias, channel_major != 0, out_dtype, y, splits,
                            (int *)workspace, (hipStream_t)stream);
}

}  // extern "C"
