// delta.h -- the gated delta rule's kernels: argument blocks, workspace layout and
// host entries.  Arguments are already validated.
//
// Per value head, with the chunk's inclusive sums of log decays G, D_ij = exp(G_i - G_j) for i >= j, e = exp(G),
// f = exp(G_last - G), queries and keys normalised and scaled as the call asks, S the state before the chunk:
//   Z = inv(I + (D * k k^T)_{i>j} diag(beta)) (v - e (k S)),   u = beta Z
//   y = e (q S) + (D * q k^T) u,   S' = e_last S + (f k)^T u
// which is the recurrence  z_t = v_t - e^{g_t} S^T k_t,  S <- e^{g_t} S + k_t (beta_t z_t)^T,  y_t = S^T q_t
// with the steps of a chunk solved together.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/miconv.h"
#include "ssm.h"

namespace miconv {

constexpr int kDeltaChunk = 64;
constexpr int kDeltaSlice = 16;            // value channels of one MFMA tile
constexpr int kDeltaStepValues = 64;       // of one work-group of the single-token step

constexpr int delta_chunks(int L) { return (L + kDeltaChunk - 1) / kDeltaChunk; }
// Key channels are padded to whole loops of the kernels, value channels to a pair of tiles.
constexpr int delta_key_pad(int P) { return P <= 64 ? 64 : (P <= 128 ? 128 : 256); }
constexpr int delta_value_pad(int V) { return (V + 31) / 32 * 32; }

constexpr int kDeltaSquare = kDeltaChunk * kDeltaChunk * 2;    // bytes of a plane of 64 x 64; inv and attn have three

// What the pass over chunks finds about each step of a chunk and value head.
struct DeltaSteps {
    double G[kDeltaChunk];                 // sums of log decays
    float ek[kDeltaChunk], eq[kDeltaChunk];   // exp(G) times the key's / query's factor
    float fk[kDeltaChunk];                 // exp(G_last - G) times the key's factor
    float beta[kDeltaChunk];
    float rk[kDeltaChunk], rq[kDeltaChunk];   // 1 / norm of key and query, or 1; eq holds the call's scale too
    float last;                            // exp(G_last)
    float pad[3];
};

// A slice of the problem: sequences b0 .. b0 + nb, chunks c0 .. c0 + nc.
struct DeltaSlice {
    int b0, nb, c0, nc;
};

// Places in the workspace, in bytes.  Matrices are stored in the order in which a wave's lanes take
// the row operand of 16x16x32 MFMAs: [row tile of 16][32 columns][lane][8].
struct DeltaWork {
    size_t k, q;                           // k and (forward) q, [t][p], a plane of bf16 after the other
    size_t inv, attn;                      // planes of the inverse and of (D * q k^T), transposed in the backward pass
    size_t steps;                          // DeltaSteps
    size_t state;                          // [nb][Hv][Pp][Vp] fp32: carried between slices of time
    size_t F, after;                       // backward: [chunk][Vp][64], [chunk][Pp][Vp] fp32
    size_t sums;                           // backward, 256 key channels: dq and dk over a key head's value heads so far
    size_t bytes;
};

struct DeltaArgs {
    miconv_gated_delta_t d;
    DeltaSlice s;
    int rep, chunks;                       // Hv / Hk, chunks of L
    int slices;                            // value slices of the scan kernels
    int Vp;
    char *ws;
    DeltaWork w;
    int first, last;                       // whether the slice holds the first / the last chunk of time
    int more;                              // a dispatch's first work-group
};

// Saved by the forward pass for the backward pass, per [b][head][chunk]: the state before the chunk [Pp][Vp] and
// Z transposed [Vp][64], fp32.
constexpr size_t delta_saved(int P, int V) {
    return ((size_t)delta_key_pad(P) + kDeltaChunk) * delta_value_pad(V);
}

DeltaWork delta_work(const miconv_gated_delta_t &d, int dtype, const DeltaSlice &s, bool backward);
// The largest slice within the budget, or the smallest there is.
DeltaSlice delta_slice(const miconv_gated_delta_t &d, int dtype, size_t budget, bool backward);

int launch_delta_prepare(const DeltaArgs &a, int dtype, bool backward, hipStream_t st);
int launch_delta_fwd(const DeltaArgs &a, int dtype, hipStream_t st);
int launch_delta_bwd(const DeltaArgs &a, int dtype, hipStream_t st);
int launch_delta_grads(const DeltaArgs &a, int dtype, hipStream_t st);
int launch_delta_step(const miconv_gated_delta_t &d, int dtype, const float *state, int slots, const int *slot_of,
                      float *state_out, hipStream_t st);

}  // namespace miconv
