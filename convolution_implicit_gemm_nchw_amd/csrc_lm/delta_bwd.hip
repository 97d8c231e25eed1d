// delta_bwd.hip -- gradients of the gated delta rule.
//
// With dS the gradient of the state after a chunk and T = inv(I + diag(beta) (D * k k^T)_{i>j}):
//   du = (D * q k^T)^T dy + f (k dS),   F = T^T du,   dv = beta F,
//   dS <- e_last dS + (e q)^T dy - (e k)^T (beta F)
// goes from the last chunk to the first (delta_bwd_kernel).  The rest of a chunk needs nothing but what stands
// on its two ends, and runs for all chunks side by side (delta_grads_kernel): with Z and the state S before the
// chunk, which the forward pass saved,
//   dP_ij = beta_j D_ij dy_i.Z_j (i >= j),   dA_ij = -beta_i beta_j D_ij F_i.Z_j (i > j),   dbeta_i = F_i.Z_i
//   dq = e (S dy) + dP k,   read = dA k - e beta (S F),   write = f beta (dS Z) + dP^T q + dA^T k,   dk = read + write
// A key reads with the decays up to its step and writes against them, so the gradient of the sum G_i is
// q_i.dq_i + k_i.read_i - k_i.write_i, and that of g_t the sum of those from t on, with what the chunk's end adds:
// e_last <S, dS> + sum_j k_j.(f beta dS Z)_j.
#include "delta_device.h"

namespace miconv {

namespace {

// Laid out and split as the forward scan; the state here is dS.  Four waves go along the chain k dS, the transposed inverse
// times du, dS - (e k)^T (beta F); the others compute attn^T dy, for the chunk that comes next, and meanwhile
// (e q)^T dy for all key channels, half of which they hand over through LDS.  Bound like that one by the chain's
// latency: 2 x 2048 steps of 16 heads of 128 and 128 channels in bf16, 32 chunks, take 100 us.
template <int DT, int DK>
__global__ __launch_bounds__(512) void delta_bwd_kernel(DeltaArgs a, float *state_in, float *state_out) {
    constexpr int TI = in_planes(DT), kKS = DK / 32, kTiles = DK / 16, kMT = kTiles > 8 ? kTiles / 8 : 1, kN = kDeltaSlice;
    constexpr int kPitchS = DK + 8, kPitchT = kDeltaChunk + 8, kPlaneS = kN * kPitchS, kPlaneT = kN * kPitchT;
    constexpr int kPitchF = kDeltaChunk + 4, kHalf = kTiles < 8 ? kTiles : kTiles / 2;   // tiles of the chain's waves
    typedef typename Elem<DT>::T T;
    __shared__ __attribute__((aligned(16))) uint16_t Sp[3 * kPlaneS], Up[3 * kPlaneT], Wp[3 * kPlaneT];
    __shared__ __attribute__((aligned(16))) float Bs[2][kN * kPitchF];   // attn^T dy of this chunk and the next
    __shared__ __attribute__((aligned(16))) float Qs[kHalf * 64 * 4];   // (e q)^T dy as accumulators
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), col = lane & 15, grp = lane >> 4;
    const bool queries = wave >= 4, owner = wave * kMT < kTiles;
    const int part = wave & 3, row4 = grp * 4, mine = part * 16 + row4;
    const int total = a.s.nb * a.d.Hv * a.slices;
    const int id = xcd_remap(blockIdx.x, total);
    const int slice = id % a.slices, bh = id / a.slices, h = bh % a.d.Hv, b = bh / a.d.Hv, B = a.s.b0 + b;
    const int hk = h / a.rep, v0 = slice * kN;
    const int valid = valid_steps(a.d.lengths, B, a.d.L);
    const int steps_first = a.s.c0 * kDeltaChunk;
    int chunks = (valid - steps_first + kDeltaChunk - 1) / kDeltaChunk;
    chunks = chunks < 0 ? 0 : (chunks > a.s.nc ? a.s.nc : chunks);

    f32x4 S[kMT];
    {
        const int P = a.last ? a.d.P : DK, V = a.last ? a.d.V : a.Vp;
        const float *in = a.last ? a.d.d_final_state : state_in;
        const long long at = a.last ? (long long)B * a.d.Hv + h : bh;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int p = (wave * kMT + i) * 16 + row4 + r, v = v0 + col;
                S[i][r] = in && p < P && v < V ? in[(at * P + p) * V + v] : 0.0f;
            }
    }
    const auto put_state = [&] {
        if (!owner) return;
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const float v[4] = {S[i][0], S[i][1], S[i][2], S[i][3]};
            put_planes<3>(Sp + col * kPitchS + (wave * kMT + i) * 16 + row4, kPlaneS, v);
        }
    };
    put_state();
    for (int i = threadIdx.x; i < 3 * kN * 8; i += 512)        // the zeros behind du's steps
        Up[i / (kN * 8) * kPlaneT + i / 8 % kN * kPitchT + kDeltaChunk + i % 8] = 0;

    const size_t of_k = ((size_t)b * a.s.nc * a.d.Hk + hk) * TI * 64 * DK * 2, step_k = (size_t)a.d.Hk * TI * 64 * DK * 2;
    const size_t of_v = (size_t)b * a.s.nc * a.d.Hv + h;
    constexpr int kPlaneK = 64 * DK * 2;
    // three planes of 256 key channels are more than the registers hold ahead of their use
    constexpr bool kLate = TI == 3 && DK == 256;
    const T *krow[kMT];
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
        const int p = (wave * kMT + i) * 16 + col;
        krow[i] = row_of<DT>(a.d.k, B, hk * a.d.P + (p < a.d.P ? p : 0));
    }
    Raw8<DT> ft[kMT][2];
    float last = 0.0f;
    const auto steps_of = [&](int c) {
        return (const DeltaSteps *)(a.ws + a.w.steps + (of_v + (size_t)c * a.d.Hv) * sizeof(DeltaSteps));
    };
    const auto load_turned = [&](int c, bool whole) {
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                ft[i][ks] = steps8<DT>(krow[i], whole, steps_first + c * kDeltaChunk + ks * 32 + grp * 8, valid);
    };
    // The transposed inverse and attn are upper triangular: the first 32 columns of rows 32.. are zero and not stored.
    const bool lower = part < 2;
    const auto load_m = [&](size_t place, int c, u32x4 (&fm)[2][3]) {
        const char *at = a.ws + place + (of_v + (size_t)c * a.d.Hv) * 3 * kDeltaSquare;
        fragment<3>(at, part * 2 + (lower ? 0 : 1), kDeltaSquare, fm[0]);
        fragment<3>(at, part * 2 + 1, kDeltaSquare, fm[1]);
    };
    const auto save_state = [&](int c) {
        if (!owner) return;
        float *after = (float *)(a.ws + a.w.after) + (of_v + (size_t)c * a.d.Hv) * DK * a.Vp;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                after[(size_t)((wave * kMT + i) * 16 + row4 + r) * a.Vp + v0 + col] = S[i][r];
    };
    // dS from `given`, (e q)^T dy of the wave's own tiles
    const auto update = [&](int c, bool whole, f32x4 (&given)[kMT]) {
        if (!owner) return;
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            if constexpr (kLate) {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    ft[i][ks] = steps8<DT>(krow[i], whole, steps_first + c * kDeltaChunk + ks * 32 + grp * 8, valid);
            }
            u32x4 k0[TI], k1[TI];
            const int tile = wave * kMT + i;
            planes_of<DT>(only<DT>(ft[i][0], tile * 16 + col < a.d.P), k0);
            planes_of<DT>(only<DT>(ft[i][1], tile * 16 + col < a.d.P), k1);
            Sums<2> sum;
            u32x4 w[3];
            const uint16_t *from = Wp + col * kPitchT + grp * 8;
            get_planes<3>(from, kPlaneT, w);
            sum.add(k0, w);
            get_planes<3>(from + 32, kPlaneT, w);
            sum.add(k1, w);
            S[i] = S[i] * last + (given[i] + sum.total());
        }
        put_state();
    };
    // as in the forward scan; here the chunk that ends inside comes first
    int full = (valid - steps_first) / kDeltaChunk;
    full = valid <= steps_first ? 0 : (full < chunks ? full : chunks);
    const int begin = chunks - 1;
    if (chunks) {
        if constexpr (!kLate) load_turned(begin, full == chunks);
        last = steps_of(begin)->last;
    }
    if (!chunks) {
    } else if (!queries) {
        u32x4 fk[kLate ? 1 : kKS][TI], fi[2][3];
        T *const out = row_of<DT>(a.d.dv, B, h * a.d.V + (v0 + col < a.d.V ? v0 + col : 0));
        const auto load_k = [&](int c) {
#pragma unroll
            for (int ks = 0; ks < kKS && !kLate; ++ks)
                fragment<TI>(a.ws + a.w.k + of_k + c * step_k, part * kKS + ks, kPlaneK, fk[ks]);
        };
        load_k(begin);
        load_m(a.w.inv, begin, fi);
        f32x4 vek = *(const f32x4 *)(steps_of(begin)->ek + mine), vfk = *(const f32x4 *)(steps_of(begin)->fk + mine);
        f32x4 vbeta = *(const f32x4 *)(steps_of(begin)->beta + mine);
        // rows 32.. meet the first fragment with the zeros behind each channel's 64 steps
        const int first_half = lower ? 0 : kDeltaChunk - grp * 8;
        const auto chunk = [&](const int c, auto is_full) {
            constexpr bool FULL = decltype(is_full)::value;
            const int next = c ? c - 1 : 0;
            save_state(c);
            __syncthreads();
            Sums<2> kd;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                if constexpr (kLate) fragment<TI>(a.ws + a.w.k + of_k + c * step_k, part * kKS + ks, kPlaneK, fk[0]);
                u32x4 s[3];
                get_planes<3>(Sp + col * kPitchS + ks * 32 + grp * 8, kPlaneS, s);
                kd.add(fk[kLate ? 0 : ks], s);
            }
            const f32x4 k = kd.total(), back = *(const f32x4 *)(Bs[c & 1] + col * kPitchF + mine);
            float du[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) du[r] = __builtin_fmaf(vfk[r], k[r], back[r]);
            put_planes<3>(Up + col * kPitchT + mine, kPlaneT, du);
            load_k(next);
            vfk = *(const f32x4 *)(steps_of(next)->fk + mine);
            __syncthreads();
            float *Fout = (float *)(a.ws + a.w.F) + (of_v + (size_t)c * a.d.Hv) * a.Vp * kDeltaChunk;
            Sums<2> sum;
            u32x4 u[3];
            const uint16_t *from = Up + col * kPitchT + grp * 8;
            get_planes<3>(from + first_half, kPlaneT, u);
            sum.add(fi[0], u);
            get_planes<3>(from + 32, kPlaneT, u);
            sum.add(fi[1], u);
            const f32x4 F = sum.total();
            float w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = -(vek[r] * (vbeta[r] * F[r]));
            put_planes<3>(Wp + col * kPitchT + mine, kPlaneT, w);
            // ahead of the stores: loads come back in their order, stores among them
            const f32x4 beta = vbeta;
            load_m(a.w.inv, next, fi);
            vek = *(const f32x4 *)(steps_of(next)->ek + mine);
            vbeta = *(const f32x4 *)(steps_of(next)->beta + mine);
            __syncthreads();
            f32x4 given[kMT];
            if (owner) {
#pragma unroll
                for (int i = 0; i < kMT; ++i)
                    given[i] = *(const f32x4 *)(Qs + ((wave * kMT + i) * 64 + lane) * 4);
            }
            update(c, FULL, given);
            last = steps_of(next)->last;
            if constexpr (!kLate) load_turned(next, FULL || c);
            *(f32x4 *)(Fout + (size_t)(v0 + col) * kDeltaChunk + mine) = F;
            if (v0 + col < a.d.V) {
                const int t = steps_first + c * kDeltaChunk + mine;
                float dv[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) dv[r] = FULL || t + r < valid ? beta[r] * F[r] : 0.0f;
                store4_until<DT>(out, FULL, t, a.d.L, dv);
            }
        };
        if (full < chunks) chunk(full, Whole<false>());
        for (int c = full - 1; c >= 0; --c) chunk(c, Whole<true>());
    } else {
        constexpr bool kAhead = TI == 1 && DK <= 128;    // queries likewise, where the registers hold them
        u32x4 fa[2][3];
        Raw8<DT> fq[kAhead ? 2 * kMT : 1][2];
        Raw8<DT> fg[2], fn[2];                 // dy as column operand: of this chunk, and of the next
        f32x4 veq[2][2];                       // of the steps that fg holds
        const T *const grow = row_of<DT>(a.d.dy, B, h * a.d.V + (v0 + col < a.d.V ? v0 + col : 0)), *qrow[2 * kMT];
        // tiles of queries that this wave multiplies: its own and those of the wave that it hands over to
        const auto tile_of = [&](int i) { return (i < kMT ? wave : part) * kMT + i % kMT; };
#pragma unroll
        for (int i = 0; i < 2 * kMT; ++i) {
            const int p = tile_of(i) * 16 + col;
            qrow[i] = row_of<DT>(a.d.q, B, hk * a.d.P + (p < a.d.P ? p : 0));
        }
        const auto load_dy = [&](int c, bool whole) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                fn[ks] = steps8<DT>(grow, whole, steps_first + c * kDeltaChunk + ks * 32 + grp * 8, valid);
        };
        const auto turned_q = [&](int i, int c, int ks, bool whole) {
            return steps8<DT>(qrow[i], whole, steps_first + c * kDeltaChunk + ks * 32 + grp * 8, valid);
        };
        const auto load_q = [&](int c, bool whole) {
#pragma unroll
            for (int i = 0; i < 2 * kMT && kAhead; ++i)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) fq[i][ks] = turned_q(i, c, ks, whole);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) veq[ks][e] = *(const f32x4 *)(steps_of(c)->eq + ks * 32 + grp * 8 + e * 4);
        };
        // attn^T dy of chunk c, whose attn is in fa and dy in fn, to Bs[c & 1]; then the next one's are loaded
        const auto put_back = [&](int c, int next, bool whole) {
            Sums<2> sum;
            u32x4 g[TI];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                planes_of<DT>(only<DT>(fn[ks], v0 + col < a.d.V && (ks || lower)), g);
                sum.add(fa[ks], g);
            }
            *(f32x4 *)(Bs[c & 1] + col * kPitchF + mine) = sum.total();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) fg[ks] = fn[ks];
            load_m(a.w.attn, next, fa);
            load_dy(next, whole);
        };
        load_m(a.w.attn, begin, fa);
        load_dy(begin, full == chunks);
        load_q(begin, full == chunks);
        put_back(begin, begin ? begin - 1 : 0, begin || full == chunks);
        const auto chunk = [&](const int c, auto is_full) {
            constexpr bool FULL = decltype(is_full)::value;
            const int next = c ? c - 1 : 0;
            u32x4 g[2][3];                         // e dy, split while the other waves finish the chunk before
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                float x[8];
                widen8<DT>(only<DT>(fg[ks], v0 + col < a.d.V), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= veq[ks][e >> 2][e & 3];
                split8<3>(x, g[ks]);
#pragma unroll
                for (int o = 0; o < 3; ++o) asm volatile("" : "+v"(g[ks][o]));
            }
            save_state(c);
            __syncthreads();
            f32x4 given[kMT];
#pragma unroll
            for (int i = 0; i < 2 * kMT; ++i) {
                const int tile = tile_of(i);
                if (kTiles < 8 && i < kMT) continue;     // with 64 key channels these waves own no tile
                Sums<2> sum;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    u32x4 q[TI];
                    if constexpr (!kAhead) fq[0][ks] = turned_q(i, c, ks, FULL);
                    planes_of<DT>(only<DT>(fq[kAhead ? i : 0][ks], tile * 16 + col < a.d.P), q);
                    sum.add(q, g[ks]);
                }
                const f32x4 t = sum.total();
                if (i < kMT)
                    given[i % kMT] = t;
                else
                    *(f32x4 *)(Qs + (tile * 64 + lane) * 4) = t;
            }
            load_q(next, FULL || c);
            __syncthreads();
            put_back(next, c > 1 ? c - 2 : 0, FULL || c);      // after the first chunk of time, for nothing
            __syncthreads();
            update(c, FULL, given);
            last = steps_of(next)->last;
            if constexpr (!kLate) load_turned(next, FULL || c);
        };
        if (full < chunks) chunk(full, Whole<false>());
        for (int c = full - 1; c >= 0; --c) chunk(c, Whole<true>());
    }
    // chunks past the sequence's end
    for (int c = chunks; queries && c < a.s.nc; ++c) {
        const float zeros[4] = {};
        if (v0 + col < a.d.V)
            store4_until<DT>(row_of<DT>(a.d.dv, B, h * a.d.V + v0 + col), steps_first + (c + 1) * kDeltaChunk <= a.d.L,
                             steps_first + c * kDeltaChunk + mine, a.d.L, zeros);
    }
    float *to = a.first ? a.d.d_initial_state : state_out;
    if (to && owner) {
        const int P = a.first ? a.d.P : DK, V = a.first ? a.d.V : a.Vp;
        const long long at = a.first ? (long long)B * a.d.Hv + h : bh;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int p = (wave * kMT + i) * 16 + row4 + r, v = v0 + col;
                if (p < P && v < V) to[(at * P + p) * V + v] = S[i][r];
            }
    }
}

// ------------------------------------------------------------------ the rest of each chunk
//
// A work-group takes one chunk of one key head, its value heads in turn, whose gradients of q and k add up in
// registers.  A wave owns a quarter of the key channels, NC tiles of 16, for half of the 64 steps; the state and dS
// are its column operands, read from memory and split in registers.  Z, F and dy stand in LDS as planes
// [step][value channel], 64 channels at a time; after them, in the same place, dP and dA in both orders.
// One work-group fits a CU (122 KB of LDS, 248 registers), and no phase hides another's waits: of some 60000 cycles
// 14000 go to Z, F and dy, 15000 to the products with the states (9000 of matrix instructions), 8000 to those with dP
// and dA.  An eighth of the channels for all steps would split the states once instead of twice: 64 key channels then
// have 4 waves, and 13 heads of 6599 steps take 230 us instead of 172; at 128 channels both take as long.
// 2 x 2048 steps of 16 heads, 128 and 128 channels, bf16: 136 us, 2 TB/s of states, Z, F and operands.
template <int DT, int DK>
struct Grads {
    static constexpr int kWaves = 8, kThreads = kWaves * 64, kNC = DK / 64;
    static constexpr int kPair = kNC > 1 ? 2 : 1;          // tiles that share what is read of Z, F, dy, dP and dA
    static constexpr int kTiles = 2;                       // column tiles of the 64 x 64 products per wave
    static constexpr int kPitch = 72, kPlane = 64 * kPitch;   // bf16 elements
    static constexpr int TI = in_planes(DT);
    static constexpr bool kKeep = DK < 256, kHold = DK < 256, kAhead = DK == 64;
    static constexpr int kValues = 6 + TI, kPlanes = kValues > 12 ? kValues : 12;
};

// Sums over the 16 lanes of a row.
DEVI float sum16(float v) {
    v += cross<0xB1>(v);                       // quad_perm 1,0,3,2
    v += cross<0x4E>(v);                       // quad_perm 2,3,0,1
    v += cross<0x141>(v);                      // row_half_mirror
    v += cross<0x140>(v);                      // row_mirror
    return v;
}

template <int DT, int DK>
__global__ __launch_bounds__((Grads<DT, DK>::kThreads)) void delta_grads_kernel(DeltaArgs a) {
    typedef Grads<DT, DK> X;
    constexpr int TI = X::TI, NC = X::kNC, NP = X::kPair, W = X::kWaves, TILES = X::kTiles;
    typedef typename Elem<DT>::T T;
    __shared__ __attribute__((aligned(16))) uint16_t shared[X::kPlanes * X::kPlane];
    __shared__ float rows[W][4][64];           // a wave's part of q.dq, k.(read - write), and q.dq, k.dk in full
    __shared__ float part[W];                  // of what the chunk's end adds
    __shared__ float norm_q[64], norm_k[64];   // q.dq and k.dk of all heads, for the normalisation
    __shared__ float diag[64], diag_p[64], e[64], f[64];
    __shared__ __attribute__((aligned(16))) DeltaSteps steps;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), m0 = (wave >> 2) * 2;   // tiles m0, m0 + 1 of 16 steps
    const int id = a.more + blockIdx.x;
    const int hk = id % a.d.Hk, bc = id / a.d.Hk, c = bc % a.s.nc, b = bc / a.s.nc, B = a.s.b0 + b;
    const int t0 = (a.s.c0 + c) * kDeltaChunk, valid = valid_steps(a.d.lengths, B, a.d.L), end = valid - t0;
    const int stop = a.d.L - t0 < kDeltaChunk ? a.d.L - t0 : kDeltaChunk;     // steps of this chunk in the tensors
    if (end <= 0) {                            // a chunk past the sequence's end
        for (int i = tid; i < a.d.P * kDeltaChunk; i += X::kThreads) {
            const int d = i / kDeltaChunk, t = i % kDeltaChunk;
            if (t >= stop) continue;
            row_of<DT>(a.d.dq, B, hk * a.d.P + d)[t0 + t] = Elem<DT>::put(0.0f);
            row_of<DT>(a.d.dk, B, hk * a.d.P + d)[t0 + t] = Elem<DT>::put(0.0f);
        }
        for (int i = tid; i < a.rep * kDeltaChunk; i += X::kThreads) {
            const int h = hk * a.rep + i / kDeltaChunk, t = i % kDeltaChunk;
            if (t >= stop) continue;
            const size_t at = ((size_t)B * a.d.Hv + h) * a.d.L + t0 + t;
            a.d.dg[at] = a.d.dbeta[at] = 0.0f;
        }
        return;
    }
    const auto chunk = [&](auto is_whole) {
        constexpr bool whole = decltype(is_whole)::value;
        // The sums over heads stay in registers where these hold them, else in the workspace, each lane's own.
        f32x4 dq[X::kKeep ? 2 : 1][NC], dk[X::kKeep ? 2 : 1][NC];
        if constexpr (X::kKeep) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NC; ++n) dq[m][n] = dk[m][n] = f32x4{0, 0, 0, 0};
        }
        if (tid < 64) norm_q[tid] = norm_k[tid] = 0.0f;
        // four steps of this lane's channels of key and query, where the registers hold them: they are used three times
        Raw4<DT> held_k[X::kHold ? NC : 1][2], held_q[X::kHold ? NC : 1][2];
        if constexpr (X::kHold) {
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const int d = (wave & 3) * NC * 16 + n * 16 + (tid & 15), row = hk * a.d.P + (d < a.d.P ? d : 0);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int t = (m0 + m) * 16 + (tid >> 4 & 3) * 4;
                    held_k[n][m] = steps4<DT>(row_of<DT>(a.d.k, B, row) + t0, whole, t, end);
                    held_q[n][m] = steps4<DT>(row_of<DT>(a.d.q, B, row) + t0, whole, t, end);
                }
            }
        }

        for (int hr = 0; hr < a.rep; ++hr) {
            const int h = hk * a.rep + hr;
            // a lane's place, of which the compiler does not know that it is the same for all heads: what is made from
            // it is then not held in registers from one to the next
            const int lane = again(tid & 63), col = lane & 15, grp = lane >> 4, row4 = grp * 4;
            const int d0 = (wave & 3) * NC * 16 + col;   // key channels d0 + 16 n
            const size_t of_v = (size_t)bc * a.d.Hv + h;
            const float *S0 = (const float *)a.d.states + (((size_t)B * a.d.Hv + h) * a.chunks + a.s.c0 + c) * delta_saved(a.d.P, a.d.V);
            const float *Zs = S0 + (size_t)DK * a.Vp;
            const float *S1 = (const float *)(a.ws + a.w.after) + of_v * DK * a.Vp;
            const float *Fs = (const float *)(a.ws + a.w.F) + of_v * a.Vp * kDeltaChunk;
            if (hr) __syncthreads();               // the head before has read steps, shared and rows
            if (tid < (int)(sizeof(DeltaSteps) / 16))
                ((u32x4 *)&steps)[tid] = ((const u32x4 *)(a.ws + a.w.steps + of_v * sizeof(DeltaSteps)))[tid];
            f32x4 q_[2][NC], read[2][NC], write[2][NC], FZ[TILES], OZ[TILES];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NC; ++n) q_[m][n] = read[m][n] = write[m][n] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < TILES; ++j) FZ[j] = OZ[j] = f32x4{0, 0, 0, 0};
            float ends = 0.0f;
            const int mi = wave * 4 / W, j0 = wave % (W / 4);         // the wave's tiles: row mi, columns j0 + j W / 4

            // eight value channels of this lane's rows of the state and of dS: the next 32 columns' while these are multiplied
            f32x4 states0[NP][2], states1[NP][2];
            const auto load_states = [&](int n, int v) {
                const unsigned from = again(d0 + n * 16) * a.Vp + (v < a.Vp ? v : 0) + grp * 8;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    states0[n % NP][k] = *(const f32x4 *)(S0 + from + k * 4);
                    states1[n % NP][k] = *(const f32x4 *)(S1 + from + k * 4);
                }
            };
            if constexpr (X::kAhead) {
#pragma unroll
                for (int n = 0; n < NC; ++n) load_states(n, 0);
            }
            for (int v0 = 0; v0 < a.Vp; v0 += 64) {
                if (v0) __syncthreads();           // the channels before are used up
                // blocks of 4 steps x 8 channels: Z, F, dy; each of them loads and stores in a branch of its own
                const auto put = [&](int which, int t, int vl, const float (&x)[8][4]) {
                    uint16_t *to = shared + which * 3 * X::kPlane + t * X::kPitch + vl;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float eight[8] = {x[0][r], x[1][r], x[2][r], x[3][r], x[4][r], x[5][r], x[6][r], x[7][r]};
                        u32x4 s[3];
                        split8<3>(eight, s);
                        *(u32x4 *)(to + r * X::kPitch) = s[0];
                        if (which < 2 || TI == 3) {
                            *(u32x4 *)(to + r * X::kPitch + X::kPlane) = s[1];
                            *(u32x4 *)(to + r * X::kPitch + 2 * X::kPlane) = s[2];
                        }
                    }
                };
                for (int i = again(tid); i < 3 * 128; i += X::kThreads) {
                    const int which = uniform(i >> 7), t = (i & 15) * 4, vl = (i >> 4 & 7) * 8, v = v0 + vl;
                    float x[8][4];
                    if (which == 2) {
                        Raw4<DT> held[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            held[c] = steps4<DT>(row_of<DT>(a.d.dy, B, h * a.d.V + (v + c < a.d.V ? v + c : 0)) + t0, whole, t, end);
#pragma unroll
                        for (int c = 0; c < 8; ++c) widen4<DT>(held[c], v + c < a.d.V, x[c]);
                        put(2, t, vl, x);
                    } else {
                        const float *from = which ? Fs : Zs;
                        f32x4 held[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) held[c] = *(const f32x4 *)(from + (size_t)(v + c < a.Vp ? v + c : 0) * kDeltaChunk + t);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
#pragma unroll
                            for (int r = 0; r < 4; ++r) x[c][r] = v + c < a.Vp ? held[c][r] : 0.0f;
                        put(which, t, vl, x);
                    }
                }
                __syncthreads();
                const uint16_t *Zp = shared, *Fp = shared + 3 * X::kPlane, *Op = shared + 6 * X::kPlane;
#pragma unroll 1
                for (int ks = 0; ks < 2; ++ks) {
                    if (v0 + ks * 32 >= a.Vp) break;
                    const int at = again(ks * 32 + grp * 8);
                    // F Z^T and dy Z^T up to the diagonal
                    {
                        u32x4 fr[3], og[TI];
                        get_planes<3>(Fp + (mi * 16 + col) * X::kPitch + at, X::kPlane, fr);
                        get_planes<TI>(Op + (mi * 16 + col) * X::kPitch + at, X::kPlane, og);
#pragma unroll
                        for (int j = 0; j < TILES; ++j) {
                            const int jt = j0 + j * (W / 4);
                            if (jt > mi) break;
                            u32x4 z[3];
                            get_planes<3>(Zp + (jt * 16 + col) * X::kPitch + at, X::kPlane, z);
                            multiply<3, 3, 2>(fr, z, FZ[j]);
                            multiply<TI, 3, 2>(og, z, OZ[j]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NC; n += NP) {
                        u32x4 s0[NP][3], s1[NP][3];
#pragma unroll
                        for (int w = 0; w < NP; ++w) {
                            if constexpr (!X::kAhead) load_states(n + w, v0 + ks * 32);
                            float x[8], y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                x[k] = states0[w][k >> 2][k & 3];
                                y[k] = states1[w][k >> 2][k & 3];
                                ends = __builtin_fmaf(x[k], y[k], ends);
                            }
                            split8<3>(x, s0[w]);
                            split8<3>(y, s1[w]);
                            if constexpr (X::kAhead) load_states(n + w, v0 + ks * 32 + 32);
                        }
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const int from = again(((m0 + m) * 16 + col) * X::kPitch) + at;
                            u32x4 og[TI], r3[3];
                            get_planes<TI>(Op + from, X::kPlane, og);
#pragma unroll
                            for (int w = 0; w < NP; ++w) multiply<TI, 3, 2>(og, s0[w], q_[m][n + w]);
                            get_planes<3>(Fp + from, X::kPlane, r3);
#pragma unroll
                            for (int w = 0; w < NP; ++w) multiply<3, 3, 2>(r3, s0[w], read[m][n + w]);
                            get_planes<3>(Zp + from, X::kPlane, r3);
#pragma unroll
                            for (int w = 0; w < NP; ++w) multiply<3, 3, 2>(r3, s1[w], write[m][n + w]);
                            __builtin_amdgcn_sched_barrier(0);   // loads further ahead would not fit the registers
                        }
                    }
                }
            }
            if (tid < 64) {
                e[tid] = exp_any((float)steps.G[tid]);
                f[tid] = exp_any((float)(steps.G[63] - steps.G[tid]));
            }
            __syncthreads();                       // and the products have left the planes
            settle(q_, read, write, FZ, OZ);
            ends = m0 ? 0.0f : ends * steps.last;   // both halves of the steps have read the states
            // the rows' factors; the chunk's end reaches its decays through the last of them
            const auto four = [&](const miconv_rows_t &rows, const auto &held, int n, int m, float (&v)[4]) {
                const int at = again(d0 + n * 16);
                if constexpr (X::kHold)
                    widen4<DT>(held[n][m], at < a.d.P, v);
                else
                    widen4<DT>(steps4<DT>(row_of<DT>(rows, B, hk * a.d.P + (at < a.d.P ? at : 0)) + t0, whole, (m0 + m) * 16 + row4, end),
                               at < a.d.P, v);
            };
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int t = again((m0 + m) * 16 + row4);
                    float k[4];
                    four(a.d.k, held_k, n, m, k);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float beta = steps.beta[t + r];
                        q_[m][n][r] *= e[t + r];
                        read[m][n][r] *= -(e[t + r] * beta);
                        write[m][n][r] *= f[t + r] * beta;
                        ends = __builtin_fmaf(k[r] * steps.rk[t + r], write[m][n][r], ends);
                    }
                    // here, not where the sum is used, with all its terms in registers till then
                    asm volatile("" : "+v"(ends), "+v"(q_[m][n]), "+v"(read[m][n]), "+v"(write[m][n]));
                    __builtin_amdgcn_sched_barrier(0);
                }
            // dP and dA as row operands: [i][j] times the key's factor of j, for q and read, and [j][i] times the query's
            // or key's factor of i, for write
            uint16_t *Mq = shared, *Mr = shared + 3 * X::kPlane, *Mp = shared + 6 * X::kPlane, *Ma = shared + 9 * X::kPlane;
#pragma unroll
            for (int j = 0; j < TILES; ++j) {
                const int jt = j0 + j * (W / 4);
                if (jt > (mi | 1)) break;          // a block of 32 columns past the diagonal is never read
                const int cj = again(jt * 16 + col);
                const double Gj = steps.G[cj];
                const float bj = steps.beta[cj], rkj = steps.rk[cj];
                float pq[4], ar[4], pw[4], aw[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = mi * 16 + row4 + r;
                    const float D = i >= cj ? exp_any((float)(steps.G[i] - Gj)) * bj : 0.0f;
                    const float dP = i > cj ? D * OZ[j][r] : 0.0f, dA = i > cj ? -(D * steps.beta[i]) * FZ[j][r] : 0.0f;
                    pq[r] = dP * rkj;
                    ar[r] = dA * rkj;
                    pw[r] = dP * (steps.rq[i] * a.d.scale);
                    aw[r] = dA * steps.rk[i];
                    if (i == cj) {
                        diag[i] = FZ[j][r];
                        diag_p[i] = D * OZ[j][r];
                    }
                }
                u32x2 s[3];
                const auto across = [&](uint16_t *to) {
#pragma unroll
                    for (int p = 0; p < 3; ++p)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            to[p * X::kPlane + (mi * 16 + row4 + r) * X::kPitch + cj] =
                                (uint16_t)(r & 1 ? s[p][r >> 1] >> 16 : s[p][r >> 1]);
                };
                split4<3>(pq, s);
                across(Mq);
                split4<3>(ar, s);
                across(Mr);
                put_planes<3>(Mp + cj * X::kPitch + mi * 16 + row4, X::kPlane, pw);
                put_planes<3>(Ma + cj * X::kPitch + mi * 16 + row4, X::kPlane, aw);
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NC; n += NP)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    u32x4 fk[NP][TI], fq[NP][TI];
#pragma unroll
                    for (int w = 0; w < NP; ++w) {
                        const int d = again(d0 + (n + w) * 16), row = hk * a.d.P + (d < a.d.P ? d : 0), t = ks * 32 + grp * 8;
                        planes_of<DT>(only<DT>(steps8<DT>(row_of<DT>(a.d.k, B, row) + t0, whole, t, end), d < a.d.P), fk[w]);
                        planes_of<DT>(only<DT>(steps8<DT>(row_of<DT>(a.d.q, B, row) + t0, whole, t, end), d < a.d.P), fq[w]);
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int at = again(((m0 + m) * 16 + col) * X::kPitch + ks * 32 + grp * 8);
                        u32x4 s[3];
                        if (m0 >= 2 * ks) {        // columns up to the diagonal
                            get_planes<3>(Mq + at, X::kPlane, s);
#pragma unroll
                            for (int w = 0; w < NP; ++w) multiply<3, TI, 2>(s, fk[w], q_[m][n + w]);
                            get_planes<3>(Mr + at, X::kPlane, s);
#pragma unroll
                            for (int w = 0; w < NP; ++w) multiply<3, TI, 2>(s, fk[w], read[m][n + w]);
                        }
                        if (m0 < 2 * ks + 2) {     // columns from the diagonal on
                            get_planes<3>(Mp + at, X::kPlane, s);
#pragma unroll
                            for (int w = 0; w < NP; ++w) multiply<3, TI, 2>(s, fq[w], write[m][n + w]);
                            get_planes<3>(Ma + at, X::kPlane, s);
#pragma unroll
                            for (int w = 0; w < NP; ++w) multiply<3, TI, 2>(s, fk[w], write[m][n + w]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            settle(q_, read, write);
            // The rows' products with normalised query and key.  A step's own dP_ii k_i and dP_ii q_i add the same to
            // q_i.dq_i and k_i.write_i, so they enter after the decays' part: its terms then cancel no further than its
            // definition's do, and the first step from a zero state gets a zero.
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float x[4] = {}, y[4] = {}, z[4] = {}, w[4] = {};
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    float k[4], q[4];
                    four(a.d.k, held_k, n, m, k);
                    four(a.d.q, held_q, n, m, q);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = (m0 + m) * 16 + row4 + r;
                        x[r] = __builtin_fmaf(q[r], q_[m][n][r], x[r]);
                        y[r] = __builtin_fmaf(k[r], read[m][n][r] - write[m][n][r], y[r]);
                        q_[m][n][r] = __builtin_fmaf(diag_p[t] * steps.rk[t], k[r], q_[m][n][r]);
                        write[m][n][r] = __builtin_fmaf(diag_p[t] * (steps.rq[t] * a.d.scale), q[r], write[m][n][r]);
                        z[r] = __builtin_fmaf(q[r], q_[m][n][r], z[r]);
                        w[r] = __builtin_fmaf(k[r], read[m][n][r] + write[m][n][r], w[r]);
                        if constexpr (X::kKeep) {
                            dq[m][n][r] += q_[m][n][r];
                            dk[m][n][r] += read[m][n][r] + write[m][n][r];
                        }
                    }
                    if constexpr (!X::kKeep) {
                        f32x4 *const sums = (f32x4 *)(a.ws + a.w.sums) + (((size_t)bc * a.d.Hk + hk) * 2 * 2 * NC + (m * NC + n) * 2) * X::kThreads + again(tid);
                        read[m][n] += write[m][n];
                        if (hr) {
                            q_[m][n] += sums[0];
                            read[m][n] += sums[X::kThreads];
                        }
                        if (hr + 1 < a.rep) {
                            sums[0] = q_[m][n];
                            sums[X::kThreads] = read[m][n];
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = (m0 + m) * 16 + row4 + r;
                    x[r] = sum16(x[r]);
                    y[r] = sum16(y[r]);
                    z[r] = sum16(z[r]);
                    w[r] = sum16(w[r]);
                    if (col == 0) {
                        rows[wave][0][t] = x[r] * steps.rq[t];
                        rows[wave][1][t] = y[r] * steps.rk[t];
                        rows[wave][2][t] = z[r] * steps.rq[t];
                        rows[wave][3][t] = w[r] * steps.rk[t];
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int o = 32; o; o /= 2) ends += __shfl_xor(ends, o);
            if (lane == 0) part[wave] = ends;
            __syncthreads();
            if (wave == 0) {
                float x = 0.0f, y = 0.0f, z = 0.0f, u = 0.0f, w = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int from = (lane >> 5) * 4 + i;
                    x += rows[from][0][lane];
                    y += rows[from][1][lane];
                    z += rows[from][2][lane];
                    u += rows[from][3][lane];
                    w += part[i] + part[4 + i];
                }
                norm_q[lane] += z;
                norm_k[lane] += u;
                // sums of the decays' gradients from each step on, in 64 bits like the decays' own
                double s = (double)x * a.d.scale + y;
#pragma unroll
                for (int o = 1; o < 64; o *= 2) {
                    const double other = __shfl_down(s, o);
                    if (lane + o < 64) s += other;
                }
                if (lane < stop) {
                    const size_t at = ((size_t)B * a.d.Hv + h) * a.d.L + t0 + lane;
                    a.d.dg[at] = lane < end ? (float)(s + w) : 0.0f;
                    a.d.dbeta[at] = lane < end ? diag[lane] : 0.0f;
                }
            }
            if (hr + 1 < a.rep) continue;
            __syncthreads();
            // through the normalisation n = r x: dx = r (dn - n (n . dn))
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const int d = again(d0 + n * 16);
                if (d >= a.d.P) continue;
                T *const qrow = row_of<DT>(a.d.dq, B, hk * a.d.P + d) + t0, *const krow = row_of<DT>(a.d.dk, B, hk * a.d.P + d) + t0;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int t = (m0 + m) * 16 + row4;
                    float k[4], q[4], x[4], y[4];
                    four(a.d.k, held_k, n, m, k);
                    four(a.d.q, held_q, n, m, q);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float rq = steps.rq[t + r], rk = steps.rk[t + r];
                        float g, u;
                        if constexpr (X::kKeep) {
                            g = dq[m][n][r], u = dk[m][n][r];
                        } else {
                            g = q_[m][n][r], u = read[m][n][r];
                        }
                        if (a.d.l2norm) {
                            g -= q[r] * rq * norm_q[t + r];
                            u -= k[r] * rk * norm_k[t + r];
                        }
                        x[r] = t + r < end ? g * (rq * a.d.scale) : 0.0f;
                        y[r] = t + r < end ? u * rk : 0.0f;
                    }
                    store4_until<DT>(qrow, stop == kDeltaChunk, t, stop, x);
                    store4_until<DT>(krow, stop == kDeltaChunk, t, stop, y);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };
    if (end >= kDeltaChunk)
        chunk(Whole<true>());
    else
        chunk(Whole<false>());
}

template <int DT, int DK>
int backward(DeltaArgs a, hipStream_t st) {
    float *carry = (float *)(a.ws + a.w.state);
    a.slices = a.Vp / kDeltaSlice;
    hipLaunchKernelGGL((delta_bwd_kernel<DT, DK>), dim3((unsigned)(a.s.nb * a.d.Hv * a.slices)), dim3(512), 0, st, a,
                       carry, carry);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

template <int DT, int DK>
int gradients(DeltaArgs a, hipStream_t st) {
    return launch_groups((long long)a.s.nb * a.s.nc * a.d.Hk, Grads<DT, DK>::kThreads, [&](unsigned n, unsigned first) {
        a.more = (int)first;
        hipLaunchKernelGGL((delta_grads_kernel<DT, DK>), dim3(n), dim3(Grads<DT, DK>::kThreads), 0, st, a);
    });
}

}  // namespace

int launch_delta_bwd(const DeltaArgs &a, int dtype, hipStream_t st) {
    switch (delta_key_pad(a.d.P)) {
        case 64: return dtype == MICONV_BF16 ? backward<1, 64>(a, st) : backward<0, 64>(a, st);
        case 128: return dtype == MICONV_BF16 ? backward<1, 128>(a, st) : backward<0, 128>(a, st);
        default: return dtype == MICONV_BF16 ? backward<1, 256>(a, st) : backward<0, 256>(a, st);
    }
}

int launch_delta_grads(const DeltaArgs &a, int dtype, hipStream_t st) {
    switch (delta_key_pad(a.d.P)) {
        case 64: return dtype == MICONV_BF16 ? gradients<1, 64>(a, st) : gradients<0, 64>(a, st);
        case 128: return dtype == MICONV_BF16 ? gradients<1, 128>(a, st) : gradients<0, 128>(a, st);
        default: return dtype == MICONV_BF16 ? gradients<1, 256>(a, st) : gradients<0, 256>(a, st);
    }
}

}  // namespace miconv
