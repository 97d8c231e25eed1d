// delta_prepare.hip -- the gated delta rule's pass over single chunks: everything of a chunk that does not wait for
// the state before it.  Normalised products of queries and keys, the inverse of the chunk's triangular system, and
// the operands in the order in which the scan's MFMAs take them, so that the scan reads them without LDS.
//
// One work-group of four waves per (sequence, chunk, value head), three on a CU in bf16.  Latency bounds it: barriers between
// the products, the substitution of 16 dependent rows and the inverse's blocks down each column, 12 us for a single
// chunk.  2048 of them (a prompt of 4096 steps, 32 value heads on 16 key heads of 128 channels, bf16): 50 us.
#include "delta_device.h"

namespace miconv {

namespace {

// LDS matrices of 64 x 64 fp32 have rows of 68: 16-byte aligned, and 16 rows of a column block on different banks.
constexpr int kRow = 68;

template <int TI, int DK>
struct Prepare {
    static constexpr int kCols = DK < 128 ? DK : 128;      // channels at a time
    static constexpr int kSteps = kCols / 32;
    static constexpr int kPlane = 64 * kCols * 2;          // bytes of one plane in LDS
    static constexpr int kFrags = 2 * TI * kPlane;
    static constexpr int kSolve = 64 * kRow * 4 + 4 * 16 * 20 * 4;
    static constexpr int kShared = kFrags > kSolve ? kFrags : kSolve;
};

template <int DT, int DK, bool BWD>
__global__ __launch_bounds__(256) void delta_prepare_kernel(DeltaArgs a) {
    constexpr int TI = in_planes(DT);
    typedef Prepare<TI, DK> X;
    __shared__ __attribute__((aligned(16))) char shared[X::kShared];
    __shared__ __attribute__((aligned(16))) float A[64 * kRow];
    float (*const part)[X::kCols / 8][64] = (float (*)[X::kCols / 8][64])A;     // before A: sums of squares
    __shared__ __attribute__((aligned(16))) DeltaSteps steps;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int id = a.more + blockIdx.x;
    const int h = id % a.d.Hv, bc = id / a.d.Hv, c = bc % a.s.nc, b = bc / a.s.nc;
    const int hk = h / a.rep, B = a.s.b0 + b, t0 = (a.s.c0 + c) * kDeltaChunk;
    const int end = valid_steps(a.d.lengths, B, a.d.L) - t0;      // valid steps of this chunk, or less than 1
    if (end <= 0) return;
    const bool leads = h == hk * a.rep;                           // writes the operands that heads share
    const size_t of_k = ((size_t)bc * a.d.Hk + hk) * TI * 64 * DK * 2, of_v = (size_t)bc * a.d.Hv + h;

    // the decays' loads and those of the first operands are in flight together
    const int own = lane < end ? lane : 0;
    const float decay = ((const float *)a.d.g.data + (long long)B * a.d.g.stride_b + (long long)h * a.d.g.stride_d + t0)[own];
    const float size = ((const float *)a.d.beta.data + (long long)B * a.d.beta.stride_b +
                        (long long)h * a.d.beta.stride_d + t0)[own];
    const auto decays = [&] {
        // sums of log decays in 64 bits: their differences are the exponents between near steps, however far
        // the sums have gone.  A decay of exp(-200) is 0 in fp32, so that also stands for less, minus infinity included.
        if (wave == 0) {
            double G = lane >= end ? 0.0 : decay < -200.0f ? -200.0 : (double)decay;
#pragma unroll
            for (int o = 1; o < 64; o *= 2) {
                const double other = __shfl_up(G, o);
                if (lane >= o) G += other;
            }
            const double last = __shfl(G, 63);
            steps.G[lane] = G;
            steps.ek[lane] = exp_any((float)G);                      // the keys' factors are applied below
            steps.fk[lane] = exp_any((float)(last - G));
            steps.beta[lane] = lane < end ? size : 0.0f;
            if (lane == 0) steps.last = exp_any((float)last);
        }
    };
    // operands, in blocks of 8 steps x 8 channels per thread: keys first, then queries
    constexpr int kBlocks = X::kCols;                             // per operand: 8 x kCols / 8
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) kk[n] = qk[n] = f32x4{0, 0, 0, 0};
    float squares[8] = {};
    for (int d0 = 0; d0 < DK; d0 += X::kCols) {
        if (d0) __syncthreads();                                  // the products of the columns before are done
        const int operand = tid / kBlocks, in = tid % kBlocks;
        const auto block = [&](auto is_whole) {
            constexpr bool whole = decltype(is_whole)::value;
            const int tb = (in & 7) * 8, db = (in >> 3) * 8;
            const miconv_rows_t &rows = operand ? a.d.q : a.d.k;
            float x[8][8];
            Raw8<DT> raw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int d = d0 + db + i;
                raw[i] = steps8<DT>(row_of<DT>(rows, B, hk * a.d.P + (d < a.d.P ? d : 0)) + t0, whole, tb, end);
            }
            if (d0 == 0) decays();                                // while they are in flight
#pragma unroll
            for (int i = 0; i < 8; ++i) widen8<DT>(only<DT>(raw[i], d0 + db + i < a.d.P), x[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) squares[j] = __builtin_fmaf(x[i][j], x[i][j], squares[j]);
            // [t][p]: to LDS, and k (forward: q too) to memory
            const bool rows_out = leads && (!operand || !BWD);
            char *const flat = a.ws + (operand ? a.w.q : a.w.k) + of_k;
#pragma unroll
            for (int p = 0; p < TI; ++p) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const u32x4 v = {take_plane<TI>(p, x[0][j], x[1][j]), take_plane<TI>(p, x[2][j], x[3][j]),
                                     take_plane<TI>(p, x[4][j], x[5][j]), take_plane<TI>(p, x[6][j], x[7][j])};
                    const int t = tb + j, lane_at = (t & 15) + (db >> 3 & 3) * 16;
                    *(u32x4 *)(shared + (operand * TI + p) * X::kPlane + ((t >> 4) * X::kSteps + (db >> 5)) * 1024 +
                               lane_at * 16) = v;
                    if (rows_out)
                        *(u32x4 *)(flat + (size_t)p * 64 * DK * 2 + ((t >> 4) * (DK / 32) + ((d0 + db) >> 5)) * 1024 +
                                   lane_at * 16) = v;
                }
            }
        };
        if (operand < 2) {
            if (end >= kDeltaChunk)
                block(Whole<true>());
            else
                block(Whole<false>());
        }
        __syncthreads();
        // k k^T and q k^T: the wave's 16 rows, column tiles up to the diagonal
#pragma unroll
        for (int ks = 0; ks < X::kSteps; ++ks) {
            u32x4 rk[TI], rq[TI];
            fragment<TI>(shared, wave * X::kSteps + ks, X::kPlane, rk);
            fragment<TI>(shared + TI * X::kPlane, wave * X::kSteps + ks, X::kPlane, rq);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (n > wave) break;
                u32x4 col[TI];
                fragment<TI>(shared, n * X::kSteps + ks, X::kPlane, col);
                multiply<TI, TI, 2>(rk, col, kk[n]);
                // q k^T with four neighbouring keys to a lane (backward: queries), as attn is stored
                if constexpr (BWD)
                    multiply<TI, TI, 2>(rq, col, qk[n]);
                else
                    multiply<TI, TI, 2>(col, rq, qk[n]);
            }
        }
    }
    settle(kk, qk);
    {
        const int operand = tid / kBlocks, in = tid % kBlocks;
        if (operand < 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) part[operand][in >> 3][(in & 7) * 8 + j] = squares[j];
        }
    }
    __syncthreads();
    if (wave < 2) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < X::kCols / 8; ++i) s += part[wave][i][lane];
        const float r = a.d.l2norm ? 1.0f / __builtin_sqrtf(s + MICONV_DELTA_NORM_EPS) : 1.0f;
        (wave ? steps.rq : steps.rk)[lane] = r;
    }
    __syncthreads();
    if (wave == 0) {
        steps.eq[lane] = steps.ek[lane] * (steps.rq[lane] * a.d.scale);
        steps.ek[lane] *= steps.rk[lane];
        steps.fk[lane] *= steps.rk[lane];
    }
    // The system's matrix (its diagonal of ones left out), and the products of queries with keys, which go to memory
    // from here.  A block of 32 columns past the diagonal is never read.
    const int col = lane & 15, row4 = (lane >> 4) * 4;
    char *const inv = a.ws + a.w.inv + of_v * 3 * kDeltaSquare, *const attn = a.ws + a.w.attn + of_v * 3 * kDeltaSquare;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        if (n > (wave | 1)) break;
        const int j = n * 16 + col;
        const double Gj = steps.G[j];
        const float rkj = steps.rk[j], bj = steps.beta[j];
        float m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = wave * 16 + row4 + r;
            const float D = i > j ? exp_any((float)(steps.G[i] - Gj)) : 0.0f;
            A[i * kRow + j] = i > j ? kk[n][r] * (steps.rk[i] * rkj) * D * (BWD ? steps.beta[i] : bj) : 0.0f;
            if constexpr (BWD) m[r] = i >= j ? qk[n][r] * (steps.rq[i] * a.d.scale * rkj) * (i == j ? 1.0f : D) : 0.0f;
        }
        if constexpr (!BWD) {
            const int i = wave * 16 + col;
            const double Gi = steps.G[i];
            const float ri = steps.rq[i] * a.d.scale;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = n * 16 + row4 + r;
                m[r] = i >= key ? qk[n][r] * (ri * steps.rk[key]) * exp_any((float)(Gi - steps.G[key])) : 0.0f;
            }
        }
        // row tile, block of 32 columns, and the half of it, of the four values
        const int tile = BWD ? n : wave, block = (BWD ? wave : n) >> 1, eight = ((BWD ? wave : n) & 1) * 2 + (lane >> 5);
        put_planes<3>((uint16_t *)(attn + (tile * 2 + block) * 1024 + (col + eight * 16) * 16 + (lane >> 4 & 1) * 8),
                      kDeltaSquare / 2, m);
    }
    __syncthreads();

    // The inverse of I + A: the diagonal blocks of 16 by substitution, a lane per column; then
    // T_ij = -T_ii sum_{j <= m < i} A_im T_mj down each block column, a wave per column, on fp32 MFMAs: a lane's
    // four accumulators are rows 4 (lane / 16) + r, so with k taken in that order they are the next
    // product's column operand as they stand.
    float *const Tm = (float *)shared, *const Dm = Tm + 64 * kRow;    // Dm: [block][row][20]
    {
        float x[16];
        const float *blk = A + wave * 16 * kRow + wave * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == col ? 1.0f : 0.0f;
#pragma unroll
            for (int m4 = 0; m4 < i; m4 += 4) {
                const f32x4 v = *(const f32x4 *)(blk + i * kRow + m4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m4 + e < i) s = __builtin_fmaf(-v[e], x[m4 + e], s);
            }
            x[i] = s;
        }
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) Dm[(wave * 16 + i) * 20 + col] = x[i];
        }
    }
    __syncthreads();
    {
        f32x4 Tc[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) Tc[0][r] = Dm[(wave * 16 + row4 + r) * 20 + col];
#pragma unroll
        for (int di = 1; di < 4; ++di) {
            Tc[di] = f32x4{0, 0, 0, 0};
            if (wave + di < 4) {
                const int i = wave + di;
                f32x4 y = {0, 0, 0, 0};
#pragma unroll
                for (int dm = 0; dm < di; ++dm) {
                    const f32x4 left = *(const f32x4 *)(A + (i * 16 + col) * kRow + (wave + dm) * 16 + row4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y = __builtin_amdgcn_mfma_f32_16x16x4f32(left[r], Tc[dm][r], y, 0, 0, 0);
                }
                const f32x4 left = *(const f32x4 *)(Dm + (i * 16 + col) * 20 + row4);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    Tc[di] = __builtin_amdgcn_mfma_f32_16x16x4f32(-left[r], y[r], Tc[di], 0, 0, 0);
                settle(Tc[di]);
            }
        }
        // block column `wave` of the inverse, zeros above the diagonal; transposed for the backward pass
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 v = {0, 0, 0, 0};
#pragma unroll
            for (int di = 0; di < 4; ++di)
                if (wave + di == i) v = Tc[di];
            if constexpr (BWD) {
                *(f32x4 *)(Tm + (wave * 16 + col) * kRow + i * 16 + row4) = v;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) Tm[(i * 16 + row4 + r) * kRow + wave * 16 + col] = v[r];
            }
        }
    }
    __syncthreads();
    // Out in operand order, without the quarter that is zero: columns 32.. of rows 0..31 (forward), columns 0..31 of
    // rows 32.. (backward).
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int f = half * 4 + wave, tile = f >> 1, ks = f & 1;
        if (BWD ? (tile >= 2 && ks == 0) : (tile < 2 && ks == 1)) continue;
        const float *from = Tm + (tile * 16 + col) * kRow + ks * 32 + (lane >> 4) * 8;
        const f32x4 lo = *(const f32x4 *)from, hi = *(const f32x4 *)(from + 4);
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        u32x4 planes[3];
        split8<3>(v, planes);
#pragma unroll
        for (int p = 0; p < 3; ++p) *(u32x4 *)(inv + p * kDeltaSquare + f * 1024 + lane * 16) = planes[p];
    }
    if (tid < (int)(sizeof(DeltaSteps) / 16))
        ((u32x4 *)(a.ws + a.w.steps + of_v * sizeof(DeltaSteps)))[tid] = ((const u32x4 *)&steps)[tid];
}

template <int DT, bool BWD>
int by_width(DeltaArgs a, hipStream_t st) {
    const long long groups = (long long)a.s.nb * a.s.nc * a.d.Hv;
    return launch_groups(groups, 256, [&](unsigned n, unsigned first) {
        a.more = (int)first;
        switch (delta_key_pad(a.d.P)) {
            case 64: hipLaunchKernelGGL((delta_prepare_kernel<DT, 64, BWD>), dim3(n), dim3(256), 0, st, a); break;
            case 128: hipLaunchKernelGGL((delta_prepare_kernel<DT, 128, BWD>), dim3(n), dim3(256), 0, st, a); break;
            default: hipLaunchKernelGGL((delta_prepare_kernel<DT, 256, BWD>), dim3(n), dim3(256), 0, st, a);
        }
    });
}

}  // namespace

int launch_delta_prepare(const DeltaArgs &a, int dtype, bool backward, hipStream_t st) {
    if (dtype == MICONV_BF16) return backward ? by_width<1, true>(a, st) : by_width<1, false>(a, st);
    return backward ? by_width<0, true>(a, st) : by_width<0, false>(a, st);
}

}  // namespace miconv
