// delta_fwd.hip -- the gated delta rule from chunk to chunk, forward, and its single-token step.
#include "delta_device.h"

namespace miconv {

namespace {

// One work-group carries a value slice of 16 channels of one head through time; the state [DK][16] stays in
// accumulators, key channels of it in each of the eight waves.  A chunk is a chain of which no step can wait:
// k S, the inverse times X = v - e (k S), the state's update.  Four waves (16 steps each) go along it; the four others meanwhile compute y,
// of the chunk before while the first ones multiply k S, and q S while those multiply by the inverse.  Row operands come from memory in
// operand order, the next chunk's as soon as this one's are used; what waves exchange (planes of the state, X and u f, and u) are column
// operands in LDS, [channel][step or key channel], rows padded by 16 bytes against bank conflicts.
//
// The chain's latency bounds it: some 3900 cycles a chunk (of 3700 with a plane less of the scores, k S took 650, x to LDS 400,
// the inverse 850, u f to LDS 500, the update 700, the state to LDS 450), 119 us at best and 135 in the median for a prompt
// of 64 chunks, 32 heads of 128 and 128 channels in bf16, 256 work-groups.  Wider slices have fewer work-groups and
// chains as long, so a slice is one MFMA's 16 channels.
// One role for all waves, in turn, took 152 us.
template <int DK>
struct Scan {
    static constexpr int kKS = DK / 32, kTiles = DK / 16, kMT = kTiles > 8 ? kTiles / 8 : 1, kN = kDeltaSlice;
    static constexpr int kPitchS = DK + 8, kPitchT = kDeltaChunk + 8;   // bf16 elements
    static constexpr int kPlaneS = kN * kPitchS, kPlaneT = kN * kPitchT;
};

template <int DT, int DK, bool SAVE>
__global__ __launch_bounds__(512) void delta_fwd_kernel(DeltaArgs a, float *state_in, float *state_out) {
    constexpr int TI = in_planes(DT);
    typedef Scan<DK> X;
    typedef typename Elem<DT>::T T;
    constexpr int kPitchU = kDeltaChunk + 4;   // floats
    __shared__ __attribute__((aligned(16))) uint16_t Sp[3 * X::kPlaneS], Xp[3 * X::kPlaneT], Uf[3 * X::kPlaneT];
    __shared__ __attribute__((aligned(16))) float Us[2][X::kN * kPitchU];      // u of this chunk and the one before
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), col = lane & 15, grp = lane >> 4;
    const bool queries = wave >= 4, owner = wave * X::kMT < X::kTiles;
    const int part = wave & 3, row4 = grp * 4, mine = part * 16 + row4;     // a lane's four steps
    // the slices of a head side by side on one XCD: they share its operands in the L2
    const int total = a.s.nb * a.d.Hv * a.slices;
    const int id = xcd_remap(blockIdx.x, total);
    const int slice = id % a.slices, bh = id / a.slices, h = bh % a.d.Hv, b = bh / a.d.Hv, B = a.s.b0 + b;
    const int hk = h / a.rep, v0 = slice * X::kN;
    const int valid = valid_steps(a.d.lengths, B, a.d.L);
    const int steps_first = a.s.c0 * kDeltaChunk;
    int chunks = (valid - steps_first + kDeltaChunk - 1) / kDeltaChunk;
    chunks = chunks < 0 ? 0 : (chunks > a.s.nc ? a.s.nc : chunks);

    // the state: from the caller, from the slice of time before, or zeros
    f32x4 S[X::kMT];
    {
        const int P = a.first ? a.d.P : DK, V = a.first ? a.d.V : a.Vp;
        const float *in = a.first ? a.d.initial_state : state_in;
        const long long at = a.first ? (long long)B * a.d.Hv + h : bh;
#pragma unroll
        for (int i = 0; i < X::kMT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int p = (wave * X::kMT + i) * 16 + row4 + r, v = v0 + col;
                S[i][r] = in && p < P && v < V ? in[(at * P + p) * V + v] : 0.0f;
            }
    }
    const auto put_state = [&] {
        if (!owner) return;
#pragma unroll
        for (int i = 0; i < X::kMT; ++i) {
            const float v[4] = {S[i][0], S[i][1], S[i][2], S[i][3]};
            put_planes<3>(Sp + col * X::kPitchS + (wave * X::kMT + i) * 16 + row4, X::kPlaneS, v);
        }
    };
    put_state();
    for (int i = threadIdx.x; i < 3 * X::kN * 8; i += 512)      // the zeros behind X's steps
        Xp[i / (X::kN * 8) * X::kPlaneT + i / 8 % X::kN * X::kPitchT + kDeltaChunk + i % 8] = 0;

    const size_t of_k = ((size_t)b * a.s.nc * a.d.Hk + hk) * TI * 64 * DK * 2, step_k = (size_t)a.d.Hk * TI * 64 * DK * 2;
    const size_t of_v = (size_t)b * a.s.nc * a.d.Hv + h;
    constexpr int kPlaneK = 64 * DK * 2;
    // three planes of 128 key channels are more than the registers hold ahead of their use
    constexpr bool kLate = TI == 3 && DK >= 128;
    u32x4 fx[kLate ? 1 : X::kKS][TI];          // keys or queries
    const char *px = a.ws + (queries ? a.w.q : a.w.k) + of_k, *pi = a.ws + a.w.inv + of_v * 3 * kDeltaSquare;
    const char *pa = a.ws + a.w.attn + of_v * 3 * kDeltaSquare, *ps = a.ws + a.w.steps + of_v * sizeof(DeltaSteps);
    const T *krow[X::kMT];
#pragma unroll
    for (int i = 0; i < X::kMT; ++i) {
        const int p = (wave * X::kMT + i) * 16 + col;
        krow[i] = row_of<DT>(a.d.k, B, hk * a.d.P + (p < a.d.P ? p : 0));
    }
    Raw8<DT> ft[X::kMT][2];
    float last = 0.0f;
    const auto steps_of = [&](int c) { return (const DeltaSteps *)(ps + (size_t)c * a.d.Hv * sizeof(DeltaSteps)); };
    const auto load_x = [&](int c) {
#pragma unroll
        for (int ks = 0; ks < X::kKS && !kLate; ++ks) fragment<TI>(px + c * step_k, part * X::kKS + ks, kPlaneK, fx[ks]);
    };
    const auto load_kt = [&](int c, bool whole) {
#pragma unroll
        for (int i = 0; i < X::kMT; ++i)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                ft[i][ks] = steps8<DT>(krow[i], whole, steps_first + c * kDeltaChunk + ks * 32 + grp * 8, valid);
    };
    const auto times_state = [&](int c, f32x4 &xS) {
        Sums<2> sum;
#pragma unroll
        for (int ks = 0; ks < X::kKS; ++ks) {
            if constexpr (kLate) fragment<TI>(px + c * step_k, part * X::kKS + ks, kPlaneK, fx[0]);
            u32x4 s[3];
            get_planes<3>(Sp + col * X::kPitchS + ks * 32 + grp * 8, X::kPlaneS, s);
            sum.add(fx[kLate ? 0 : ks], s);
        }
        xS = sum.total();
    };
    float *saved = SAVE ? (float *)a.d.states + (((size_t)B * a.d.Hv + h) * a.chunks + a.s.c0) * delta_saved(a.d.P, a.d.V) : nullptr;
    const auto save_state = [&] {
        if (SAVE && owner) {
#pragma unroll
            for (int i = 0; i < X::kMT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    saved[(size_t)((wave * X::kMT + i) * 16 + row4 + r) * a.Vp + v0 + col] = S[i][r];
        }
    };
    const auto update = [&] {
        if (!owner) return;
#pragma unroll
        for (int i = 0; i < X::kMT; ++i) {
            u32x4 k0[TI], k1[TI];
            const bool in = (wave * X::kMT + i) * 16 + col < a.d.P;
            planes_of<DT>(only<DT>(ft[i][0], in), k0);
            planes_of<DT>(only<DT>(ft[i][1], in), k1);
            Sums<2> sum;
            u32x4 u[3];
            const uint16_t *from = Uf + col * X::kPitchT + grp * 8;
            get_planes<3>(from, X::kPlaneT, u);
            sum.add(k0, u);
            get_planes<3>(from + 32, X::kPlaneT, u);
            sum.add(k1, u);
            S[i] = S[i] * last + sum.total();
        }
        put_state();
    };

    // Chunks of 64 valid steps, and the one that ends inside, if any, whose loads look at each step.  Both kinds of waves have a loop of
    // their own, and a chunk's loads for the next one (after the last, for itself again) depend on no branch: where two
    // ways meet, what they loaded is moved, and waited for.
    int full = (valid - steps_first) / kDeltaChunk;
    full = valid <= steps_first ? 0 : (full < chunks ? full : chunks);
    const bool upper = part >= 2;              // the second 32 columns of rows 0..31 of the inverse and of attn are not stored
    if (chunks) {
        load_x(0);
        if (full) load_kt(0, true);
        last = steps_of(0)->last;
    }
    if (!chunks) {
    } else if (!queries) {
        u32x4 fi[2][3];
        Raw4<DT> vin;
        const T *const vrow = row_of<DT>(a.d.v, B, h * a.d.V + (v0 + col < a.d.V ? v0 + col : 0));
        const auto load_inverse = [&](int c) {
            const char *at = pi + (size_t)c * a.d.Hv * 3 * kDeltaSquare;
            fragment<3>(at, part * 2, kDeltaSquare, fi[0]);
            fragment<3>(at, part * 2 + upper, kDeltaSquare, fi[1]);
        };
        const auto load_v = [&](int c, bool whole) {
            vin = steps4<DT>(vrow, whole, steps_first + c * kDeltaChunk + mine, valid);
        };
        load_inverse(0);
        f32x4 vek = *(const f32x4 *)(steps_of(0)->ek + mine), vfk = *(const f32x4 *)(steps_of(0)->fk + mine);
        f32x4 vbeta = *(const f32x4 *)(steps_of(0)->beta + mine);
        if (full) load_v(0, true);
        // rows 0..31 meet the second fragment with the zeros behind each channel's 64 steps
        const int second = upper ? 32 : kDeltaChunk - grp * 8;
        const auto chunk = [&](const int c, auto is_full) {
            constexpr bool FULL = decltype(is_full)::value;
            const int next = c + 1 < chunks ? c + 1 : c, next_full = c + 1 < full ? c + 1 : c;
            if constexpr (!FULL) {
                load_v(c, false);
                load_kt(c, false);
            }
            save_state();
            __syncthreads();
            f32x4 kS;
            times_state(c, kS);
            load_x(next);
            float x[4];
            widen4<DT>(vin, v0 + col < a.d.V, x);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(-vek[r], kS[r], x[r]);
            put_planes<3>(Xp + col * X::kPitchT + mine, X::kPlaneT, x);
            vek = *(const f32x4 *)(steps_of(next)->ek + mine);
            if constexpr (FULL) load_v(next_full, true);
            __syncthreads();
            Sums<2> sum;
            u32x4 planes[3];
            const uint16_t *from = Xp + col * X::kPitchT + grp * 8;
            get_planes<3>(from, X::kPlaneT, planes);
            sum.add(fi[0], planes);
            get_planes<3>(from + second, X::kPlaneT, planes);
            sum.add(fi[1], planes);
            const f32x4 z = sum.total(), u = z * vbeta;
            float uf[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) uf[r] = u[r] * vfk[r];
            put_planes<3>(Uf + col * X::kPitchT + mine, X::kPlaneT, uf);
            *(f32x4 *)(Us[c & 1] + col * kPitchU + mine) = u;
            if constexpr (SAVE)
                *(f32x4 *)(saved + (size_t)DK * a.Vp + (size_t)(v0 + col) * kDeltaChunk + mine) = z;
            load_inverse(next);
            vfk = *(const f32x4 *)(steps_of(next)->fk + mine);
            vbeta = *(const f32x4 *)(steps_of(next)->beta + mine);
            __syncthreads();
            update();
            last = steps_of(next)->last;
            if constexpr (FULL) load_kt(next_full, true);
            if constexpr (SAVE) saved += delta_saved(a.d.P, a.d.V);
        };
        for (int c = 0; c < full; ++c) chunk(c, Whole<true>());
        if (full < chunks) chunk(full, Whole<false>());
    } else {
        u32x4 fa[2][3];
        f32x4 veq = {0, 0, 0, 0}, qS = {0, 0, 0, 0};
        T *const yrow = row_of<DT>(a.d.y, B, h * a.d.V + (v0 + col < a.d.V ? v0 + col : 0));
        const auto load_attn = [&](int c) {
            const char *at = pa + (size_t)c * a.d.Hv * 3 * kDeltaSquare;
            fragment<3>(at, part * 2, kDeltaSquare, fa[0]);
            fragment<3>(at, part * 2 + upper, kDeltaSquare, fa[1]);
            veq = *(const f32x4 *)(steps_of(c)->eq + mine);
        };
        // y of chunk c, whose u is in Us[c & 1]
        const auto make_y = [&](const int c, float (&y)[4]) {
            Sums<2> o;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const f32x4 *from = (const f32x4 *)(Us[c & 1] + col * kPitchU + ks * 32 + grp * 8);
                const f32x4 lo = from[0], hi = from[1];
                float u[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = ks == 0 || upper ? u[e] : 0.0f;
                u32x4 planes[3];
                split8<3>(u, planes);
                o.add(fa[ks], planes);
            }
            const f32x4 p = o.total();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[r] = __builtin_fmaf(veq[r], qS[r], p[r]);
                asm volatile("" : "+v"(y[r]));
            }
        };
        const auto put_y = [&](const int c, auto is_full, float (&y)[4]) {
            constexpr bool FULL = decltype(is_full)::value;
            const int t = steps_first + c * kDeltaChunk + mine;
            if (v0 + col < a.d.V) {
                // past the sequence's end: zeros, up to the end of the rows
                if constexpr (!FULL) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = t + r < valid ? y[r] : 0.0f;
                }
                store4_until<DT>(yrow, FULL, t, a.d.L, y);
            }
        };
        const auto finish = [&](const int c, auto is_full) {
            float y[4];
            make_y(c, y);
            put_y(c, is_full, y);
        };
        const auto chunk = [&](const int c, auto is_full, auto is_first) {
            constexpr bool FULL = decltype(is_full)::value, FIRST = decltype(is_first)::value;
            const int next = c + 1 < chunks ? c + 1 : c, next_full = c + 1 < full ? c + 1 : c;
            if constexpr (!FULL) load_kt(c, false);
            save_state();
            __syncthreads();
            // the waves of the state are ahead till their x stands, and behind after it: y is stored then
            float y[4];
            if constexpr (!FIRST) make_y(c - 1, y);
            __syncthreads();
            load_attn(c);
            if constexpr (!FIRST) put_y(c - 1, Whole<true>(), y);
            times_state(c, qS);
            load_x(next);
            __syncthreads();
            update();
            last = steps_of(next)->last;
            if constexpr (FULL) load_kt(next_full, true);
            if constexpr (SAVE) saved += delta_saved(a.d.P, a.d.V);
        };
        if (full) {
            chunk(0, Whole<true>(), Whole<true>());
            for (int c = 1; c < full; ++c) chunk(c, Whole<true>(), Whole<false>());
            if (full < chunks) {
                chunk(full, Whole<false>(), Whole<false>());
                finish(full, Whole<false>());
            } else {
                finish(full - 1, Whole<true>());
            }
        } else {
            chunk(0, Whole<false>(), Whole<true>());
            finish(0, Whole<false>());
        }
    }
    // chunks past the sequence's end
    for (int c = chunks; queries && c < a.s.nc; ++c) {
        const float zeros[4] = {};
        if (v0 + col < a.d.V)
            store4_until<DT>(row_of<DT>(a.d.y, B, h * a.d.V + v0 + col), steps_first + (c + 1) * kDeltaChunk <= a.d.L,
                             steps_first + c * kDeltaChunk + mine, a.d.L, zeros);
    }
    float *out = a.last ? a.d.final_state : state_out;
    if (out && owner) {
        const int P = a.last ? a.d.P : DK, V = a.last ? a.d.V : a.Vp;
        const long long at = a.last ? (long long)B * a.d.Hv + h : bh;
#pragma unroll
        for (int i = 0; i < X::kMT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int p = (wave * X::kMT + i) * 16 + row4 + r, v = v0 + col;
                if (p < P && v < V) out[(at * P + p) * V + v] = S[i][r];
            }
    }
}

template <int DT, int DK>
int forward(DeltaArgs a, hipStream_t st) {
    float *carry = (float *)(a.ws + a.w.state);
    a.slices = a.Vp / kDeltaSlice;
    const unsigned groups = (unsigned)(a.s.nb * a.d.Hv * a.slices);
    if (a.d.states)
        hipLaunchKernelGGL((delta_fwd_kernel<DT, DK, true>), dim3(groups), dim3(512), 0, st, a, carry, carry);
    else
        hipLaunchKernelGGL((delta_fwd_kernel<DT, DK, false>), dim3(groups), dim3(512), 0, st, a, carry, carry);
    return hipGetLastError() == hipSuccess ? MICONV_OK : MICONV_ERR_HIP;
}

template <int DT>
int forward_by_width(const DeltaArgs &a, hipStream_t st) {
    switch (delta_key_pad(a.d.P)) {
        case 64: return forward<DT, 64>(a, st);
        case 128: return forward<DT, 128>(a, st);
        default: return forward<DT, 256>(a, st);
    }
}

// ------------------------------------------------------------------ one token
//
// The state's bytes: read once, held in registers between the two products with it, written once.  A work-group
// takes 64 value channels of one head; a thread four neighbouring channels of every 16th key channel.  64 sequences of
// 32 heads of 128 and 128 channels: 49 us, 268 MB at 5.5 TB/s (the rate of a large copy is 4.95); one of 8 heads of 64
// and 64: 4.6 us, a launch.
template <int DT, int DK>
__global__ __launch_bounds__(256) void delta_step_kernel(miconv_gated_delta_t d, const float *state, int slots,
                                                         const int *slot_of, float *state_out, int tiles, int first) {
    constexpr int kRows = DK / 16;
    typedef typename Elem<DT>::T T;
    __shared__ float ks[DK], qs[DK], sums[4][2];
    __shared__ __attribute__((aligned(16))) float red[4][kDeltaStepValues];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int id = first + blockIdx.x, tile = id % tiles, bh = id / tiles, h = bh % d.Hv, b = bh / d.Hv;
    const int hk = h / (d.Hv / d.Hk), v = tile * kDeltaStepValues + (tid & 15) * 4, p0 = tid >> 4;
    const int slot = slot_of ? slot_of[b] : b;
    const bool unused = slot < 0 || slot >= slots;
    T *const y = row_of<DT>(d.y, b, 0) + ((long long)h * d.V) * d.y.stride_d;
    if (unused) {
        if (tid < 16) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (v + e < d.V) y[(long long)(v + e) * d.y.stride_d] = Elem<DT>::put(0.0f);
        }
        return;
    }
    const long long head = ((long long)slot * d.Hv + h) * d.P * d.V;
    float S[kRows][4];
    const bool whole = v + 4 <= d.V && d.V % 4 == 0 && (uintptr_t)state % 16 == 0 && (uintptr_t)state_out % 16 == 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int p = i * 16 + p0;
        const float *from = state + head + (long long)p * d.V + v;
        if (p < d.P && whole) {
            const f32x4 s = __builtin_nontemporal_load((const f32x4 *)from);
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][e] = s[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][e] = p < d.P && v + e < d.V ? from[e] : 0.0f;
        }
    }
    {
        float k = 0.0f, q = 0.0f;
        if (tid < d.P) {
            k = Elem<DT>::get(*row_of<DT>(d.k, b, hk * d.P + tid));
            q = Elem<DT>::get(*row_of<DT>(d.q, b, hk * d.P + tid));
        }
        if (d.l2norm) {
            float kk = k * k, qq = q * q;
#pragma unroll
            for (int o = 32; o; o /= 2) {
                kk += __shfl_xor(kk, o);
                qq += __shfl_xor(qq, o);
            }
            if (lane == 0) {
                sums[wave][0] = kk;
                sums[wave][1] = qq;
            }
            __syncthreads();
            kk = sums[0][0] + sums[1][0] + sums[2][0] + sums[3][0];
            qq = sums[0][1] + sums[1][1] + sums[2][1] + sums[3][1];
            k *= 1.0f / __builtin_sqrtf(kk + MICONV_DELTA_NORM_EPS);
            q *= 1.0f / __builtin_sqrtf(qq + MICONV_DELTA_NORM_EPS);
        }
        if (tid < DK) {
            ks[tid] = k;
            qs[tid] = q * d.scale;
        }
    }
    const float g = ((const float *)d.g.data)[(long long)b * d.g.stride_b + (long long)h * d.g.stride_d];
    const float beta = ((const float *)d.beta.data)[(long long)b * d.beta.stride_b + (long long)h * d.beta.stride_d];
    const float decay = exp_any(g);
    float vin[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        vin[e] = v + e < d.V ? Elem<DT>::get(*row_of<DT>(d.v, b, h * d.V + v + e)) : 0.0f;
    __syncthreads();
    // a sum over the key channels: over the thread's rows, its wave's four row groups, the waves
    const auto total = [&](float (&s)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] += __shfl_xor(s[e], 16);
            s[e] += __shfl_xor(s[e], 32);
        }
        if (lane < 16) *(f32x4 *)&red[wave][lane * 4] = f32x4{s[0], s[1], s[2], s[3]};
        __syncthreads();
        f32x4 r = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w) r += *(const f32x4 *)&red[w][(tid & 15) * 4];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = r[e];
    };
    float u[4] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float k = ks[i * 16 + p0];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] *= decay;
            u[e] = __builtin_fmaf(k, S[i][e], u[e]);
        }
    }
    total(u);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = beta * (vin[e] - u[e]);
    float o[4] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int p = i * 16 + p0;
        const float k = ks[p], q = qs[p];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] = __builtin_fmaf(k, u[e], S[i][e]);
            o[e] = __builtin_fmaf(q, S[i][e], o[e]);
        }
        float *to = state_out + head + (long long)p * d.V + v;
        if (p < d.P && whole) {
            __builtin_nontemporal_store(f32x4{S[i][0], S[i][1], S[i][2], S[i][3]}, (f32x4 *)to);
        } else if (p < d.P) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (v + e < d.V) to[e] = S[i][e];
        }
    }
    total(o);
    if (tid < 16) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (v + e < d.V) y[(long long)(v + e) * d.y.stride_d] = Elem<DT>::put(o[e]);
    }
}

template <int DT>
int step(const miconv_gated_delta_t &d, const float *state, int slots, const int *slot_of, float *state_out,
         hipStream_t st) {
    const int tiles = (d.V + kDeltaStepValues - 1) / kDeltaStepValues;
    return launch_groups((long long)d.B * d.Hv * tiles, 256, [&](unsigned n, unsigned first) {
        switch (delta_key_pad(d.P)) {
            case 64:
                hipLaunchKernelGGL((delta_step_kernel<DT, 64>), dim3(n), dim3(256), 0, st, d, state, slots, slot_of,
                                   state_out, tiles, (int)first);
                break;
            case 128:
                hipLaunchKernelGGL((delta_step_kernel<DT, 128>), dim3(n), dim3(256), 0, st, d, state, slots, slot_of,
                                   state_out, tiles, (int)first);
                break;
            default:
                hipLaunchKernelGGL((delta_step_kernel<DT, 256>), dim3(n), dim3(256), 0, st, d, state, slots, slot_of,
                                   state_out, tiles, (int)first);
        }
    });
}

}  // namespace

int launch_delta_fwd(const DeltaArgs &a, int dtype, hipStream_t st) {
    return dtype == MICONV_BF16 ? forward_by_width<1>(a, st) : forward_by_width<0>(a, st);
}

int launch_delta_step(const miconv_gated_delta_t &d, int dtype, const float *state, int slots, const int *slot_of,
                      float *state_out, hipStream_t st) {
    return dtype == MICONV_BF16 ? step<1>(d, state, slots, slot_of, state_out, st)
                                : step<0>(d, state, slots, slot_of, state_out, st);
}

}  // namespace miconv
