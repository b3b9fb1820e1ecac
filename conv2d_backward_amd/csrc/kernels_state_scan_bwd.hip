// kernels_state_scan_bwd.hip -- the gradients of the selective state space scan.
//
// Two chains a state: h forwards (run again from the checkpoint before the
// chunk) and its gradient q backwards, q_t = C_t gy_t + a_{t+1} q_{t+1}; both go
// over a chunk with the lane scan of kernels_state_scan.hip and share its
// exponentials.  dB and dC sum over channels: 4 channels meet in a wave through
// lane swaps, 8 waves through LDS, and the work-groups of a group through the
// workspace, in a fixed order.
//
// A work-group walks its chunks from the last to the first.  Where there are
// too few (batch, channel tile) pairs to fill the chip, the positions are cut
// into segments: scan_tail finds what each segment sends back on its own,
// scan_carry chains those, and the segments then run side by side.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

constexpr int LANES = 16, T = 8, CHUNK = LANES * T, RPW = 64 / LANES;
static_assert(CHUNK == SEQ_SCAN_CHECKPOINT, "a chunk starts at every checkpoint");
constexpr int kWaves = 8, kThreads = 64 * kWaves, CH = kWaves * RPW;
constexpr int kNB = 16;  // states whose B and C are in LDS at once
constexpr int kNR = 4;   // states summed over waves at once
constexpr int kTailWaves = 4, kTailThreads = 64 * kTailWaves, kTailCH = kTailWaves * RPW;

struct Plan {
    int tiles, chunks, segments, pitch;  // pitch: padded positions of a partial row
    int64_t sums, params, tails, steps;  // workspace offsets, in floats
    int64_t floats;
};

Plan make_plan(int64_t B, int64_t D, int64_t L, int64_t N, int64_t G) {
    Plan p;
    p.tiles = (int)((D / G + CH - 1) / CH);
    p.chunks = (int)((L + CHUNK - 1) / CHUNK);
    p.pitch = p.chunks * CHUNK;
    const int64_t groups = B * G * p.tiles;
    p.segments = groups >= 256 ? 1 : (int)std::min<int64_t>(p.chunks, (512 + groups - 1) / groups);
    p.sums = 0;
    p.params = p.sums + p.tiles * 2 * B * G * N * (int64_t)p.pitch;
    p.tails = p.params + B * p.segments * D * (N + 2);
    p.steps = p.tails + (p.segments > 1 ? B * p.segments * D * N : 0);
    p.floats = p.steps + (p.segments > 1 ? B * p.segments * D : 0);
    return p;
}

template <class E>
struct ScanBwd {
    View<E> gout, x, dt, z, Bm, Cm, dx, ddt, dz;
    const float *A, *skip, *dt_bias, *checkpoints, *gstate;
    float *dstate;
    const int32_t *lengths;
    float *ws;
    int B, D, L, N, G;
    int softplus;
    Plan p;
};

// Steps of a lane's positions; 0 beyond the length, where the state passes unchanged.
template <class E>
__device__ __forceinline__ void load_steps(const typename E::type *dt, int t0, int len, float bias,
                                           bool soft, float (&s)[T]) {
    load_row<E, T>(dt, t0, len, s);
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const float raw = s[i] + bias;
        s[i] = t0 + i < len ? (soft ? softplus(raw) : raw) : 0.f;
    }
}

// Chains (P, Q) from the right: lane l's result is what reaches the state before
// its first position, `carry` what comes from behind lane 15.
__device__ __forceinline__ float scan_back(float P, float Q, float carry, int lane) {
    float v = __builtin_fmaf(P, lane == LANES - 1 ? carry : 0.f, Q);
    v = __builtin_fmaf(P, dpp0<kRowShl + 1>(v), v);
    P *= dpp0<kRowShl + 1>(P);
    v = __builtin_fmaf(P, dpp0<kRowShl + 2>(v), v);
    P *= dpp0<kRowShl + 2>(P);
    v = __builtin_fmaf(P, dpp0<kRowShl + 4>(v), v);
    P *= dpp0<kRowShl + 4>(P);
    return __builtin_fmaf(P, dpp0<kRowShl + 8>(v), v);
}

__device__ __forceinline__ float scan_forth(float P, float Q, float carry, int lane) {
    float v = __builtin_fmaf(P, lane == 0 ? carry : 0.f, Q);
    v = __builtin_fmaf(P, dpp0<kRowShr + 1>(v), v);
    P *= dpp0<kRowShr + 1>(P);
    v = __builtin_fmaf(P, dpp0<kRowShr + 2>(v), v);
    P *= dpp0<kRowShr + 2>(P);
    v = __builtin_fmaf(P, dpp0<kRowShr + 4>(v), v);
    P *= dpp0<kRowShr + 4>(P);
    return __builtin_fmaf(P, dpp0<kRowShr + 8>(v), v);
}

// Sum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float row_sum(float v) {
    v += dpp0<kRowRor + 8>(v);
    v += dpp0<kRowRor + 4>(v);
    v += dpp0<kRowRor + 2>(v);
    return v + dpp0<kRowRor + 1>(v);
}

// lo of the lower half wave + hi-half counterpart, for two values at once:
// lanes 0..31 get x summed over the halves, lanes 32..63 y.
__device__ __forceinline__ float meet32(float x, float y) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x),
                                                    __builtin_bit_cast(unsigned, y), false, false);
    const unsigned p = r[0], q = r[1];
    return __builtin_bit_cast(float, p) + __builtin_bit_cast(float, q);
}
// The same between the 16-lane rows of each half: even rows get x, odd rows y.
__device__ __forceinline__ float meet16(float x, float y) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x),
                                                    __builtin_bit_cast(unsigned, y), false, false);
    const unsigned p = r[0], q = r[1];
    return __builtin_bit_cast(float, p) + __builtin_bit_cast(float, q);
}

// Stages B or C of nb states from position c0, in the order the lanes read them.
template <class E>
__device__ __forceinline__ void stage(const View<E> &m, int64_t b, int64_t first, int nb, int c0,
                                      int len, float *to, int tid, int threads) {
    for (int i = tid; i < nb * (CHUNK / 4); i += threads) {
        const int n = i / (CHUNK / 4), q = i % (CHUNK / 4);
        float v[4];
        load_row<E, 4>(m.row(b, first + n), c0 + 4 * q, len, v);
        *reinterpret_cast<float4 *>(to + n * CHUNK + (q % (T / 4) * LANES + q / (T / 4)) * 4) =
            float4{v[0], v[1], v[2], v[3]};
    }
}

__device__ __forceinline__ void fetch(const float *from, int n, int lane, float (&v)[T]) {
#pragma unroll
    for (int j = 0; j < T / 4; ++j) {
        const float4 f =
            *reinterpret_cast<const float4 *>(from + n * CHUNK + (j * LANES + lane) * 4);
        v[4 * j] = f.x;
        v[4 * j + 1] = f.y;
        v[4 * j + 2] = f.z;
        v[4 * j + 3] = f.w;
    }
}

template <class E>
__global__ __launch_bounds__(kThreads, 2) void scan_backward(ScanBwd<E> a) {
    extern __shared__ float lds[];
    float *sB = lds, *sC = sB + kNB * CHUNK;
    float *sums = sC + kNB * CHUNK;                 // [kNR][2][kWaves][CHUNK]
    float *sH = sums + kNR * 2 * kWaves * CHUNK;    // [kNB][CH]: states before the chunk
    const int NP = (a.N + kNB - 1) / kNB * kNB;
    float *sA = sH + kNB * CH;                      // [NP][CH]: A log2(e)
    float *sG = sA + NP * CH;                       // [NP][CH]: what comes from behind
    float *sD = sG + NP * CH;                       // [NP][CH]: dA so far
    const int tid = threadIdx.x, lane = tid % LANES, ch = tid / LANES, wave = tid / 64;
    const int Dg = a.D / a.G;
    const int g = blockIdx.x / a.p.tiles, tile = blockIdx.x % a.p.tiles;
    const int b = blockIdx.y, seg = blockIdx.z;
    const bool live = tile * CH + ch < Dg;
    const int d = g * Dg + std::min(tile * CH + ch, Dg - 1);
    const int length = length_of(a.lengths, b, a.L);
    const int len = live ? length : 0;  // a row of no channel adds nothing to dB and dC
    const int64_t bs = (int64_t)b * a.p.segments + seg;
    for (int i = tid; i < NP * CH; i += kThreads) {
        const int n = i / CH, c = tile * CH + i % CH;
        float A2 = 0.f, q = 0.f;
        if (n < a.N && c < Dg) {
            const int64_t at = (int64_t)(g * Dg + c) * a.N + n;
            A2 = a.A[at] * kLog2e;
            if (a.p.segments > 1)
                q = a.ws[a.p.tails + bs * a.D * a.N + at];
            else if (a.gstate)
                q = a.gstate[(int64_t)b * a.D * a.N + at];
        }
        sA[i] = A2;
        sG[i] = q;
        sD[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const float skip = a.skip ? a.skip[d] : 0.f;
    float sum_skip = 0.f, sum_bias = 0.f;
    const int c_lo = (int)((int64_t)a.p.chunks * seg / a.p.segments);
    const int c_hi = (int)((int64_t)a.p.chunks * (seg + 1) / a.p.segments);
    for (int c = c_hi - 1; c >= c_lo; --c) {
        const int c0 = c * CHUNK, t0 = c0 + lane * T;
        float s[T], u[T], gy[T], total = 0.f;
        {
            float v[T];
            load_steps<E>(a.dt.row(b, d), t0, len, bias, a.softplus, s);
            load_row<E, T>(a.x.row(b, d), t0, len, v);
            load_row<E, T>(a.gout.row(b, d), t0, len, gy);
#pragma unroll
            for (int i = 0; i < T; ++i) {
                u[i] = s[i] * v[i];
                total += s[i];
            }
            if (a.z.p) {
                load_row<E, T>(a.z.row(b, d), t0, len, v);
#pragma unroll
                for (int i = 0; i < T; ++i) gy[i] *= v[i] * sigmoid(v[i]);
            }
        }
        float y[T], gB[T], ds[T];
#pragma unroll
        for (int i = 0; i < T; ++i) y[i] = gB[i] = ds[i] = 0.f;
        for (int n0 = 0; n0 < a.N; n0 += kNB) {
            const int nb = std::min(kNB, a.N - n0);
            __syncthreads();
            stage<E>(a.Bm, b, (int64_t)g * a.N + n0, nb, c0, length, sB, tid, kThreads);
            stage<E>(a.Cm, b, (int64_t)g * a.N + n0, nb, c0, length, sC, tid, kThreads);
            for (int i = tid; i < nb * CH; i += kThreads) {
                const int n = i % nb, cc = i / nb;
                const int64_t row = (int64_t)b * a.D + g * Dg + tile * CH + cc;
                sH[n * CH + cc] = tile * CH + cc < Dg
                                      ? a.checkpoints[(row * a.p.chunks + c) * a.N + n0 + n]
                                      : 0.f;
            }
            __syncthreads();
            for (int n1 = 0; n1 < nb; n1 += kNR) {
                const int nr = std::min(kNR, nb - n1);
                for (int r = 0; r < nr; ++r) {
                    const int n = n1 + r, at = (n0 + n) * CH + ch;
                    const float A2 = sA[at], carry = sG[at], h0 = sH[n * CH + ch];
                    float da[T], in[T], Bv[T], cg[T], pB[T], pC[T], ah[T];
                    fetch(sB, n, lane, Bv);
                    fetch(sC, n, lane, cg);
                    float hq = 0.f;
#pragma unroll
                    for (int i = 0; i < T; ++i) {
                        da[i] = exp2_fast(s[i] * A2);
                        in[i] = u[i] * Bv[i];
                        hq = __builtin_fmaf(da[i], hq, in[i]);
                    }
                    const float P = exp2_fast(total * A2);
                    const float hs = scan_forth(P, hq, h0, lane);
                    const float before = dpp0<kRowRor + 1>(hs);
                    float h = lane == 0 ? h0 : before;
#pragma unroll
                    for (int i = 0; i < T; ++i) {
                        ah[i] = da[i] * h;
                        h = ah[i] + in[i];
                        y[i] = __builtin_fmaf(cg[i], h, y[i]);
                        pC[i] = h * gy[i];
                        cg[i] *= gy[i];
                    }
                    float q = cg[T - 1];
#pragma unroll
                    for (int i = T - 2; i >= 0; --i) q = __builtin_fmaf(da[i + 1], q, cg[i]);
                    const float qs = scan_back(P, da[0] * q, carry, lane);
                    const float behind = dpp0<kRowRor + 15>(qs);
                    if (lane == LANES - 1) sG[at] = behind;
                    q = cg[T - 1] + (lane == LANES - 1 ? carry : behind);
                    float dA = 0.f;
#pragma unroll
                    for (int i = T - 1; i >= 0; --i) {
                        if (i < T - 1) q = __builtin_fmaf(da[i + 1], q, cg[i]);
                        const float through = q * ah[i];
                        ds[i] = __builtin_fmaf(A2, through, ds[i]);
                        dA = __builtin_fmaf(s[i], through, dA);
                        gB[i] = __builtin_fmaf(q, Bv[i], gB[i]);
                        pB[i] = q * u[i];
                    }
                    dA = row_sum(dA);
                    if (lane == 0) sD[at] += dA;
                    // Channels meet: row k of the wave ends with positions 2k, 2k+1 of each lane.
                    float *to = sums + ((r * 2) * kWaves + wave) * CHUNK + lane * T +
                                tid % 64 / LANES * 2;
                    float2 o;
                    o.x = meet16(meet32(pB[0], pB[4]), meet32(pB[2], pB[6]));
                    o.y = meet16(meet32(pB[1], pB[5]), meet32(pB[3], pB[7]));
                    *reinterpret_cast<float2 *>(to) = o;
                    o.x = meet16(meet32(pC[0], pC[4]), meet32(pC[2], pC[6]));
                    o.y = meet16(meet32(pC[1], pC[5]), meet32(pC[3], pC[7]));
                    *reinterpret_cast<float2 *>(to + kWaves * CHUNK) = o;
                }
                __syncthreads();
                for (int i = tid; i < nr * 2 * (CHUNK / 2); i += kThreads) {
                    const int t = i % (CHUNK / 2) * 2, which = i / (CHUNK / 2);  // [r][B or C]
                    const float *from = sums + which * kWaves * CHUNK + t;
                    float2 v = *reinterpret_cast<const float2 *>(from);
#pragma unroll
                    for (int w = 1; w < kWaves; ++w) {
                        const float2 m = *reinterpret_cast<const float2 *>(from + w * CHUNK);
                        v.x += m.x;
                        v.y += m.y;
                    }
                    const int64_t rows = (int64_t)a.B * a.G * a.N;
                    const int64_t row = ((int64_t)b * a.G + g) * a.N + n0 + n1 + which / 2;
                    *reinterpret_cast<float2 *>(
                        a.ws + a.p.sums +
                        (((int64_t)tile * 2 + which % 2) * rows + row) * a.p.pitch + c0 + t) = v;
                }
                if (n1 + kNR < nb) __syncthreads();
            }
        }
        if (live && t0 < a.L) {
            float x[T], v[T], o[T];
            load_row<E, T>(a.x.row(b, d), t0, len, x);
#pragma unroll
            for (int i = 0; i < T; ++i) {
                o[i] = __builtin_fmaf(skip, gy[i], s[i] * gB[i]);
                sum_skip = __builtin_fmaf(gy[i], x[i], sum_skip);
                ds[i] = __builtin_fmaf(ds[i], kLn2, x[i] * gB[i]);
            }
            store_row<E, T>(a.dx.row(b, d), t0, a.L, o);
            if (a.softplus) {
                load_row<E, T>(a.dt.row(b, d), t0, len, v);
#pragma unroll
                for (int i = 0; i < T; ++i) ds[i] *= sigmoid(v[i] + bias);
            }
#pragma unroll
            for (int i = 0; i < T; ++i) {
                ds[i] = t0 + i < len ? ds[i] : 0.f;
                sum_bias += ds[i];
            }
            store_row<E, T>(a.ddt.row(b, d), t0, a.L, ds);
            if (a.z.p) {
                float go[T];
                load_row<E, T>(a.z.row(b, d), t0, len, v);
                load_row<E, T>(a.gout.row(b, d), t0, len, go);
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    const float sg = sigmoid(v[i]);
                    o[i] = go[i] * __builtin_fmaf(skip, x[i], y[i]) *
                           (sg * __builtin_fmaf(v[i], 1.f - sg, 1.f));
                    o[i] = t0 + i < len ? o[i] : 0.f;
                }
                store_row<E, T>(a.dz.row(b, d), t0, a.L, o);
            }
        }
    }
    __syncthreads();
    float *params = a.ws + a.p.params + bs * a.D * (a.N + 2);
    for (int i = tid; i < a.N * CH; i += kThreads) {
        const int n = i % a.N, cc = i / a.N, c = tile * CH + cc;
        if (c >= Dg) continue;
        const int64_t dc = g * Dg + c;
        params[dc * (a.N + 2) + n] = sD[n * CH + cc];
        if (seg == 0 && a.dstate)
            a.dstate[((int64_t)b * a.D + dc) * a.N + n] = sG[n * CH + cc];
    }
    sum_skip = row_sum(sum_skip);
    sum_bias = row_sum(sum_bias);
    if (live && lane == 0) {
        params[(int64_t)d * (a.N + 2) + a.N] = sum_skip;
        params[(int64_t)d * (a.N + 2) + a.N + 1] = sum_bias;
    }
}

// What a segment sends back to the state before it when nothing comes from
// behind: tails[b][segment][d][n], and its summed steps [b][segment][d].
template <class E>
__global__ __launch_bounds__(kTailThreads) void scan_tail(ScanBwd<E> a, int tiles) {
    extern __shared__ float lds[];
    float *sC = lds;
    const int NP = (a.N + kNB - 1) / kNB * kNB;
    float *sA = sC + kNB * CHUNK, *sG = sA + NP * kTailCH;
    const int tid = threadIdx.x, lane = tid % LANES, ch = tid / LANES;
    const int Dg = a.D / a.G;
    const int g = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int b = blockIdx.y, seg = blockIdx.z;
    const bool live = tile * kTailCH + ch < Dg;
    const int d = g * Dg + std::min(tile * kTailCH + ch, Dg - 1);
    const int len = length_of(a.lengths, b, a.L);
    for (int i = tid; i < NP * kTailCH; i += kTailThreads) {
        const int n = i / kTailCH, c = tile * kTailCH + i % kTailCH;
        sA[i] = n < a.N && c < Dg ? a.A[(int64_t)(g * Dg + c) * a.N + n] * kLog2e : 0.f;
        sG[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    float steps = 0.f;
    const int c_lo = (int)((int64_t)a.p.chunks * seg / a.p.segments);
    const int c_hi = (int)((int64_t)a.p.chunks * (seg + 1) / a.p.segments);
    for (int c = c_hi - 1; c >= c_lo; --c) {
        const int c0 = c * CHUNK, t0 = c0 + lane * T;
        float s[T], gy[T], total = 0.f;
        load_steps<E>(a.dt.row(b, d), t0, len, bias, a.softplus, s);
        load_row<E, T>(a.gout.row(b, d), t0, len, gy);
#pragma unroll
        for (int i = 0; i < T; ++i) total += s[i];
        if (a.z.p) {
            float v[T];
            load_row<E, T>(a.z.row(b, d), t0, len, v);
#pragma unroll
            for (int i = 0; i < T; ++i) gy[i] *= v[i] * sigmoid(v[i]);
        }
        steps += total;
        for (int n0 = 0; n0 < a.N; n0 += kNB) {
            const int nb = std::min(kNB, a.N - n0);
            __syncthreads();
            stage<E>(a.Cm, b, (int64_t)g * a.N + n0, nb, c0, len, sC, tid, kTailThreads);
            __syncthreads();
            for (int n = 0; n < nb; ++n) {
                const int at = (n0 + n) * kTailCH + ch;
                const float A2 = sA[at], carry = sG[at];
                float Cv[T];
                fetch(sC, n, lane, Cv);
                float q = 0.f;
#pragma unroll
                for (int i = T - 1; i >= 0; --i)
                    q = exp2_fast(s[i] * A2) * __builtin_fmaf(Cv[i], gy[i], q);
                const float qs = scan_back(exp2_fast(total * A2), q, carry, lane);
                if (lane == 0) sG[at] = qs;
            }
        }
    }
    __syncthreads();
    const int64_t bs = (int64_t)b * a.p.segments + seg;
    for (int i = tid; i < a.N * kTailCH; i += kTailThreads) {
        const int n = i % a.N, cc = i / a.N, c = tile * kTailCH + cc;
        if (c < Dg) a.ws[a.p.tails + (bs * a.D + g * Dg + c) * a.N + n] = sG[n * kTailCH + cc];
    }
    steps = row_sum(steps);
    if (live && lane == 0) a.ws[a.p.steps + bs * a.D + d] = steps;
}

// Chains the segments of a (batch, channel, state): tails become what comes
// from behind each segment.
__global__ void scan_carry(float *ws, Plan p, const float *A, const float *gstate, int64_t B,
                           int64_t D, int64_t N) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= B * D * N) return;
    const int64_t b = i / (D * N), dn = i - b * D * N, d = dn / N;
    const float A2 = A[dn] * kLog2e;
    float carry = gstate ? gstate[i] : 0.f;
    for (int seg = p.segments - 1; seg >= 0; --seg) {
        const int64_t bs = b * p.segments + seg;
        float *tail = ws + p.tails + bs * D * N + dn;
        const float own = *tail;
        *tail = carry;
        carry = __builtin_fmaf(exp2_fast(ws[p.steps + bs * D + d] * A2), carry, own);
    }
}

// The last sums: dB and dC over channel tiles, dA, dskip and ddt_bias over the
// batch and the segments.  Blocks [0, matrix_blocks) take the former.
template <class E>
__global__ __launch_bounds__(256) void scan_join(const float *ws, Plan p, int64_t B, int64_t D,
                                                 int64_t L, int64_t N, int64_t G,
                                                 typename E::type *dB, typename E::type *dC,
                                                 float *dA, float *dskip, float *dbias,
                                                 const int32_t *lengths, int64_t matrix_blocks) {
    const int64_t rows = B * G * N;
    if (blockIdx.x < matrix_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        const int64_t per_row = p.pitch / 4;
        const int64_t r = i / per_row, t = i % per_row * 4;
        if (r >= 2 * rows || t >= L) return;
        const float *from = ws + p.sums + r * p.pitch + t;
        float4 v = {0.f, 0.f, 0.f, 0.f};
        for (int tile = 0; tile < p.tiles; ++tile) {
            const float4 m = *reinterpret_cast<const float4 *>(from + tile * 2 * rows * p.pitch);
            v.x += m.x;
            v.y += m.y;
            v.z += m.z;
            v.w += m.w;
        }
        float out[4] = {v.x, v.y, v.z, v.w};
        const int64_t br = r < rows ? r : r - rows;
        const int len = length_of(lengths, br / (G * N), (int)L);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = t + i < len ? out[i] : 0.f;
        typename E::type *to = (r < rows ? dB : dC) + br * L;
        store_row<E, 4>(to, t, L, out);
        return;
    }
    const int64_t i = (blockIdx.x - matrix_blocks) * 256 + threadIdx.x;
    if (i >= D * (N + 2)) return;
    float v = 0.f;
    for (int64_t s = 0; s < B * p.segments; ++s) v += ws[p.params + s * D * (N + 2) + i];
    const int64_t d = i / (N + 2), n = i % (N + 2);
    if (n < N) {
        dA[d * N + n] = v;
    } else if (n == N) {
        if (dskip) dskip[d] = v;
    } else if (dbias) {
        dbias[d] = v;
    }
}

template <class E>
hipError_t backward(const state_scan_backward_args &a, hipStream_t s) {
    ScanBwd<E> k{view<E>(a.gout), view<E>(a.x), view<E>(a.dt), view<E>(a.z), view<E>(a.Bm),
                 view<E>(a.Cm), view<E>(a.dx), view<E>(a.ddt), view<E>(a.dz), a.A, a.skip,
                 a.dt_bias, a.checkpoints, a.gstate, a.dstate, a.lengths,
                 static_cast<float *>(a.workspace), a.B, a.D, a.L, a.N, a.G, a.softplus,
                 make_plan(a.B, a.D, a.L, a.N, a.G)};
    const Plan &p = k.p;
    const int NP = (a.N + kNB - 1) / kNB * kNB;
    hipError_t e;
    if (p.segments > 1) {
        const int tiles = (a.D / a.G + kTailCH - 1) / kTailCH;
        const size_t bytes = (kNB * CHUNK + 2 * (size_t)NP * kTailCH) * sizeof(float);
        scan_tail<E><<<dim3((unsigned)(a.G * tiles), (unsigned)a.B, (unsigned)p.segments),
                       kTailThreads, bytes, s>>>(k, tiles);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        const int64_t n = (int64_t)a.B * a.D * a.N;
        scan_carry<<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(k.ws, p, a.A, a.gstate, a.B,
                                                                    a.D, a.N);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const size_t bytes = (2 * kNB * CHUNK + kNR * 2 * kWaves * CHUNK + kNB * CH +
                          3 * (size_t)NP * CH) * sizeof(float);
    if (bytes > 64 * 1024) {
        e = hipFuncSetAttribute((const void *)scan_backward<E>,
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != hipSuccess) return e;
    }
    scan_backward<E><<<dim3((unsigned)(a.G * p.tiles), (unsigned)a.B, (unsigned)p.segments),
                       kThreads, bytes, s>>>(k);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t matrix = (2 * (int64_t)a.B * a.G * a.N * (p.pitch / 4) + 255) / 256;
    const int64_t params = ((int64_t)a.D * (a.N + 2) + 255) / 256;
    scan_join<E><<<dim3((unsigned)(matrix + params)), 256, 0, s>>>(
        k.ws, p, a.B, a.D, a.L, a.N, a.G, static_cast<typename E::type *>(a.dBm),
        static_cast<typename E::type *>(a.dCm), a.dA, a.dskip, a.ddt_bias,
        a.lengths, matrix);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_backward(const state_scan_backward_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? backward<F32>(a, s)
           : a.dtype == SEQ_BF16 ? backward<BF16>(a, s) : backward<F16>(a, s);
}

int64_t scan_backward_workspace(int B, int D, int L, int N, int G) {
    return make_plan(B, D, L, N, G).floats * 4;
}

}  // namespace seq
