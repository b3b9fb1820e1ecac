// kernels_state_scan_bwd.hip -- the gradients of the selective state space scan.
//
// Two chains a state: h forwards (run again from the checkpoint before the
// chunk) and its gradient q backwards, q_t = C_t gy_t + a_{t+1} q_{t+1}; both go
// over a chunk with the lane scan of kernels_state_scan.hip and share its
// exponentials.  dB and dC sum over channels: 4 channels meet in a wave through
// lane swaps, a work-group's waves through LDS, and the work-groups of a group through the
// workspace, in a fixed order.
//
// A work-group walks its chunks from the last to the first.  Where there are
// too few (batch, channel tile) pairs to fill the chip, the positions are cut
// into segments: scan_tail finds what each segment sends back on its own, and
// the segments then run side by side, each chaining what is behind it.
//
// What bounds it: issue of the vector ALUs, 27 instructions for each (channel,
// state, position): an exponential, 15 of the formula's chains and sums over states
// and positions, 5 for the sums over a wave's channels, 2 for the lane scans, the
// rest selects and addresses.  A loop of the formula's 16 on registers reaches 0.389 ps
// an element with 8 waves a SIMD, 104 us at [4, 2048, 2048] bf16, N = 16; here 256
// registers a lane leave two waves, and it takes 262 us (and scan_join 12, whose
// 67 MB come from the caches).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

constexpr int LANES = 16, RPW = 64 / LANES;
constexpr int kNB = 16;  // states whose B and C are in LDS at once
constexpr int kTailT = 8, kTailNI = 4, kTailWaves = 4, kTailThreads = 64 * kTailWaves,
              kTailCH = kTailWaves * RPW;

struct Plan {
    int W, T, chunk;     // waves of a work-group, positions of a lane and of a chunk
    int tiles, chunks;   // channel tiles of a group, chunks of a row
    int segments;
    int marks;           // checkpoints of a row
    int pitch;           // padded positions of a partial row of dB or dC
    int joined;          // states summed over the waves at once
    size_t lds;
    int64_t sums, params, tails, steps;  // workspace offsets, in floats
    int64_t floats;
};

constexpr size_t kLdsBytes = 160 * 1024;

// LDS of a work-group: B and C, two halves of sums, states before, and A, q and dA.
size_t lds_bytes(int W, int T, int joined, int64_t N) {
    const size_t NP = (N + kNB - 1) / kNB * kNB, chunk = LANES * T, CH = W * RPW;
    return (2 * kNB * chunk + 2 * joined * 2 * W * chunk + kNB * CH + 3 * NP * CH) *
           sizeof(float);
}

Plan make_plan(int64_t B, int64_t D, int64_t L, int64_t N, int64_t G) {
    Plan p;
    // Work-groups of 8 waves, one on a compute unit, lanes of 16 positions (which
    // spend half as much on the lane scans as lanes of 8: 30 instructions for both
    // chains, beside some 24 a position) unless padding the row to whole chunks costs
    // more, there are too few chunks to give every compute unit one, or their sums do
    // not fit.  Where that leaves the last round of compute units mostly empty,
    // work-groups of 4 waves and lanes of 8, more of them cut finer, though they share
    // less.  Measured (us, first / second way): [4, 2048, 2048] N 16 268 / 315,
    // [1, 1024, 2048] N 16 60 / 65, [2, 547, 1364] N 64 174 / 174, but
    // [5, 1825, 3409] N 8 686 / 498, [2, 1834, 640] N 64 239 / 207,
    // [2, 340, 3307] N 64 304 / 249.
    const int64_t c16 = (L + 255) / 256, c8 = (L + 127) / 128;
    const int64_t wide = B * G * ((D / G + 8 * RPW - 1) / (8 * RPW));
    const auto deal = [&](int W, int T, int64_t want) {
        p.W = W;
        p.T = T;
        p.chunk = LANES * T;
        p.chunks = (int)((L + p.chunk - 1) / p.chunk);
        p.tiles = (int)((D / G + W * RPW - 1) / (W * RPW));
        // As many segments as `want` work-groups need, evened out.
        const int64_t groups = B * G * p.tiles;
        const int most = (int)std::min<int64_t>(p.chunks, (want + groups - 1) / groups);
        const int longest = (p.chunks + most - 1) / most;
        p.segments = (p.chunks + longest - 1) / longest;
        const int64_t rounds = (groups * p.segments + 255) / 256;
        return (double)(groups * p.chunks) / (double)(rounds * 256 * longest);
    };
    const bool longer = c16 * (16 * 24 + 30) <= c8 * (8 * 24 + 30) && wide * c16 >= 256 &&
                        lds_bytes(8, 16, 1, N) <= kLdsBytes;
    if (deal(8, longer ? 16 : 8, 256) < 0.7) deal(4, 8, 1536);
    p.joined = p.T == 16 ? 2 : 4;
    while (lds_bytes(p.W, p.T, p.joined, N) > kLdsBytes) p.joined /= 2;
    p.lds = lds_bytes(p.W, p.T, p.joined, N);
    p.marks = (int)((L + SEQ_SCAN_CHECKPOINT - 1) / SEQ_SCAN_CHECKPOINT);
    p.pitch = p.chunks * p.chunk;
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
template <class E, int T>
__device__ __forceinline__ void load_steps(const typename E::type *dt, int t0, int len, float bias,
                                           bool soft, float (&s)[T]) {
    load_row<E, T>(dt, t0, len, s);
#pragma unroll
    for (int i = 0; i < T; ++i) s[i] += bias;
    if (soft) {
#pragma unroll
        for (int i = 0; i < T; ++i) s[i] = softplus(s[i]);
    }
    if (len - t0 < T) {
#pragma unroll
        for (int i = 0; i < T; ++i) s[i] = len - t0 > i ? s[i] : 0.f;
    }
}

// Sum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float row_sum(float v) {
    v += dpp0<kRowRor + 8>(v);
    v += dpp0<kRowRor + 4>(v);
    v += dpp0<kRowRor + 2>(v);
    return v + dpp0<kRowRor + 1>(v);
}

template <int T>
__device__ __forceinline__ void fetch(const float *from, int lane, float (&v)[T]) {
#pragma unroll
    for (int j = 0; j < T / 4; ++j) {
        const float4 f = *reinterpret_cast<const float4 *>(from + (j * LANES + lane) * 4);
        v[4 * j] = f.x;
        v[4 * j + 1] = f.y;
        v[4 * j + 2] = f.z;
        v[4 * j + 3] = f.w;
    }
}

// A work-group: waves of 4 channels, 16 lanes a channel, T positions a lane,
// NI states at a time.
template <class E, int kWaves, int T, int NI>
__global__ __launch_bounds__(64 * kWaves, 2) void scan_backward(ScanBwd<E> a) {
    constexpr int kThreads = 64 * kWaves, CH = kWaves * RPW;
    constexpr int CHUNK = LANES * T, F = T / 4;  // F: sums of a lane
    constexpr int OCTETS = 2 * kNB * CHUNK / 8, PRE = OCTETS / kThreads;
    static_assert(OCTETS % kThreads == 0 && kNB * CH == kThreads, "whole rounds of threads");
    extern __shared__ float lds[];
    float *sBC = lds;                                        // [B or C][kNB][CHUNK]
    float *sums = sBC + 2 * kNB * CHUNK;                     // 2 of [joined][B or C][kWaves][64][F]
    float *sH = sums + 2 * a.p.joined * 2 * kWaves * CHUNK;  // [kNB][CH]: states before
    const int NP = (a.N + kNB - 1) / kNB * kNB;
    float *sA = sH + kNB * CH;                               // [NP][CH]: A log2(e)
    float *sG = sA + NP * CH;                                // [NP][CH]: what comes from behind
    float *sD = sG + NP * CH;                                // [NP][CH]: dA so far
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
            A2 = decay_rate(a.A[at]);
            if (a.gstate) q = a.gstate[(int64_t)b * a.D * a.N + at];
            // Through the segments behind this one.
#pragma unroll 4
            for (int later = a.p.segments - 1; later > seg; --later) {
                const int64_t ls = (int64_t)b * a.p.segments + later;
                q = __builtin_fmaf(exp2_fast(a.ws[a.p.steps + ls * a.D + g * Dg + c] * A2), q,
                                   a.ws[a.p.tails + ls * a.D * a.N + at]);
            }
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
    // B, C and the checkpoints of the next group of states travel while this one's chains run.
    Octet<E> next[PRE];
    float next_h = 0.f;
    const auto prefetch = [&](int c, int n0) {
#pragma unroll
        for (int k = 0; k < PRE; ++k) {
            const int o = k * kThreads + tid, per = kNB * CHUNK / 8;
            const int n = n0 + o % per / (CHUNK / 8), t = c * CHUNK + o % (CHUNK / 8) * 8;
            const View<E> &m = o < per ? a.Bm : a.Cm;
            next[k].load(m.row(b, (int64_t)g * a.N + n) + t, n < a.N ? length - t : 0);
        }
        const int n = n0 + tid % kNB, cc = tile * CH + tid / kNB;
        next_h = 0.f;
        if (n < a.N && cc < Dg)
            next_h = a.checkpoints[(((int64_t)b * a.D + g * Dg + cc) * a.p.marks +
                                    c * CHUNK / SEQ_SCAN_CHECKPOINT) * a.N + n];
    };
    prefetch(c_hi - 1, 0);
    // This tile's part of dB, and how far from it dC's is.
    const int64_t to_C = (int64_t)a.B * a.G * a.N * a.p.pitch;
    float *out = a.ws + a.p.sums + tile * 2 * to_C + ((int64_t)b * a.G + g) * a.N * a.p.pitch;
    // Sums of a group of states over the waves are read from one half of `sums`
    // while the next group's are written to the other.
    int half = 0;
    for (int c = c_hi - 1; c >= c_lo; --c) {
        const int c0 = c * CHUNK, t0 = c0 + lane * T;
        float s[T], u[T], gy[T], total = 0.f;
        {
            float v[T];
            load_steps<E, T>(a.dt.row(b, d), t0, len, bias, a.softplus, s);
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
#pragma unroll
            for (int k = 0; k < PRE; ++k) stage_octet<E, LANES, T>(sBC, k * kThreads + tid, next[k]);
            sH[tid % kNB * CH + tid / kNB] = next_h;
            __syncthreads();
            const bool more = n0 + kNB < a.N;
            if (more || c > c_lo) prefetch(more ? c : c - 1, more ? n0 + kNB : 0);
            for (int n1 = 0; n1 < nb; n1 += a.p.joined) {
                const int nr = std::min(a.p.joined, nb - n1);
                for (int r = 0; r < nr; r += NI) {
                    // (States past N have A, B, C and h 0 and change nothing.)
                    const int n = n1 + r, at = (n0 + n) * CH + ch;
                    float A2[NI], carry[NI], h0[NI], h[NI], q[NI], P[NI], P1[NI], turned[NI];
                    float da[NI][T], in[NI][T], Bv[NI][T], cg[NI][T], ah[NI][T];
#pragma unroll
                    for (int k = 0; k < NI; ++k) {
                        A2[k] = sA[at + k * CH];
                        carry[k] = sG[at + k * CH];
                        h0[k] = sH[(n + k) * CH + ch];
                        fetch<T>(sBC + (n + k) * CHUNK, lane, Bv[k]);
                        h[k] = lane == 0 ? h0[k] : 0.f;
                        P[k] = exp2_fast(total * A2[k]);
                        P1[k] = P[k];
                    }
#pragma unroll
                    for (int i = 0; i < T; ++i)
#pragma unroll
                        for (int k = 0; k < NI; ++k) {
                            da[k][i] = exp2_fast(s[i] * A2[k]);
                            in[k][i] = u[i] * Bv[k][i];
                            h[k] = __builtin_fmaf(da[k][i], h[k], in[k][i]);
                        }
                    scan_lanes<LANES>(h, P1, turned);
                    float *to = sums + ((half * a.p.joined + r) * 2 * kWaves + wave) * CHUNK +
                                tid % 64 * F;
#pragma unroll
                    for (int k = 0; k < NI; ++k) {
                        h[k] = lane == 0 ? h0[k] : turned[k];
                        fetch<T>(sBC + (kNB + n + k) * CHUNK, lane, cg[k]);
                        float p[T];
#pragma unroll
                        for (int i = 0; i < T; ++i) {
                            ah[k][i] = da[k][i] * h[k];
                            h[k] = ah[k][i] + in[k][i];
                            y[i] = __builtin_fmaf(cg[k][i], h[k], y[i]);
                            p[i] = h[k] * gy[i];
                            cg[k][i] *= gy[i];
                        }
                        *reinterpret_cast<Whole<F> *>(to + (k * 2 + 1) * kWaves * CHUNK) =
                            meet_rows<T>(p);
                        // q, the gradient of h; lane 15 starts from what comes from behind.
                        q[k] = cg[k][T - 1] + (lane == LANES - 1 ? carry[k] : 0.f);
                        P1[k] = P[k];
                    }
#pragma unroll
                    for (int i = T - 2; i >= 0; --i)
#pragma unroll
                        for (int k = 0; k < NI; ++k)
                            q[k] = __builtin_fmaf(da[k][i + 1], q[k], cg[k][i]);
#pragma unroll
                    for (int k = 0; k < NI; ++k) q[k] *= da[k][0];
                    scan_lanes_back<NI>(q, P1, turned);
#pragma unroll
                    for (int k = 0; k < NI; ++k) {
                        if (lane == LANES - 1) sG[at + k * CH] = turned[k];
                        q[k] = cg[k][T - 1] + (lane == LANES - 1 ? carry[k] : turned[k]);
                        if constexpr (T == 16) fetch<T>(sBC + (n + k) * CHUNK, lane, Bv[k]);
                        float dA = 0.f, p[T];
#pragma unroll
                        for (int i = T - 1; i >= 0; --i) {
                            if (i < T - 1) q[k] = __builtin_fmaf(da[k][i + 1], q[k], cg[k][i]);
                            p[i] = q[k] * u[i];
                            const float through = q[k] * ah[k][i];
                            ds[i] = __builtin_fmaf(A2[k], through, ds[i]);
                            dA = __builtin_fmaf(s[i], through, dA);
                            gB[i] = __builtin_fmaf(q[k], Bv[k][i], gB[i]);
                        }
                        dA = row_sum(dA);
                        if (lane == 0) sD[at + k * CH] += dA;
                        *reinterpret_cast<Whole<F> *>(to + k * 2 * kWaves * CHUNK) =
                            meet_rows<T>(p);
                    }
                }
                __syncthreads();
                for (int i = tid; i < nr * 2 * 64; i += kThreads) {
                    const int f = i % 64, rw = i / 64;  // [r][B or C]
                    const float *from =
                        sums + (half * a.p.joined * 2 + rw) * kWaves * CHUNK + f * F;
                    Whole<F> v = *reinterpret_cast<const Whole<F> *>(from);
#pragma unroll
                    for (int w = 1; w < kWaves; ++w) {
                        const Whole<F> o = *reinterpret_cast<const Whole<F> *>(from + w * CHUNK);
#pragma unroll
                        for (int k = 0; k < F; ++k) v.v[k] += o.v[k];
                    }
                    *reinterpret_cast<Whole<F> *>(out + (rw & 1 ? to_C : 0) +
                                                  (int64_t)(n0 + n1 + rw / 2) * a.p.pitch + c0 +
                                                  f % 16 * T + f / 16 * F) = v;
                }
                half ^= 1;
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
            if (len - t0 < T) {
#pragma unroll
                for (int i = 0; i < T; ++i) o[i] = len - t0 > i ? o[i] : 0.f;
            }
            store_row<E, T>(a.dx.row(b, d), t0, a.L, o);
            if (a.softplus) {
                load_row<E, T>(a.dt.row(b, d), t0, len, v);
#pragma unroll
                for (int i = 0; i < T; ++i) ds[i] *= sigmoid(v[i] + bias);
            }
            if (len - t0 < T) {
#pragma unroll
                for (int i = 0; i < T; ++i) ds[i] = len - t0 > i ? ds[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < T; ++i) sum_bias += ds[i];
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
                }
                if (len - t0 < T) {
#pragma unroll
                    for (int i = 0; i < T; ++i) o[i] = len - t0 > i ? o[i] : 0.f;
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

// What a segment (but the first, behind nothing) sends back to the state before it
// when nothing comes from behind: tails[b][segment][d][n], and its summed steps
// [b][segment][d].
template <class E>
__global__ __launch_bounds__(kTailThreads) void scan_tail(ScanBwd<E> a, int tiles) {
    constexpr int T = kTailT, CHUNK = LANES * T;
    extern __shared__ float lds[];
    float *sC = lds;
    const int NP = (a.N + kNB - 1) / kNB * kNB;
    float *sA = sC + kNB * CHUNK, *sG = sA + NP * kTailCH;
    const int tid = threadIdx.x, lane = tid % LANES, ch = tid / LANES;
    const int Dg = a.D / a.G;
    const int g = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int b = blockIdx.y, seg = blockIdx.z + 1;
    const bool live = tile * kTailCH + ch < Dg;
    const int d = g * Dg + std::min(tile * kTailCH + ch, Dg - 1);
    const int len = length_of(a.lengths, b, a.L);
    for (int i = tid; i < NP * kTailCH; i += kTailThreads) {
        const int n = i / kTailCH, c = tile * kTailCH + i % kTailCH;
        sA[i] = n < a.N && c < Dg ? decay_rate(a.A[(int64_t)(g * Dg + c) * a.N + n]) : 0.f;
        sG[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    float steps = 0.f;
    const int lo = (int)((int64_t)a.p.chunks * seg / a.p.segments) * a.p.chunk;
    const int hi = (int)((int64_t)a.p.chunks * (seg + 1) / a.p.segments) * a.p.chunk;
    for (int c0 = hi - CHUNK; c0 >= lo; c0 -= CHUNK) {
        const int t0 = c0 + lane * T;
        float s[T], gy[T], total = 0.f;
        load_steps<E, T>(a.dt.row(b, d), t0, len, bias, a.softplus, s);
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
            for (int o = tid; o < kNB * (CHUNK / 8); o += kTailThreads) {
                Octet<E> v;
                const int t = c0 + o % (CHUNK / 8) * 8, n = n0 + o / (CHUNK / 8);
                v.load(a.Cm.row(b, (int64_t)g * a.N + n) + t, n < a.N ? len - t : 0);
                stage_octet<E, LANES, T>(sC, o, v);
            }
            __syncthreads();
            // kTailNI states at once: there are few waves, and one chain waits for itself
            // (67 us for 61 at [4, 420, 3640] f32, N = 24).  States past N have A and C 0 and
            // change nothing.
            for (int n = 0; n < nb; n += kTailNI) {
                const int at = (n0 + n) * kTailCH + ch;
                float A2[kTailNI], q[kTailNI], P[kTailNI], turned[kTailNI], Cv[kTailNI][T];
#pragma unroll
                for (int k = 0; k < kTailNI; ++k) {
                    A2[k] = sA[at + k * kTailCH];
                    q[k] = lane == LANES - 1 ? sG[at + k * kTailCH] : 0.f;
                    fetch<T>(sC + (n + k) * CHUNK, lane, Cv[k]);
                    P[k] = exp2_fast(total * A2[k]);
                }
#pragma unroll
                for (int i = T - 1; i >= 0; --i)
#pragma unroll
                    for (int k = 0; k < kTailNI; ++k)
                        q[k] = exp2_fast(s[i] * A2[k]) * __builtin_fmaf(Cv[k][i], gy[i], q[k]);
                scan_lanes_back<kTailNI>(q, P, turned);
#pragma unroll
                for (int k = 0; k < kTailNI; ++k)
                    if (lane == 0) sG[at + k * kTailCH] = q[k];
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
        // 64 runs of 4 positions a work-group, its waves over every fourth tile each.
        __shared__ float4 part[4][64];
        const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x % 64;
        const int wave = threadIdx.x / 64;
        const int64_t per_row = p.pitch / 4;
        const int64_t r = i / per_row, t = i % per_row * 4;
        const bool here = r < 2 * rows && t < L;
        const float *from = ws + p.sums + r * p.pitch + t;
        float4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int tile = wave; here && tile < p.tiles; tile += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(from + tile * 2 * rows * p.pitch);
            v.x += m.x;
            v.y += m.y;
            v.z += m.z;
            v.w += m.w;
        }
        part[wave][threadIdx.x % 64] = v;
        __syncthreads();
        if (wave || !here) return;
        float out[4] = {v.x, v.y, v.z, v.w};
        for (int w = 1; w < 4; ++w) {
            const float4 m = part[w][threadIdx.x];
            out[0] += m.x;
            out[1] += m.y;
            out[2] += m.z;
            out[3] += m.w;
        }
        const int64_t br = r < rows ? r : r - rows;
        const int len = length_of(lengths, br / (G * N), (int)L);
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = t + k < len ? out[k] : 0.f;
        store_row<E, 4>((r < rows ? dB : dC) + br * L, (int)t, (int)L, out);
        return;
    }
    const int64_t i = (blockIdx.x - matrix_blocks) * 256 + threadIdx.x;
    if (i >= D * (N + 2)) return;
    float v = 0.f;
#pragma unroll 8
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
        const size_t bytes = (kNB * LANES * kTailT + 2 * (size_t)NP * kTailCH) * sizeof(float);
        scan_tail<E><<<dim3((unsigned)(a.G * tiles), (unsigned)a.B, (unsigned)(p.segments - 1)),
                       kTailThreads, bytes, s>>>(k, tiles);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const auto kernel = p.W == 4 ? scan_backward<E, 4, 8, 2>
                        : p.T == 16 ? scan_backward<E, 8, 16, 1> : scan_backward<E, 8, 8, 2>;
    if (p.lds > 64 * 1024) {
        e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)p.lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<dim3((unsigned)(a.G * p.tiles), (unsigned)a.B, (unsigned)p.segments), 64 * p.W, p.lds,
             s>>>(k);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t matrix = (2 * (int64_t)a.B * a.G * a.N * (p.pitch / 4) + 63) / 64;
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

void scan_backward_plan(int B, int D, int L, int N, int G, char *buf, size_t len) {
    const Plan p = make_plan(B, D, L, N, G);
    std::snprintf(buf, len, "waves=%d positions=%d segments=%d joined=%d", p.W, p.T, p.segments,
                  p.joined);
}

int64_t scan_backward_workspace(int B, int D, int L, int N, int G) {
    return make_plan(B, D, L, N, G).floats * 4;
}

}  // namespace seq
