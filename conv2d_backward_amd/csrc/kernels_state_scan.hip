// kernels_state_scan.hip -- the selective state space scan over prompts and
// one position of it against a state cache.
//
// h_t = a_t h_{t-1} + b_t with a_t = exp(s_t A), b_t = s_t x_t B_t is a chain
// along the positions, but maps compose: positions i..j send h to P h + Q with
// P = exp(A (s_i + .. + s_j)).  A lane takes T consecutive positions, runs their
// chain once from 0 for its Q, the lanes of a row combine their (P, Q) in
// log2(lanes) steps, and each lane runs its chain again from the state it then
// knows, adding C_t h_t to its outputs.  Every exponential is taken once.
//
// What bounds it: for each (channel, state, position) one v_exp_f32 (a quarter
// rate instruction) and five full-rate ones, about 10 issue slots of 4 cycles
// for 64 elements with the lane scan; the bytes (x, dt, z, y) are 1/N of that
// many elements.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kNB = 16;  // states whose B and C are in LDS at once

template <class E>
struct ScanFwd {
    View<E> x, dt, z, Bm, Cm, y;
    const float *A, *skip, *dt_bias, *state_in;
    float *state_out, *checkpoints;
    const int32_t *lengths;
    int B, D, L, N, G;
    int tiles;  // channel tiles of a group
    int softplus;
};

// A work-group: 4 waves, each RPW = 64/16 rows (channels) of 16 lanes, each lane T
// positions.  LDS: B and C of kNB states over a chunk of 16 T positions (fp32,
// in the order the lanes read them), then A log2(e) and the running state of
// every (state, channel).
template <class E, int T>
__global__ __launch_bounds__(kThreads) void scan_forward(ScanFwd<E> a) {
    constexpr int LANES = 16, RPW = 64 / LANES, CH = kWaves * RPW, CHUNK = LANES * T;
    constexpr int Q = T / 4;
    extern __shared__ float lds[];
    float *sB = lds, *sC = lds + kNB * CHUNK;
    float2 *sAh = reinterpret_cast<float2 *>(lds + 2 * kNB * CHUNK);  // [N][CH]
    const int tid = threadIdx.x, lane = tid % LANES, ch = tid / LANES;
    const int Dg = a.D / a.G;
    const int g = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles, b = blockIdx.y;
    const int in_group = tile * CH + ch;
    const bool live = in_group < Dg;
    const int d = g * Dg + (live ? in_group : Dg - 1);
    const int len = length_of(a.lengths, b, a.L);
    const int64_t row = (int64_t)b * a.D + d;
    const int NP = (a.N + kNB - 1) / kNB * kNB;
    for (int i = tid; i < NP * CH; i += kThreads) {
        const int n = i / CH, c = i % CH;
        const int dc = g * Dg + std::min(tile * CH + c, Dg - 1);
        float2 v = {0.f, 0.f};
        if (n < a.N) {
            v.x = a.A[(int64_t)dc * a.N + n] * kLog2e;
            if (a.state_in) v.y = a.state_in[((int64_t)b * a.D + dc) * a.N + n];
        }
        sAh[i] = v;
    }
    const auto *x = a.x.row(b, d), *dt = a.dt.row(b, d);
    const auto *z = a.z.p ? a.z.row(b, d) : nullptr;
    auto *y = a.y.row(b, d);
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const float skip = a.skip ? a.skip[d] : 0.f;
    const int nck = (a.L + SEQ_SCAN_CHECKPOINT - 1) / SEQ_SCAN_CHECKPOINT;
    // With checkpoints every chunk is run (their states are wanted), else those with positions.
    const int end = a.checkpoints ? a.L : len;
    int c0 = 0;
    for (; c0 < end; c0 += CHUNK) {
        const int t0 = c0 + lane * T;
        float s[T], u[T], acc[T];
        float total = 0.f;
        {
            float xv[T];
            load_row<E, T>(x, t0, len, xv);
            load_row<E, T>(dt, t0, len, s);
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const float raw = s[i] + bias;
                const float step = a.softplus ? softplus(raw) : raw;
                s[i] = t0 + i < len ? step : 0.f;  // 0: the state passes unchanged
                u[i] = s[i] * xv[i];
                acc[i] = skip * xv[i];
                total += s[i];
            }
        }
        for (int n0 = 0; n0 < a.N; n0 += kNB) {
            const int nb = std::min(kNB, a.N - n0);
            __syncthreads();
            for (int i = tid; i < nb * (CHUNK / 4); i += kThreads) {
                const int n = i / (CHUNK / 4), q = i % (CHUNK / 4);
                const int64_t t = c0 + 4 * q;
                const int at = n * CHUNK + (q % Q * LANES + q / Q) * 4;
                float v[4];
                load_row<E, 4>(a.Bm.row(b, (int64_t)g * a.N + n0 + n), t, len, v);
                *reinterpret_cast<float4 *>(sB + at) = float4{v[0], v[1], v[2], v[3]};
                load_row<E, 4>(a.Cm.row(b, (int64_t)g * a.N + n0 + n), t, len, v);
                *reinterpret_cast<float4 *>(sC + at) = float4{v[0], v[1], v[2], v[3]};
            }
            __syncthreads();
            for (int n = 0; n < nb; ++n) {
                float2 *ah = sAh + (n0 + n) * CH + ch;
                const float A2 = ah->x, carry = ah->y;
                float da[T], in[T];
                float hq = 0.f;
#pragma unroll
                for (int j = 0; j < Q; ++j) {
                    const float4 B4 =
                        *reinterpret_cast<const float4 *>(sB + n * CHUNK + (j * LANES + lane) * 4);
                    in[4 * j] = u[4 * j] * B4.x;
                    in[4 * j + 1] = u[4 * j + 1] * B4.y;
                    in[4 * j + 2] = u[4 * j + 2] * B4.z;
                    in[4 * j + 3] = u[4 * j + 3] * B4.w;
                }
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    da[i] = exp2_fast(s[i] * A2);
                    hq = __builtin_fmaf(da[i], hq, in[i]);
                }
                float P = exp2_fast(total * A2);
                // Lane 0 starts from the running state; then (P, Q) over the row.
                float hs = __builtin_fmaf(P, lane == 0 ? carry : 0.f, hq);
                hs = __builtin_fmaf(P, dpp0<kRowShr + 1>(hs), hs);
                P *= dpp0<kRowShr + 1>(P);
                hs = __builtin_fmaf(P, dpp0<kRowShr + 2>(hs), hs);
                P *= dpp0<kRowShr + 2>(P);
                hs = __builtin_fmaf(P, dpp0<kRowShr + 4>(hs), hs);
                P *= dpp0<kRowShr + 4>(P);
                hs = __builtin_fmaf(P, dpp0<kRowShr + 8>(hs), hs);
                // Lane l's state in is lane l-1's state out; lane 0 gets lane 15's: the next carry.
                const float turned = dpp0<kRowRor + 1>(hs);
                float h = lane == 0 ? carry : turned;
                if (lane == 0) ah->y = turned;
                if (a.checkpoints && live && t0 % SEQ_SCAN_CHECKPOINT == 0 && t0 < a.L)
                    a.checkpoints[(row * nck + t0 / SEQ_SCAN_CHECKPOINT) * a.N + n0 + n] = h;
#pragma unroll
                for (int j = 0; j < Q; ++j) {
                    const float4 C4 =
                        *reinterpret_cast<const float4 *>(sC + n * CHUNK + (j * LANES + lane) * 4);
                    h = __builtin_fmaf(da[4 * j], h, in[4 * j]);
                    acc[4 * j] = __builtin_fmaf(C4.x, h, acc[4 * j]);
                    h = __builtin_fmaf(da[4 * j + 1], h, in[4 * j + 1]);
                    acc[4 * j + 1] = __builtin_fmaf(C4.y, h, acc[4 * j + 1]);
                    h = __builtin_fmaf(da[4 * j + 2], h, in[4 * j + 2]);
                    acc[4 * j + 2] = __builtin_fmaf(C4.z, h, acc[4 * j + 2]);
                    h = __builtin_fmaf(da[4 * j + 3], h, in[4 * j + 3]);
                    acc[4 * j + 3] = __builtin_fmaf(C4.w, h, acc[4 * j + 3]);
                }
            }
        }
        if (live && t0 < a.L) {
            if (z) {
                float zv[T];
                load_row<E, T>(z, t0, len, zv);
#pragma unroll
                for (int i = 0; i < T; ++i) acc[i] *= zv[i] * sigmoid(zv[i]);
            }
#pragma unroll
            for (int i = 0; i < T; ++i) acc[i] = t0 + i < len ? acc[i] : 0.f;
            store_row<E, T>(y, t0, a.L, acc);
        }
    }
    if (live) {
        float zero[T];
#pragma unroll
        for (int i = 0; i < T; ++i) zero[i] = 0.f;
        for (int64_t t = c0 + lane * T; t < a.L; t += CHUNK) store_row<E, T>(y, t, a.L, zero);
    }
    if (a.state_out) {
        __syncthreads();
        for (int i = tid; i < a.N * CH; i += kThreads) {
            const int c = i / a.N, n = i % a.N;
            if (tile * CH + c < Dg)
                a.state_out[((int64_t)b * a.D + g * Dg + tile * CH + c) * a.N + n] =
                    sAh[n * CH + c].y;
        }
    }
}

template <class E>
struct ScanStep {
    View<E> x, dt, z, Bm, Cm, y;
    const float *A, *skip, *dt_bias;
    float *state;
    const int32_t *slots;
    int B, D, N, G, lines, softplus;
    int row_lanes;  // lanes on one channel's states, a power of two
};

// One position: the states are read and written once and everything else is
// 1/N of them.  A lane takes V consecutive states at a time (16 bytes for V = 4).
template <class E, int V>
__global__ __launch_bounds__(kThreads) void scan_step(ScanStep<E> a) {
    const int lane = threadIdx.x % a.row_lanes;
    const int d = blockIdx.x * (kThreads / a.row_lanes) + threadIdx.x / a.row_lanes;
    const int b = blockIdx.y;
    if (d >= a.D) return;
    const int slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.lines) {
        if (lane == 0) *a.y.row(b, d) = E::down(0.f);
        return;
    }
    const float raw = E::up(*a.dt.row(b, d)) + (a.dt_bias ? a.dt_bias[d] : 0.f);
    const float s = a.softplus ? softplus(raw) : raw;
    const float x = E::up(*a.x.row(b, d));
    const float u = s * x;
    const int64_t first = (int64_t)(d / (a.D / a.G)) * a.N;
    float *state = a.state + ((int64_t)slot * a.D + d) * a.N;
    const float *A = a.A + (int64_t)d * a.N;
    float sum = 0.f;
    for (int n = lane * V; n < a.N; n += a.row_lanes * V) {
        float h[V], Av[V];
        load_vec<F32, V>(state + n, h);
        load_vec<F32, V>(A + n, Av);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float Bv = E::up(*a.Bm.row(b, first + n + i));
            const float Cv = E::up(*a.Cm.row(b, first + n + i));
            h[i] = __builtin_fmaf(exp2_fast(s * (Av[i] * kLog2e)), h[i], u * Bv);
            sum = __builtin_fmaf(Cv, h[i], sum);
        }
        store_vec<F32, V>(state + n, h);
    }
    for (int m = 1; m < a.row_lanes; m *= 2) sum += lane_xor(sum, m);
    if (lane == 0) {
        float out = a.skip ? __builtin_fmaf(a.skip[d], x, sum) : sum;
        if (a.z.p) {
            const float z = E::up(*a.z.row(b, d));
            out *= z * sigmoid(z);
        }
        *a.y.row(b, d) = E::down(out);
    }
}

template <class E>
hipError_t forward(const state_scan_args &a, hipStream_t s) {
    constexpr int T = 8, CH = kWaves * 4;
    ScanFwd<E> k{view<E>(a.x), view<E>(a.dt), view<E>(a.z), view<E>(a.Bm), view<E>(a.Cm),
                 view<E>(a.y), a.A, a.skip, a.dt_bias, a.state_in, a.state_out, a.checkpoints,
                 a.lengths, a.B, a.D, a.L, a.N, a.G, (a.D / a.G + CH - 1) / CH, a.softplus};
    const int NP = (a.N + kNB - 1) / kNB * kNB;
    const size_t bytes = (2 * kNB * 16 * T + 2 * (size_t)NP * CH) * sizeof(float);
    scan_forward<E, T><<<dim3((unsigned)(a.G * k.tiles), (unsigned)a.B), kThreads, bytes, s>>>(k);
    return hipGetLastError();
}

template <class E>
hipError_t step(const state_scan_step_args &a, hipStream_t s) {
    ScanStep<E> k{view<E>(a.x), view<E>(a.dt), view<E>(a.z), view<E>(a.Bm), view<E>(a.Cm),
                  view<E>(a.y), a.A, a.skip, a.dt_bias, a.state, a.slots, a.B, a.D, a.N, a.G,
                  a.lines, a.softplus, 1};
    const int V = a.N % 4 == 0 ? 4 : 1;
    while (k.row_lanes < 16 && k.row_lanes * V < a.N) k.row_lanes *= 2;
    const int rows = kThreads / k.row_lanes;
    const dim3 grid((unsigned)((a.D + rows - 1) / rows), (unsigned)a.B);
    if (V == 4)
        scan_step<E, 4><<<grid, kThreads, 0, s>>>(k);
    else
        scan_step<E, 1><<<grid, kThreads, 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_forward(const state_scan_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? forward<F32>(a, s)
           : a.dtype == SEQ_BF16 ? forward<BF16>(a, s) : forward<F16>(a, s);
}
hipError_t launch_scan_step(const state_scan_step_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? step<F32>(a, s)
           : a.dtype == SEQ_BF16 ? step<BF16>(a, s) : step<F16>(a, s);
}

}  // namespace seq
