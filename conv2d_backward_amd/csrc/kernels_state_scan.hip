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
// What bounds it: for each (channel, state, position) one v_exp_f32 and five fp32
// instructions; the bytes (x, dt, z, y) are 1/N of that many elements.  A loop of
// those six on registers reaches 0.182 ps an element with 8 waves a SIMD.
// [1, 4096, 8192] bf16, N = 16: 178 us for that rate's 98; the lane scan, the steps
// and gates and the staging of B and C add 3.8 instructions to the six, and there
// are 4 waves a SIMD (their vector instructions, at 4 cycles each and 8 an
// exponential, make 0.89 of the time).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

// Floats of B, and as many of C, in LDS at once.  Rows of 64 lanes come through so
// many states between two waits only with more of them; with T = 16 the registers
// to carry them are not there (spilled, [2, 340, 3307] f32, N = 64, takes 166 us for 127).
constexpr int staged_floats(int lanes, int T) { return lanes == 64 && T == 8 ? 8192 : 4096; }

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

// A work-group: W waves, each 64/LANES rows (channels) of LANES lanes, each lane
// T consecutive positions of a chunk of LANES * T; NI states at a time, whose
// chains have nothing to do with each other.  NS waves share their rows, each
// with every NS-th group of NI states; their outputs meet in LDS.  LDS: B and C of
// NB states over the chunk (fp32, in the order the lanes read them), then A log2(e)
// and the running state of every (state, channel).
template <class E, int W, int LANES, int T, int NI, int NS, int OCC>
__global__ __launch_bounds__(64 * W, OCC) void scan_forward(ScanFwd<E> a) {
    constexpr int kThreads = 64 * W, CH = W / NS * 64 / LANES, CHUNK = LANES * T;
    constexpr int kStaged = staged_floats(LANES, T), NB = kStaged / CHUNK, Q = T / 4;
    static_assert(NB % (NI * NS) == 0, "whole groups of states");
    static_assert(NS == 1 || (W - W / NS) * 64 * T <= 2 * kStaged, "outputs fit where B and C were");
    extern __shared__ float lds[];
    float *sB = lds, *sC = lds + kStaged;
    float2 *sAh = reinterpret_cast<float2 *>(lds + 2 * kStaged);  // [N][CH]
    const int tid = threadIdx.x, lane = tid % LANES, ch = tid / LANES % CH;
    const int share = tid / LANES / CH;
    const int Dg = a.D / a.G;
    const int g = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles, b = blockIdx.y;
    const int in_group = tile * CH + ch;
    const bool live = in_group < Dg;
    const int d = g * Dg + (live ? in_group : Dg - 1);
    const int len = length_of(a.lengths, b, a.L);
    const int64_t row = (int64_t)b * a.D + d;
    const int NP = (a.N + NB - 1) / NB * NB;
    for (int i = tid; i < NP * CH; i += kThreads) {
        const int n = i / CH, c = i % CH;
        const int dc = g * Dg + std::min(tile * CH + c, Dg - 1);
        float2 v = {0.f, 0.f};
        if (n < a.N) {
            v.x = decay_rate(a.A[(int64_t)dc * a.N + n]);
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
    // B and C of the next group of states travel while this one's chains run.
    constexpr int PRE = kStaged / 8 / kThreads;
    Octet<E> next[2 * PRE];
    const auto prefetch = [&](int c, int n0) {
#pragma unroll
        for (int k = 0; k < PRE; ++k) {
            const int o = k * kThreads + tid, n = n0 + o / (CHUNK / 8);
            const int t = c + o % (CHUNK / 8) * 8;
            const int left = n < a.N ? len - t : 0;  // past N: zeros
            const int64_t state = (int64_t)g * a.N + n;
            next[k].load(a.Bm.row(b, state) + t, left);
            next[PRE + k].load(a.Cm.row(b, state) + t, left);
        }
    };
    if (end > 0) prefetch(0, 0);
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
            for (int i = 0; i < T; ++i) s[i] += bias;
            if (a.softplus) {
#pragma unroll
                for (int i = 0; i < T; ++i) s[i] = softplus(s[i]);
            }
            if (c0 + CHUNK > len) {
#pragma unroll
                for (int i = 0; i < T; ++i)  // 0: the state passes unchanged
                    s[i] = len - t0 > i ? s[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < T; ++i) {
                u[i] = s[i] * xv[i];
                acc[i] = share == 0 ? skip * xv[i] : 0.f;
                total += s[i];
            }
        }
        const bool mark = a.checkpoints && live && t0 % SEQ_SCAN_CHECKPOINT == 0 && t0 < a.L;
        for (int n0 = 0; n0 < a.N; n0 += NB) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < PRE; ++k) stage_octet<E, LANES, T>(sB, k * kThreads + tid, next[k]);
#pragma unroll
            for (int k = 0; k < PRE; ++k)
                stage_octet<E, LANES, T>(sC, k * kThreads + tid, next[PRE + k]);
            __syncthreads();
            const bool more = n0 + NB < a.N;
            if (more || c0 + CHUNK < end)
                prefetch(more ? c0 : c0 + CHUNK, more ? n0 + NB : 0);
            const int nb = std::min(NB, a.N - n0);
            for (int n = share * NI; n < nb; n += NS * NI) {
                float2 *ah = sAh + (n0 + n) * CH + ch;
                const float *pB = sB + n * CHUNK + lane * 4, *pC = sC + n * CHUNK + lane * 4;
                float da[NI][T], in[NI][T], h[NI], P[NI], carry[NI];
#pragma unroll
                for (int k = 0; k < NI; ++k) {
                    const float2 v = ah[k * CH];
                    carry[k] = v.y;
                    P[k] = exp2_fast(total * v.x);
#pragma unroll
                    for (int j = 0; j < Q; ++j) {
                        const float4 B4 =
                            *reinterpret_cast<const float4 *>(pB + k * CHUNK + j * LANES * 4);
                        const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            da[k][4 * j + i] = exp2_fast(s[4 * j + i] * v.x);
                            in[k][4 * j + i] = u[4 * j + i] * Bv[i];
                        }
                    }
                    // Lane 0 starts from the running state.
                    h[k] = lane == 0 ? carry[k] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < T; ++i)
#pragma unroll
                    for (int k = 0; k < NI; ++k)
                        h[k] = __builtin_fmaf(da[k][i], h[k], in[k][i]);
                // Lane l's state in is lane l-1's state out; lane 0 gets the last lane's, the
                // next chunk's running state.
                float turned[NI];
                scan_lanes<LANES>(h, P, turned);
#pragma unroll
                for (int k = 0; k < NI; ++k) {
                    h[k] = lane == 0 ? carry[k] : turned[k];
                    if (lane == 0) ah[k * CH].y = turned[k];
                    if (mark && n0 + n + k < a.N)
                        a.checkpoints[(row * nck + t0 / SEQ_SCAN_CHECKPOINT) * a.N + n0 + n + k] =
                            h[k];
                }
#pragma unroll
                for (int j = 0; j < Q; ++j)
#pragma unroll
                    for (int k = 0; k < NI; ++k) {
                        const float4 C4 =
                            *reinterpret_cast<const float4 *>(pC + k * CHUNK + j * LANES * 4);
                        const float Cv[4] = {C4.x, C4.y, C4.z, C4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[k] = __builtin_fmaf(da[k][4 * j + i], h[k], in[k][4 * j + i]);
                            acc[4 * j + i] = __builtin_fmaf(Cv[i], h[k], acc[4 * j + i]);
                        }
                    }
            }
        }
        if constexpr (NS > 1) {
            __syncthreads();
            float4 *meet = reinterpret_cast<float4 *>(lds) + (share - 1) * Q * (CH * LANES) +
                           tid % (CH * LANES);
            if (share > 0) {
#pragma unroll
                for (int j = 0; j < Q; ++j)
                    meet[j * CH * LANES] =
                        float4{acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]};
            }
            __syncthreads();
            if (share == 0) {
                for (int k = 1; k < NS; ++k) {
                    const float4 *from = meet + k * Q * (CH * LANES);
#pragma unroll
                    for (int j = 0; j < Q; ++j) {
                        const float4 v = from[j * CH * LANES];
                        acc[4 * j] += v.x;
                        acc[4 * j + 1] += v.y;
                        acc[4 * j + 2] += v.z;
                        acc[4 * j + 3] += v.w;
                    }
                }
            }
        }
        if (live && t0 < a.L && share == 0) {
            if (z) {
                float zv[T];
                load_row<E, T>(z, t0, len, zv);
#pragma unroll
                for (int i = 0; i < T; ++i) acc[i] *= zv[i] * sigmoid(zv[i]);
            }
            if (c0 + CHUNK > len) {
#pragma unroll
                for (int i = 0; i < T; ++i) acc[i] = len - t0 > i ? acc[i] : 0.f;
            }
            store_row<E, T>(y, t0, a.L, acc);
        }
    }
    if (live && share == 0) {
        float zero[T];
#pragma unroll
        for (int i = 0; i < T; ++i) zero[i] = 0.f;
        for (int t = c0 + lane * T; t < a.L; t += CHUNK) store_row<E, T>(y, t, a.L, zero);
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

constexpr int kThreads = 256;  // of scan_step

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
// 1/N of them, so memory bounds it.  A lane takes V consecutive states at a time
// (16 bytes for V = 4) of R channels, which share B and C; the R channels' states
// are on their way together.
template <class E, int V, int R>
__global__ __launch_bounds__(kThreads) void scan_step(ScanStep<E> a) {
    const int lane = threadIdx.x % a.row_lanes, rows = kThreads / a.row_lanes;
    const int d0 = blockIdx.x * rows * R + threadIdx.x / a.row_lanes;
    const int b = blockIdx.y, Dg = a.D / a.G;
    const int slot = a.slots ? a.slots[b] : b;
    const bool dead = slot < 0 || slot >= a.lines;
    float s[R], u[R], sum[R];
    if (!dead) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = std::min(d0 + r * rows, a.D - 1);
            const float raw = E::up(*a.dt.row(b, d)) + (a.dt_bias ? a.dt_bias[d] : 0.f);
            s[r] = a.softplus ? softplus(raw) : raw;
            u[r] = s[r] * E::up(*a.x.row(b, d));
            sum[r] = 0.f;
        }
        for (int n = lane * V; n < a.N; n += a.row_lanes * V) {
            float h[R][V], Av[R][V];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int d = std::min(d0 + r * rows, a.D - 1);
                load_vec<F32, V>(a.state + ((int64_t)slot * a.D + d) * a.N + n, h[r]);
                load_vec<F32, V>(a.A + (int64_t)d * a.N + n, Av[r]);
            }
            float Bv[V], Cv[V];
            int of = -1;  // the group whose B and C are there
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int d = std::min(d0 + r * rows, a.D - 1), g = R > 1 && a.G == 1 ? 0 : d / Dg;
                if (g != of) {
                    const int64_t first = (int64_t)g * a.N + n;
                    if (V > 1 && a.Bm.channel == 1 && a.Cm.channel == 1) {
                        load_vec<E, V>(a.Bm.row(b, first), Bv);
                        load_vec<E, V>(a.Cm.row(b, first), Cv);
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            Bv[i] = E::up(*a.Bm.row(b, first + i));
                            Cv[i] = E::up(*a.Cm.row(b, first + i));
                        }
                    }
                    of = g;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    h[r][i] = __builtin_fmaf(exp2_fast(s[r] * (Av[r][i] * kLog2e)), h[r][i],
                                             u[r] * Bv[i]);
                    sum[r] = __builtin_fmaf(Cv[i], h[r][i], sum[r]);
                }
                if (d0 + r * rows < a.D)
                    store_vec<F32, V>(a.state + ((int64_t)slot * a.D + d) * a.N + n, h[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int d = d0 + r * rows;
        if (!dead)
            for (int m = 1; m < a.row_lanes; m *= 2) sum[r] += lane_xor(sum[r], m);
        if (lane || d >= a.D) continue;
        float out = 0.f;
        if (!dead) {
            out = a.skip ? __builtin_fmaf(a.skip[d], E::up(*a.x.row(b, d)), sum[r]) : sum[r];
            if (a.z.p) {
                const float z = E::up(*a.z.row(b, d));
                out *= z * sigmoid(z);
            }
        }
        *a.y.row(b, d) = E::down(out);
    }
}

template <class E, int W, int LANES, int T, int NI, int NS, int OCC>
hipError_t forward(const state_scan_args &a, hipStream_t s) {
    constexpr int kStaged = staged_floats(LANES, T);
    constexpr int CH = W / NS * 64 / LANES, NB = kStaged / (LANES * T);
    ScanFwd<E> k{view<E>(a.x), view<E>(a.dt), view<E>(a.z), view<E>(a.Bm), view<E>(a.Cm),
                 view<E>(a.y), a.A, a.skip, a.dt_bias, a.state_in, a.state_out, a.checkpoints,
                 a.lengths, a.B, a.D, a.L, a.N, a.G, (a.D / a.G + CH - 1) / CH, a.softplus};
    const int NP = (a.N + NB - 1) / NB * NB;
    const size_t bytes = (2 * kStaged + 2 * (size_t)NP * CH) * sizeof(float);
    if (bytes > 64 * 1024) {
        hipError_t e =
            hipFuncSetAttribute((const void *)scan_forward<E, W, LANES, T, NI, NS, OCC>,
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != hipSuccess) return e;
    }
    scan_forward<E, W, LANES, T, NI, NS, OCC>
        <<<dim3((unsigned)(a.G * k.tiles), (unsigned)a.B), 64 * W, bytes, s>>>(k);
    return hipGetLastError();
}

// How the work is dealt: waves of a work-group, lanes of a row, positions of a
// lane, waves that share a row's states.
struct Deal {
    int W, lanes, T, shares;
};
constexpr Deal kDeals[] = {{8, 64, 16, 1}, {8, 64, 16, 2}, {8, 64, 16, 4}, {8, 64, 8, 1},
                           {8, 64, 8, 2},  {8, 64, 8, 4},  {4, 16, 16, 1}, {4, 16, 4, 1},
                           {8, 16, 8, 2},  {8, 16, 8, 4}};
constexpr int kDealCount = sizeof(kDeals) / sizeof(kDeals[0]);

// The deal with the least time by a count of issue slots.  Per chunk a wave has
//   N / shares * (7.6 T + 15 (64 lanes: 18 for the lane scan))   its chains
//   + N' T lanes / (16 W)   its part of B and C, of N' states: N in whole stages
//   + 20 T                  steps, gates, stores
// and 2560 waves, 2.5 a SIMD, run as fast as one: more take their turns; a stage
// costs 100 more for its waits.  At 29 shapes the choice is within 3% of the
// fastest on average and 19% at worst.  Measured (us, in the order above):
// [1, 4096, 8192] bf16 N 16 180 / 214 / 284 / 200 / 230 / 313 / 277 / 681 / 328 / 311,
// [1, 1024, 8192] bf16 N 16 107 / 78 / 76 / 122 / 79 / 85 / 252 / 628 / 299 / 221,
// [2, 340, 3307] f32 N 64 199 / 131 / 127 / 185 / 114 / 114 / 345 / 623 / 310 / 187,
// [5, 1825, 3409] f32 N 8 186 / 219 / 296 / 162 / 188 / 280 / 193 / 268 / 237 / 285,
// [5, 1000, 301] bf16 N 16 39 / 43 / 62 / 23 / 26 / 37 / 26 / 30 / 24 / 27,
// [16, 1024, 60] bf16 N 16 88 / 119 / 179 / 49 / 66 / 103 / 26 / 12 / 18 / 25.
int pick_deal(const state_scan_args &a) {
    int best = 0;
    double least = 0;
    for (int i = 0; i < kDealCount; ++i) {
        const Deal &v = kDeals[i];
        const int channels = v.W / v.shares * 64 / v.lanes, chunk = v.lanes * v.T;
        const int NB = staged_floats(v.lanes, v.T) / chunk, stages = (a.N + NB - 1) / NB;
        const int64_t tiles = (a.D / a.G + channels - 1) / channels;
        const double waves = (double)a.B * a.G * tiles * v.W;
        const double work = (double)a.N / v.shares * (7.6 * v.T + (v.lanes == 64 ? 18 : 15)) +
                            (double)stages * NB * v.T * v.lanes / (16 * v.W) + 20. * v.T;
        const double cost = ((a.L + chunk - 1) / chunk) *
                            (work * std::max(1., waves / 2560) + 100. * stages);
        if (i == 0 || cost < least) best = i, least = cost;
    }
    return best;
}

template <class E>
hipError_t forward_any(const state_scan_args &a, hipStream_t s) {
    switch (pick_deal(a)) {
        case 0: return forward<E, 8, 64, 16, 1, 1, 4>(a, s);
        case 1: return forward<E, 8, 64, 16, 1, 2, 4>(a, s);
        case 2: return forward<E, 8, 64, 16, 1, 4, 4>(a, s);
        case 3: return forward<E, 8, 64, 8, 1, 1, 4>(a, s);
        case 4: return forward<E, 8, 64, 8, 1, 2, 4>(a, s);
        case 5: return forward<E, 8, 64, 8, 1, 4, 4>(a, s);
        case 6: return forward<E, 4, 16, 16, 1, 1, 3>(a, s);
        case 7: return forward<E, 4, 16, 4, 2, 1, 4>(a, s);
        case 8: return forward<E, 8, 16, 8, 1, 2, 4>(a, s);
        default: return forward<E, 8, 16, 8, 1, 4, 4>(a, s);
    }
}

template <class E>
hipError_t step(const state_scan_step_args &a, hipStream_t s) {
    ScanStep<E> k{view<E>(a.x), view<E>(a.dt), view<E>(a.z), view<E>(a.Bm), view<E>(a.Cm),
                  view<E>(a.y), a.A, a.skip, a.dt_bias, a.state, a.slots, a.B, a.D, a.N, a.G,
                  a.lines, a.softplus, 1};
    const int V = a.N % 4 == 0 ? 4 : 1;
    while (k.row_lanes < 16 && k.row_lanes * V < a.N) k.row_lanes *= 2;
    // Two channels a lane where half the work-groups still fill the chip many times
    // over ([256, 4096], N = 16: 32.3 us, 4.4 TB/s; one 36.6, four 37.6), one where
    // latency counts.
    const int64_t rows = kThreads / k.row_lanes, groups = (a.D + rows - 1) / rows * a.B;
    const int R = groups >= 8192 ? 2 : 1;
    const dim3 grid((unsigned)((a.D + rows * R - 1) / (rows * R)), (unsigned)a.B);
    const auto kernel = V == 4 ? (R == 2 ? scan_step<E, 4, 2> : scan_step<E, 4, 1>)
                               : (R == 2 ? scan_step<E, 1, 2> : scan_step<E, 1, 1>);
    kernel<<<grid, kThreads, 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

int64_t scan_forward_items(const state_scan_args &a) {
    // A work-group has two channels at least and eight waves at most.
    const int64_t most = ((int64_t)a.D + a.G) / 2 * 512;
    if (most >> 32 == 0) return most;
    const Deal &v = kDeals[pick_deal(a)];
    const int channels = v.W / v.shares * 64 / v.lanes;
    return (int64_t)a.G * ((a.D / a.G + channels - 1) / channels) * 64 * v.W;
}
void scan_forward_plan(const state_scan_args &a, char *buf, size_t len) {
    const Deal &v = kDeals[pick_deal(a)];
    std::snprintf(buf, len, "waves=%d lanes=%d positions=%d shares=%d staged=%d", v.W, v.lanes, v.T,
                  v.shares, staged_floats(v.lanes, v.T) / (v.lanes * v.T));
}
hipError_t launch_scan_forward(const state_scan_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? forward_any<F32>(a, s)
           : a.dtype == SEQ_BF16 ? forward_any<BF16>(a, s) : forward_any<F16>(a, s);
}
hipError_t launch_scan_step(const state_scan_step_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? step<F32>(a, s)
           : a.dtype == SEQ_BF16 ? step<BF16>(a, s) : step<F16>(a, s);
}

}  // namespace seq
