// kernels_gated_scan.hip -- the gated recurrence: prompts, its gradients, and one
// position of it against a state cache.
//
// h_t = a_t h_{t-1} + m_t e_t with a = exp(A sr), sr = sigmoid(r + r_bias), m =
// sqrt(1 - a^2) and e = sigmoid(i + i_bias) x is a chain along the positions, and
// maps h -> P h + Q compose.  A lane takes 8 consecutive positions, runs their chain
// once from 0 for its map, 16 lanes (a DPP row) combine their maps in four steps, the
// rows of a wave and the waves of a work-group theirs one after the other, and each
// lane runs its chain again from the state it then knows.  The gradient q of h is the
// same chain from the right, c -> a_t (gy_t + c), whose maps have the same P; h is run
// again from the checkpoint that the forward call leaves every 128 positions, one
// for each row of lanes.
//
// What bounds it: memory, with the instructions close behind.  A position has 5 activations
// forward and 9 backward, and some 40 and 70 fp32 instructions beside 8 of the slow ones
// (exponentials, roots, reciprocals).  With z, operands from memory (the same ones again, of which the
// memory-side cache has a part): bf16 [1, 4096, 8192] forward 70 us, 4.8 TB/s (67), backward 123, 4.9
// TB/s (123); [4, 2048, 2048] 40 (33) and 76 (66); f32 [2, 602, 777] 9.7 (6.1) and 17.4 (13.0), the
// latency of a chunk.  Backward, a SIMD has three waves of 16-bit types (150 to 158 registers) and of
// float32 with one wave a row (166), two of float32 with more (170 to 178); 16 waves a row are held to
// 128 registers, for which 16-bit types spill 2 and float32 29.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

constexpr int T = 8;            // positions of a lane
constexpr int kRow = 16 * T;    // positions of a row of lanes
static_assert(kRow == SEQ_SCAN_CHECKPOINT, "a checkpoint for every row of lanes");

// 1 - a^2 loses all digits in fp32 where a is near 1, which is where such layers work (u is
// -1e-4 to -0.1).  It is -2 a sinh(u), and sinh(u) / u has a short series in u^2: up to u^6 / 5040
// the next term is 1e-8 of it at |u| = 0.5.  Below that 1 - a^2 itself has lost less than a bit.
// Everything is in l = u log2(e), so that no u is needed.
struct Decay {
    float a, n;  // e^u, 1 - e^2u
};
__device__ __forceinline__ Decay decay(float sr, float A2) {
    constexpr float k = kLn2 * kLn2;
    const float l = sr * A2, w = l * l;
    Decay d;
    d.a = exp2_fast(l);
    float s = __builtin_fmaf(w, -2 * kLn2 * k * k * k / 5040, -2 * kLn2 * k * k / 120);
    s = __builtin_fmaf(w, s, -2 * kLn2 * k / 6);
    s = __builtin_fmaf(w, s, -2 * kLn2);
    const float near = d.a * (l * s), far = __builtin_fmaf(-d.a, d.a, 1.f);
    d.n = l > -0.5f * kLog2e ? near : far;
    return d;
}
// sigmoid(v + bias), the bias times -log2(e).
__device__ __forceinline__ float gate(float v, float bias) {
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(__builtin_fmaf(v, -kLog2e, bias)));
}

template <int CTRL>
__device__ __forceinline__ float dpp(float old, float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        __builtin_bit_cast(int, old), __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
constexpr int kRowShl1 = 0x101, kRowShr1 = 0x111, kRowFirst = 0x150, kRowLast = 0x15f;
// Of four lanes, each other's: the lane that each takes from.
constexpr int kQuad3012 = 0x93, kQuad1230 = 0x39, kQuad2301 = 0x4e, kQuadFirst = 0x00, kQuadLast = 0xff;

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Inclusive maps of 16 lanes (or of 4), from the first lane (or, BACK, from the last).
template <int LANES, bool BACK>
__device__ __forceinline__ void scan_row(float &P, float &Q) {
    if constexpr (LANES == 4) {
        const unsigned lane = BACK ? 3 - threadIdx.x % 4 : threadIdx.x % 4;
        const float p1 = dpp<BACK ? kQuad1230 : kQuad3012>(0.f, P), q1 = dpp<BACK ? kQuad1230 : kQuad3012>(0.f, Q);
        Q = lane >= 1 ? __builtin_fmaf(P, q1, Q) : Q;
        P = lane >= 1 ? P * p1 : P;
        const float p2 = dpp<kQuad2301>(0.f, P), q2 = dpp<kQuad2301>(0.f, Q);
        Q = lane >= 2 ? __builtin_fmaf(P, q2, Q) : Q;
        P = lane >= 2 ? P * p2 : P;
    } else if constexpr (BACK)
        asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP1, "shl") SEQ_STEP1("row_shl:8" SEQ_ALL)
            "s_nop 0" : "+v"(Q), "+v"(P));
    else
        asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP1, "shr") SEQ_STEP1("row_shr:8" SEQ_ALL)
            "s_nop 0" : "+v"(Q), "+v"(P));
}

// The value that enters each lane, from its map (P, Q) and the value `start` that enters
// the row of W * LANES lanes; start becomes what leaves it.  W > 1: `meet` has W maps of the
// row, which nothing else uses before the barrier after the next one.
template <int LANES, int W, bool BACK>
__device__ __forceinline__ float enter(float P, float Q, float &start, float2 *meet) {
    scan_row<LANES, BACK>(P, Q);
    if constexpr (LANES == 4) {
        static_assert(W == 1, "rows of 4 lanes are in one wave");
        const bool end = threadIdx.x % 4 == (BACK ? 3 : 0);
        const float p = dpp<BACK ? kQuad1230 : kQuad3012>(0.f, P), q = dpp<BACK ? kQuad1230 : kQuad3012>(0.f, Q);
        const float into = end ? start : __builtin_fmaf(p, start, q);
        const float all_P = dpp<BACK ? kQuadFirst : kQuadLast>(0.f, P);
        const float all_Q = dpp<BACK ? kQuadFirst : kQuadLast>(0.f, Q);
        start = __builtin_fmaf(all_P, start, all_Q);
        return into;
    }
    const float before_P = BACK ? dpp<kRowShl1>(1.f, P) : dpp<kRowShr1>(1.f, P);
    const float before_Q = BACK ? dpp<kRowShl1>(0.f, Q) : dpp<kRowShr1>(0.f, Q);
    if constexpr (LANES == 16) {
        static_assert(W == 1, "rows of 16 lanes are in one wave");
        const float into = __builtin_fmaf(before_P, start, before_Q);
        const float all_P = BACK ? dpp<kRowFirst>(0.f, P) : dpp<kRowLast>(0.f, P);
        const float all_Q = BACK ? dpp<kRowFirst>(0.f, Q) : dpp<kRowLast>(0.f, Q);
        start = __builtin_fmaf(all_P, start, all_Q);
        return into;
    } else if constexpr (LANES == 64) {
        // The rows in the chain's order.
        float rP[4], rQ[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int lane = BACK ? 48 - 16 * k : 16 * k + 15;
            rP[k] = lane_value(P, lane);
            rQ[k] = lane_value(Q, lane);
        }
        float mine = start;
        if constexpr (W > 1) {
            float wP = rP[0], wQ = rQ[0];
#pragma unroll
            for (int k = 1; k < 4; ++k) {
                wQ = __builtin_fmaf(rP[k], wQ, rQ[k]);
                wP *= rP[k];
            }
            const int wave = threadIdx.x / 64 % W;
            if (threadIdx.x % 64 == 0) meet[wave] = float2{wP, wQ};
            __syncthreads();
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const int w = BACK ? W - 1 - k : k;
                const float2 v = meet[w];
                if (w == wave) mine = start;
                start = __builtin_fmaf(v.x, start, v.y);
            }
        }
        const int place = threadIdx.x % 64 / 16, row = BACK ? 3 - place : place;
        float s = mine, at = mine;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            s = __builtin_fmaf(rP[k], s, rQ[k]);
            if (row > k) at = s;
        }
        if constexpr (W == 1) start = __builtin_fmaf(rP[3], s, rQ[3]);
        return __builtin_fmaf(before_P, at, before_Q);
    }
}

template <class E>
struct GatedFwd {
    View<E> x, r, i, z, y;
    const float *A, *r_bias, *i_bias, *state_in;
    float *state_out, *checkpoints;
    const int32_t *lengths;
    int rows, D, L, marks;
};

// Rows of a work-group: one of W waves, or, W = 1, four waves with 64 / LANES rows each.
template <int LANES, int W>
constexpr int kThreadsOf = W == 1 ? 256 : 64 * W;
template <int LANES, int W>
constexpr int kRowsOf = kThreadsOf<LANES, W> / (LANES * W);

template <class E, int LANES, int W>
__global__ __launch_bounds__((kThreadsOf<LANES, W>)) void gated_forward(GatedFwd<E> a) {
    constexpr int CHUNK = LANES * W * T, ROWS = kRowsOf<LANES, W>;
    __shared__ float2 meet[2][W];
    const int lane = threadIdx.x % (LANES * W);
    const int row = blockIdx.x * ROWS + threadIdx.x / (LANES * W);
    if (row >= a.rows) return;  // (W > 1: one row, all or none)
    const int b = row / a.D, d = row - b * a.D;
    const int len = length_of(a.lengths, b, a.L);
    const float A2 = decay_rate(a.A[d]);
    const float r_bias = a.r_bias ? a.r_bias[d] * -kLog2e : 0.f;
    const float i_bias = a.i_bias ? a.i_bias[d] * -kLog2e : 0.f;
    const auto *x = a.x.row(b, d), *r = a.r.row(b, d), *i = a.i.row(b, d);
    const auto *z = a.z.p ? a.z.row(b, d) : nullptr;
    auto *y = a.y.row(b, d);
    float state = a.state_in ? a.state_in[row] : 0.f;
    float *marks = a.checkpoints ? a.checkpoints + (int64_t)row * a.marks : nullptr;
    Octet<E> nx, nr, ni, nz;
    const auto prefetch = [&](int t) {
        nx.load(x + t, len - t);
        nr.load(r + t, len - t);
        ni.load(i + t, len - t);
        if (z) nz.load(z + t, len - t);
    };
    if (len > 0) prefetch(lane * T);
    int c0 = 0;
    for (int turn = 0; c0 < len; c0 += CHUNK, turn ^= 1) {
        const int t0 = c0 + lane * T;
        float av[T], in[T], f[T], P = 1.f, Q = 0.f;
#pragma unroll
        for (int k = 0; k < T; ++k) {
            const float sr = gate(nr.at(k), r_bias), si = gate(ni.at(k), i_bias);
            const Decay v = decay(sr, A2);
            av[k] = v.a;
            in[k] = __builtin_amdgcn_sqrtf(v.n) * (si * nx.at(k));
            if (z) f[k] = nz.at(k) * sigmoid(nz.at(k));
        }
        if (c0 + CHUNK > len) {
#pragma unroll
            for (int k = 0; k < T; ++k) {  // beyond the length the state passes unchanged
                av[k] = len - t0 > k ? av[k] : 1.f;
                in[k] = len - t0 > k ? in[k] : 0.f;
            }
        }
        if (c0 + CHUNK < len) prefetch(t0 + CHUNK);
#pragma unroll
        for (int k = 0; k < T; ++k) {
            Q = __builtin_fmaf(av[k], Q, in[k]);
            P *= av[k];
        }
        float h = enter<LANES, W, false>(P, Q, state, meet[turn]);
        if (marks && t0 % SEQ_SCAN_CHECKPOINT == 0 && t0 < a.L)
            marks[t0 / SEQ_SCAN_CHECKPOINT] = h;
        float out[T];
#pragma unroll
        for (int k = 0; k < T; ++k) {
            h = __builtin_fmaf(av[k], h, in[k]);
            out[k] = z ? h * f[k] : h;
        }
        if (c0 + CHUNK > len) {
#pragma unroll
            for (int k = 0; k < T; ++k) out[k] = len - t0 > k ? out[k] : 0.f;
        }
        if (t0 < a.L) store_row<E, T>(y, t0, a.L, out);
    }
    float zero[T];
#pragma unroll
    for (int k = 0; k < T; ++k) zero[k] = 0.f;
    for (int t = c0 + lane * T; t < a.L; t += CHUNK) {
        store_row<E, T>(y, t, a.L, zero);
        if (marks && t % SEQ_SCAN_CHECKPOINT == 0) marks[t / SEQ_SCAN_CHECKPOINT] = state;
    }
    if (a.state_out && lane == 0) a.state_out[row] = state;
}

template <class E>
struct GatedBwd {
    View<E> gout, x, r, i, z, dx, dr, di, dz;
    const float *A, *r_bias, *i_bias, *checkpoints, *gstate;
    float *dA, *dr_bias, *di_bias;
    float *params;  // [B][D][3], where a work-group has not all batch items of its channels
    float *dstate;
    const int32_t *lengths;
    int D, L, marks;
    int channels, items;  // of a work-group: items of the batch, each with these channels
};

// A work-group has some channels of all batch items, where those are few: then the
// parameters' sums meet in LDS and need no second kernel ([2, 602, 777] f32: 14.8 -> 12.8 us).
// Else it has them of one, and `gated_join` sums over the batch.
template <class E, int LANES, int W>
__global__ __launch_bounds__((W > 8 ? 1024 : 512)) void gated_backward(GatedBwd<E> a) {
    constexpr int CHUNK = LANES * W * T;
    constexpr int kH = LANES == 4 ? 4 : 16;   // lanes that run h again from a checkpoint together
    __shared__ float2 meet[2][16];
    __shared__ float sums[1024 / (LANES * W)][3];
    const int lane = threadIdx.x % (LANES * W), own = threadIdx.x / (LANES * W);
    const int b = blockIdx.y * a.items + own / a.channels;
    const int wanted = blockIdx.x * a.channels + own % a.channels;
    const bool live = wanted < a.D;   // (a row of no channel reads and writes nothing)
    const int d = live ? wanted : a.D - 1;
    const int64_t row = (int64_t)b * a.D + d;
    const int len = live ? length_of(a.lengths, b, a.L) : 0, L = live ? a.L : 0;
    const float A2 = decay_rate(a.A[d]), A = A2 * kLn2;
    const float r_bias = a.r_bias ? a.r_bias[d] * -kLog2e : 0.f;
    const float i_bias = a.i_bias ? a.i_bias[d] * -kLog2e : 0.f;
    const auto *x = a.x.row(b, d), *r = a.r.row(b, d), *i = a.i.row(b, d), *g = a.gout.row(b, d);
    const auto *z = a.z.p ? a.z.row(b, d) : nullptr;
    auto *dx = a.dx.row(b, d), *dr = a.dr.row(b, d), *di = a.di.row(b, d);
    auto *dz = z ? a.dz.row(b, d) : nullptr;
    const float *marks = a.checkpoints + row * a.marks;
    float back = a.gstate && live ? a.gstate[row] : 0.f;  // the gradient that comes from behind
    float sum_A = 0.f, sum_r = 0.f, sum_i = 0.f;
    int chunks = (len + CHUNK - 1) / CHUNK;
    if constexpr (W > 1) {   // the same number of barriers for all rows
        for (int k = 0; k < a.items; ++k)
            chunks = std::max(chunks, (length_of(a.lengths, blockIdx.y * a.items + k, a.L) + CHUNK - 1) / CHUNK);
    }
    Octet<E> nx, nr, ni, nz, ng;
    float next_h = 0.f;
    const auto prefetch = [&](int t) {
        nx.load(x + t, len - t);
        nr.load(r + t, len - t);
        ni.load(i + t, len - t);
        ng.load(g + t, len - t);
        if (z) nz.load(z + t, len - t);
        next_h = 0.f;
        if (lane % kH == 0 && t < len) next_h = marks[t / SEQ_SCAN_CHECKPOINT];
    };
    {
        float zero[T];
#pragma unroll
        for (int k = 0; k < T; ++k) zero[k] = 0.f;
        for (int t = chunks * CHUNK + lane * T; t < L; t += CHUNK) {
            store_row<E, T>(dx, t, L, zero);
            store_row<E, T>(dr, t, L, zero);
            store_row<E, T>(di, t, L, zero);
            if (z) store_row<E, T>(dz, t, L, zero);
        }
    }
    if (chunks > 0) prefetch((chunks - 1) * CHUNK + lane * T);
    for (int c = chunks - 1, turn = 0; c >= 0; --c, turn ^= 1) {
        const int c0 = c * CHUNK, t0 = c0 + lane * T;
        float av[T], m[T], inv[T], si[T], sr[T], e[T], gy[T], slope[T], h = next_h, P = 1.f, Q = 0.f;
#pragma unroll
        for (int k = 0; k < T; ++k) {
            sr[k] = gate(nr.at(k), r_bias);
            si[k] = gate(ni.at(k), i_bias);
            const Decay v = decay(sr[k], A2);
            av[k] = v.a;
            // 1 / m; where a is 1 the normaliser's slope, infinite there, counts as 0 (and
            // below the normal range, whose root v_sqrt_f32 too takes for 0).  A rate above 0
            // has no root: NaN, as in the forward call.
            inv[k] = __builtin_fabsf(v.n) < 1.17549435e-38f ? 0.f : __builtin_amdgcn_rsqf(v.n);
            m[k] = v.n * inv[k];
            e[k] = si[k] * nx.at(k);
            gy[k] = ng.at(k);
            if (z) {
                const float sz = sigmoid(nz.at(k));
                slope[k] = gy[k] * (sz * __builtin_fmaf(nz.at(k), 1.f - sz, 1.f));
                gy[k] *= nz.at(k) * sz;
            }
        }
        if (c0 + CHUNK > len) {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const bool in = len - t0 > k;
                av[k] = in ? av[k] : 1.f;
                m[k] = in ? m[k] : 0.f;
                inv[k] = in ? inv[k] : 0.f;
                e[k] = in ? e[k] : 0.f;
                gy[k] = in ? gy[k] : 0.f;
            }
        }
        if (c > 0) prefetch(t0 - CHUNK);
        // h again, from the checkpoint before the row of lanes.
#pragma unroll
        for (int k = 0; k < T; ++k) {
            Q = __builtin_fmaf(av[k], Q, m[k] * e[k]);
            P *= av[k];
        }
        {
            float at = dpp<kH == 4 ? kQuadFirst : kRowFirst>(0.f, h), row_P = P;
            h = enter<kH, 1, false>(row_P, Q, at, nullptr);
        }
        float before[T];  // h before the position
#pragma unroll
        for (int k = 0; k < T; ++k) {
            before[k] = h;
            h = __builtin_fmaf(av[k], h, m[k] * e[k]);
            if (z) slope[k] *= h;
        }
        if (z && t0 < L) {
            if (c0 + CHUNK > len) {
#pragma unroll
                for (int k = 0; k < T; ++k) slope[k] = len - t0 > k ? slope[k] : 0.f;
            }
            store_row<E, T>(dz, t0, L, slope);
        }
        Q = 0.f;
#pragma unroll
        for (int k = T - 1; k >= 0; --k) Q = av[k] * (gy[k] + Q);
        float q = enter<LANES, W, true>(P, Q, back, meet[turn] + threadIdx.x / 64 / W * W);
        float odx[T], odr[T], odi[T];
#pragma unroll
        for (int k = T - 1; k >= 0; --k) {
            q += gy[k];
            const float du = q * (av[k] * (before[k] - av[k] * inv[k] * e[k])) * sr[k];
            const float qm = q * m[k];
            odx[k] = qm * si[k];
            odi[k] = qm * e[k] * (1.f - si[k]);
            odr[k] = du * A * (1.f - sr[k]);
            q *= av[k];
            if (c0 + CHUNK > len) {
                const bool in = len - t0 > k;
                odx[k] = in ? odx[k] : 0.f;
                odi[k] = in ? odi[k] : 0.f;
                odr[k] = in ? odr[k] : 0.f;
                sum_A += in ? du : 0.f;
            } else {
                sum_A += du;
            }
            sum_r += odr[k];
            sum_i += odi[k];
        }
        if (t0 < L) {
            store_row<E, T>(dx, t0, L, odx);
            store_row<E, T>(dr, t0, L, odr);
            store_row<E, T>(di, t0, L, odi);
        }
    }
    if (a.dstate && lane == 0 && live) a.dstate[row] = back;
    float sum[3] = {sum_A, sum_r, sum_i};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int s = 1; s < LANES; s *= 2) sum[k] += lane_xor(sum[k], s);
    }
    // [row][wave], then the batch items in their order, each with its waves.
    __shared__ float parts[3][16];
    if constexpr (W > 1) {
        if (lane % 64 == 0) {
#pragma unroll
            for (int k = 0; k < 3; ++k) parts[k][threadIdx.x / 64] = sum[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            sum[k] = 0.f;
            for (int w = 0; w < W; ++w) sum[k] += parts[k][own * W + w];
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k) sums[own][k] = sum[k];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.channels * 3; i += blockDim.x) {
        const int c = i / 3, k = i % 3, dc = blockIdx.x * a.channels + c;
        if (dc >= a.D) continue;
        float total = 0.f;
        for (int n = 0; n < a.items; ++n) total += sums[n * a.channels + c][k];
        if (a.params) {
            a.params[((int64_t)blockIdx.y * a.D + dc) * 3 + k] = total;
        } else {
            float *const to = k == 0 ? a.dA : k == 1 ? a.dr_bias : a.di_bias;
            if (to) to[dc] = total;
        }
    }
}

// Sums over the batch, in its order, of [B][D][3]: dA, dr_bias, di_bias.
__global__ __launch_bounds__(256) void gated_join(const float *params, float *dA, float *dr_bias,
                                                  float *di_bias, int B, int D) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= 3 * D) return;
    float sum = 0.f;
#pragma unroll 8
    for (int b = 0; b < B; ++b) sum += params[(int64_t)b * 3 * D + i];
    float *const to = i % 3 == 0 ? dA : i % 3 == 1 ? dr_bias : di_bias;
    if (to) to[i / 3] = sum;
}

template <class E>
struct GatedStep {
    View<E> x, r, i, z, y;
    const float *A, *r_bias, *i_bias;
    float *state;
    const int32_t *slots;
    int D, lines;
};

// One position: each number is read and written once, V channels a thread (contiguous ones
// where V > 1), 16 bytes of states for V = 4.  Up to some 100000 channels the launch and one
// round trip ([8, 2048] bf16 2.4 us), beyond memory ([256, 4096] 4.5 us and 4.2 TB/s where the
// operands are in the memory-side cache, 7.2 from memory).
template <class E, int V>
__global__ __launch_bounds__(256) void gated_step(GatedStep<E> a) {
    const int d = (blockIdx.x * 256 + threadIdx.x) * V, b = blockIdx.y;
    if (d >= a.D) return;
    const int slot = a.slots ? a.slots[b] : b;
    float out[V];
    if (slot >= 0 && slot < a.lines) {
        float *state = a.state + (int64_t)slot * a.D + d;
        float x[V], r[V], i[V], z[V], h[V], A[V], rb[V], ib[V];
        load_vec<F32, V>(state, h);
        load_vec<E, V>(a.x.row(b, d), x);
        load_vec<E, V>(a.r.row(b, d), r);
        load_vec<E, V>(a.i.row(b, d), i);
        if (a.z.p) load_vec<E, V>(a.z.row(b, d), z);
        load_vec<F32, V>(a.A + d, A);
#pragma unroll
        for (int k = 0; k < V; ++k) rb[k] = ib[k] = 0.f;
        if (a.r_bias) load_vec<F32, V>(a.r_bias + d, rb);
        if (a.i_bias) load_vec<F32, V>(a.i_bias + d, ib);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float sr = gate(r[k], rb[k] * -kLog2e), si = gate(i[k], ib[k] * -kLog2e);
            const Decay v = decay(sr, decay_rate(A[k]));
            h[k] = __builtin_fmaf(v.a, h[k], __builtin_amdgcn_sqrtf(v.n) * (si * x[k]));
            out[k] = a.z.p ? h[k] * (z[k] * sigmoid(z[k])) : h[k];
        }
        store_vec<F32, V>(state, h);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) out[k] = 0.f;
    }
    store_vec<E, V>(a.y.row(b, d), out);
}

// How the rows are dealt: lanes of a row in a wave, waves of a row.
struct Deal {
    int lanes, waves;
};
// Rows that fit into few lanes take no more (4 lanes only where that is the whole row:
// a checkpoint is for 16).  Longer ones take a wave, several where there are too few rows to
// fill the chip, and where that leaves four chunks to read ahead in; the backward call, whose
// waves have twice the work, takes two chunks at least instead of a wave more.  Measured (us,
// forward / backward, 16 lanes, 64 lanes with 1, 2, 4, 8, 16 waves):
// [1, 4096, 8192] bf16 108 75 74 71 77 87 / 144 134 136 129 154 169,
// [4, 2048, 2048] bf16 37 30 31 32 64 153 / 65 61 64 71 168 262,
// [1, 256, 8192] bf16 85 24 14 8.8 6.9 6.4 / 129 38 24 16.5 14.4 14.8,
// [2, 602, 777] f32 12 7.5 6.3 8.7 13 26 / 23 14.7 17.7 22 32 59,
// [1, 300, 3000] f16 34 11 8.5 7.3 6.4 11 / 54 19 15 13 15 21,
// [4, 2000, 500] bf16 13 14 21 34 70 165 / 24 27 43 73 183 268,
// [1, 600, 500] f32 8.4 4.8 5.3 6.1 8.9 16 / 15.5 9.6 10.2 14 21 34.
// Forward, a row that two or four waves cover in one chunk, with little over, takes them: all of
// it is on its way at once.  On three sets of operands in turn (1, 2, 4 waves): [4, 2048, 2048] bf16
// 38.6 37.6 34.5, [2, 4096, 2048] 38.9 36.8 32.5, [16, 1024, 1024] 36.3 33.9 59.
Deal pick_deal(int64_t rows, int64_t L, bool backward) {
    if (L <= 4 * T) return {4, 1};
    if (L <= kRow || (L <= 4 * kRow && rows >= 4096)) return {16, 1};
    constexpr int kWave = 64 * T;
    Deal v{64, 1};
    if (!backward)
        for (int W = 2; W <= 4; W *= 2)
            if (L <= W * kWave && L > W * kWave * 7 / 8) return {64, W};
    while (v.waves < 16 && v.waves * kWave * (backward ? 2 : 1) < L && rows * v.waves < 4096) v.waves *= 2;
    while (v.waves < 16 && v.waves * kWave * 8 <= L && rows * v.waves < 16384) v.waves *= 2;
    return v;
}

template <class E, int LANES, int W>
hipError_t forward(const gated_scan_args &a, hipStream_t s) {
    GatedFwd<E> k{view<E>(a.x), view<E>(a.r), view<E>(a.i), view<E>(a.z), view<E>(a.y), a.A,
                  a.r_bias, a.i_bias, a.state_in, a.state_out, a.checkpoints, a.lengths,
                  a.B * a.D, a.D, a.L, (a.L + kRow - 1) / kRow};
    constexpr int ROWS = kRowsOf<LANES, W>;
    gated_forward<E, LANES, W>
        <<<(unsigned)((k.rows + ROWS - 1) / ROWS), kThreadsOf<LANES, W>, 0, s>>>(k);
    return hipGetLastError();
}

// Batch items of a work-group of the backward call, and its channels: whole waves of them,
// four at least.  All items where that is up to four waves, or eight (512 threads, for
// registers) and all rows run at once; beyond, groups of so many waves leave places empty
// ([5, 1000, 1237] f16: 52 us for 34, [8, 4000, 100] bf16: 31 for 26).
struct Share {
    int items, channels;
};
Share pick_share(int64_t B, int64_t D, const Deal &v) {
    const int per_wave = 64 / v.lanes;   // channels
    Share k{(int)B, per_wave};
    if (B * v.waves > (B * D / per_wave * v.waves <= 2048 ? 8 : 4)) k.items = 1;
    while (k.items * v.waves * (k.channels / per_wave) * 2 <= 4) k.channels *= 2;
    return k;
}

template <class E, int LANES, int W>
hipError_t backward(const gated_scan_backward_args &a, hipStream_t s) {
    const Share v = pick_share(a.B, a.D, {LANES, W});
    const bool whole = v.items == a.B;
    GatedBwd<E> k{view<E>(a.gout), view<E>(a.x), view<E>(a.r), view<E>(a.i), view<E>(a.z),
                  view<E>(a.dx), view<E>(a.dr), view<E>(a.di), view<E>(a.dz), a.A, a.r_bias,
                  a.i_bias, a.checkpoints, a.gstate, a.dA, a.dr_bias, a.di_bias,
                  whole ? nullptr : static_cast<float *>(a.workspace), a.dstate, a.lengths,
                  a.D, a.L, (a.L + kRow - 1) / kRow, v.channels, v.items};
    const dim3 grid((unsigned)((a.D + v.channels - 1) / v.channels), (unsigned)(a.B / v.items));
    gated_backward<E, LANES, W><<<grid, v.channels * v.items * LANES * W, 0, s>>>(k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || whole) return e;
    gated_join<<<(unsigned)((3 * (int64_t)a.D + 255) / 256), 256, 0, s>>>(k.params, a.dA, a.dr_bias, a.di_bias,
                                                                         a.B, a.D);
    return hipGetLastError();
}

template <class E>
hipError_t forward_any(const gated_scan_args &a, hipStream_t s) {
    const Deal v = pick_deal((int64_t)a.B * a.D, a.L, false);
    if (v.lanes == 4) return forward<E, 4, 1>(a, s);
    if (v.lanes == 16) return forward<E, 16, 1>(a, s);
    switch (v.waves) {
        case 1: return forward<E, 64, 1>(a, s);
        case 2: return forward<E, 64, 2>(a, s);
        case 4: return forward<E, 64, 4>(a, s);
        case 8: return forward<E, 64, 8>(a, s);
        default: return forward<E, 64, 16>(a, s);
    }
}

template <class E>
hipError_t backward_any(const gated_scan_backward_args &a, hipStream_t s) {
    const Deal v = pick_deal((int64_t)a.B * a.D, a.L, true);
    if (v.lanes == 4) return backward<E, 4, 1>(a, s);
    if (v.lanes == 16) return backward<E, 16, 1>(a, s);
    switch (v.waves) {
        case 1: return backward<E, 64, 1>(a, s);
        case 2: return backward<E, 64, 2>(a, s);
        case 4: return backward<E, 64, 4>(a, s);
        case 8: return backward<E, 64, 8>(a, s);
        default: return backward<E, 64, 16>(a, s);
    }
}

template <class E>
hipError_t step(const gated_scan_step_args &a, hipStream_t s) {
    GatedStep<E> k{view<E>(a.x), view<E>(a.r), view<E>(a.i), view<E>(a.z), view<E>(a.y), a.A,
                   a.r_bias, a.i_bias, a.state, a.slots, a.D, a.lines};
    const bool dense = a.D % 4 == 0 && a.x.channel == 1 && a.r.channel == 1 && a.i.channel == 1 &&
                       (a.z.channel == 1 || !a.z.data) && a.y.channel == 1;
    // Four channels a thread where that still leaves the chip work-groups enough (us, 1 / 4): [32,
    // 4096] 2.65 / 2.77, [64, 4096] 2.91 / 2.84, [256, 4096] 5.2 / 4.6, [512, 4096] 10.1 / 8.7.
    const int V = dense && (int64_t)a.B * a.D >= 262144 ? 4 : 1;
    const dim3 grid((unsigned)((a.D + 256 * V - 1) / (256 * V)), (unsigned)a.B);
    if (V == 4)
        gated_step<E, 4><<<grid, 256, 0, s>>>(k);
    else
        gated_step<E, 1><<<grid, 256, 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

int64_t gated_backward_workspace(int B, int D, int L) {
    const Share v = pick_share(B, D, pick_deal((int64_t)B * D, L, true));
    return v.items == B ? 0 : (int64_t)B * D * 3 * sizeof(float);
}

void gated_plan(int64_t rows, int64_t L, int backward, char *buf, size_t len) {
    const Deal v = pick_deal(rows, L, backward != 0);
    std::snprintf(buf, len, "lanes=%d waves=%d", v.lanes, v.waves);
}
hipError_t launch_gated_forward(const gated_scan_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? forward_any<F32>(a, s)
           : a.dtype == SEQ_BF16 ? forward_any<BF16>(a, s) : forward_any<F16>(a, s);
}
hipError_t launch_gated_backward(const gated_scan_backward_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? backward_any<F32>(a, s)
           : a.dtype == SEQ_BF16 ? backward_any<BF16>(a, s) : backward_any<F16>(a, s);
}
hipError_t launch_gated_step(const gated_scan_step_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? step<F32>(a, s)
           : a.dtype == SEQ_BF16 ? step<BF16>(a, s) : step<F16>(a, s);
}

}  // namespace seq
