// kernels_causal_conv.hip -- the depthwise causal convolution: forward, its
// gradients, and one position against a state cache.
//
// p[t] = bias + sum_k w[k] full[t+k] is K multiply-adds an element beside one
// read and one write, so memory bounds all three kernels.  A thread owns V = 8
// consecutive positions of one row (one 16-byte access for 16-bit types) and
// takes the K-1 positions before them from its neighbour's registers.
// [4, 4096, 2048] bf16, 4 taps: forward 33 us (134 MB, 4.0 TB/s), backward 43 us
// (201 MB, 4.7 TB/s); one position of [8, 2048] 2.4 us, the latency of its loads.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

constexpr int kV = 8;
constexpr int kThreads = 256;

int pow2_at_least(int64_t v, int most) {
    int p = 1;
    while (p < v && p < most) p *= 2;
    return p;
}

template <class E>
struct ConvFwd {
    View<E> x, y;
    const float *w, *bias;
    const typename E::type *state_in;
    typename E::type *state_out;
    const int32_t *lengths;
    int B, D, L;
    int row_threads;  // threads along a row, a power of two
    int silu;
};

// Threads [row][position octet]; grid.x over rows, grid.y over the row's rest.  A
// thread has R octets, `row_threads` octets apart, all on their way together.
template <class E, int K, int R>
__global__ __launch_bounds__(kThreads) void conv_forward(ConvFwd<E> a) {
    const int rows = kThreads / a.row_threads, lane = threadIdx.x % a.row_threads;
    const int64_t r = (int64_t)blockIdx.x * rows + threadIdx.x / a.row_threads;
    if (r >= (int64_t)a.B * a.D) return;
    const int b = (int)(r / a.D), d = (int)(r - (int64_t)b * a.D);
    const int start = (int)(blockIdx.y * R) * a.row_threads * kV;
    const int len = length_of(a.lengths, b, a.L);
    const auto *x = a.x.row(b, d);
    Octet<E> own[R];
#pragma unroll
    for (int c = 0; c < R; ++c) {
        // (What lies beyond the length is not read: 9.5 us for 10.7 at [5, 1000, 1237] fp16
        // with half of the positions there, though the length must arrive first.)
        const int t = start + (c * a.row_threads + lane) * kV;
        own[c].load(x + t, len - t);
    }
    float past[K], w[K];  // K-1 of past used
#pragma unroll
    for (int j = 0; j < K; ++j) past[j] = 0.f;
    if (start == 0 && lane == 0) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            if (a.state_in) past[j] = E::up(a.state_in[r * (K - 1) + j]);
        if (a.state_out) {
            // The last K-1 positions of the sequence; of the given state where it is shorter.
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                const int t = len + j;  // into full
                float v = 0.f;
                if (t >= K - 1) {
                    v = E::up(x[t - (K - 1)]);
                } else {
#pragma unroll
                    for (int i = 0; i < K - 1; ++i)
                        if (t == i) v = past[i];
                }
                a.state_out[r * (K - 1) + j] = E::down(v);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = a.w[(int64_t)d * K + k];
    const float bias = a.bias ? a.bias[d] : 0.f;
#pragma unroll
    for (int c = 0; c < R; ++c) {
        const int t0 = start + (c * a.row_threads + lane) * kV, left = len - t0;
        float v[kV + K], out[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[K - 1 + i] = own[c].at(i);
        // The positions before: the lane before's last; for a wave's first lane its last
        // lane's of the octet before, or a read of them.
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            v[j] = dpp0<kWaveShr>(v[kV + j]);
            if (c > 0) {
                const float turned = dpp0<kWaveRor>(own[c > 0 ? c - 1 : 0].at(kV - (K - 1) + j));
                if (lane == 0) v[j] = turned;
            }
        }
        if (c == 0 && threadIdx.x % 64 == 0 && t0 > 0 && left > 0) {
            Octet<E> o;
            o.load(x + t0 - kV, 8);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) v[j] = o.at(kV - (K - 1) + j);
        }
        if (t0 == 0) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) v[j] = past[j];
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float p = bias;
#pragma unroll
            for (int k = 0; k < K; ++k) p = __builtin_fmaf(w[k], v[i + k], p);
            const float q = a.silu ? p * sigmoid(p) : p;
            out[i] = left > i ? q : 0.f;
        }
        if (t0 < a.L) store_row<E, kV>(a.y.row(b, d), t0, a.L, out);
    }
}

// How the threads of a backward work-group are dealt: `along` along a row,
// `batch` batch items and `channels` channels at once (all powers of two), and
// how many work-groups share a channel's (batch, row segment) list.
struct BwdShape {
    int along, batch, channels;
    int segments, batches, splits;  // segments of a row, batch groups
};

BwdShape bwd_shape(int B, int D, int L) {
    BwdShape s;
    // A row beyond 256 octets in pieces of 256, 128 or 64 lanes, whichever leave the
    // fewest idle (shorter rows lose more to the borders of pieces than to idle lanes).
    const int64_t octets = ((int64_t)L + kV - 1) / kV;
    s.along = pow2_at_least(octets, kThreads);
    for (int n = s.along / 2; octets > kThreads && n >= 64; n /= 2)
        if ((octets + n - 1) / n * n < (octets + s.along - 1) / s.along * s.along) s.along = n;
    s.batch = pow2_at_least(B, kThreads / s.along);
    s.channels = kThreads / (s.along * s.batch);
    s.segments = (int)(((int64_t)L + (int64_t)s.along * kV - 1) / ((int64_t)s.along * kV));
    s.batches = (B + s.batch - 1) / s.batch;
    // Eight work-groups a compute unit keep enough loads in flight; a channel's
    // list is split no further than that needs.
    const int64_t tiles = (D + s.channels - 1) / s.channels;
    const int64_t list = (int64_t)s.segments * s.batches;
    const int64_t want = (2048 + tiles - 1) / tiles;
    s.splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(list, want), 65535));
    return s;
}

__device__ __forceinline__ float silu_slope(float p) {
    const float s = sigmoid(p);
    return s * (1.f + p * (1.f - s));
}

template <class E>
struct ConvBwd {
    View<E> gy, x, dx;
    const float *w, *bias;
    float *dw, *db;   // results, where one work-group has a channel
    float *part;      // [splits][D][K+1] otherwise
    const int32_t *lengths;
    int B, D, L;
    BwdShape s;
    int silu;
};

template <class E, int K>
__global__ __launch_bounds__(kThreads) void conv_backward(ConvBwd<E> a) {
    const int along = a.s.along;
    const int lane = threadIdx.x % along;
    const int bb = threadIdx.x / along % a.s.batch;
    const int dd = threadIdx.x / (along * a.s.batch);
    const int d = blockIdx.x * a.s.channels + dd;
    const int list = a.s.segments * a.s.batches;
    const int first = (int)((int64_t)list * blockIdx.y / a.s.splits);
    const int last = (int)((int64_t)list * (blockIdx.y + 1) / a.s.splits);
    float sums[K + 1];
#pragma unroll
    for (int k = 0; k <= K; ++k) sums[k] = 0.f;
    const bool channel = d < a.D;
    float w[K], bias = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = channel ? a.w[(int64_t)d * K + k] : 0.f;
    if (channel && a.bias) bias = a.bias[d];
    // Each wave's first dp, for the lane before it.
    __shared__ float edge[2][kThreads / 64 + 1][K];
    const int wave = threadIdx.x / 64;
    // This thread's channel in the first batch item, and its place in the list.
    const auto *x0 = a.x.row(0, d), *gy0 = a.gy.row(0, d);
    auto *dx0 = a.dx.row(0, d);
    int b = first / a.s.segments * a.s.batch + bb, segment = first % a.s.segments;
    for (int i = first; i < last; ++i) {
        const int t0 = (segment * along + lane) * kV;
        const bool here = channel && b < a.B && t0 < a.L;
        const int len = here ? length_of(a.lengths, b, a.L) : 0, left = len - t0;
        const auto *x = x0 + b * a.x.batch, *gy = gy0 + b * a.gy.batch;
        auto *dx = dx0 + b * a.dx.batch;
        if (++segment == a.s.segments) segment = 0, b += a.s.batch;
        // x of positions t0-(K-1) .. t0+V-1, dp of t0 .. t0+V-1+(K-1).
        float xs[kV + K], dp[kV + K];
        Octet<E> own, g, before;
        own.load(x + t0, left);
        g.load(gy + t0, left);
        // A wave's first lane reads the positions before its own, others have their
        // neighbour's.
        const bool border = threadIdx.x % 64 == 0 && t0 > 0;
        if (border) before.load(x + t0 - kV, left + kV);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            xs[K - 1 + j] = own.at(j);
            dp[j] = g.at(j);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            xs[j] = dpp0<kWaveShr>(xs[kV + j]);
            if (border) xs[j] = before.at(kV - (K - 1) + j);
            if (t0 == 0) xs[j] = 0.f;
        }
        if (a.silu) {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                float p = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) p = __builtin_fmaf(w[k], xs[j + k], p);
                // (Beyond the length p may come from NaN inside it.)
                dp[j] = left > j ? dp[j] * silu_slope(p) : 0.f;
            }
        }
        if (left >= kV) {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
#pragma unroll
                for (int k = 0; k < K; ++k) sums[k] = __builtin_fmaf(dp[j], xs[j + k], sums[k]);
                sums[K] += dp[j];
            }
        } else {
            // A position beyond the length multiplies none of the values inside, which
            // may be infinite: 0 for its dp is not enough.
#pragma unroll
            for (int j = 0; j < kV - 1; ++j) {
                if (left <= j) continue;
#pragma unroll
                for (int k = 0; k < K; ++k) sums[k] = __builtin_fmaf(dp[j], xs[j + k], sums[k]);
                sums[K] += dp[j];
            }
        }
        if (!a.dx.p) continue;
        // The next positions' dp: the lane after's first, or the wave after's; the last
        // lane of a piece of a longer row works them out.
        if (K > 1 && along > 64) {
            if (threadIdx.x % 64 == 0) {
#pragma unroll
                for (int j = 0; j < K - 1; ++j) edge[i & 1][wave][j] = dp[j];
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            dp[kV + j] = dpp0<kWaveShl>(dp[j]);
            if (along > 64 && threadIdx.x % 64 == 63) dp[kV + j] = edge[i & 1][wave + 1][j];
            if (left <= kV) dp[kV + j] = 0.f;
        }
        if (left > kV && lane == along - 1) {
            float xn[kV], gn[kV], tail[2 * K];
            load_row<E, kV>(x, t0 + kV, len, xn);
            load_row<E, kV>(gy, t0 + kV, len, gn);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                tail[j] = xs[kV + j];
                tail[K - 1 + j] = xn[j];
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                float p = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) p = __builtin_fmaf(w[k], tail[j + k], p);
                dp[kV + j] = left > kV + j ? (a.silu ? gn[j] * silu_slope(p) : gn[j]) : 0.f;
            }
        }
        if (!here) continue;
        float out[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            out[j] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) out[j] = __builtin_fmaf(w[K - 1 - k], dp[j + k], out[j]);
        }
        if (left < kV) {
#pragma unroll
            for (int j = 0; j < kV; ++j)  // 0 beyond the length also where a weight is infinite
                out[j] = left > j ? out[j] : 0.f;
        }
        store_row<E, kV>(dx, t0, a.L, out);
    }
    if (!a.dw && !a.db) return;
    // Sum over the threads of a channel: within waves, then over its waves in order.
    const int group = along * a.s.batch;
    __shared__ float waves[kThreads / 64][K + 1];
#pragma unroll
    for (int k = 0; k <= K; ++k)
        for (int m = 1; m < group && m < 64; m *= 2) sums[k] += lane_xor(sums[k], m);
    if (group > 64) {
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int k = 0; k <= K; ++k) waves[threadIdx.x / 64][k] = sums[k];
        __syncthreads();
        if (threadIdx.x % group == 0)
#pragma unroll
            for (int k = 0; k <= K; ++k) {
                sums[k] = 0.f;
                for (int v = 0; v < group / 64; ++v) sums[k] += waves[threadIdx.x / 64 + v][k];
            }
    }
    if (threadIdx.x % group == 0 && d < a.D) {
        if (a.s.splits > 1) {
#pragma unroll
            for (int k = 0; k <= K; ++k)
                a.part[((int64_t)blockIdx.y * a.D + d) * (K + 1) + k] = sums[k];
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (a.dw) a.dw[(int64_t)d * K + k] = sums[k];
            if (a.db) a.db[d] = sums[K];
        }
    }
}

__global__ void conv_backward_join(const float *part, float *dw, float *db, int D, int K,
                                   int splits) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t n = (int64_t)D * (K + 1);
    if (i >= n) return;
    float sum = 0.f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) sum += part[s * n + i];
    const int64_t d = i / (K + 1);
    const int k = (int)(i - d * (K + 1));
    if (k == K) {
        if (db) db[d] = sum;
    } else if (dw) {
        dw[d * K + k] = sum;
    }
}

template <class E>
struct ConvStep {
    View<E> x, y;
    const float *w, *bias;
    typename E::type *state;
    const int32_t *slots;
    int B, D, lines, silu;
};

template <class E, int K>
__global__ __launch_bounds__(kThreads) void conv_step(ConvStep<E> a) {
    const int d = blockIdx.x * kThreads + threadIdx.x;
    const int b = blockIdx.y;
    if (d >= a.D) return;
    const int slot = a.slots ? a.slots[b] : b;
    auto *y = a.y.row(b, d);
    if (slot < 0 || slot >= a.lines) {
        *y = E::down(0.f);
        return;
    }
    auto *state = a.state + ((int64_t)slot * a.D + d) * (K - 1);
    typename E::type line[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) line[j] = state[j];
    line[K - 1] = *a.x.row(b, d);
    float p = a.bias ? a.bias[d] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) p = __builtin_fmaf(a.w[(int64_t)d * K + k], E::up(line[k]), p);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) state[j] = line[j + 1];
    *y = E::down(a.silu ? p * sigmoid(p) : p);
}

template <class F>
void with_taps(int K, F f) {
    switch (K) {
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        case 3: f(std::integral_constant<int, 3>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        case 5: f(std::integral_constant<int, 5>()); break;
        case 6: f(std::integral_constant<int, 6>()); break;
        case 7: f(std::integral_constant<int, 7>()); break;
        case 8: f(std::integral_constant<int, 8>()); break;
    }
}

template <class E>
hipError_t forward(const causal_conv_args &a, hipStream_t s) {
    ConvFwd<E> k{view<E>(a.x), view<E>(a.y), a.w, a.bias,
                 static_cast<const typename E::type *>(a.state_in),
                 static_cast<typename E::type *>(a.state_out), a.lengths, a.B, a.D, a.L, 0,
                 a.silu};
    // Rows of more than two waves' octets go to one wave, four octets a lane: fewer
    // waves to start and no reads at their borders.
    const int64_t octets = ((int64_t)a.L + kV - 1) / kV;
    const int R = octets > 128 ? 4 : 1;
    k.row_threads = R == 4 ? 64 : pow2_at_least(octets, kThreads);
    const int64_t rows = kThreads / k.row_threads, span = (int64_t)k.row_threads * R;
    const dim3 grid((unsigned)(((int64_t)a.B * a.D + rows - 1) / rows),
                    (unsigned)((octets + span - 1) / span));
    with_taps(a.K, [&](auto taps) {
        constexpr int K = decltype(taps)::value;
        const auto kernel = R == 4 ? conv_forward<E, K, 4> : conv_forward<E, K, 1>;
        kernel<<<grid, kThreads, 0, s>>>(k);
    });
    return hipGetLastError();
}

template <class E>
hipError_t backward(const causal_conv_backward_args &a, hipStream_t s) {
    ConvBwd<E> k{view<E>(a.gy), view<E>(a.x), view<E>(a.dx), a.w, a.bias, a.dw, a.db,
                 static_cast<float *>(a.workspace), a.lengths, a.B, a.D, a.L,
                 bwd_shape(a.B, a.D, a.L), a.silu};
    const dim3 grid((unsigned)((a.D + k.s.channels - 1) / k.s.channels), (unsigned)k.s.splits);
    with_taps(a.K, [&](auto taps) {
        conv_backward<E, decltype(taps)::value><<<grid, kThreads, 0, s>>>(k);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || k.s.splits == 1 || (!a.dw && !a.db)) return e;
    const int64_t n = (int64_t)a.D * (a.K + 1);
    conv_backward_join<<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(
        k.part, a.dw, a.db, a.D, a.K, k.s.splits);
    return hipGetLastError();
}

template <class E>
hipError_t step(const causal_conv_step_args &a, hipStream_t s) {
    ConvStep<E> k{view<E>(a.x), view<E>(a.y), a.w, a.bias,
                  static_cast<typename E::type *>(a.state), a.slots, a.B, a.D, a.lines, a.silu};
    const dim3 grid((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)a.B);
    with_taps(a.K, [&](auto taps) {
        conv_step<E, decltype(taps)::value><<<grid, kThreads, 0, s>>>(k);
    });
    return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_forward(const causal_conv_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? forward<F32>(a, s)
           : a.dtype == SEQ_BF16 ? forward<BF16>(a, s) : forward<F16>(a, s);
}
hipError_t launch_conv_backward(const causal_conv_backward_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? backward<F32>(a, s)
           : a.dtype == SEQ_BF16 ? backward<BF16>(a, s) : backward<F16>(a, s);
}
hipError_t launch_conv_step(const causal_conv_step_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? step<F32>(a, s)
           : a.dtype == SEQ_BF16 ? step<BF16>(a, s) : step<F16>(a, s);
}

int64_t conv_backward_workspace(int B, int D, int L, int K) {
    const BwdShape s = bwd_shape(B, D, L);
    return s.splits > 1 ? (int64_t)s.splits * D * (K + 1) * 4 : 0;
}

}  // namespace seq
