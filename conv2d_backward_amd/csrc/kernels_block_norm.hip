// kernels_block_norm.hip -- the norms between two residual blocks with the gate
// and the residual sum, and their gradients.
//
// The means run over channels, which are a row apart, while positions are
// contiguous: in the forward a work-group owns a tile of columns (positions) and
// all D channels of them, so one launch holds both means.  Memory bounds it (y,
// gate, r in, r_out, u out): a tile of few channels is read once, into
// registers, one of many again, which finds much of it in the caches.  A tile's
// rows are pieces of a cache line; the tiles that share the line run at the same
// time on the same die (tile_of), whose L2 has it.  [4, 2048, 2048] bf16: 76 us
// forward (235 MB, 3.1 TB/s): its work-groups, one a compute unit, read and write in
// turn, with the sums between.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

constexpr int kV = 8;
constexpr int kDies = 8;  // work-groups go to the dies in turn

// The tile of a work-group of n: those of one die follow each other.
__device__ __forceinline__ int tile_of(int wg, int n) {
    const int per = n / kDies, rest = n % kDies, die = wg % kDies;
    return die * per + std::min(die, rest) + wg / kDies;
}

// Sum over the lanes l, l + CV, .. of each row of 16, then over the wave's rows:
// row k of 16 lanes ends with columns 2k and 2k+1 of its lanes' vectors.
template <int CV>
__device__ __forceinline__ Whole<2> wave_sums(float (&v)[kV]) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        if constexpr (CV <= 1) v[i] += dpp0<kRowRor + 1>(v[i]);
        if constexpr (CV <= 2) v[i] += dpp0<kRowRor + 2>(v[i]);
        if constexpr (CV <= 4) v[i] += dpp0<kRowRor + 4>(v[i]);
        v[i] += dpp0<kRowRor + 8>(v[i]);
    }
    return meet_rows<kV>(v);
}

// Sums v over the threads that share a column vector (threads i, i + CV, ..);
// every thread gets the sums of its columns.  `scratch`: [NT/64 + 1][S][CV * kV].
template <int S, int CV, int NT>
__device__ __forceinline__ void column_sums(float (&v)[S][kV], float *scratch) {
    constexpr int N = S * CV * kV, kWaves = NT / 64;
    const int tid = threadIdx.x, cv = tid % CV;
    __syncthreads();  // (the results of an earlier call are read)
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const Whole<2> w = wave_sums<CV>(v[s]);
        if (tid % 16 < CV)
            *reinterpret_cast<Whole<2> *>(scratch + tid / 64 * N + (s * CV + cv) * kV +
                                          tid % 64 / 16 * 2) = w;
    }
    __syncthreads();
    if (tid < N) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += scratch[w * N + tid];
        scratch[kWaves * N + tid] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < kV; ++i) v[s][i] = scratch[kWaves * N + (s * CV + cv) * kV + i];
}

__device__ __forceinline__ float inverse_rms(float squares, int D, float eps) {
    return rsqrtf(squares / (float)D + eps);
}

template <class E>
struct NormFwd {
    View<E> y, gate, u;
    View<F32> r, r_out;
    const float *scale, *w_post, *w_pre;
    const int32_t *lengths;
    int B, D, L, tiles;  // tiles of a batch item
    float eps;
};

// One element vector of the residual sum.
template <class E>
__device__ __forceinline__ void residual_sum(const NormFwd<E> &a, int d, int left,
                                             const Octet<E> &y, const Octet<E> &gate,
                                             const float (&i_post)[kV], float (&r)[kV]) {
    const float f = (a.scale ? a.scale[d] : 1.f) * (a.w_post ? a.w_post[d] : 1.f);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        float n = y.at(i) * (i_post[i] * f);
        if (a.gate.p) n *= sigmoid(gate.at(i));
        r[i] = left > i ? r[i] + n : 0.f;
    }
}

// Threads [row][CV]; a thread has rows first, first + NT/CV, ..  ITER of
// them stay in its registers; ITER 0: any number, read again for each use.
template <class E, int NT, int CV, int ITER>
__global__ __launch_bounds__(NT) void norm_forward(NormFwd<E> a) {
    __shared__ float scratch[(NT / 64 + 1) * CV * kV];
    constexpr int ROWS = NT / CV, KEPT = ITER ? ITER : 1;
    const int wg = tile_of(blockIdx.x, gridDim.x), b = wg / a.tiles;
    const int t0 = (wg % a.tiles * CV + threadIdx.x % CV) * kV, first = threadIdx.x / CV;
    const int len = length_of(a.lengths, b, a.L), left = len - t0;
    const int rounds = ITER ? ITER : (a.D + ROWS - 1) / ROWS;
    Octet<E> y[KEPT], gate[KEPT];
    float r[KEPT][kV];
    const auto read = [&](int k, int d) {
        const int n = d < a.D ? left : 0;
        y[k].load(a.y.row(b, d) + t0, n);
        if (a.gate.p) gate[k].load(a.gate.row(b, d) + t0, n);
        load_row<F32, kV>(a.r.row(b, d), t0, t0 + n, r[k]);
    };
    if constexpr (ITER > 0) {
#pragma unroll
        for (int k = 0; k < ITER; ++k) read(k, first + k * ROWS);
    }
    float sum[1][kV], i_post[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) i_post[i] = 1.f, sum[0][i] = 0.f;
    if (a.w_post) {
#pragma unroll KEPT
        for (int k = 0; k < rounds; ++k) {
            const int d = first + k * ROWS, q = ITER ? k : 0;
            if constexpr (ITER == 0) y[0].load(a.y.row(b, d) + t0, d < a.D ? left : 0);
#pragma unroll
            for (int i = 0; i < kV; ++i)
                sum[0][i] = __builtin_fmaf(y[q].at(i), y[q].at(i), sum[0][i]);
        }
        column_sums<1, CV, NT>(sum, scratch);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            i_post[i] = inverse_rms(sum[0][i], a.D, a.eps);
            sum[0][i] = 0.f;
        }
    }
#pragma unroll KEPT
    for (int k = 0; k < rounds; ++k) {
        const int d = first + k * ROWS, q = ITER ? k : 0;
        if constexpr (ITER == 0) read(0, d);
        if (d < a.D && t0 < a.L) {
            residual_sum(a, d, left, y[q], gate[q], i_post, r[q]);
            store_row<F32, kV>(a.r_out.row(b, d), t0, a.L, r[q]);
#pragma unroll
            for (int i = 0; i < kV; ++i) sum[0][i] = __builtin_fmaf(r[q][i], r[q][i], sum[0][i]);
        }
    }
    if (!a.w_pre) return;
    column_sums<1, CV, NT>(sum, scratch);
    if (t0 >= a.L) return;
#pragma unroll
    for (int i = 0; i < kV; ++i) sum[0][i] = inverse_rms(sum[0][i], a.D, a.eps);
#pragma unroll KEPT
    for (int k = 0; k < rounds; ++k) {
        const int d = first + k * ROWS, q = ITER ? k : 0;
        if (d >= a.D) break;
        if constexpr (ITER == 0) load_row<F32, kV>(a.r_out.row(b, d), t0, len, r[0]);
        const float w = a.w_pre[d];
        float u[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) u[i] = r[q][i] * (sum[0][i] * w);
        if (left < kV) {
#pragma unroll
            for (int i = 0; i < kV; ++i)  // 0 beyond the length also where eps or w leave 0 * inf
                u[i] = left > i ? u[i] : 0.f;
        }
        store_row<E, kV>(a.u.row(b, d), t0, a.L, u);
    }
}

// One position a batch item: the channels of a row lie together (V of them an
// access where they are contiguous), and a work-group owns the row.
constexpr int kTokenThreads = 512;

__device__ __forceinline__ float group_sum(float v, float *scratch) {
    v += dpp0<kRowRor + 1>(v);
    v += dpp0<kRowRor + 2>(v);
    v += dpp0<kRowRor + 4>(v);
    v += dpp0<kRowRor + 8>(v);
    __syncthreads();
    if (threadIdx.x % 16 == 0) scratch[threadIdx.x / 16] = v;
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kTokenThreads / 16; ++i) sum += scratch[i];
    return sum;
}

template <class E, int V>
__device__ __forceinline__ void load_channels(const typename E::type *p, int64_t stride, int d,
                                              int D, float (&v)[V]) {
    if constexpr (V == 1)
        v[0] = d < D ? E::up(p[d * stride]) : 0.f;
    else
        load_row<E, V>(p, d, D, v);
}

template <class E, int V>
__device__ __forceinline__ void store_channels(typename E::type *p, int64_t stride, int d, int D,
                                               const float (&v)[V]) {
    if constexpr (V == 1) {
        if (d < D) p[d * stride] = E::down(v[0]);
    } else {
        store_row<E, V>(p, d, D, v);
    }
}

template <class E, int V, int ITER>
__global__ __launch_bounds__(kTokenThreads) void norm_token(NormFwd<E> a) {
    __shared__ float scratch[kTokenThreads / 16];
    constexpr int KEPT = ITER ? ITER : 1;
    const int b = blockIdx.x, D = a.D;
    const bool in = length_of(a.lengths, b, 1) > 0;
    const int rounds = ITER ? ITER : (D + kTokenThreads * V - 1) / (kTokenThreads * V);
    const int live = in ? D : 0;
    float y[KEPT][V], r[KEPT][V];
    float i_post = 1.f, sum = 0.f;
#pragma unroll KEPT
    for (int k = 0; k < rounds; ++k) {
        const int d = (k * kTokenThreads + threadIdx.x) * V, q = ITER ? k : 0;
        load_channels<E, V>(a.y.row(b, 0), a.y.channel, d, live, y[q]);
        if constexpr (ITER > 0)
            load_channels<F32, V>(a.r.row(b, 0), a.r.channel, d, live, r[q]);
#pragma unroll
        for (int i = 0; i < V; ++i) sum = __builtin_fmaf(y[q][i], y[q][i], sum);
    }
    if (a.w_post) i_post = inverse_rms(group_sum(sum, scratch), D, a.eps);
    sum = 0.f;
#pragma unroll KEPT
    for (int k = 0; k < rounds; ++k) {
        const int d = (k * kTokenThreads + threadIdx.x) * V, q = ITER ? k : 0;
        if constexpr (ITER == 0) {
            load_channels<E, V>(a.y.row(b, 0), a.y.channel, d, live, y[0]);
            load_channels<F32, V>(a.r.row(b, 0), a.r.channel, d, live, r[0]);
        }
        float f[V], v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i_post;
        if (a.w_post) {
            load_channels<F32, V>(a.w_post, 1, d, D, v);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= v[i];
        }
        if (a.scale) {
            load_channels<F32, V>(a.scale, 1, d, D, v);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= v[i];
        }
        if (a.gate.p) {
            load_channels<E, V>(a.gate.row(b, 0), a.gate.channel, d, live, v);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= sigmoid(v[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            r[q][i] = in ? __builtin_fmaf(y[q][i], f[i], r[q][i]) : 0.f;
            sum = __builtin_fmaf(r[q][i], r[q][i], sum);
        }
        store_channels<F32, V>(a.r_out.row(b, 0), a.r_out.channel, d, D, r[q]);
    }
    if (!a.w_pre) return;
    const float i_pre = inverse_rms(group_sum(sum, scratch), D, a.eps);
#pragma unroll KEPT
    for (int k = 0; k < rounds; ++k) {
        const int d = (k * kTokenThreads + threadIdx.x) * V, q = ITER ? k : 0;
        if constexpr (ITER == 0)
            load_channels<F32, V>(a.r_out.row(b, 0), a.r_out.channel, d, live, r[0]);
        float w[V];
        load_channels<F32, V>(a.w_pre, 1, d, D, w);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = in ? w[i] * (r[q][i] * i_pre) : 0.f;
        store_channels<E, V>(a.u.row(b, 0), a.u.channel, d, D, w);
    }
}

// Backward: two passes over tiles of 64 columns by a share of the rows, so that
// rows are read in whole cache lines and any shape fills the chip: the first
// sums over channels, the second has every gradient of its elements.
// [4, 2048, 2048] bf16: 40 + 66 us, the second at 5.6 TB/s, partly out of the
// memory-side cache.  A single pass with a work-group per 32 columns and all
// channels, reading its tile twice, took 150 us.
constexpr int kBwdThreads = 256, kBwdCV = 8, kBwdRows = kBwdThreads / kBwdCV;

struct BwdShape {
    int tiles, splits;     // column tiles of a batch item, shares of the rows
    int64_t sums, params;  // workspace offsets, in floats
    int64_t floats;
};

BwdShape bwd_shape(int64_t B, int64_t D, int64_t L) {
    BwdShape s;
    s.tiles = (int)((L + kV * kBwdCV - 1) / (kV * kBwdCV));
    // Four work-groups a compute unit; a share has a round of rows at least.
    const int64_t most = std::min<int64_t>(64, (D + kBwdRows - 1) / kBwdRows);
    s.splits = (int)std::max<int64_t>(1, std::min(most, 1024 / (B * s.tiles)));
    s.sums = 0;
    s.params = s.sums + s.splits * 6 * B * s.tiles * kV * kBwdCV;
    s.floats = s.params + B * s.tiles * 3 * D;
    return s;
}

template <class E>
struct NormBwd {
    View<E> gu, y, gate, dy, dgate;
    View<F32> gr, r_out, dr;
    const float *scale, *w_post, *w_pre;
    const int32_t *lengths;
    float *ws;
    int B, D, L;
    BwdShape s;
    int params;  // whether the parameters' gradients are wanted
    float eps;
};

// An element vector of every input; missing ones are zeros, and so is the new residual
// without a norm of it.
template <class E>
struct NormIn {
    Octet<E> y, gate, gu;
    Octet<F32> r, gr;
    __device__ __forceinline__ void load(const NormBwd<E> &a, int b, int d, int t0, int left) {
        y.load(a.y.row(b, d) + t0, left);
        if (a.w_pre)
            r.load(a.r_out.row(b, d) + t0, left);
        else
            r.zero();
        if (a.gr.p)
            gr.load(a.gr.row(b, d) + t0, left);
        else
            gr.zero();
        if (a.gu.p)
            gu.load(a.gu.row(b, d) + t0, left);
        else
            gu.zero();
        if (a.gate.p) gate.load(a.gate.row(b, d) + t0, left);
    }
    __device__ __forceinline__ float open(const NormBwd<E> &a, int i) const {
        return a.gate.p ? sigmoid(gate.at(i)) : 1.f;
    }
};

// With v the gradient of rms(x) = x i, x's is i (v - (x i) k), k = i mean(v x): x i and
// k are of order 1 and of v, where x i^3 mean(v x) overflows for x under 2^-42.
// With q = scale sigmoid(gate) w_post y the mean that dy's norm needs, sum_d q dr,
// splits over dr = gr + i (gu w_pre - (r i) k) into sums of the inputs, so that one
// pass has all six sums.
template <class E>
__global__ __launch_bounds__(kBwdThreads) void norm_backward_sums(NormBwd<E> a) {
    constexpr int COLS = kV * kBwdCV;
    __shared__ float waves[kBwdThreads / 64][6][COLS];
    const int cv = threadIdx.x % kBwdCV, tid = threadIdx.x;
    const int all = a.B * a.s.tiles, wg = tile_of(blockIdx.x, gridDim.x);
    const int bt = wg % all, b = bt / a.s.tiles, split = wg / all;
    const int t0 = bt % a.s.tiles * COLS + cv * kV;
    const int left = length_of(a.lengths, b, a.L) - t0;
    const int lo = (int)((int64_t)a.D * split / a.s.splits);
    const int hi = (int)((int64_t)a.D * (split + 1) / a.s.splits);
    float sum[6][kV];
#pragma unroll
    for (int s = 0; s < 6; ++s)
#pragma unroll
        for (int i = 0; i < kV; ++i) sum[s][i] = 0.f;
    if (left > 0) {
        for (int d = lo + tid / kBwdCV; d < hi; d += kBwdRows) {
            NormIn<E> in;
            in.load(a, b, d, t0, left);
            const float f = (a.scale ? a.scale[d] : 1.f) * (a.w_post ? a.w_post[d] : 1.f);
            const float w = a.w_pre ? a.w_pre[d] : 0.f;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float y = in.y.at(i), r = in.r.at(i);
                const float q = f * y * in.open(a, i), guw = in.gu.at(i) * w;
                sum[0][i] = __builtin_fmaf(y, y, sum[0][i]);
                sum[1][i] = __builtin_fmaf(r, r, sum[1][i]);
                sum[2][i] = __builtin_fmaf(guw, r, sum[2][i]);
                sum[3][i] = __builtin_fmaf(q, in.gr.at(i), sum[3][i]);
                sum[4][i] = __builtin_fmaf(q, guw, sum[4][i]);
                sum[5][i] = __builtin_fmaf(q, r, sum[5][i]);
            }
        }
    }
#pragma unroll
    for (int s = 0; s < 6; ++s) {
        const Whole<2> w = wave_sums<kBwdCV>(sum[s]);
        if (tid % 16 < kBwdCV)
            *reinterpret_cast<Whole<2> *>(&waves[tid / 64][s][cv * kV + tid % 64 / 16 * 2]) = w;
    }
    __syncthreads();
    for (int i = tid; i < 6 * COLS; i += kBwdThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kBwdThreads / 64; ++w) v += waves[w][i / COLS][i % COLS];
        a.ws[a.s.sums + (((int64_t)split * 6 + i / COLS) * a.B * a.s.tiles + bt) * COLS +
             i % COLS] = v;
    }
}

// Sum over groups of 8 lanes, in every lane.
__device__ __forceinline__ float sum_of_8(float v) {
    v += dpp0<0xb1>(v);   // lane ^ 1
    v += dpp0<0x4e>(v);   // lane ^ 2
    return v + dpp0<0x141>(v);  // 7 - lane
}

template <class E>
__global__ __launch_bounds__(kBwdThreads) void norm_backward_apply(NormBwd<E> a) {
    constexpr int COLS = kV * kBwdCV;
    __shared__ float sums[6][COLS];
    __shared__ float coef[4][COLS];  // i_post, i_pre, k_pre, k_post
    const int cv = threadIdx.x % kBwdCV, tid = threadIdx.x;
    // From the last tile back: the caches hold what the first pass read last.
    const int all = a.B * a.s.tiles, wg = tile_of(gridDim.x - 1 - blockIdx.x, gridDim.x);
    const int bt = wg % all, b = bt / a.s.tiles, split = wg / all;
    const int t0 = bt % a.s.tiles * COLS + cv * kV;
    const int left = length_of(a.lengths, b, a.L) - t0;
    const int lo = (int)((int64_t)a.D * split / a.s.splits);
    const int hi = (int)((int64_t)a.D * (split + 1) / a.s.splits);
    for (int i = tid; i < 6 * COLS; i += kBwdThreads) {
        float v = 0.f;
#pragma unroll 8
        for (int s = 0; s < a.s.splits; ++s)
            v += a.ws[a.s.sums + (((int64_t)s * 6 + i / COLS) * a.B * a.s.tiles + bt) * COLS +
                      i % COLS];
        sums[i / COLS][i % COLS] = v;
    }
    __syncthreads();
    if (tid < COLS) {
        const float D = (float)a.D;
        // Columns without a position get 0 for both roots (1/0 at eps = 0): their zeros
        // go through the same sums as the others' values and add nothing.
        const bool here = bt % a.s.tiles * COLS + tid < length_of(a.lengths, b, a.L);
        const float i_pre = here && a.w_pre ? inverse_rms(sums[1][tid], a.D, a.eps) : 0.f;
        const float k_pre = i_pre * (sums[2][tid] / D);
        const float i_post = !here ? 0.f : a.w_post ? inverse_rms(sums[0][tid], a.D, a.eps) : 1.f;
        const float m = sums[3][tid] + i_pre * (sums[4][tid] - k_pre * (i_pre * sums[5][tid]));
        coef[0][tid] = i_post;
        coef[1][tid] = i_pre;
        coef[2][tid] = k_pre;
        coef[3][tid] = a.w_post ? i_post * (m / D) : 0.f;
    }
    __syncthreads();
    float i_post[kV], i_pre[kV], k_pre[kV], k_post[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        i_post[i] = coef[0][cv * kV + i];
        i_pre[i] = coef[1][cv * kV + i];
        k_pre[i] = coef[2][cv * kV + i];
        k_post[i] = coef[3][cv * kV + i];
    }
    for (int d = lo + tid / kBwdCV; d < hi; d += kBwdRows) {
        float p[3] = {0.f, 0.f, 0.f};
        if (t0 < a.L) {
            NormIn<E> in;
            in.load(a, b, d, t0, left);
            float dy[kV], dr[kV], dgate[kV];
            const float scale = a.scale ? a.scale[d] : 1.f;
            const float wq = a.w_post ? a.w_post[d] : 1.f;
            const float w = a.w_pre ? a.w_pre[d] : 0.f;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float y = in.y.at(i), r = in.r.at(i), gu = in.gu.at(i);
                const float open = in.open(a, i);
                const float ri = r * i_pre[i];
                const float drv = in.gr.at(i) + i_pre[i] * (gu * w - ri * k_pre[i]);
                const float yi = y * i_post[i], n = yi * wq, dn = drv * scale * open;
                p[0] = __builtin_fmaf(drv * open, n, p[0]);
                p[1] = __builtin_fmaf(dn, yi, p[1]);
                p[2] = __builtin_fmaf(gu, ri, p[2]);
                const bool inside = left > i;
                dr[i] = inside ? drv : 0.f;
                dgate[i] = inside ? dn * n * (1.f - open) : 0.f;
                // (Without a norm of y its value has no part in dy, though it be infinite.)
                const float part = a.w_post ? yi * k_post[i] : 0.f;
                dy[i] = inside ? i_post[i] * (dn * wq - part) : 0.f;
            }
            store_row<F32, kV>(a.dr.row(b, d), t0, a.L, dr);
            store_row<E, kV>(a.dy.row(b, d), t0, a.L, dy);
            if (a.dgate.p) store_row<E, kV>(a.dgate.row(b, d), t0, a.L, dgate);
        }
        if (a.params) {
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                p[s] = sum_of_8(p[s]);
                if (cv == 0) a.ws[a.s.params + ((int64_t)bt * 3 + s) * a.D + d] = p[s];
            }
        }
    }
}

__global__ __launch_bounds__(256) void norm_join(const float *part, float *dscale, float *dw_post,
                                                 float *dw_pre, int64_t D, int parts) {
    // 32 channels a work-group, 8 threads each over every eighth part.
    __shared__ float sums[8][32];
    const int64_t i = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
    const int q = threadIdx.x / 32;
    float v = 0.f;
    if (i < 3 * D) {
#pragma unroll 4
        for (int t = q; t < parts; t += 8) v += part[(int64_t)t * 3 * D + i];
    }
    sums[q][threadIdx.x % 32] = v;
    __syncthreads();
    if (q || i >= 3 * D) return;
    for (int k = 1; k < 8; ++k) v += sums[k][threadIdx.x];
    float *to = i < D ? dscale : i < 2 * D ? dw_post : dw_pre;
    if (to) to[i % D] = v;
}

int64_t tiles_of(int64_t L, int CV) { return (L + kV * CV - 1) / (kV * CV); }

// How the columns are dealt to work-groups, and how many rows of them a thread keeps
// (0: none).  A tile stays in registers where its channels fit: 32 columns of up to 1024, 16
// of 2048 or 8 of 4096.  Pieces of rows should be long and tiles enough for the
// chip: 32 columns where those make 128 tiles, 8 where 16 make fewer than 96 (or
// none fit, up to 512 tiles of 8).  Else it is read again, with 32 columns where
// those make 256 tiles.  Measured (us, 32 / 16 / 8 columns kept, 32 / 16 again):
// [8, 1024, 2001] bf16 50 / 69 / 75, again 74 / 95; [3, 1000, 1025] f32 24 / 21 / 24;
// [1, 600, 1500] bf16 - / 12 / 10; [3, 1800, 2805] f16 - / 77 / 96, again 110;
// [64, 1500, 16] bf16 - / 13 / 10; [1, 4000, 1000] bf16 - / - / 31, again 52;
// [2, 4096, 2048] bf16 - / - / 67, again 59.
struct Deal {
    int CV, kept;
};
Deal pick_deal(int64_t B, int64_t D, int64_t L) {
    const int64_t t32 = B * tiles_of(L, 4), t16 = B * tiles_of(L, 2), t8 = B * tiles_of(L, 1);
    if (D <= 1024 && t32 >= 128) return {4, 4};
    if (D <= 2048 && t16 >= 96) return {2, D <= 1024 ? 2 : 4};
    if (D <= 4096 && t8 < 512) return {1, D <= 1024 ? 1 : D <= 2048 ? 2 : 4};
    return {t32 >= 256 ? 4 : 2, 0};
}

template <class E>
hipError_t forward(const block_norm_args &a, hipStream_t s) {
    NormFwd<E> k{view<E>(a.y), view<E>(a.gate), view<E>(a.u), view<F32>(a.r), view<F32>(a.r_out),
                 a.scale, a.w_post, a.w_pre, a.lengths, a.B, a.D, a.L, 0, a.eps};
    if (a.L == 1) {
        const bool together = a.y.channel == 1 && a.r.channel == 1 && a.r_out.channel == 1 &&
                              (!a.gate.data || a.gate.channel == 1) &&
                              (!a.u.data || a.u.channel == 1);
        const int rounds = (a.D + kTokenThreads * 8 - 1) / (kTokenThreads * 8);
        auto kernel = norm_token<E, 1, 0>;
        if (together)
            kernel = rounds == 1 ? norm_token<E, 8, 1>
                     : rounds == 2 ? norm_token<E, 8, 2> : norm_token<E, 8, 0>;
        kernel<<<dim3((unsigned)a.B), kTokenThreads, 0, s>>>(k);
        return hipGetLastError();
    }
    const Deal deal = pick_deal(a.B, a.D, a.L);
    void (*kernel)(NormFwd<E>);
    if (deal.CV == 4)
        kernel = deal.kept ? norm_forward<E, 1024, 4, 4> : norm_forward<E, 1024, 4, 0>;
    else if (deal.CV == 2)
        kernel = deal.kept == 2   ? norm_forward<E, 1024, 2, 2>
                 : deal.kept == 4 ? norm_forward<E, 1024, 2, 4> : norm_forward<E, 1024, 2, 0>;
    else
        kernel = deal.kept == 1   ? norm_forward<E, 1024, 1, 1>
                 : deal.kept == 2 ? norm_forward<E, 1024, 1, 2> : norm_forward<E, 1024, 1, 4>;
    k.tiles = (int)tiles_of(a.L, deal.CV);
    kernel<<<dim3((unsigned)(a.B * k.tiles)), 1024, 0, s>>>(k);
    return hipGetLastError();
}

template <class E>
hipError_t backward(const block_norm_backward_args &a, hipStream_t s) {
    const bool params = a.dscale || a.dw_post || a.dw_pre;
    NormBwd<E> k{view<E>(a.gu), view<E>(a.y), view<E>(a.gate), view<E>(a.dy), view<E>(a.dgate),
                 view<F32>(a.gr), view<F32>(a.r_out), view<F32>(a.dr), a.scale, a.w_post, a.w_pre,
                 a.lengths, static_cast<float *>(a.workspace), a.B, a.D, a.L,
                 bwd_shape(a.B, a.D, a.L), params, a.eps};
    const dim3 grid((unsigned)(a.B * k.s.tiles * k.s.splits));
    norm_backward_sums<E><<<grid, kBwdThreads, 0, s>>>(k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm_backward_apply<E><<<grid, kBwdThreads, 0, s>>>(k);
    e = hipGetLastError();
    if (e != hipSuccess || !params) return e;
    norm_join<<<dim3((unsigned)((3 * (int64_t)a.D + 31) / 32)), 256, 0, s>>>(
        k.ws + k.s.params, a.dscale, a.dw_post, a.dw_pre, a.D, a.B * k.s.tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_forward(const block_norm_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? forward<F32>(a, s)
           : a.dtype == SEQ_BF16 ? forward<BF16>(a, s) : forward<F16>(a, s);
}
hipError_t launch_norm_backward(const block_norm_backward_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? backward<F32>(a, s)
           : a.dtype == SEQ_BF16 ? backward<BF16>(a, s) : backward<F16>(a, s);
}

int norm_columns(int64_t B, int64_t D, int64_t L) { return L == 1 ? 1 : kV * pick_deal(B, D, L).CV; }

int64_t norm_workspace(int B, int D, int L, int backward) {
    return backward ? bwd_shape(B, D, L).floats * 4 : 0;
}

}  // namespace seq
