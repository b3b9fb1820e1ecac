// kernels_block_norm.hip -- the norms between two residual blocks with the gate
// and the residual sum, and their gradients.
//
// The means run over channels, which are a row apart, while positions are
// contiguous: a work-group owns a tile of columns (positions) and all D
// channels of them, so one launch holds every mean.  Memory bounds it: forward
// y, gate, r in, r_out, u out; the second pass over a tile finds what the first
// one read in the caches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

constexpr int kThreads = 512;

// A tile is CV column vectors of V positions, side by side.

// Sums v over the threads that share a column vector (threads i, i + CV, ...);
// every thread gets the sums of its columns.  `scratch`: [kThreads/64][S][CV*V].
template <int S, int V, int CV>
__device__ __forceinline__ void column_sums(float (&v)[S][V], float *scratch) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, cv = threadIdx.x % CV;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int m = CV; m < 64; m *= 2) v[s][i] += lane_xor(v[s][i], m);
    __syncthreads();
    if (lane < CV) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) scratch[(wave * S + s) * CV * V + cv * V + i] = v[s][i];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 64; ++w) sum += scratch[(w * S + s) * CV * V + cv * V + i];
            v[s][i] = sum;
        }
}

template <class E>
struct NormFwd {
    View<E> y, gate, u;
    View<F32> r, r_out;
    const float *scale, *w_post, *w_pre;
    const int32_t *lengths;
    int B, D, L, tiles;
    float eps;
};

template <class E, int V, int CV>
__global__ __launch_bounds__(kThreads) void norm_forward(NormFwd<E> a) {
    __shared__ float scratch[kThreads / 64 * CV * V];
    constexpr int ROWS = kThreads / CV;
    const int b = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int t0 = (tile * CV + threadIdx.x % CV) * V, first = threadIdx.x / CV;
    const int len = length_of(a.lengths, b, a.L);
    float i_post[V], sum[1][V];
#pragma unroll
    for (int i = 0; i < V; ++i) i_post[i] = 1.f;
    if (a.w_post) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0][i] = 0.f;
        for (int d = first; d < a.D; d += ROWS) {
            float y[V];
            load_row<E, V>(a.y.row(b, d), t0, len, y);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[0][i] = __builtin_fmaf(y[i], y[i], sum[0][i]);
        }
        column_sums<1, V, CV>(sum, scratch);
#pragma unroll
        for (int i = 0; i < V; ++i) i_post[i] = rsqrtf(sum[0][i] / a.D + a.eps);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sum[0][i] = 0.f;
    for (int d = first; d < a.D; d += ROWS) {
        if (t0 >= a.L) break;
        float y[V], r[V], v[V];
        load_row<E, V>(a.y.row(b, d), t0, len, y);
        load_row<F32, V>(a.r.row(b, d), t0, len, r);
        const float f = (a.scale ? a.scale[d] : 1.f) * (a.w_post ? a.w_post[d] : 1.f);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] *= i_post[i] * f;
        if (a.gate.p) {
            load_row<E, V>(a.gate.row(b, d), t0, len, v);
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] *= sigmoid(v[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            r[i] = t0 + i < len ? r[i] + y[i] : 0.f;
            sum[0][i] = __builtin_fmaf(r[i], r[i], sum[0][i]);
        }
        store_row<F32, V>(a.r_out.row(b, d), t0, a.L, r);
    }
    if (!a.w_pre) return;
    column_sums<1, V, CV>(sum, scratch);
    if (t0 >= a.L) return;
    float i_pre[V];
#pragma unroll
    for (int i = 0; i < V; ++i) i_pre[i] = rsqrtf(sum[0][i] / a.D + a.eps);
    for (int d = first; d < a.D; d += ROWS) {
        float r[V];
        load_row<F32, V>(a.r_out.row(b, d), t0, len, r);
        const float w = a.w_pre[d];
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] *= i_pre[i] * w;
        store_row<E, V>(a.u.row(b, d), t0, a.L, r);
    }
}

template <class E>
struct NormBwd {
    View<E> gu, y, gate, dy, dgate;
    View<F32> gr, r_out, dr;
    const float *scale, *w_post, *w_pre;
    const int32_t *lengths;
    float *part;  // [B * tiles][3][D]: dscale, dw_post, dw_pre; NULL: none wanted
    int B, D, L, tiles;
    float eps;
};

// With q = scale sigmoid(gate) w_post y the mean that dy's norm needs,
// sum_d q dr, splits over dr = gr + i (gu w_pre) - r i^3 c into sums of the
// inputs, so that one pass over the tile has all six sums.
template <class E, int V, int CV>
__global__ __launch_bounds__(kThreads) void norm_backward(NormBwd<E> a) {
    __shared__ float scratch[kThreads / 64 * 6 * CV * V];
    constexpr int ROWS = kThreads / CV;
    const int b = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int t0 = (tile * CV + threadIdx.x % CV) * V, first = threadIdx.x / CV;
    const int len = length_of(a.lengths, b, a.L);
    float sum[6][V];
#pragma unroll
    for (int s = 0; s < 6; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[s][i] = 0.f;
    for (int d = first; d < a.D; d += ROWS) {
        float y[V], r[V], gr[V], gu[V], v[V];
        load_row<E, V>(a.y.row(b, d), t0, len, y);
        load_row<F32, V>(a.r_out.row(b, d), t0, len, r);
        load_row<F32, V>(a.gr.row(b, d), t0, a.gr.p ? len : 0, gr);
        load_row<E, V>(a.gu.row(b, d), t0, a.gu.p ? len : 0, gu);
        load_row<E, V>(a.gate.row(b, d), t0, a.gate.p ? len : 0, v);
        const float f = (a.scale ? a.scale[d] : 1.f) * (a.w_post ? a.w_post[d] : 1.f);
        const float w = a.w_pre ? a.w_pre[d] : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float q = f * y[i] * (a.gate.p ? sigmoid(v[i]) : 1.f);
            const float guw = gu[i] * w;
            sum[0][i] = __builtin_fmaf(y[i], y[i], sum[0][i]);
            sum[1][i] = __builtin_fmaf(r[i], r[i], sum[1][i]);
            sum[2][i] = __builtin_fmaf(guw, r[i], sum[2][i]);
            sum[3][i] = __builtin_fmaf(q, gr[i], sum[3][i]);
            sum[4][i] = __builtin_fmaf(q, guw, sum[4][i]);
            sum[5][i] = __builtin_fmaf(q, r[i], sum[5][i]);
        }
    }
    column_sums<6, V, CV>(sum, scratch);
    float i_post[V], i_pre[V], c_pre[V], c_post[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float D = (float)a.D;
        i_pre[i] = rsqrtf(sum[1][i] / D + a.eps);
        c_pre[i] = i_pre[i] * i_pre[i] * i_pre[i] * (sum[2][i] / D);
        i_post[i] = a.w_post ? rsqrtf(sum[0][i] / D + a.eps) : 1.f;
        const float m = sum[3][i] + i_pre[i] * sum[4][i] - c_pre[i] * sum[5][i];
        c_post[i] = a.w_post ? i_post[i] * i_post[i] * i_post[i] * (m / D) : 0.f;
    }
    for (int d = first; d < a.D; d += ROWS) {
        float y[V], r[V], gr[V], gu[V], v[V], p[3] = {0.f, 0.f, 0.f};
        if (t0 < a.L) {
            load_row<E, V>(a.y.row(b, d), t0, len, y);
            load_row<F32, V>(a.r_out.row(b, d), t0, len, r);
            load_row<F32, V>(a.gr.row(b, d), t0, a.gr.p ? len : 0, gr);
            load_row<E, V>(a.gu.row(b, d), t0, a.gu.p ? len : 0, gu);
            load_row<E, V>(a.gate.row(b, d), t0, a.gate.p ? len : 0, v);
            const float scale = a.scale ? a.scale[d] : 1.f;
            const float wq = a.w_post ? a.w_post[d] : 1.f;
            const float w = a.w_pre ? a.w_pre[d] : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float open = a.gate.p ? sigmoid(v[i]) : 1.f;
                const float dr = gr[i] + i_pre[i] * (gu[i] * w) - r[i] * c_pre[i];
                const float yi = y[i] * i_post[i], n = yi * wq;
                const float dn = dr * scale * open;
                p[0] = __builtin_fmaf(dr * open, n, p[0]);
                p[1] = __builtin_fmaf(dn, yi, p[1]);
                p[2] = __builtin_fmaf(gu[i] * r[i], i_pre[i], p[2]);
                const bool in = t0 + i < len;
                gr[i] = in ? dr : 0.f;
                v[i] = in ? dn * n * (1.f - open) : 0.f;
                y[i] = in ? i_post[i] * (dn * wq) - y[i] * c_post[i] : 0.f;
            }
            store_row<F32, V>(a.dr.row(b, d), t0, a.L, gr);
            store_row<E, V>(a.dy.row(b, d), t0, a.L, y);
            if (a.dgate.p) store_row<E, V>(a.dgate.row(b, d), t0, a.L, v);
        }
        if (a.part) {
#pragma unroll
            for (int s = 0; s < 3; ++s) {
#pragma unroll
                for (int m = 1; m < CV; m *= 2) p[s] += lane_xor(p[s], m);
                if (threadIdx.x % CV == 0) a.part[((int64_t)blockIdx.x * 3 + s) * a.D + d] = p[s];
            }
        }
    }
}

__global__ __launch_bounds__(256) void norm_join(const float *part, float *dscale, float *dw_post,
                                                 float *dw_pre, int64_t D, int tiles) {
    // 64 channels a work-group, 4 threads each over every fourth tile.
    __shared__ float sums[4][64];
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x % 64;
    const int q = threadIdx.x / 64;
    float v = 0.f;
    if (i < 3 * D)
        for (int t = q; t < tiles; t += 4) v += part[(int64_t)t * 3 * D + i];
    sums[q][threadIdx.x % 64] = v;
    __syncthreads();
    if (q || i >= 3 * D) return;
    v = sums[0][threadIdx.x] + sums[1][threadIdx.x] + sums[2][threadIdx.x] + sums[3][threadIdx.x];
    float *to = i < D ? dscale : i < 2 * D ? dw_post : dw_pre;
    if (to) to[i % D] = v;
}

constexpr int kV = 4, kCV = 8;

int64_t tiles_of(int64_t L) { return (L + kV * kCV - 1) / (kV * kCV); }

template <class E>
hipError_t forward(const block_norm_args &a, hipStream_t s) {
    NormFwd<E> k{view<E>(a.y), view<E>(a.gate), view<E>(a.u), view<F32>(a.r), view<F32>(a.r_out),
                 a.scale, a.w_post, a.w_pre, a.lengths, a.B, a.D, a.L, (int)tiles_of(a.L), a.eps};
    norm_forward<E, kV, kCV><<<dim3((unsigned)(a.B * k.tiles)), kThreads, 0, s>>>(k);
    return hipGetLastError();
}

template <class E>
hipError_t backward(const block_norm_backward_args &a, hipStream_t s) {
    const bool params = a.dscale || a.dw_post || a.dw_pre;
    NormBwd<E> k{view<E>(a.gu), view<E>(a.y), view<E>(a.gate), view<E>(a.dy), view<E>(a.dgate),
                 view<F32>(a.gr), view<F32>(a.r_out), view<F32>(a.dr), a.scale, a.w_post, a.w_pre,
                 a.lengths, params ? static_cast<float *>(a.workspace) : nullptr, a.B, a.D, a.L,
                 (int)tiles_of(a.L), a.eps};
    const int tiles = a.B * k.tiles;
    norm_backward<E, kV, kCV><<<dim3((unsigned)tiles), kThreads, 0, s>>>(k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !params) return e;
    norm_join<<<dim3((unsigned)((3 * (int64_t)a.D + 63) / 64)), 256, 0, s>>>(
        k.part, a.dscale, a.dw_post, a.dw_pre, a.D, tiles);
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

int64_t norm_workspace(int B, int D, int L, int backward) {
    return backward ? B * tiles_of(L) * 3 * (int64_t)D * 4 : 0;
}

}  // namespace seq
