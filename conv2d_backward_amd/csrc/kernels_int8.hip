// kernels_int8.hip -- projections in 8-bit integers: codes of activations or weights
// with a scale for each row, and the product of two matrices of codes.
//
// y[e, n] = scales[n] w_scales[e] sum over k of w[e, k] codes[n, k] + bias[e], where n
// counts the positions of all batch items.  Both operands have k contiguous, in rows of
// whole 128 bytes, so that the product needs no ends along k; the sums are int32 and
// exact.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gi_common.h"
#include "lds_barrier.h"
#include "seq_common.h"
#include "seq_kernels.h"

namespace seq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// ---- codes ---------------------------------------------------------------------------------------

// The code of v in a row whose largest magnitude is most: rint(127 v / most), decided
// exactly.  Rows of very large or small numbers are scaled by a power of two first, so
// that 127 v and 1 / most stay in range.
struct Coder {
    float factor, most, inv;   // of the scaled row: most, 1 / most
};
__device__ __forceinline__ Coder coder(uint32_t most_bits) {
    Coder c;
    const float most = __builtin_bit_cast(float, most_bits);
    c.factor = most > 0x1p100f ? 0x1p-64f : most < 0x1p-60f ? 0x1p64f : 1.f;
    c.most = most * c.factor;
    const bool coded = most_bits != 0 && most_bits < 0x7f800000u;
    c.inv = coded ? __builtin_amdgcn_rcpf(c.most) : 0.f;
    c.factor = coded ? c.factor : 0.f;
    return c;
}
__device__ __forceinline__ float row_scale(uint32_t most_bits) {
    return most_bits < 0x7f800000u ? __builtin_bit_cast(float, most_bits) / 127.f
                                   : __builtin_bit_cast(float, 0x7fc00000u);
}
// 16-bit numbers: 127 v is exact in fp32.  One step of Newton's method makes the quotient
// exact wherever it is half a step between two codes (it is a float then), and off by at
// most 2^-24 of it elsewhere, where it is at least 2^-18 of it away from the border.
// float32: the remainder of the nearest candidate, against half of most; 127 v has a low
// part, and every other term is exact.
template <class E>
__device__ __forceinline__ int code(float v, const Coder &c) {
    v *= c.factor;
    v = v != v || c.inv == 0.f ? 0.f : v;
    const float hi = v * 127.f;
    const float q = hi * c.inv;
    if constexpr (!std::is_same_v<E, F32>) {
        return (int)__builtin_rintf(__builtin_fmaf(__builtin_fmaf(-q, c.most, hi), c.inv, q));
    } else {
        const float k = __builtin_rintf(q);
        const float r = __builtin_fmaf(-k, c.most, hi), lo = __builtin_fmaf(v, 127.f, -hi);
        const float over = (__builtin_fabsf(r) - 0.5f * c.most) + (r < 0.f ? -lo : lo);
        const int n = (int)k, on = r < 0.f ? -1 : 1;
        return over > 0.f || (over == 0.f && (n & 1)) ? n + on : n;
    }
}
__device__ __forceinline__ uint32_t pack(int a, int b, int c, int d) {
    return (a & 255) | (b & 255) << 8 | (c & 255) << 16 | (uint32_t)d << 24;
}

template <class E>
struct Quantize {
    View<E> x;
    uint32_t *codes;   // [B, L, K / 4]
    float *scales;
    const int32_t *lengths;
    int B, D, L, K, tiles;
};

// Bits of |v|: they order like the numbers, infinities and NaN above all.
__device__ __forceinline__ uint32_t magnitude(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

// Positions along the lanes: a work-group has 32 positions, its threads 8 of them and
// every 64th quad of channels.
template <class E>
__global__ __launch_bounds__(256) void quantize_tile(Quantize<E> a) {
    __shared__ uint32_t meet[4][32];
    const int b = blockIdx.x / a.tiles, t0 = blockIdx.x % a.tiles * 32;
    const int len = length_of(a.lengths, b, a.L);
    const int t = t0 + threadIdx.x % 4 * 8, quad = threadIdx.x / 4;
    uint32_t most[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (t < len) {
        for (int d = quad; d < a.D; d += 64) {
            Octet<E> v;
            v.load(a.x.row(b, d) + t, len - t);
#pragma unroll
            for (int k = 0; k < 8; ++k) most[k] = max(most[k], magnitude(v.at(k)));
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int s = 4; s < 64; s *= 2)
            most[k] = max(most[k], (uint32_t)__shfl_xor((int)most[k], s, 64));
    }
    if (threadIdx.x % 64 < 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) meet[threadIdx.x / 64][threadIdx.x % 4 * 8 + k] = most[k];
    }
    __syncthreads();
    Coder c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int p = threadIdx.x % 4 * 8 + k;
        most[k] = max(max(meet[0][p], meet[1][p]), max(meet[2][p], meet[3][p]));
        c[k] = coder(most[k]);
        if (quad == 0 && t + k < a.L)
            a.scales[(int64_t)b * a.L + t + k] = row_scale(most[k]);
    }
    for (int d = quad * 4; d < a.K; d += 256) {
        Octet<E> v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j].zero();
            if (d + j < a.D && t < len) v[j].load(a.x.row(b, d + j) + t, len - t);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (t + k < a.L)
                a.codes[((int64_t)b * a.L + t + k) * (a.K / 4) + d / 4] =
                    pack(code<E>(v[0].at(k), c[k]), code<E>(v[1].at(k), c[k]),
                         code<E>(v[2].at(k), c[k]), code<E>(v[3].at(k), c[k]));
    }
}

// Channels along the lanes (one position, contiguous channels): a work-group a row.
template <class E>
__global__ __launch_bounds__(256) void quantize_row(Quantize<E> a) {
    __shared__ uint32_t meet[4];
    const int b = blockIdx.x;
    const int D = length_of(a.lengths, b, 1) ? a.D : 0;
    const auto *x = a.x.row(b, 0);
    uint32_t most = 0;
    for (int d = threadIdx.x * 8; d < D; d += 2048) {
        Octet<E> v;
        v.load(x + d, D - d);
#pragma unroll
        for (int k = 0; k < 8; ++k) most = max(most, magnitude(v.at(k)));
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2) most = max(most, (uint32_t)__shfl_xor((int)most, s, 64));
    if (threadIdx.x % 64 == 0) meet[threadIdx.x / 64] = most;
    __syncthreads();
    most = max(max(meet[0], meet[1]), max(meet[2], meet[3]));
    const Coder c = coder(most);
    if (threadIdx.x == 0) a.scales[b] = row_scale(most);
    for (int d = threadIdx.x * 8; d < a.K; d += 2048) {
        Octet<E> v;
        v.load(x + d, D - d);
        int n[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k] = code<E>(v.at(k), c);
        uint2 *to = reinterpret_cast<uint2 *>(a.codes + ((int64_t)b * a.K + d) / 4);
        *to = uint2{pack(n[0], n[1], n[2], n[3]), pack(n[4], n[5], n[6], n[7])};
    }
}

template <class E>
hipError_t quantize(const quantize_tokens_args &a, hipStream_t s) {
    Quantize<E> k{view<E>(a.x), static_cast<uint32_t *>(a.codes), a.scales, a.lengths,
                  a.B, a.D, a.L, a.K, (a.L + 31) / 32};
    if (a.L == 1 && (a.x.channel == 1 || a.D == 1))
        quantize_row<E><<<(unsigned)a.B, 256, 0, s>>>(k);
    else
        quantize_tile<E><<<(unsigned)(a.B * (int64_t)k.tiles), 256, 0, s>>>(k);
    return hipGetLastError();
}

// ---- the product ---------------------------------------------------------------------------------

template <class E>
struct Project {
    const uint8_t *codes, *w;   // [N, K], [E, K]
    const float *scales, *w_scales, *bias;
    View<E> y;
    const int32_t *lengths;
    int N, E_, L, K, n_tiles, e_tiles;
};

constexpr int kStep = 128;   // bytes of k staged at once

typedef __attribute__((address_space(3))) void *lds_ptr_t;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t *p, long bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, bytes, 0x00020000);
}
// 16 bytes a lane straight to LDS, lanes one after another.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint8_t *lds, uint32_t at, int from) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)lds, 16, at, from, 0, 0);
}
__device__ __forceinline__ v16i mfma(v4i a, v4i b, v16i c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// Tiles of TM positions and TE channels; waves in WM x WE, each with BM x BE blocks of
// 32 x 32.  Stages of 128 bytes of k go to LDS by direct loads, one stage ahead.  In
// LDS a row is eight 16-byte units, unit u at u ^ (row / 2 % 8): the 16 lanes that a
// cycle of ds_read_b128 serves then read 16 different units of 256 bytes.
template <class E, int WM, int WE, int BM, int BE>
__global__ __launch_bounds__(64 * WM * WE, 2) void project(Project<E> a) {
    constexpr int kThreads = 64 * WM * WE, TM = 32 * WM * BM, TE = 32 * WE * BE;
    constexpr int kLoads = (TM + TE) * 8 / kThreads, kStage = (TM + TE) * kStep;
    static_assert((TM + TE) * 8 % kThreads == 0 && TM * 8 % kThreads == 0, "whole rounds of loads");
    extern __shared__ uint8_t smem[];
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int id = gi::xcd_order(blockIdx.x, gridDim.x);
    // Eight tiles of positions by the tiles of channels, then the next eight.
    const int band = id / (8 * a.e_tiles), in_band = id - band * 8 * a.e_tiles;
    const int wide = min(8, a.n_tiles - band * 8);
    const int n0 = (band * 8 + in_band % wide) * TM, e0 = in_band / wide * TE;
    const int wm = wave % WM, we = wave / WM, half = lane / 32, col = lane % 32;

    bool any = a.lengths == nullptr;
    if (a.lengths) {
        for (int n = n0 + tid; n < min(n0 + TM, a.N); n += kThreads) {
            const int b = n / a.L;
            any = any || n - b * a.L < length_of(a.lengths, b, a.L);
        }
        any = __syncthreads_or(any);
    }

    v16i acc[BM][BE];
#pragma unroll
    for (int i = 0; i < BM; ++i)
#pragma unroll
        for (int j = 0; j < BE; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[i][j][k] = 0;

    if (any) {
        // Each thread's share of a stage: unit tid + p kThreads, at the same offset in every
        // stage.  Rows past the end are the last one again.
        uint32_t from[kLoads];
        const uint8_t *x0 = a.codes + (int64_t)n0 * a.K, *w0 = a.w + (int64_t)e0 * a.K;
        const __amdgpu_buffer_rsrc_t xr = rsrc(x0, (long)min(TM, a.N - n0) * a.K);
        const __amdgpu_buffer_rsrc_t wr = rsrc(w0, (long)min(TE, a.E_ - e0) * a.K);
#pragma unroll
        for (int p = 0; p < kLoads; ++p) {
            const int unit = tid + p * kThreads, row = unit / 8 % (TM + TE);
            const int r = row < TM ? min(row, a.N - n0 - 1) : min(row - TM, a.E_ - e0 - 1);
            from[p] = r * a.K + (unit % 8 ^ (row / 2 % 8)) * 16;
        }
        const auto stage = [&](int to, int k) {
            uint8_t *lds = smem + to * kStage + wave * 1024;
#pragma unroll
            for (int p = 0; p < kLoads; ++p)
                load_lds(p * kThreads < TM * 8 ? xr : wr, lds + p * kThreads * 16, from[p], k * kStep);
        };
        // A block's row r holds position r / 4 % 2 * 16 + r / 8 * 4 + r % 4, so that a lane's 16
        // sums are consecutive positions.
        const int pos = col / 4 % 2 * 16 + col / 8 * 4 + col % 4;
        const int steps = a.K / kStep;
        stage(0, 0);
        for (int k = 0; k < steps; ++k) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            gi::lds_barrier();
            if (k + 1 < steps) stage((k + 1) & 1, k + 1);
            const uint8_t *x = smem + (k & 1) * kStage, *w = x + TM * kStep;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                v4i fx[BM], fw[BE];
                const int u = kk * 2 + half;
#pragma unroll
                for (int i = 0; i < BM; ++i) {
                    const int row = (wm * BM + i) * 32 + pos;
                    fx[i] = *reinterpret_cast<const v4i *>(x + row * kStep + (u ^ (row / 2 % 8)) * 16);
                }
#pragma unroll
                for (int j = 0; j < BE; ++j) {
                    const int row = (we * BE + j) * 32 + col;
                    fw[j] = *reinterpret_cast<const v4i *>(w + row * kStep + (u ^ (row / 2 % 8)) * 16);
                }
#pragma unroll
                for (int i = 0; i < BM; ++i)
#pragma unroll
                    for (int j = 0; j < BE; ++j)
                        acc[i][j] = mfma(fx[i], fw[j], acc[i][j]);
            }
        }
    }

#pragma unroll
    for (int i = 0; i < BM; ++i) {
        const int n = n0 + (wm * BM + i) * 32 + half * 16;
        if (n >= a.N) continue;
        int b = n / a.L, l = n - b * a.L;
        const bool whole = n + 16 <= a.N && l + 16 <= a.L;
        float sx[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) sx[k] = a.scales[min(n + k, a.N - 1)];
#pragma unroll
        for (int j = 0; j < BE; ++j) {
            const int e = e0 + (we * BE + j) * 32 + col;
            if (e >= a.E_) continue;
            const float sw = a.w_scales[e], bias = a.bias ? a.bias[e] : 0.f;
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int sum = acc[i][j][k];
                v[k] = __builtin_fmaf((float)sum, sx[k] * sw, bias);
            }
            if (whole) {
                if (a.lengths) {
                    const int left = length_of(a.lengths, b, a.L) - l;
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = left > k ? v[k] : 0.f;
                }
                store_vec<E, 16>(a.y.row(b, e) + l, v);
            } else {
                int bk = b, lk = l;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    if (n + k >= a.N) continue;
                    const bool in = lk < length_of(a.lengths, bk, a.L);
                    a.y.row(bk, e)[lk] = E::down(in ? v[k] : 0.f);
                    if (++lk == a.L) lk = 0, ++bk;
                }
            }
        }
    }
}

template <class E, int WM, int WE, int BM, int BE>
hipError_t product(const project_int8_args &a, hipStream_t s) {
    constexpr int TM = 32 * WM * BM, TE = 32 * WE * BE;
    const int64_t N = (int64_t)a.B * a.L;
    Project<E> k{static_cast<const uint8_t *>(a.codes), static_cast<const uint8_t *>(a.w), a.scales,
                 a.w_scales, a.bias, view<E>(a.y), a.lengths, (int)N, a.E, a.L, a.K,
                 (int)((N + TM - 1) / TM), (a.E + TE - 1) / TE};
    constexpr int bytes = 2 * (TM + TE) * kStep;
    if (bytes > 64 * 1024) {
        hipError_t e = hipFuncSetAttribute((const void *)project<E, WM, WE, BM, BE>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    project<E, WM, WE, BM, BE>
        <<<(unsigned)((int64_t)k.n_tiles * k.e_tiles), 64 * WM * WE, bytes, s>>>(k);
    return hipGetLastError();
}

template <class E>
hipError_t product_any(const project_int8_args &a, hipStream_t s) {
    const int64_t N = (int64_t)a.B * a.L;
    const auto tiles = [&](int64_t t) { return (N + t - 1) / t * ((a.E + t - 1) / t); };
    if (tiles(256) >= 192) return product<E, 2, 4, 4, 2>(a, s);
    if (tiles(128) >= 192) return product<E, 2, 2, 2, 2>(a, s);
    return product<E, 2, 2, 1, 1>(a, s);
}

int64_t code_row(int64_t D) { return (D + SEQ_INT8_ROW - 1) / SEQ_INT8_ROW * SEQ_INT8_ROW; }

template <class E>
hipError_t step(const project_int8_step_args &a, hipStream_t s) {
    quantize_tokens_args q = {};
    q.dtype = a.dtype, q.B = a.B, q.D = a.D, q.L = 1, q.K = a.K, q.x = a.x;
    q.codes = a.workspace;
    q.scales = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + (int64_t)a.B * a.K);
    hipError_t e = quantize<E>(q, s);
    if (e != hipSuccess) return e;
    project_int8_args p = {};
    p.dtype = a.dtype, p.B = a.B, p.E = a.E, p.L = 1, p.K = a.K;
    p.codes = q.codes, p.scales = q.scales, p.w = a.w, p.w_scales = a.w_scales, p.bias = a.bias;
    p.y = a.y;
    return product_any<E>(p, s);
}

}  // namespace

int64_t project_step_workspace(int B, int D, int) { return B * (code_row(D) + (int64_t)sizeof(float)); }

hipError_t launch_quantize(const quantize_tokens_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? quantize<F32>(a, s)
           : a.dtype == SEQ_BF16 ? quantize<BF16>(a, s) : quantize<F16>(a, s);
}
hipError_t launch_project(const project_int8_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? product_any<F32>(a, s)
           : a.dtype == SEQ_BF16 ? product_any<BF16>(a, s) : product_any<F16>(a, s);
}
hipError_t launch_project_step(const project_int8_step_args &a, hipStream_t s) {
    return a.dtype == SEQ_F32 ? step<F32>(a, s)
           : a.dtype == SEQ_BF16 ? step<BF16>(a, s) : step<F16>(a, s);
}

}  // namespace seq
