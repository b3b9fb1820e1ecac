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
    float times, most, inv;   // 127 2^k, 2^k most, 1 / (2^k most)
    uint32_t keep;            // 0 where the row has no codes: zeros, or no numbers
};
__device__ __forceinline__ Coder coder(uint32_t most_bits) {
    Coder c;
    const float most = __builtin_bit_cast(float, most_bits);
    const float power = most > 0x1p100f ? 0x1p-64f : most < 0x1p-60f ? 0x1p64f : 1.f;
    c.times = 127.f * power;
    c.most = most * power;
    c.inv = __builtin_amdgcn_rcpf(c.most);
    c.keep = most_bits != 0 && most_bits < 0x7f800000u ? ~0u : 0u;
    return c;
}
__device__ __forceinline__ float row_scale(uint32_t most_bits) {
    return most_bits < 0x7f800000u ? __builtin_bit_cast(float, most_bits) / 127.f
                                   : __builtin_bit_cast(float, 0x7fc00000u);
}
// The code is the low byte of what is returned: adding 1.5 2^23 rounds to an integer, ties
// to even, and leaves it in the low bits.
//
// 16-bit numbers: 127 v is exact in fp32.  One step of Newton's method makes the quotient
// exact wherever it is half a step between two codes (it is a float then), and off by at
// most 2^-24 of it elsewhere, where it is at least 2^-18 of it away from the border.
// float32: the remainder of the nearest candidate, against half of most; 127 v has a low
// part, and every other term is exact.
template <class E>
__device__ __forceinline__ uint32_t code(float v, const Coder &c) {
    const float hi = v * c.times, q = hi * c.inv;
    if constexpr (!std::is_same_v<E, F32>) {
        const float exact = __builtin_fmaf(__builtin_fmaf(-q, c.most, hi), c.inv, q);
        return __builtin_bit_cast(uint32_t, exact + 12582912.f);
    } else {
        const float k = __builtin_rintf(q);
        const float r = __builtin_fmaf(-k, c.most, hi), lo = __builtin_fmaf(v, c.times, -hi);
        const float over = (__builtin_fabsf(r) - 0.5f * c.most) + (r < 0.f ? -lo : lo);
        const uint32_t n = __builtin_bit_cast(uint32_t, k + 12582912.f);
        return over > 0.f || (over == 0.f && (n & 1)) ? n + (r < 0.f ? -1 : 1) : n;
    }
}
// Four low bytes.
__device__ __forceinline__ uint32_t pack(const uint32_t (&n)[4], uint32_t keep) {
    const uint32_t lo = __builtin_amdgcn_perm(n[1], n[0], 0x0c0c0400u);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[3], n[2], 0x04000c0cu), lo, 0x07060100u) & keep;
}

// The largest magnitudes of rows, as bits: those of |v| order like the numbers, infinities
// and NaN above all.  16-bit numbers come in pairs.
__device__ __forceinline__ uint32_t raise(uint32_t most, uint32_t bits, F32) {
    return max(most, bits & 0x7fffffffu);
}
template <class E>
__device__ __forceinline__ uint32_t raise(uint32_t most, uint32_t bits, E) {
    typedef unsigned short Pair __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
        __builtin_bit_cast(Pair, most), __builtin_bit_cast(Pair, bits & 0x7fff7fffu)));
}
// Bits of the float that a magnitude is.
template <class E>
__device__ __forceinline__ uint32_t wide(uint32_t bits) {
    return __builtin_bit_cast(uint32_t, E::up(__builtin_bit_cast(
        typename E::type, (std::conditional_t<sizeof(typename E::type) == 4, uint32_t, uint16_t>)bits)));
}

template <class E>
struct Quantize {
    View<E> x;
    uint32_t *codes;   // [B, L, K / 4]
    float *scales;
    const int32_t *lengths;
    int B, D, L, K, tiles;
};

// Positions along the lanes.  A work-group has 64 bytes of positions, its 1024 threads V
// of them (16 bytes) and four channels at a time, 1024 channels in a round.  The first
// KEPT rounds stay in registers between the two passes, over the maximum and over the
// codes; what is beyond is read again.  A wave's loads are 64 bytes of 16 channels, its
// stores 64 bytes of codes of 4 positions.
template <class E>
constexpr int kTilePositions = 64 / (int)sizeof(typename E::type);

template <class E, int KEPT>
__global__ __launch_bounds__(1024) void quantize_tile(Quantize<E> a) {
    using T = typename E::type;
    constexpr int V = 16 / (int)sizeof(T), TT = 4 * V;
    typedef typename Vec<T, V>::type Some;
    __shared__ uint32_t meet[16][16];
    const int id = gi::xcd_order(blockIdx.x, gridDim.x);
    const int b = id / a.tiles, t0 = id % a.tiles * TT;
    const int len = length_of(a.lengths, b, a.L);
    const int group = threadIdx.x % 4, quad = threadIdx.x / 4, t = t0 + group * V;
    const int left = len - t;
    const auto load = [&](int d) {
        Some v;
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = 0;
        if (d < a.D && left > 0) {
            const T *p = a.x.row(b, d) + t;
            if (left >= V) {
                v = *reinterpret_cast<const Some *>(p);
            } else {
                T u[V];
                load_end(p, left, u);
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = u[k];
            }
        }
        return v;
    };
    Some kept[KEPT][4];
#pragma unroll
    for (int r = 0; r < KEPT; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) kept[r][j] = load(r * 1024 + quad * 4 + j);
    // Four words of V positions each.
    uint32_t words[4] = {0, 0, 0, 0};
    const auto see = [&](const Some &v) {
        const v4i bits = __builtin_bit_cast(v4i, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int word = bits[k];
            words[k] = raise(words[k], word, E{});
        }
    };
#pragma unroll
    for (int r = 0; r < KEPT; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) see(kept[r][j]);
    for (int d = KEPT * 1024 + quad * 4; d < a.D; d += 1024) {
        Some v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load(d + j);
#pragma unroll
        for (int j = 0; j < 4; ++j) see(v[j]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int s = 4; s < 64; s *= 2)
            words[k] = raise(words[k], (uint32_t)__shfl_xor((int)words[k], s, 64), E{});
        if (threadIdx.x % 64 < 4) meet[threadIdx.x / 64][group * 4 + k] = words[k];
    }
    __syncthreads();
    Coder c[V];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int w = 0; w < 16; ++w) words[k] = raise(words[k], meet[w][group * 4 + k], E{});
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            const int at = k * (V / 4) + h;
            const uint32_t most = wide<E>(words[k] >> 16 * h);
            c[at] = coder(most);
            if (quad == 0 && t + at < a.L) a.scales[(int64_t)b * a.L + t + at] = row_scale(most);
        }
    }
    uint32_t *codes = a.codes + ((int64_t)b * a.L + t) * (a.K / 4);
    const auto write = [&](int d, const Some (&v)[4]) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            uint32_t n[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const T e = v[j][k];
                n[j] = code<E>(E::up(e), c[k]);
            }
            if (t + k < a.L) codes[k * (a.K / 4) + d / 4] = pack(n, c[k].keep);
        }
    };
#pragma unroll
    for (int r = 0; r < KEPT; ++r) {
        const int d = r * 1024 + quad * 4;
        if (d < a.K) write(d, kept[r]);
    }
    for (int d = KEPT * 1024 + quad * 4; d < a.K; d += 1024) {
        Some v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load(d + j);
        write(d, v);
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
        for (int k = 0; k < 8; ++k) most = raise(most, __builtin_bit_cast(uint32_t, v.at(k)), F32{});
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
        uint32_t n[2][4];
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k / 4][k % 4] = code<E>(v.at(k), c);
        uint2 *to = reinterpret_cast<uint2 *>(a.codes + ((int64_t)b * a.K + d) / 4);
        *to = uint2{pack(n[0], c.keep), pack(n[1], c.keep)};
    }
}

template <class E>
hipError_t quantize(const quantize_tokens_args &a, hipStream_t s) {
    Quantize<E> k{view<E>(a.x), static_cast<uint32_t *>(a.codes), a.scales, a.lengths,
                  a.B, a.D, a.L, a.K, (a.L + kTilePositions<E> - 1) / kTilePositions<E>};
    if (a.L == 1 && (a.x.channel == 1 || a.D == 1)) {
        quantize_row<E><<<(unsigned)a.B, 256, 0, s>>>(k);
    } else {
        const auto kernel = a.D <= 1024 ? quantize_tile<E, 1>
                            : a.D <= 2048 ? quantize_tile<E, 2> : quantize_tile<E, 4>;
        kernel<<<(unsigned)(a.B * (int64_t)k.tiles), 1024, 0, s>>>(k);
    }
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
