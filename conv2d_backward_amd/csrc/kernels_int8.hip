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
// Until at most N of this wave's loads are on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ v16i mfma(v4i a, v4i b, v16i c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v4i mfma16(v4i a, v4i b, v4i c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Writes consecutive positions n .. n + V - 1 (n < N, counted over the batch) of channel e.
template <class E, int V>
__device__ __forceinline__ void store_positions(const Project<E> &a, int n, int e, float (&v)[V]) {
    int b = n / a.L, l = n - b * a.L;
    if (n + V <= a.N && l + V <= a.L) {
        if (a.lengths) {
            const int left = length_of(a.lengths, b, a.L) - l;
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = left > k ? v[k] : 0.f;
        }
        store_vec<E, V>(a.y.row(b, e) + l, v);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (n + k >= a.N) continue;
            const bool in = l < length_of(a.lengths, b, a.L);
            a.y.row(b, e)[l] = E::down(in ? v[k] : 0.f);
            if (++l == a.L) l = 0, ++b;
        }
    }
}

// Tiles of TM positions and TE channels; waves in WM x WE, each with BM x BE blocks of
// 32 x 32.  Steps of 128 bytes of k go to LDS by direct loads, ST - 1 ahead.  In
// LDS a row is eight 16-byte units, unit u at u ^ (row / 2 % 8): the 16 lanes that a
// cycle of ds_read_b128 serves then read 16 different units of 256 bytes.
template <class E, int WM, int WE, int BM, int BE, int ST>
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
#pragma unroll
        for (int k = 0; k < ST - 1; ++k)
            if (k < steps) stage(k, k);
        for (int k = 0, at = 0; k < steps; ++k, at = at + 1 < ST ? at + 1 : 0) {
            // Step k is there: all but the ST - 2 behind it, or, at the end, all.
            if (steps - k > ST - 2)
                wait_loads<(ST - 2) * kLoads>();
            else
                wait_loads<0>();
            gi::lds_barrier();
            if (k + ST - 1 < steps) stage(at ? at - 1 : ST - 1, k + ST - 1);
            const uint8_t *x = smem + at * kStage, *w = x + TM * kStep;
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
            store_positions<E, 16>(a, n, e, v);
        }
    }
}

template <class E>
Project<E> project_of(const project_int8_args &a) {
    return {static_cast<const uint8_t *>(a.codes), static_cast<const uint8_t *>(a.w), a.scales,
            a.w_scales, a.bias, view<E>(a.y), a.lengths, (int)((int64_t)a.B * a.L), a.E, a.L, a.K, 0, 0};
}

template <class E, int WM, int WE, int BM, int BE, int ST>
hipError_t product(const project_int8_args &a, hipStream_t s) {
    constexpr int TM = 32 * WM * BM, TE = 32 * WE * BE;
    Project<E> k = project_of<E>(a);
    k.n_tiles = (k.N + TM - 1) / TM, k.e_tiles = (a.E + TE - 1) / TE;
    constexpr int bytes = ST * (TM + TE) * kStep;
    if (bytes > 64 * 1024) {
        hipError_t e = hipFuncSetAttribute((const void *)project<E, WM, WE, BM, BE, ST>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    project<E, WM, WE, BM, BE, ST>
        <<<(unsigned)((int64_t)k.n_tiles * k.e_tiles), 64 * WM * WE, bytes, s>>>(k);
    return hipGetLastError();
}

// The largest of `lanes` (a power of two, 32 or 64) lanes, in each of them.
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int lanes) {
    const auto turned = [](uint32_t u, auto by) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, kRowRor + decltype(by)::value, 0xf, 0xf, true);
    };
    v = max(v, turned(v, std::integral_constant<int, 1>{}));
    v = max(v, turned(v, std::integral_constant<int, 2>{}));
    v = max(v, turned(v, std::integral_constant<int, 4>{}));
    v = max(v, turned(v, std::integral_constant<int, 8>{}));
    // Rows of 16 lanes.
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    const uint32_t low = max(a, b), high = max(c, d);
    return lanes == 64 ? max(low, high) : threadIdx.x % 64 < 32 ? low : high;
}

// Products too small to fill the chip with whole rows of k: a work-group has RB blocks of 16
// channels and NB of 16 positions, and its S waves share k by steps of 128 bytes, wave w with
// every S-th; their sums meet in LDS.  Each wave brings its steps by direct loads through a
// ring of DEPTH steps of its own, without a barrier: lanes 8 to a row, because loads straight
// into operands (each lane another row) reach 9.4 TB/s from the caches where these reach 28.
// Rows are swizzled as in `project`.
//
// What the results are laid out along decides which operand is the first: a lane has four
// consecutive rows of it.  Along channels (one position a row), the weights.  Along
// positions, the positions, in the order that gives a lane 4 NB consecutive ones.  With
// codes inside (at most 16 positions, along channels) they are made here, from x, by every
// work-group for itself, and wait in LDS, unit u of row r at u ^ r in each 256 bytes.
enum Form { kAlongChannels, kCodesInside, kAlongPositions };

template <class E>
struct Split {
    Project<E> p;
    View<E> x;   // [N, D]
    int D, share;
};

template <class E, int RB, int NB, int S, int DEPTH, int FORM>
__global__ __launch_bounds__(64 * S) void project_split(Split<E> t) {
    constexpr bool CODES = FORM == kCodesInside;
    static_assert(!CODES || NB == 1, "the codes of 16 rows");
    constexpr int ROWS = 16 * (RB + (CODES ? 0 : NB)), kLoads = ROWS / 8, kEntry = ROWS * kStep;
    const Project<E> &a = t.p;
    extern __shared__ uint8_t smem[];
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    constexpr int kRing = DEPTH * kEntry, kMeet = RB * NB * 1024;   // bytes of a wave
    uint8_t *const ring = smem + wave * kRing;
    v4i *const meet = reinterpret_cast<v4i *>(smem);   // after the rings
    float *const own_scales = reinterpret_cast<float *>(smem + S * (kRing > kMeet ? kRing : kMeet));
    uint8_t *const own = reinterpret_cast<uint8_t *>(own_scales + 64);   // [16][pitch]
    const int pitch = (a.K + 255) / 256 * 256;
    // Work-groups of the same positions or, where there are more of those, channels follow
    // each other on one die.
    const int id = gi::xcd_order(blockIdx.x, gridDim.x);
    const int e0 = id % a.e_tiles * RB * 16, n0 = id / a.e_tiles * NB * 16;
    const int row = lane % 16, part = lane / 16;
    const int steps = a.K / kStep;
    // Work-groups start at different places, so that rows a power of two apart do not all
    // come from the same channel of the caches (1 position, 4096 x 4096: 5.7 -> 5.2 us).
    const int turn = id % steps;
    const int mine = (steps - wave + S - 1) / S;   // steps of this wave
    const auto place = [&](int j) {
        const int k = wave + j * S + turn;
        return k < steps ? k : k - steps;
    };

    // Codes inside: a row of x has `share` threads, a power of two; its numbers are on their
    // way before the weights.
    constexpr int KEPT = CODES ? 8 : 1;   // octets of a thread that stay in registers
    const int share = t.share, own_row = tid / share, first = tid % share * 8;
    const auto load = [&](int d) {
        Octet<E> v;
        if (t.x.channel == 1) {
            v.load(t.x.row(own_row, 0) + d, t.D - d);
        } else {
            v.zero();
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (d + k < t.D) v.v[k] = *t.x.row(own_row, d + k);
        }
        return v;
    };
    Octet<E> kept[KEPT];
    const int end = CODES && own_row < a.N ? t.D : 0;
    if constexpr (CODES) {
#pragma unroll
        for (int i = 0; i < KEPT; ++i) {
            kept[i].zero();
            if (first + i * share * 8 < end) kept[i] = load(first + i * share * 8);
        }
    }

    const auto wr = rsrc(a.w + (int64_t)e0 * a.K, (long)min(16 * RB, a.E_ - e0) * a.K);
    const auto xr = rsrc(a.codes + (CODES ? 0 : (int64_t)n0 * a.K),
                         CODES ? 0 : (long)min(16 * NB, a.N - n0) * a.K);
    uint32_t from[kLoads];
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
        const int r = p * 8 + lane / 8, unit = lane % 8 ^ (r / 2 % 8);
        const int held = r < 16 * RB ? min(r, a.E_ - e0 - 1) : min(r - 16 * RB, a.N - n0 - 1);
        from[p] = held * a.K + unit * 16;
    }
    const auto bring = [&](int j) {
#pragma unroll
        for (int p = 0; p < kLoads; ++p)
            load_lds(p < 2 * RB ? wr : xr, ring + j % DEPTH * kEntry + p * 1024, from[p],
                     place(j) * kStep);
    };
#pragma unroll
    for (int j = 0; j < DEPTH; ++j)
        if (j < mine) bring(j);

    if constexpr (CODES) {
        uint32_t most = 0;
        const auto see = [&](const Octet<E> &v) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                most = raise(most, __builtin_bit_cast(uint32_t, v.at(k)), F32{});
        };
#pragma unroll
        for (int i = 0; i < KEPT; ++i) see(kept[i]);
        for (int d = first + KEPT * share * 8; d < end; d += share * 8) see(load(d));
        most = lanes_max(most, share < 64 ? share : 64);
        if (share > 64) {
            uint32_t *const parts = reinterpret_cast<uint32_t *>(own_scales + 16);
            if (lane == 0) parts[wave] = most;
            gi::lds_barrier();
            for (int w = 0; w < share / 64; ++w) most = max(most, parts[tid / share * (share / 64) + w]);
        }
        const Coder c = coder(most);
        if (first == 0) own_scales[own_row] = row_scale(most);
        const auto write = [&](int d, const Octet<E> &v) {
            uint32_t q[2][4];
#pragma unroll
            for (int k = 0; k < 8; ++k) q[k / 4][k % 4] = code<E>(v.at(k), c);
            *reinterpret_cast<uint2 *>(own + own_row * pitch + ((d / 16) ^ own_row) * 16 + d % 16) =
                uint2{pack(q[0], c.keep), pack(q[1], c.keep)};
        };
        const int bytes = own_row < a.N ? a.K : 0;
#pragma unroll
        for (int i = 0; i < KEPT; ++i)
            if (first + i * share * 8 < bytes) write(first + i * share * 8, kept[i]);
        for (int d = first + KEPT * share * 8; d < bytes; d += share * 8) write(d, load(d));
        gi::lds_barrier();
    }

    v4i acc[RB][NB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[r][n] = v4i{0, 0, 0, 0};
    // Along positions, row r of block n is position r / 4 * 4 NB + n * 4 + r % 4.
    const int x_row = FORM == kAlongPositions ? row / 4 * 4 * NB + row % 4 : row;
    for (int j = 0; j < mine; ++j) {
        // Step j is there: all but the DEPTH - 1 behind it, or, at the end, all.
        if (mine - j >= DEPTH)
            wait_loads<(DEPTH - 1) * kLoads>();
        else
            wait_loads<0>();
        const uint8_t *at = ring + j % DEPTH * kEntry;
        v4i fw[RB][2], fx[NB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int u = h * 4 + part;
#pragma unroll
            for (int r = 0; r < RB; ++r)
                fw[r][h] = *reinterpret_cast<const v4i *>(at + (r * 16 + row) * kStep +
                                                          (u ^ (row / 2 % 8)) * 16);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int xn = x_row + n * (FORM == kAlongPositions ? 4 : 16);
                fx[n][h] = *reinterpret_cast<const v4i *>(
                    CODES ? own + row * pitch + ((place(j) * 8 + u) ^ row) * 16
                          : at + (RB * 16 + xn) * kStep + (u ^ (xn / 2 % 8)) * 16);
            }
        }
        if (j + DEPTH < mine) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the ring's place is read
            bring(j + DEPTH);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    acc[r][n] = FORM == kAlongPositions ? mfma16(fx[n][h], fw[r][h], acc[r][n])
                                                        : mfma16(fw[r][h], fx[n][h], acc[r][n]);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < NB; ++n) meet[((r * NB + n) * S + wave) * 64 + lane] = acc[r][n];
    __syncthreads();
    const auto sum_of = [&](int block) {
        v4i sum = meet[block * S * 64 + lane];
#pragma unroll
        for (int s = 1; s < S; ++s) sum += meet[(block * S + s) * 64 + lane];
        return sum;
    };
    if constexpr (FORM == kAlongPositions) {
        for (int r = wave; r < RB; r += S) {
            const int e = e0 + r * 16 + row, n = n0 + part * 4 * NB;
            if (e >= a.E_ || n >= a.N) continue;
            float v[4 * NB];
            const float sw = a.w_scales[e], bias = a.bias ? a.bias[e] : 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const v4i sum = sum_of(r * NB + i);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int one = sum[k];
                    v[4 * i + k] = __builtin_fmaf(
                        (float)one, a.scales[min(n + 4 * i + k, a.N - 1)] * sw, bias);
                }
            }
            store_positions<E, 4 * NB>(a, n, e, v);
        }
    } else {
        for (int block = wave; block < RB * NB; block += S) {
            const int n = n0 + block % NB * 16 + lane % 16;
            const int e = e0 + block / NB * 16 + lane / 16 * 4;
            if (n >= a.N || e >= a.E_) continue;
            const v4i sum = sum_of(block);
            const int b = n / a.L, l = n - b * a.L;
            const bool in = l < length_of(a.lengths, b, a.L);
            const float sx = CODES ? own_scales[n] : a.scales[n];
            auto *y = a.y.row(b, e) + l;
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int ek = min(e + k, a.E_ - 1), one = sum[k];
                v[k] = __builtin_fmaf((float)one, sx * a.w_scales[ek], a.bias ? a.bias[ek] : 0.f);
                v[k] = in ? v[k] : 0.f;
            }
            if (a.y.channel == 1 && e + 4 <= a.E_) {
                store_vec<E, 4>(y, v);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (e + k < a.E_) y[k * a.y.channel] = E::down(v[k]);
            }
        }
    }
}

template <class E, int RB, int NB, int S, int DEPTH, int FORM>
hipError_t split(const project_int8_args &a, const seq_tensor &x, int D, hipStream_t s) {
    constexpr bool CODES = FORM == kCodesInside;
    Split<E> k{project_of<E>(a), view<E>(x), D, 64 * S / 16};
    k.p.n_tiles = (k.p.N + 16 * NB - 1) / (16 * NB), k.p.e_tiles = (a.E + 16 * RB - 1) / (16 * RB);
    if constexpr (CODES)
        while (k.share < 64 * S && 64 * S / k.share / 2 >= k.p.N) k.share *= 2;
    constexpr int kRing = DEPTH * 16 * (RB + (CODES ? 0 : NB)) * kStep, kMeet = RB * NB * 1024;
    const int bytes = S * std::max(kRing, kMeet) + 256 + (CODES ? 16 * ((a.K + 255) / 256 * 256) : 0);
    if (bytes > 64 * 1024) {
        hipError_t e = hipFuncSetAttribute((const void *)project_split<E, RB, NB, S, DEPTH, FORM>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    project_split<E, RB, NB, S, DEPTH, FORM>
        <<<(unsigned)((int64_t)k.p.n_tiles * k.p.e_tiles), 64 * S, bytes, s>>>(k);
    return hipGetLastError();
}

template <class E, int FORM>
hipError_t split_any(const project_int8_args &a, hipStream_t s) {
    const int64_t N = (int64_t)a.B * a.L;
    if (N <= 16) return a.E > 4096 ? split<E, 2, 1, 8, 2, FORM>(a, {}, 0, s) : split<E, 1, 1, 8, 2, FORM>(a, {}, 0, s);
    if (N <= 32) return a.E > 4096 ? split<E, 2, 2, 8, 1, FORM>(a, {}, 0, s) : split<E, 1, 2, 8, 1, FORM>(a, {}, 0, s);
    if (N <= 64 && a.E <= 2048) return split<E, 1, 2, 8, 2, FORM>(a, {}, 0, s);
    return split<E, 2, 4, 8, 1, FORM>(a, {}, 0, s);
}

template <class E>
hipError_t product_any(const project_int8_args &a, hipStream_t s) {
    const int64_t N = (int64_t)a.B * a.L;
    const auto tiles = [&](int64_t t) { return (N + t - 1) / t * ((a.E + t - 1) / t); };
    if (N <= 64 || tiles(64) <= 128)
        return a.L == 1 ? split_any<E, kAlongChannels>(a, s) : split_any<E, kAlongPositions>(a, s);
    if (tiles(256) >= 192) return product<E, 2, 4, 4, 2, 2>(a, s);
    if (tiles(128) >= 192) return product<E, 2, 4, 2, 1, 2>(a, s);
    return product<E, 2, 2, 1, 1, 3>(a, s);
}

int64_t code_row(int64_t D) { return (D + SEQ_INT8_ROW - 1) / SEQ_INT8_ROW * SEQ_INT8_ROW; }

// Whether every work-group makes the codes of a single-position call for itself: at most 16
// rows, few enough numbers, and room in LDS for their codes.
bool codes_inside(int64_t B, int64_t D) {
    return B <= 16 && B * D <= 32768 && D <= 8192;
}

template <class E>
hipError_t step(const project_int8_step_args &a, hipStream_t s) {
    project_int8_args p = {};
    p.dtype = a.dtype, p.B = a.B, p.E = a.E, p.L = 1, p.K = a.K;
    p.w = a.w, p.w_scales = a.w_scales, p.bias = a.bias, p.y = a.y;
    if (codes_inside(a.B, a.D))
        return a.E > 4096 ? split<E, 2, 1, 8, 2, kCodesInside>(p, a.x, a.D, s)
                          : split<E, 1, 1, 8, 2, kCodesInside>(p, a.x, a.D, s);
    quantize_tokens_args q = {};
    q.dtype = a.dtype, q.B = a.B, q.D = a.D, q.L = 1, q.K = a.K, q.x = a.x;
    q.codes = a.workspace;
    q.scales = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + (int64_t)a.B * a.K);
    hipError_t e = quantize<E>(q, s);
    if (e != hipSuccess) return e;
    p.codes = q.codes, p.scales = q.scales;
    return product_any<E>(p, s);
}

}  // namespace

int64_t project_step_workspace(int B, int D) {
    return codes_inside(B, D) ? 0 : B * (code_row(D) + (int64_t)sizeof(float));
}

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
