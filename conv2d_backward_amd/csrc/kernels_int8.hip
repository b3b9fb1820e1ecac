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

// V positions from t of channel d, `left` of them inside the length: what is not is 0.
template <class E, int V>
__device__ __forceinline__ typename Vec<typename E::type, V>::type positions_of(
    const Quantize<E> &a, int b, int d, int t, int left) {
    using T = typename E::type;
    typedef typename Vec<T, V>::type Some;
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
}
// 16 bytes of them into four words of maxima.
template <class E, int V>
__device__ __forceinline__ void see_positions(const typename Vec<typename E::type, V>::type &v,
                                              uint32_t (&words)[4]) {
    const v4i bits = __builtin_bit_cast(v4i, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int word = bits[k];
        words[k] = raise(words[k], word, E{});
    }
}
// Four channels of position k, as codes.
template <class E, int V>
__device__ __forceinline__ uint32_t codes_of(const typename Vec<typename E::type, V>::type (&v)[4], int k,
                                             const Coder &c) {
    uint32_t n[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const typename E::type e = v[j][k];
        n[j] = code<E>(E::up(e), c);
    }
    return pack(n, c.keep);
}

// Positions along the lanes.  A work-group has 16 G bytes of positions, each thread of its W
// waves V of them (16 bytes) and four channels at a time, 256 W / G channels in a round.  The
// first KEPT rounds stay in registers between the two passes, over the maximum and over the
// codes; what is beyond is read again.  With G = 4 a wave's loads are 64 bytes of 16
// channels, its stores 64 bytes of codes of 4 positions.  [1, 4096, 8192] bf16 33.6 us from memory, 3.0
// TB/s of the 4.9 that a copy reaches (23.9 for operands of which the memory-side cache has a part): one
// work-group of 16 waves a compute unit (109 registers), which all read, then all write.
// [4, 2048, 2048] 19.2 (13.1); f32 [2, 2051, 777] 11.9 (8.9): 196 work-groups, one each for 256 units,
// whose numbers take twice the instructions.
template <class E, int G, int W, int KEPT>
__global__ __launch_bounds__(64 * W) void quantize_tile(Quantize<E> a) {
    using T = typename E::type;
    constexpr int V = 16 / (int)sizeof(T), TT = G * V, kRound = 256 * W / G;
    typedef typename Vec<T, V>::type Some;
    __shared__ uint32_t meet[W][4 * G];
    const int id = gi::xcd_order(blockIdx.x, gridDim.x);
    const int b = id / a.tiles, t0 = id % a.tiles * TT;
    const int len = length_of(a.lengths, b, a.L);
    const int group = threadIdx.x % G, quad = threadIdx.x / G, t = t0 + group * V;
    const int left = len - t;
    const auto load = [&](int d) { return positions_of<E, V>(a, b, d, t, left); };
    Some kept[KEPT][4];
#pragma unroll
    for (int r = 0; r < KEPT; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) kept[r][j] = load(r * kRound + quad * 4 + j);
    // Four words of V positions each.
    uint32_t words[4] = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < KEPT; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) see_positions<E, V>(kept[r][j], words);
    for (int d = KEPT * kRound + quad * 4; d < a.D; d += kRound) {
        Some v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load(d + j);
#pragma unroll
        for (int j = 0; j < 4; ++j) see_positions<E, V>(v[j], words);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int s = G; s < 64; s *= 2)
            words[k] = raise(words[k], (uint32_t)__shfl_xor((int)words[k], s, 64), E{});
        if (threadIdx.x % 64 < G) meet[threadIdx.x / 64][group * 4 + k] = words[k];
    }
    __syncthreads();
    Coder c[V];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int w = 0; w < W; ++w) words[k] = raise(words[k], meet[w][group * 4 + k], E{});
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
        for (int k = 0; k < V; ++k)
            if (t + k < a.L) codes[k * (a.K / 4) + d / 4] = codes_of<E, V>(v, k, c[k]);
    };
#pragma unroll
    for (int r = 0; r < KEPT; ++r) {
        const int d = r * kRound + quad * 4;
        if (d < a.K) write(d, kept[r]);
    }
    for (int d = KEPT * kRound + quad * 4; d < a.K; d += kRound) {
        Some v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load(d + j);
        write(d, v);
    }
}

// Few positions with many channels: the channels are shared out too, kSlice to a work-group, and
// two kernels run one after the other.  The first leaves the maxima of each slice where the codes
// of the row will be: a copy of all of them in every slice's place, from where the work-groups
// of the second, which have the same slices, take them before they write their codes over them.
constexpr int kSlice = 512, kSliceG = 4, kSliceW = 8;
constexpr int kMaxSlices = 32;   // copies of so many fit into the 128 bytes that the last slice may have
static_assert(kSlice == 256 * kSliceW / kSliceG, "a slice is a round");

template <class E, bool CODES>
__global__ __launch_bounds__(64 * kSliceW) void quantize_slice(Quantize<E> a) {
    constexpr int G = kSliceG, W = kSliceW, V = 16 / (int)sizeof(typename E::type), TT = G * V;
    typedef typename Vec<typename E::type, V>::type Some;
    __shared__ uint32_t meet[W][4 * G], most[TT];
    const int id = gi::xcd_order(blockIdx.x, gridDim.x), slice = blockIdx.y, slices = gridDim.y;
    const int b = id / a.tiles, t0 = id % a.tiles * TT;
    const int len = length_of(a.lengths, b, a.L);
    const int group = threadIdx.x % G, quad = threadIdx.x / G, t = t0 + group * V;
    const int d = slice * kSlice + quad * 4;
    uint32_t *const row = a.codes + ((int64_t)b * a.L + t0) * (a.K / 4);   // of position t0
    Some v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = positions_of<E, V>(a, b, d + j, t, len - t);
    if constexpr (!CODES) {
        uint32_t words[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) see_positions<E, V>(v[j], words);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int s = G; s < 64; s *= 2)
                words[k] = raise(words[k], (uint32_t)__shfl_xor((int)words[k], s, 64), E{});
            if (threadIdx.x % 64 < G) meet[threadIdx.x / 64][group * 4 + k] = words[k];
        }
        __syncthreads();
        if (threadIdx.x < TT) {
            const int at = threadIdx.x;   // position: V / 4 of them in a word
            uint32_t word = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) word = raise(word, meet[w][at / (V / 4)], E{});
            most[at] = wide<E>(word >> 16 * (at % (V / 4)));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < TT * slices; i += 64 * W) {
            const int at = i / slices, copy = i % slices;
            if (t0 + at < a.L) row[at * (a.K / 4) + copy * (kSlice / 4) + slice] = most[at];
        }
    } else {
        // 64 W / TT threads a position, the first ones of a group of lanes.
        constexpr int kShare = 64 * W / TT;
        const int at = threadIdx.x / kShare;
        uint32_t own = 0;
        if (t0 + at < a.L)
            for (int s = threadIdx.x % kShare; s < slices; s += kShare)
                own = max(own, row[at * (a.K / 4) + slice * (kSlice / 4) + s]);
#pragma unroll
        for (int s = 1; s < kShare; s *= 2) own = max(own, (uint32_t)__shfl_xor((int)own, s, 64));
        if (threadIdx.x % kShare == 0) {
            most[at] = own;
            if (slice == 0 && t0 + at < a.L) a.scales[(int64_t)b * a.L + t0 + at] = row_scale(own);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (t + k < a.L && d < a.K)
                row[(group * V + k) * (a.K / 4) + d / 4] = codes_of<E, V>(v, k, coder(most[group * V + k]));
    }
}

template <class E>
hipError_t quantize_slices(Quantize<E> k, hipStream_t s) {
    constexpr int TT = kSliceG * 16 / (int)sizeof(typename E::type);
    k.tiles = (k.L + TT - 1) / TT;
    const dim3 grid((unsigned)(k.B * (int64_t)k.tiles), (unsigned)((k.D + kSlice - 1) / kSlice));
    quantize_slice<E, false><<<grid, 64 * kSliceW, 0, s>>>(k);
    quantize_slice<E, true><<<grid, 64 * kSliceW, 0, s>>>(k);
    return hipGetLastError();
}

// Channels along the lanes (one position, contiguous channels): a work-group a row.  Two round
// trips and the launch: [64, 4096] bf16 3.2 us.
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

// For more than LOW channels and at most HIGH: the rounds kept are 1, 2 or 4.
template <class E, int G, int W, int LOW, int HIGH>
hipError_t quantize_tiles(Quantize<E> k, hipStream_t s) {
    constexpr int TT = G * 16 / (int)sizeof(typename E::type), kRound = 256 * W / G;
    constexpr int kFewest = LOW < kRound ? 1 : LOW < 2 * kRound ? 2 : 4;
    constexpr int kMost = HIGH <= kRound ? 1 : HIGH <= 2 * kRound ? 2 : 4;
    k.tiles = (k.L + TT - 1) / TT;
    const int kept = k.D <= kRound ? 1 : k.D <= 2 * kRound ? 2 : 4;
    const auto kernel = kept <= kFewest ? quantize_tile<E, G, W, kFewest>
                        : kept < kMost ? quantize_tile<E, G, W, (kMost > 2 && kFewest < 2 ? 2 : kMost)>
                                       : quantize_tile<E, G, W, kMost>;
    kernel<<<(unsigned)(k.B * (int64_t)k.tiles), 64 * W, 0, s>>>(k);
    return hipGetLastError();
}

template <class E>
hipError_t quantize(const quantize_tokens_args &a, hipStream_t s) {
    Quantize<E> k{view<E>(a.x), static_cast<uint32_t *>(a.codes), a.scales, a.lengths,
                  a.B, a.D, a.L, a.K, 0};
    if (a.L == 1 && (a.x.channel == 1 || a.D == 1)) {
        quantize_row<E><<<(unsigned)a.B, 256, 0, s>>>(k);
        return hipGetLastError();
    }
    const int64_t bytes = a.L * (int64_t)sizeof(typename E::type);
    // The channels are shared out too where even the finest share leaves half of the compute
    // units without positions and each of the others with many channels, which bound it ([1,
    // 4096, 100] as long as [1, 4096, 500]); it costs a second launch.  Measured (us, the same
    // operands again and again, as in the table below; shared out / not, bf16): [1, 4096, 500] 8.3 /
    // 11.2, [1, 8192, 100] 7.7 / 18.7, [1, 4096, 2000] 13.7 / 11.0, [1, 2048, 500] 7.7 / 7.2, [64, 4096,
    // 8] 8.5 / 6.1 (a slice has 64 bytes of positions).
    const int64_t groups = a.B * ((bytes + 15) / 16);
    const int slices = (a.D + kSlice - 1) / kSlice;
    if (groups <= 128 && slices > 5 && slices <= kMaxSlices && bytes >= 64)
        return quantize_slices<E>(k, s);
    // Few positions are shared out finer, so that more compute units have some, though a cache
    // line then goes to several of them; positions that end early have no lanes beyond.  More
    // waves to a position where its channels would not stay in registers otherwise.  Measured
    // (us; G, W of 4, 16 / 4, 8 / 2, 16 / 2, 8 / 1, 8): [1, 4096, 8192] bf16 23.9 - 27.6 25.5
    // 29.8, [1, 1024, 8192] 9.6 8.6 11.3 9.7 12.1, [1, 4096, 4096] 18.9 21.9 16.1 15.2 17.0, [2,
    // 2051, 777] f32 13.2 - 9.5 10.1 11.3, [2, 1024, 1000] bf16 6.7 5.8 6.1 5.1 5.6, [5, 1000,
    // 301] f16 8.3 7.3 7.7 6.9 5.8, [512, 2048, 16] bf16 18.5 16.2 15.3 13.3 15.0; 1, 8 / 1, 4:
    // [1024, 2048, 2] 10.7 / 9.0, [2000, 300, 3] 13.3 / 8.4, [256, 4096, 4] 11.7 / 12.3.
    constexpr int kAll = SEQ_MAX_INT8_CHANNELS, kHalf = 8192 / (int)sizeof(typename E::type);
    if (groups < 256) return quantize_tiles<E, 1, 8, 0, kAll>(k, s);
    if (bytes <= 16)
        return a.D <= 2048 ? quantize_tiles<E, 1, 4, 0, 2048>(k, s) : quantize_tiles<E, 1, 8, 2048, kAll>(k, s);
    if (groups >= 1024 && bytes > 32)
        return a.D <= 2048 ? quantize_tiles<E, 4, 8, 0, 2048>(k, s) : quantize_tiles<E, 4, 16, 2048, kAll>(k, s);
    return a.D <= kHalf ? quantize_tiles<E, 2, 8, 0, kHalf>(k, s) : quantize_tiles<E, 2, 16, kHalf, kAll>(k, s);
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
// 4 bytes a lane.
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, uint8_t *lds, uint32_t at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)lds, 4, at, 0, 0, 0);
}
// Until at most N of this wave's loads are on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ v4i mfma16(v4i a, v4i b, v4i c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// The result sum sx sw + bias.  The scales' product is a float of its own, which the sum then multiplies
// in one fused step; of rows near either end of the range that product would leave it where the
// result does not (a sum of 0 times infinity, or digits below the normal range that a sum of 2^30
// brings back), so a scale `is_far` from 1 takes `far_scaled`: the product of the fractions, and
// the powers of two dealt over both factors of the fused step.  Where the product is a normal
// number both give the same bits, so that either may be taken for several results at once.
__device__ __forceinline__ int is_far(float scale) {
    const float size = __builtin_fabsf(scale);
    return (int)(size > 0x1p62f) | ((int)(size < 0x1p-62f) & (int)(size > 0.f));   // (no branches)
}
__device__ __forceinline__ float scaled(float sum, float sx, float sw, float bias) {
    return __builtin_fmaf(sum, sx * sw, bias);
}
__device__ __forceinline__ float far_scaled(float sum, float sx, float sw, float bias) {
    const float fraction = __builtin_amdgcn_frexp_mantf(sx) * __builtin_amdgcn_frexp_mantf(sw);
    const int power = __builtin_amdgcn_frexp_expf(sx) + __builtin_amdgcn_frexp_expf(sw);
    // (1 <= |sum| < 2^31 and 1/4 <= |fraction| < 1 stay normal numbers; powers that both ends cut
    // off make every sum infinite, or nothing.)
    const int of_sum = min(max(power, -126), 96), of_fraction = min(max(power - of_sum, -124), 128);
    return __builtin_fmaf(__builtin_amdgcn_ldexpf(sum, of_sum), __builtin_amdgcn_ldexpf(fraction, of_fraction), bias);
}

// Between the fused step and the rounding to 16 bits: merged into one instruction (v_fma_mixlo_f16)
// they would round once, in some kernels and for some channels, and a result would depend on how many
// positions a call has.
template <int V>
__device__ __forceinline__ void keep_apart(float (&v)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) asm("" : "+v"(v[k]));
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

// 16 bytes of results.
template <class E>
__device__ __forceinline__ uint4 packed(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (std::is_same_v<E, F32>) {
            w[k] = __builtin_bit_cast(uint32_t, v[k]);
        } else {
            using H = std::conditional_t<std::is_same_v<E, BF16>, __bf16, _Float16>;
            typedef float Floats __attribute__((ext_vector_type(2)));
            typedef H Halves __attribute__((ext_vector_type(2)));
            w[k] = __builtin_bit_cast(
                uint32_t, __builtin_convertvector((Floats{v[2 * k], v[2 * k + 1]}), Halves));
        }
    }
    return uint4{w[0], w[1], w[2], w[3]};
}

// The results of a wave, 16 NB positions from n by 16 RB channels from e, whose sums sum(r, k)
// a lane has for position part * 4 NB + k and channel r * 16 + row.  They turn in `turn`, 16
// channels (float32: 8) at a time, so that a store writes whole lines; where the positions are
// not all in one batch item and inside its length, or channels are missing, they leave one by
// one, a lane a position, all of them read before the first leaves (3000 positions, 1024 -> 4096
// channels in tiles of 256: 20.5 us; read one by one 27.5).  Returns whether that took exactly
// RB NB sizeof(T) / 4 stores.  SWAPPED: the bias goes by positions.  far: a scale of the wave's is.
template <class E, int NB, int RB, bool SWAPPED, class Sx, class Sw, class Bias, class Sum>
__device__ __forceinline__ bool leave(const Project<E> &a, int n, int e, uint8_t *turn, bool far, Sx scale_of,
                                      Sw w_scale_of, Bias bias_of, Sum sum) {
    using T = typename E::type;
    // (opaque: addresses that depend on the lane alone would be kept over the caller's steps)
    unsigned lane = threadIdx.x % 64;
    asm volatile("" : "+v"(lane));
    lane &= 63;
    const unsigned row = lane % 16, part = lane / 16;
    constexpr int P = 16 * NB;   // positions, at most a lane each
    const int at = n + (int)(lane % P), b = min(at, a.N - 1) / a.L, l = at - b * a.L;
    const bool here = at < a.N, inside = here && l < length_of(a.lengths, b, a.L);
    const int b0 = __builtin_amdgcn_readfirstlane(b);
    const bool whole = __all(inside && b == b0) && e + 16 * RB <= a.E_;
    float sn[4 * NB], bn[SWAPPED ? 4 * NB : 1];
#pragma unroll
    for (int k = 0; k < 4 * NB; ++k) {
        sn[k] = scale_of(part * 4 * NB + k);
        if constexpr (SWAPPED) bn[k] = bias_of(part * 4 * NB + k);
    }
    // Unit u of row c is at u ^ turned(c).
    constexpr int kLine = P * (int)sizeof(T), kRows = sizeof(T) == 2 ? 16 : 8, kUnits = kLine / 16;
    constexpr int kOwn = kUnits / 4, V = 16 / (int)sizeof(T);   // units of a lane, results of a unit
    constexpr int kPart = 64 / kUnits, kTimes = kRows / kPart;  // rows of a store, stores
    const auto turned = [](unsigned c) {
        return ((c & 2) | (c >> 2 & 1) | (c >> 1 & 4)) & (kUnits - 1);
    };
    uint8_t *put[kOwn];
    const uint8_t *get[kTimes];
#pragma unroll
    for (int u = 0; u < kOwn; ++u)
        put[u] = turn + row % kRows * kLine + ((part * kOwn + u) ^ turned(row % kRows)) * 16;
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
        const unsigned c = i * kPart + lane / kUnits;
        get[i] = turn + c * kLine + (lane % kUnits ^ turned(c)) * 16;
    }
    // (not followed where there is no position)
    T *y = a.y.row(b, e + lane / P) + l;
    if (whole)
        y = a.y.row(b0, e + lane / kUnits) + __builtin_amdgcn_readfirstlane(l) + lane % kUnits * V;
    const int64_t channel = a.y.channel;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        __builtin_amdgcn_sched_barrier(0);
        const float sw = w_scale_of(r * 16 + row);
        float bias = 0.f, v[4 * NB];
        if constexpr (!SWAPPED) bias = bias_of(r * 16 + row);
        if (__builtin_expect(far, 0)) {
#pragma unroll
            for (int k = 0; k < 4 * NB; ++k) {
                const int one = sum(r, k);
                v[k] = far_scaled((float)one, sn[k], sw, SWAPPED ? bn[SWAPPED ? k : 0] : bias);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4 * NB; ++k) {
                const int one = sum(r, k);
                v[k] = scaled((float)one, sn[k], sw, SWAPPED ? bn[SWAPPED ? k : 0] : bias);
            }
        }
        keep_apart(v);
#pragma unroll
        for (int half = 0; half < 16 / kRows; ++half) {
            if (row / kRows == half) {
#pragma unroll
                for (int u = 0; u < kOwn; ++u) *reinterpret_cast<uint4 *>(put[u]) = packed<E>(v + u * V);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            const int c0 = r * 16 + half * kRows;   // the first row's channel
            if (whole) {
                typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
                for (int i = 0; i < kTimes; ++i) {
                    const uint4 o = *reinterpret_cast<const uint4 *>(get[i]);
                    *reinterpret_cast<Words *>(y + (c0 + i * kPart) * channel) = Words{o.x, o.y, o.z, o.w};
                }
            } else {
                // kSide channels at once, kSome of a lane.
                constexpr int kSide = 64 / P, kSome = kRows / kSide;
                const int first = lane / P, rows = a.E_ - e - c0;
                T o[kSome], *to = y + c0 * channel;
#pragma unroll
                for (int i = 0; i < kSome; ++i) {
                    const int c = first + i * kSide;
                    o[i] = *reinterpret_cast<const T *>(
                        turn + c * kLine + ((lane % P / V) ^ turned(c)) * 16 + lane % V * sizeof(T));
                }
                if (here) {
#pragma unroll
                    for (int i = 0; i < kSome; ++i, to += kSide * channel) {
                        asm volatile("" : "+v"(to));   // (opaque: all addresses would be kept)
                        if (first + i * kSide < rows) *to = inside ? o[i] : (T)0;
                    }
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    }
    return whole;
}

// f(row) for positions, and for channels row / 2 % 8 (above `project`).
template <int NB>
__device__ __forceinline__ int position_turn(int row) {
    return row / 2 % 2 + row / (4 * NB) % 4 * 2;
}

// Tiles of positions by channels; waves in WM x WE, each with NB x RB blocks of 16 x 16.
// (The 16 x 16 x 64 product: on numbers that use all bits the chip's power holds it to 4.2
// POP/s where 32 x 32 x 32 is held to 3.4; on zeros both reach 4.9.)  Steps of 128 bytes of
// k go to LDS by direct loads, ST of them there or on their way.  A step is two halves of
// 64 bytes; the operands of a half are read while the products of the one before run, and
// the barrier that hands over a step lies between the halves, so that the matrix cores have
// work across it.
//
// What bounds it: the latency of a step's way from the caches through LDS, which a compute unit hides
// with what other work-groups it has (tiles of 64: three fit; 425 tiles are one or two a unit).
// [5, 1000, 301] x 2000 bf16 12.1 us from memory, 8.9 again (680 TOP/s), [2, 2051, 777] x 1027 f32 13.6
// and 10.1 (650).  Two groups of waves that share the steps of a tile, with half as many barriers,
// took 11.6 and 10.4 where this took 9.1 and 10.2.
//
// SWAPPED: single positions, whose results lie along the channels.  The caller gives the weights
// as positions and the positions as weights; the bias then goes by positions.
//
// In LDS a row is eight 16-byte units, unit u at u ^ f(row), so that the 16 lanes that a
// cycle of ds_read_b128 serves (rows 0..3 and 12..15 of one unit, 4..11 of its neighbour, or
// the others) read 16 different units of 256 bytes.  Row r of block n of the positions is
// position r / 4 * 4 NB + n * 4 + r % 4 of the wave's, which gives a lane 4 NB consecutive ones.
template <class E, int WM, int WE, int NB, int RB, int ST, bool SWAPPED>
__global__ __launch_bounds__(64 * WM * WE, 2) void project(Project<E> a) {
    constexpr int kThreads = 64 * WM * WE, TM = 16 * WM * NB, TE = 16 * WE * RB;
    constexpr int kLoads = (TM + TE) * 8 / kThreads, kStage = (TM + TE) * kStep;
    static_assert((TM + TE) * 8 % kThreads == 0 && TM * 8 % kThreads == 0, "whole rounds of loads");
    static_assert(NB <= 4 && RB <= 4, "a wave's scales of a kind in its lanes");
    extern __shared__ uint8_t smem[];
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int id = gi::xcd_order(blockIdx.x, gridDim.x);
    // Eight tiles of positions by the tiles of channels, then the next eight.
    const int band = id / (8 * a.e_tiles), in_band = id - band * 8 * a.e_tiles;
    const int wide = min(8, a.n_tiles - band * 8);
    const int n0 = (band * 8 + in_band % wide) * TM, e0 = in_band / wide * TE;
    const int wm = wave % WM, we = wave / WM, row = lane % 16, part = lane / 16;

    bool any = a.lengths == nullptr;
    if (a.lengths) {
        for (int n = n0 + tid; n < min(n0 + TM, a.N); n += kThreads) {
            const int b = n / a.L;
            any = any || n - b * a.L < length_of(a.lengths, b, a.L);
        }
        any = __syncthreads_or(any);
    }

    v4i acc[RB][NB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[r][n] = v4i{0, 0, 0, 0};

    // One of the wave's scales of each kind in a lane; on their way beside the first steps.
    const int n = n0 + wm * 16 * NB, e = e0 + we * 16 * RB;
    const float seen_x = a.scales[min(n + lane % (16 * NB), a.N - 1)];
    const float seen_w = a.w_scales[min(e + lane % (16 * RB), a.E_ - 1)];
    if (any) {
        // Each thread's share of a step: unit tid + p kThreads, at the same offset in every
        // step.  Rows past the end are the last one again.
        uint32_t from[kLoads];
        const auto xr = rsrc(a.codes + (int64_t)n0 * a.K, (long)min(TM, a.N - n0) * a.K);
        const auto wr = rsrc(a.w + (int64_t)e0 * a.K, (long)min(TE, a.E_ - e0) * a.K);
#pragma unroll
        for (int p = 0; p < kLoads; ++p) {
            const int r = (tid + p * kThreads) / 8, unit = tid % 8;
            from[p] = r < TM ? min(r, a.N - n0 - 1) * a.K + (unit ^ position_turn<NB>(r)) * 16
                             : min(r - TM, a.E_ - e0 - 1) * a.K + (unit ^ r / 2 % 8) * 16;
        }
        const auto stage = [&](int to, int k) {
            uint8_t *lds = smem + to * kStage + wave * 1024;
#pragma unroll
            for (int p = 0; p < kLoads; ++p)
                load_lds(p * kThreads < TM * 8 ? xr : wr, lds + p * kThreads * 16, from[p], k * kStep);
        };
        // Half h of this lane's rows of block 0; block n of the positions is 512 bytes on,
        // block r of the channels 2048.
        const int x_row = wm * 16 * NB + row / 4 * 4 * NB + row % 4, w_row = we * 16 * RB + row;
        const int x_at = x_row * kStep + (part ^ position_turn<NB>(x_row)) * 16;
        const int w_at = (TM + w_row) * kStep + (part ^ w_row / 2 % 8) * 16;
        struct Operands {
            v4i x[NB], w[RB];
        };
        const auto read = [&](Operands &o, int at, int h) {
            const uint8_t *x = smem + at * kStage + (x_at ^ h * 64), *w = smem + at * kStage + (w_at ^ h * 64);
#pragma unroll
            for (int r = 0; r < RB; ++r) o.w[r] = *reinterpret_cast<const v4i *>(w + r * 2048);
#pragma unroll
            for (int n = 0; n < NB; ++n) o.x[n] = *reinterpret_cast<const v4i *>(x + n * 512);
        };
        const auto multiply = [&](const Operands &o) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int r = 0; r < RB; ++r) acc[r][n] = mfma16(o.x[n], o.w[r], acc[r][n]);
        };
        const int steps = a.K / kStep;
#pragma unroll
        for (int k = 0; k < ST; ++k)
            if (k < steps) stage(k, k);
        if (steps >= ST)
            wait_loads<(ST - 1) * kLoads>();
        else
            wait_loads<0>();
        gi::lds_barrier();
        Operands first, second;
        read(first, 0, 0);
        for (int k = 0, at = 0; k < steps; ++k) {
            const int next = at + 1 < ST ? at + 1 : 0;
            read(second, at, 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(first);
            __builtin_amdgcn_sched_barrier(0);
            // Step k + 1 is there (all but the ST - 2 behind it, or, at the end, all), and
            // everyone has read step k.
            if (steps - k > ST - 1)
                wait_loads<(ST - 2) * kLoads>();
            else
                wait_loads<0>();
            gi::lds_barrier();
            if (k + 1 < steps) read(first, next, 0);
            if (k + ST < steps) stage(at, k + ST);
            __builtin_amdgcn_sched_barrier(0);
            multiply(second);
            __builtin_amdgcn_sched_barrier(0);
            at = next;
        }
    }

    // (every wave has read its last operands before the last barrier)
    const bool far = __any(is_far(seen_x) | is_far(seen_w));
    leave<E, NB, RB, SWAPPED>(
        a, n, e, smem + wave * 2048, far, [&](int k) { return a.scales[min(n + k, a.N - 1)]; },
        [&](int c) { return a.w_scales[min(e + c, a.E_ - 1)]; },
        [&](int i) {
            return !a.bias ? 0.f : SWAPPED ? a.bias[min(n + i, a.N - 1)] : a.bias[min(e + i, a.E_ - 1)];
        },
        [&](int r, int k) { return acc[r][k / 4][k % 4]; });
}

// The same for products that fill the chip: tiles of 256 x 256, one work-group a compute
// unit, which goes through its tiles as one stream of steps: the first steps of the next tile
// are on their way before the last products of this one, and the results leave while they
// come.  [1, 4096, 8192] x 8192 bf16: 224 us from memory, 200 again, 2450 and 2750 TOP/s (a tile by a
// work-group of its own took 250 where this took 207); 8192 x 8192 x 8192: 417 and 381 us, where the
// library's product with int32 results takes 456 again.  What bounds it: LDS and power.  A step takes
// 1.33 us on numbers that use all bits and 1.13 on zeros, at the clock of which the matrix cores alone
// would need 0.85: its 192 KB of reads by eight waves and 64 KB of loads are 2048 cycles of LDS, as many
// as its products take, and do not all lie beside them; the other 0.2 us are power.  The results
// of a tile take 2.9 us beside the steps.
constexpr int kStreamWM = 4, kStreamWE = 2, kStreamNB = 4, kStreamRB = 8;
constexpr int kStreamTile = 256, kStreamWaves = kStreamWM * kStreamWE;
constexpr int kStreamStage = 2 * kStreamTile * kStep;
// LDS: two steps, two sets of the tile's scales and biases, 2 KB a wave for results.
constexpr int kStreamScales = 2 * kStreamStage, kStreamTurn = kStreamScales + 2 * 4096;
constexpr int kStreamBytes = kStreamTurn + kStreamWaves * 2048;

template <class E, bool SWAPPED>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void project_stream(Project<E> a) {
    constexpr int NB = kStreamNB, RB = kStreamRB, TM = kStreamTile, TE = kStreamTile;
    constexpr int kThreads = 64 * kStreamWaves, kLoads = (TM + TE) * 8 / kThreads;
    using T = typename E::type;
    constexpr int kStores = RB * 64 * (int)sizeof(T) / 64;   // of a wave and whole tile
    extern __shared__ uint8_t smem[];
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int wm = wave % kStreamWM, we = wave / kStreamWM, row = lane % 16, part = lane / 16;
    const int tiles = a.n_tiles * a.e_tiles, steps = a.K / kStep;

    struct Tile {
        int n0, e0;
        bool any;   // a position inside a length
    };
    const auto tile_of = [&](int number) {
        const int id = gi::xcd_order(number, tiles);
        const int band = id / (8 * a.e_tiles), in_band = id - band * 8 * a.e_tiles;
        const int wide = min(8, a.n_tiles - band * 8);
        Tile t{(band * 8 + in_band % wide) * TM, in_band / wide * TE, true};
        if (a.lengths) {
            bool any = false;
#pragma unroll 1
            for (int i = 0; i < TM; i += 64) {
                const int n = t.n0 + i + lane, b = min(n, a.N - 1) / a.L;
                any = any || (n < a.N && n - b * a.L < length_of(a.lengths, b, a.L));
            }
            t.any = __any(any);
        }
        return t;
    };

    // Each thread's share of a step: unit tid + p kThreads, 64 rows on each time (which turns
    // the units no further).  Rows past the end are past the resource, and come as zeros.
    __amdgpu_buffer_rsrc_t xr, wr;
    const auto aim = [&](const Tile &t) {
        xr = rsrc(a.codes + (int64_t)t.n0 * a.K, t.any ? (long)min(TM, a.N - t.n0) * a.K : 0);
        wr = rsrc(a.w + (int64_t)t.e0 * a.K, t.any ? (long)min(TE, a.E_ - t.e0) * a.K : 0);
    };
    uint32_t x_from = tid / 8 * a.K + (tid % 8 ^ position_turn<NB>(tid / 8)) * 16;
    uint32_t w_from = tid / 8 * a.K + (tid % 8 ^ tid / 16 % 8) * 16;
    // Load p of a step's kLoads.
    const auto load_one = [&](int to, int k, int p) {
        uint8_t *lds = smem + to * kStreamStage + wave * 1024 + p * kThreads * 16;
        const int rows = p % (kLoads / 2) * 64;
        if (p < kLoads / 2)
            load_lds(xr, lds, x_from + rows * a.K, k * kStep);
        else
            load_lds(wr, lds, w_from + rows * a.K, k * kStep);
    };
    const auto stage = [&](int to, int k) {
#pragma unroll
        for (int p = 0; p < kLoads; ++p) load_one(to, k, p);
    };
    // Scales of the positions, scales of the channels, biases: 256 floats each, 64 a load and
    // two loads a wave (a fourth part is loaded in vain); what is past the end is 0.
    const auto stage_scales = [&](int to, const Tile &t) {
        const int which = wave / 2, of_n = min(TM, a.N - t.n0), of_e = min(TE, a.E_ - t.e0);
        const float *p = which == 0 ? a.scales + t.n0 : a.w_scales + t.e0;
        int held = which == 0 ? of_n : which == 1 ? of_e : 0;
        if (which == 2 && a.bias) p = a.bias + (SWAPPED ? t.n0 : t.e0), held = SWAPPED ? of_n : of_e;
        const auto r = rsrc(reinterpret_cast<const uint8_t *>(p), held * 4L);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int first = wave % 2 * 128 + i * 64;
            load_lds4(r, smem + kStreamScales + to * 4096 + which * 1024 + first * 4, (first + lane) * 4);
        }
    };

    // Half h of this lane's rows of block 0; block n of the positions is 512 bytes on, block r
    // of the channels 2048.
    const int x_row = wm * 16 * NB + row / 4 * 4 * NB + row % 4, w_row = we * 16 * RB + row;
    const int x_at = x_row * kStep + (part ^ position_turn<NB>(x_row)) * 16;
    const int w_at = (TM + w_row) * kStep + (part ^ w_row / 2 % 8) * 16;
    struct Operands {
        v4i x[NB], w[RB];
    };
    // Read i of a half's NB + RB.
    const auto read_one = [&](Operands &o, int at, int h, int i) {
        if (i < NB)
            o.x[i] = *reinterpret_cast<const v4i *>(smem + at * kStreamStage + (x_at ^ h * 64) + i * 512);
        else
            o.w[i - NB] = *reinterpret_cast<const v4i *>(smem + at * kStreamStage + (w_at ^ h * 64) +
                                                         (i - NB) * 2048);
    };
    v4i acc[RB][NB];
    // The products of a half.  Among them, a few apart, go the reads of the half after it and,
    // LOAD, the loads of a step: all at once they would fill the queues in front of the LDS and
    // the caches, and the products behind them would wait (a step 1.6 us for 1.4).
    const auto multiply = [&](const Operands &o, Operands &fill, int from, int h, auto load, int to, int k) {
        constexpr bool LOAD = decltype(load)::value;
        if constexpr (LOAD) asm volatile("" : "+v"(x_from), "+v"(w_from));   // (opaque: nothing kept)
#pragma unroll
        for (int i = 0; i < RB * NB; ++i) {
            acc[i / NB][i % NB] = mfma16(o.x[i % NB], o.w[i / NB], acc[i / NB][i % NB]);
            if (i % 2 == 1 && i / 2 < NB + RB) read_one(fill, from, h, i / 2);
            if (LOAD && i % 4 == 2) load_one(to, k, i / 4);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    static_assert(RB * NB / 2 >= NB + RB && RB * NB / 4 == kLoads, "a place for every read and load");

    // Tiles without a position inside a length have no products: they are written here.
    const auto empty = [&](const Tile &t) {
        const int n = t.n0 + wave % 4 * 64 + lane, b = min(n, a.N - 1) / a.L;
        T *y = a.y.row(b, t.e0) + (n - b * a.L);
#pragma unroll 1
        for (int c = wave / 4; c < min(TE, a.E_ - t.e0); c += 2)
            if (n < a.N) y[c * a.y.channel] = 0;
    };
    int number = blockIdx.x;
    const auto following = [&](Tile &t) {   // the next tile with products
        for (; number < tiles; number += gridDim.x) {
            t = tile_of(number);
            if (t.any) {
                number += gridDim.x;
                return true;
            }
            empty(t);
        }
        return false;
    };

    Tile now;
    if (!following(now)) return;
    aim(now);
    stage_scales(0, now);
    stage(0, 0);
    stage(1, 1);
    wait_loads<kLoads>();
    gi::lds_barrier();
    Operands first, second;
    int at = 0, set = 0;
    bool whole_stores = false;   // whether the tile before has left in exactly kStores stores
    for (bool more = true; more;) {
        Tile next{0, 0, false};
        more = following(next);
        next.any = more;
#pragma unroll
        for (int i = 0; i < NB + RB; ++i) read_one(first, at, 0, i);
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int n = 0; n < NB; ++n) acc[r][n] = v4i{0, 0, 0, 0};
#pragma clang loop unroll(disable)
        for (int k = 0; k < steps; ++k, at ^= 1) {
            multiply(first, second, at, 1, std::false_type{}, 0, 0);
            // The following step is there, and everyone has read this one.  Before a tile's
            // second step the stores of the tile before may still be on their way.
            if (k == 0 && whole_stores)
                wait_loads<kStores>();
            else
                wait_loads<0>();
            gi::lds_barrier();
            if (k == steps - 2) {
                if (more) stage_scales(set ^ 1, next);
                aim(next);   // (after the last tile: at nothing)
            }
            multiply(second, first, at ^ 1, 0, std::true_type{}, at, k + 2 < steps ? k + 2 : k + 2 - steps);
        }
        const float *sx = reinterpret_cast<const float *>(smem + kStreamScales + set * 4096);
        const float *const sw = sx + 256 + we * 128;
        const bool far = __any(is_far(sx[wm * 64 + lane]) | is_far(sw[lane]) | is_far(sw[64 + lane]));
        whole_stores = leave<E, NB, RB, SWAPPED>(
            a, now.n0 + wm * 64, now.e0 + we * 128, smem + kStreamTurn + wave * 2048, far,
            [&](int k) { return sx[wm * 64 + k]; }, [&](int c) { return sw[c]; },
            [&](int i) { return sx[512 + (SWAPPED ? wm * 64 : we * 128) + i]; },
            [&](int r, int k) { return acc[r][k / 4][k % 4]; });
        now = next;
        set ^= 1;
    }
}

template <class E>
Project<E> project_of(const project_int8_args &a) {
    return {static_cast<const uint8_t *>(a.codes), static_cast<const uint8_t *>(a.w), a.scales,
            a.w_scales, a.bias, view<E>(a.y), a.lengths, (int)((int64_t)a.B * a.L), a.E, a.L, a.K, 0, 0};
}

template <class E, int WM, int WE, int NB, int RB, int ST, bool SWAPPED>
hipError_t product(Project<E> k, hipStream_t s) {
    constexpr int TM = 16 * WM * NB, TE = 16 * WE * RB;
    k.n_tiles = (k.N + TM - 1) / TM, k.e_tiles = (k.E_ + TE - 1) / TE;
    constexpr int bytes = ST * (TM + TE) * kStep;
    if (bytes > 64 * 1024) {
        hipError_t e = hipFuncSetAttribute((const void *)project<E, WM, WE, NB, RB, ST, SWAPPED>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    project<E, WM, WE, NB, RB, ST, SWAPPED>
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
// every S-th; their sums meet in LDS.  Each wave brings its steps by direct loads to a place of
// its own, without a barrier: lanes 8 to a row, because loads straight into operands (each lane
// another row) reach 9.4 TB/s from the caches where these reach 28.  The next step is on its way
// while this one's products run; one more ahead was slower ([32, 4096] x 8192 9.1 us for 8.0,
// [8, 2048] x 4096 3.33 for 3.30): fewer work-groups share a compute unit.
// Rows are swizzled as in `project`.  Bound by memory where the weights are many ([64, 4096] x 8192
// bf16 8.3 us and 4.2 TB/s with weights in the memory-side cache, 12.2 from memory), else by the chain
// of launch, one round trip to memory, one through LDS and the sums' meeting ([8, 2048] x 4096
// 3.4 and 4.6 us).
//
// What the results are laid out along decides which operand is the first: a lane has four
// consecutive rows of it.  Along channels (one position a row), the weights.  Along
// positions, the positions, in the order that gives a lane 4 NB consecutive ones.  With
// codes inside (at most 16 positions, along channels) they are made here, from x, by every
// work-group for itself, and wait in LDS, unit u of row r at u ^ r in each 256 bytes; the
// operand's rows without a position are the last one again.
enum Form { kAlongChannels, kCodesInside, kAlongPositions };

template <class E>
struct Split {
    Project<E> p;
    View<E> x;   // [N, D]
    int D, share;
};

// (128 registers, for two work-groups a compute unit)
template <class E, int RB, int NB, int S, int FORM>
__global__ __launch_bounds__(64 * S, 4) void project_split(Split<E> t) {
    constexpr bool CODES = FORM == kCodesInside;
    static_assert(!CODES || NB == 1, "the codes of 16 rows");
    static_assert(NB <= 4 && RB <= 4, "the scales of a kind in a wave's lanes");
    constexpr int ROWS = 16 * (RB + (CODES ? 0 : NB)), kLoads = ROWS / 8;
    const Project<E> &a = t.p;
    extern __shared__ uint8_t smem[];
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    constexpr int kPlace = ROWS * kStep, kMeet = RB * NB * 1024;   // bytes of a wave
    uint8_t *const here = smem + wave * kPlace;
    v4i *const meet = reinterpret_cast<v4i *>(smem);   // after the steps
    float *const own_scales = reinterpret_cast<float *>(smem + S * std::max(kPlace, kMeet));
    uint8_t *const own = reinterpret_cast<uint8_t *>(own_scales + 64);   // [N][pitch]
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
        const int r = p * 8 + lane / 8;
        const int unit = lane % 8 ^ (FORM == kAlongPositions && r >= 16 * RB
                                         ? position_turn<NB>(r - 16 * RB) : r / 2 % 8);
        const int held = r < 16 * RB ? min(r, a.E_ - e0 - 1) : min(r - 16 * RB, a.N - n0 - 1);
        from[p] = held * a.K + unit * 16;
    }
    const auto bring = [&](int j) {
#pragma unroll
        for (int p = 0; p < kLoads; ++p)
            load_lds(p < 2 * RB ? wr : xr, here + p * 1024, from[p], place(j) * kStep);
    };
    // One of the work-group's scales of each kind, to see whether any is far (asked for behind the first
    // step they would hold it up: [1, 4096] x 4096 0.2 us more).
    const float seen_w = a.w_scales[min(e0 + lane % (16 * RB), a.E_ - 1)];
    const float seen_x = CODES ? 0.f : a.scales[min(n0 + lane % (16 * NB), a.N - 1)];
    if (mine > 0) bring(0);

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
    const int held = min(row, a.N - 1);
    const uint8_t *const own_at = own + held * pitch;
    for (int j = 0; j < mine; ++j) {
        wait_loads<0>();
        v4i fw[RB][2], fx[NB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int u = h * 4 + part;
#pragma unroll
            for (int r = 0; r < RB; ++r)
                fw[r][h] = *reinterpret_cast<const v4i *>(here + (r * 16 + row) * kStep +
                                                          (u ^ (row / 2 % 8)) * 16);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int xn = x_row + n * (FORM == kAlongPositions ? 4 : 16);
                const int turned = u ^ (FORM == kAlongPositions ? position_turn<NB>(xn) : xn / 2 % 8);
                fx[n][h] = *reinterpret_cast<const v4i *>(
                    CODES ? own_at + ((place(j) * 8 + u) ^ held) * 16
                          : here + (RB * 16 + xn) * kStep + turned * 16);
            }
        }
        if (j + 1 < mine) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // this one is read
            bring(j + 1);
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
    const bool far = __any(is_far(seen_w) | is_far(CODES ? own_scales[min(lane % 16, a.N - 1)] : seen_x));
    if constexpr (FORM == kAlongPositions) {
        for (int r = wave; r < RB; r += S) {
            const int e = e0 + r * 16 + row, n = n0 + part * 4 * NB;
            if (e >= a.E_ || n >= a.N) continue;
            float v[4 * NB], sx[4 * NB];
            const float sw = a.w_scales[e], bias = a.bias ? a.bias[e] : 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const v4i sum = sum_of(r * NB + i);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int one = sum[k];
                    sx[4 * i + k] = a.scales[min(n + 4 * i + k, a.N - 1)];
                    v[4 * i + k] = (float)one;
                }
            }
            if (__builtin_expect(far, 0)) {
#pragma unroll
                for (int k = 0; k < 4 * NB; ++k) v[k] = far_scaled(v[k], sx[k], sw, bias);
            } else {
#pragma unroll
                for (int k = 0; k < 4 * NB; ++k) v[k] = scaled(v[k], sx[k], sw, bias);
            }
            keep_apart(v);
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
            float v[4], sw[4], bias[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int ek = min(e + k, a.E_ - 1);
                sw[k] = a.w_scales[ek];
                bias[k] = a.bias ? a.bias[ek] : 0.f;
            }
            if (__builtin_expect(far, 0)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = far_scaled((float)sum[k], sx, sw[k], bias[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = scaled((float)sum[k], sx, sw[k], bias[k]);
            }
            keep_apart(v);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = in ? v[k] : 0.f;
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

template <class E, int RB, int NB, int S, int FORM>
hipError_t split(const project_int8_args &a, const seq_tensor &x, int D, hipStream_t s) {
    constexpr bool CODES = FORM == kCodesInside;
    Split<E> k{project_of<E>(a), view<E>(x), D, 64 * S / 16};
    k.p.n_tiles = (k.p.N + 16 * NB - 1) / (16 * NB), k.p.e_tiles = (a.E + 16 * RB - 1) / (16 * RB);
    if constexpr (CODES)
        while (k.share < 64 * S && 64 * S / k.share / 2 >= k.p.N) k.share *= 2;
    constexpr int kPlace = 16 * (RB + (CODES ? 0 : NB)) * kStep, kMeet = RB * NB * 1024;
    const int bytes = S * std::max(kPlace, kMeet) + 256 + (CODES ? k.p.N * ((a.K + 255) / 256 * 256) : 0);
    if (bytes > 64 * 1024) {
        hipError_t e = hipFuncSetAttribute((const void *)project_split<E, RB, NB, S, FORM>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    project_split<E, RB, NB, S, FORM>
        <<<(unsigned)((int64_t)k.p.n_tiles * k.p.e_tiles), 64 * S, bytes, s>>>(k);
    return hipGetLastError();
}

template <class E, bool SWAPPED>
hipError_t stream(Project<E> k, hipStream_t s) {
    k.n_tiles = (k.N + kStreamTile - 1) / kStreamTile, k.e_tiles = (k.E_ + kStreamTile - 1) / kStreamTile;
    hipError_t e = hipFuncSetAttribute((const void *)project_stream<E, SWAPPED>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes);
    if (e != hipSuccess) return e;
    const int64_t tiles = (int64_t)k.n_tiles * k.e_tiles;
    project_stream<E, SWAPPED>
        <<<(unsigned)std::min<int64_t>(tiles, 256), 64 * kStreamWaves, kStreamBytes, s>>>(k);
    return hipGetLastError();
}

// Blocks of channels RB and positions NB of a work-group: the fewest whose work-groups have a
// compute unit each, or else more of them, which read less.  Measured (us; RB NB of 1 1, 2 1 /
// 1 2, 2 2, 2 4): [8, 2048] x 4096 3.3 3.5, [16, 8192] x 8192 12.9 12.1 / [32, 4096] x 4096 5.0
// 5.5 6.7, [32, 4096] x 8192 8.0 7.2 8.1, [64, 4096] x 2048 5.0 5.6 6.9, [64, 1024] x 4096 3.8
// 3.6 3.9, [64, 4096] x 8192 12.1 11.9 8.5.
template <class E, int FORM>
hipError_t split_any(const project_int8_args &a, hipStream_t s) {
    const int64_t N = (int64_t)a.B * a.L;
    const auto fits = [&](int64_t RB, int64_t NB) {
        return (a.E + 16 * RB - 1) / (16 * RB) * ((N + 16 * NB - 1) / (16 * NB)) <= 256;
    };
    if (N <= 16)
        return fits(1, 1) ? split<E, 1, 1, 8, FORM>(a, {}, 0, s) : split<E, 2, 1, 8, FORM>(a, {}, 0, s);
    if (fits(1, 2)) return split<E, 1, 2, 8, FORM>(a, {}, 0, s);
    if (N <= 32 || fits(2, 2)) return split<E, 2, 2, 8, FORM>(a, {}, 0, s);
    return split<E, 2, 4, 8, FORM>(a, {}, 0, s);
}

// Larger tiles read less, smaller ones leave fewer compute units without one.  Tiles of 256 where
// at least two thirds of the units' turns have one; measured (us, tiles of 256 / 128, N x E from
// K): 3300 x 4096 from 2048 (208 of 256 turns) 30 / 36, 2500 x 4096 from 1024 (160) 19.8 / 20.2,
// 4400 x 4096 from 2048 (288 of 512) 48 / 45, 9000 x 4096 from 2048 (576 of 768) 71 / 75, 8192 x
// 8192 from 4096 207 / 262.  Tiles of 128 from 208 on, four fifths of a turn (tiles of 128 / 64):
// 192 tiles 11.0 / 9.2, 208 9.7 / 9.9, 256 8.8 / 11.9, 512 14.5 / 19.8.
template <class E, bool SWAPPED>
hipError_t tiles_any(const Project<E> &k, hipStream_t s) {
    const auto tiles = [&](int64_t t) { return (k.N + t - 1) / t * ((k.E_ + t - 1) / t); };
    const int64_t large = tiles(256), places = (large + 255) / 256 * 256;
    if (large * 3 >= places * 2 && k.K >= 2 * kStep) return stream<E, SWAPPED>(k, s);
    if (tiles(128) >= 208) return product<E, 2, 4, 4, 2, 2, SWAPPED>(k, s);
    return product<E, 2, 2, 2, 2, 3, SWAPPED>(k, s);
}

// k is shared out where tiles of whole rows would leave half of the chip without one, and for up
// to 32 positions, half a tile (us, shared / tiles of 64): 500 x 1024 from 1024 (128 tiles) 4.8 /
// 5.4, 200 x 2048 from 2048 (128) 6.6 / 7.2, 120 x 4096 from 4096 (128) 9.3 / 11.2, 700 x 1500
// from 300 (264) 8.4 / 5.3, 300 x 4096 from 4096 (320) 22 / 13.6, 64 x 16384 from 4096 (256) 17.6
// / 16.2; 17 x 65536 from 4096 50 / 63.
template <class E>
hipError_t product_any(const project_int8_args &a, hipStream_t s) {
    Project<E> k = project_of<E>(a);
    if (k.N <= 32 || (int64_t)((k.N + 63) / 64) * ((a.E + 63) / 64) <= 128)
        return a.L == 1 ? split_any<E, kAlongChannels>(a, s) : split_any<E, kAlongPositions>(a, s);
    if (a.L > 1 || a.lengths || a.y.channel != 1) return tiles_any<E, false>(k, s);
    // One position a row, results along the channels: they are the positions of one batch item.
    std::swap(k.codes, k.w);
    std::swap(k.scales, k.w_scales);
    std::swap(k.N, k.E_);
    k.L = k.N;
    k.y.channel = k.y.batch;
    k.y.batch = 0;
    return tiles_any<E, true>(k, s);
}

int64_t code_row(int64_t D) { return (D + SEQ_INT8_ROW - 1) / SEQ_INT8_ROW * SEQ_INT8_ROW; }

// Whether every work-group makes the codes of a single-position call for itself: one block of
// positions, few numbers for each thread, and not too many work-groups to do that again and again.  A
// row has 512 / P threads, P the rows rounded up to a power of two, which keep 64 numbers each in
// registers; float32 numbers take twice the instructions.  What it saves is the codes' own kernel
// (longer for long rows, whatever their number) and the host's time for a second launch: eager calls
// take 5.3 us of the host with the codes made inside and 9.2 without.  So the border is where
// the product with the codes inside takes longer than those 9.2 too.  Measured (us, made inside / by
// a kernel before it, both in graphs, the weights from memory; | the border):
// bf16 x 4096: [1, 8192] 9.3 / 11.5, [1, 32768] 29.3 / 38.5, [3, 10900] 15.7 / 16.6, [8, 2048] 6.3 /
// 6.5, [8, 4096] 8.2 / 8.2, [9, 2048] 6.8 / 6.5, [16, 2048] 7.0 / 6.5 | [5, 5400] 11.5 / 10.5, [5,
// 6500] 12.5 / 10.5, [9, 2700] 9.4 / 7.7, [9, 3640] 11.9 / 8.3;
// f32 x 4096: [1, 32768] 33.1 / 44.9, [2, 16384] 22.8 / 26.2, [4, 4096] 9.0 / 8.7, [8, 2048] 7.9 / 6.9,
// [16, 1024] 7.1 / 5.8 | [4, 8192] 14.2 / 13.5, [5, 4096] 11.5 / 8.8, [9, 2048] 10.5 / 7.0, [16, 2048]
// 11.0 / 7.0;
// bf16 x 16384 | x 24576, x 32768, x 49152: [1, 1024] 7.2 / 7.7 | 9.7 / 8.7, 11.7 / 11.1, 17.9 / 14.7,
// [4, 4096] 15.4 / 18.0 | 23.6 / 21.3, 27.8 / 29.0, 39.5 / 39.6, [8, 2048] 9.0 / 10.2 | 16.4 / 14.9, 18.4 /
// 18.6, 25.4 / 22.0, [16, 1024] 7.9 / 7.8 | 11.0 / 9.1, 13.4 / 11.1, 20.2 / 15.1.
bool codes_inside(int32_t dtype, int64_t B, int64_t D, int64_t E) {
    if (B > 16 || B * D > 32768) return false;
    int64_t P = 1;
    while (P < B) P *= 2;
    const bool few = dtype == SEQ_F32 ? P <= 2 || P * D <= 16384 : P <= 4 || P * D <= 32768;
    return few && E <= 16384;
}

template <class E>
hipError_t step(const project_int8_step_args &a, hipStream_t s) {
    project_int8_args p = {};
    p.dtype = a.dtype, p.B = a.B, p.E = a.E, p.L = 1, p.K = a.K;
    p.w = a.w, p.w_scales = a.w_scales, p.bias = a.bias, p.y = a.y;
    if (codes_inside(a.dtype, a.B, a.D, a.E))
        return a.E > 4096 ? split<E, 2, 1, 8, kCodesInside>(p, a.x, a.D, s)
                          : split<E, 1, 1, 8, kCodesInside>(p, a.x, a.D, s);
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

int64_t project_step_workspace(int32_t dtype, int B, int D, int E) {
    return codes_inside(dtype, B, D, E) ? 0 : B * (code_row(D) + (int64_t)sizeof(float));
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
