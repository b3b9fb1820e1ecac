// seq_common.h -- element types, vector memory access and lane operations
// shared by the sequence kernels (causal_conv, state_scan, block_norm).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sequence_ops.h"

namespace seq {

// Element types: storage, widening (exact) and rounding (to nearest even).
struct F32 {
    using type = float;
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
struct BF16 {
    using type = uint16_t;
    static __device__ __forceinline__ float up(uint16_t v) {
        return __builtin_bit_cast(float, (uint32_t)v << 16);
    }
    static __device__ __forceinline__ uint16_t down(float v) {
        const __bf16 h = (__bf16)v;
        return __builtin_bit_cast(uint16_t, h);
    }
};
struct F16 {
    using type = uint16_t;
    static __device__ __forceinline__ float up(uint16_t v) {
        return (float)__builtin_bit_cast(_Float16, v);
    }
    static __device__ __forceinline__ uint16_t down(float v) {
        const _Float16 h = (_Float16)v;
        return __builtin_bit_cast(uint16_t, h);
    }
};

// V elements in one or more wide accesses.  Rows of any length and stride start
// at any multiple of the element size, so the accesses claim no more alignment
// than that (gfx950 serves unaligned wide global accesses).
template <class T, int V>
struct Vec {
    typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};

template <class E, int V>
__device__ __forceinline__ void load_vec(const typename E::type *p, float (&out)[V]) {
    using T = typename E::type;
    constexpr int W = 16 / (int)sizeof(T) < V ? 16 / (int)sizeof(T) : V;
    using U = typename Vec<T, W>::type;
#pragma unroll
    for (int j = 0; j < V; j += W) {
        const U u = *reinterpret_cast<const U *>(p + j);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const T e = u[i];
            out[j + i] = E::up(e);
        }
    }
}

template <class E, int V>
__device__ __forceinline__ void store_vec(typename E::type *p, const float (&in)[V]) {
    using T = typename E::type;
    constexpr int W = 16 / (int)sizeof(T) < V ? 16 / (int)sizeof(T) : V;
    using U = typename Vec<T, W>::type;
#pragma unroll
    for (int j = 0; j < V; j += W) {
        U u;
#pragma unroll
        for (int i = 0; i < W; ++i) u[i] = E::down(in[j + i]);
        *reinterpret_cast<U *>(p + j) = u;
    }
}

// The first `left` of V positions as they are stored, 0 for the others.  The reads
// go out one by one under their conditions; the empty statements keep what uses
// them from moving up there, where it would cost the end of a row V latencies.
template <class T, int V>
__device__ __forceinline__ void load_end(const T *p, int left, T (&out)[V]) {
    using Word = std::conditional_t<sizeof(T) == 4, T, uint32_t>;
    Word u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        u[i] = 0;
        if (i < left) u[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) asm volatile("" : "+v"(u[i]));
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = (T)u[i];
}

// Positions t .. t+V-1 of a row (t >= 0); those from `end` on are 0 and not read.
template <class E, int V>
__device__ __forceinline__ void load_row(const typename E::type *row, int t, int end,
                                         float (&out)[V]) {
    const int left = end - t;
    if (left >= V) {
        load_vec<E, V>(row + t, out);
    } else {
        typename E::type u[V];
        load_end(row + t, left, u);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = E::up(u[i]);
    }
}

// Eight positions as they are stored, for a load whose use comes later; those
// from the left-th on are 0 and not read.
template <class E>
struct Octet {
    typename Vec<typename E::type, 8>::type v;
    __device__ __forceinline__ void load(const typename E::type *p, int left) {
        if (left >= 8) {
            v = *reinterpret_cast<const typename Vec<typename E::type, 8>::type *>(p);
        } else {
            typename E::type u[8];
            load_end(p, left, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = u[i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const {
        const typename E::type e = v[i];
        return E::up(e);
    }
};

// Writes positions t .. t+V-1 of a row of L positions (t >= 0).
template <class E, int V>
__device__ __forceinline__ void store_row(typename E::type *row, int t, int L,
                                          const float (&v)[V]) {
    typename E::type *p = row + t;
    if (L - t >= V) {
        store_vec<E, V>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (L - t > i) p[i] = E::down(v[i]);
    }
}

// One activation on the device: rows of contiguous positions.
template <class E>
struct View {
    typename E::type *p;
    int64_t batch, channel;
    __device__ __forceinline__ typename E::type *row(int64_t b, int64_t c) const {
        return p + b * batch + c * channel;
    }
};

template <class E>
inline View<E> view(const seq_tensor &t) {
    return {static_cast<typename E::type *>(t.data), t.batch, t.channel};
}

__device__ __forceinline__ int length_of(const int32_t *lengths, int64_t b, int L) {
    if (!lengths) return L;
    const int n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// v_exp_f32, v_log_f32 and v_rcp_f32 are good to 1 ulp; results below the
// normal range become 0, which the sums they enter cannot tell from the truth.
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
}

// A log2(e) of a scan.  -inf becomes the lowest float, whose decay is 0 for any step
// above 1e-36 too: positions beyond a length have step 0, where exp(0 A) has to be 1.
__device__ __forceinline__ float decay_rate(float A) {
    const float v = A * kLog2e;
    return v < -3.4028234664e38f ? -3.4028234664e38f : v;
}

// log(1 + e^v) = max(v, 0) + log(1 + e) with e = exp(-|v|) in (0, 1].  The sum
// w = 1 + e loses c = e - (w - 1) <= 2^-24 of e, exactly known; log(1 + e) is
// log(w) + c / w to second order in c, and c stands for c / w: they differ by
// c e / w, at most 2^-25 of the result.  Where e is too small to change w the
// result is c = e.
__device__ __forceinline__ float softplus(float v) {
    const float e = exp2_fast(__builtin_fabsf(v) * -kLog2e);
    const float w = 1.f + e;
    const float c = e - (w - 1.f);
    return __builtin_fmaxf(v, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(w), kLn2, c);
}

// Lane moves (DPP), with 0 in lanes without a source (folds into the consuming instruction).
template <int CTRL>
__device__ __forceinline__ float dpp0(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
constexpr int kRowRor = 0x120;  // + distance 1..15, inside rows of 16 lanes
constexpr int kWaveShl = 0x130, kWaveShr = 0x138, kWaveRor = 0x13c;  // by a lane of the wave

// Maps h -> P h + Q compose along the lanes of a row of LANES (16 or 64): with Q
// in h, h[k] becomes the composition of lanes 0 .. l applied to 0, and turned[k]
// lane l-1's result, in lane 0 the last lane's.  NI independent chains.  A DPP
// operand must be two instructions older than its use, which the compiler does
// not see to inside an asm block: chains alternate, and one alone waits.
#define SEQ_STEP1(M) \
    "v_fmac_f32_dpp %0, %0, %1 " M "\n\tv_mul_f32_dpp %1, %1, %1 " M "\n\ts_nop 0\n\t"
#define SEQ_STEP2(M)                                                                  \
    "v_fmac_f32_dpp %0, %0, %2 " M "\n\tv_fmac_f32_dpp %1, %1, %3 " M "\n\t"          \
    "v_mul_f32_dpp %2, %2, %2 " M "\n\tv_mul_f32_dpp %3, %3, %3 " M "\n\t"
#define SEQ_ALL " row_mask:0xf bank_mask:0xf"
#define SEQ_ROW_STEPS(S, DIR) \
    S("row_" DIR ":1" SEQ_ALL) S("row_" DIR ":2" SEQ_ALL) S("row_" DIR ":4" SEQ_ALL)

template <int LANES>
__device__ __forceinline__ void scan_chain(float &h, float &P, float &turned) {
    if constexpr (LANES == 16) {
        asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP1, "shr")
            "v_fmac_f32_dpp %0, %0, %1 row_shr:8" SEQ_ALL "\n\ts_nop 1\n\t"
            "v_mov_b32_dpp %2, %0 row_ror:1" SEQ_ALL
            : "+v"(h), "+v"(P), "=&v"(turned));
    } else {
        asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP1, "shr") SEQ_STEP1("row_shr:8" SEQ_ALL)
            SEQ_STEP1("row_bcast:15 row_mask:0xa bank_mask:0xf")
            "v_fmac_f32_dpp %0, %0, %1 row_bcast:31 row_mask:0xc bank_mask:0xf\n\ts_nop 1\n\t"
            "v_mov_b32_dpp %2, %0 wave_ror:1" SEQ_ALL
            : "+v"(h), "+v"(P), "=&v"(turned));
    }
}

template <int LANES>
__device__ __forceinline__ void scan_chains(float &h0, float &h1, float &P0, float &P1,
                                            float &turned0, float &turned1) {
    if constexpr (LANES == 16) {
        asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP2, "shr")
            "v_fmac_f32_dpp %0, %0, %2 row_shr:8" SEQ_ALL "\n\t"
            "v_fmac_f32_dpp %1, %1, %3 row_shr:8" SEQ_ALL "\n\ts_nop 0\n\t"
            "v_mov_b32_dpp %4, %0 row_ror:1" SEQ_ALL "\n\t"
            "v_mov_b32_dpp %5, %1 row_ror:1" SEQ_ALL
            : "+v"(h0), "+v"(h1), "+v"(P0), "+v"(P1), "=&v"(turned0), "=&v"(turned1));
    } else {
        asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP2, "shr") SEQ_STEP2("row_shr:8" SEQ_ALL)
            SEQ_STEP2("row_bcast:15 row_mask:0xa bank_mask:0xf")
            "v_fmac_f32_dpp %0, %0, %2 row_bcast:31 row_mask:0xc bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %1, %1, %3 row_bcast:31 row_mask:0xc bank_mask:0xf\n\ts_nop 0\n\t"
            "v_mov_b32_dpp %4, %0 wave_ror:1" SEQ_ALL "\n\t"
            "v_mov_b32_dpp %5, %1 wave_ror:1" SEQ_ALL
            : "+v"(h0), "+v"(h1), "+v"(P0), "+v"(P1), "=&v"(turned0), "=&v"(turned1));
    }
}

// The same from the right over 16 lanes: h becomes the composition of lanes
// 15 .. l, turned lane l+1's result, in lane 15 lane 0's.
__device__ __forceinline__ void scan_chain_back(float &h, float &P, float &turned) {
    asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP1, "shl")
        "v_fmac_f32_dpp %0, %0, %1 row_shl:8" SEQ_ALL "\n\ts_nop 1\n\t"
        "v_mov_b32_dpp %2, %0 row_ror:15" SEQ_ALL
        : "+v"(h), "+v"(P), "=&v"(turned));
}
__device__ __forceinline__ void scan_chains_back(float &h0, float &h1, float &P0, float &P1,
                                                 float &turned0, float &turned1) {
    asm("s_nop 1\n\t" SEQ_ROW_STEPS(SEQ_STEP2, "shl")
        "v_fmac_f32_dpp %0, %0, %2 row_shl:8" SEQ_ALL "\n\t"
        "v_fmac_f32_dpp %1, %1, %3 row_shl:8" SEQ_ALL "\n\ts_nop 0\n\t"
        "v_mov_b32_dpp %4, %0 row_ror:15" SEQ_ALL "\n\t"
        "v_mov_b32_dpp %5, %1 row_ror:15" SEQ_ALL
        : "+v"(h0), "+v"(h1), "+v"(P0), "+v"(P1), "=&v"(turned0), "=&v"(turned1));
}
template <int NI>
__device__ __forceinline__ void scan_lanes_back(float (&h)[NI], float (&P)[NI],
                                                float (&turned)[NI]) {
    if constexpr (NI == 1) {
        scan_chain_back(h[0], P[0], turned[0]);
    } else {
#pragma unroll
        for (int k = 0; k < NI; k += 2)
            scan_chains_back(h[k], h[k + 1], P[k], P[k + 1], turned[k], turned[k + 1]);
    }
}

template <int LANES, int NI>
__device__ __forceinline__ void scan_lanes(float (&h)[NI], float (&P)[NI], float (&turned)[NI]) {
    if constexpr (NI == 1) {
        scan_chain<LANES>(h[0], P[0], turned[0]);
    } else {
#pragma unroll
        for (int k = 0; k < NI; k += 2)
            scan_chains<LANES>(h[k], h[k + 1], P[k], P[k + 1], turned[k], turned[k + 1]);
    }
}

// x summed over the half waves in lanes 0..31, y in lanes 32..63.
__device__ __forceinline__ float meet32(float x, float y) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x),
                                                    __builtin_bit_cast(unsigned, y), false, false);
    const unsigned p = r[0], q = r[1];
    return __builtin_bit_cast(float, p) + __builtin_bit_cast(float, q);
}
// x summed over the two rows of 16 lanes of each half in its first row, y in its second.
__device__ __forceinline__ float meet16(float x, float y) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x),
                                                    __builtin_bit_cast(unsigned, y), false, false);
    const unsigned p = r[0], q = r[1];
    return __builtin_bit_cast(float, p) + __builtin_bit_cast(float, q);
}

// F floats at an address that is a multiple of their size.
template <int F>
struct alignas(4 * F) Whole {
    float v[F];
};

// Sums over the four rows of 16 lanes: row k ends with those of values k T/4 ..
// (k+1) T/4 - 1 of each of its lanes.
template <int T>
__device__ __forceinline__ Whole<T / 4> meet_rows(const float (&v)[T]) {
    Whole<T / 4> sum;
#pragma unroll
    for (int i = 0; i < T / 4; ++i)
        sum.v[i] = meet16(meet32(v[i], v[T / 2 + i]), meet32(v[T / 4 + i], v[3 * T / 4 + i]));
    return sum;
}

// v of lane ^ M.
__device__ __forceinline__ float lane_xor(float v, int m) { return __shfl_xor(v, m, 64); }

// Octet o of a group of states goes where its lanes read it: [state][T/4][LANES][4].
template <class E, int LANES, int T>
__device__ __forceinline__ void stage_octet(float *to, int o, const Octet<E> &v) {
    constexpr int PER = LANES * T / 8;  // octets of a state
    const int n = o / PER, t = o % PER * 8;
    float4 *p = reinterpret_cast<float4 *>(to + n * (LANES * T));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lane = (t + 4 * h) / T, q = (t + 4 * h) % T / 4;
        p[q * LANES + lane] =
            float4{v.at(4 * h), v.at(4 * h + 1), v.at(4 * h + 2), v.at(4 * h + 3)};
    }
}

}  // namespace seq
