// seq_common.h -- element types, vector memory access and lane operations
// shared by the sequence kernels (causal_conv, state_scan, block_norm).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

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

// Positions t .. t+V-1 of a row; those outside [0, end) are 0 and not read.
template <class E, int V>
__device__ __forceinline__ void load_row(const typename E::type *row, int64_t t, int64_t end,
                                         float (&out)[V]) {
    if (t >= 0 && t + V <= end) {
        load_vec<E, V>(row + t, out);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            out[i] = 0.f;
            if (t + i >= 0 && t + i < end) out[i] = E::up(row[t + i]);
        }
    }
}

// Writes positions t .. t+V-1 of a row of L positions (t >= 0).
template <class E, int V>
__device__ __forceinline__ void store_row(typename E::type *row, int64_t t, int64_t L,
                                          const float (&v)[V]) {
    if (t + V <= L) {
        store_vec<E, V>(row + t, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (t + i < L) row[t + i] = E::down(v[i]);
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

// log(1 + e^v).  For the logarithm of 1 + e the rounded sum w = 1 + e stands in
// for it with the factor e / (w - 1), which takes the rounding of w back out:
// log(1 + e) = log(w) * e / (w - 1) up to a relative 2^-23 or so, for any e.
__device__ __forceinline__ float softplus(float v) {
    const float e = exp2_fast(-__builtin_fabsf(v) * kLog2e);
    const float w = 1.f + e;
    const float d = w - 1.f;
    const float l = __builtin_amdgcn_logf(w) * kLn2;
    const float r = d == 0.f ? e : l * (e * __builtin_amdgcn_rcpf(d));
    return __builtin_fmaxf(v, 0.f) + r;
}

// Lane moves inside rows of 16 lanes (DPP): lanes without a source get `old`.
template <int CTRL>
__device__ __forceinline__ float dpp(float old, float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        __builtin_bit_cast(int, old), __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// The same with 0 in lanes without a source (folds into the consuming instruction).
template <int CTRL>
__device__ __forceinline__ float dpp0(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
constexpr int kRowShl = 0x100, kRowShr = 0x110, kRowRor = 0x120;  // + distance 1..15

// v of lane ^ M.
__device__ __forceinline__ float lane_xor(float v, int m) { return __shfl_xor(v, m, 64); }

}  // namespace seq
