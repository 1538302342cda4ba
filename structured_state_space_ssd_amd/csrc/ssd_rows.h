// Row-vector access shared by the convolution, selective-scan and
// normalisation kernels: up to V consecutive elements of one row as floats,
// from addresses aligned only to the element. Rows may start anywhere (odd
// widths, slices of a wider projection), and gfx950 loads and stores 16 bytes
// at any byte address, so a full vector is one instruction whatever the row's
// alignment and only a row's ragged last vector goes element by element.
#pragma once

#include "ssd_common.h"

namespace ssd {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2_any __attribute__((ext_vector_type(2), aligned(4)));

// A ragged vector's element count (or a lane's number) as a value the compiler
// cannot know ahead: comparisons with it are then made where they are needed
// instead of being kept, one lane mask each, across the whole loop.
__device__ __forceinline__ int ragged(int n) {
    asm volatile("" : "+v"(n));
    return n;
}

// V consecutive elements as loaded, still packed.
template <typename T, int V> struct RowRaw;

template <> struct RowRaw<bf16_t, 8> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const bf16_t *p) {
        const u32x4_any u = *reinterpret_cast<const u32x4_any *>(p);
        w[0] = u[0]; w[1] = u[1]; w[2] = u[2]; w[3] = u[3];
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ void load(const bf16_t *p, int n) {
        if (n >= 8) return load(p);
        zero();
        n = ragged(n);
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) w[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
    }
    __device__ __forceinline__ float get(int e) const {
        const uint32_t v = w[e >> 1];
        return __uint_as_float((e & 1) ? (v & 0xffff0000u) : (v << 16));
    }
};
template <> struct RowRaw<bf16_t, 4> {
    uint32_t w[2];
    __device__ __forceinline__ void load(const bf16_t *p) {
        const u32x2_any u = *reinterpret_cast<const u32x2_any *>(p);
        w[0] = u[0]; w[1] = u[1];
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = 0; }
    __device__ __forceinline__ void load(const bf16_t *p, int n) {
        if (n >= 4) return load(p);
        zero();
        n = ragged(n);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) w[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
    }
    __device__ __forceinline__ float get(int e) const {
        const uint32_t v = w[e >> 1];
        return __uint_as_float((e & 1) ? (v & 0xffff0000u) : (v << 16));
    }
};
template <int V> struct RowRaw<float, V> {
    static_assert(V % 4 == 0, "whole 16-byte loads");
    float w[V];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4_any u = *reinterpret_cast<const f32x4_any *>(p + i);
            w[i] = u[0]; w[i + 1] = u[1]; w[i + 2] = u[2]; w[i + 3] = u[3];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = 0.0f;
    }
    __device__ __forceinline__ void load(const float *p, int n) {
        if (n >= V) return load(p);
        zero();
        n = ragged(n);
#pragma unroll
        for (int e = 0; e < V - 1; ++e)
            if (e < n) w[e] = p[e];
    }
    __device__ __forceinline__ float get(int e) const { return w[e]; }
};

// Two values rounded to bf16 (nearest even, one instruction), the first one low.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2));
}

// The first n of V values, rounded to nearest even where T is bf16.
template <int V> __device__ __forceinline__ void row_store(float *p, const float (&v)[V], int n) {
    if (n >= V) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<f32x4_any *>(p + i) = f32x4_any{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
        n = ragged(n);
#pragma unroll
        for (int e = 0; e < V - 1; ++e)
            if (e < n) p[e] = v[e];
    }
}
template <int V> __device__ __forceinline__ void row_store(bf16_t *p, const float (&v)[V], int n) {
    static_assert(V == 4 || V == 8, "8 or 16 bytes");
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (n >= V) {
        if constexpr (V == 8)
            *reinterpret_cast<u32x4_any *>(p) = u32x4_any{w[0], w[1], w[2], w[3]};
        else
            *reinterpret_cast<u32x2_any *>(p) = u32x2_any{w[0], w[1]};
    } else {
        n = ragged(n);
#pragma unroll
        for (int e = 0; e < V - 1; ++e)
            if (e < n) p[e] = static_cast<bf16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
}

// 1 / (1 + e^-v): one exponential and one reciprocal, each within 1 ulp. At
// the ends e^-v is infinity or 0 and the quotient 0 or 1.
__device__ __forceinline__ float sigmoid_f32(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
}
// v sigmoid(v), and its derivative p (1 + v (1 - p)) with p = sigmoid(v).
// v = -inf gives 0 * -inf: NaN, as the product of the two factors does.
__device__ __forceinline__ float silu_f32(float v) { return v * sigmoid_f32(v); }
__device__ __forceinline__ float silu_grad_f32(float v) {
    const float p = sigmoid_f32(v);
    return p * (1.0f + v * (1.0f - p));
}

// log(1 + e^v) = max(v, 0) + log(1 + t) with t = e^-|v| in (0, 1]. 1 + t is
// rounded to u; log(u) + (t - (u - 1)) / u puts back what the rounding lost,
// so the result keeps its relative accuracy where t is tiny (the step sizes'
// usual range).
__device__ __forceinline__ float softplus_f32(float v) {
    const float t = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
    const float u = 1.0f + t;
    const float c = t - (u - 1.0f);
    const float l = __builtin_amdgcn_logf(u) * 0.6931471805599453f;
    // the larger of v and 0: one instruction where fmaxf first quiets its operands
    return __builtin_amdgcn_fmed3f(v, 0.0f, __builtin_inff()) + fmaf(c, __builtin_amdgcn_rcpf(u), l);
}

}  // namespace ssd
