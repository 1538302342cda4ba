// Row-vector access shared by the convolution, selective-scan and
// normalisation kernels: up to V consecutive elements of one row as floats,
// from addresses aligned only to the element. Rows may start anywhere (odd
// widths, slices of a wider projection), and gfx950 loads and stores 16 bytes
// at any byte address, so a full vector is one instruction whatever the row's
// alignment and only a row's ragged last vector goes element by element.
#pragma once

#include <type_traits>

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
    // 0 in its place unless `keep`
    __device__ __forceinline__ void clear(int e, bool keep) {
        w[e >> 1] = keep ? w[e >> 1] : w[e >> 1] & ((e & 1) ? 0x0000ffffu : 0xffff0000u);
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
    __device__ __forceinline__ void clear(int e, bool keep) { w[e] = keep ? w[e] : 0.0f; }
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

// ---- rows held by groups of lanes (the normalisations) ---------------------------

// Lanes that share a row, as the kernels see it: `lpr` <= 64 lanes of one
// wavefront (a power of two), or the workgroup (lpr = 0).
struct RowGroup {
    int lpr, lane, group, groups;
};
__device__ __forceinline__ RowGroup row_group(int lpr) {
    RowGroup r;
    r.lpr = lpr;
    if (lpr) {
        r.lane = threadIdx.x & (lpr - 1);
        r.group = threadIdx.x / lpr;
        r.groups = blockDim.x / lpr;
    } else {
        r.lane = threadIdx.x;
        r.group = 0;
        r.groups = 1;
    }
    return r;
}

// Sums over groups of `top` lanes (a power of two), in every one of them: moves
// within the vector unit, which a row's sums, one after the other, wait for far
// less than for the permutes through LDS that __shfl_xor makes.
template <int K> __device__ __forceinline__ void lane_sum(float (&v)[K], int top) {
    auto dpp = [&](auto ctrl) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[k]),
                                                               decltype(ctrl)::value, 0xf, 0xf, true));
    };
    if (top > 1) dpp(std::integral_constant<int, 0xB1>());    // the other of two
    if (top > 2) dpp(std::integral_constant<int, 0x4E>());    // the other two of four
    if (top > 4) dpp(std::integral_constant<int, 0x141>());   // eight, mirrored
    if (top > 8) dpp(std::integral_constant<int, 0x140>());   // sixteen, mirrored
    if (top > 16)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]),
                                                            __float_as_uint(v[k]), false, false);
            v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        }
    if (top > 32)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]),
                                                            __float_as_uint(v[k]), false, false);
            v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        }
}

// Sums of K values over the lanes of a row, in every one of them. `buf` holds
// K floats per wavefront (at most 16 wavefronts); the caller alternates between
// two of them, so that one barrier per sum is enough (a wavefront can write a
// buffer again only after it has passed the barrier of the other one).
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int lpr, float *buf) {
    lane_sum(v, lpr ? lpr : 64);
    const int waves = blockDim.x >> 6;
    if (lpr || waves == 1) return;
    if (lane_id() == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[wave_id() * K + k] = v[k];
    __syncthreads();
    const int w = lane_id() & 15;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = w < waves ? buf[w * K + k] : 0.0f;
    lane_sum(v, 16);
}

constexpr int kShortWaves = 4;  // wavefronts of a workgroup that takes several rows at once

template <typename T> constexpr int vec_of() { return sizeof(T) == 2 ? 8 : 4; }

struct NormShape {
    int lpr, threads, nv, groups;
};
// One vector per lane where the row allows it: more lanes per row keep more
// loads in flight than more vectors per lane do. `most`: lanes of a workgroup
// that a row may take.
inline NormShape norm_shape(int D, int V, int most) {
    const int nvec = (D + V - 1) / V;
    NormShape s;
    if (nvec <= 64) {
        s.lpr = 1;
        while (s.lpr < nvec) s.lpr <<= 1;
        s.threads = 64 * kShortWaves;
        s.nv = 1;
        s.groups = s.threads / s.lpr;
        return s;
    }
    s.lpr = 0;
    s.groups = 1;
    s.nv = 1;
    while ((nvec + s.nv - 1) / s.nv > most) s.nv *= 2;
    s.threads = ((nvec + s.nv - 1) / s.nv + 63) / 64 * 64;
    return s;
}

}  // namespace ssd
