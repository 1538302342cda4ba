// Shared by the selective scan's forward, backward and single-token kernels.
#pragma once

#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

// How a workgroup holds channels and states (NK: the state size rounded up to
// 4, 8, 16, 32 or 64). A lane holds NS states of one channel; the WS wavefronts
// that share 64 channels hold different states. So the B and C of a token are
// the same for a whole wavefront and come from scalar loads, and sums over
// channels or states never mix the two axes. The backward (BACK) keeps a
// tile's states and decays in registers, so its lanes hold 4 states (8 at NK
// 64) and the workgroup has more wavefronts instead.
template <int NK, bool BACK = false> struct SelShape {
    static constexpr int NS = BACK ? (NK <= 32 ? 4 : 8) : NK <= 16 ? 4 : NK / 4;  // states per lane
    static constexpr int WS = NK / NS;                           // wavefronts across the states
    static constexpr int THREADS = WS > 4 ? 64 * WS : 256;
    static constexpr int CH = THREADS / WS;                      // channels per workgroup
    static constexpr int TILE = 2048 / CH;                       // tokens staged at a time
};
// Tokens between the states that the backward's first walk keeps: a tile of
// its second one, whose partial sums (12 bytes per channel, token and
// wavefront) stay within 48 KB of LDS and whose states within the registers.
template <int NK> constexpr int sel_keep() { return NK <= 8 ? 8 : NK == 16 ? 16 : NK == 32 ? 8 : 4; }

// B and C as the scans read them: float32 [Bt][G][tokens][NK / 4][B, C][4], the
// tokens rounded up to a whole number of tiles and zero behind the last. Four
// states' B and C are one 32-byte scalar load (SelBC: B in 0 .. 3, C in 4 .. 7).
constexpr int kSelPad = 32;
__host__ __device__ constexpr int sel_padded(int seqlen) { return (seqlen + kSelPad - 1) / kSelPad * kSelPad; }
typedef float SelBC __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(4))) SelBC sel_const;

// The step size of raw value v (bias included): softplus and clamp as chosen.
__device__ __forceinline__ float sel_step(const DtOpts &o, float v) {
    if (o.softplus) v = softplus_f32(v);
    if (o.clamp) v = clamp_step(o, v);
    return v;
}
// The same of a vector's values, the choices outside the loops; zero (which
// moves no state and passes no gradient) past the segment's last row.
template <int V>
__device__ __forceinline__ void sel_steps(const DtOpts &o, float (&d)[V], bool in) {
    if (o.softplus) {
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = softplus_f32(d[e]);
    }
    if (o.clamp) {
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = clamp_step(o, d[e]);
    }
    if (!in) {
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = 0.0f;
    }
}

// Where a workgroup of the scan stands: sequence b, segment seg, channels
// first .. first + n - 1, all of group g, its block-th workgroup.
struct SelBlock {
    int b, seg, g, block, first, n;
};
// (units: a sequence's workgroups, one sequence after the other)
template <int CH> __device__ __forceinline__ SelBlock sel_block(int unit, int seg, int channels, int ngroups) {
    const int each = channels / ngroups, per = (each + CH - 1) / CH;
    SelBlock k;
    const int cb = unit % (per * ngroups);
    k.seg = seg;
    k.b = unit / (per * ngroups);
    k.g = cb / per;
    k.block = cb % per;
    const int at = k.block * CH;
    k.first = k.g * each + at;
    k.n = each - at < CH ? each - at : CH;
    return k;
}

// A lane's NS states in scratch, [..][NK / 4][E][4] from its first four on, E
// channels: 16 bytes a lane and a kilobyte a wavefront at a time.
template <int NS> __device__ __forceinline__ void lane_load(const float *p, int E, float (&v)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(p + (size_t)i * E);
        v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
}
template <int NS> __device__ __forceinline__ void lane_store(float *p, int E, const float (&v)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; i += 4)
        *reinterpret_cast<float4 *>(p + (size_t)i * E) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

// Waits for the scalar loads and LDS reads under way (their counter to 0, the others
// at their most).
__device__ __forceinline__ void wait_lgkm() { __builtin_amdgcn_s_waitcnt(0xc07f); }

// A row vector's place within a tile, in bytes from the tile's first row: with
// the tile's address uniform it is the 32-bit offset of the load or store, and
// no lane computes an address (rows of a tile are at most 32, and token strides
// below 2^24 elements).
template <typename T>
__device__ __forceinline__ uint32_t row_offset(int r, size_t stride, int c) {
    return (static_cast<uint32_t>(r) * static_cast<uint32_t>(stride) + static_cast<uint32_t>(c)) *
           static_cast<uint32_t>(sizeof(T));
}
template <typename T> __device__ __forceinline__ const T *row_at(const T *tile, uint32_t off) {
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(tile) + off);
}
template <typename T> __device__ __forceinline__ T *row_at(T *tile, uint32_t off) {
    return reinterpret_cast<T *>(reinterpret_cast<char *>(tile) + off);
}

// The state that n spans of tokens leave one after another: h = state of span
// 0, then h = exp(sum of span s) h + state of span s. Span s lies s * step rows
// of [NK / 4][E][4] from `state` (this lane's place in row 0) and of [E] from
// `sum`; four spans are fetched at a time.
template <int NK, int NS>
__device__ __forceinline__ void sel_fold(const float *state, const float *sum, long long step, int E,
                                         int n, const float (&A2)[NS], float (&h)[NS]) {
    for (int s0 = 0; s0 < n; s0 += 4) {
        float v[4][NS], m[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long s = s0 + u < n ? s0 + u : n - 1;
            lane_load(state + s * step * E * NK, E, v[u]);
            m[u] = s ? sum[s * step * E] : 0.0f;  // the first one's decays nothing here
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (s0 + u < n)
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    h[i] = s0 + u == 0 ? v[u][i] : fmaf(__builtin_amdgcn_exp2f(A2[i] * m[u]), h[i], v[u][i]);
    }
}

// A decay rate times log2(e), so that a decay is one exp2. -inf becomes the lowest
// float: the same decay for any step size but zero, which it leaves at 1.
__device__ __forceinline__ float sel_rate(float a) {
    const float v = a * kLog2e;
    return v < -3.402823466e38f ? -3.402823466e38f : v;
}
// This lane's rates; states past the state size get 0.
template <int NS>
__device__ __forceinline__ void load_rates(const float *A, int nn, float (&A2)[NS]) {
    RowRaw<float, NS> r;
    r.zero();
    if (nn > 0) r.load(A, nn);
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] = sel_rate(r.get(i));
}

// FN<type, kernel state size>(...) for a's state size; returns its result.
#define SSD_SEL_DISPATCH(FN, ...)                                                        \
    switch (selective_kernel_dstate(a.dstate)) {                                         \
        case 4: return bf16 ? FN<bf16_t, 4>(__VA_ARGS__) : FN<float, 4>(__VA_ARGS__);    \
        case 8: return bf16 ? FN<bf16_t, 8>(__VA_ARGS__) : FN<float, 8>(__VA_ARGS__);    \
        case 16: return bf16 ? FN<bf16_t, 16>(__VA_ARGS__) : FN<float, 16>(__VA_ARGS__); \
        case 32: return bf16 ? FN<bf16_t, 32>(__VA_ARGS__) : FN<float, 32>(__VA_ARGS__); \
        case 64: return bf16 ? FN<bf16_t, 64>(__VA_ARGS__) : FN<float, 64>(__VA_ARGS__); \
        default: return hipErrorInvalidValue;                                            \
    }

}  // namespace ssd
