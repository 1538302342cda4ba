// Shared by the selective scan's forward, backward and single-token kernels.
#pragma once

#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

// A lane holds 4 states of one channel; the NK/4 lanes that share the channel
// (NK: the state size rounded up to 4, 8, 16, 32 or 64) are neighbours, so a
// workgroup of 256 lanes holds 1024 / NK channels.
template <int NK> struct SelShape {
    static constexpr int SL = NK / 4;           // lanes per channel
    static constexpr int CH = 256 / SL;         // channels per workgroup
    static constexpr int TILE = NK < 16 ? 2 * NK : 32;  // tokens staged at a time
    static constexpr int BACK = NK < 16 ? 8 : 16;       // and by the backward, which keeps the
                                                        // states before every so many tokens
};

// Sum over the SL neighbouring lanes, in each of them: DPP moves within a row
// of 16 lanes (neighbour, neighbour pair, half row, row).
template <int SL> __device__ __forceinline__ float lanes_sum(float v) {
    auto add = [](float a, int b) { return a + __int_as_float(b); };
    if constexpr (SL >= 2) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));
    if constexpr (SL >= 4) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));
    if constexpr (SL >= 8) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));
    if constexpr (SL >= 16) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));
    return v;
}

// The step size of raw value v (bias included): softplus and clamp as chosen.
__device__ __forceinline__ float sel_step(const DtOpts &o, float v) {
    if (o.softplus) v = softplus_f32(v);
    if (o.clamp) v = fminf(fmaxf(v, o.lo), o.hi);
    return v;
}

// Where a workgroup of the scan stands: sequence b, segment seg, channels
// first .. first + n - 1, all of group g.
struct SelBlock {
    int b, seg, g, first, n;
};
template <int NK> __device__ __forceinline__ SelBlock sel_block(int id, int channels, int ngroups, int segs) {
    constexpr int CH = SelShape<NK>::CH;
    const int each = channels / ngroups, per = (each + CH - 1) / CH;
    SelBlock k;
    const int cb = id % (per * ngroups), rest = id / (per * ngroups);
    k.seg = rest % segs;
    k.b = rest / segs;
    k.g = cb / per;
    const int at = (cb % per) * CH;
    k.first = k.g * each + at;
    k.n = each - at < CH ? each - at : CH;
    return k;
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
