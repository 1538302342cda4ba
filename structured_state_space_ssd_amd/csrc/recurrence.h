// Device code shared by the gated recurrence's walks, forward (recurrence.hip) and
// back (recurrence_bwd.hip). The layout of a workgroup:
//   it holds 32 channels of one sequence; a strand of 16 lanes with two channels
//   each holds S (4 or 8) consecutive tokens, a wavefront four strands one after the
//   other, the workgroup `waves` wavefronts one after the other: a tile of
//   4 S waves tokens, which it walks along the token axis.
// A strand's tokens are a map h -> A h + H of the state entering it; maps are put
// together across the strands of a wavefront by swaps of registers and across the
// wavefronts through LDS, so one barrier a tile is all that the walk waits for.
//
// A map that starts a sequence anew inside (packed sequences) is marked by a
// negative A (a product of decays is not): the state before it does not
// enter, not even as 0 times an infinity.
#pragma once

#include "ssd_common.h"
#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

// The code of a token that no sequence of a packed axis holds: padding, which starts from a
// zero state like a first token and gives zeros, whatever it holds.
constexpr int kRecNone = -0x7fffffff;
constexpr int kRecCols = 32;

// Two channels' values of one token.
template <typename T> struct RecPair;
typedef uint32_t u32_any __attribute__((aligned(2)));
template <> struct RecPair<bf16_t> {
    uint32_t w;
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void load(const char *p) { w = *reinterpret_cast<const u32_any *>(p); }
    __device__ __forceinline__ void load_one(const char *p) { w = *reinterpret_cast<const bf16_t *>(p); }
    __device__ __forceinline__ float get(int e) const {
        return __uint_as_float(e ? (w & 0xffff0000u) : (w << 16));
    }
    static __device__ __forceinline__ void store(char *p, float a, float b) {
        *reinterpret_cast<u32_any *>(p) = pack_bf16(a, b);
    }
    static __device__ __forceinline__ void store_one(char *p, float a) {
        *reinterpret_cast<bf16_t *>(p) = static_cast<bf16_t>(pack_bf16(a, 0.0f));
    }
};
template <> struct RecPair<float> {
    float w[2];
    __device__ __forceinline__ void zero() { w[0] = w[1] = 0.0f; }
    __device__ __forceinline__ void load(const char *p) {
        const f32x2_any u = *reinterpret_cast<const f32x2_any *>(p);
        w[0] = u[0]; w[1] = u[1];
    }
    __device__ __forceinline__ void load_one(const char *p) {
        w[0] = *reinterpret_cast<const float *>(p);
        w[1] = 0.0f;
    }
    __device__ __forceinline__ float get(int e) const { return w[e]; }
    static __device__ __forceinline__ void store(char *p, float a, float b) {
        *reinterpret_cast<f32x2_any *>(p) = f32x2_any{a, b};
    }
    static __device__ __forceinline__ void store_one(char *p, float a) { *reinterpret_cast<float *>(p) = a; }
};

// Where a lane is: its strand, channels and the workgroup's unit.
struct RecPlace {
    int batch, seg, ch, nch;      // nch: channels of the lane inside the tensor, 0 to 2
    int wave, sub, col;           // strand `sub` of wavefront `wave`, lane `col` of the strand
    int begin, end;               // the segment's tokens
    bool live;                    // a unit of the grid that there is
};
// Units one after the other along the channels go to the same XCD (workgroups
// are dealt to the eight XCDs in turn): they share cache lines.
__device__ __forceinline__ RecPlace rec_place(const RecArgs &a, int segs) {
    RecPlace p;
    const int units = a.batch * a.blocks * segs, each = (units + 7) >> 3;
    const int id = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    p.live = (int)(blockIdx.x >> 3) < each && id < units;
    const int rest = id / a.blocks, block = id - rest * a.blocks;
    p.batch = rest / segs;
    p.seg = rest - p.batch * segs;
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p.sub = (threadIdx.x >> 4) & 3;
    p.col = threadIdx.x & 15;
    p.ch = block * kRecCols + 2 * p.col;
    p.nch = min(max(a.channels - p.ch, 0), 2);
    p.begin = p.seg * a.seg_len;
    p.end = min(p.begin + a.seg_len, a.seqlen);
    return p;
}

// Bytes between tokens, as a value that the compiler takes anew in every tile: offsets
// made of it ahead of the walk would fill the registers.
template <typename T> __device__ __forceinline__ uint32_t rec_bytes(size_t token) {
    uint32_t step = static_cast<uint32_t>(token * sizeof(T));
    asm volatile("" : "+s"(step));
    return step;
}
// Byte offset of a lane's first token and channel (strides are below 2^24 elements).
template <typename T, int S> __device__ __forceinline__ uint32_t rec_offset(uint32_t step, const RecPlace &p) {
    return static_cast<uint32_t>(p.sub * S) * step + p.ch * static_cast<uint32_t>(sizeof(T));
}
// A lane's tokens of one tensor, whose wavefront's first is element `at` (uniform).
// WHOLE: every token and channel is there.
template <typename T, bool WHOLE, int S>
__device__ __forceinline__ void rec_load(RecPair<T> (&r)[S], const void *t, size_t at, size_t token,
                                         const RecPlace &p, int nt) {
    const char *base = static_cast<const char *>(t) + at * sizeof(T);
    const uint32_t step = rec_bytes<T>(token);
    uint32_t off = rec_offset<T, S>(step, p);
#pragma unroll
    for (int j = 0; j < S; ++j, off += step) {
        if (WHOLE) r[j].load(base + off);
        else {
            r[j].zero();
            if (j < nt) {
                if (p.nch == 2) r[j].load(base + off);
                else if (p.nch == 1) r[j].load_one(base + off);
            }
        }
    }
}
// A token of a dense tensor, `base` as above and `off` its byte offset.
template <typename T, bool WHOLE>
__device__ __forceinline__ void rec_store(char *base, uint32_t off, int nch, float a, float b) {
    if (WHOLE || nch == 2) RecPair<T>::store(base + off, a, b);
    else if (nch == 1) RecPair<T>::store_one(base + off, a);
}

// ---- gates ------------------------------------------------------------------------

// -c softplus(decay) log2(e): what a channel's open gate decays by, in log2.
__device__ __forceinline__ float rec_rate(float decay, float c) { return -c * softplus_f32(decay) * kLog2e; }

// 1 - e^t for t <= 0, to a few roundings of itself: the series up to t^6 where 1 and
// e^t cancel (the next term is below 2^-24 of the sum), else 1 - a^2 with the given
// a = e^(t/2).
__device__ __forceinline__ float one_minus_square(float t, float a) {
    float s = fmaf(t, 1.0f / 720.0f, 1.0f / 120.0f);
    s = fmaf(t, s, 1.0f / 24.0f);
    s = fmaf(t, s, 1.0f / 6.0f);
    s = fmaf(t, s, 0.5f);
    s = fmaf(t, s, 1.0f);
    return t > -0.25f ? -t * s : fmaf(-a, a, 1.0f);
}

constexpr float kLn2 = 0.6931471805599453f;

// ---- maps -------------------------------------------------------------------------

struct RecMap {
    float a, h;
};
// first, then second
template <bool PACKED> __device__ __forceinline__ RecMap rec_then(RecMap first, RecMap second) {
    if (PACKED) {
        const bool cut = second.a < 0.0f;
        return {cut || first.a < 0.0f ? -1.0f : first.a * second.a,
                cut ? second.h : fmaf(second.a, first.h, second.h)};
    }
    return {first.a * second.a, fmaf(second.a, first.h, second.h)};
}
template <bool PACKED> __device__ __forceinline__ float rec_apply(RecMap m, float h) {
    return PACKED && m.a < 0.0f ? m.h : fmaf(m.a, h, m.h);
}

// The wavefront's four strands put together in the order of their tokens, or against
// it (REVERSE): `whole` all of them, `before` those that come before the lane's own.
template <bool PACKED, bool REVERSE>
__device__ __forceinline__ void rec_wave(RecMap m, int sub, RecMap &before, RecMap &whole) {
    auto swap16 = [](float v, float &even, float &odd) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        even = __uint_as_float(r[0]);
        odd = __uint_as_float(r[1]);
    };
    auto swap32 = [](float v, float &low, float &high) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        low = __uint_as_float(r[0]);
        high = __uint_as_float(r[1]);
    };
    RecMap even, odd, low, high;
    swap16(m.a, even.a, odd.a);
    swap16(m.h, even.h, odd.h);
    const RecMap pair = REVERSE ? rec_then<PACKED>(odd, even) : rec_then<PACKED>(even, odd);
    swap32(pair.a, low.a, high.a);
    swap32(pair.h, low.h, high.h);
    whole = REVERSE ? rec_then<PACKED>(high, low) : rec_then<PACKED>(low, high);
    // within the pair, the second of the two comes after the first; the same for the pairs
    const bool second = REVERSE ? !(sub & 1) : (sub & 1), later = REVERSE ? !(sub & 2) : (sub & 2) != 0;
    const RecMap mate = REVERSE ? odd : even, pairs = REVERSE ? high : low;
    const RecMap none = {1.0f, 0.0f};
    const RecMap in = second ? mate : none;
    const RecMap joined = rec_then<PACKED>(pairs, in);
    before = later ? (second ? joined : pairs) : in;
}

}  // namespace ssd
