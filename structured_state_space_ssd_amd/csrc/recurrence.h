// Device code shared by the gated recurrence's passes, forward (recurrence.hip) and back
// (recurrence_bwd.hip). The layout of a workgroup:
//   it holds one tile: 32 channels of one sequence (a unit) for 4 S waves consecutive
//   tokens. A strand of 16 lanes with two channels each holds S (4 or 8) consecutive
//   tokens, a wavefront four strands one after the other, the workgroup `waves`
//   wavefronts one after the other.
// A strand's tokens are a map h -> A h + H of the state entering it; maps are put
// together across the strands of a wavefront by swaps of registers, across the
// wavefronts through LDS and across the tiles of a unit through memory (rec_enter), so
// that every operand is read once, whatever the number of channels, and tokens fill the
// GPU as channels do. Few units are the exception (rec_place).
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
constexpr int kRecCols = 32, kRecWaves = 4;  // a workgroup's channels, and wavefronts at most

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
    // as a value that the compiler has not seen
    __device__ __forceinline__ void fresh() { asm volatile("" : "+v"(w)); }
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
    __device__ __forceinline__ void fresh() {
        float u = w[0], v = w[1];
        asm volatile("" : "+v"(u));
        asm volatile("" : "+v"(v));
        w[0] = u; w[1] = v;
    }
    static __device__ __forceinline__ void store(char *p, float a, float b) {
        *reinterpret_cast<f32x2_any *>(p) = f32x2_any{a, b};
    }
    static __device__ __forceinline__ void store_one(char *p, float a) { *reinterpret_cast<float *>(p) = a; }
};

// Where a lane is: its strand and channels, and the workgroup's unit.
struct RecPlace {
    int unit, batch, ch, nch;     // nch: channels of the lane inside the tensor, 0 to 2
    int wave, sub, col;           // strand `sub` of wavefront `wave`, lane `col` of the strand
    bool live;                    // a unit of the grid that there is
};
__device__ __forceinline__ int rec_quotient(int n, const RecDivisor &d) {
    return static_cast<int>(static_cast<unsigned long long>(n) * d.mul >> d.shift);
}
// Every unit has as many workgroups as tiles. Units one after the other along the channels
// go to the same XCD (workgroups are dealt to the eight XCDs in turn): they share
// cache lines. So every XCD takes ceil(units / 8) of them from the first one on, and few units
// leave XCDs without: 1 of 8 works on one unit, 5 on 9 or 10. 1 x 16384 tokens bf16 without z:
// 17 us forward and 27 back with 32 channels, 21 and 32 with 256 (8 units), 22 and 40 with 288
// (9), 22 and 40 with 512 (16): with so few a state's way through the 128 tiles (256 back)
// takes the time, and where the units lie shows back from 9 on.
__device__ __forceinline__ RecPlace rec_place(const RecArgs &a) {
    RecPlace p;
    const int units = a.batch * a.blocks, each = (units + 7) >> 3, slot = blockIdx.x >> 3;
    p.unit = (blockIdx.x & 7) * each + (slot - rec_quotient(slot, a.by_each) * each);
    p.live = p.unit < units;
    p.batch = rec_quotient(p.unit, a.by_blocks);
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p.sub = (threadIdx.x >> 4) & 3;
    p.col = threadIdx.x & 15;
    p.ch = (p.unit - p.batch * a.blocks) * kRecCols + 2 * p.col;
    p.nch = min(max(a.channels - p.ch, 0), 2);
    return p;
}

// Whether any of a tile's n tokens of a packed axis is a first or last one of a sequence, or
// in none: of most tiles none is, and they go without the selections (1 x 16384 tokens x 2560
// channels in 55 sequences, bf16 without z: back 217 us with them everywhere, 207 so; forward
// 97 to 103 both ways, float32 157 and 153). cuts: per 64
// tokens, whether any is; a tile begins at the first of 64 and has 128 at most.
__device__ __forceinline__ bool rec_cuts(const int *cuts, int from, int n) {
    const int *at = cuts + from / 64;
    return (at[0] | at[n > 64]) != 0;
}

// Byte offset of a lane's first token and channel (strides are below 2^24 elements).
template <typename T, int S> __device__ __forceinline__ uint32_t rec_offset(size_t token, const RecPlace &p) {
    return (static_cast<uint32_t>(p.sub * S) * static_cast<uint32_t>(token) + p.ch) * static_cast<uint32_t>(sizeof(T));
}
// A lane's tokens of one tensor, whose wavefront's first is element `at`: uniform bases, one
// offset. WHOLE: every token and channel is there.
template <typename T, bool WHOLE, int S>
__device__ __forceinline__ void rec_load(RecPair<T> (&r)[S], const void *t, size_t at, size_t token,
                                         const RecPlace &p, int nt) {
    const uint32_t off = rec_offset<T, S>(token, p);
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const char *base = static_cast<const char *>(t) + (at + j * token) * sizeof(T);
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
// A token of a dense tensor: `base` uniform, `off` the lane's byte offset.
template <typename T, bool WHOLE>
__device__ __forceinline__ void rec_store(char *base, uint32_t off, int nch, float a, float b) {
    if (WHOLE || nch == 2) RecPair<T>::store(base + off, a, b);
    else if (nch == 1) RecPair<T>::store_one(base + off, a);
}

// ---- gates ------------------------------------------------------------------------

// -c softplus(decay) log2(e): what a channel's open gate decays by, in log2.
__device__ __forceinline__ float rec_rate(float decay, float c) { return -c * softplus_f32(decay) * kLog2e; }
// The lane's channels' (0 past the last one).
__device__ __forceinline__ void rec_rates(float (&rate)[2], const RecArgs &a, const RecPlace &p) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
        rate[e] = e < p.nch ? a.rate ? a.rate[p.ch + e] : rec_rate(a.decay[p.ch + e], a.c) : 0.0f;
}

// 1 - a^2 for a = 2^l with l <= 0, to a few roundings of itself. Where 1 and a^2 cancel (a
// above e^-0.25) it is -2 a sinh(log a): a l (c1 + c3 l^2 + c5 l^4) with c_n = -2 ln(2)^n / n!
// (the next term is below 2^-24 of the sum).
__device__ __forceinline__ float one_minus_square(float l, float a) {
    const float l2 = l * l;
    float s = fmaf(l2, -0.0026672267f, -0.11100822f);
    s = fmaf(l2, s, -1.3862944f);
    return l > -0.36067376f ? a * (l * s) : fmaf(-a, a, 1.0f);
}

constexpr float kLn2 = 0.6931471805599453f;

// ---- maps -------------------------------------------------------------------------

struct RecMap {
    float a, h;
};
// a h + v. GROWS (the direct form, where decays may pass 1): the product of many may be
// infinite, and a state of zero stays out of it.
template <bool GROWS> __device__ __forceinline__ float rec_carry(float a, float h, float v) {
    return GROWS && h == 0.0f ? v : fmaf(a, h, v);
}
// first, then second
template <bool PACKED, bool GROWS> __device__ __forceinline__ RecMap rec_then(RecMap first, RecMap second) {
    if (PACKED) {
        const bool cut = second.a < 0.0f;
        return {cut || first.a < 0.0f ? -1.0f : first.a * second.a,
                cut ? second.h : rec_carry<GROWS>(second.a, first.h, second.h)};
    }
    return {first.a * second.a, rec_carry<GROWS>(second.a, first.h, second.h)};
}
template <bool PACKED, bool GROWS> __device__ __forceinline__ float rec_apply(RecMap m, float h) {
    return PACKED && m.a < 0.0f ? m.h : rec_carry<GROWS>(m.a, h, m.h);
}

// The wavefront's four strands put together in the order of their tokens, or against
// it (REVERSE): `whole` all of them, `before` those that come before the lane's own.
template <bool PACKED, bool GROWS, bool REVERSE>
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
    const RecMap pair = REVERSE ? rec_then<PACKED, GROWS>(odd, even) : rec_then<PACKED, GROWS>(even, odd);
    swap32(pair.a, low.a, high.a);
    swap32(pair.h, low.h, high.h);
    whole = REVERSE ? rec_then<PACKED, GROWS>(high, low) : rec_then<PACKED, GROWS>(low, high);
    // within the pair, the second of the two comes after the first; the same for the pairs
    const bool second = REVERSE ? !(sub & 1) : (sub & 1), later = REVERSE ? !(sub & 2) : (sub & 2) != 0;
    const RecMap mate = REVERSE ? odd : even, pairs = REVERSE ? high : low;
    const RecMap none = {1.0f, 0.0f};
    const RecMap in = second ? mate : none, joined = rec_then<PACKED, GROWS>(pairs, in);
    before = later ? joined : in;
}


// ---- across the tiles of a unit -------------------------------------------------------
//
// A unit's tiles are taken in the order in which its workgroups start: the first one
// to start takes the first tile (the last one, back). So the tiles that come before a
// workgroup's own are held by workgroups that have started, which wait for tiles before
// theirs only: every wait ends, in whatever order and however few at a time the GPU
// runs the workgroups.
//
// A tile first makes the map of all its tokens known, then waits for those of the tiles
// before it in its group of kRecGroup and for the state that enters the group, which the last tile
// of the group before makes known: its state comes from the same maps in the same
// order every time, and the way of a state through a long sequence is one wait for
// kRecGroup tiles. Each value travels in a 64-bit word of its own with what says that it is
// there, so nothing has to be ordered; before the pass all words are set to ~0.

constexpr int kRecGroup = 16, kRecAtOnce = 2;  // tiles that a lane looks at together
constexpr uint32_t kRecUnset = 0xffffffffu;

struct RecShared {
    int tile;
    float map[kRecWaves][kRecCols][2];                     // the wavefronts' maps, by channel
    float before[kRecGroup / kRecAtOnce][kRecCols][2];     // those of the tiles before
    float state[kRecCols];                                 // what enters the group
    float enters[kRecWaves][kRecCols];                     // what enters the wavefronts
};

// The workgroup's tile, in the order of starting (one that there is not, where another call has
// written over the workspace).
__device__ __forceinline__ int rec_ticket(const RecArgs &a, const RecPlace &p, RecShared &sh) {
    if (a.tiles == 1) return 0;
    if (threadIdx.x == 0)
        sh.tile = static_cast<int>(__hip_atomic_fetch_add(a.ticket + (size_t)p.unit * kRecTicketStep, 1u, __ATOMIC_RELAXED,
                                                          __HIP_MEMORY_SCOPE_AGENT) + 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(sh.tile);
}
__device__ __forceinline__ void rec_tell(unsigned long long *at, float value, uint32_t mark) {
    __hip_atomic_store(at, static_cast<unsigned long long>(__float_as_uint(value)) << 32 | mark, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long rec_look(const unsigned long long *at) {
    return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// `v`: what rec_look has seen there. A wait of about a second (a tile takes microseconds) means
// that another call has written over the workspace; it ends with what is not a number.
constexpr int kRecLooks = 1 << 20;
__device__ __forceinline__ RecMap rec_wait(const unsigned long long *at, unsigned long long v) {
    for (int k = 0; static_cast<uint32_t>(v) == kRecUnset && k < kRecLooks; ++k) {
        __builtin_amdgcn_s_sleep(1);
        v = rec_look(at);
    }
    return {__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32))};
}

// All lanes of the workgroup, with the maps of their wavefronts (the same in every strand):
// what enters the lane's wavefront. first: what enters the unit's first tile, [Bt][E] or
// NULL (zeros); last: what leaves its last one, the same. REVERSE: the last wavefront comes
// first. order: the tile's place in the order of the walk. For the wait and what follows
// a lane is a channel, and half a wavefront looks at kRecAtOnce tiles.
template <bool PACKED, bool GROWS, bool REVERSE>
__device__ __forceinline__ void rec_enter(const RecArgs &a, const RecPlace &p, int order, const RecMap (&whole)[2],
                                          const float *first, float *last, float (&enters)[2], RecShared &sh) {
    if (p.sub == 0)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sh.map[p.wave][2 * p.col + e][0] = whole[e].a;
            sh.map[p.wave][2 * p.col + e][1] = whole[e].h;
        }
    __syncthreads();
    auto wave_map = [&](int k, int c) {
        const float *v = sh.map[REVERSE ? a.waves - 1 - k : k][c];
        return RecMap{v[0], v[1]};
    };
    const int place = order % kRecGroup, group = order / kRecGroup;
    const size_t words = (size_t)a.batch * a.blocks * kRecCols;  // of one tile of every unit
    const int c = threadIdx.x & (kRecCols - 1), part = threadIdx.x / kRecCols, parts = 2 * a.waves;
    const size_t at = (size_t)p.unit * kRecCols + c;
    if (a.tiles > 1) {
        if (part == 0 && place < kRecGroup - 1 && order + 1 < a.tiles) {
            RecMap all = wave_map(0, c);
            for (int k = 1; k < a.waves; ++k) all = rec_then<PACKED, GROWS>(all, wave_map(k, c));
            // (any number but the mark of none; a decay that is not a number is one of its own)
            rec_tell(a.maps + order * words + at, all.h, all.a != all.a ? 0x7fc00000u : __float_as_uint(all.a));
        }
        for (int q = part; q * kRecAtOnce < place; q += parts) {
            const int n = place - q * kRecAtOnce;
            const unsigned long long *maps = a.maps + ((size_t)group * kRecGroup + q * kRecAtOnce) * words + at;
            unsigned long long seen[kRecAtOnce];
#pragma unroll
            for (int k = 0; k < kRecAtOnce; ++k)
                if (k < n) seen[k] = rec_look(maps + k * words);
            RecMap tiles = {1.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < kRecAtOnce; ++k)
                if (k < n) tiles = rec_then<PACKED, GROWS>(tiles, rec_wait(maps + k * words, seen[k]));
            sh.before[q][c][0] = tiles.a;
            sh.before[q][c][1] = tiles.h;
        }
        if (group > 0 && part == parts - 1) {
            const unsigned long long *enter = a.enter + group * words + at;
            sh.state[c] = rec_wait(enter, rec_look(enter)).h;
        }
        __syncthreads();
    }
    if (part == 0) {
        const int ch = (p.unit - p.batch * a.blocks) * kRecCols + c;
        float in = group > 0 ? sh.state[c] : first && ch < a.channels ? first[(size_t)p.batch * a.channels + ch] : 0.0f;
        for (int q = 0; q * kRecAtOnce < place; ++q) in = rec_apply<PACKED, GROWS>({sh.before[q][c][0], sh.before[q][c][1]}, in);
        for (int k = 0; k < a.waves; ++k) {
            sh.enters[REVERSE ? a.waves - 1 - k : k][c] = in;
            in = rec_apply<PACKED, GROWS>(wave_map(k, c), in);
        }
        if (place == kRecGroup - 1 && order + 1 < a.tiles) rec_tell(a.enter + (group + 1) * words + at, in, 0);
        if (last && order == a.tiles - 1 && ch < a.channels) last[(size_t)p.batch * a.channels + ch] = in;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) enters[e] = sh.enters[p.wave][2 * p.col + e];
}

}  // namespace ssd
