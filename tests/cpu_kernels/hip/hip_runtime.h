// A stand-in for the HIP runtime under which the layers' kernels run on the CPU,
// one workgroup after another: every lane is a fiber that runs until it meets
// its wavefront (an exchange between lanes) or its workgroup (a barrier).
// What it is for: memory comes from allocations with an unmapped page on either
// side, arrays are compiled with bounds checks, and lanes can be run in any
// order, so that an access out of range ends the program and a missing barrier
// changes results. Rounding, timing and memory order are not the GPU's.
#pragma once
#include <math.h>
#include <setjmp.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <sys/mman.h>
#include <ucontext.h>

#include <algorithm>
#include <array>
#include <functional>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static

typedef void *hipStream_t;
typedef void *hipEvent_t;
enum hipError_t { hipSuccess = 0, hipErrorInvalidValue = 1, hipErrorNotSupported = 801 };
inline hipError_t hipGetLastError() { return hipSuccess; }
struct dim3 {
    unsigned x, y, z;
    dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
struct float2 { float x, y; };
struct float4 { float x, y, z, w; };
inline float2 make_float2(float a, float b) { return {a, b}; }
inline float4 make_float4(float a, float b, float c, float d) { return {a, b, c, d}; }
using std::max;
using std::min;

inline dim3 threadIdx, blockIdx, blockDim, gridDim;

namespace cpu {

constexpr size_t kStack = 256 << 10;
constexpr int kBarrier = 1 << 30;  // "line" of a barrier

struct Lane {
    ucontext_t ctx;
    jmp_buf at;
    bool started, live;
    int line;      // where it waits, 0: nowhere
    uint32_t out;  // what it gives
};
struct Wave {
    uint32_t val[64];
    uint64_t mask;  // lanes that meet
};
inline Lane lanes[1024];
inline Wave waves[16];
inline char *stacks;
inline jmp_buf scheduler;
inline int current;
inline int order = 0;  // 0: lanes in order, 1: backward, else: shuffled by it
inline const std::function<void()> *body;

inline void entry() {
    (*body)();
    lanes[current].live = false;
    _longjmp(scheduler, 1);
}

inline void resume(int t) {
    current = t;
    threadIdx = dim3(t, 0, 0);
    if (_setjmp(scheduler)) return;
    Lane &l = lanes[t];
    if (l.started) _longjmp(l.at, 1);
    l.started = true;
    getcontext(&l.ctx);
    l.ctx.uc_stack.ss_sp = stacks + (size_t)t * kStack;
    l.ctx.uc_stack.ss_size = kStack;
    l.ctx.uc_link = nullptr;
    makecontext(&l.ctx, entry, 0);
    setcontext(&l.ctx);
}

// The calling lane waits at `line`; the scheduler runs the others.
inline void wait_at(int line) {
    Lane &l = lanes[current];
    l.line = line;
    if (_setjmp(l.at)) return;
    _longjmp(scheduler, 1);
}

inline void fail(const char *what) {
    fprintf(stderr, "cpu kernels: %s\n", what);
    abort();
}

inline void run_block(int threads) {
    std::vector<int> seq(threads);
    for (int t = 0; t < threads; ++t) {
        lanes[t].started = false;
        lanes[t].live = true;
        lanes[t].line = 0;
        seq[t] = order == 1 ? threads - 1 - t : t;
    }
    uint32_t rnd = order * 2654435761u + 1;
    const int nw = (threads + 63) / 64;
    for (;;) {
        if (order > 1)
            for (int i = threads - 1; i > 0; --i) {
                rnd = rnd * 1664525u + 1013904223u;
                std::swap(seq[i], seq[(rnd >> 8) % (i + 1)]);
            }
        bool any = false;
        for (int t : seq)
            if (lanes[t].live && lanes[t].line == 0) {
                resume(t);
                any |= lanes[t].live;
            } else any |= lanes[t].live;
        if (!any) return;
        // Lanes of a wavefront that exchange: those furthest back in the source are the
        // ones that the others wait for.
        bool met = false;
        for (int w = 0; w < nw; ++w) {
            int line = kBarrier;
            for (int t = w * 64; t < min(threads, w * 64 + 64); ++t)
                if (lanes[t].live) line = min(line, lanes[t].line);
            if (line == kBarrier) continue;
            waves[w].mask = 0;
            for (int t = w * 64; t < min(threads, w * 64 + 64); ++t)
                if (lanes[t].live && lanes[t].line == line) {
                    waves[w].mask |= 1ull << (t & 63);
                    waves[w].val[t & 63] = lanes[t].out;
                    lanes[t].line = 0;
                }
            met = true;
        }
        if (met) continue;
        for (int t = 0; t < threads; ++t)  // all at the barrier
            if (lanes[t].live) lanes[t].line = 0;
    }
}

inline void launch(dim3 grid, int threads, const std::function<void()> &f) {
    if (threads < 1 || threads > 1024) fail("workgroup size");
    if ((uint64_t)grid.x * threads >> 32) fail("grid size");
    if (!stacks)
        stacks = (char *)mmap(nullptr, 1024 * kStack, PROT_READ | PROT_WRITE,
                              MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
    body = &f;
    gridDim = grid;
    blockDim = dim3(threads);
    for (unsigned y = 0; y < grid.y; ++y)
        for (unsigned x = 0; x < grid.x; ++x) {
            blockIdx = dim3(x, y);
            run_block(threads);
        }
}

// The value of lane `from` of the wavefront; `ok`: whether it takes part.
inline uint32_t taken(int from, bool &ok) {
    const Wave &w = waves[threadIdx.x >> 6];
    ok = w.mask >> from & 1;
    return ok ? w.val[from] : 0;
}
inline void give(uint32_t v, int line) {
    lanes[current].out = v;
    wait_at(line);
}

inline int dpp(int old, int v, int ctrl, int line) {
    (void)old;
    const int l = threadIdx.x & 63, row = l & ~15, i = l & 15;
    int from;
    if (ctrl < 0x100) from = (l & ~3) | ((ctrl >> (2 * (l & 3))) & 3);  // within four
    else if (ctrl == 0x140) from = row | (15 - i);                     // row mirrored
    else if (ctrl == 0x141) from = (l & ~7) | (7 - (l & 7));           // half row mirrored
    else if (ctrl > 0x120 && ctrl < 0x130) from = row | ((i - (ctrl - 0x120)) & 15);  // row rotated
    else fail("dpp control"), from = 0;
    give((uint32_t)v, line);
    bool ok;
    const uint32_t r = taken(from, ok);
    if (!ok) fail("a lane reads one that is not there");
    return (int)r;
}
// permlane{16,32}_swap of a lane's (a, b) with a == b or not: `half` odd groups of a
// change places with the even groups of b.
inline std::array<uint32_t, 2> swap(uint32_t a, uint32_t b, int half, int line) {
    const int l = threadIdx.x & 63;
    const bool odd = l & half;
    // an odd group gives its a and takes the even one's b, and the other way round
    give(odd ? a : b, line);
    bool ok;
    const uint32_t r = taken(l ^ half, ok);
    if (!ok) fail("a lane reads one that is not there");
    return odd ? std::array<uint32_t, 2>{r, b} : std::array<uint32_t, 2>{a, r};
}
inline float shfl_xor(float v, int off, int line) {
    uint32_t u;
    memcpy(&u, &v, 4);
    give(u, line);
    bool ok;
    u = taken((threadIdx.x & 63) ^ off, ok);
    if (!ok) fail("a lane reads one that is not there");
    memcpy(&v, &u, 4);
    return v;
}
inline float med3(float a, float b, float c) { return fmaxf(fminf(fmaxf(a, b), c), fminf(a, b)); }

}  // namespace cpu

#define __syncthreads() cpu::wait_at(cpu::kBarrier)
#define __shfl_xor(v, off) cpu::shfl_xor(v, off, __LINE__)
#define __builtin_amdgcn_update_dpp(o, v, c, a, b, z) cpu::dpp(o, v, c, __LINE__)
#define __builtin_amdgcn_permlane16_swap(a, b, c, d) cpu::swap(a, b, 16, __LINE__)
#define __builtin_amdgcn_permlane32_swap(a, b, c, d) cpu::swap(a, b, 32, __LINE__)
#define __builtin_amdgcn_sched_barrier(x)
#define __builtin_amdgcn_s_waitcnt(x) ((void)0)
#define __builtin_amdgcn_readfirstlane(x) (x)
#define __builtin_amdgcn_exp2f exp2f
#define __builtin_amdgcn_logf log2f
#define __builtin_amdgcn_rcpf(x) (1.0f / (x))
#define __builtin_amdgcn_fmed3f cpu::med3

inline float __uint_as_float(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
inline uint32_t __float_as_uint(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
inline float __int_as_float(int u) { float f; memcpy(&f, &u, 4); return f; }
inline int __float_as_int(float f) { int u; memcpy(&u, &f, 4); return u; }
