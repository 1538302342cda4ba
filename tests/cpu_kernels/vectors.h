// Types of the HIP runtime that the recurrent block's kernels use beside those in
// hip/hip_runtime.h here.
#pragma once
struct uint4 { unsigned x, y, z, w; };
inline uint4 make_uint4(unsigned a, unsigned b, unsigned c, unsigned d) { return {a, b, c, d}; }
// Buffer loads and stores, from a base that all lanes have alike.
#include <string.h>
typedef char *cpu_buffer;
typedef unsigned cpu_word2 __attribute__((ext_vector_type(2)));
#define __amdgpu_buffer_rsrc_t cpu_buffer
#define __builtin_amdgcn_make_buffer_rsrc(p, stride, n, flags) ((cpu_buffer)(p))
template <typename W> inline W cpu_buffer_load(cpu_buffer p, unsigned off, unsigned row) {
    W w;
    memcpy(&w, p + ((size_t)off + row), sizeof(w));
    return w;
}
template <typename W> inline void cpu_buffer_store(W w, cpu_buffer p, unsigned off, unsigned row) {
    memcpy(p + ((size_t)off + row), &w, sizeof(w));
}
#define __builtin_amdgcn_raw_buffer_load_b32(p, off, row, aux) cpu_buffer_load<unsigned>(p, off, row)
#define __builtin_amdgcn_raw_buffer_load_b64(p, off, row, aux) cpu_buffer_load<cpu_word2>(p, off, row)
#define __builtin_amdgcn_raw_buffer_store_b32(w, p, off, row, aux) cpu_buffer_store<unsigned>(w, p, off, row)
#define __builtin_amdgcn_raw_buffer_store_b64(w, p, off, row, aux) cpu_buffer_store<cpu_word2>(w, p, off, row)
