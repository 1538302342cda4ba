// Types of the HIP runtime that the recurrent block's kernels use beside those in
// hip/hip_runtime.h here.
#pragma once
struct uint4 { unsigned x, y, z, w; };
inline uint4 make_uint4(unsigned a, unsigned b, unsigned c, unsigned d) { return {a, b, c, d}; }
