// Random bits of dropout, the same wherever an element's mask is formed: Philox
// 4x32 with 10 rounds (J. K. Salmon, M. A. Moraes, R. O. Dror and D. E. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011), which turns a counter and
// a key into 128 bits. Counter: (column / 8, row, offset low, offset high); key:
// the seed. Eight columns of a row share a call and take 16 bits each: bits
// 16 (c & 1) and up of word (c & 7) / 2. An element is dropped where these
// are below `threshold` = round(65536 p).
#pragma once

#include "ssd_common.h"

namespace ssd {

__device__ __forceinline__ void philox_words(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t p0 = static_cast<uint64_t>(c[0]) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
        c[0] = static_cast<uint32_t>(p1 >> 32) ^ c[1] ^ k0;
        c[1] = static_cast<uint32_t>(p1);
        c[2] = static_cast<uint32_t>(p0 >> 32) ^ c[3] ^ k1;
        c[3] = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Seed and offset, the GPU's where the caller keeps them there.
struct DropState {
    uint32_t seed0, seed1, off0, off1;
};
__device__ __forceinline__ DropState drop_state(const DropArgs &d) {
    const unsigned long long seed = d.rng ? d.rng[0] : d.seed, off = d.rng ? d.rng[1] : d.offset;
    return {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32),
            static_cast<uint32_t>(off), static_cast<uint32_t>(off >> 32)};
}

// Bits of the eight columns of which `col` is one (two of them a word).
struct DropBits {
    uint32_t w[4];
    __device__ __forceinline__ void set(const DropState &s, uint32_t col, uint32_t row) {
        w[0] = col >> 3; w[1] = row; w[2] = s.off0; w[3] = s.off1;
        philox_words(w, s.seed0, s.seed1);
    }
    // whether the column c stays (c & 7 known where this is compiled)
    __device__ __forceinline__ bool keep(int c, uint32_t threshold) const {
        const uint32_t v = w[(c & 7) >> 1];
        return ((c & 1) ? v >> 16 : v & 0xffffu) >= threshold;
    }
};

}  // namespace ssd
