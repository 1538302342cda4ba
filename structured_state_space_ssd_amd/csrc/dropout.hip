// Dropout with a mask that is computed where it is needed and never stored
// (dropout.h): y = x / (1 - p) where an element stays, 0 where it is dropped,
// whatever it held. The same call on the gradient is the backward pass.
//
// Bound by memory (an element in, one out) with the generator's 20 products of 32
// bits for 8 elements close behind. A lane takes vectors of 8 columns, one generator
// call each, a grid's stride apart; row and column advance by additions, so
// that odd widths need no division per vector. 16384 x 5120 bf16: 63 us, 5.3 TB/s, a
// large copy's rate.
#include "dropout.h"
#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

constexpr int kDropLanes = 256, kDropVec = 8;

// WHOLE: rows are whole vectors. nvec: vectors of a row; a grid's stride is
// step_rows rows and step_vecs vectors.
template <typename T, bool WHOLE, int AHEAD>
__global__ __launch_bounds__(kDropLanes) void dropout_kernel(
    const T *__restrict__ x, size_t x_stride, long long rows, int D, int nvec, int step_rows,
    int step_vecs, DropArgs drop, T *__restrict__ y) {
    constexpr int V = kDropVec;
    const DropState rng = drop_state(drop);
    const uint32_t first = blockIdx.x * kDropLanes + threadIdx.x;
    long long row = first / static_cast<uint32_t>(nvec);
    int vec = static_cast<int>(first % static_cast<uint32_t>(nvec));
    while (row < rows) {
        RowRaw<T, V> raw[AHEAD];
        long long at_row[AHEAD];
        int at_vec[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            at_row[k] = row;
            at_vec[k] = vec;
            if (row < rows) {
                const T *p = x + row * x_stride + vec * V;
                if (WHOLE) raw[k].load(p);
                else raw[k].load(p, D - vec * V);
            }
            vec += step_vecs;
            row += step_rows;
            if (vec >= nvec) {
                vec -= nvec;
                ++row;
            }
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (at_row[k] >= rows) break;
            DropBits bits;
            bits.set(rng, static_cast<uint32_t>(at_vec[k]) * V, static_cast<uint32_t>(at_row[k]));
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                o[e] = bits.keep(e, drop.threshold) ? raw[k].get(e) * drop.scale : 0.0f;
            row_store(y + at_row[k] * D + at_vec[k] * V, o, WHOLE ? V : D - at_vec[k] * V);
        }
    }
}

template <typename T> hipError_t dropout(const DropoutArgs &a, hipStream_t stream) {
    constexpr int AHEAD = 2;
    const long long nvec = (a.width + kDropVec - 1LL) / kDropVec, items = a.rows * nvec;
    const long long want = (items + kDropLanes * AHEAD - 1) / (kDropLanes * AHEAD);
    const int grid = static_cast<int>(want < kDropGrid ? want : kDropGrid);
    const long long step = (long long)grid * kDropLanes;
    const int rows = static_cast<int>(step / nvec), vecs = static_cast<int>(step % nvec);
#define SSD_DROPOUT(WHOLE)                                                                        \
    dropout_kernel<T, WHOLE, AHEAD><<<grid, kDropLanes, 0, stream>>>(                             \
        static_cast<const T *>(a.x), a.x_stride, a.rows, a.width, static_cast<int>(nvec), rows,   \
        vecs, a.drop, static_cast<T *>(a.y))
    if (a.width % kDropVec == 0) SSD_DROPOUT(true);
    else SSD_DROPOUT(false);
#undef SSD_DROPOUT
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, bool bf16, hipStream_t stream) {
    return bf16 ? dropout<bf16_t>(a, stream) : dropout<float>(a, stream);
}

}  // namespace ssd
