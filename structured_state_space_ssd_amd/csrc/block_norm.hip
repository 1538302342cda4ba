// What joins a block's output x to the residual stream r and makes the next
// block's input, in one pass over both, and its gradients. For a row:
//   v = norm(x) w1 + b1   (the norm after the block; without it v = x)
//   b = v g silu(z)       (layer scale g per column, gate z per element)
//   d = b / (1 - p) where the element stays, else 0                (dropout.h)
//   s = alpha r + beta d  (kept in the stream's type)
//   y = norm(s) w2 + b2   (the norm before the next block, of s as it is kept)
// norm(u) = (u - m) / sqrt(mean((u - m)^2) + eps) = n, m the mean or, in the
// root-mean-square form, 0; its gradient of dn is rstd (dn - mean(dn) - n mean(dn n)).
// Backward, with ds the gradient of s (dsum and, through the norm before, dy's):
//   dr = alpha ds,  db = beta ds / (1 - p) or 0,  dz = db v g silu'(z),
//   e = db silu(z),  dx = gradient of norm(x) for e g w1,
//   dw2 = sum dy n2, db2 = sum dy, and from P = sum e n1 and Q = sum e over the rows
//   dw1 = g P, db1 = g Q, dg = w1 P + b1 Q (without the norm after: dg = sum e x).
// So four sums per column give all five parameters' gradients.
//
// Bound by memory: every tensor is read once and written once. A row stays in
// registers from the load to the stores, held by a group of lanes as in norm.hip;
// the two norms are two rounds of sums over it. Nothing between x and y goes
// through memory but the stream and, for training, four numbers a row. Measured, bf16 with a
// float32 stream: 16384 x 2560, both norms in the root-mean-square form, scale and dropout, forward
// 108 us (4.7 TB/s), backward 189 (4.0 TB/s) and 8 for the sums of the partial rows; 4099 x
// 5120, layer norms with gate, 71, 130 and 8 (4.1 and 3.6 TB/s). float32 throughout, the same
// number of elements as the latter: 8192 x 2560 all options 114, 184 and 8, without biases and gate 69, 136
// and 6 (4.9 and 3.7 TB/s); 2560 x 8192 118, 182 and 9, and 82, 116 and 6. Rows of little more
// than 64 vectors leave most of their second wavefront without work: 80659 x 520 bf16 202, 350
// and 8, where 40960 x 1024 takes 118, 205 and 8.
#include "dropout.h"
#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

// Every kernel is there twice: for all options, and (FULL false) without biases and gate,
// as models with root-mean-square norms have it, which leaves registers for more
// wavefronts.

// A column parameter's values at c .. c + V - 1; none given: `none`.
template <int V>
__device__ __forceinline__ void col_load(float (&v)[V], const float *p, int c, int n, float none) {
    RowRaw<float, V> r;
    if (p) r.load(p + c, n);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = p ? r.get(e) : none;
}

// The bits of columns c .. c + V - 1 (c a multiple of V, 4 or 8), the first one's first.
template <int V>
__device__ __forceinline__ DropBits drop_bits(const DropState &rng, int c, long long row) {
    DropBits b;
    b.set(rng, c, static_cast<uint32_t>(row));
    if (V == 4 && (c & 4)) {
        b.w[0] = b.w[2];
        b.w[1] = b.w[3];
    }
    return b;
}

// T: type of x, z, y. R: type of the stream.
template <typename T, typename R, int NV, bool FULL>
__global__ __launch_bounds__(1024, NV == 1 ? 6 : 5) void block_fwd_kernel(BlockArgs a, int lpr) {
    constexpr int V = vec_of<T>();
    __shared__ float buf[2][16];
    int turn = 0;  // sums take the two buffers in turn (row_sum)
    if (NV > 1) lpr = 0;  // only whole workgroups hold more than a vector per lane
    const RowGroup g = row_group(lpr);
    const int D = a.width, step = (lpr ? lpr : (int)blockDim.x) * V;
    const float inv = 1.0f / static_cast<float>(D);
    const long long stride = (long long)gridDim.x * g.groups;
    const T *x = static_cast<const T *>(a.x), *z = FULL ? static_cast<const T *>(a.z) : nullptr;
    const R *res = static_cast<const R *>(a.residual);
    T *y = static_cast<T *>(a.y);
    R *sum = static_cast<R *>(a.sum);
    DropState rng{};
    if (a.drop.threshold) rng = drop_state(a.drop);
    RowRaw<T, V> xr[NV];
    RowRaw<R, V> rr[NV];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            xr[i].zero();
            if (row < a.rows && n > 0) {
                xr[i].load(x + row * a.x_stride + c, n);
                if (!FULL) rr[i].load(res + row * D + c, n);
            }
        }
    };
    // u - m for the norm's mean m (0 past the row's end), and 1 / deviation
    auto norm = [&](float (&u)[NV][V], float &m) {
        m = 0.0f;
        if (!a.rms) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] += u[i][e];
            row_sum(s, lpr, buf[turn]);
            turn ^= 1;
            m = s[0] * inv;
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = D - (g.lane * V + i * step);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < n) {
                    u[i][e] -= m;
                    q[0] += u[i][e] * u[i][e];
                }
        }
        row_sum(q, lpr, buf[turn]);
        turn ^= 1;
        return 1.0f / sqrtf(q[0] * inv + a.eps);
    };
    long long row = (long long)blockIdx.x * g.groups + g.group;
    constexpr bool AHEAD = NV == 1 && !(FULL && sizeof(R) > sizeof(T));
    if (AHEAD) fetch(row);
    for (; row < a.rows; row += stride) {
        if (!AHEAD) fetch(row);
        float u[NV][V], s[NV][V];
        RowRaw<T, V> zk[NV];
        RowRaw<R, V> rk[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) u[i][e] = xr[i].get(e);
            if (!FULL) rk[i] = rr[i];
            const int c = g.lane * V + i * step, n = D - c;
            if (FULL && n > 0) {  // all options leave no registers to fetch these a row ahead
                rk[i].load(res + row * D + c, n);
                if (z) zk[i].load(z + row * a.z_stride + c, n);
            }
        }
        if (AHEAD) fetch(row + stride);
        if (a.post_weight) {
            float m;
            const float r = norm(u, m);
            if (g.lane == 0) {
                if (a.post_mean && !a.rms) a.post_mean[row] = m;
                if (a.post_rstd) a.post_rstd[row] = r;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = g.lane * V + i * step, n = D - c;
                if (n <= 0) continue;
                float w[V], b[V];
                col_load(w, a.post_weight, c, n, 0.0f);
                col_load(b, FULL ? a.post_bias : nullptr, c, n, 0.0f);
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] = u[i][e] * r * w[e] + b[e];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n <= 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) s[i][e] = 0.0f;
                continue;
            }
            if (a.scale) {
                float k[V];
                col_load(k, a.scale, c, n, 1.0f);
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] *= k[e];
            }
            if (z)
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] *= silu_f32(zk[i].get(e));
            if (a.drop.threshold) {
                const DropBits bits = drop_bits<V>(rng, c, row);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    u[i][e] = bits.keep(e, a.drop.threshold) ? u[i][e] * a.drop.scale : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < V; ++e)  // the next norm reads the stream as it is kept
                s[i][e] = to_f32(from_f32<R>(fmaf(a.beta, u[i][e], a.alpha * rk[i].get(e))));
            row_store(sum + row * D + c, s[i], n);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e >= n) s[i][e] = 0.0f;
        }
        if (!a.weight) continue;
        float m;
        const float r = norm(s, m);
        if (g.lane == 0) {
            if (a.mean && !a.rms) a.mean[row] = m;
            if (a.rstd) a.rstd[row] = r;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n <= 0) continue;
            float w[V], b[V];
            col_load(w, a.weight, c, n, 0.0f);
            col_load(b, FULL ? a.bias : nullptr, c, n, 0.0f);
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] = s[i][e] * r * w[e] + b[e];
            row_store(y + row * D + c, w, n);
        }
    }
}

// A row's lanes in the backward: `lpr` <= 64 of one wavefront (a power of two), or `waves`
// whole wavefronts, of which a workgroup has several sets where that packs better.
// The sums of K values over a row's lanes, in every one of them; buf as in row_sum.
template <int K>
__device__ __forceinline__ void set_sum(float (&v)[K], const BlockSets &s, int set, float (*buf)[K]) {
    lane_sum(v, s.lpr ? s.lpr : 64);
    if (s.lpr || blockDim.x == 64) return;
    if (lane_id() == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[wave_id()][k] = v[k];
    __syncthreads();
    const int w = lane_id() & 15;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = w < s.waves ? buf[set * s.waves + w][k] : 0.0f;
    lane_sum(v, 16);
}

// Lanes of a workgroup at most: with 12 wavefronts to a CU (all options) or 16.
template <typename T, int NV, bool FULL> constexpr int block_bwd_lanes() {
    return FULL && sizeof(T) == 2 ? (NV == 1 ? 768 : 512) : NV == 4 ? 512 : FULL && NV == 2 ? 768 : 1024;
}

// Each set of lanes (for short rows, each workgroup) keeps its columns' four sums in
// registers over its rows and writes them once at its end, those that are wanted:
// part[set][dw2, db2, P, Q][D]. block_sum_kernel adds them up in a fixed order.
template <typename T, typename R, int NV, bool FULL>
__global__ __launch_bounds__((block_bwd_lanes<T, NV, FULL>()), (block_bwd_lanes<T, NV, FULL>() / 256))
void block_bwd_kernel(BlockBwdArgs a, BlockSets sets) {
    constexpr int V = vec_of<T>();
    constexpr bool AHEAD = NV == 1;  // wider rows leave no registers for the next one
    __shared__ float buf[2][16][2];
    __shared__ float acc[NV == 1 ? kShortWaves * V * 64 : 1];
    if (NV > 1) sets.lpr = 0;  // only whole wavefronts hold more than a vector per lane
    const int lpr = sets.lpr, width = lpr ? lpr : 64 * sets.waves;
    const int set = threadIdx.x / width, lane = threadIdx.x - set * width;
    const int D = a.width;
    int step = width * V;
    const float inv = 1.0f / static_cast<float>(D);
    const long long stride = (long long)gridDim.x * sets.sets;
    const T *dy = static_cast<const T *>(a.dy), *x = static_cast<const T *>(a.x);
    const T *z = FULL ? static_cast<const T *>(a.z) : nullptr;
    const R *dsum = static_cast<const R *>(a.dsum), *sum = static_cast<const R *>(a.sum);
    DropState rng{};
    if (a.drop.threshold) rng = drop_state(a.drop);
    float dw[NV][V], db[NV][V], sp[NV][V], sq[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = sp[i][e] = sq[i][e] = 0.0f;
    RowRaw<T, V> yn[NV], xn[NV], zn[NV];
    RowRaw<R, V> sn[NV];
    float m2n = 0.0f, r2n = 0.0f, m1n = 0.0f, r1n = 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        yn[i].zero();
        xn[i].zero();
        zn[i].zero();
        sn[i].zero();
    }
    auto fetch = [&](long long row) {
        if (row >= a.rows) return;
        if (a.weight) {
            m2n = a.mean ? a.mean[row] : 0.0f;
            r2n = a.rstd[row];
        }
        if (a.post_weight) {
            m1n = a.post_mean ? a.post_mean[row] : 0.0f;
            r1n = a.post_rstd[row];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane * V + i * step, n = D - c;
            if (n <= 0) continue;
            if (a.weight) {
                yn[i].load(dy + row * D + c, n);
                sn[i].load(sum + row * D + c, n);
            }
            xn[i].load(x + row * a.x_stride + c, n);
            if (z) zn[i].load(z + row * a.z_stride + c, n);
        }
    };
    int turn = 0;  // sums take the two buffers in turn (row_sum)
    // (the sets of a workgroup go round together: the last rows may be there for some)
    long long row0 = (long long)blockIdx.x * sets.sets;
    if (AHEAD) fetch(row0 + set);
    for (; row0 < a.rows; row0 += stride) {
        const long long row = row0 + set;
        const bool live = row < a.rows;
        if (!AHEAD) {
            asm volatile("" : "+s"(step));  // the offsets anew each row: kept, they spill
            fetch(row);
        }
        RowRaw<T, V> yr[NV], xr[NV], zr[NV];
        RowRaw<R, V> sr[NV], dr[NV];
        const float m1 = m1n, r1 = r1n, m2 = m2n, r2 = r2n;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            yr[i] = yn[i];
            xr[i] = xn[i];
            zr[i] = zn[i];
            sr[i] = sn[i];
            const int c = lane * V + i * step, n = D - c;
            dr[i].zero();
            if (dsum && n > 0 && live) dr[i].load(dsum + row * D + c, n);
        }
        if (AHEAD) fetch(row + stride);
        if (lpr && !live) continue;
        float ds[NV][V];
        if (!a.weight) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) ds[i][e] = dr[i].get(e);
        } else {
            float s[2] = {0.0f, 0.0f};
            // (past the row's end s = 0, but s - m is not)
            auto normal = [&](int i, int e, int n) { return e < n ? (sr[i].get(e) - m2) * r2 : 0.0f; };
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = lane * V + i * step, n = D - c;
                if (n <= 0) continue;
                float w[V];
                col_load(w, a.weight, c, n, 0.0f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = yr[i].get(e), nn = normal(i, e, n), t = d * w[e];
                    if (live) dw[i][e] += d * nn;
                    if (FULL && live) db[i][e] += d;
                    s[0] += t;
                    s[1] += t * nn;
                }
            }
            set_sum(s, sets, set, buf[turn]);
            turn ^= 1;
            const float c0 = a.mean ? s[0] * inv : 0.0f, c1 = s[1] * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = lane * V + i * step, n = D - c;
                if (n <= 0) continue;
                float w[V];
                col_load(w, a.weight, c, n, 0.0f);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    ds[i][e] = dr[i].get(e) + r2 * (yr[i].get(e) * w[e] - c0 - normal(i, e, n) * c1);
            }
        }
        float s[2] = {0.0f, 0.0f};
        // x as it goes into the gate's product: normalised, or itself
        auto inner = [&](int i, int e, int n) { return e < n ? (xr[i].get(e) - m1) * r1 : 0.0f; };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane * V + i * step, n = D - c;
            if (n <= 0) continue;
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                o[e] = a.alpha * ds[i][e];
                ds[i][e] *= a.beta;
            }
            if (live) row_store(static_cast<R *>(a.dresidual) + row * D + c, o, n);
            if (a.drop.threshold) {
                const DropBits bits = drop_bits<V>(rng, c, row);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const bool keep = bits.keep(e, a.drop.threshold);
                    ds[i][e] = keep ? ds[i][e] * a.drop.scale : 0.0f;
                    // (what a dropped element holds is not multiplied by that zero: it may be infinite)
                    if (z) zr[i].clear(e, keep);
                    if (!a.post_weight) xr[i].clear(e, keep);
                }
            }
            float k[V], w[V];
            col_load(k, a.scale, c, n, 1.0f);
            col_load(w, a.post_weight, c, n, 1.0f);
            if (z) {
                float b[V];
                col_load(b, FULL ? a.post_bias : nullptr, c, n, 0.0f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float zv = zr[i].get(e);
                    o[e] = ds[i][e] * (inner(i, e, n) * w[e] + b[e]) * k[e] * silu_grad_f32(zv);
                    ds[i][e] *= silu_f32(zv);
                }
                if (live) row_store(static_cast<T *>(a.dz) + row * D + c, o, n);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float nn = inner(i, e, n);
                if (live) sp[i][e] += ds[i][e] * nn;
                if (FULL && live) sq[i][e] += ds[i][e];
                ds[i][e] *= k[e] * w[e];
                if (e < n) s[0] += ds[i][e];
                s[1] += ds[i][e] * nn;
            }
        }
        float c0 = 0.0f, c1 = 0.0f;
        if (a.post_weight) {
            set_sum(s, sets, set, buf[turn]);
            turn ^= 1;
            c0 = a.post_mean ? s[0] * inv : 0.0f;
            c1 = s[1] * inv;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane * V + i * step, n = D - c;
            if (n <= 0) continue;
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                o[e] = a.post_weight ? r1 * (ds[i][e] - c0 - inner(i, e, n) * c1) : ds[i][e];
            if (live) row_store(static_cast<T *>(a.dx) + row * D + c, o, n);
        }
    }
    float *p = a.part + ((size_t)blockIdx.x * (lpr ? 1 : sets.sets) + (lpr ? 0 : set)) * a.sums * D;
    auto put = [&](float (&v)[NV][V]) {
        if (NV == 1 && lpr) {  // short rows: the groups of a wavefront meet, then the wavefronts
            const int w = wave_id(), l = lane_id();
            for (int off = lpr; off < 64; off <<= 1)
#pragma unroll
                for (int e = 0; e < V; ++e) v[0][e] += __shfl_xor(v[0][e], off);
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) acc[(w * V + e) * 64 + l] = v[0][e];
            __syncthreads();
            if (!w && l < lpr)
#pragma unroll
                for (int e = 0; e < V; ++e)
#pragma unroll
                    for (int k = 1; k < kShortWaves; ++k) v[0][e] += acc[(k * V + e) * 64 + l];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane * V + i * step, n = D - c;
            if (n > 0 && (!lpr || threadIdx.x < (unsigned)lpr)) row_store(p + c, v[i], n);
        }
        p += D;
    };
    if (a.dweight) put(dw);
    if (FULL && a.dbias) put(db);
    if (a.want_p) put(sp);
    if (FULL && a.want_q) put(sq);
}

// Adds up the partial rows, 1024 / COLS strands of them to a column, and makes the
// parameters' gradients of the sums: blockIdx.y 0 the norm before's, 1 what lies after the
// block. 16 columns to a workgroup where there are many rows, else 32. Measured, 16 and 32 columns:
// 768 rows of 2 x 2560 columns 7.6 and 10.9 us, 768 of 4 x 520 10.6 and 17.8; 256 rows of 4 x 5120
// 11.0 and 8.6, of 4 x 8192 13.0 and 9.2, of 2 x 8192 8.7 and 6.1. Between them the columns
// count for more than the rows, which this rule leaves: 512 rows of 4 x 2560 9.2 and 12.8, 501 of
// 2 x 2560 7.3 and 9.4, 256 of 4 x 520 5.1 and 7.5, 64 of 2 x 2560 3.4 both.
template <int COLS> __global__ __launch_bounds__(1024) void block_sum_kernel(BlockBwdArgs a, int rows) {
    constexpr int STRANDS = 1024 / COLS;
    __shared__ float buf[2][16][COLS];
    const int col = threadIdx.x % COLS, strand = threadIdx.x / COLS, D = a.width;
    const int c = blockIdx.x * COLS + col;
    const bool before = blockIdx.y == 0;
    const int pre = (a.dweight != nullptr) + (a.dbias != nullptr);
    const bool one = before ? a.dweight != nullptr : a.want_p, two = before ? a.dbias != nullptr : a.want_q;
    const float *part = a.part + (size_t)(before ? 0 : pre) * D + c;
    float s[2] = {0.0f, 0.0f};
    if (c < D)
#pragma unroll 8
        for (int k = strand; k < rows; k += STRANDS) {
            const float *p = part + (size_t)k * a.sums * D;
            if (one) s[0] += p[0];
            if (two) s[1] += p[one ? D : 0];
        }
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // the strands of a wavefront, then the wavefronts
        if (COLS == 16) {
            const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(s[k]), __float_as_uint(s[k]), false, false);
            s[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        }
        const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(s[k]), __float_as_uint(s[k]), false, false);
        s[k] = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    }
    if (lane_id() < COLS) {
        buf[0][wave_id()][col] = s[0];
        buf[1][wave_id()][col] = s[1];
    }
    __syncthreads();
    if (strand || c >= D) return;
    s[0] = s[1] = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        s[0] += buf[0][k][col];
        s[1] += buf[1][k][col];
    }
    if (before) {
        if (one) a.dweight[c] = s[0];
        if (two) a.dbias[c] = s[1];
        return;
    }
    const float g = a.scale ? a.scale[c] : 1.0f;
    if (a.dpost_weight) a.dpost_weight[c] = g * s[0];
    if (a.dpost_bias) a.dpost_bias[c] = g * s[1];
    if (a.dscale)
        a.dscale[c] = a.post_weight ? a.post_weight[c] * s[0] + (a.post_bias ? a.post_bias[c] * s[1] : 0.0f) : s[0];
}

// Workgroups: as many as run at once, but no more than there are rows for. A SIMD holds
// `waves` wavefronts, and a workgroup's start on the first one.
int block_blocks(long long rows, int sets, int threads, int waves) {
    const long long want = (rows + sets - 1) / sets;
    const int first = (threads / 64 + 3) / 4, resident = 256 * (waves / first > 1 ? waves / first : 1);
    return static_cast<int>(want < resident ? want : resident);
}

template <typename T, typename R, bool FULL> hipError_t block_fwd(const BlockArgs &a, hipStream_t stream) {
    const NormShape s = norm_shape(a.width, vec_of<T>(), 1024);
    const int grid = block_blocks(a.rows, s.groups, s.threads, s.nv == 1 ? 6 : 5);
    if (s.nv == 1) {
        block_fwd_kernel<T, R, 1, FULL><<<grid, s.threads, 0, stream>>>(a, s.lpr);
        return hipGetLastError();
    }
    if constexpr (sizeof(T) == 4)  // 8192 float32 values are two vectors of 4 for 1024 lanes
        if (s.nv == 2) {
            block_fwd_kernel<T, R, 2, FULL><<<grid, s.threads, 0, stream>>>(a, s.lpr);
            return hipGetLastError();
        }
    return hipErrorInvalidValue;
}

// The backward's lanes for rows of D: vectors to a lane, sets of lanes to a workgroup.
struct BlockBwdShape {
    int nv, threads, lanes;  // lanes: of a CU
    BlockSets sets;
};
template <typename T, bool FULL> BlockBwdShape block_bwd_shape(int D) {
    const int nvec = (D + vec_of<T>() - 1) / vec_of<T>();
    BlockBwdShape s;
    s.sets.lpr = 0;
    s.nv = 1;
    s.lanes = FULL && sizeof(T) == 2 ? 768 : 1024;
    if (nvec <= 64) {
        s.sets.lpr = 1;
        while (s.sets.lpr < nvec) s.sets.lpr <<= 1;
        s.threads = 64 * kShortWaves;
        s.sets.waves = 1;
        s.sets.sets = s.threads / s.sets.lpr;
        return s;
    }
    if (nvec > block_bwd_lanes<T, 1, FULL>()) {
        s.nv = 2;
        s.lanes = block_bwd_lanes<T, 2, FULL>();
    }
    if (sizeof(T) == 4 && nvec > 2 * s.lanes) {
        s.nv = 4;
        s.lanes = block_bwd_lanes<T, 4, FULL>();
    }
    const int w = ((nvec + s.nv - 1) / s.nv + 63) / 64;
    s.sets.waves = w;
    // Wavefronts of a workgroup start on the first SIMD: unless they fill all four alike, the
    // first one is full before the others. So sets that do not are put together, as many as
    // the CU holds (16384 rows of 2560, five wavefronts each: 284 us one by one, 185 so). Rows of
    // two wavefronts go one by one, which is not the faster way: back, with the sums of the partial
    // rows, 40960 x 1024 bf16 212 us, together 187, 54613 x 768 261 and 210, 80659 x 520 357 and 273;
    // with gate 20480 x 1024 167 and 138; float32 40960 x 512 160 and 120, with gate 221 and 178.
    s.sets.sets = w % 4 == 0 || w < 3 || s.lanes / (64 * w) < 1 ? 1 : s.lanes / (64 * w);
    s.threads = 64 * w * s.sets.sets;
    return s;
}
int block_bwd_rows(const BlockBwdShape &s, int grid) { return s.sets.lpr ? grid : grid * s.sets.sets; }

template <typename T, typename R, bool FULL> hipError_t block_bwd(const BlockBwdArgs &a, hipStream_t stream) {
    const BlockBwdShape s = block_bwd_shape<T, FULL>(a.width);
    const int grid = block_blocks(a.rows, s.sets.sets, s.threads, s.lanes / 256);
    if (s.nv == 1) block_bwd_kernel<T, R, 1, FULL><<<grid, s.threads, 0, stream>>>(a, s.sets);
    else if (s.nv == 2) {
        if constexpr (sizeof(T) == 4 || FULL) block_bwd_kernel<T, R, 2, FULL><<<grid, s.threads, 0, stream>>>(a, s.sets);
        else return hipErrorInvalidValue;  // 8192 values are one vector of 8 for 1024 lanes
    } else {
        if constexpr (sizeof(T) == 4 && FULL) block_bwd_kernel<T, R, 4, FULL><<<grid, s.threads, 0, stream>>>(a, s.sets);
        else return hipErrorInvalidValue;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.sums == 0) return e;
    const int rows = block_bwd_rows(s, grid), per = rows > 512 ? 16 : 32;
    const dim3 sums((a.width + per - 1) / per, a.want_p || a.want_q ? 2 : 1);
    if (per == 16) block_sum_kernel<16><<<sums, 1024, 0, stream>>>(a, rows);
    else block_sum_kernel<32><<<sums, 1024, 0, stream>>>(a, rows);
    return hipGetLastError();
}

template <typename T, bool FULL> size_t block_part_rows(long long rows, int width) {
    const BlockBwdShape s = block_bwd_shape<T, FULL>(width);
    return block_bwd_rows(s, block_blocks(rows, s.sets.sets, s.threads, s.lanes / 256));
}

}  // namespace

size_t block_bwd_part_bytes(long long rows, int width, bool bf16, bool full, int sums) {
    const size_t n = bf16 ? full ? block_part_rows<bf16_t, true>(rows, width) : block_part_rows<bf16_t, false>(rows, width)
                          : full ? block_part_rows<float, true>(rows, width) : block_part_rows<float, false>(rows, width);
    return n * sums * width * sizeof(float);
}

hipError_t launch_block_fwd(const BlockArgs &a, bool bf16, bool stream_bf16, hipStream_t stream) {
    const bool full = a.z || a.bias || a.post_bias;
    if (!bf16) return full ? block_fwd<float, float, true>(a, stream) : block_fwd<float, float, false>(a, stream);
    if (stream_bf16)
        return full ? block_fwd<bf16_t, bf16_t, true>(a, stream) : block_fwd<bf16_t, bf16_t, false>(a, stream);
    return full ? block_fwd<bf16_t, float, true>(a, stream) : block_fwd<bf16_t, float, false>(a, stream);
}

hipError_t launch_block_bwd(const BlockBwdArgs &a, bool bf16, bool stream_bf16, hipStream_t stream) {
    const bool full = block_bwd_full(a);
    if (!bf16) return full ? block_bwd<float, float, true>(a, stream) : block_bwd<float, float, false>(a, stream);
    if (stream_bf16)
        return full ? block_bwd<bf16_t, bf16_t, true>(a, stream) : block_bwd<bf16_t, bf16_t, false>(a, stream);
    return full ? block_bwd<bf16_t, float, true>(a, stream) : block_bwd<bf16_t, float, false>(a, stream);
}

}  // namespace ssd
