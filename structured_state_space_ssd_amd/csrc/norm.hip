// Normalisation of rows and its gradients: layer norm and its root-mean-square
// form, over x, over the sum of x and a residual stream, or over x gated by
// silu(z). For a row u of D values with mean m (0 in the root-mean-square form):
//   s = 1 / sqrt(mean((u - m)^2) + eps),  n = (u - m) s,  y = n w + b,
//   dn = dy w,  du = s (dn - mean(dn) - n mean(dn n))      (no mean(dn) without m),
//   dw = sum over rows of dy n,  db = sum over rows of dy;
// with the gate, u = x silu(z): dx = du silu(z), dz = du x silu'(z).
//
// Both passes are bound by memory: each tensor is read once and written once.
// A row stays in registers between the sums and the output (the mean is
// subtracted before the squares are summed, so no cancellation), held by a
// group of lanes: the smallest power of two of one wavefront that has a lane
// for every vector of the row, or the whole workgroup for longer rows, whose
// wavefronts meet once through LDS per sum.
//
// Measured where a large copy runs at 4.9 to 5.3 TB/s (read and written): 16384
// rows of 2560 bf16 values with a float32 residual stream, forward 100 us (5.0
// TB/s), backward 132 us (5.1 TB/s) and 5 us for the sum of the partial rows;
// gated, 4099 rows of 5120, forward 33 us (3.8 TB/s) and backward 61 us (3.4
// TB/s): 640 lanes to a row leave a CU two, backward one workgroup, whose
// wavefronts wait for the sums together; 4096 gated rows of 8192 53 and 82 us. Short
// rows: 1048576 of 16 values 15 us forward, 24 + 4 us backward, 65536 of 256 values 16
// and 23 + 4 us. 4 rows of 2560: 3.4 us, a launch.
#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

// Rows are taken with the stride of the grid, which holds as many as run at
// once; the next row sets out while one is worked on, so that its way from
// memory hides behind the sums and their barriers (backward, 16384 rows of 2560:
// 163 us with a grid of all rows, 132 so).
//
// T: type of x, z, y. R: type of the residual stream.
template <typename T, typename R, int NV>
__global__ __launch_bounds__(1024, NV == 1 ? 7 : 4) void norm_fwd_kernel(
    const T *__restrict__ x, size_t x_stride, const R *__restrict__ res,
    const float *__restrict__ weight, const float *__restrict__ bias, const T *__restrict__ z,
    size_t z_stride, long long rows, int D, int lpr, int rms, float eps, T *__restrict__ y,
    R *__restrict__ res_out, float *__restrict__ mean_out, float *__restrict__ rstd_out) {
    constexpr int V = vec_of<T>();
    __shared__ float buf[3][16];
    if (NV > 1) lpr = 0;  // only whole workgroups hold more than a vector per lane
    const RowGroup g = row_group(lpr);
    const int step = (lpr ? lpr : (int)blockDim.x) * V;
    const float inv = 1.0f / static_cast<float>(D);
    const long long stride = (long long)gridDim.x * g.groups;
    RowRaw<T, V> xr[NV], zr[NV];
    RowRaw<R, V> rr[NV];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            xr[i].zero();
            if (row < rows && n > 0) {
                xr[i].load(x + row * x_stride + c, n);
                if (res) rr[i].load(res + row * D + c, n);
                else if (z) zr[i].load(z + row * z_stride + c, n);
            }
        }
    };
    constexpr bool AHEAD = NV * V < 16;  // wider rows leave no registers for it
    long long row = (long long)blockIdx.x * g.groups + g.group;
    if (AHEAD) fetch(row);
    for (int turn = 0; row < rows; row += stride, turn ^= 1) {
        if (!AHEAD) fetch(row);
        float u[NV][V];
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
#pragma unroll
            for (int e = 0; e < V; ++e) u[i][e] = xr[i].get(e);
            if (n <= 0) continue;
            if (res) {
#pragma unroll
                for (int e = 0; e < V; ++e)  // the norm reads the stream as it is kept
                    u[i][e] = to_f32(from_f32<R>(u[i][e] + rr[i].get(e)));
                row_store(res_out + row * D + c, u[i], n);
            } else if (z) {
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] *= silu_f32(zr[i].get(e));
            }
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] += u[i][e];
        }
        if (AHEAD) fetch(row + stride);
        float m = 0.0f;
        if (!rms) {
            row_sum(s, lpr, buf[2]);
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
        const float rstd = 1.0f / sqrtf(q[0] * inv + eps);
        if (g.lane == 0) {
            if (mean_out && !rms) mean_out[row] = m;
            if (rstd_out) rstd_out[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n > 0) {
                RowRaw<float, V> w, b;
                w.load(weight + c, n);
                if (bias) b.load(bias + c, n);
                else b.zero();
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = u[i][e] * rstd * w.get(e) + b.get(e);
                row_store(y + row * D + c, o, n);
            }
        }
    }
}

// Each workgroup (or, for short rows, each group of lanes) keeps its columns'
// dw and db in registers over its rows; a workgroup writes them once at its end;
// colsum_kernel adds the partial rows in their order, so the result does not
// depend on timing. A row's own values stay as they were loaded: what the sums
// need of them is computed again for the output, in the shadow of memory.
// X: type of x (the residual stream's, where there is one).
template <typename T, typename X, int NV, bool GATE>
__global__ __launch_bounds__(NV * vec_of<T>() < 16 ? 1024 : 512, NV == 1 ? 4 : NV == 2 ? 4 : 2) void norm_bwd_kernel(
    const T *__restrict__ dy, const X *__restrict__ x, size_t x_stride,
    const float *__restrict__ weight, const T *__restrict__ z, size_t z_stride,
    const float *__restrict__ mean, const float *__restrict__ rstd, const X *__restrict__ dres,
    long long rows, int D, int lpr, T *__restrict__ dx, X *__restrict__ dres_in,
    T *__restrict__ dz, float *__restrict__ part, int want_db) {
    constexpr int V = vec_of<T>();
    __shared__ float buf[2][32];
    __shared__ float acc[2][NV == 1 ? kShortWaves * V * 64 : 1];
    if (NV > 1) lpr = 0;  // only whole workgroups hold more than a vector per lane
    const RowGroup g = row_group(lpr);
    int step = (lpr ? lpr : (int)blockDim.x) * V;
    const float inv = 1.0f / static_cast<float>(D);
    const long long stride = (long long)gridDim.x * g.groups;
    float dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.0f;
    RowRaw<T, V> yn[NV], zn[NV];
    RowRaw<X, V> xn[NV];
    float mn = 0.0f, rn = 0.0f;
    auto fetch = [&](long long row) {
        if (row >= rows) return;
        mn = mean ? mean[row] : 0.0f;
        rn = rstd[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n > 0) {
                yn[i].load(dy + row * D + c, n);
                xn[i].load(x + row * x_stride + c, n);
                if (GATE) zn[i].load(z + row * z_stride + c, n);
            }
        }
    };
    long long row = (long long)blockIdx.x * g.groups + g.group;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        yn[i].zero();
        xn[i].zero();
        if (GATE) zn[i].zero();
    }
    constexpr bool AHEAD = NV * V < 16;  // wider rows leave no registers for it
    if (AHEAD) fetch(row);
    for (int turn = 0; row < rows; row += stride, turn ^= 1) {
        if (!AHEAD) {
            asm volatile("" : "+s"(step));  // the offsets anew each row: kept, they spill
            fetch(row);
        }
        RowRaw<T, V> yr[NV], zr[NV];
        RowRaw<X, V> xr[NV];
        const float m = mn, r = rn;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            yr[i] = yn[i];
            xr[i] = xn[i];
            if (GATE) zr[i] = zn[i];
        }
        if (AHEAD) fetch(row + stride);
        float s[2] = {0.0f, 0.0f};
        // normalised value and weighted gradient of element e of vector i
        auto normal = [&](int i, int e, int n) {
            float u = xr[i].get(e);
            if (GATE) u *= silu_f32(zr[i].get(e));
            return e < n ? (u - m) * r : 0.0f;  // past the row's end u = 0, but u - m is not
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n <= 0) continue;
            RowRaw<float, V> w;
            w.load(weight + c, n);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = yr[i].get(e), nn = normal(i, e, n), dn = d * w.get(e);
                dw[i][e] += d * nn;
                db[i][e] += d;
                s[0] += dn;
                s[1] += dn * nn;
            }
        }
        RowRaw<X, V> ar[NV];
        if (!GATE && AHEAD && dres)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = g.lane * V + i * step, n = D - c;
                if (n > 0) ar[i].load(dres + row * D + c, n);
            }
        row_sum(s, lpr, buf[turn]);
        const float c0 = mean ? s[0] * inv : 0.0f, c1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n <= 0) continue;
            RowRaw<float, V> w;
            w.load(weight + c, n);
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                o[e] = r * (yr[i].get(e) * w.get(e) - c0 - normal(i, e, n) * c1);
            if (GATE) {
                float oz[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float zv = zr[i].get(e);
                    oz[e] = o[e] * xr[i].get(e) * silu_grad_f32(zv);
                    o[e] *= silu_f32(zv);
                }
                row_store(dz + row * D + c, oz, n);
            } else {
                if (dres) {
                    if (!AHEAD) ar[i].load(dres + row * D + c, n);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += ar[i].get(e);
                }
                if (dres_in) row_store(dres_in + row * D + c, o, n);
            }
            row_store(dx + row * D + c, o, n);
        }
    }
    if (NV == 1 && lpr) {  // short rows: the groups of a wavefront meet, then the wavefronts
        const int w = wave_id(), l = lane_id();
        for (int off = lpr; off < 64; off <<= 1)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                dw[0][e] += __shfl_xor(dw[0][e], off);
                db[0][e] += __shfl_xor(db[0][e], off);
            }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            acc[0][(w * V + e) * 64 + l] = dw[0][e];
            acc[1][(w * V + e) * 64 + l] = db[0][e];
        }
        __syncthreads();
        if (w || l >= lpr) return;
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
            for (int k = 1; k < kShortWaves; ++k) {
                dw[0][e] += acc[0][(k * V + e) * 64 + l];
                db[0][e] += acc[1][(k * V + e) * 64 + l];
            }
    }
    // [workgroup][dw, db][D]
    float *p = part + (size_t)blockIdx.x * (want_db ? 2 : 1) * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = g.lane * V + i * step, n = D - c;
        if (n <= 0) continue;
        row_store(p + c, dw[i], n);
        if (want_db) row_store(p + D + c, db[i], n);
    }
}

// out[c] = sum over k < n of part[k][c]: 1024 / COLS strands of rows to a column,
// added in a fixed order; with several workgroups to a column (blockIdx.y) each
// takes `chunk` rows and leaves a row of its own. 32 columns to a workgroup while that gives each CU two
// workgroups at most, else 64, a wavefront's full width: 768 rows of 5120 columns
// 4.8 us with 32 and 6.0 with 64, 24 rows of 81920 9.2 and 6.1.
template <int COLS>
__global__ __launch_bounds__(1024) void colsum_kernel(const float *__restrict__ part, int n,
                                                      int chunk, long long cols, long long first,
                                                      float *__restrict__ out0,
                                                      float *__restrict__ out1) {
    constexpr int STRANDS = 1024 / COLS;
    __shared__ float buf[STRANDS][COLS];
    const int col = threadIdx.x % COLS, strand = threadIdx.x / COLS;
    const long long c = (long long)blockIdx.x * COLS + col;
    float s = 0.0f;
    const long long end = min((long long)n, (blockIdx.y + 1LL) * chunk);
    if (c < cols)
#pragma unroll 4
        for (long long k = (long long)blockIdx.y * chunk + strand; k < end; k += STRANDS) s += part[k * cols + c];
    buf[strand][col] = s;
    __syncthreads();
    if (strand == 0 && c < cols) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < STRANDS; ++k) s += buf[k][col];
        if (c < first) {
            if (out0) out0[blockIdx.y * cols + c] = s;
        } else if (out1) out1[c - first] = s;
    }
}

NormShape norm_fwd_shape(int D, int V) { return norm_shape(D, V, 1024); }
// The widest rows of the backward (above 8192 values) take half the lanes, which
// then have twice the registers: 1024 lanes of 128 spilled up to 411 of them.
NormShape norm_bwd_shape(int D, int V) {
    const NormShape s = norm_shape(D, V, 1024);
    return s.nv * V < 16 ? s : norm_shape(D, V, 512);
}

// Workgroups: as many as run at once (about 1536 lanes to a CU forward, 1024
// backward, which needs more registers and writes a partial row for each), but
// no more than there are rows for. At 16384 x 2560: forward 106, 99 and 131 us
// with 1024, 1536 and 2048 lanes to a CU (the last do not all fit, and a second
// round begins), backward 145, 132 and 156 us with 640, 1024 and 1280.
int norm_blocks(long long rows, const NormShape &s, int lanes) {
    const long long want = (rows + s.groups - 1) / s.groups;
    const int resident = 256 * (lanes / s.threads > 1 ? lanes / s.threads : 1);
    return static_cast<int>(want < resident ? want : resident);
}
constexpr int kFwdLanes = 1536, kBwdLanes = 1024;

template <typename T, typename R>
hipError_t norm_fwd(const NormArgs &a, hipStream_t stream) {
    const NormShape s = norm_fwd_shape(a.width, vec_of<T>());
    const int grid = norm_blocks(a.rows, s, kFwdLanes);
#define SSD_NORM_FWD(NV)                                                                          \
    norm_fwd_kernel<T, R, NV><<<grid, s.threads, 0, stream>>>(                                    \
        static_cast<const T *>(a.x), a.x_stride, static_cast<const R *>(a.residual), a.weight,    \
        a.bias, static_cast<const T *>(a.z), a.z_stride, a.rows, a.width, s.lpr, a.rms, a.eps,    \
        static_cast<T *>(a.y), static_cast<R *>(a.residual_out), a.mean, a.rstd)
    switch (s.nv) {
        case 1: SSD_NORM_FWD(1); break;
        case 2: SSD_NORM_FWD(2); break;
        case 4:  // float32 only: 16384 values are two vectors of 8 or four of 4 for 1024 lanes
            if constexpr (sizeof(T) == 4) {
                SSD_NORM_FWD(4);
                break;
            }
        default: return hipErrorInvalidValue;
    }
#undef SSD_NORM_FWD
    return hipGetLastError();
}

template <typename T, typename X, bool GATE>
hipError_t norm_bwd(const NormBwdArgs &a, hipStream_t stream) {
    const NormShape s = norm_bwd_shape(a.width, vec_of<T>());
    const int blocks = norm_blocks(a.rows, s, kBwdLanes);
#define SSD_NORM_BWD(NV)                                                                          \
    norm_bwd_kernel<T, X, NV, GATE><<<blocks, s.threads, 0, stream>>>(                            \
        static_cast<const T *>(a.dy), static_cast<const X *>(a.x), a.x_stride, a.weight,          \
        static_cast<const T *>(a.z), a.z_stride, a.mean, a.rstd,                                  \
        static_cast<const X *>(a.dresidual), a.rows, a.width, s.lpr, static_cast<T *>(a.dx),      \
        static_cast<X *>(a.dresidual_in), static_cast<T *>(a.dz), a.part, a.dbias != nullptr)
    constexpr int V = vec_of<T>();  // one vector per lane, float32 two, and the widest rows
    switch (s.nv) {
        case 1: SSD_NORM_BWD(1); break;
        case 2:
            if constexpr (V == 4) {
                SSD_NORM_BWD(2);
                break;
            }
            return hipErrorInvalidValue;
        case 32 / V: SSD_NORM_BWD(32 / V); break;
        default: return hipErrorInvalidValue;
    }
#undef SSD_NORM_BWD
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long cols = (long long)a.width * (a.dbias ? 2 : 1);
    return launch_colsum(a.part, blocks, cols, a.width, a.dweight, a.dbias, stream);
}

}  // namespace

// Columns of a workgroup in a sum's only or last pass.
static int colsum_cols(long long cols) { return cols <= 16384 ? 32 : 64; }

bool colsum_grid_ok(int n, long long cols, bool spare) {
    const auto fits = [&](int per) { return (cols + per - 1) / per < (1LL << 32) / 1024; };
    return fits(colsum_cols(cols)) && (!spare || n <= kColsumRows || fits(32));
}

hipError_t launch_colsum(const float *part, int n, long long cols, long long first, float *out0,
                         float *out1, hipStream_t stream, float *spare) {
    const auto grid = [&](int per) { return static_cast<unsigned>((cols + per - 1) / per); };
    if (spare && n > kColsumRows) {
        const int chunk = (n + kColsumChunks - 1) / kColsumChunks;
        colsum_kernel<32><<<dim3(grid(32), kColsumChunks), 1024, 0, stream>>>(part, n, chunk, cols,
                                                                              cols, spare, nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        part = spare;
        n = kColsumChunks;
    }
    if (colsum_cols(cols) == 32)
        colsum_kernel<32><<<grid(32), 1024, 0, stream>>>(part, n, n, cols, first, out0, out1);
    else colsum_kernel<64><<<grid(64), 1024, 0, stream>>>(part, n, n, cols, first, out0, out1);
    return hipGetLastError();
}

size_t norm_bwd_part_bytes(long long rows, int width, bool bf16, bool want_db) {
    const NormShape s = norm_bwd_shape(width, bf16 ? 8 : 4);
    return (size_t)norm_blocks(rows, s, kBwdLanes) * (want_db ? 2 : 1) * width * sizeof(float);
}

hipError_t launch_norm_fwd(const NormArgs &a, bool bf16, bool res_bf16, hipStream_t stream) {
    if (!bf16) return norm_fwd<float, float>(a, stream);
    return a.residual && !res_bf16 ? norm_fwd<bf16_t, float>(a, stream)
                                   : norm_fwd<bf16_t, bf16_t>(a, stream);
}

hipError_t launch_norm_bwd(const NormBwdArgs &a, bool bf16, bool x_bf16, hipStream_t stream) {
    // The gate and the residual stream exclude each other, so a gated x has z's type.
    if (a.z)
        return bf16 ? norm_bwd<bf16_t, bf16_t, true>(a, stream)
                    : norm_bwd<float, float, true>(a, stream);
    if (!bf16) return norm_bwd<float, float, false>(a, stream);
    return x_bf16 ? norm_bwd<bf16_t, bf16_t, false>(a, stream)
                  : norm_bwd<bf16_t, float, false>(a, stream);
}

}  // namespace ssd
