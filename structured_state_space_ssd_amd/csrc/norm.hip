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
#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

// Lanes that share a row, as the kernels see it: `lpr` <= 64 lanes of one
// wavefront (a power of two), or the workgroup (lpr = 0).
struct RowGroup {
    int lpr, lane, group, groups;
};
__device__ __forceinline__ RowGroup row_group(int lpr) {
    RowGroup r;
    r.lpr = lpr;
    if (lpr) {
        r.lane = threadIdx.x & (lpr - 1);
        r.group = threadIdx.x / lpr;
        r.groups = blockDim.x / lpr;
    } else {
        r.lane = threadIdx.x;
        r.group = 0;
        r.groups = 1;
    }
    return r;
}

// Sums of K values over the lanes of a row, in every one of them. `buf` holds
// K floats per wavefront; the caller alternates between two of them, so that
// one barrier per sum is enough (a wavefront can write a buffer again only
// after it has passed the barrier of the other one).
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int lpr, float *buf) {
    const int top = lpr ? lpr : 64;
    for (int off = 1; off < top; off <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], off);
    const int waves = blockDim.x >> 6;
    if (lpr || waves == 1) return;
    if (lane_id() == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[wave_id() * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
    for (int w = 0; w < waves; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += buf[w * K + k];
}

template <typename T> constexpr int vec_of() { return sizeof(T) == 2 ? 8 : 4; }

// T: type of x, z, y. R: type of the residual stream (RES).
template <typename T, typename R, int NV>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(
    const T *__restrict__ x, size_t x_stride, const R *__restrict__ res,
    const float *__restrict__ weight, const float *__restrict__ bias, const T *__restrict__ z,
    size_t z_stride, long long rows, int D, int lpr, int rms, float eps, T *__restrict__ y,
    R *__restrict__ res_out, float *__restrict__ mean_out, float *__restrict__ rstd_out) {
    constexpr int V = vec_of<T>();
    __shared__ float buf[3][16];
    const RowGroup g = row_group(lpr);
    const int step = (lpr ? lpr : (int)blockDim.x) * V;
    const float inv = 1.0f / static_cast<float>(D);
    int turn = 0;
    for (long long row = (long long)blockIdx.x * g.groups + g.group; row < rows;
         row += (long long)gridDim.x * g.groups, turn ^= 1) {
        const T *xr = x + row * x_stride;
        float u[NV][V];
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n > 0) {
                RowRaw<T, V> a;
                a.load(xr + c, n);
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] = a.get(e);
                if (res) {
                    RowRaw<R, V> b;
                    b.load(res + row * D + c, n);
#pragma unroll
                    for (int e = 0; e < V; ++e)  // the norm reads the stream as it is kept
                        u[i][e] = to_f32(from_f32<R>(u[i][e] + b.get(e)));
                    row_store(res_out + row * D + c, u[i], n);
                } else if (z) {
                    RowRaw<T, V> b;
                    b.load(z + row * z_stride + c, n);
#pragma unroll
                    for (int e = 0; e < V; ++e) u[i][e] *= silu_f32(b.get(e));
                }
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] += u[i][e];
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] = 0.0f;
            }
        }
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

// Each workgroup (or, for short rows, each group of lanes) takes rows with a
// stride of the grid and keeps its columns' dw and db in registers; it writes
// them once at its end, and colsum_kernel adds the partial rows in their
// order, so the result does not depend on timing.
// X: type of x (the residual stream's, where there is one).
template <typename T, typename X, int NV>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(
    const T *__restrict__ dy, const X *__restrict__ x, size_t x_stride,
    const float *__restrict__ weight, const T *__restrict__ z, size_t z_stride,
    const float *__restrict__ mean, const float *__restrict__ rstd, const X *__restrict__ dres,
    long long rows, int D, int lpr, T *__restrict__ dx, X *__restrict__ dres_in,
    T *__restrict__ dz, float *__restrict__ part, int want_db) {
    constexpr int V = vec_of<T>();
    __shared__ float buf[2][32];
    const RowGroup g = row_group(lpr);
    const int step = (lpr ? lpr : (int)blockDim.x) * V;
    const float inv = 1.0f / static_cast<float>(D);
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = g.lane * V + i * step, n = D - c;
        RowRaw<float, V> a;
        a.zero();
        if (n > 0) a.load(weight + c, n);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[i][e] = a.get(e);
            dw[i][e] = db[i][e] = 0.0f;
        }
    }
    int turn = 0;
    for (long long row = (long long)blockIdx.x * g.groups + g.group; row < rows;
         row += (long long)gridDim.x * g.groups, turn ^= 1) {
        const float m = mean ? mean[row] : 0.0f, r = rstd[row];
        float n_[NV][V], dn[NV][V];
        RowRaw<X, V> xr[NV];
        RowRaw<T, V> zr[NV];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            RowRaw<T, V> a;
            a.zero();
            xr[i].zero();
            zr[i].zero();
            if (n > 0) {
                a.load(dy + row * D + c, n);
                xr[i].load(x + row * x_stride + c, n);
                if (z) zr[i].load(z + row * z_stride + c, n);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float u = xr[i].get(e);
                if (z) u *= silu_f32(zr[i].get(e));
                const float d = a.get(e);
                // past the row's end u = 0, but u - m is not
                const float nn = e < n ? (u - m) * r : 0.0f;
                n_[i][e] = nn;
                dw[i][e] += d * nn;
                db[i][e] += d;
                dn[i][e] = d * w[i][e];
                s[0] += dn[i][e];
                s[1] += dn[i][e] * nn;
            }
        }
        row_sum(s, lpr, buf[turn]);
        const float c0 = mean ? s[0] * inv : 0.0f, c1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.lane * V + i * step, n = D - c;
            if (n <= 0) continue;
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = r * (dn[i][e] - c0 - n_[i][e] * c1);
            if (z) {
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
                    RowRaw<X, V> a;
                    a.load(dres + row * D + c, n);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += a.get(e);
                }
                if (dres_in) row_store(dres_in + row * D + c, o, n);
            }
            row_store(dx + row * D + c, o, n);
        }
    }
    // [partial row][dw, db][D]
    float *p = part + ((size_t)blockIdx.x * g.groups + g.group) * (want_db ? 2 : 1) * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = g.lane * V + i * step, n = D - c;
        if (n <= 0) continue;
        row_store(p + c, dw[i], n);
        if (want_db) row_store(p + D + c, db[i], n);
    }
}

// out[c] = sum over k < n of part[k][c]: 64 columns per workgroup, 16 strands
// of rows each, added in a fixed order.
__global__ __launch_bounds__(1024) void colsum_kernel(const float *__restrict__ part, int n,
                                                      long long cols, long long first,
                                                      float *__restrict__ out0,
                                                      float *__restrict__ out1) {
    __shared__ float acc[16][64];
    const int l = threadIdx.x & 63, strand = threadIdx.x >> 6;
    const long long c = (long long)blockIdx.x * 64 + l;
    float a = 0.0f, b = 0.0f;
    if (c < cols) {
        int k = strand;
        for (; k + 16 < n; k += 32) {
            a += part[(size_t)k * cols + c];
            b += part[(size_t)(k + 16) * cols + c];
        }
        if (k < n) a += part[(size_t)k * cols + c];
    }
    acc[strand][l] = a + b;
    __syncthreads();
    if (strand == 0 && c < cols) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += acc[k][l];
        if (c < first) {
            if (out0) out0[c] = s;
        } else if (out1) out1[c - first] = s;
    }
}

struct NormShape {
    int lpr, threads, nv, groups;
};
// One vector per lane where the row allows it: more lanes per row keep more
// loads in flight than more vectors per lane do. `most`: lanes of a workgroup
// that a row may take.
NormShape norm_shape(int D, int V, int most) {
    const int nvec = (D + V - 1) / V;
    NormShape s;
    if (nvec <= 64) {
        s.lpr = 1;
        while (s.lpr < nvec) s.lpr <<= 1;
        s.threads = 256;
        s.nv = 1;
        s.groups = 256 / s.lpr;
        return s;
    }
    s.lpr = 0;
    s.groups = 1;
    s.nv = 1;
    while ((nvec + s.nv - 1) / s.nv > most) s.nv *= 2;
    s.threads = ((nvec + s.nv - 1) / s.nv + 63) / 64 * 64;
    return s;
}
constexpr int kNormLanes = 1024;

// Workgroups of the backward: as many as stay resident (2048 lanes per CU at
// most), but no more than there are rows for, so that few partial rows are
// written and added up.
int norm_bwd_blocks(long long rows, const NormShape &s) {
    const long long want = (rows + s.groups - 1) / s.groups;
    const int resident = 256 * (1024 / s.threads > 4 ? 4 : 1024 / s.threads);
    return static_cast<int>(want < resident ? want : resident);
}

template <typename T, typename R>
hipError_t norm_fwd(const NormArgs &a, hipStream_t stream) {
    const NormShape s = norm_shape(a.width, vec_of<T>(), kNormLanes);
    const long long want = (a.rows + s.groups - 1) / s.groups;
    const dim3 grid(static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20)));
#define SSD_NORM_FWD(NV)                                                                          \
    norm_fwd_kernel<T, R, NV><<<grid, s.threads, 0, stream>>>(                                    \
        static_cast<const T *>(a.x), a.x_stride, static_cast<const R *>(a.residual), a.weight,    \
        a.bias, static_cast<const T *>(a.z), a.z_stride, a.rows, a.width, s.lpr, a.rms, a.eps,    \
        static_cast<T *>(a.y), static_cast<R *>(a.residual_out), a.mean, a.rstd)
    switch (s.nv) {
        case 1: SSD_NORM_FWD(1); break;
        case 2: SSD_NORM_FWD(2); break;
        case 4: SSD_NORM_FWD(4); break;
        default: return hipErrorInvalidValue;
    }
#undef SSD_NORM_FWD
    return hipGetLastError();
}

template <typename T, typename X>
hipError_t norm_bwd(const NormBwdArgs &a, hipStream_t stream) {
    const NormShape s = norm_shape(a.width, vec_of<T>(), kNormLanes);
    const int blocks = norm_bwd_blocks(a.rows, s);
#define SSD_NORM_BWD(NV)                                                                          \
    norm_bwd_kernel<T, X, NV><<<blocks, s.threads, 0, stream>>>(                                  \
        static_cast<const T *>(a.dy), static_cast<const X *>(a.x), a.x_stride, a.weight,          \
        static_cast<const T *>(a.z), a.z_stride, a.mean, a.rstd,                                  \
        static_cast<const X *>(a.dresidual), a.rows, a.width, s.lpr, static_cast<T *>(a.dx),      \
        static_cast<X *>(a.dresidual_in), static_cast<T *>(a.dz), a.part, a.dbias != nullptr)
    switch (s.nv) {
        case 1: SSD_NORM_BWD(1); break;
        case 2: SSD_NORM_BWD(2); break;
        case 4: SSD_NORM_BWD(4); break;
        default: return hipErrorInvalidValue;
    }
#undef SSD_NORM_BWD
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long cols = (long long)a.width * (a.dbias ? 2 : 1);
    return launch_colsum(a.part, blocks * s.groups, cols, a.width, a.dweight, a.dbias, stream);
}

}  // namespace

hipError_t launch_colsum(const float *part, int n, long long cols, long long first, float *out0,
                         float *out1, hipStream_t stream) {
    colsum_kernel<<<static_cast<unsigned>((cols + 63) / 64), 1024, 0, stream>>>(part, n, cols,
                                                                                 first, out0, out1);
    return hipGetLastError();
}

size_t norm_bwd_part_bytes(long long rows, int width, bool bf16, bool want_db) {
    const NormShape s = norm_shape(width, bf16 ? 8 : 4, kNormLanes);
    return (size_t)norm_bwd_blocks(rows, s) * s.groups * (want_db ? 2 : 1) * width * sizeof(float);
}

hipError_t launch_norm_fwd(const NormArgs &a, bool bf16, bool res_bf16, hipStream_t stream) {
    if (!bf16) return norm_fwd<float, float>(a, stream);
    return a.residual && !res_bf16 ? norm_fwd<bf16_t, float>(a, stream)
                                   : norm_fwd<bf16_t, bf16_t>(a, stream);
}

hipError_t launch_norm_bwd(const NormBwdArgs &a, bool bf16, bool x_bf16, hipStream_t stream) {
    if (!bf16) return norm_bwd<float, float>(a, stream);
    return x_bf16 ? norm_bwd<bf16_t, bf16_t>(a, stream) : norm_bwd<bf16_t, float>(a, stream);
}

}  // namespace ssd
