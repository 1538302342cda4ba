// Short causal convolution along the token axis, one filter of W = 2, 3 or 4
// taps per channel, with an optional SiLU:
//   v_t = b + sum_{k < W} w_k x_{t-W+1+k},   y_t = v_t or v_t sigmoid(v_t),
// where tokens before the first come from a state of W-1 rows (or are zero),
// its gradients and its step for single tokens ("Mamba-2架构深度解析", section
// 2.1, puts a short convolution before the state-space layer).
//
// Bound by memory (2W operations per element read and written). A lane owns
// a vector of four channels and walks a tile of tokens with the last W-1 rows in
// registers, so each row is read once per tile and W-1 rows more (its halo);
// consecutive lanes own consecutive vectors, so a wavefront reads 512 bytes or
// more of a row at once. Eight channels to a lane (16-byte loads in bf16) took
// 81 us where four take 72: twice the registers, half the wavefronts.
//
// Measured in bf16 with W = 4 where a large copy runs at 4.9 to 5.3 TB/s: 16384
// tokens of 5248 channels 72 us (4.8 TB/s), as 55 packed sequences 75 us,
// backward 132 us (3.9 TB/s) and 5 us for the sum of the partial rows; one
// token for 256 sequences of 7168 channels 8.7 us (3.4 TB/s). Float32, W = 3,
// 3 x 1021 tokens of 1312 channels: 8.8 us forward, 13.8 + 4.0 us backward.
#include <type_traits>

#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

// Vectors of V channels never straddle two parts of the channel axis.
struct PartVec {
    int part, count, col, chan, n;  // part, its width, first column in it, first channel, elements
};
template <int V> __device__ __forceinline__ PartVec part_vec(const ConvParts &p, int v) {
    PartVec r;
    r.part = 0;
    while (r.part + 1 < p.n) {
        const int nv = (p.count[r.part] + V - 1) / V;
        if (v < nv) break;
        v -= nv;
        ++r.part;
    }
    r.count = r.part == 0 ? p.count[0] : r.part == 1 ? p.count[1] : p.count[2];
    const int first = r.part == 0 ? p.first[0] : r.part == 1 ? p.first[1] : p.first[2];
    r.col = v * V;
    r.chan = first + r.col;
    r.n = r.count - r.col;
    return r;
}
int part_vecs(const ConvParts &p, int V) {
    int s = 0;
    for (int i = 0; i < p.n; ++i) s += (p.count[i] + V - 1) / V;
    return s;
}
// The part's tensor and row length.
template <typename T> __device__ __forceinline__ T *part_row(const ConvParts &p, int part, size_t row) {
    T *base = static_cast<T *>(part == 0 ? p.ptr[0] : part == 1 ? p.ptr[1] : p.ptr[2]);
    return base + row * (part == 0 ? p.count[0] : part == 1 ? p.count[1] : p.count[2]);
}

// The filters of n channels, tap by tap (a full vector's V * W weights are contiguous).
template <int V, int W>
__device__ __forceinline__ void load_filter(const float *weight, const float *bias, int chan, int n,
                                            float (&w)[W][V], float (&b)[V]) {
    RowRaw<float, V * W> r;
    RowRaw<float, V> rb;
    r.load(weight + (size_t)chan * W, n >= V ? V * W : n * W);
    if (bias) rb.load(bias + chan, n);
    else rb.zero();
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][e] = r.get(e * W + k);
        b[e] = rb.get(e);
    }
}

// The sequence that token t lies in: the last s with cu[s] <= t. Any contents
// of cu give an index in [0, nseq).
__device__ __forceinline__ int find_seq(const int *cu, int nseq, int t) {
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Items: (tile of T tokens, vector), vectors fastest, then (sequence, vector)
// for the states after each sequence.
template <typename T, int V, int W, int U>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int nvec, int tile, int tiles,
                                                       long long walks, long long items) {
    const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
    if (item >= items) return;
    const T *x = static_cast<const T *>(a.x), *init = static_cast<const T *>(a.init);
    const int K = a.channels, L = a.seqlen;
    if (item >= walks) {
        // the last W-1 rows of a sequence, in front of it its initial state's (or zeros)
        const long long q = item - walks;
        const int seq = static_cast<int>(q / nvec);
        const PartVec pv = part_vec<V>(a.y, static_cast<int>(q % nvec));
        int begin = 0, end = L, b = seq;
        if (a.cu_seqlens) {
            begin = a.cu_seqlens[seq];
            end = a.cu_seqlens[seq + 1];
            b = 0;
        }
        T *out = static_cast<T *>(a.final_state) + (size_t)seq * (W - 1) * K + pv.chan;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long t = (long long)end - (W - 1) + j;
            RowRaw<T, V> r;
            r.zero();
            if (t >= begin && t >= 0 && t < L)
                r.load(x + (size_t)b * a.x_batch + (size_t)t * a.x_row + pv.chan, pv.n);
            else if (t < begin && init && t - begin + (W - 1) >= 0)
                r.load(init + ((size_t)b * (W - 1) + (t - begin + (W - 1))) * K + pv.chan, pv.n);
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = r.get(e);
            row_store(out + (size_t)j * K, v, pv.n);
        }
        return;
    }
    const PartVec pv = part_vec<V>(a.y, static_cast<int>(item % nvec));
    const long long ti = item / nvec;
    const int b = static_cast<int>(ti / tiles), t0 = static_cast<int>(ti % tiles) * tile;
    const int t1 = min(t0 + tile, L);
    const T *xp = x + (size_t)b * a.x_batch + pv.chan;
    float w[W][V], bias[V], win[W - 1][V];
    load_filter<V, W>(a.weight, a.bias, pv.chan, pv.n, w, bias);
    int begin = 0, next = 0x7fffffff, seq = 0;
    if (a.cu_seqlens) {
        seq = find_seq(a.cu_seqlens, a.nseq, t0);
        begin = a.cu_seqlens[seq];
        next = a.cu_seqlens[seq + 1];
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int t = t0 - (W - 1) + j;
        RowRaw<T, V> r;
        r.zero();
        if (t >= begin && t >= 0) r.load(xp + (size_t)t * a.x_row, pv.n);
        else if (t < 0 && init) r.load(init + ((size_t)b * (W - 1) + (t + W - 1)) * K + pv.chan, pv.n);
#pragma unroll
        for (int e = 0; e < V; ++e) win[j][e] = r.get(e);
    }
    // U tokens: their rows are fetched together, so U loads are in flight per lane.
    // `whole`: all of them are in this tile and this sequence and the vector is full,
    // so nothing is checked row by row.
    auto rows = [&](int t, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        RowRaw<T, V> raw[U];
        const T *from = xp + (size_t)t * a.x_row;
#pragma unroll
        for (int u = 0; u < U; ++u, from += a.x_row)
            if constexpr (WHOLE) raw[u].load(from);
            else if (t + u < t1) raw[u].load(from, pv.n);
            else raw[u].zero();
        T *to = part_row<T>(a.y, pv.part, (size_t)b * L + t) + pv.col;
#pragma unroll
        for (int u = 0; u < U; ++u, to += pv.count) {
            if (!WHOLE && t + u >= t1) break;
            if (!WHOLE && t + u >= next) {
                // a new sequence: nothing before it is seen
                while (seq + 1 < a.nseq && a.cu_seqlens[seq + 1] <= t + u) ++seq;
                next = seq + 1 < a.nseq ? a.cu_seqlens[seq + 1] : 0x7fffffff;
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) win[j][e] = 0.0f;
            }
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xv = raw[u].get(e);
                float v = bias[e];
#pragma unroll
                for (int k = 0; k < W - 1; ++k) v = fmaf(w[k][e], win[k][e], v);
                v = fmaf(w[W - 1][e], xv, v);
#pragma unroll
                for (int k = 0; k + 1 < W - 1; ++k) win[k][e] = win[k + 1][e];
                win[W - 2][e] = xv;
                o[e] = a.silu ? silu_f32(v) : v;
            }
            row_store(to, o, WHOLE ? V : pv.n);
        }
    };
    for (int t = t0; t < t1; t += U)
        if (pv.n >= V && t + U <= t1 && t + U <= next) rows(t, std::true_type());
        else rows(t, std::false_type());
}

// Gradients. With g_t = dy_t silu'(v_t) (v recomputed):
//   dx_t = sum_k w_k g_{t+W-1-k},   dw_k = sum_t g_t x_{t-W+1+k},   db = sum_t g_t.
// A lane walks its tile's tokens and W-1 more, since dx_t needs the g of the
// W-1 tokens after t; dw and db take only the tile's own tokens. The first
// tile starts W-1 rows early, in the initial state. Partial sums go to
// part[tile][W + 1][K], added up in order by colsum.
template <typename T, int V, int W>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvBwdArgs a, int nvec, int tile, int tiles,
                                                       long long items) {
    const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
    if (item >= items) return;
    const T *x = static_cast<const T *>(a.x), *init = static_cast<const T *>(a.init);
    const T *dfinal = static_cast<const T *>(a.dfinal);
    T *dx = static_cast<T *>(a.dx), *dinit = static_cast<T *>(a.dinit);
    const int K = a.channels, L = a.seqlen;
    const PartVec pv = part_vec<V>(a.dy, static_cast<int>(item % nvec));
    const long long ti = item / nvec;
    const int b = static_cast<int>(ti / tiles), t0 = static_cast<int>(ti % tiles) * tile;
    const int t1 = min(t0 + tile, L);
    const T *xp = x + (size_t)b * a.x_batch + pv.chan;
    float w[W][V], bias[V], win[W - 1][V], g[W - 1][V], dw[W][V], db[V];
    load_filter<V, W>(a.weight, a.bias, pv.chan, pv.n, w, bias);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) g[k][e] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int t = t0 - (W - 1) + j;
        RowRaw<T, V> r;
        r.zero();
        if (t >= 0) r.load(xp + (size_t)t * a.x_row, pv.n);
        else if (init) r.load(init + ((size_t)b * (W - 1) + (t + W - 1)) * K + pv.chan, pv.n);
#pragma unroll
        for (int e = 0; e < V; ++e) win[j][e] = r.get(e);
    }
    // tokens fetched together: 2, 4 and 8 took 150, 137 and 153 us at the size above
    constexpr int U = 4;
    const int last = t1 + W - 1;  // one past the last token whose g a row of dx here needs
    // `whole`: these tokens are the tile's own (so the rows of dx they write lie
    // before those that take a gradient of the final state) and the vector is full:
    // little is checked row by row.
    auto rows = [&](int t, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        RowRaw<T, V> xr[U], dr[U];
        const T *from = xp + (size_t)t * a.x_row;
        const T *grad = part_row<const T>(a.dy, pv.part, (size_t)b * L + t) + pv.col;
#pragma unroll
        for (int u = 0; u < U; ++u, from += a.x_row, grad += pv.count) {
            if constexpr (WHOLE) {
                xr[u].load(from);
                dr[u].load(grad);
            } else {
                xr[u].zero();
                dr[u].zero();
                if (t + u < last && t + u < L) {
                    xr[u].load(from, pv.n);
                    dr[u].load(grad, pv.n);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = t + u;
            if (!WHOLE && j >= last) break;
            const bool own = WHOLE || j < t1;
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xv = xr[u].get(e);
                float v = bias[e];
#pragma unroll
                for (int k = 0; k < W - 1; ++k) v = fmaf(w[k][e], win[k][e], v);
                v = fmaf(w[W - 1][e], xv, v);
                float gv = dr[u].get(e);
                if (a.silu) gv *= silu_grad_f32(v);
                if (!WHOLE && j >= L) gv = 0.0f;  // past the last token, whatever v is
                if (own) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) dw[k][e] = fmaf(gv, win[k][e], dw[k][e]);
                    dw[W - 1][e] = fmaf(gv, xv, dw[W - 1][e]);
                    db[e] += gv;
                }
                // g[i] holds the gradient of token j - (W-1) + i
                float d = w[0][e] * gv;
#pragma unroll
                for (int i = 0; i < W - 1; ++i) d = fmaf(w[W - 1 - i][e], g[i][e], d);
                o[e] = d;
#pragma unroll
                for (int k = 0; k + 1 < W - 1; ++k) {
                    win[k][e] = win[k + 1][e];
                    g[k][e] = g[k + 1][e];
                }
                win[W - 2][e] = xv;
                g[W - 2][e] = gv;
            }
            const int t_out = j - (W - 1);  // token of this row of dx
            if (t_out < t0 && t0 > 0) continue;  // the tile before has it
            if (!WHOLE && dfinal && t_out >= L - (W - 1)) {
                RowRaw<T, V> r;
                r.load(dfinal + ((size_t)b * (W - 1) + (t_out - (L - (W - 1)))) * K + pv.chan, pv.n);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] += r.get(e);
            }
            if (t_out >= 0)
                row_store(dx + ((size_t)b * L + t_out) * K + pv.chan, o, WHOLE ? V : pv.n);
            else if (dinit)
                row_store(dinit + ((size_t)b * (W - 1) + (t_out + W - 1)) * K + pv.chan, o, pv.n);
        }
    };
    for (int t = t0; t < last; t += U)
        if (pv.n >= V && t + U <= t1) rows(t, std::true_type());
        else rows(t, std::false_type());
    // dweight's own layout [K][W], then the bias's [K]
    float *p = a.part + (size_t)ti * (W + 1) * K;
    float flat[V * W];
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
        for (int k = 0; k < W; ++k) flat[e * W + k] = dw[k][e];
    row_store(p + (size_t)pv.chan * W, flat, pv.n >= V ? V * W : pv.n * W);
    row_store(p + (size_t)W * K + pv.chan, db, pv.n);
}

// One token: the state's rows move up by one and the token's input becomes the last.
template <typename T, int V, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(T *__restrict__ state,
                                                        const T *__restrict__ x, size_t x_row,
                                                        const float *__restrict__ weight,
                                                        const float *__restrict__ bias_, int K,
                                                        int silu, ConvParts y, int nvec,
                                                        long long items) {
    const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
    if (item >= items) return;
    const PartVec pv = part_vec<V>(y, static_cast<int>(item % nvec));
    const size_t b = static_cast<size_t>(item / nvec);
    T *st = state + b * (W - 1) * K + pv.chan;
    RowRaw<T, V> r[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j].load(st + (size_t)j * K, pv.n);
    r[W - 1].load(x + b * x_row + pv.chan, pv.n);
    float w[W][V], bias[V], o[V];
    load_filter<V, W>(weight, bias_, pv.chan, pv.n, w, bias);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float v = bias[e];
#pragma unroll
        for (int k = 0; k < W; ++k) v = fmaf(w[k][e], r[k].get(e), v);
        o[e] = silu ? silu_f32(v) : v;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = r[j + 1].get(e);
        row_store(st + (size_t)j * K, v, pv.n);
    }
    row_store(part_row<T>(y, pv.part, b) + pv.col, o, pv.n);
}

// Measured at 16384 tokens x 5248 channels: forward 73, 75 and 78 us with tiles
// of 16, 32 and 64 tokens; backward 146, 137 and 132 us with 32, 64 and 128 (of
// which 12, 6 and 5 us more go to the partial sums).
constexpr int kFwdTile = 16, kFwdTileMin = 8;
constexpr int kBwdTile = 128, kBwdTileMin = 8;

// Tokens per tile: long tiles read fewer halo rows (and, backward, write fewer
// partial sums), short ones give every CU work; the longest power of two that
// still leaves `want` lanes.
int tile_of(int batch, int seqlen, int nvec, int most, int least, long long want) {
    int t = most;
    while (t > least && (long long)batch * ((seqlen + t - 1) / t) * nvec < want) t /= 2;
    return t;
}
constexpr long long kFwdLanes = 256LL * 2048 / 2, kBwdLanes = 256LL * 512;

int bwd_tile(int batch, int seqlen, int channels) {
    return tile_of(batch, seqlen, (channels + 3) / 4, kBwdTile, kBwdTileMin, kBwdLanes);
}

template <typename T>
hipError_t conv_fwd(const ConvArgs &a, hipStream_t stream) {
    constexpr int V = 4, U = 8;
    const int nvec = part_vecs(a.y, V);
    const int tile = tile_of(a.batch, a.seqlen, nvec, kFwdTile, kFwdTileMin, kFwdLanes);
    const int tiles = (a.seqlen + tile - 1) / tile;
    const long long walks = (long long)a.batch * tiles * nvec;
    const long long items =
        walks + (a.final_state ? (long long)(a.cu_seqlens ? a.nseq : a.batch) * nvec : 0);
    const long long blocks = (items + 255) / 256;
    if (blocks >= (1LL << 24)) return hipErrorNotSupported;
    const dim3 grid(static_cast<unsigned>(blocks));
    switch (a.width) {
        case 2: conv_fwd_kernel<T, V, 2, U><<<grid, 256, 0, stream>>>(a, nvec, tile, tiles, walks, items); break;
        case 3: conv_fwd_kernel<T, V, 3, U><<<grid, 256, 0, stream>>>(a, nvec, tile, tiles, walks, items); break;
        case 4: conv_fwd_kernel<T, V, 4, U><<<grid, 256, 0, stream>>>(a, nvec, tile, tiles, walks, items); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <typename T>
hipError_t conv_bwd(const ConvBwdArgs &a, hipStream_t stream) {
    constexpr int V = 4;
    const int nvec = part_vecs(a.dy, V);
    const int tile = bwd_tile(a.batch, a.seqlen, a.channels);
    const int tiles = (a.seqlen + tile - 1) / tile;
    const long long items = (long long)a.batch * tiles * nvec;
    const long long blocks = (items + 255) / 256;
    const dim3 grid(static_cast<unsigned>(blocks));
    switch (a.width) {
        case 2: conv_bwd_kernel<T, V, 2><<<grid, 256, 0, stream>>>(a, nvec, tile, tiles, items); break;
        case 3: conv_bwd_kernel<T, V, 3><<<grid, 256, 0, stream>>>(a, nvec, tile, tiles, items); break;
        case 4: conv_bwd_kernel<T, V, 4><<<grid, 256, 0, stream>>>(a, nvec, tile, tiles, items); break;
        default: return hipErrorInvalidValue;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long K = a.channels;
    const size_t rows = (size_t)a.batch * tiles;
    return launch_colsum(a.part, a.batch * tiles, K * (a.width + 1), K * a.width, a.dweight,
                         a.dbias, stream, a.part + rows * K * (a.width + 1));
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs &a, bool bf16, hipStream_t stream) {
    return bf16 ? conv_fwd<bf16_t>(a, stream) : conv_fwd<float>(a, stream);
}

size_t conv_bwd_part_bytes(int batch, int seqlen, int channels, int width) {
    const int tile = bwd_tile(batch, seqlen, channels);
    const size_t rows = (size_t)batch * ((seqlen + tile - 1) / tile);
    return (rows + (rows > kColsumRows ? kColsumChunks : 0)) * channels * (width + 1) * sizeof(float);
}

bool conv_bwd_grid_ok(int batch, int seqlen, int channels, int width, const ConvParts &dy) {
    const int tile = bwd_tile(batch, seqlen, channels);
    const long long rows = (long long)batch * ((seqlen + tile - 1) / tile);
    return rows <= 0x7fffffff && (rows * part_vecs(dy, 4) + 255) / 256 < (1LL << 24) &&
           colsum_grid_ok(static_cast<int>(rows), (long long)channels * (width + 1), true);
}

hipError_t launch_conv_bwd(const ConvBwdArgs &a, bool bf16, hipStream_t stream) {
    return bf16 ? conv_bwd<bf16_t>(a, stream) : conv_bwd<float>(a, stream);
}

template <typename T>
static hipError_t conv_step(void *state, const void *x, size_t x_row, const float *weight,
                            const float *bias, int batch, int K, int width, int silu,
                            const ConvParts &y, hipStream_t stream) {
    constexpr int V = 4;
    const int nvec = part_vecs(y, V);
    const long long items = (long long)batch * nvec, blocks = (items + 255) / 256;
    if (blocks >= (1LL << 24)) return hipErrorNotSupported;
    const dim3 grid(static_cast<unsigned>(blocks));
    T *st = static_cast<T *>(state);
    const T *xx = static_cast<const T *>(x);
    switch (width) {
        case 2: conv_step_kernel<T, V, 2><<<grid, 256, 0, stream>>>(st, xx, x_row, weight, bias, K, silu, y, nvec, items); break;
        case 3: conv_step_kernel<T, V, 3><<<grid, 256, 0, stream>>>(st, xx, x_row, weight, bias, K, silu, y, nvec, items); break;
        case 4: conv_step_kernel<T, V, 4><<<grid, 256, 0, stream>>>(st, xx, x_row, weight, bias, K, silu, y, nvec, items); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch_conv_step(void *state, const void *x, size_t x_row, const float *weight,
                            const float *bias, int batch, int channels, int width, int silu,
                            const ConvParts &y, bool bf16, hipStream_t stream) {
    return bf16 ? conv_step<bf16_t>(state, x, x_row, weight, bias, batch, channels, width, silu, y, stream)
                : conv_step<float>(state, x, x_row, weight, bias, batch, channels, width, silu, y, stream);
}

}  // namespace ssd
