// Backward of the selective scan. With q_t[n] = exp(dt_t A[n]) h_{t-1}[n], the
// adjoint runs back in time:
//   g_t[n] = dy_t C_t[n] + exp(dt_{t+1} A[n]) g_{t+1}[n]      (dy after the gate's silu(z))
//   dx_t = dt_t sum_n g_t B_t + D dy_t,  ddt_t = sum_n g_t (x_t B_t + A q_t),
//   dA[n] = sum_t dt_t g_t q_t,  dB_t = sum_e dt_t x_t g_t,  dC_t = sum_e dy_t h_t,
//   dz_t = dy'_t (sum_n C_t h_t + D x_t) silu'(z_t),  ddt then through softplus and clamp.
//
// States are recomputed, not stored by the forward: a first walk (the
// forward's, SEL_KEEP) keeps the state before every 16 tokens (8 at small
// state sizes), and the walk back rebuilds a tile's 16 states in registers from there,
// with their decays, then runs the adjoint over them. As in the forward a lane
// holds 4 states of one channel. Bound by vector issue: about 25 slots per
// element, of which the rebuilding takes 7.
//
// Sums over channels (dB, dC): per token a wavefront adds its channels' eight
// values by exchanging halves and rows of lanes between two registers (each
// exchange and addition halves the number of values as it doubles the lanes
// summed), then within the rows of 16 lanes; wavefronts meet in LDS, and
// workgroups in partial tensors that are added in a fixed order. Sums over
// tokens (dA, dD, the bias) stay in registers and end in partial rows the same way.
//
// With segments (see the forward) every segment's adjoint from zero is made
// first, and a walk starts by folding the segments after its own.
#include "selective.h"

namespace ssd {

namespace {

// a's and b's halves (or odd and even rows of 16 lanes) exchanged and added:
// lower half (even rows): a summed over both, upper half (odd rows): b.
__device__ __forceinline__ float fold32(float a, float b) {
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    const u2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float a, float b) {
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    const u2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sum over the lanes of a row of 16 that share lane % SL, in each of them.
template <int SL> __device__ __forceinline__ float row_fold(float v) {
    auto add = [](float a, int b) { return a + __int_as_float(b); };
    if constexpr (SL <= 8) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, true));
    if constexpr (SL <= 4) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xf, 0xf, true));
    if constexpr (SL <= 2) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xf, 0xf, true));
    if constexpr (SL <= 1) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xf, 0xf, true));
    return v;
}

__device__ __forceinline__ float4 f4(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }

// A segment's adjoint from zero (from dfinal for the last one): the gradient
// of the state entering it, for segments 1 .. segs - 1.
template <typename T, int NK>
__global__ __launch_bounds__(256) void selective_adj_kernel(SelBwdArgs ba) {
    using S = SelShape<NK>;
    constexpr int SL = S::SL, CH = S::CH, TILE = S::TILE;
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    constexpr int VPR = CH / V, IT = (TILE * VPR + 255) / 256, IB = (TILE * NK + 255) / 256;
    __shared__ float2 dd[TILE * CH];  // (dt, dy)
    __shared__ __attribute__((aligned(16))) float cs[TILE * NK];
    const SelArgs &a = ba.f;
    SelBlock k = sel_block<NK>(blockIdx.x, a.channels, a.ngroups, a.segs - 1);
    k.seg += 1;
    const int tid = threadIdx.x, sl = tid & (SL - 1), ch = tid / SL, n0 = sl * 4;
    const int N = a.dstate, E = a.channels, nn = ch < k.n ? N - n0 : 0;
    const int t_begin = k.seg * a.seg_len, t_end = min(a.seqlen, t_begin + a.seg_len);
    const T *dt = static_cast<const T *>(a.dt) + k.b * a.dt_batch + k.first;
    const T *z = a.z ? static_cast<const T *>(a.z) + k.b * a.z_batch + k.first : nullptr;
    const T *C = static_cast<const T *>(a.C) + k.b * a.C_batch + (size_t)k.g * N;
    const T *dy = static_cast<const T *>(ba.dy) + (size_t)k.b * a.seqlen * E + k.first;
    float A2[4], g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    {
        RowRaw<float, 4> r;
        r.zero();
        if (nn > 0) r.load(a.A + (size_t)(k.first + ch) * N + n0, nn);
#pragma unroll
        for (int i = 0; i < 4; ++i) A2[i] = r.get(i) * kLog2e;
        r.zero();
        if (nn > 0 && ba.dfinal && k.seg == a.segs - 1)
            r.load(ba.dfinal + ((size_t)k.b * E + k.first + ch) * N + n0, nn);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = r.get(i);
    }
    const int tiles = (t_end - t_begin + TILE - 1) / TILE;
    for (int ti = tiles - 1; ti >= 0; --ti) {
        const int t0 = t_begin + ti * TILE, nt = min(TILE, t_end - t0);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * 256, r = id / VPR, c = (id % VPR) * V;
            if (r < nt && c < k.n) {
                RowRaw<T, V> dr, zr, yr;
                const size_t t = t0 + r;
                dr.load(dt + t * a.dt_token + c, k.n - c);
                yr.load(dy + t * E + c, k.n - c);
                if (z) zr.load(z + t * a.z_token + c, k.n - c);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float b = a.opts.bias && c + e < k.n ? a.opts.bias[k.first + c + e] : 0.0f;
                    const float w = z ? silu_f32(zr.get(e)) : 1.0f;
                    dd[r * CH + c + e] = make_float2(sel_step(a.opts, dr.get(e) + b), yr.get(e) * w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int id = tid + i * 256, r = id / NK, n = id % NK;
            if (r < nt) cs[id] = n < N ? to_f32(C[(size_t)(t0 + r) * a.C_token + n]) : 0.0f;
        }
        __syncthreads();
        if (nn > 0)
#pragma unroll 4
            for (int t = nt - 1; t >= 0; --t) {
                const float2 d = dd[t * CH + ch];
                const float4 c4 = *reinterpret_cast<const float4 *>(&cs[t * NK + n0]);
                const float cv[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    g[i] = __builtin_amdgcn_exp2f(d.x * A2[i]) * fmaf(d.y, cv[i], g[i]);
            }
        __syncthreads();
    }
    if (nn > 0)
        *reinterpret_cast<float4 *>(
            ba.seg_adj + (((size_t)k.b * (a.segs - 1) + k.seg - 1) * E + k.first + ch) * NK + n0) = f4(g);
}

template <typename T, int NK, bool GATE>
__global__ __launch_bounds__(256, 2) void selective_bwd_kernel(SelBwdArgs ba) {
    using S = SelShape<NK>;
    constexpr int SL = S::SL, CH = S::CH, TB = S::BACK, V = 4;
    constexpr int VPR = CH / V, IT = (TB * VPR + 255) / 256, IB = (TB * NK + 255) / 256;
    __shared__ float2 du[TB * CH];  // (dt, dt x); after the walk back sum_n (g B), sum_n (A2 g q)
    __shared__ float dys[TB * CH];  // dy silu(z)
    __shared__ float ys[GATE ? TB * CH : 1];
    __shared__ __attribute__((aligned(16))) float bs[TB * NK];
    __shared__ __attribute__((aligned(16))) float cs[TB * NK];
    // dB and dC of every wavefront; after the last tile every lane's dD and bias sums
    constexpr int RED = 4 * TB * 2 * NK, ACC = 2 * 256 * V;
    __shared__ __attribute__((aligned(16))) float red[RED > ACC ? RED : ACC];

    const SelArgs &a = ba.f;
    const SelBlock k = sel_block<NK>(blockIdx.x, a.channels, a.ngroups, a.segs);
    const int tid = threadIdx.x, sl = tid & (SL - 1), ch = tid / SL, n0 = sl * 4;
    const int w = tid >> 6, row16 = (tid >> 4) & 3;
    const int N = a.dstate, E = a.channels, L = a.seqlen;
    const bool live = ch < k.n;
    const int nn = live ? N - n0 : 0;
    const int t_begin = k.seg * a.seg_len, t_end = min(L, t_begin + a.seg_len);
    const T *x = static_cast<const T *>(a.x) + k.b * a.x_batch + k.first;
    const T *dt = static_cast<const T *>(a.dt) + k.b * a.dt_batch + k.first;
    const T *z = GATE ? static_cast<const T *>(a.z) + k.b * a.z_batch + k.first : nullptr;
    const T *B = static_cast<const T *>(a.B) + k.b * a.B_batch + (size_t)k.g * N;
    const T *C = static_cast<const T *>(a.C) + k.b * a.C_batch + (size_t)k.g * N;
    const T *dy = static_cast<const T *>(ba.dy) + (size_t)k.b * L * E + k.first;

    float A2[4], h_in[4] = {0.0f, 0.0f, 0.0f, 0.0f}, ag[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float dA[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    {
        RowRaw<float, 4> r;
        r.zero();
        if (nn > 0) r.load(a.A + (size_t)(k.first + ch) * N + n0, nn);
#pragma unroll
        for (int i = 0; i < 4; ++i) A2[i] = r.get(i) * kLog2e;
    }
    if (live) {
        const size_t at = (size_t)k.b * (a.segs - 1) * E + k.first + ch;
        for (int s = 0; s < k.seg; ++s) {
            const float sum = a.seg_sum[at + (size_t)s * E];
            const float4 st = *reinterpret_cast<const float4 *>(a.seg_state + (at + (size_t)s * E) * NK + n0);
            const float v[4] = {st.x, st.y, st.z, st.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h_in[i] = s == 0 ? v[i] : fmaf(__builtin_amdgcn_exp2f(A2[i] * sum), h_in[i], v[i]);
        }
        if (k.seg == a.segs - 1) {
            RowRaw<float, 4> r;
            r.zero();
            if (ba.dfinal && nn > 0) r.load(ba.dfinal + ((size_t)k.b * E + k.first + ch) * N + n0, nn);
#pragma unroll
            for (int i = 0; i < 4; ++i) ag[i] = r.get(i);
        }
        for (int s = a.segs - 1; s > k.seg; --s) {
            // the gradient of the state entering segment s
            const float4 st = *reinterpret_cast<const float4 *>(ba.seg_adj + (at + (size_t)(s - 1) * E) * NK + n0);
            const float v[4] = {st.x, st.y, st.z, st.w};
            const float sum = s < a.segs - 1 ? a.seg_sum[at + (size_t)s * E] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ag[i] = s == a.segs - 1 ? v[i] : fmaf(__builtin_amdgcn_exp2f(A2[i] * sum), ag[i], v[i]);
        }
    }

    float bias[IT][V], Dv[IT][V], dD[IT][V], db[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = ((tid + i * 256) % VPR) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            bias[i][e] = a.opts.bias && c + e < k.n ? a.opts.bias[k.first + c + e] : 0.0f;
            Dv[i][e] = a.D && c + e < k.n ? a.D[k.first + c + e] : 0.0f;
            dD[i][e] = db[i][e] = 0.0f;
        }
    }

    const int tiles = (t_end - t_begin + TB - 1) / TB;
    for (int ti = tiles - 1; ti >= 0; --ti) {
        const int t0 = t_begin + ti * TB, nt = min(TB, t_end - t0);
        RowRaw<T, V> xr[IT], zr[IT], yr[IT], dr[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * 256, r = id / VPR, c = (id % VPR) * V;
            xr[i].zero();
            dr[i].zero();
            zr[i].zero();
            yr[i].zero();
            if (r < nt && c < k.n) {
                const size_t t = t0 + r;
                xr[i].load(x + t * a.x_token + c, k.n - c);
                dr[i].load(dt + t * a.dt_token + c, k.n - c);
                if (GATE) zr[i].load(z + t * a.z_token + c, k.n - c);
                yr[i].load(dy + t * E + c, k.n - c);
            }
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int id = tid + i * 256, r = id / NK, n = id % NK;
            if (r < TB) {
                const bool ok = r < nt && n < N;
                bs[id] = ok ? to_f32(B[(size_t)(t0 + r) * a.B_token + n]) : 0.0f;
                cs[id] = ok ? to_f32(C[(size_t)(t0 + r) * a.C_token + n]) : 0.0f;
            }
        }
        float hk[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // the state entering the tile
        if (live) {
            const size_t at = ((size_t)k.b * a.keeps + t0 / TB) * E + k.first + ch;
            const float4 st = *reinterpret_cast<const float4 *>(a.keep_state + at * NK + n0);
            const float v[4] = {st.x, st.y, st.z, st.w};
            const float sum = k.seg ? a.keep_sum[at] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                hk[i] = k.seg ? fmaf(__builtin_amdgcn_exp2f(A2[i] * sum), h_in[i], v[i]) : v[i];
        }
        float delta[IT][V], dyg[IT][V];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * 256, r = id / VPR, c = (id % VPR) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                // rows past the end neither move the state nor take a gradient
                delta[i][e] = r < nt ? sel_step(a.opts, dr[i].get(e) + bias[i][e]) : 0.0f;
                dyg[i][e] = yr[i].get(e);
                if (GATE) dyg[i][e] *= silu_f32(zr[i].get(e));
                if (r < TB) {
                    du[r * CH + c + e] = make_float2(delta[i][e], delta[i][e] * xr[i].get(e));
                    dys[r * CH + c + e] = dyg[i][e];
                }
            }
        }
        __syncthreads();

        float h[TB][4], dec[TB][4];
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            // LDS reads of at most two tokens ahead: more would not fit the registers
            if (t % 2 == 0) __builtin_amdgcn_sched_barrier(0);
            const float2 d = du[t * CH + ch];
            const float4 b4 = *reinterpret_cast<const float4 *>(&bs[t * NK + n0]);
            const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dec[t][i] = __builtin_amdgcn_exp2f(d.x * A2[i]);
                h[t][i] = fmaf(dec[t][i], t ? h[t - 1][i] : hk[i], d.y * bv[i]);
            }
            if constexpr (GATE) {
                const float4 c4 = *reinterpret_cast<const float4 *>(&cs[t * NK + n0]);
                float p = c4.x * h[t][0];
                p = fmaf(c4.y, h[t][1], p);
                p = fmaf(c4.z, h[t][2], p);
                p = fmaf(c4.w, h[t][3], p);
                p = lanes_sum<SL>(p);
                if (sl == 0) ys[t * CH + ch] = p;
            }
        }
#pragma unroll
        for (int t = TB - 1; t >= 0; --t) {
            if (t % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            const float2 d = du[t * CH + ch];
            const float dyv = dys[t * CH + ch];
            const float4 b4 = *reinterpret_cast<const float4 *>(&bs[t * NK + n0]);
            const float4 c4 = *reinterpret_cast<const float4 *>(&cs[t * NK + n0]);
            const float bv[4] = {b4.x, b4.y, b4.z, b4.w}, cv[4] = {c4.x, c4.y, c4.z, c4.w};
            float gB = 0.0f, gA = 0.0f, v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g = fmaf(dyv, cv[i], ag[i]);
                gB = fmaf(g, bv[i], gB);
                const float gq = g * (dec[t][i] * (t ? h[t - 1][i] : hk[i]));
                gA = fmaf(A2[i], gq, gA);
                dA[i] = fmaf(d.x, gq, dA[i]);
                ag[i] = dec[t][i] * g;
                v[i] = d.y * g;
                v[4 + i] = dyv * h[t][i];
            }
            gB = lanes_sum<SL>(gB);
            gA = lanes_sum<SL>(gA);
            // every lane of the channel has read du[t] (they are of one wavefront)
            if (sl == 0) du[t * CH + ch] = make_float2(gB, gA);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fold32(v[i], v[4 + i]);
            float q0 = row_fold<SL>(fold16(v[0], v[2])), q1 = row_fold<SL>(fold16(v[1], v[3]));
            // row 0: dB of states n0, n0 + 1; row 1: n0 + 2, n0 + 3; rows 2, 3: dC
            if ((tid & 15) < SL) {
                float *p = &red[((w * TB + t) * 2 + (row16 >> 1)) * NK + n0 + 2 * (row16 & 1)];
                *reinterpret_cast<float2 *>(p) = make_float2(q0, q1);
            }
        }
        __syncthreads();

#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * 256, r = id / VPR, c = (id % VPR) * V;
            if (r < nt && c < k.n) {
                float ox[V], ot[V], oz[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 s = du[r * CH + c + e];
                    const float xv = xr[i].get(e), raw = dr[i].get(e) + bias[i][e];
                    ox[e] = fmaf(delta[i][e], s.x, Dv[i][e] * dyg[i][e]);
                    float dd = fmaf(xv, s.x, s.y * 0.6931471805599453f);
                    if (a.opts.clamp) {
                        const float free = a.opts.softplus ? softplus_f32(raw) : raw;
                        if (free < a.opts.lo || free > a.opts.hi) dd = 0.0f;
                    }
                    if (a.opts.softplus) dd *= sigmoid_f32(raw);
                    ot[e] = dd;
                    if (c + e < k.n) {
                        dD[i][e] = fmaf(dyg[i][e], xv, dD[i][e]);
                        db[i][e] += dd;
                    }
                    if constexpr (GATE)
                        oz[e] = yr[i].get(e) * fmaf(Dv[i][e], xv, ys[r * CH + c + e]) *
                                silu_grad_f32(zr[i].get(e));
                }
                const size_t o = ((size_t)k.b * L + t0 + r) * E + k.first + c;
                row_store(static_cast<T *>(ba.dx) + o, ox, k.n - c);
                row_store(static_cast<T *>(ba.ddt) + o, ot, k.n - c);
                if constexpr (GATE) row_store(static_cast<T *>(ba.dz) + o, oz, k.n - c);
            }
        }
        // the wavefronts' dB and dC, to this workgroup's partial tensors
        const int each = E / a.ngroups, part = (k.first - k.g * each) / CH;
        const size_t count = (size_t)a.batch * L * a.ngroups * N;
        for (int id = tid; id < nt * 2 * NK; id += 256) {
            const int t = id / (2 * NK), m = (id / NK) & 1, n = id % NK;
            if (n < N) {
                float s = 0.0f;
#pragma unroll
                for (int u = 0; u < 4; ++u) s += red[(u * TB + t) * 2 * NK + m * NK + n];
                ba.dbc_part[((size_t)part * 2 + m) * count +
                            (((size_t)k.b * L + t0 + t) * a.ngroups + k.g) * N + n] = s;
            }
        }
        __syncthreads();
    }

    const size_t unit = (size_t)k.b * a.segs + k.seg;
    if (nn > 0) {
        row_store(ba.dA_part + (unit * E + k.first + ch) * N + n0, dA, nn);
        if (ba.dinit && k.seg == 0)
            row_store(ba.dinit + ((size_t)k.b * E + k.first + ch) * N + n0, ag, nn);
    }
    // dD and the bias: a channel's sums lie in the 256 / VPR lanes (or IT vectors) of its column
    float sD[V], sb[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sD[e] = sb[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            sD[e] += dD[i][e];
            sb[e] += db[i][e];
        }
        red[tid * V + e] = sD[e];
        red[256 * V + tid * V + e] = sb[e];
    }
    __syncthreads();
    for (int c = tid; c < k.n; c += 256) {
        float s0 = 0.0f, s1 = 0.0f;
        for (int r = c / V; r < 256; r += VPR) {
            s0 += red[r * V + c % V];
            s1 += red[256 * V + r * V + c % V];
        }
        ba.de_part[(unit * 2) * E + k.first + c] = s0;
        ba.de_part[(unit * 2 + 1) * E + k.first + c] = s1;
    }
}

// out (dB, then dC) = sums over `n` partial tensors of `count` values, four to a lane
template <typename T>
__global__ __launch_bounds__(256) void selective_dbc_kernel(const float *__restrict__ part, int n,
                                                            size_t count, T *__restrict__ dB,
                                                            T *__restrict__ dC) {
    const size_t vecs = (count + 3) / 4, id = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= 2 * vecs) return;
    const int m = id >= vecs;
    const size_t c = (id - m * vecs) * 4;
    const int left = count - c < 4 ? static_cast<int>(count - c) : 4;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int p = 0; p < n; ++p) {
        RowRaw<float, 4> r;
        r.load(part + ((size_t)p * 2 + m) * count + c, left);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += r.get(e);
    }
    row_store((m ? dC : dB) + c, s, left);
}

template <typename T, int NK> hipError_t sel_bwd(const SelBwdArgs &ba, hipStream_t stream) {
    const SelArgs &a = ba.f;
    const int blocks = selective_blocks(a.channels, a.ngroups, a.dstate);
    hipError_t e = launch_selective_keep(a, sizeof(T) == 2, stream);
    if (e != hipSuccess) return e;
    if (a.segs > 1) {
        selective_adj_kernel<T, NK>
            <<<static_cast<unsigned>(blocks * (a.segs - 1) * a.batch), 256, 0, stream>>>(ba);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const unsigned grid = static_cast<unsigned>(blocks * a.segs * a.batch);
    if (a.z) selective_bwd_kernel<T, NK, true><<<grid, 256, 0, stream>>>(ba);
    else selective_bwd_kernel<T, NK, false><<<grid, 256, 0, stream>>>(ba);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const size_t count = (size_t)a.batch * a.seqlen * a.ngroups * a.dstate;
    selective_dbc_kernel<T><<<static_cast<unsigned>((2 * ((count + 3) / 4) + 255) / 256), 256, 0, stream>>>(
        ba.dbc_part, blocks / a.ngroups, count, static_cast<T *>(ba.dB), static_cast<T *>(ba.dC));
    e = hipGetLastError();
    const int units = a.batch * a.segs;
    const long long en = (long long)a.channels * a.dstate;
    if (e == hipSuccess) e = launch_colsum(ba.dA_part, units, en, en, ba.dA, nullptr, stream);
    if (e == hipSuccess && (ba.dD || ba.ddt_bias))
        e = launch_colsum(ba.de_part, units, 2LL * a.channels, a.channels, ba.dD, ba.ddt_bias, stream);
    return e;
}

}  // namespace

int selective_keep_tokens(int dstate) { return selective_kernel_dstate(dstate) < 16 ? 8 : 16; }

// As the forward's: the walks back cost about 32 slots per element with the
// kept states, a segment's adjoint 7 more.
SelPlan selective_bwd_plan(int batch, int seqlen, int channels, int ngroups, int dstate) {
    return selective_plan(batch, seqlen, channels, ngroups, dstate);
}

hipError_t launch_selective_bwd(const SelBwdArgs &ba, bool bf16, hipStream_t stream) {
    const SelArgs &a = ba.f;
    SSD_SEL_DISPATCH(sel_bwd, ba, stream)
}

}  // namespace ssd
