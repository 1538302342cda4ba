// Selective scan with a decay rate for every channel and state, forward
// ("从Transformer到Mamba" tutorial, section 3.2): per channel e and state n,
//   h_t[n] = exp(dt_t A[e][n]) h_{t-1}[n] + dt_t x_t B_t[n],
//   y_t    = (sum_n C_t[n] h_t[n] + D[e] x_t) silu(z_t),
// with B_t, C_t shared by the channels of a group.
//
// The decay differs from state to state, so nothing here is a matrix product:
// an element (token, channel, state) costs one exponential (a quarter-rate
// instruction) and four multiply-adds, 8 vector-issue slots, and 16 states of
// one channel-token more time than its 8 bytes do. The kernel is bound by
// vector issue; what it can do is to issue little else. So
// * a lane keeps 4 states in registers for the whole walk, and the lanes of a
//   channel are neighbours: y_t takes two DPP additions at 16 states;
// * step sizes (softplus) and gates are computed once per (token, channel) by
//   the lanes that load them, 16 bytes each, and reach the walk through LDS as
//   (dt, dt x); B and C reach it as float, one 16-byte read each per 4 states;
// * the next tile's rows are fetched into registers while a tile is walked.
// With few channels the token axis is cut into segments: a first kernel makes
// every segment's state from zero and its sum of step sizes (the decay over
// any span is exp(A sum dt)), and the walk of a segment starts by folding the
// segments before it, in their order.
#include "selective.h"

namespace ssd {

namespace {

// What the walk leaves: outputs; a segment's state and step-size sum; or (for
// the backward) those and, before every BACK tokens, the state from the
// segment's start (zero, or the first one's initial state) with its step-size sum.
enum SelMode { SEL_OUT, SEL_STATE, SEL_KEEP };

template <typename T, int NK, SelMode MODE>
__global__ __launch_bounds__(256) void selective_fwd_kernel(SelArgs a) {
    constexpr bool STATE = MODE != SEL_OUT;
    using S = SelShape<NK>;
    constexpr int SL = S::SL, CH = S::CH, TILE = S::TILE;
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    constexpr int VPR = CH / V;                              // vectors per row
    constexpr int IT = (TILE * VPR + 255) / 256;             // row vectors per lane
    constexpr int IB = (TILE * NK + 255) / 256;              // B and C elements per lane
    __shared__ float2 du[TILE * CH];                         // (dt, dt x)
    __shared__ __attribute__((aligned(16))) float bs[TILE * NK];
    __shared__ __attribute__((aligned(16))) float cs[STATE ? 4 : TILE * NK];
    __shared__ float ys[STATE ? 1 : TILE * CH];

    const int segs = MODE == SEL_STATE ? a.segs - 1 : a.segs;
    const SelBlock k = sel_block<NK>(blockIdx.x, a.channels, a.ngroups, segs);
    const int tid = threadIdx.x, sl = tid & (SL - 1), ch = tid / SL;
    const int N = a.dstate, E = a.channels;
    const int t_begin = k.seg * a.seg_len, t_end = min(a.seqlen, t_begin + a.seg_len);
    const T *x = static_cast<const T *>(a.x) + k.b * a.x_batch + k.first;
    const T *dt = static_cast<const T *>(a.dt) + k.b * a.dt_batch + k.first;
    const T *z = a.z ? static_cast<const T *>(a.z) + k.b * a.z_batch + k.first : nullptr;
    const T *B = static_cast<const T *>(a.B) + k.b * a.B_batch + (size_t)k.g * N;
    const T *C = static_cast<const T *>(a.C) + k.b * a.C_batch + (size_t)k.g * N;

    // this lane's states (those past the state size stay zero: A = B = C = 0)
    const bool live = ch < k.n;
    const int n0 = sl * 4, nn = live ? N - n0 : 0;
    float A2[4], h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dsum = 0.0f;
    {
        RowRaw<float, 4> r;
        r.zero();
        if (nn > 0) r.load(a.A + (size_t)(k.first + ch) * N + n0, nn);
#pragma unroll
        for (int i = 0; i < 4; ++i) A2[i] = r.get(i) * kLog2e;
    }
    if (k.seg == 0 && a.init && nn > 0) {
        RowRaw<float, 4> r;
        r.load(a.init + ((size_t)k.b * E + k.first + ch) * N + n0, nn);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = r.get(i);
    }
    if (!STATE && live) {
        // segment s's own state (the first one's goes on from the initial state) and
        // step-size sum, [b][segs - 1][E], states NK wide
        const size_t at = (size_t)k.b * (segs - 1) * E + k.first + ch;
        for (int s = 0; s < k.seg; ++s) {
            const float sum = a.seg_sum[at + (size_t)s * E];
            const float4 st = *reinterpret_cast<const float4 *>(a.seg_state + (at + (size_t)s * E) * NK + n0);
            const float v[4] = {st.x, st.y, st.z, st.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = s == 0 ? v[i] : fmaf(__builtin_amdgcn_exp2f(A2[i] * sum), h[i], v[i]);
        }
    }

    // this lane's row vectors: row r, channels c .. of the tile
    RowRaw<T, V> xr[2][IT], dr[2][IT], zr[2][IT];
    float br[2][IB], cr[2][IB];
    auto fetch = [&](int t0, int w) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * 256, r = id / VPR, c = (id % VPR) * V;
            xr[w][i].zero();
            dr[w][i].zero();
            zr[w][i].zero();
            if (r < TILE && t0 + r < t_end && c < k.n) {
                const size_t t = t0 + r;
                xr[w][i].load(x + t * a.x_token + c, k.n - c);
                dr[w][i].load(dt + t * a.dt_token + c, k.n - c);
                if (!STATE && z) zr[w][i].load(z + t * a.z_token + c, k.n - c);
            }
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int id = tid + i * 256, r = id / NK, n = id % NK;
            const bool ok = r < TILE && t0 + r < t_end && n < N;
            br[w][i] = ok ? to_f32(B[(size_t)(t0 + r) * a.B_token + n]) : 0.0f;
            if (!STATE) cr[w][i] = ok ? to_f32(C[(size_t)(t0 + r) * a.C_token + n]) : 0.0f;
        }
    };

    float bias[IT][V], Dv[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = ((tid + i * 256) % VPR) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            bias[i][e] = a.opts.bias && c + e < k.n ? a.opts.bias[k.first + c + e] : 0.0f;
            Dv[i][e] = !STATE && a.D && c + e < k.n ? a.D[k.first + c + e] : 0.0f;
        }
    }

    fetch(t_begin, 0);
    auto tile = [&](int t0, int w) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * 256, r = id / VPR, c = (id % VPR) * V;
            if (r < TILE) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = sel_step(a.opts, dr[w][i].get(e) + bias[i][e]);
                    du[r * CH + c + e] = make_float2(d, d * xr[w][i].get(e));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int id = tid + i * 256;
            if (id < TILE * NK) {
                bs[id] = br[w][i];
                if (!STATE) cs[id] = cr[w][i];
            }
        }
        __syncthreads();
        if (t0 + TILE < t_end) fetch(t0 + TILE, w ^ 1);
        const int nt = min(TILE, t_end - t0);
#pragma unroll 4
        for (int t = 0; t < nt; ++t) {
            const float2 d = du[t * CH + ch];
            const float4 b4 = *reinterpret_cast<const float4 *>(&bs[t * NK + n0]);
            const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
            float p = 0.0f;
            if constexpr (STATE) {
                if constexpr (MODE == SEL_KEEP)
                    if (t % S::BACK == 0 && live) {
                        const size_t at = ((size_t)k.b * a.keeps + (t0 + t) / S::BACK) * E + k.first + ch;
                        *reinterpret_cast<float4 *>(a.keep_state + at * NK + n0) =
                            make_float4(h[0], h[1], h[2], h[3]);
                        if (sl == 0) a.keep_sum[at] = dsum;
                    }
                dsum += d.x;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[i] = fmaf(__builtin_amdgcn_exp2f(d.x * A2[i]), h[i], d.y * bv[i]);
            } else {
                const float4 c4 = *reinterpret_cast<const float4 *>(&cs[t * NK + n0]);
                const float cv[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = fmaf(__builtin_amdgcn_exp2f(d.x * A2[i]), h[i], d.y * bv[i]);
                    p = fmaf(cv[i], h[i], p);
                }
                p = lanes_sum<SL>(p);
                if (sl == 0) ys[t * CH + ch] = p;
            }
        }
        __syncthreads();
        if constexpr (!STATE) {
            T *y = static_cast<T *>(a.y);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int id = tid + i * 256, r = id / VPR, c = (id % VPR) * V;
                if (r < nt && c < k.n) {
                    float o[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        o[e] = fmaf(Dv[i][e], xr[w][i].get(e), ys[r * CH + c + e]);
                        if (z) o[e] *= silu_f32(zr[w][i].get(e));
                    }
                    row_store(y + ((size_t)k.b * a.seqlen + t0 + r) * E + k.first + c, o, k.n - c);
                }
            }
        }
    };
    for (int t0 = t_begin; t0 < t_end; t0 += 2 * TILE) {
        tile(t0, 0);
        if (t0 + TILE < t_end) tile(t0 + TILE, 1);
    }

    if constexpr (STATE) {
        if (!live || k.seg >= a.segs - 1) return;
        const size_t at = ((size_t)k.b * (a.segs - 1) + k.seg) * E + k.first + ch;
        *reinterpret_cast<float4 *>(a.seg_state + at * NK + n0) = make_float4(h[0], h[1], h[2], h[3]);
        if (sl == 0) a.seg_sum[at] = dsum;
    } else if (a.final_state && k.seg == segs - 1 && nn > 0) {
        row_store(a.final_state + ((size_t)k.b * E + k.first + ch) * N + n0, h, nn);
    }
}

// One token. Bound by the float32 state, read once and written once: a lane
// takes 4 states (16 bytes), neighbours the rest of the channel.
template <typename T, int NK>
__global__ __launch_bounds__(256) void selective_step_kernel(SelArgs a, float *__restrict__ state,
                                                             long long items) {
    constexpr int SL = SelShape<NK>::SL;
    const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
    const int sl = threadIdx.x & (SL - 1), n0 = sl * 4;
    const int N = a.dstate, E = a.channels, nn = N - n0;
    if (item >= items) return;
    const long long be = item / SL;
    const int b = static_cast<int>(be / E), e = static_cast<int>(be % E), g = e / (E / a.ngroups);
    RowRaw<float, 4> hr, Ar;
    RowRaw<T, 4> Br, Cr;
    hr.zero(); Ar.zero(); Br.zero(); Cr.zero();
    float *st = state + (size_t)be * N + n0;
    if (nn > 0) {
        hr.load(st, nn);
        Ar.load(a.A + (size_t)e * N + n0, nn);
        Br.load(static_cast<const T *>(a.B) + b * a.B_batch + (size_t)g * N + n0, nn);
        Cr.load(static_cast<const T *>(a.C) + b * a.C_batch + (size_t)g * N + n0, nn);
    }
    const float xv = to_f32(static_cast<const T *>(a.x)[b * a.x_batch + e]);
    const float d = sel_step(a.opts, to_f32(static_cast<const T *>(a.dt)[b * a.dt_batch + e]) +
                                         (a.opts.bias ? a.opts.bias[e] : 0.0f));
    const float u = d * xv;
    float h[4], p = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(__builtin_amdgcn_exp2f(d * (Ar.get(i) * kLog2e)), hr.get(i), u * Br.get(i));
        p = fmaf(Cr.get(i), h[i], p);
    }
    if (nn > 0) row_store(st, h, nn);
    p = lanes_sum<SL>(p);
    if (sl == 0) {
        float o = p + (a.D ? a.D[e] : 0.0f) * xv;
        if (a.z) o *= silu_f32(to_f32(static_cast<const T *>(a.z)[b * a.z_batch + e]));
        static_cast<T *>(a.y)[be] = from_f32<T>(o);
    }
}

template <typename T, int NK> hipError_t sel_fwd(const SelArgs &a, hipStream_t stream) {
    const int blocks = selective_blocks(a.channels, a.ngroups, a.dstate);
    if (a.segs > 1) {
        selective_fwd_kernel<T, NK, SEL_STATE>
            <<<static_cast<unsigned>(blocks * (a.segs - 1) * a.batch), 256, 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    selective_fwd_kernel<T, NK, SEL_OUT>
        <<<static_cast<unsigned>(blocks * a.segs * a.batch), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int NK> hipError_t sel_keep(const SelArgs &a, hipStream_t stream) {
    selective_fwd_kernel<T, NK, SEL_KEEP>
        <<<static_cast<unsigned>(selective_blocks(a.channels, a.ngroups, a.dstate) * a.segs * a.batch),
           256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int NK>
hipError_t sel_step_launch(const SelArgs &a, float *state, hipStream_t stream) {
    const long long items = (long long)a.batch * a.channels * SelShape<NK>::SL;
    selective_step_kernel<T, NK>
        <<<static_cast<unsigned>((items + 255) / 256), 256, 0, stream>>>(a, state, items);
    return hipGetLastError();
}

}  // namespace

int selective_kernel_dstate(int n) {
    for (int k = 4; k <= 64; k *= 2)
        if (n <= k) return k;
    return 0;
}

int selective_blocks(int channels, int ngroups, int dstate) {
    const int CH = 1024 / selective_kernel_dstate(dstate), each = channels / ngroups;
    return ngroups * ((each + CH - 1) / CH);
}

// Segments of the token axis. One walk costs 8 issue slots per element, a
// segment's state 7 more, so cutting pays only while the uncut walks leave
// most of the GPU idle.
SelPlan selective_plan(int batch, int seqlen, int channels, int ngroups, int dstate) {
    const int nk = selective_kernel_dstate(dstate), tile = nk < 16 ? 2 * nk : 32;
    const long long wgs = (long long)batch * selective_blocks(channels, ngroups, dstate);
    SelPlan p{1, seqlen, 0};
    if (wgs < 512) {
        long long s = (1024 + wgs - 1) / wgs;
        const int tiles = (seqlen + tile - 1) / tile;
        if (s > tiles / 2) s = tiles / 2;
        if (s > 1) {
            const int per = static_cast<int>((tiles + s - 1) / s);
            p.seg_len = per * tile;
            p.segs = (seqlen + p.seg_len - 1) / p.seg_len;
        }
    }
    if (p.segs <= 1) return SelPlan{1, seqlen, 0};
    p.scratch_bytes = (size_t)batch * (p.segs - 1) * channels * (nk + 1) * sizeof(float);
    return p;
}

hipError_t launch_selective_fwd(const SelArgs &a, bool bf16, hipStream_t stream) {
    SSD_SEL_DISPATCH(sel_fwd, a, stream)
}
hipError_t launch_selective_keep(const SelArgs &a, bool bf16, hipStream_t stream) {
    SSD_SEL_DISPATCH(sel_keep, a, stream)
}
hipError_t launch_selective_step(const SelArgs &a, float *state, bool bf16, hipStream_t stream) {
    SSD_SEL_DISPATCH(sel_step_launch, a, state, stream)
}

}  // namespace ssd
