// Selective scan with a decay rate for every channel and state, forward
// ("从Transformer到Mamba" tutorial, section 3.2): per channel e and state n,
//   h_t[n] = exp(dt_t A[e][n]) h_{t-1}[n] + dt_t x_t B_t[n],
//   y_t    = (sum_n C_t[n] h_t[n] + D[e] x_t) silu(z_t),
// with B_t, C_t shared by the channels of a group.
//
// The decay differs from state to state, so nothing here is a matrix product:
// an element (token, channel, state) costs one exponential (half rate) and
// four multiplies or multiply-adds, more issue time at 16 states than the 8
// bytes of its channel-token take to move. The kernel is bound by vector
// issue, so it issues little else:
// * lanes are channels and a lane holds 4 states (16 at 64 states), the other
//   states of the channel being in the other wavefronts: B_t and C_t are then
//   uniform, come from scalar loads (a first small kernel writes them as
//   float, padded) and are scalar operands of the multiply-adds; with the
//   states across lanes they came through LDS, 20 clocks of it per 256
//   elements, and LDS was as busy as the vector units;
// * step sizes (softplus) and gates are computed once per (token, channel) by
//   the lanes that load them, 16 bytes each, and reach the walk through LDS as
//   (dt, dt x); the wavefronts' parts of y_t meet there too, and the lanes
//   that loaded x and z finish and store the rows;
// * the next tile's rows are fetched into registers while a tile is walked, the
//   next tokens' B, C and step sizes while a group of tokens is.
// With few channels the token axis is cut into segments: a first kernel makes
// every segment's state from zero and its sum of step sizes (the decay over
// any span is exp(A sum dt)), and the walk of a segment starts by folding the
// segments before it, in their order.
//
// Measured in bf16 with 5120 channels and 16 states: 1 x 8192 tokens 154 us for
// the segments' states and 209 us for the walk, whose vector units are busy 94%
// of the time; 4 x 2048 tokens 39 + 241 us (63%: mostly one workgroup to a CU), with
// 32 states 56 + 367 us, with 64 104 + 626 us.
// One token for 256 sequences 38 us (4.7 TB/s, bound by the states' way from
// memory and back), for one 3.7 us, a launch. Float32, 2 x 777 tokens of 1000
// channels and 24 states: 21 + 22 us, the time that one segment of 96 tokens takes (an
// uncut walk takes 0.145 us a token), with vector units busy 45 to 50%: segments are two
// tiles at least and rounded up to whole ones, too long to fill the GPU here.
#include "selective.h"

namespace ssd {

namespace {

// B and C in the walks' layout, zero past the state size and past the last token.
template <typename T, int NK>
__global__ __launch_bounds__(256) void selective_bc_kernel(SelArgs a, size_t count) {
    const size_t id = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= count) return;
    const int slot = id % (2 * NK), n = slot / 8 * 4 + slot % 4;
    const size_t row = id / (2 * NK);
    const int padded = sel_padded(a.seqlen), t = row % padded, bg = static_cast<int>(row / padded);
    const int b = bg / a.ngroups, g = bg % a.ngroups;
    float v = 0.0f;
    if (t < a.seqlen && n < a.dstate) {
        const size_t at = (size_t)g * a.dstate + n;
        v = slot / 4 % 2 ? to_f32(static_cast<const T *>(a.C)[b * a.C_batch + t * a.C_token + at])
                          : to_f32(static_cast<const T *>(a.B)[b * a.B_batch + t * a.B_token + at]);
    }
    a.bc[id] = v;
}

// What the walk leaves: outputs; a segment's state and step-size sum; or (for
// the backward) those and, before every few tokens, the state from the
// segment's start (zero, or the first one's initial state) with its step-size
// sum; or all that and the segment's adjoint, the gradient of the state
// entering it when nothing comes from behind it:
//   sum_t P_t C_t dy_t + P_T dfinal,  P_t = exp(A (dt_1 + .. + dt_t)),
// which a walk forward can add up as well, P being a product of the decays
// that it computes anyway: three more instructions per element, where a walk
// backward of its own takes five and loads the step sizes again.
enum SelMode { SEL_OUT, SEL_STATE, SEL_KEEP, SEL_BOTH };

template <typename T, int NK, SelMode MODE>
__global__ __launch_bounds__((SelShape<NK, (MODE >= SEL_KEEP)>::THREADS)) void selective_fwd_kernel(SelArgs a) {
    constexpr bool OUT = MODE == SEL_OUT, BACK = MODE >= SEL_KEEP, ADJ = MODE == SEL_BOTH;
    using S = SelShape<NK, BACK>;
    constexpr int NS = S::NS, WS = S::WS, CH = S::CH, TILE = S::TILE, THREADS = S::THREADS;
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    constexpr int VPR = CH / V;                               // vectors per row
    constexpr int IT = (TILE * VPR + THREADS - 1) / THREADS;  // row vectors per lane
    constexpr int KEEP = sel_keep<NK>();
    constexpr int U = BACK && KEEP < 8 ? KEEP : 8;            // tokens per turn of the inner loop
    __shared__ float2 du[TILE * CH];                          // (dt, dt x)
    __shared__ float ys[OUT ? WS * TILE * CH : ADJ ? TILE * CH : 1];  // parts of y; or dy silu(z)

    // the first `whole` units in one piece, the others segment by segment
    const int first = MODE == SEL_STATE ? a.whole : 0, id = blockIdx.x + first;
    const bool uncut = id < a.whole;
    const int cut = a.units - a.whole;
    const SelBlock k = uncut ? sel_block<CH>(id, 0, a.channels, a.ngroups)
                             : sel_block<CH>(a.whole + (id - a.whole) % cut, (id - a.whole) / cut,
                                             a.channels, a.ngroups);
    const bool last_seg = uncut || k.seg == a.segs - 1;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ws = w % WS, ch = w / WS * 64 + (tid & 63), n0 = ws * NS;
    const int N = a.dstate, E = a.channels;
    const int t_begin = k.seg * a.seg_len, t_end = last_seg ? a.seqlen : t_begin + a.seg_len;
    const bool gate = (OUT || ADJ) && a.z != nullptr;
    // rows of the tile at hand
    const T *x = static_cast<const T *>(a.x) + k.b * a.x_batch + k.first + t_begin * a.x_token;
    const T *dt = static_cast<const T *>(a.dt) + k.b * a.dt_batch + k.first + t_begin * a.dt_token;
    const T *z = gate ? static_cast<const T *>(a.z) + k.b * a.z_batch + k.first + t_begin * a.z_token : nullptr;
    const size_t dense = ((size_t)k.b * a.seqlen + t_begin) * E + k.first;
    const T *dy = ADJ ? static_cast<const T *>(a.dy) + dense : nullptr;
    T *y = OUT ? static_cast<T *>(a.y) + dense : nullptr;
    sel_const *bc = (sel_const *)(a.bc + ((size_t)(k.b * a.ngroups + k.g) * sel_padded(a.seqlen) + t_begin) * 2 * NK +
                                  ws * 2 * NS);

    // this lane's states of scratch row `at`
    auto seg_at = [&](size_t at) { return (at * (NK / 4) + n0 / 4) * E * 4 + (size_t)(k.first + ch) * 4; };
    const bool live = ch < k.n;
    const int nn = live ? N - n0 : 0;  // states of this lane (those past them stay zero)
    float A2[NS], h[NS], P[ADJ ? NS : 1], G[ADJ ? NS : 1], dsum = 0.0f;
    load_rates(a.A + (size_t)(k.first + ch) * N + n0, nn, A2);
    {
        RowRaw<float, NS> r;
        r.zero();
        if (k.seg == 0 && a.init && nn > 0)
            r.load(a.init + ((size_t)k.b * E + k.first + ch) * N + n0, nn);
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = r.get(i);
    }
    if constexpr (ADJ)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            P[i] = 1.0f;
            G[i] = 0.0f;
        }
    if (OUT && live) {
        const size_t at = (size_t)k.b * (a.segs - 1);
        sel_fold<NK>(a.seg_state + seg_at(at), a.seg_sum + at * E + k.first + ch, 1, E, k.seg, A2, h);
    }

    // this lane's row vectors: row r, channels c .. of the tile
    RowRaw<T, V> xr[2][IT], dr[2][IT], zr[2][IT], yr[2][IT];
    uint32_t xo[IT], dto[IT], zo[IT], yo[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
        xo[i] = row_offset<T>(r, a.x_token, c);
        dto[i] = row_offset<T>(r, a.dt_token, c);
        zo[i] = row_offset<T>(r, a.z_token, c);
        yo[i] = row_offset<T>(r, E, c);
    }
    // the tile `ahead` tokens from the one at hand, which begins at t0
    auto fetch = [&](int t0, int ahead, int p) {
        const T *xt = x + ahead * a.x_token, *dtt = dt + ahead * a.dt_token;
        const T *zt = gate ? z + ahead * a.z_token : nullptr, *yt = ADJ ? dy + (size_t)ahead * E : nullptr;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
            xr[p][i].zero();
            dr[p][i].zero();
            if (OUT || ADJ) zr[p][i].zero();
            if (ADJ) yr[p][i].zero();
            if (r < TILE && t0 + ahead + r < t_end && c < k.n) {
                xr[p][i].load(row_at(xt, xo[i]), k.n - c);
                dr[p][i].load(row_at(dtt, dto[i]), k.n - c);
                if (gate) zr[p][i].load(row_at(zt, zo[i]), k.n - c);
                if (ADJ) yr[p][i].load(row_at(yt, yo[i]), k.n - c);
            }
        }
    };
    RowRaw<float, V> bias, Dv;
    bias.zero();
    Dv.zero();
    if (const int c = (tid % VPR) * V; c < k.n) {
        if (a.opts.bias) bias.load(a.opts.bias + k.first + c, k.n - c);
        if (OUT && a.D) Dv.load(a.D + k.first + c, k.n - c);
    }

    // What GR tokens from the t-th of the tile at hand on need: B and C (past the tile,
    // the next one's; the buffer has a tile to spare at its end), the step sizes and,
    // for the adjoint, the gradients (past the tile, any).
    constexpr int GR = 16 / NS;
    SelBC bcv[2][GR][NS / 4];
    float2 dv[2][GR];
    float gv[2][GR];
    auto scalars = [&](int t, int s) {
#pragma unroll
        for (int u = 0; u < GR; ++u)
#pragma unroll
            for (int i = 0; i < NS / 4; ++i) bcv[s][u][i] = bc[(t + u) * (NK / 4) + i];
    };
    auto steps = [&](int t, int s) {
        const int r = t % TILE;
#pragma unroll
        for (int u = 0; u < GR; ++u) {
            dv[s][u] = du[(r + u) * CH + ch];
            if (ADJ) gv[s][u] = ys[(r + u) * CH + ch];
        }
    };

    fetch(t_begin, 0, 0);
    scalars(0, 0);
    auto tile = [&](int t0, int p) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
            const bool in = t0 + r < t_end;  // rows past the end do not move the state
            if (r < TILE) {
                float d[V];
#pragma unroll
                for (int e = 0; e < V; ++e) d[e] = dr[p][i].get(e) + bias.get(e);
                sel_steps(a.opts, d, in);
#pragma unroll
                for (int e = 0; e < V; ++e) du[r * CH + c + e] = make_float2(d[e], d[e] * xr[p][i].get(e));
                if constexpr (ADJ) {
                    float g[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) g[e] = yr[p][i].get(e);
                    if (gate)
#pragma unroll
                        for (int e = 0; e < V; ++e) g[e] *= silu_f32(zr[p][i].get(e));
#pragma unroll
                    for (int e = 0; e < V; ++e) ys[r * CH + c + e] = g[e];
                }
            }
        }
        __syncthreads();
        steps(0, 0);
        if (t0 + TILE < t_end) fetch(t0, TILE, p ^ 1);
        const int nt = min(TILE, t_end - t0);
        for (int tb = 0; tb < nt; tb += U) {
            if constexpr (BACK)
                if (tb % KEEP == 0 && live) {
                    const size_t at = (size_t)k.b * a.keeps + (t0 + tb) / KEEP;
                    lane_store(a.keep_state + seg_at(at), E, h);
                    if (ws == 0) a.keep_sum[at * E + k.first + ch] = dsum;
                }
#pragma unroll
            for (int g = 0; g < U; g += GR) {
                // The next tokens' operands set out while these are used. Scalar loads
                // come back in any order, so whoever uses one waits for all under way:
                // these have to be here before the next are sent for.
                const int s = g / GR % 2;
                __builtin_amdgcn_sched_barrier(0);
                wait_lgkm();
                scalars(tb + g + GR, s ^ 1);
                steps(tb + g + GR, s ^ 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int u = 0; u < GR; ++u) {
                    const int t = tb + g + u;
                    const float2 d = dv[s][u];
                    const float dyv = ADJ ? gv[s][u] : 0.0f;
                    float yv = 0.0f;
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const SelBC v = bcv[s][u][i / 4];
                        const float decay = __builtin_amdgcn_exp2f(d.x * A2[i]);
                        h[i] = fmaf(decay, h[i], d.y * v[i % 4]);
                        if constexpr (OUT) yv = fmaf(v[4 + i % 4], h[i], yv);
                        if constexpr (ADJ) {
                            P[i] *= decay;
                            G[i] = fmaf(P[i], dyv * v[4 + i % 4], G[i]);
                        }
                    }
                    if constexpr (OUT) ys[(ws * TILE + t) * CH + ch] = yv;
                    else dsum += d.x;
                }
            }
        }
        __syncthreads();
        if constexpr (OUT) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
                if (r < nt && c < k.n) {
                    float o[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float s = ys[r * CH + c + e];
#pragma unroll
                        for (int j = 1; j < WS; ++j) s += ys[(j * TILE + r) * CH + c + e];
                        o[e] = fmaf(Dv.get(e), xr[p][i].get(e), s);
                    }
                    if (gate)
#pragma unroll
                        for (int e = 0; e < V; ++e) o[e] *= silu_f32(zr[p][i].get(e));
                    row_store(row_at(y, yo[i]), o, k.n - c);
                }
            }
        }
        x += TILE * a.x_token;
        dt += TILE * a.dt_token;
        if (gate) z += TILE * a.z_token;
        if (ADJ) dy += TILE * E;
        if (OUT) y += TILE * E;
        bc += TILE * (NK / 4);
    };
    for (int t0 = t_begin; t0 < t_end; t0 += 2 * TILE) {
        tile(t0, 0);
        if (t0 + TILE < t_end) tile(t0 + TILE, 1);
    }

    if constexpr (!OUT) {
        if (!live) return;
        const size_t at = (size_t)k.b * (a.segs - 1) + k.seg;
        if (k.seg < a.segs - 1) {
            lane_store(a.seg_state + seg_at(at), E, h);
            if (ws == 0) a.seg_sum[at * E + k.first + ch] = dsum;
        }
        if constexpr (ADJ)
            if (k.seg > 0) {
                if (k.seg == a.segs - 1 && a.dfinal && nn > 0) {
                    RowRaw<float, NS> r;
                    r.load(a.dfinal + ((size_t)k.b * E + k.first + ch) * N + n0, nn);
#pragma unroll
                    for (int i = 0; i < NS; ++i) G[i] = fmaf(P[i], r.get(i), G[i]);
                }
                lane_store(a.seg_adj + seg_at(at - 1), E, G);
            }
    } else if (a.final_state && last_seg && nn > 0) {
        row_store(a.final_state + ((size_t)k.b * E + k.first + ch) * N + n0, h, nn);
    }
}

// Sum over the SL neighbouring lanes, in each of them: DPP moves within a row
// of 16 lanes (neighbour, neighbour pair, half row, row).
template <int SL> __device__ __forceinline__ float lanes_sum(float v) {
    auto add = [](float a, int b) { return a + __int_as_float(b); };
    if constexpr (SL >= 2) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));
    if constexpr (SL >= 4) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));
    if constexpr (SL >= 8) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));
    if constexpr (SL >= 16) v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));
    return v;
}

// One token. Bound by the float32 state, read once and written once: a lane
// takes 4 states (16 bytes), neighbours the rest of the channel.
template <typename T, int NK>
__global__ __launch_bounds__(256) void selective_step_kernel(SelArgs a, float *__restrict__ state,
                                                             long long items) {
    constexpr int SL = NK / 4;  // lanes per channel
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
        h[i] = fmaf(__builtin_amdgcn_exp2f(d * (sel_rate(Ar.get(i)))), hr.get(i), u * Br.get(i));
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

template <typename T, int NK> hipError_t sel_bc(const SelArgs &a, hipStream_t stream) {
    const size_t count = (size_t)a.batch * a.ngroups * sel_padded(a.seqlen) * 2 * NK;
    selective_bc_kernel<T, NK><<<static_cast<unsigned>((count + 255) / 256), 256, 0, stream>>>(a, count);
    return hipGetLastError();
}

template <typename T, int NK> hipError_t sel_fwd(const SelArgs &a, hipStream_t stream) {
    hipError_t e = sel_bc<T, NK>(a, stream);
    const int cut = a.units - a.whole;
    if (e == hipSuccess && a.segs > 1) {
        selective_fwd_kernel<T, NK, SEL_STATE>
            <<<static_cast<unsigned>(cut * (a.segs - 1)), 256, 0, stream>>>(a);
        e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
    selective_fwd_kernel<T, NK, SEL_OUT>
        <<<static_cast<unsigned>(a.whole + cut * a.segs), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int NK> hipError_t sel_keep_launch(const SelArgs &a, hipStream_t stream) {
    const hipError_t e = sel_bc<T, NK>(a, stream);
    if (e != hipSuccess) return e;
    const unsigned grid = a.units * a.segs;
    constexpr int threads = SelShape<NK, true>::THREADS;
    if (a.segs > 1) selective_fwd_kernel<T, NK, SEL_BOTH><<<grid, threads, 0, stream>>>(a);
    else selective_fwd_kernel<T, NK, SEL_KEEP><<<grid, threads, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int NK>
hipError_t sel_step_launch(const SelArgs &a, float *state, hipStream_t stream) {
    const long long items = (long long)a.batch * a.channels * (NK / 4);
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

static int selective_ch(int dstate) {
    const int nk = selective_kernel_dstate(dstate);
    return nk <= 16 ? 1024 / nk : 64;
}

int selective_blocks(int channels, int ngroups, int dstate) {
    const int ch = selective_ch(dstate), each = channels / ngroups;
    return ngroups * ((each + ch - 1) / ch);
}

// Units from the `whole`-th on cut along the token axis into at most `most`
// segments, whole tiles to a segment and two at least.
static SelPlan sel_cut(int batch, int seqlen, int channels, int ngroups, int dstate, int whole,
                       long long most) {
    const int nk = selective_kernel_dstate(dstate), tile = 2048 / selective_ch(dstate);
    const int units = static_cast<int>((long long)batch * selective_blocks(channels, ngroups, dstate));
    const int tiles = (seqlen + tile - 1) / tile;
    long long s = most;
    if (s > tiles / 2) s = tiles / 2;
    if (s > 128) s = 128;  // every segment folds the ones before it
    SelPlan p{units, whole, 1, seqlen, 0};
    if (s > 1) {
        const int per = static_cast<int>((tiles + s - 1) / s);
        p.seg_len = per * tile;
        p.segs = (seqlen + p.seg_len - 1) / p.seg_len;
    }
    if (p.segs <= 1) p = SelPlan{units, 0, 1, seqlen, 0};
    p.seg_floats = (size_t)batch * (p.segs - 1) * channels * nk;
    return p;
}

// Cut forward, a walk costs two passes, so it pays only while the uncut walks
// leave CUs without work: with fewer workgroups than CUs all are cut, and with
// few more than a multiple of the CUs (up to four times) those few, so that they
// spread over all CUs instead of doubling the work of some. Measured with 16
// states and 2048 tokens in bf16: 80 workgroups 297 us uncut, 111 in 24 segments;
// 160 299 and 186 (in 16); 260 301 and 249 (four of them in 8); 320 327 and 281
// (64 in 8; in 4 or 16 within 4 us of that); 640 443 and 386 (128 in 4).
SelPlan selective_plan(int batch, int seqlen, int channels, int ngroups, int dstate) {
    constexpr long long CUS = 256;
    const long long units = (long long)batch * selective_blocks(channels, ngroups, dstate);
    if (units < CUS) return sel_cut(batch, seqlen, channels, ngroups, dstate, 0, 2048 / units);
    const long long rest = units % CUS;
    if (units < 4 * CUS && rest > 0 && rest <= CUS / 2)
        return sel_cut(batch, seqlen, channels, ngroups, dstate, static_cast<int>(units - rest),
                       rest <= 64 ? 8 : 512 / rest);
    return sel_cut(batch, seqlen, channels, ngroups, dstate, 0, 1);
}

// The backward's first walk is made either way, so cutting costs it little and
// evens out the load; 2048 are four rounds of the two workgroups that a CU
// holds. Measured as above: 640 workgroups 2543 us uncut, 1979 in 3 segments,
// 1892 in 8; 320 1624 and 972 (in 6; 1106 in 4, whose last round is half
// empty); 160 1400 and 523 (in 12); 80 1369 and 296 (in 24).
SelPlan selective_bwd_plan(int batch, int seqlen, int channels, int ngroups, int dstate) {
    const long long units = (long long)batch * selective_blocks(channels, ngroups, dstate);
    return sel_cut(batch, seqlen, channels, ngroups, dstate, 0, 2048 / units);
}

size_t selective_bc_floats(int batch, int seqlen, int ngroups, int dstate) {
    return ((size_t)batch * ngroups * sel_padded(seqlen) + kSelPad) * 2 * selective_kernel_dstate(dstate);
}

hipError_t launch_selective_fwd(const SelArgs &a, bool bf16, hipStream_t stream) {
    SSD_SEL_DISPATCH(sel_fwd, a, stream)
}
hipError_t launch_selective_keep(const SelArgs &a, bool bf16, hipStream_t stream) {
    SSD_SEL_DISPATCH(sel_keep_launch, a, stream)
}
hipError_t launch_selective_step(const SelArgs &a, float *state, bool bf16, hipStream_t stream) {
    SSD_SEL_DISPATCH(sel_step_launch, a, state, stream)
}

}  // namespace ssd
