// Backward of the selective scan. With q_t[n] = exp(dt_t A[n]) h_{t-1}[n], the
// adjoint runs back in time:
//   g_t[n] = dy_t C_t[n] + exp(dt_{t+1} A[n]) g_{t+1}[n]      (dy after the gate's silu(z))
//   dx_t = dt_t sum_n g_t B_t + D dy_t,  ddt_t = sum_n g_t (x_t B_t + A q_t),
//   dA[n] = sum_t dt_t g_t q_t,  dB_t = sum_e dt_t x_t g_t,  dC_t = sum_e dy_t h_t,
//   dz_t = dy'_t (sum_n C_t h_t + D x_t) silu'(z_t),  ddt then through softplus and clamp.
//
// States are recomputed, not stored by the forward: a first walk (the
// forward's, SEL_KEEP) keeps the state before every 16 tokens (4 or 8 at other
// state sizes), and the walk back rebuilds a tile's states in registers from
// there, with their decays, then runs the adjoint over them. Channels and
// states lie over lanes and wavefronts as in the forward. Bound by vector
// issue, of which the rebuilding is a quarter. Measured in bf16 at 4 x 2048
// tokens of 5120 channels and 16 states: first walk 227 us, walk back 640 us
// (vector units busy 81% of the time, two workgroups to a CU by their registers
// and LDS), partial dB and dC 15 us; with 32 states 404, 1463 and 33 us, with 64, where
// a state is kept every 4 tokens, 878, 3047 and 130 us; float32, 2 x 777 tokens of 1000
// channels and 24 states: 24, 68 and 5 us (segments of 96 tokens, see the forward).
//
// What the first walk keeps is 4 bytes per (token, channel) at 16 states, 16 at 32 and
// 64 at 64: 4 x 2048 tokens of 5120 channels take a workspace of 0.29, 0.91 and 3.5 GB.
//
// Sums over channels (dB, dC) are sums over lanes, of eight values per token
// and four states: three steps swap halves between registers, so that each
// leaves half the values, spread over half the lanes, and three more add up the
// eight lanes that then hold a value: 24 instructions, where eight butterflies
// over 64 lanes take 96, and no LDS (through which the same took as long, and
// 11% of the time in bank conflicts). Workgroups meet in partial tensors that are
// added in a fixed order. Sums over tokens (dA, dD, the bias) stay in
// registers and end in partial rows the same way.
//
// With segments (see the forward) the first walk also makes every segment's
// adjoint from zero, and a walk back starts by folding the segments after its own.
#include "selective.h"

namespace ssd {

namespace {

// Tokens of a row of dbc_part, and the rows a sequence and group take: every
// row holds 64 values per four states, dB of each state for 8 tokens, then dC.
template <int NK> constexpr int sel_row_tokens() { return sel_keep<NK>() < 8 ? sel_keep<NK>() : 8; }

template <typename T, int NK, bool GATE>
__global__ __launch_bounds__((SelShape<NK, true>::THREADS), 2) void selective_bwd_kernel(SelBwdArgs ba) {
    using S = SelShape<NK, true>;
    constexpr int NS = S::NS, WS = S::WS, CH = S::CH, THREADS = S::THREADS, TB = sel_keep<NK>(), V = 4;
    constexpr int VPR = CH / V, IT = (TB * VPR + THREADS - 1) / THREADS, TOK = sel_row_tokens<NK>();
    __shared__ float2 du[TB * CH];        // (dt, dt x)
    __shared__ float dys[TB * CH];        // dy silu(z)
    __shared__ float2 pg[WS * TB * CH];   // each wavefront's sum_n (g B), sum_n (A2 g q)
    __shared__ float py[GATE ? WS * TB * CH : 1];  // and sum_n (C h)
    // the channels' bias and D, which the walk leaves no registers for
    __shared__ __attribute__((aligned(16))) float biases[CH], Ds[CH];
    __shared__ float tr[2 * THREADS * V];  // after the last tile every lane's dD and bias sums

    const SelArgs &a = ba.f;
    const SelBlock k = sel_block<CH>(blockIdx.x % a.units, blockIdx.x / a.units, a.channels, a.ngroups);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ws = w % WS, ch = w / WS * 64 + lane, n0 = ws * NS;
    const int N = a.dstate, E = a.channels, L = a.seqlen;
    // this lane's states of scratch row `at`
    auto seg_at = [&](size_t at) { return (at * (NK / 4) + n0 / 4) * E * 4 + (size_t)(k.first + ch) * 4; };
    const bool live = ch < k.n;
    const int nn = live ? N - n0 : 0;
    const int t_begin = k.seg * a.seg_len, t_end = min(L, t_begin + a.seg_len);
    const int t_last = t_begin + (t_end - t_begin - 1) / TB * TB;  // the first tile walked
    // rows of the tile at hand
    const T *x = static_cast<const T *>(a.x) + k.b * a.x_batch + k.first + t_last * a.x_token;
    const T *dt = static_cast<const T *>(a.dt) + k.b * a.dt_batch + k.first + t_last * a.dt_token;
    const T *z = GATE ? static_cast<const T *>(a.z) + k.b * a.z_batch + k.first + t_last * a.z_token : nullptr;
    size_t dense = ((size_t)k.b * L + t_last) * E + k.first;  // in dy and the outputs
    sel_const *q = (sel_const *)(a.bc + ((size_t)(k.b * a.ngroups + k.g) * sel_padded(L) + t_last) * 2 * NK +
                                 ws * 2 * NS);

    float A2[NS], h_in[NS], ag[NS], dA[NS];
    load_rates(a.A + (size_t)(k.first + ch) * N + n0, nn, A2);
    {
        RowRaw<float, NS> r;
        r.zero();
        if (k.seg == a.segs - 1 && a.dfinal && nn > 0)
            r.load(a.dfinal + ((size_t)k.b * E + k.first + ch) * N + n0, nn);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            ag[i] = r.get(i);
            h_in[i] = dA[i] = 0.0f;
        }
    }
    if (live) {
        const size_t at = (size_t)k.b * (a.segs - 1), e = k.first + ch;
        sel_fold<NK>(a.seg_state + seg_at(at), a.seg_sum + at * E + e, 1, E, k.seg, A2, h_in);
        // the gradients of the states entering the segments behind, from the last one on
        if (k.seg < a.segs - 1)
            sel_fold<NK>(a.seg_adj + seg_at(at + a.segs - 2), a.seg_sum + (at + a.segs - 1) * E + e, -1, E,
                         a.segs - 1 - k.seg, A2, ag);
    }

    float dD[V], db[V];
    for (int c = tid; c < CH; c += THREADS) {
        biases[c] = a.opts.bias && c < k.n ? a.opts.bias[k.first + c] : 0.0f;
        Ds[c] = a.D && c < k.n ? a.D[k.first + c] : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) dD[e] = db[e] = 0.0f;
    // this wavefront's rows of dbc_part
    const int part = k.block * (CH / 64) + w / WS;
    float *rows = ba.dbc_part + (((size_t)part * a.batch + k.b) * a.ngroups + k.g) *
                                    ((L + TOK - 1) / TOK) * (NK / 4) * 64;

    // A tile's rows and the state before it. The next tile's rows set out halfway back,
    // when half the tile's states are done with (in float32, and at 64 states, only when
    // all are: the registers would not do), its state when the walk is done.
    constexpr bool EARLY = sizeof(T) == 2 && NK <= 32;
    RowRaw<T, V> xr[IT], zr[IT], yr[IT], dr[IT];
    float hk[NS], hsum = 0.0f;
    uint32_t xo[IT], dto[IT], zo[IT], yo[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
        xo[i] = row_offset<T>(r, a.x_token, c);
        dto[i] = row_offset<T>(r, a.dt_token, c);
        zo[i] = row_offset<T>(r, a.z_token, c);
        yo[i] = row_offset<T>(r, E, c);
    }
    auto fetch = [&](int t0, size_t dense, RowRaw<T, V>(&xr)[IT], RowRaw<T, V>(&dr)[IT], RowRaw<T, V>(&zr)[IT],
                     RowRaw<T, V>(&yr)[IT]) {
        const T *dy = static_cast<const T *>(a.dy) + dense;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
            xr[i].zero();
            dr[i].zero();
            zr[i].zero();
            yr[i].zero();
            if (r < TB && t0 + r < t_end && c < k.n) {
                xr[i].load(row_at(x, xo[i]), k.n - c);
                dr[i].load(row_at(dt, dto[i]), k.n - c);
                if (GATE) zr[i].load(row_at(z, zo[i]), k.n - c);
                yr[i].load(row_at(dy, yo[i]), k.n - c);
            }
        }
    };
    auto state = [&](int t0) {
#pragma unroll
        for (int i = 0; i < NS; ++i) hk[i] = 0.0f;
        if (live) {
            const size_t at = (size_t)k.b * a.keeps + t0 / TB;
            lane_load(a.keep_state + seg_at(at), E, hk);
            if (k.seg) hsum = a.keep_sum[at * E + k.first + ch];
        }
    };
    fetch(t_last, dense, xr, dr, zr, yr);
    state(t_last);
    for (int t0 = t_last; t0 >= t_begin; t0 -= TB) {
        const int nt = min(TB, t_end - t0);
        if (k.seg)
#pragma unroll
            for (int i = 0; i < NS; ++i)
                hk[i] = fmaf(__builtin_amdgcn_exp2f(A2[i] * hsum), h_in[i], hk[i]);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
            if (r < TB) {
                float d[V];
#pragma unroll
                for (int e = 0; e < V; ++e) d[e] = dr[i].get(e) + biases[c + e];
                sel_steps(a.opts, d, r < nt);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    du[r * CH + c + e] = make_float2(d[e], d[e] * xr[i].get(e));
                    dys[r * CH + c + e] = GATE ? yr[i].get(e) * silu_f32(zr[i].get(e)) : yr[i].get(e);
                }
            }
        }
        __syncthreads();

        // B and C of GR tokens at a time, the next ones on their way while these
        // are used (one in float32 at 16 states, where two would spill)
        constexpr int GR = NS == 4 && (sizeof(T) == 2 || NK != 16) ? 2 : 1;
        SelBC bcv[2][GR][NS / 4];
        float2 dv[2][GR];
        float gv[2][GR];
        auto operands = [&](int t, int s, bool back) {
#pragma unroll
            for (int u = 0; u < GR; ++u) {
#pragma unroll
                for (int i = 0; i < NS / 4; ++i) bcv[s][u][i] = q[(t + u) * (NK / 4) + i];
                dv[s][u] = du[(t + u) * CH + ch];
                if (back) gv[s][u] = dys[(t + u) * CH + ch];
            }
        };
        float h[TB][NS], dec[TB][NS], res[NS / 4];
        operands(0, 0, false);
#pragma unroll
        for (int tg = 0; tg < TB; tg += GR) {
            const int s = tg / GR % 2;
            if (tg + GR < TB) operands(tg + GR, s ^ 1, false);
            else operands(TB - GR, s, true);  // the walk back begins where this one ends
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < GR; ++u) {
                const int t = tg + u;
                const float2 d = dv[s][u];
                float y = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    dec[t][i] = __builtin_amdgcn_exp2f(d.x * A2[i]);
                    h[t][i] = fmaf(dec[t][i], t ? h[t - 1][i] : hk[i], d.y * bcv[s][u][i / 4][i % 4]);
                    if constexpr (GATE) y = fmaf(bcv[s][u][i / 4][4 + i % 4], h[t][i], y);
                }
                if constexpr (GATE) py[(ws * TB + t) * CH + ch] = y;
            }
        }
        RowRaw<T, V> xn[IT], zn[IT], yn[IT], dn[IT];
        auto fetch_next = [&]() {
            x -= TB * a.x_token;
            dt -= TB * a.dt_token;
            if (GATE) z -= TB * a.z_token;
            fetch(t0 - TB, dense - (size_t)TB * E, xn, dn, zn, yn);
        };
        // not a constant of the loop: eight lane masks would be kept for the comparisons below
        const int turn = ragged(lane & 7);
        // The sums over the lanes of a token's eight values with four states. Each of the
        // first three steps halves the lanes that a value is spread over and with them the
        // values that a lane holds; lane 8 v + u ends with value v and keeps it for the
        // row's u-th token.
        auto sums = [&](int t, int s4, const float (&v)[8]) {
            auto add = [](float x, int o) { return x + __int_as_float(o); };
            float p[4], q2[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[j]), __float_as_uint(v[j + 4]), false, false);
                p[j] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(p[j]), __float_as_uint(p[j + 2]), false, false);
                q2[j] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
            }
            const bool odd = lane & 8;
            const float send = odd ? q2[0] : q2[1];
            float sum = add(odd ? q2[1] : q2[0],
                            __builtin_amdgcn_update_dpp(0, __float_as_int(send), 0x128, 0xf, 0xf, true));
            sum = add(sum, __builtin_amdgcn_update_dpp(0, __float_as_int(sum), 0xB1, 0xf, 0xf, true));
            sum = add(sum, __builtin_amdgcn_update_dpp(0, __float_as_int(sum), 0x4E, 0xf, 0xf, true));
            sum = add(sum, __builtin_amdgcn_update_dpp(0, __float_as_int(sum), 0x141, 0xf, 0xf, true));
            if (t % TOK == TOK - 1) res[s4] = sum;
            else res[s4] = turn == t % TOK ? sum : res[s4];
            if (t % TOK == 0 && t < nt)  // nt: rows past the sequence's are another's
                rows[((size_t)(t0 + t) / TOK * (NK / 4) + n0 / 4 + s4) * 64 + lane] = res[s4];
        };
#pragma unroll
        for (int tg = TB - GR; tg >= 0; tg -= GR) {
            const int s = tg / GR % 2;
            if (tg) operands(tg - GR, s ^ 1, true);
            if (EARLY && tg == TB / 2 && t0 > t_begin) fetch_next();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = GR - 1; u >= 0; --u) {
                const int t = tg + u;
                const float2 d = dv[s][u];
                const float dyv = gv[s][u];
                float gB = 0.0f, gA = 0.0f;
#pragma unroll
                for (int s4 = 0; s4 < NS / 4; ++s4) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = s4 * 4 + j;
                        const float g = fmaf(dyv, bcv[s][u][i / 4][4 + i % 4], ag[i]);
                        gB = fmaf(g, bcv[s][u][i / 4][i % 4], gB);
                        ag[i] = dec[t][i] * g;
                        const float gq = ag[i] * (t ? h[t - 1][i] : hk[i]);
                        gA = fmaf(A2[i], gq, gA);
                        dA[i] = fmaf(d.x, gq, dA[i]);
                        v[j] = d.y * g;
                        v[4 + j] = dyv * h[t][i];
                    }
                    sums(t, s4, v);
                }
                pg[(ws * TB + t) * CH + ch] = make_float2(gB, gA);
            }
        }
        T *const dx = static_cast<T *>(ba.dx) + dense, *const ddt = static_cast<T *>(ba.ddt) + dense;
        T *const dz = GATE ? static_cast<T *>(ba.dz) + dense : nullptr;
        if (t0 > t_begin) {
            if (!EARLY) fetch_next();
            dense -= (size_t)TB * E;
            q -= TB * (NK / 4);
            state(t0 - TB);
        }
        __syncthreads();

#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int id = tid + i * THREADS, r = id / VPR, c = (id % VPR) * V;
            if (r < nt && c < k.n) {
                float ox[V], ot[V], oz[V], raws[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int at = r * CH + c + e;
                    float sB = pg[at].x, sA = pg[at].y;
#pragma unroll
                    for (int j = 1; j < WS; ++j) {
                        sB += pg[j * TB * CH + at].x;
                        sA += pg[j * TB * CH + at].y;
                    }
                    const float xv = xr[i].get(e), raw = dr[i].get(e) + biases[c + e], dyg = dys[at];
                    ox[e] = fmaf(du[at].x, sB, Ds[c + e] * dyg);
                    raws[e] = raw;
                    ot[e] = fmaf(xv, sB, sA * 0.6931471805599453f);
                    dD[e] = fmaf(dyg, xv, dD[e]);  // zero past the last channel
                    if constexpr (GATE) {
                        float y = py[at];
#pragma unroll
                        for (int j = 1; j < WS; ++j) y += py[j * TB * CH + at];
                        oz[e] = yr[i].get(e) * fmaf(Ds[c + e], xv, y) * silu_grad_f32(zr[i].get(e));
                    }
                }
                if (a.opts.clamp)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float free = a.opts.softplus ? softplus_f32(raws[e]) : raws[e];
                        if (free < a.opts.lo || free > a.opts.hi) ot[e] = 0.0f;
                    }
                if (a.opts.softplus)
#pragma unroll
                    for (int e = 0; e < V; ++e) ot[e] *= sigmoid_f32(raws[e]);
#pragma unroll
                for (int e = 0; e < V; ++e) db[e] += ot[e];
                row_store(row_at(dx, yo[i]), ox, k.n - c);
                row_store(row_at(ddt, yo[i]), ot, k.n - c);
                if constexpr (GATE) row_store(row_at(dz, yo[i]), oz, k.n - c);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            xr[i] = xn[i];
            dr[i] = dn[i];
            zr[i] = zn[i];
            yr[i] = yn[i];
        }
    }

    const size_t unit = (size_t)k.b * a.segs + k.seg;
    if (nn > 0) {
        row_store(ba.dA_part + (unit * E + k.first + ch) * N + n0, dA, nn);
        if (ba.dinit && k.seg == 0)
            row_store(ba.dinit + ((size_t)k.b * E + k.first + ch) * N + n0, ag, nn);
    }
    // dD and the bias: a channel's sums lie in the lanes of its column
#pragma unroll
    for (int e = 0; e < V; ++e) {
        tr[tid * V + e] = dD[e];
        tr[THREADS * V + tid * V + e] = db[e];
    }
    __syncthreads();
    for (int c = tid; c < k.n; c += THREADS) {
        float s0 = 0.0f, s1 = 0.0f;
        for (int r = c / V; r < THREADS; r += VPR) {
            s0 += tr[r * V + c % V];
            s1 += tr[THREADS * V + r * V + c % V];
        }
        ba.de_part[(unit * 2) * E + k.first + c] = s0;
        ba.de_part[(unit * 2 + 1) * E + k.first + c] = s1;
    }
}

// dB and dC: sums of the workgroups' rows, in order; `per` rows' values in one part.
template <typename T, int NK>
__global__ __launch_bounds__(256) void selective_dbc_kernel(const float *__restrict__ parts, int n,
                                                            size_t per, int L, int G, int N,
                                                            T *__restrict__ dB, T *__restrict__ dC) {
    constexpr int TOK = sel_row_tokens<NK>();
    const size_t id = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= per) return;
    const int v = (id >> 3) & 7, u = id & 7;
    const size_t row = id / 64;
    const int state = static_cast<int>(row % (NK / 4)) * 4 + (v & 3);
    const size_t at = row / (NK / 4), chunks = (L + TOK - 1) / TOK;
    const size_t t = at % chunks * TOK + u, bg = at / chunks;
    if (u >= TOK || t >= (size_t)L || state >= N) return;
    float s = 0.0f;
#pragma unroll 8
    for (int p = 0; p < n; ++p) s += parts[p * per + id];
    (v >> 2 ? dC : dB)[((bg / G * L + t) * G + bg % G) * N + state] = from_f32<T>(s);
}

template <int NK> size_t sel_dbc_part(int batch, int seqlen, int ngroups) {
    constexpr int TOK = sel_row_tokens<NK>();
    return (size_t)batch * ngroups * ((seqlen + TOK - 1) / TOK) * (NK / 4) * 64;
}

template <typename T, int NK> hipError_t sel_bwd(const SelBwdArgs &ba, hipStream_t stream) {
    const SelArgs &a = ba.f;
    const int blocks = selective_blocks(a.channels, a.ngroups, a.dstate);
    hipError_t e = launch_selective_keep(a, sizeof(T) == 2, stream);
    if (e != hipSuccess) return e;
    const unsigned grid = static_cast<unsigned>(a.units * a.segs);
    if (a.z) selective_bwd_kernel<T, NK, true><<<grid, SelShape<NK, true>::THREADS, 0, stream>>>(ba);
    else selective_bwd_kernel<T, NK, false><<<grid, SelShape<NK, true>::THREADS, 0, stream>>>(ba);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const size_t per = sel_dbc_part<NK>(a.batch, a.seqlen, a.ngroups);
    selective_dbc_kernel<T, NK><<<static_cast<unsigned>((per + 255) / 256), 256, 0, stream>>>(
        ba.dbc_part, blocks / a.ngroups * (SelShape<NK, true>::CH / 64), per, a.seqlen, a.ngroups, a.dstate,
        static_cast<T *>(ba.dB), static_cast<T *>(ba.dC));
    e = hipGetLastError();
    const int units = a.batch * a.segs;
    const long long en = (long long)a.channels * a.dstate;
    if (e == hipSuccess) e = launch_colsum(ba.dA_part, units, en, en, ba.dA, nullptr, stream);
    if (e == hipSuccess && (ba.dD || ba.ddt_bias))
        e = launch_colsum(ba.de_part, units, 2LL * a.channels, a.channels, ba.dD, ba.ddt_bias, stream);
    return e;
}

}  // namespace

template <int NK> static size_t sel_dbc_floats(int batch, int seqlen, int ngroups, int blocks) {
    return sel_dbc_part<NK>(batch, seqlen, ngroups) * (blocks / ngroups) * (SelShape<NK, true>::CH / 64);
}

size_t selective_dbc_floats(int batch, int seqlen, int channels, int ngroups, int dstate) {
    const int blocks = selective_blocks(channels, ngroups, dstate);
    switch (selective_kernel_dstate(dstate)) {
        case 4: return sel_dbc_floats<4>(batch, seqlen, ngroups, blocks);
        case 8: return sel_dbc_floats<8>(batch, seqlen, ngroups, blocks);
        case 16: return sel_dbc_floats<16>(batch, seqlen, ngroups, blocks);
        case 32: return sel_dbc_floats<32>(batch, seqlen, ngroups, blocks);
        default: return sel_dbc_floats<64>(batch, seqlen, ngroups, blocks);
    }
}

template <int NK>
static bool sel_bwd_grid_ok(int batch, int seqlen, int channels, int ngroups, int dstate, int segs) {
    const long long units = (long long)batch * selective_blocks(channels, ngroups, dstate) * segs;
    return units < (1LL << 32) / SelShape<NK, true>::THREADS &&
           (sel_dbc_part<NK>(batch, seqlen, ngroups) + 255) / 256 < (1u << 24) &&
           colsum_grid_ok(batch * segs, (long long)channels * dstate, false) &&
           colsum_grid_ok(batch * segs, 2LL * channels, false);
}

bool selective_bwd_grid_ok(int batch, int seqlen, int channels, int ngroups, int dstate, int segs) {
    switch (selective_kernel_dstate(dstate)) {
        case 4: return sel_bwd_grid_ok<4>(batch, seqlen, channels, ngroups, dstate, segs);
        case 8: return sel_bwd_grid_ok<8>(batch, seqlen, channels, ngroups, dstate, segs);
        case 16: return sel_bwd_grid_ok<16>(batch, seqlen, channels, ngroups, dstate, segs);
        case 32: return sel_bwd_grid_ok<32>(batch, seqlen, channels, ngroups, dstate, segs);
        default: return sel_bwd_grid_ok<64>(batch, seqlen, channels, ngroups, dstate, segs);
    }
}

int selective_keep_tokens(int dstate) {
    switch (selective_kernel_dstate(dstate)) {
        case 4: return sel_keep<4>();
        case 8: return sel_keep<8>();
        case 16: return sel_keep<16>();
        case 32: return sel_keep<32>();
        default: return sel_keep<64>();
    }
}

hipError_t launch_selective_bwd(const SelBwdArgs &ba, bool bf16, hipStream_t stream) {
    const SelArgs &a = ba.f;
    SSD_SEL_DISPATCH(sel_bwd, ba, stream)
}

}  // namespace ssd
