// Gated linear recurrence with one state per channel:
//   h_t = a_t h_{t-1} + u_t,  y_t = h_t  or  h_t silu(z_t)
// gated:  log a_t = -c softplus(decay) sigmoid(r_t),  u_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t
// direct: log a_t = r_t,  u_t = x_t.
// Forward walk, single tokens and the plan; recurrence.h has the layout.
//
// The inputs are read once: a tile's tokens stay in registers between the map that they
// make and the states that the entering state gives them. What the vector unit does for an
// element (three exponentials, two reciprocals, a square root, each four
// cycles of a wavefront's issue, and some 20 others) takes about as long as
// its 8 bytes take from memory, so neither waits for long.
#include "recurrence.h"

namespace ssd {

namespace {

// What tokens of a packed axis are: bit 0, the first of its sequence; above, 1 + the
// number of the sequence whose last token it is; kRecNone: in no sequence. `final`: set to
// the state of an empty sequence. Any contents of `cu` are read within its nseq + 1 entries.
__global__ __launch_bounds__(256) void rec_token_kernel(const int *__restrict__ cu, int nseq, int L,
                                                        int *__restrict__ token, float *__restrict__ final,
                                                        long long finals) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x, all = (long long)gridDim.x * 256;
    if (final)
        for (long long k = id; k < finals; k += all) final[k] = 0.0f;
    for (long long t = id; t < L; t += all) {
        int lo = 0, hi = nseq;  // the last sequence that begins at or before t
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int from = cu[lo], to = cu[lo + 1];
        token[t] = t < from || t >= to ? kRecNone : (from == t ? 1 : 0) | (to - 1 == t ? 2 * (lo + 1) : 0);
    }
}

// Tokens of a strand: float32 operands of 8 do not fit the registers.
template <typename T> constexpr int rec_fwd_strand() { return sizeof(T) == 2 ? 8 : 4; }

// OUT: the outputs, from the state that the segments before give. Else what a segment
// does to the state entering it: seg_a, seg_h.
template <typename T, bool GATED, bool PACKED, bool OUT>
__global__ __launch_bounds__(1024) void rec_fwd_kernel(RecArgs a) {
    constexpr int S = rec_fwd_strand<T>();
    __shared__ float buf[2][16][16][4];
    const RecPlace p = rec_place(a, OUT ? a.segs : a.segs - 1);
    if (!p.live) return;
    const int tile = a.waves * 4 * S, E = a.channels;
    const size_t row0 = (size_t)p.batch * E + p.ch;
    float rate[2] = {0.0f, 0.0f}, h[2] = {0.0f, 0.0f}, A[2] = {1.0f, 1.0f};
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (e < p.nch) {
            if (GATED) rate[e] = rec_rate(a.decay[p.ch + e], a.c);
            if (OUT && a.init) h[e] = a.init[row0 + e];
            if (OUT)
                for (int s = 0; s < p.seg; ++s) {
                    const size_t k = ((size_t)p.batch * (a.segs - 1) + s) * E + p.ch + e;
                    h[e] = rec_apply<PACKED>({a.seg_a[k], a.seg_h[k]}, h[e]);
                }
        }
    const size_t xb = p.batch * a.x_batch, rb = p.batch * a.r_batch, ib = p.batch * a.i_batch, zb = p.batch * a.z_batch;
    const size_t yb = (size_t)p.batch * a.seqlen * E;
    int turn = 0;
    const bool inner = p.ch - 2 * p.col + kRecCols <= E;
    // The next tile's operands are on their way while this one's states are put together.
    RecPair<T> x[S], r[S], in[S];
    auto fetch = [&](int t0) {
        if (t0 >= p.end) return;
        const int tw = t0 + p.wave * 4 * S, nt = min(max(p.end - tw - p.sub * S, 0), S);
        auto load = [&](auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            rec_load<T, WHOLE>(r, a.r, rb + tw * a.r_token, a.r_token, p, nt);
            if (GATED) rec_load<T, WHOLE>(in, a.i, ib + tw * a.i_token, a.i_token, p, nt);
            rec_load<T, WHOLE>(x, a.x, xb + tw * a.x_token, a.x_token, p, nt);
        };
        if (inner && t0 + tile <= p.end) load(std::true_type());
        else load(std::false_type());
    };
    auto walk = [&](auto whole, int t0) {
        constexpr bool WHOLE = decltype(whole)::value;
        const int tw = t0 + p.wave * 4 * S, ts = tw + p.sub * S;
        const int nt = min(max(p.end - ts, 0), S);
        RecPair<T> z[S];
        if (OUT && a.z) rec_load<T, WHOLE>(z, a.z, zb + tw * a.z_token, a.z_token, p, nt);
        int code[S];
        if (PACKED)
#pragma unroll
            for (int j = 0; j < S; ++j) code[j] = WHOLE || j < nt ? a.token[ts + j] : 0;
        float av[S][2], uv[S][2];
        RecMap m[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
#pragma unroll
        for (int j = 0; j < S; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float d, u;
                if (GATED) {
                    const float la = rate[e] * sigmoid_f32(r[j].get(e));
                    d = __builtin_amdgcn_exp2f(la);
                    u = __builtin_amdgcn_sqrtf(one_minus_square(2.0f * kLn2 * la, d)) *
                        sigmoid_f32(in[j].get(e)) * x[j].get(e);
                } else {
                    d = __builtin_amdgcn_exp2f(kLog2e * r[j].get(e));
                    u = x[j].get(e);
                }
                if (!WHOLE && j >= nt) {
                    d = 1.0f;
                    u = 0.0f;
                }
                if (PACKED && (code[j] & 1)) d = -1.0f;
                if (PACKED && code[j] < 0) u = 0.0f;
                av[j][e] = d;
                uv[j][e] = u;
                m[e] = rec_then<PACKED>(m[e], {d, u});
            }
        fetch(t0 + tile);
        RecMap before[2], all[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) rec_wave<PACKED, false>(m[e], p.sub, before[e], all[e]);
        if (p.sub == 0) {
            float *w = buf[turn][p.wave][p.col];
            w[0] = all[0].a; w[1] = all[0].h; w[2] = all[1].a; w[3] = all[1].h;
        }
        __syncthreads();
        float hs[2] = {h[0], h[1]};
        for (int w = 0; w < a.waves; ++w) {
            const float *v = buf[turn][w][p.col];
            const RecMap mw[2] = {{v[0], v[1]}, {v[2], v[3]}};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (w == p.wave) hs[e] = h[e];
                h[e] = rec_apply<PACKED>(mw[e], h[e]);
                if (!OUT) A[e] = PACKED && (A[e] < 0.0f || mw[e].a < 0.0f) ? -1.0f : A[e] * mw[e].a;
            }
        }
        turn ^= 1;
        if (!OUT) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) hs[e] = rec_apply<PACKED>(before[e], hs[e]);
        if (a.states && ts % kRecKeep == 0 && (WHOLE || nt > 0)) {
            float *s = a.states + ((size_t)p.batch * a.keeps + ts / kRecKeep) * E + p.ch;
            if (p.nch > 0) s[0] = hs[0];
            if (p.nch > 1) s[1] = hs[1];
        }
        char *y = static_cast<char *>(a.y) + (yb + (size_t)tw * E) * sizeof(T);
        const uint32_t step = rec_bytes<T>(E);
        uint32_t off = rec_offset<T, S>(step, p);
#pragma unroll
        for (int j = 0; j < S; ++j, off += step) {
            float o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                hs[e] = rec_apply<PACKED>({av[j][e], uv[j][e]}, hs[e]);
                o[e] = hs[e];
                if (a.z) o[e] *= silu_f32(z[j].get(e));
                if (PACKED && code[j] < 0) o[e] = 0.0f;
            }
            if (a.y && (WHOLE || j < nt)) rec_store<T, WHOLE>(y, off, p.nch, o[0], o[1]);
            if (PACKED && a.final_state && (WHOLE || j < nt) && code[j] > 1) {
                float *f = a.final_state + (size_t)((code[j] >> 1) - 1) * E + p.ch;
                if (p.nch > 0) f[0] = hs[0];
                if (p.nch > 1) f[1] = hs[1];
            }
        }
    };
    int t0 = p.begin;
    fetch(t0);
    if (inner)
        for (; t0 + tile <= p.end; t0 += tile) walk(std::true_type(), t0);
    for (; t0 < p.end; t0 += tile) walk(std::false_type(), t0);
    if (p.wave || p.sub) return;
    const bool last = p.seg == a.segs - 1;
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (e < p.nch) {
            if (!OUT) {
                const size_t k = ((size_t)p.batch * (a.segs - 1) + p.seg) * E + p.ch + e;
                a.seg_a[k] = A[e];
                a.seg_h[k] = h[e];
            } else if (!PACKED && last && a.final_state) a.final_state[row0 + e] = h[e];
        }
}

// One token: a lane takes four channels of one sequence.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void rec_step_kernel(RecArgs a, float *__restrict__ state, int vecs) {
    constexpr int V = 4;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= (long long)a.batch * vecs) return;
    const int b = static_cast<int>(id / vecs), c = static_cast<int>(id - (long long)b * vecs) * V, n = a.channels - c;
    RowRaw<T, V> x, r, in, z;
    RowRaw<float, V> s, d;
    x.load(static_cast<const T *>(a.x) + b * a.x_batch + c, n);
    r.load(static_cast<const T *>(a.r) + b * a.r_batch + c, n);
    if (GATED) {
        in.load(static_cast<const T *>(a.i) + b * a.i_batch + c, n);
        d.load(a.decay + c, n);
    }
    if (a.z) z.load(static_cast<const T *>(a.z) + b * a.z_batch + c, n);
    s.load(state + (size_t)b * a.channels + c, n);
    float h[V], o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (GATED) {
            const float la = rec_rate(d.get(e), a.c) * sigmoid_f32(r.get(e)), k = __builtin_amdgcn_exp2f(la);
            h[e] = fmaf(k, s.get(e), __builtin_amdgcn_sqrtf(one_minus_square(2.0f * kLn2 * la, k)) *
                                         sigmoid_f32(in.get(e)) * x.get(e));
        } else h[e] = fmaf(__builtin_amdgcn_exp2f(kLog2e * r.get(e)), s.get(e), x.get(e));
        o[e] = a.z ? h[e] * silu_f32(z.get(e)) : h[e];
    }
    row_store(state + (size_t)b * a.channels + c, h, n);
    row_store(static_cast<T *>(a.y) + (size_t)b * a.channels + c, o, n);
}

template <typename T, bool GATED, bool PACKED> hipError_t fwd(const RecArgs &a, hipStream_t stream) {
    const int threads = a.waves * 64;
    if (a.segs > 1) {
        rec_fwd_kernel<T, GATED, PACKED, false><<<rec_grid(a, a.segs - 1), threads, 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    rec_fwd_kernel<T, GATED, PACKED, true><<<rec_grid(a, a.segs), threads, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, bool GATED> hipError_t step(const RecArgs &a, float *state, hipStream_t stream) {
    const int vecs = (a.channels + 3) / 4;
    const unsigned grid = static_cast<unsigned>(((long long)a.batch * vecs + 255) / 256);
    rec_step_kernel<T, GATED><<<grid, 256, 0, stream>>>(a, state, vecs);
    return hipGetLastError();
}

}  // namespace

// Wavefronts of a workgroup and segments of the token axis, for strands of `strand` tokens.
static RecPlan rec_plan(int batch, int seqlen, int channels, int strand, int most_waves) {
    RecPlan p;
    p.blocks = (channels + kRecCols - 1) / kRecCols;
    const long long units = (long long)batch * p.blocks;
    const int wanted = (seqlen + 4 * strand - 1) / (4 * strand);  // wavefronts that have tokens
    p.waves = units >= 512 ? 4 : units >= 128 ? 8 : 16;
    if (p.waves > most_waves) p.waves = most_waves;
    while (p.waves > 1 && p.waves / 2 >= wanted) p.waves /= 2;
    const int tile = p.waves * 4 * strand;
    const long long tiles = (seqlen + tile - 1LL) / tile;
    long long segs = 2048 / (units * p.waves);
    if (segs > tiles / 2) segs = tiles / 2;
    if (segs > 32) segs = 32;
    if (segs < 1) segs = 1;
    const long long each = (tiles + segs - 1) / segs;  // tiles of a segment
    p.seg_len = static_cast<int>(each * tile);
    p.segs = static_cast<int>((tiles + each - 1) / each);
    p.keeps = (seqlen + kRecKeep - 1) / kRecKeep;
    return p;
}
RecPlan rec_fwd_plan(int batch, int seqlen, int channels, bool bf16) {
    return rec_plan(batch, seqlen, channels, bf16 ? rec_fwd_strand<bf16_t>() : rec_fwd_strand<float>(), 16);
}
RecPlan rec_bwd_plan(int batch, int seqlen, int channels) {
    return rec_plan(batch, seqlen, channels, kRecBwdStrand, kRecBwdWaves);
}

unsigned rec_grid(const RecArgs &a, int segs) {
    return static_cast<unsigned>(((long long)a.batch * a.blocks * segs + 7) / 8 * 8);
}

hipError_t launch_rec_tokens(const RecArgs &a, const int *cu, int nseq, int *token, float *final, hipStream_t stream) {
    const unsigned want = static_cast<unsigned>((a.seqlen + 255LL) / 256), grid = want < 2048 ? want : 2048;
    rec_token_kernel<<<grid, 256, 0, stream>>>(
        cu, nseq, a.seqlen, token, final, (long long)nseq * a.channels);
    return hipGetLastError();
}

hipError_t launch_rec_fwd(const RecArgs &a, bool bf16, hipStream_t stream) {
    const bool gated = a.decay != nullptr, packed = a.token != nullptr;
    if (bf16) {
        if (gated) return packed ? fwd<bf16_t, true, true>(a, stream) : fwd<bf16_t, true, false>(a, stream);
        return packed ? fwd<bf16_t, false, true>(a, stream) : fwd<bf16_t, false, false>(a, stream);
    }
    if (gated) return packed ? fwd<float, true, true>(a, stream) : fwd<float, true, false>(a, stream);
    return packed ? fwd<float, false, true>(a, stream) : fwd<float, false, false>(a, stream);
}

hipError_t launch_rec_step(const RecArgs &a, float *state, bool bf16, hipStream_t stream) {
    if (bf16) return a.decay ? step<bf16_t, true>(a, state, stream) : step<bf16_t, false>(a, state, stream);
    return a.decay ? step<float, true>(a, state, stream) : step<float, false>(a, state, stream);
}

}  // namespace ssd
