// Gated linear recurrence with one state per channel:
//   h_t = a_t h_{t-1} + u_t,  y_t = h_t  or  h_t silu(z_t)
// gated:  log a_t = -c softplus(decay) sigmoid(r_t),  u_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t
// direct: log a_t = r_t,  u_t = x_t.
// Forward walk, single tokens and the plan; recurrence.h has the layout.
//
// The inputs are read once: a tile's tokens stay in registers between the map that they
// make and the states that the entering state gives them. Bound by memory with the vector
// unit close behind: an element's 38 instructions without z (three exponentials, two
// reciprocals and a square root among them), 46 with, keep it busy for half of the time.
// Measured (bf16): 1 x 8192 x 2560 without z 45 us, 3.7 TB/s; 8 x 2048 x 2560 with z
// 105 us, 4.1 TB/s. With arithmetic and exchange left out the same loads and stores of 64
// bytes a token take 35 and 92 us. Ways that took longer: two passes, the first of which
// makes the segments' maps (94 us where the exchange between tiles took 61), workgroups that
// stay for several tiles (70 to 81, where 57), 64 channels to a unit (prompt 74, where 57,
// training 129, where 111), strands of 4 tokens in bf16 (124, where 113); each against the
// step that it was tried on. float32 at 8 x 2048 x 2560: gated 140 us, with z 175 (4.9 TB/s).
// Packed, the kernel holds its body four times (whole or ragged, with ends or without): 16384 x
// 2560 bf16 without z 99 us, with 27 % more vector instructions than without sequences and 72
// scalar registers spilled to lanes of vector registers, where there are none otherwise.
#include "recurrence.h"

namespace ssd {

namespace {

// Before a pass: the words that its tiles wait for are set to ~0 (`words` vectors of 16
// bytes), the channels' rates are made, and, for a packed axis, the tokens' codes: bit 0, the first of its
// sequence; above, 1 + the number of the sequence whose last token it is; kRecNone: in no
// sequence; and per 64 tokens whether any code is not 0 (rec_cuts). `final`: set to the state of an empty sequence. Any contents of `cu` are read
// within its nseq + 1 entries.
__global__ __launch_bounds__(256) void rec_prepare_kernel(uint4 *__restrict__ unset, long long words,
                                                          const int *__restrict__ cu, int nseq, int L,
                                                          int *__restrict__ token, int *__restrict__ cuts,
                                                          float *__restrict__ final,
                                                          long long finals, const float *__restrict__ decay,
                                                          float c, int E, float *__restrict__ rate) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x, all = (long long)gridDim.x * 256;
    for (long long k = id; k < words; k += all) unset[k] = make_uint4(kRecUnset, kRecUnset, kRecUnset, kRecUnset);
    if (decay)
        for (long long k = id; k < E; k += all) rate[k] = rec_rate(decay[k], c);
    if (!cu) return;
    if (final)
        for (long long k = id; k < finals; k += all) final[k] = 0.0f;
    for (long long t = id; t - lane_id() < L; t += all) {
        int lo = 0, hi = nseq;  // the last sequence that begins at or before t
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int from = cu[lo], to = cu[lo + 1];
        const int code = t < from || t >= to ? kRecNone : (from == t ? 1 : 0) | (to - 1 == t ? 2 * (lo + 1) : 0);
        if (t < L) token[t] = code;
        float any[1] = {t < L && code != 0 ? 1.0f : 0.0f};
        lane_sum(any, 64);
        if (lane_id() == 0) cuts[t / 64] = any[0] != 0.0f;
    }
}

// Tokens of a strand: float32 operands of 8 do not fit the registers.
template <typename T> constexpr int rec_fwd_strand() { return sizeof(T) == 2 ? 8 : 4; }

// GATE: whether there is a z (known to the compiler: see the backward's). The wavefronts of a
// SIMD are what fits without spilling vector registers. Left to the compiler: packed bf16 without
// z 104 us (so 97 to 103), packed float32 156 and 183 with z (so 153 and 179), bf16 with z 102
// (so 104).
template <typename T, bool GATED, bool PACKED, bool GATE>
__global__ __launch_bounds__(kRecWaves * 64, sizeof(T) == 2 ? GATE ? 5 : 6 : 7) void rec_fwd_kernel(RecArgs a) {
    constexpr int S = rec_fwd_strand<T>();
    __shared__ RecShared sh;
    const RecPlace p = rec_place(a);
    if (!p.live) return;
    const int order = rec_ticket(a, p, sh);
    if (static_cast<unsigned>(order) >= static_cast<unsigned>(a.tiles)) return;
    const int E = a.channels, tw = (order * a.waves + p.wave) * 4 * S, ts = tw + p.sub * S;
    const int nt = min(max(a.seqlen - ts, 0), S);
    auto run = [&](auto whole_tile, auto cuts) {
        constexpr bool WHOLE = decltype(whole_tile)::value, CUTS = decltype(cuts)::value;
        RecPair<T> x[S], r[S], in[S], z[S];
        rec_load<T, WHOLE>(r, a.r, p.batch * a.r_batch + tw * a.r_token, a.r_token, p, nt);
        if (GATED) rec_load<T, WHOLE>(in, a.i, p.batch * a.i_batch + tw * a.i_token, a.i_token, p, nt);
        rec_load<T, WHOLE>(x, a.x, p.batch * a.x_batch + tw * a.x_token, a.x_token, p, nt);
        if (GATE) rec_load<T, WHOLE>(z, a.z, p.batch * a.z_batch + tw * a.z_token, a.z_token, p, nt);
        int code[S];
        if (CUTS)
#pragma unroll
            for (int j = 0; j < S; ++j) code[j] = WHOLE || j < nt ? a.token[ts + j] : 0;
        float rate[2];
        if (GATED) rec_rates(rate, a, p);
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
                    u = __builtin_amdgcn_sqrtf(one_minus_square(la, d)) *
                        sigmoid_f32(in[j].get(e)) * x[j].get(e);
                } else {
                    d = __builtin_amdgcn_exp2f(kLog2e * r[j].get(e));
                    u = x[j].get(e);
                }
                if (!WHOLE && j >= nt) {
                    d = 1.0f;
                    u = 0.0f;
                }
                if (CUTS && (code[j] & 1)) d = -1.0f;
                if (CUTS && code[j] < 0) u = 0.0f;
                av[j][e] = d;
                uv[j][e] = u;
                m[e] = rec_then<CUTS, false>(m[e], {d, u});
            }
        RecMap before[2], whole[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) rec_wave<CUTS, !GATED, false>(m[e], p.sub, before[e], whole[e]);
        float h[2];
        rec_enter<PACKED, !GATED, false>(a, p, order, whole, a.init, PACKED ? nullptr : a.final_state, h, sh);
#pragma unroll
        for (int e = 0; e < 2; ++e) h[e] = rec_apply<CUTS, !GATED>(before[e], h[e]);
        if (a.states && ts % kRecKeep == 0 && (WHOLE || nt > 0)) {
            float *s = a.states + ((size_t)p.batch * a.keeps + ts / kRecKeep) * E + p.ch;
            if (p.nch > 0) s[0] = h[0];
            if (p.nch > 1) s[1] = h[1];
        }
        char *y = static_cast<char *>(a.y) + ((size_t)p.batch * a.seqlen + tw) * E * sizeof(T);
        const uint32_t off = rec_offset<T, S>(E, p);
#pragma unroll
        for (int j = 0; j < S; ++j) {
            float o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                h[e] = rec_apply<CUTS, false>({av[j][e], uv[j][e]}, h[e]);
                o[e] = h[e];
                if (GATE) o[e] *= silu_f32(z[j].get(e));
                if (CUTS && code[j] < 0) o[e] = 0.0f;
            }
            if (a.y && (WHOLE || j < nt)) rec_store<T, WHOLE>(y + (size_t)j * E * sizeof(T), off, p.nch, o[0], o[1]);
            if (CUTS && a.final_state && (WHOLE || j < nt) && code[j] > 1) {
                float *f = a.final_state + (size_t)((code[j] >> 1) - 1) * E + p.ch;
                if (p.nch > 0) f[0] = h[0];
                if (p.nch > 1) f[1] = h[1];
            }
        }
    };
    const bool whole = p.ch - 2 * p.col + kRecCols <= E && (order + 1) * a.waves * 4 * S <= a.seqlen;
    if constexpr (PACKED) {
        const int t0 = order * a.waves * 4 * S;
        if (rec_cuts(a.cuts, t0, min(a.waves * 4 * S, a.seqlen - t0))) {
            if (whole) run(std::true_type(), std::true_type());
            else run(std::false_type(), std::true_type());
            return;
        }
    }
    if (whole) run(std::true_type(), std::false_type());
    else run(std::false_type(), std::false_type());
}

// One token: a lane takes four channels of one sequence. 256 sequences of 5120 channels, bf16
// with z, 6.7 us (23.6 MB; a launch by itself is 4).
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
            h[e] = fmaf(k, s.get(e), __builtin_amdgcn_sqrtf(one_minus_square(la, k)) *
                                         sigmoid_f32(in.get(e)) * x.get(e));
        } else h[e] = fmaf(__builtin_amdgcn_exp2f(kLog2e * r.get(e)), s.get(e), x.get(e));
        o[e] = a.z ? h[e] * silu_f32(z.get(e)) : h[e];
    }
    row_store(state + (size_t)b * a.channels + c, h, n);
    row_store(static_cast<T *>(a.y) + (size_t)b * a.channels + c, o, n);
}

template <typename T, bool GATED, bool PACKED> hipError_t fwd(const RecArgs &a, hipStream_t stream) {
    if (a.z) rec_fwd_kernel<T, GATED, PACKED, true><<<rec_grid(a), a.waves * 64, 0, stream>>>(a);
    else rec_fwd_kernel<T, GATED, PACKED, false><<<rec_grid(a), a.waves * 64, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, bool GATED> hipError_t step(const RecArgs &a, float *state, hipStream_t stream) {
    const int vecs = (a.channels + 3) / 4;
    const unsigned grid = static_cast<unsigned>(((long long)a.batch * vecs + 255) / 256);
    rec_step_kernel<T, GATED><<<grid, 256, 0, stream>>>(a, state, vecs);
    return hipGetLastError();
}

}  // namespace

static RecDivisor rec_divisor(int d) {  // of numbers below 2^28
    int bits = 0;
    while (1LL << bits < d) ++bits;
    return {static_cast<uint32_t>(((1ULL << (28 + bits)) + d - 1) / d), 28 + bits};
}

// Wavefronts of a workgroup, and tiles, for strands of `strand` tokens.
static RecPlan rec_plan(int batch, int seqlen, int channels, int strand) {
    RecPlan p;
    p.blocks = (channels + kRecCols - 1) / kRecCols;
    const int wanted = (seqlen + 4 * strand - 1) / (4 * strand);  // wavefronts that have tokens
    p.waves = kRecWaves;
    while (p.waves > 1 && p.waves / 2 >= wanted) p.waves /= 2;
    p.tiles = (wanted + p.waves - 1) / p.waves;
    p.keeps = (seqlen + kRecKeep - 1) / kRecKeep;
    const size_t units = (size_t)batch * p.blocks, words = units * kRecCols;
    p.map_words = p.tiles > 1 ? words * p.tiles : 0;
    p.enter_words = p.tiles > 1 ? words * ((p.tiles + kRecGroup - 1) / kRecGroup) : 0;
    p.tickets = p.tiles > 1 ? units * kRecTicketStep : 0;
    p.by_blocks = rec_divisor(p.blocks);
    p.by_each = rec_divisor(static_cast<int>((units + 7) / 8 < (1u << 28) ? (units + 7) / 8 : 1));
    return p;
}
RecPlan rec_fwd_plan(int batch, int seqlen, int channels, bool bf16) {
    return rec_plan(batch, seqlen, channels, bf16 ? rec_fwd_strand<bf16_t>() : rec_fwd_strand<float>());
}
RecPlan rec_bwd_plan(int batch, int seqlen, int channels) {
    return rec_plan(batch, seqlen, channels, kRecBwdStrand);
}

unsigned rec_grid(const RecArgs &a) {
    return static_cast<unsigned>(((long long)a.batch * a.blocks + 7) / 8 * 8 * a.tiles);
}

hipError_t launch_rec_prepare(const RecArgs &a, void *unset, size_t bytes, float *rate, const int *cu, int nseq,
                              int *token, int *cuts, float *final, hipStream_t stream) {
    const long long words = bytes / 16, finals = (long long)nseq * a.channels;
    // its loops' extents: 32 packed tokens of 5120 channels in 32 sequences with final states take
    // 31 us where the tokens alone set the grid, 8 so
    long long most = words;
    for (long long n : {cu ? a.seqlen : 0LL, cu && final ? finals : 0LL, a.decay ? a.channels : 0LL})
        if (n > most) most = n;
    const unsigned want = static_cast<unsigned>(most / 256 + 1), grid = want < 2048 ? want : 2048;
    rec_prepare_kernel<<<grid, 256, 0, stream>>>(static_cast<uint4 *>(unset), words, cu, nseq, a.seqlen, token, cuts, final,
                                                 finals, a.decay, a.c, a.channels, rate);
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
