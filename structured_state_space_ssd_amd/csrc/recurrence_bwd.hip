// Gradients of the gated recurrence (recurrence.hip). With g_t the gradient of h_t,
//   g_t = dy_t silu(z_t) + a_{t+1} g_{t+1},  dinit = a_0 g_0,  dz = dy h silu'(z);
// gated, with b = sqrt(1 - a^2), p = sigmoid(i) and w the gradient of log a times log a,
//   dx = g b p,  di = g u (1 - p),  w = g log a (a h_{t-1} - u a^2 / b^2),  u = b p x,
//   dr = w (1 - sigmoid(r)),  ddecay = sum of w, times sigmoid(decay) / softplus(decay);
// direct, dx = g and dr = g a h_{t-1}.
// (u log a / b^2 goes to 0 with log a, so w does too, where the gradient of log a itself
// grows without bound.)
//
// A wavefront's 16 tokens find the state entering them in memory, where the forward
// kept one every kRecKeep = 16 tokens (1/4 of a byte a channel and token), and make their
// states from it again in registers; the adjoint is put together like the forward's
// state, against the tokens' order.
//
// 8 x 2048 x 2560 bf16 with z: 209 us for 765 MB, 3.7 TB/s. The same loads and stores
// alone take 185 us, the 94 vector instructions of an element 114; a SIMD holds four
// wavefronts (about 120 registers), which hide most of the one behind the other. Two
// wavefronts to a tile in place of four, and stores that pass the caches by, gained nothing.
// float32, gated: 266 us, with z 331 (4.6 TB/s). Packed, bf16 without z, 16384 x 2560: 201 us; its
// four bodies spill 67 scalar registers, 105 with z, where the kernel without sequences spills 9 and 17.
// Without kept states the forward kernel runs first, with its z if there is one, though only the
// states are kept of it: 8 x 2048 x 2560 bf16 with z 93 us more, without 74.
#include "recurrence.h"

namespace ssd {

namespace {

// Whole tiles go through buffer loads and stores: a wavefront's base and a token's distance
// from it in scalar registers, one offset per lane. By addresses, which the compiler adds
// up per lane in 64 bits, a tile takes 7 % more vector instructions (8 x 2048 x 2560 bf16
// with z: 234 us, so 216; float32 340 and 331; forward, with fewer tensors, no gain). A pair of
// channels has to lie on 32-bit words, else the tile goes the way of ragged ones (254 us).
typedef __amdgpu_buffer_rsrc_t rec_buffer;
__device__ __forceinline__ rec_buffer rec_buffer_at(const void *t, size_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(t) + bytes;
    const uint64_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at)) & 0xffffffffu,
                   hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(hi << 32 | lo), 0, -1, 0x00020000);
}
__device__ __forceinline__ void rec_get(RecPair<bf16_t> &r, rec_buffer t, uint32_t off, uint32_t row) {
    r.w = __builtin_amdgcn_raw_buffer_load_b32(t, off, row, 0);
}
__device__ __forceinline__ void rec_get(RecPair<float> &r, rec_buffer t, uint32_t off, uint32_t row) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(t, off, row, 0);
    r.w[0] = __uint_as_float(v[0]);
    r.w[1] = __uint_as_float(v[1]);
}
template <typename T, bool WHOLE, int S>
__device__ __forceinline__ void rec_get(RecPair<T> (&r)[S], const void *t, size_t at, size_t token,
                                        const RecPlace &p, int nt) {
    if (!WHOLE) return rec_load<T, false>(r, t, at, token, p, nt);
    const rec_buffer from = rec_buffer_at(t, at * sizeof(T));
    const uint32_t off = rec_offset<T, S>(token, p), row = static_cast<uint32_t>(token) * static_cast<uint32_t>(sizeof(T));
#pragma unroll
    for (int j = 0; j < S; ++j) rec_get(r[j], from, off, j * row);
}
typedef unsigned rec_word2 __attribute__((ext_vector_type(2)));
template <typename T, bool WHOLE>
__device__ __forceinline__ void rec_put(void *t, size_t at, uint32_t row, uint32_t off, int nch, const float (&v)[2]) {
    if (!WHOLE) rec_store<T, false>(static_cast<char *>(t) + at + row, off, nch, v[0], v[1]);
    else if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(v[0], v[1]), rec_buffer_at(t, at), off, row, 0);
    else {
        const rec_word2 w = {__float_as_uint(v[0]), __float_as_uint(v[1])};
        __builtin_amdgcn_raw_buffer_store_b64(w, rec_buffer_at(t, at), off, row, 0);
    }
}

// GATE: whether there is a z (known to the compiler: 8 to 12 registers fewer without, and forward
// and back each 2 to 4 % faster, with and without).
template <typename T, bool GATED, bool PACKED, bool GATE>
__global__ __launch_bounds__(kRecWaves * 64, sizeof(T) == 2 ? 4 : 3) void rec_bwd_kernel(RecBwdArgs b) {
    constexpr int S = kRecBwdStrand;
    __shared__ RecShared sh;
    const RecArgs &a = b.f;
    const RecPlace p = rec_place(a);
    if (!p.live) return;
    const int order = rec_ticket(a, p, sh), tile = a.tiles - 1 - order;
    if (static_cast<unsigned>(order) >= static_cast<unsigned>(a.tiles)) return;
    const int E = a.channels, tw = (tile * a.waves + p.wave) * 4 * S, ts = tw + p.sub * S;
    const int nt = min(max(a.seqlen - ts, 0), S);
    auto run = [&](auto whole_tile, auto cuts) {
        constexpr bool WHOLE = decltype(whole_tile)::value, CUTS = decltype(cuts)::value;
        RecPair<T> x[S], r[S], in[S], z[S], dy[S];
        const size_t at = ((size_t)p.batch * a.seqlen + tw) * E;
        rec_get<T, WHOLE>(r, a.r, p.batch * a.r_batch + tw * a.r_token, a.r_token, p, nt);
        rec_get<T, WHOLE>(dy, b.dy, at, E, p, nt);
        if (GATE) rec_get<T, WHOLE>(z, a.z, p.batch * a.z_batch + tw * a.z_token, a.z_token, p, nt);
        if (GATED) rec_get<T, WHOLE>(in, a.i, p.batch * a.i_batch + tw * a.i_token, a.i_token, p, nt);
        rec_get<T, WHOLE>(x, a.x, p.batch * a.x_batch + tw * a.x_token, a.x_token, p, nt);
        float hw[2] = {0.0f, 0.0f};  // the state entering the wavefront's tokens
        if (WHOLE || tw < a.seqlen) {
            const float *s = a.states + ((size_t)p.batch * a.keeps + tw / kRecKeep) * E + p.ch;
            if (p.nch > 0) hw[0] = s[0];
            if (p.nch > 1) hw[1] = s[1];
        }
        int code[S];
        if (CUTS)
#pragma unroll
            for (int j = 0; j < S; ++j) code[j] = WHOLE || j < nt ? a.token[ts + j] : 0;
        float rate[2], sum[2] = {0.0f, 0.0f};
        if (GATED) rec_rates(rate, a, p);
        const float rate_e[2] = {rate[0] * kLn2, rate[1] * kLn2};
        float av[S][2], hv[S][2];
        float rv[S][2], iv[S][2], bv[S][2];  // the gates, and sqrt(1 - a^2)
        RecMap m[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}}, mg[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
#pragma unroll
        for (int j = 0; j < S; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float d, u;
                if (GATED) {
                    rv[j][e] = sigmoid_f32(r[j].get(e));
                    const float la = rate[e] * rv[j][e];
                    d = __builtin_amdgcn_exp2f(la);
                    bv[j][e] = __builtin_amdgcn_sqrtf(one_minus_square(la, d));
                    iv[j][e] = sigmoid_f32(in[j].get(e));
                    u = bv[j][e] * iv[j][e] * x[j].get(e);
                } else {
                    d = __builtin_amdgcn_exp2f(kLog2e * r[j].get(e));
                    u = x[j].get(e);
                }
                if (!WHOLE && j >= nt) {
                    d = 1.0f;
                    u = 0.0f;
                }
                if (CUTS) {
                    if (code[j] & 1) d = -1.0f;
                    if (code[j] < 0) u = 0.0f;
                }
                av[j][e] = d;
                hv[j][e] = u;
                m[e] = rec_then<CUTS, false>(m[e], {d, u});
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            RecMap before, whole;
            rec_wave<CUTS, !GATED, false>(m[e], p.sub, before, whole);
            float h = rec_apply<CUTS, !GATED>(before, hw[e]);
#pragma unroll
            for (int j = 0; j < S; ++j) {  // what each token takes of the state before, in its input's place
                const float carried = CUTS && av[j][e] < 0.0f ? 0.0f : av[j][e] * h;
                h = carried + hv[j][e];
                hv[j][e] = carried;
            }
        }
        // What reaches a token's state by its output, formed twice. The gate's sigmoid stays where
        // the registers that it takes leave the wavefronts of a SIMD as many (8 x 2048 x 2560 222 us
        // without, 216 so); with float32 operands they do not.
        constexpr bool KEEP = sizeof(T) == 2;
        float zv[S][2];
        if (GATE && KEEP)
#pragma unroll
            for (int j = 0; j < S; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) zv[j][e] = sigmoid_f32(z[j].get(e));
        auto own = [&](int j, int e) {
            float g = dy[j].get(e);
            if (GATE) g *= KEEP ? z[j].get(e) * zv[j][e] : silu_f32(z[j].get(e));
            if ((!WHOLE && j >= nt) || (CUTS && code[j] < 0)) g = 0.0f;
            if (CUTS && b.dfinal && code[j] > 1 && e < p.nch)
                g += b.dfinal[(size_t)((code[j] >> 1) - 1) * E + p.ch + e];
            return g;
        };
        // a token passes a (g + what comes to it) on to the one before, nothing from a first one
#pragma unroll
        for (int j = S - 1; j >= 0; --j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool first = CUTS && av[j][e] < 0.0f;
                mg[e] = {first || (CUTS && mg[e].a < 0.0f) ? -1.0f : av[j][e] * mg[e].a,
                         first ? 0.0f : av[j][e] * (own(j, e) + mg[e].h)};
            }
        RecMap after[2], whole[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) rec_wave<CUTS, !GATED, true>(mg[e], p.sub, after[e], whole[e]);
        // what comes to the wavefront's last token from behind
        float qs[2];
        rec_enter<PACKED, !GATED, true>(a, p, order, whole, PACKED ? nullptr : b.dfinal, PACKED ? nullptr : b.dinit, qs, sh);
#pragma unroll
        for (int e = 0; e < 2; ++e) qs[e] = rec_apply<CUTS, !GATED>(after[e], qs[e]);
        // (the values anew: what the compiler keeps of them from above fills the registers)
#pragma unroll
        for (int j = 0; j < S; ++j) {
            dy[j].fresh();
            z[j].fresh();
        }
        const uint32_t off = rec_offset<T, S>(E, p);
#pragma unroll
        for (int j = S - 1; j >= 0; --j) {
            float ox[2], orr[2], oi[2], oz[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool first = CUTS && av[j][e] < 0.0f;
                const float xv = x[j].get(e), d = av[j][e], g = own(j, e) + qs[e];
                const float carried = hv[j][e];  // a h_{t-1}
                float u = xv;
                if (GATED) {
                    const float sr = rv[j][e], si = iv[j][e], beta = bv[j][e], la = rate_e[e] * sr;
                    u = beta * si * xv;
                    ox[e] = g * (beta * si);
                    oi[e] = g * u * (1.0f - si);
                    // d sqrt(1 - a^2) / d log a = -a^2 / b, so p x times that is -u a^2 / b^2
                    const float a2 = CUTS && first ? __builtin_amdgcn_exp2f(2.0f * rate[e] * sr) : d * d;
                    // (where b is 0, so is u)
                    const float q2 = a2 * __builtin_amdgcn_rcpf(fmaxf(beta * beta, 1.17549435e-38f));
                    const float w = g * la * fmaf(-u, q2, carried);
                    orr[e] = w * (1.0f - sr);
                    if ((WHOLE || j < nt) && !(CUTS && code[j] < 0)) sum[e] += w;
                } else {
                    ox[e] = g;
                    orr[e] = g * carried;
                }
                if (GATE) {
                    const float sz = KEEP ? zv[j][e] : sigmoid_f32(z[j].get(e));
                    oz[e] = dy[j].get(e) * (carried + u) * (sz * fmaf(z[j].get(e), 1.0f - sz, 1.0f));
                }
                qs[e] = first ? 0.0f : d * g;
            }
            if (!WHOLE && j >= nt) continue;
            if (CUTS && code[j] < 0) ox[0] = ox[1] = orr[0] = orr[1] = oi[0] = oi[1] = oz[0] = oz[1] = 0.0f;
            const auto out = [&](void *t, float (&v)[2]) {
                rec_put<T, WHOLE>(t, at * sizeof(T), static_cast<uint32_t>(j * E) * static_cast<uint32_t>(sizeof(T)), off, p.nch, v);
            };
            out(b.dx, ox);
            out(b.dr, orr);
            if (GATED) out(b.di, oi);
            if (GATE) out(b.dz, oz);
        }
        if (!GATED) return;
        // the strands' sums of w, then the wavefronts'
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(sum[e]), __float_as_uint(sum[e]), false, false);
            sum[e] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
            const auto k = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum[e]), __float_as_uint(sum[e]), false, false);
            sum[e] = __uint_as_float(k[0]) + __uint_as_float(k[1]);
        }
        __syncthreads();
        if (p.sub == 0) {
            sh.map[p.wave][2 * p.col][0] = sum[0];
            sh.map[p.wave][2 * p.col + 1][0] = sum[1];
        }
        __syncthreads();
        if (p.wave || p.sub) return;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (e < p.nch) {
                float s = 0.0f;
                for (int w = 0; w < a.waves; ++w) s += sh.map[w][2 * p.col + e][0];
                // sigmoid / softplus goes to 1 as both go to e^decay, and beyond what 32 bits hold of that
                const float v = a.decay[p.ch + e], k = v < -20.0f ? 1.0f : sigmoid_f32(v) / softplus_f32(v);
                b.part[((size_t)p.batch * a.tiles + tile) * E + p.ch + e] = k * s;
            }
    };
    const bool whole = b.words && p.ch - 2 * p.col + kRecCols <= E && (tile + 1) * a.waves * 4 * S <= a.seqlen;
    if constexpr (PACKED) {
        const int t0 = tile * a.waves * 4 * S;
        if (rec_cuts(a.cuts, t0, min(a.waves * 4 * S, a.seqlen - t0))) {
            if (whole) run(std::true_type(), std::true_type());
            else run(std::false_type(), std::true_type());
            return;
        }
    }
    if (whole) run(std::true_type(), std::false_type());
    else run(std::false_type(), std::false_type());
}

template <typename T, bool GATED, bool PACKED> hipError_t bwd(const RecBwdArgs &b, hipStream_t stream) {
    const RecArgs &a = b.f;
    if (a.z) rec_bwd_kernel<T, GATED, PACKED, true><<<rec_grid(a), a.waves * 64, 0, stream>>>(b);
    else rec_bwd_kernel<T, GATED, PACKED, false><<<rec_grid(a), a.waves * 64, 0, stream>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !GATED) return e;
    return launch_colsum(b.part, a.batch * a.tiles, a.channels, a.channels, b.ddecay, nullptr, stream, b.spare);
}

}  // namespace

hipError_t launch_rec_bwd(const RecBwdArgs &b, bool bf16, hipStream_t stream) {
    const bool gated = b.f.decay != nullptr, packed = b.f.token != nullptr;
    if (bf16) {
        if (gated) return packed ? bwd<bf16_t, true, true>(b, stream) : bwd<bf16_t, true, false>(b, stream);
        return packed ? bwd<bf16_t, false, true>(b, stream) : bwd<bf16_t, false, false>(b, stream);
    }
    if (gated) return packed ? bwd<float, true, true>(b, stream) : bwd<float, true, false>(b, stream);
    return packed ? bwd<float, false, true>(b, stream) : bwd<float, false, false>(b, stream);
}

}  // namespace ssd
