// C ABI of the operators that make a recurrent block: the gated recurrence, the join of
// a block with the residual stream and its norms, and dropout. Argument checks, workspace
// sizes and launches; every declaration and its contract is in include/ssd.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_launch.h"

namespace {

constexpr size_t kAlign = 256;
// token and channel counts above this leave no room for tile arithmetic in int
constexpr int kMaxExtent = 1 << 30;
// offsets within a tile of tokens are 32 bits of bytes
constexpr long long kMaxTokenStride = 1LL << 24;
// rows of dropout are counted in 32 bits
constexpr long long kMaxRows = 0x7fffffffLL;

bool valid_dtype(int d) { return d == SSD_F32 || d == SSD_BF16; }
int status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

int check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return SSD_OK;
    if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0)
        return SSD_ERR_WORKSPACE;
    return SSD_OK;
}

struct Taker {
    size_t o = 0;
    size_t take(size_t words) {  // of 32 bits
        const size_t at = o;
        o += (words * 4 + kAlign - 1) / kAlign * kAlign;
        return at;
    }
};

// ---- recurrence

int check_recurrence(int batch, int seqlen, int channels, int dtype) {
    if (batch < 1 || seqlen < 1 || channels < 1) return SSD_ERR_SHAPE;
    if (seqlen > kMaxExtent || channels > kMaxExtent) return SSD_ERR_SHAPE;
    if (!valid_dtype(dtype) || channels >= kMaxTokenStride) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Fewer than 2^32 lanes, and tokens of a last tile in an int.
bool plan_fits(int batch, const ssd::RecPlan &p) {
    const long long units = (long long)batch * p.blocks;
    return units < (1LL << 28) && (units + 8) * p.tiles < (1LL << 32) / 64 / p.waves;
}

// Inputs, strides (NULL: dense) and checks that go beyond sizes.
int recurrence_args(ssd::RecArgs &a, const void *x, const void *r, const void *i, const float *decay,
                    float c, const void *z, int batch, int seqlen, int channels,
                    const ssd_recurrence_strides *st) {
    a = ssd::RecArgs{};
    if (decay && !i) return SSD_ERR_NULL;
    if (!decay && i) return SSD_ERR_UNSUPPORTED;
    if (decay && !(c > 0.0f && isfinite(c))) return SSD_ERR_OPTION;
    a.x = x; a.r = r; a.i = i; a.z = z; a.decay = decay; a.c = c;
    a.batch = batch; a.seqlen = seqlen; a.channels = channels;
    const long long e = channels, s = e * seqlen;
    ssd_recurrence_strides d = {s, e, s, e, s, e, s, e};
    if (st) {
        d = *st;
        if (seqlen == 1) d.x_token = d.r_token = d.i_token = d.z_token = 0;  // never stepped over
        for (long long v : {d.x_batch, d.x_token, d.r_batch, d.r_token, d.i_batch, d.i_token, d.z_batch,
                            d.z_token})
            if (v < 0) return SSD_ERR_SHAPE;
        for (long long v : {d.x_token, d.r_token, d.i_token, d.z_token})
            if (v >= kMaxTokenStride) return SSD_ERR_UNSUPPORTED;
    }
    a.x_batch = d.x_batch; a.x_token = d.x_token; a.r_batch = d.r_batch; a.r_token = d.r_token;
    a.i_batch = d.i_batch; a.i_token = d.i_token; a.z_batch = d.z_batch; a.z_token = d.z_token;
    return SSD_OK;
}

// (a token's code holds twice the number of a sequence)
int check_packed(const int *cu_seqlens, int nseq, int batch, const float *init) {
    if (!cu_seqlens) return SSD_OK;
    if (batch != 1 || nseq < 1 || nseq >= kMaxExtent) return SSD_ERR_SHAPE;
    return init ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

// What a pass needs beside its tensors: the words that its tiles exchange, all one after the
// other, and the codes of a packed axis.
struct RecScratch {
    size_t maps, enter, ticket, end, rate, token;
    void take(Taker &k, const ssd::RecPlan &p, int channels, int packed_tokens) {
        maps = k.take(2 * p.map_words);
        enter = k.take(2 * p.enter_words);
        ticket = k.take(p.tickets);
        end = k.o;
        rate = k.take(p.tiles > 1 || packed_tokens ? channels : 0);
        token = k.take(packed_tokens ? (size_t)packed_tokens + (packed_tokens + 63) / 64 : 0);  // and cuts behind
    }
    void use(ssd::RecArgs &a, const ssd::RecPlan &p, char *base) const {
        a.blocks = p.blocks; a.waves = p.waves; a.tiles = p.tiles; a.keeps = p.keeps;
        a.by_blocks = p.by_blocks; a.by_each = p.by_each;
        a.maps = reinterpret_cast<unsigned long long *>(base + maps);
        a.enter = reinterpret_cast<unsigned long long *>(base + enter);
        a.ticket = reinterpret_cast<unsigned *>(base + ticket);
        a.rate = nullptr;
        a.token = a.cuts = nullptr;
    }
    // What a pass over one tile of each unit does without is left out.
    hipError_t prepare(ssd::RecArgs &a, const int *cu, int nseq, float *final, char *base, hipStream_t s) const {
        if (a.tiles == 1 && !cu) return hipSuccess;
        int *t = reinterpret_cast<int *>(base + token), *u = t + a.seqlen;
        float *r = reinterpret_cast<float *>(base + rate);
        a.token = cu ? t : nullptr;
        a.cuts = cu ? u : nullptr;
        a.rate = a.decay ? r : nullptr;
        return ssd::launch_rec_prepare(a, base + maps, end - maps, r, cu, nseq, t, u, final, s);
    }
};

struct RecLayout {
    ssd::RecPlan plan;
    RecScratch scratch;
    size_t total;
};
RecLayout recurrence_layout(int batch, int seqlen, int channels, bool packed, int dtype) {
    RecLayout w{};
    w.plan = ssd::rec_fwd_plan(batch, seqlen, channels, dtype == SSD_BF16);
    Taker k;
    w.scratch.take(k, w.plan, channels, packed ? seqlen : 0);
    w.total = k.o;
    return w;
}

// Backward: its own pass and, where the caller has no states, the one that makes them.
struct RecBwdLayout {
    ssd::RecPlan plan, keep;
    RecScratch scratch, keep_scratch;
    size_t part, spare, states, total;
};
RecBwdLayout recurrence_bwd_layout(int batch, int seqlen, int channels, bool packed, bool have_states,
                                   int dtype) {
    RecBwdLayout w{};
    w.plan = ssd::rec_bwd_plan(batch, seqlen, channels);
    w.keep = ssd::rec_fwd_plan(batch, seqlen, channels, dtype == SSD_BF16);
    const size_t be = (size_t)batch * channels;
    Taker k;
    w.scratch.take(k, w.plan, channels, packed ? seqlen : 0);
    w.part = k.take(be * w.plan.tiles);
    w.spare = k.take((long long)batch * w.plan.tiles > ssd::kColsumRows ? (size_t)ssd::kColsumChunks * channels : 0);
    if (!have_states) {
        w.keep_scratch.take(k, w.keep, channels, packed ? seqlen : 0);
        w.states = k.take(be * w.plan.keeps);
    }
    w.total = k.o;
    return w;
}

// ---- dropout

// p, seed and offset as the kernels take them (NULL: nothing is dropped).
int drop_args(ssd::DropArgs &d, const ssd_random *r) {
    d = ssd::DropArgs{};
    d.scale = 1.0f;
    if (!r) return SSD_OK;
    if (!(r->p >= 0.0 && r->p <= 1.0)) return SSD_ERR_OPTION;  // NaN fails too
    if ((reinterpret_cast<uintptr_t>(r->state) & 7u) != 0) return SSD_ERR_UNSUPPORTED;
    d.seed = r->seed;
    d.offset = r->offset;
    d.rng = r->state;
    d.threshold = static_cast<uint32_t>(floor(r->p * 65536.0 + 0.5));
    d.scale = d.threshold < 65536 ? static_cast<float>(65536.0 / (65536 - d.threshold)) : 0.0f;
    return SSD_OK;
}

// ---- block norm

int check_block(const ssd_block *o, int stream_dtype, const void *z, long long z_row_stride,
                long long x_row_stride, long long rows, int width, int dtype) {
    if (!o || (!o->weight && !o->post_weight)) return SSD_ERR_NULL;
    if ((o->bias && !o->weight) || (o->post_bias && !o->post_weight)) return SSD_ERR_NULL;
    if (rows < 1 || width < 1 || x_row_stride < 0 || (z && z_row_stride < 0)) return SSD_ERR_SHAPE;
    if (width > ssd::kMaxBlockWidth || rows > kMaxRows || !valid_dtype(dtype)) return SSD_ERR_UNSUPPORTED;
    if (stream_dtype != dtype && stream_dtype != SSD_F32) return SSD_ERR_UNSUPPORTED;
    if (!isfinite(o->residual_scale) || !isfinite(o->branch_scale)) return SSD_ERR_OPTION;
    if (!(o->eps >= 0.0f)) return SSD_ERR_OPTION;
    return SSD_OK;
}

// The columns' sums that the wanted gradients take.
int block_sums(bool dweight, bool dbias, bool dpost_weight, bool dpost_bias, bool dscale, bool post_bias,
               int *p, int *q) {
    *p = dpost_weight || dscale;
    *q = dpost_bias || (dscale && post_bias);
    return dweight + dbias + *p + *q;
}

}  // namespace

extern "C" {

size_t ssd_recurrence_forward_workspace_size(int batch, int seqlen, int channels, int packed, int dtype) {
    if (check_recurrence(batch, seqlen, channels, dtype) != SSD_OK) return 0;
    return recurrence_layout(batch, seqlen, channels, packed != 0, dtype).total;
}

int ssd_recurrence_forward(const void *x, const void *r, const void *i, const float *decay, float c,
                           const void *z, int batch, int seqlen, int channels, int dtype,
                           const float *init_state, const int *cu_seqlens, int nseq, void *y,
                           float *final_state, float *states, void *workspace, size_t workspace_bytes,
                           const ssd_recurrence_strides *strides, void *stream) {
    if (!x || !r || !y) return SSD_ERR_NULL;
    int rc = check_recurrence(batch, seqlen, channels, dtype);
    if (rc != SSD_OK) return rc;
    ssd::RecArgs a;
    rc = recurrence_args(a, x, r, i, decay, c, z, batch, seqlen, channels, strides);
    if (rc != SSD_OK) return rc;
    rc = check_packed(cu_seqlens, nseq, batch, init_state);
    if (rc != SSD_OK) return rc;
    const RecLayout w = recurrence_layout(batch, seqlen, channels, cu_seqlens != nullptr, dtype);
    if (!plan_fits(batch, w.plan)) return SSD_ERR_UNSUPPORTED;
    rc = check_workspace(workspace, workspace_bytes, w.total);
    if (rc != SSD_OK) return rc;
    char *base = static_cast<char *>(workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    w.scratch.use(a, w.plan, base);
    a.init = init_state;
    a.y = y;
    a.final_state = final_state;
    a.states = states;
    const hipError_t e = w.scratch.prepare(a, cu_seqlens, nseq, final_state, base, s);
    if (e != hipSuccess) return status_of(e);
    return status_of(ssd::launch_rec_fwd(a, dtype == SSD_BF16, s));
}

int ssd_recurrence_step(float *state, const void *x, const void *r, const void *i, const float *decay,
                        float c, const void *z, int batch, int channels, int dtype, void *y,
                        const ssd_recurrence_strides *strides, void *stream) {
    if (!state || !x || !r || !y) return SSD_ERR_NULL;
    int rc = check_recurrence(batch, 1, channels, dtype);
    if (rc != SSD_OK) return rc;
    ssd::RecArgs a;
    rc = recurrence_args(a, x, r, i, decay, c, z, batch, 1, channels, strides);
    if (rc != SSD_OK) return rc;
    if ((long long)batch * ((channels + 3) / 4) >= (1LL << 32) - 256) return SSD_ERR_UNSUPPORTED;
    a.y = y;
    return status_of(ssd::launch_rec_step(a, state, dtype == SSD_BF16, static_cast<hipStream_t>(stream)));
}

size_t ssd_recurrence_backward_workspace_size(int batch, int seqlen, int channels, int packed,
                                              int have_states, int dtype) {
    if (check_recurrence(batch, seqlen, channels, dtype) != SSD_OK) return 0;
    return recurrence_bwd_layout(batch, seqlen, channels, packed != 0, have_states != 0, dtype).total;
}

int ssd_recurrence_backward(const void *x, const void *r, const void *i, const float *decay, float c,
                            const void *z, const float *init_state, const int *cu_seqlens, int nseq,
                            const float *states, const void *dy, const float *dfinal_state, int batch,
                            int seqlen, int channels, int dtype, void *dx, void *dr, void *di,
                            float *ddecay, void *dz, float *dinit_state, void *workspace,
                            size_t workspace_bytes, const ssd_recurrence_strides *strides, void *stream) {
    if (!x || !r || !dy || !dx || !dr || (decay && (!di || !ddecay)) || (z && !dz)) return SSD_ERR_NULL;
    int rc = check_recurrence(batch, seqlen, channels, dtype);
    if (rc != SSD_OK) return rc;
    ssd::RecBwdArgs b{};
    ssd::RecArgs &a = b.f;
    rc = recurrence_args(a, x, r, i, decay, c, z, batch, seqlen, channels, strides);
    if (rc != SSD_OK) return rc;
    rc = check_packed(cu_seqlens, nseq, batch, init_state);
    if (rc != SSD_OK) return rc;
    if (cu_seqlens && dinit_state) return SSD_ERR_UNSUPPORTED;
    const RecBwdLayout w = recurrence_bwd_layout(batch, seqlen, channels, cu_seqlens != nullptr,
                                                 states != nullptr, dtype);
    if (!plan_fits(batch, w.plan) || !plan_fits(batch, w.keep) ||
        (long long)batch * w.plan.tiles > kMaxExtent ||
        !ssd::colsum_grid_ok(batch * w.plan.tiles, channels, true))
        return SSD_ERR_UNSUPPORTED;
    rc = check_workspace(workspace, workspace_bytes, w.total);
    if (rc != SSD_OK) return rc;
    char *base = static_cast<char *>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(base + off); };
    const hipStream_t s = static_cast<hipStream_t>(stream);
    a.states = const_cast<float *>(states);
    hipError_t e;
    if (!states) {
        w.keep_scratch.use(a, w.keep, base);
        a.init = init_state;
        a.states = at(w.states);
        e = w.keep_scratch.prepare(a, cu_seqlens, nseq, nullptr, base, s);
        if (e == hipSuccess) e = ssd::launch_rec_fwd(a, dtype == SSD_BF16, s);
        if (e != hipSuccess) return status_of(e);
    }
    w.scratch.use(a, w.plan, base);
    e = w.scratch.prepare(a, cu_seqlens, nseq, nullptr, base, s);
    if (e != hipSuccess) return status_of(e);
    b.dy = dy;
    b.dfinal = dfinal_state;
    b.dx = dx; b.dr = dr; b.di = di; b.dz = dz;
    b.ddecay = ddecay;
    b.dinit = dinit_state;
    b.part = at(w.part);
    b.words = true;
    if (dtype == SSD_BF16) {
        for (const void *t : {x, r, i, z, dy, static_cast<const void *>(dx), static_cast<const void *>(dr),
                              static_cast<const void *>(di), static_cast<const void *>(dz)})
            if (reinterpret_cast<uintptr_t>(t) & 3u) b.words = false;
        for (size_t v : {a.x_batch, a.x_token, a.r_batch, a.r_token, a.i_batch, a.i_token, a.z_batch, a.z_token,
                         static_cast<size_t>(channels)})
            if (v & 1u) b.words = false;
    }
    b.spare = (long long)batch * w.plan.tiles > ssd::kColsumRows ? at(w.spare) : nullptr;
    return status_of(ssd::launch_rec_bwd(b, dtype == SSD_BF16, s));
}

int ssd_dropout(const void *x, long long x_row_stride, long long rows, int width, const ssd_random *random,
                int dtype, void *y, void *stream) {
    if (!x || !y || !random) return SSD_ERR_NULL;
    if (rows < 1 || width < 1 || x_row_stride < 0) return SSD_ERR_SHAPE;
    if (width > kMaxExtent || rows > kMaxRows || !valid_dtype(dtype)) return SSD_ERR_UNSUPPORTED;
    ssd::DropoutArgs a{};
    const int rc = drop_args(a.drop, random);
    if (rc != SSD_OK) return rc;
    a.x = x;
    a.x_stride = static_cast<size_t>(x_row_stride);
    a.rows = rows;
    a.width = width;
    a.y = y;
    return status_of(ssd::launch_dropout(a, dtype == SSD_BF16, static_cast<hipStream_t>(stream)));
}

int ssd_block_norm_forward(const void *x, long long x_row_stride, const void *residual, int stream_dtype,
                           const void *z, long long z_row_stride, const ssd_block *block,
                           const ssd_random *random, long long rows, int width, int dtype, void *y,
                           void *sum, float *mean, float *rstd, float *post_mean, float *post_rstd,
                           void *stream) {
    if (!x || !residual || !sum) return SSD_ERR_NULL;
    int rc = check_block(block, stream_dtype, z, z_row_stride, x_row_stride, rows, width, dtype);
    if (rc != SSD_OK) return rc;
    if (block->weight && !y) return SSD_ERR_NULL;
    ssd::BlockArgs a{};
    rc = drop_args(a.drop, random);
    if (rc != SSD_OK) return rc;
    a.x = x; a.residual = residual; a.z = z;
    a.x_stride = static_cast<size_t>(x_row_stride);
    a.z_stride = static_cast<size_t>(z_row_stride);
    a.weight = block->weight; a.bias = block->bias;
    a.post_weight = block->post_weight; a.post_bias = block->post_bias;
    a.scale = block->scale;
    a.alpha = block->residual_scale; a.beta = block->branch_scale; a.eps = block->eps;
    a.rows = rows;
    a.width = width;
    a.rms = block->rms != 0;
    a.y = y; a.sum = sum;
    a.mean = mean; a.rstd = rstd; a.post_mean = post_mean; a.post_rstd = post_rstd;
    return status_of(ssd::launch_block_fwd(a, dtype == SSD_BF16, stream_dtype == SSD_BF16,
                                           static_cast<hipStream_t>(stream)));
}

size_t ssd_block_norm_backward_workspace_size(long long rows, int width, int dtype) {
    if (rows < 1 || rows > kMaxRows || width < 1 || width > ssd::kMaxBlockWidth || !valid_dtype(dtype)) return 0;
    const size_t full = ssd::block_bwd_part_bytes(rows, width, dtype == SSD_BF16, true, 4);
    const size_t lean = ssd::block_bwd_part_bytes(rows, width, dtype == SSD_BF16, false, 2);
    return full > lean ? full : lean;
}

int ssd_block_norm_backward(const void *dy, const void *dsum, const void *x, long long x_row_stride,
                            const void *sum, int stream_dtype, const void *z, long long z_row_stride,
                            const ssd_block *block, const ssd_random *random, const float *mean,
                            const float *rstd, const float *post_mean, const float *post_rstd,
                            long long rows, int width, int dtype, void *dx, void *dresidual, void *dz,
                            float *dweight, float *dbias, float *dpost_weight, float *dpost_bias,
                            float *dscale, void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !dx || !dresidual || (z && !dz)) return SSD_ERR_NULL;
    int rc = check_block(block, stream_dtype, z, z_row_stride, x_row_stride, rows, width, dtype);
    if (rc != SSD_OK) return rc;
    const bool means = !block->rms;
    if (block->weight && (!dy || !sum || !rstd || (means && !mean))) return SSD_ERR_NULL;
    if (block->post_weight && (!post_rstd || (means && !post_mean))) return SSD_ERR_NULL;
    // gradients of what is not there
    if ((!block->weight && (dy || dweight || dbias)) || (!block->post_weight && (dpost_weight || dpost_bias)) ||
        (!block->scale && dscale))
        return SSD_ERR_UNSUPPORTED;
    ssd::BlockBwdArgs a{};
    rc = drop_args(a.drop, random);
    if (rc != SSD_OK) return rc;
    a.sums = block_sums(dweight, dbias, dpost_weight, dpost_bias, dscale, block->post_bias, &a.want_p, &a.want_q);
    a.dy = dy; a.dsum = dsum; a.x = x; a.sum = sum; a.z = z;
    a.x_stride = static_cast<size_t>(x_row_stride);
    a.z_stride = static_cast<size_t>(z_row_stride);
    a.weight = block->weight;
    a.post_weight = block->post_weight; a.post_bias = block->post_bias;
    a.scale = block->scale;
    a.mean = means ? mean : nullptr; a.rstd = rstd;
    a.post_mean = means ? post_mean : nullptr; a.post_rstd = post_rstd;
    a.alpha = block->residual_scale; a.beta = block->branch_scale;
    a.rows = rows;
    a.width = width;
    a.dx = dx; a.dresidual = dresidual; a.dz = dz;
    a.dweight = dweight; a.dbias = dbias;
    a.dpost_weight = dpost_weight; a.dpost_bias = dpost_bias; a.dscale = dscale;
    a.part = static_cast<float *>(workspace);
    rc = check_workspace(workspace, workspace_bytes,
                         ssd::block_bwd_part_bytes(rows, width, dtype == SSD_BF16, ssd::block_bwd_full(a), a.sums));
    if (rc != SSD_OK) return rc;
    return status_of(ssd::launch_block_bwd(a, dtype == SSD_BF16, stream_dtype == SSD_BF16,
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
