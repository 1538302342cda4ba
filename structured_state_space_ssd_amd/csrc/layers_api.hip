// C ABI of the operators around the state-space layers: the short causal
// convolution, the selective scan and the normalisation. Argument checks,
// workspace sizes and launches; every declaration and its contract is in
// include/ssd.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_launch.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxNormWidth = 16384;
// token and channel counts above this leave no room for tile arithmetic in int
constexpr int kMaxExtent = 1 << 30;

bool valid_dtype(int d) { return d == SSD_F32 || d == SSD_BF16; }
// (hipErrorNotSupported: a launch's own refusal of a grid, before anything is enqueued)
int status_of(hipError_t e) {
    return e == hipSuccess ? SSD_OK : e == hipErrorNotSupported ? SSD_ERR_UNSUPPORTED : SSD_ERR_HIP;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return SSD_OK;
    if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0)
        return SSD_ERR_WORKSPACE;
    return SSD_OK;
}

// The parts of the channel axis (split NULL: one part, all of it).
int conv_parts(const int *split, int nsplit, int channels, void *const *ptr, ssd::ConvParts &p) {
    p = ssd::ConvParts{};
    if (!ptr) return SSD_ERR_NULL;
    if (!split) {
        p.n = 1;
        p.count[0] = channels;
        p.ptr[0] = ptr[0];
        return p.ptr[0] ? SSD_OK : SSD_ERR_NULL;
    }
    if (nsplit < 1 || nsplit > 3) return SSD_ERR_SHAPE;
    p.n = nsplit;
    long long at = 0;
    for (int i = 0; i < nsplit; ++i) {
        if (split[i] < 1) return SSD_ERR_SHAPE;
        if (!ptr[i]) return SSD_ERR_NULL;
        p.first[i] = static_cast<int>(at);
        p.count[i] = split[i];
        p.ptr[i] = ptr[i];
        at += split[i];
        if (at > channels) return SSD_ERR_SHAPE;
    }
    return at == channels ? SSD_OK : SSD_ERR_SHAPE;
}

int check_conv(int batch, int seqlen, int channels, int width, int dtype, long long x_batch,
               long long x_row) {
    if (batch < 1 || seqlen < 1 || channels < 1) return SSD_ERR_SHAPE;
    if (seqlen > kMaxExtent || channels > kMaxExtent) return SSD_ERR_SHAPE;
    if (width < 2 || width > 4 || !valid_dtype(dtype)) return SSD_ERR_UNSUPPORTED;
    if (x_batch < 0 || x_row < 0) return SSD_ERR_SHAPE;
    return SSD_OK;
}

int check_norm(long long rows, int width, int dtype) {
    if (rows < 1 || width < 1) return SSD_ERR_SHAPE;
    if (width > kMaxNormWidth || !valid_dtype(dtype)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
// The stream beside x has x's type or is float32.
bool stream_dtype_ok(int stream, int dtype) { return stream == dtype || stream == SSD_F32; }

constexpr long long kMaxTokenStride = 1LL << 24;
// Grids hold fewer than 2^24 workgroups of 256 lanes.
constexpr long long kMaxBlocks = 1LL << 24;

int check_selective(int batch, int seqlen, int channels, int ngroups, int dstate, int dtype) {
    if (batch < 1 || seqlen < 1 || channels < 1 || ngroups < 1 || dstate < 1) return SSD_ERR_SHAPE;
    if (channels % ngroups != 0 || seqlen > kMaxExtent || channels > kMaxExtent)
        return SSD_ERR_SHAPE;
    if (!ssd::selective_kernel_dstate(dstate) || !valid_dtype(dtype)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Strides (NULL: dense) and options into the kernels' arguments.
int selective_args(ssd::SelArgs &a, const void *x, const void *dt, const float *A, const void *B,
                   const void *C, const float *D, const void *z, int batch, int seqlen,
                   int channels, int ngroups, int dstate, const ssd_selective_strides *st,
                   const ssd_options *o) {
    a = ssd::SelArgs{};
    a.x = x; a.dt = dt; a.z = z; a.B = B; a.C = C; a.A = A; a.D = D;
    a.batch = batch; a.seqlen = seqlen; a.channels = channels; a.ngroups = ngroups;
    a.dstate = dstate;
    const long long e = channels, n = (long long)ngroups * dstate;
    ssd_selective_strides d = {e * seqlen, e, e * seqlen, e, e * seqlen, e, n * seqlen, n,
                               n * seqlen, n};
    if (st) {
        d = *st;
        if (seqlen == 1)  // a single token has no stride between tokens
            d.x_token = d.dt_token = d.z_token = d.B_token = d.C_token = 0;
        for (long long v : {d.x_batch, d.x_token, d.dt_batch, d.dt_token, d.z_batch, d.z_token,
                            d.B_batch, d.B_token, d.C_batch, d.C_token})
            if (v < 0) return SSD_ERR_SHAPE;
    }
    // offsets within a tile of tokens are 32 bits of bytes, in dense tensors as well
    if (e >= kMaxTokenStride) return SSD_ERR_UNSUPPORTED;
    for (long long v : {d.x_token, d.dt_token, d.z_token, d.B_token, d.C_token})
        if (v >= kMaxTokenStride) return SSD_ERR_UNSUPPORTED;
    a.x_batch = d.x_batch; a.x_token = d.x_token; a.dt_batch = d.dt_batch; a.dt_token = d.dt_token;
    a.z_batch = d.z_batch; a.z_token = d.z_token; a.B_batch = d.B_batch; a.B_token = d.B_token;
    a.C_batch = d.C_batch; a.C_token = d.C_token;
    a.opts = ssd::DtOpts{nullptr, 0.0f, 0.0f, 0, 0, 0};
    if (!o) return SSD_OK;
    if (o->discretization != SSD_DISC_EULER) return SSD_ERR_OPTION;
    if (o->dt_clamp && !(o->dt_min <= o->dt_max)) return SSD_ERR_OPTION;  // NaN bounds fail too
    if ((reinterpret_cast<uintptr_t>(o->dt_bias) & 3u) != 0) return SSD_ERR_UNSUPPORTED;
    a.opts = ssd::DtOpts{o->dt_bias, o->dt_min, o->dt_max, o->dt_softplus != 0, o->dt_clamp != 0, 0};
    return SSD_OK;
}

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct Taker {
    size_t o = 0;
    size_t take(size_t floats) {
        const size_t at = o;
        o += align_up(floats * sizeof(float));
        return at;
    }
};

// The selective scan's plan and where its workspace's parts begin.
struct SelLayout {
    ssd::SelPlan plan;
    size_t bc, seg_state, seg_sum, total;
};
SelLayout selective_layout(int batch, int seqlen, int channels, int ngroups, int dstate) {
    SelLayout w{};
    w.plan = ssd::selective_plan(batch, seqlen, channels, ngroups, dstate);
    Taker k;
    w.bc = k.take(ssd::selective_bc_floats(batch, seqlen, ngroups, dstate));
    w.seg_state = k.take(w.plan.seg_floats);
    w.seg_sum = k.take((size_t)batch * channels * (w.plan.segs - 1));
    w.total = k.o;
    return w;
}

// The layout of B and C, and the walks' workgroups of 256 lanes.
bool selective_grid_ok(int batch, int seqlen, int channels, int ngroups, int dstate, int segs) {
    return (long long)ssd::selective_blocks(channels, ngroups, dstate) * segs * batch < kMaxBlocks &&
           ssd::selective_bc_floats(batch, seqlen, ngroups, dstate) / 256 < (size_t)kMaxBlocks - 1;
}

// The selective scan's backward: its plan and where its workspace's parts begin.
struct SelBwdLayout {
    ssd::SelPlan plan;
    int keeps;
    size_t bc, keep_state, keep_sum, seg_state, seg_sum, seg_adj, dbc, dA, de, total;
};
SelBwdLayout selective_bwd_layout(int batch, int seqlen, int channels, int ngroups, int dstate) {
    SelBwdLayout w{};
    w.plan = ssd::selective_bwd_plan(batch, seqlen, channels, ngroups, dstate);
    const size_t nk = ssd::selective_kernel_dstate(dstate), be = (size_t)batch * channels;
    const int keep = ssd::selective_keep_tokens(dstate);
    w.keeps = (seqlen + keep - 1) / keep;
    const size_t segs = w.plan.segs, later = segs - 1;
    Taker k;
    w.bc = k.take(ssd::selective_bc_floats(batch, seqlen, ngroups, dstate));
    w.keep_state = k.take(be * w.keeps * nk);
    w.keep_sum = k.take(be * w.keeps);
    w.seg_state = k.take(w.plan.seg_floats);
    w.seg_sum = k.take(be * later);
    w.seg_adj = k.take(w.plan.seg_floats);
    w.dbc = k.take(ssd::selective_dbc_floats(batch, seqlen, channels, ngroups, dstate));
    w.dA = k.take(be * segs * dstate);
    w.de = k.take(2 * be * segs);
    w.total = k.o;
    return w;
}

}  // namespace

extern "C" {

int ssd_conv_forward(const void *x, long long x_batch_stride, long long x_token_stride,
                     const float *weight, const float *bias, const void *init_state,
                     const int *cu_seqlens, int nseq, int batch, int seqlen, int channels,
                     int width, int silu, int dtype, const int *split, int nsplit, void *const *y,
                     void *final_state, void *stream) {
    if (!x || !weight) return SSD_ERR_NULL;
    int rc = check_conv(batch, seqlen, channels, width, dtype, x_batch_stride, x_token_stride);
    if (rc != SSD_OK) return rc;
    ssd::ConvArgs a{};
    rc = conv_parts(split, nsplit, channels, y, a.y);
    if (rc != SSD_OK) return rc;
    if (cu_seqlens) {
        if (batch != 1 || nseq < 1) return SSD_ERR_SHAPE;
        if (init_state) return SSD_ERR_UNSUPPORTED;
    }
    a.x = x;
    a.init = init_state;
    a.x_batch = static_cast<size_t>(x_batch_stride);
    a.x_row = static_cast<size_t>(x_token_stride);
    a.weight = weight;
    a.bias = bias;
    a.cu_seqlens = cu_seqlens;
    a.nseq = nseq;
    a.batch = batch;
    a.seqlen = seqlen;
    a.channels = channels;
    a.width = width;
    a.silu = silu != 0;
    a.final_state = final_state;
    return status_of(ssd::launch_conv_fwd(a, dtype == SSD_BF16, static_cast<hipStream_t>(stream)));
}

size_t ssd_conv_backward_workspace_size(int batch, int seqlen, int channels, int width, int dtype) {
    if (check_conv(batch, seqlen, channels, width, dtype, 0, 0) != SSD_OK) return 0;
    return ssd::conv_bwd_part_bytes(batch, seqlen, channels, width);
}

int ssd_conv_backward(const void *x, long long x_batch_stride, long long x_token_stride,
                      const float *weight, const float *bias, const void *init_state,
                      const int *split, int nsplit, void *const *dy, const void *dfinal_state,
                      int batch, int seqlen, int channels, int width, int silu, int dtype,
                      void *dx, float *dweight, float *dbias, void *dinit_state, void *workspace,
                      size_t workspace_bytes, void *stream) {
    if (!x || !weight || !dx || !dweight) return SSD_ERR_NULL;
    int rc = check_conv(batch, seqlen, channels, width, dtype, x_batch_stride, x_token_stride);
    if (rc != SSD_OK) return rc;
    ssd::ConvBwdArgs a{};
    rc = conv_parts(split, nsplit, channels, dy, a.dy);
    if (rc != SSD_OK) return rc;
    if (!ssd::conv_bwd_grid_ok(batch, seqlen, channels, width, a.dy)) return SSD_ERR_UNSUPPORTED;
    rc = check_workspace(workspace, workspace_bytes,
                         ssd::conv_bwd_part_bytes(batch, seqlen, channels, width));
    if (rc != SSD_OK) return rc;
    a.x = x;
    a.init = init_state;
    a.dfinal = dfinal_state;
    a.x_batch = static_cast<size_t>(x_batch_stride);
    a.x_row = static_cast<size_t>(x_token_stride);
    a.weight = weight;
    a.bias = bias;
    a.batch = batch;
    a.seqlen = seqlen;
    a.channels = channels;
    a.width = width;
    a.silu = silu != 0;
    a.dx = dx;
    a.dinit = dinit_state;
    a.dweight = dweight;
    a.dbias = dbias;
    a.part = static_cast<float *>(workspace);
    return status_of(ssd::launch_conv_bwd(a, dtype == SSD_BF16, static_cast<hipStream_t>(stream)));
}

int ssd_conv_step(void *state, const void *x, long long x_batch_stride, const float *weight,
                  const float *bias, int batch, int channels, int width, int silu, int dtype,
                  const int *split, int nsplit, void *const *y, void *stream) {
    if (!state || !x || !weight) return SSD_ERR_NULL;
    int rc = check_conv(batch, 1, channels, width, dtype, x_batch_stride, 0);
    if (rc != SSD_OK) return rc;
    ssd::ConvParts parts;
    rc = conv_parts(split, nsplit, channels, y, parts);
    if (rc != SSD_OK) return rc;
    return status_of(ssd::launch_conv_step(state, x, static_cast<size_t>(x_batch_stride), weight,
                                           bias, batch, channels, width, silu != 0, parts,
                                           dtype == SSD_BF16, static_cast<hipStream_t>(stream)));
}

int ssd_norm_forward(const void *x, long long x_row_stride, const void *residual,
                     int residual_dtype, const void *z, long long z_row_stride,
                     const float *weight, const float *bias, long long rows, int width, int rms,
                     float eps, int dtype, void *y, void *residual_out, float *mean, float *rstd,
                     void *stream) {
    if (!x || !weight || !y || (residual && !residual_out)) return SSD_ERR_NULL;
    const int rc = check_norm(rows, width, dtype);
    if (rc != SSD_OK) return rc;
    if (x_row_stride < 0 || z_row_stride < 0) return SSD_ERR_SHAPE;
    if (!(eps >= 0.0f)) return SSD_ERR_OPTION;
    if (residual && (z || !stream_dtype_ok(residual_dtype, dtype))) return SSD_ERR_UNSUPPORTED;
    ssd::NormArgs a{};
    a.x = x;
    a.residual = residual;
    a.z = z;
    a.x_stride = static_cast<size_t>(x_row_stride);
    a.z_stride = static_cast<size_t>(z_row_stride);
    a.weight = weight;
    a.bias = bias;
    a.rows = rows;
    a.width = width;
    a.rms = rms != 0;
    a.eps = eps;
    a.y = y;
    a.residual_out = residual_out;
    a.mean = mean;
    a.rstd = rstd;
    return status_of(ssd::launch_norm_fwd(a, dtype == SSD_BF16, residual_dtype == SSD_BF16,
                                          static_cast<hipStream_t>(stream)));
}

size_t ssd_norm_backward_workspace_size(long long rows, int width, int dtype, int want_dbias) {
    if (check_norm(rows, width, dtype) != SSD_OK) return 0;
    return ssd::norm_bwd_part_bytes(rows, width, dtype == SSD_BF16, want_dbias != 0);
}

int ssd_norm_backward(const void *dy, const void *x, long long x_row_stride, int x_dtype,
                      const void *z, long long z_row_stride, const float *weight,
                      const float *mean, const float *rstd, const void *dresidual, long long rows,
                      int width, int dtype, void *dx, void *dresidual_in, void *dz,
                      float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                      void *stream) {
    if (!dy || !x || !weight || !rstd || !dx || !dweight || (z && !dz)) return SSD_ERR_NULL;
    int rc = check_norm(rows, width, dtype);
    if (rc != SSD_OK) return rc;
    if (x_row_stride < 0 || z_row_stride < 0) return SSD_ERR_SHAPE;
    if (!stream_dtype_ok(x_dtype, dtype)) return SSD_ERR_UNSUPPORTED;
    if (z && (x_dtype != dtype || dresidual || dresidual_in)) return SSD_ERR_UNSUPPORTED;
    rc = check_workspace(workspace, workspace_bytes,
                         ssd::norm_bwd_part_bytes(rows, width, dtype == SSD_BF16, dbias != nullptr));
    if (rc != SSD_OK) return rc;
    ssd::NormBwdArgs a{};
    a.dy = dy;
    a.x = x;
    a.z = z;
    a.dresidual = dresidual;
    a.x_stride = static_cast<size_t>(x_row_stride);
    a.z_stride = static_cast<size_t>(z_row_stride);
    a.weight = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.width = width;
    a.dx = dx;
    a.dresidual_in = dresidual_in;
    a.dz = dz;
    a.dweight = dweight;
    a.dbias = dbias;
    a.part = static_cast<float *>(workspace);
    return status_of(ssd::launch_norm_bwd(a, dtype == SSD_BF16, x_dtype == SSD_BF16,
                                          static_cast<hipStream_t>(stream)));
}

size_t ssd_selective_forward_workspace_size(int batch, int seqlen, int channels, int ngroups,
                                            int dstate, int dtype) {
    if (check_selective(batch, seqlen, channels, ngroups, dstate, dtype) != SSD_OK) return 0;
    return selective_layout(batch, seqlen, channels, ngroups, dstate).total;
}

int ssd_selective_forward(const void *x, const void *dt, const float *A, const void *B,
                          const void *C, const float *D, const void *z, int batch, int seqlen,
                          int channels, int ngroups, int dstate, int dtype,
                          const float *init_state, void *y, float *final_state, void *workspace,
                          size_t workspace_bytes, const ssd_selective_strides *strides,
                          const ssd_options *opts, void *stream) {
    if (!x || !dt || !A || !B || !C || !y) return SSD_ERR_NULL;
    int rc = check_selective(batch, seqlen, channels, ngroups, dstate, dtype);
    if (rc != SSD_OK) return rc;
    ssd::SelArgs a;
    rc = selective_args(a, x, dt, A, B, C, D, z, batch, seqlen, channels, ngroups, dstate, strides,
                        opts);
    if (rc != SSD_OK) return rc;
    const SelLayout w = selective_layout(batch, seqlen, channels, ngroups, dstate);
    if (!selective_grid_ok(batch, seqlen, channels, ngroups, dstate, w.plan.segs))
        return SSD_ERR_UNSUPPORTED;
    rc = check_workspace(workspace, workspace_bytes, w.total);
    if (rc != SSD_OK) return rc;
    char *base = static_cast<char *>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(base + off); };
    a.units = w.plan.units;
    a.whole = w.plan.whole;
    a.segs = w.plan.segs;
    a.seg_len = w.plan.seg_len;
    a.bc = at(w.bc);
    a.seg_state = at(w.seg_state);
    a.seg_sum = at(w.seg_sum);
    a.init = init_state;
    a.y = y;
    a.final_state = final_state;
    return status_of(ssd::launch_selective_fwd(a, dtype == SSD_BF16, static_cast<hipStream_t>(stream)));
}

int ssd_selective_step(float *state, const void *x, const void *dt, const float *A, const void *B,
                       const void *C, const float *D, const void *z, int batch, int channels,
                       int ngroups, int dstate, int dtype, void *y,
                       const ssd_selective_strides *strides, const ssd_options *opts,
                       void *stream) {
    if (!state || !x || !dt || !A || !B || !C || !y) return SSD_ERR_NULL;
    int rc = check_selective(batch, 1, channels, ngroups, dstate, dtype);
    if (rc != SSD_OK) return rc;
    if ((long long)batch * channels * (ssd::selective_kernel_dstate(dstate) / 4) / 256 >= kMaxBlocks - 1)
        return SSD_ERR_UNSUPPORTED;
    ssd::SelArgs a;
    rc = selective_args(a, x, dt, A, B, C, D, z, batch, 1, channels, ngroups, dstate, strides, opts);
    if (rc != SSD_OK) return rc;
    a.y = y;
    return status_of(ssd::launch_selective_step(a, state, dtype == SSD_BF16,
                                                static_cast<hipStream_t>(stream)));
}

size_t ssd_selective_backward_workspace_size(int batch, int seqlen, int channels, int ngroups,
                                             int dstate, int dtype) {
    if (check_selective(batch, seqlen, channels, ngroups, dstate, dtype) != SSD_OK) return 0;
    return selective_bwd_layout(batch, seqlen, channels, ngroups, dstate).total;
}

int ssd_selective_backward(const void *x, const void *dt, const float *A, const void *B,
                           const void *C, const float *D, const void *z, const float *init_state,
                           const void *dy, const float *dfinal_state, int batch, int seqlen,
                           int channels, int ngroups, int dstate, int dtype, void *dx, void *ddt,
                           float *dA, void *dB, void *dC, float *dD, void *dz, float *dinit_state,
                           float *ddt_bias, void *workspace, size_t workspace_bytes,
                           const ssd_selective_strides *strides, const ssd_options *opts,
                           void *stream) {
    if (!x || !dt || !A || !B || !C || !dy || !dx || !ddt || !dA || !dB || !dC || (z && !dz))
        return SSD_ERR_NULL;
    int rc = check_selective(batch, seqlen, channels, ngroups, dstate, dtype);
    if (rc != SSD_OK) return rc;
    ssd::SelBwdArgs b{};
    rc = selective_args(b.f, x, dt, A, B, C, D, z, batch, seqlen, channels, ngroups, dstate,
                        strides, opts);
    if (rc != SSD_OK) return rc;
    const SelBwdLayout w = selective_bwd_layout(batch, seqlen, channels, ngroups, dstate);
    if (!selective_grid_ok(batch, seqlen, channels, ngroups, dstate, w.plan.segs) ||
        !ssd::selective_bwd_grid_ok(batch, seqlen, channels, ngroups, dstate, w.plan.segs))
        return SSD_ERR_UNSUPPORTED;
    rc = check_workspace(workspace, workspace_bytes, w.total);
    if (rc != SSD_OK) return rc;
    char *base = static_cast<char *>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(base + off); };
    b.f.init = init_state;
    b.f.units = w.plan.units;
    b.f.whole = w.plan.whole;
    b.f.segs = w.plan.segs;
    b.f.seg_len = w.plan.seg_len;
    b.f.bc = at(w.bc);
    b.f.seg_state = at(w.seg_state);
    b.f.seg_sum = at(w.seg_sum);
    b.f.keeps = w.keeps;
    b.f.keep_state = at(w.keep_state);
    b.f.keep_sum = at(w.keep_sum);
    b.f.dy = dy;
    b.f.dfinal = dfinal_state;
    b.f.seg_adj = at(w.seg_adj);
    b.dbc_part = at(w.dbc);
    b.dA_part = at(w.dA);
    b.de_part = at(w.de);
    b.dx = dx; b.ddt = ddt; b.dz = dz; b.dB = dB; b.dC = dC;
    b.dA = dA; b.dD = dD; b.ddt_bias = ddt_bias; b.dinit = dinit_state;
    return status_of(ssd::launch_selective_bwd(b, dtype == SSD_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
