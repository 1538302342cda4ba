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
int status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

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

}  // extern "C"
