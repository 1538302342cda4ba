// Host-side launchers of the SSD kernels (one per kernel source file). They
// assume arguments were validated by the C-ABI layer (ssd_api.hip) and return
// the hipError_t of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace ssd {

// Step-size preprocessing and input discretisation, passed to the kernels by
// value. The selection mechanism makes the step size a projection of the
// input made positive by softplus ("从Transformer到Mamba" tutorial, section
// 3.2): `bias` is that projection's per-head constant term, added first; an
// optional clamp to [lo, hi] follows softplus (the tutorial's section 8.2
// adjusts the range step sizes are produced in). The input term is weighted by
// the step size (Euler) or, with `zoh`, by the zero-order hold's
// (exp(dt A) - 1) / A (tutorial section 2.2; "Mamba 模型" section 2.3.1).
struct DtOpts {
    const float *bias;  // [H], or nullptr
    float lo, hi;       // clamp bounds, read when clamp != 0
    int softplus, clamp, zoh;
};

// delta (nullable): each token's input weight (the preprocessed step size, or
// its zero-order-hold weight) as float32 in dA_cumsum's chunk-padded layout,
// zero past the end. The later stages read it in place of dt.
hipError_t launch_chunk_cumsum(const void *dt, const float *A, int batch, int seqlen, int nheads,
                               int chunk, bool bf16, const DtOpts &opts, float *dA_cumsum,
                               float *delta, hipStream_t stream);

// seg (nullable): packed sequences, one int per token in dA_cumsum's chunk-padded
// layout: the first token of the token's sequence relative to its chunk's first
// token, or -1 if that sequence began in an earlier chunk (launch_varlen_seg).
// dout (backward): the same contraction with token weights exp(s_j) instead of
// exp(s_end - s_j) delta_j, i.e. sum_j exp(s_j) x_j B_j^T with x := dy and
// B := C: how a chunk's outputs depend on the state entering it (delta unused).
hipError_t launch_chunk_state(const void *x, const void *B, const float *delta,
                              const float *dA_cumsum, const int *seg,
                              int batch, int seqlen, int nheads, int ngroups, int dstate, int chunk,
                              bool bf16, float *states, hipStream_t stream, bool dout = false);

// The single-pass bf16 forward (fwd_onepass.hip): whether it applies; how
// it cuts each sequence; and the launch (two kernels when there are several
// segments: the segment states, then the forward proper; `between`
// (nullable) is recorded between them).
bool forward_onepass_ok(int batch, int nheads, int dstate, bool bf16, const void *dt);
// S segments of per_seg 64-token blocks each (the last may hold fewer); when
// S > 1 the first S - 1 segments are cut into k pieces of psub blocks, whose
// states (float32 [Bt][H][(S-1)k][P][N]) and log2-decays (float32
// [Bt][H][(S-1)k]) take scratch_bytes of scratch. S == 1: k == 0, no scratch.
struct OnepassPlan {
    int S, k, per_seg, psub;
    size_t scratch_bytes;
};
// cap: the most scratch the plan may take (SIZE_MAX: no limit); a smaller cap
// lowers k, then gives up the segments.
OnepassPlan forward_onepass_plan(int batch, int seqlen, int nheads, int dstate, size_t cap);
// Packed sequences (batch 1, no init_state / final_state): `varlen_meta`
// holds one int4 per token made by launch_onepass_varlen_prep from cu_seqlens
// (16 * seqlen bytes, 16-byte aligned); each sequence's final state goes to
// seq_states (nullable) [nseq][H][P][N]; the prep also zeroes the empty ones.
// `scratch` must hold pl.scratch_bytes (it may be NULL when that is 0).
hipError_t launch_forward_onepass(const void *x, const void *dt, const float *A, const void *B,
                                  const void *C, const float *D, const float *init,
                                  const DtOpts &opts, int batch, int seqlen, int nheads,
                                  int ngroups, int dstate, const OnepassPlan &pl, float *scratch,
                                  void *y, float *final_state, hipEvent_t between,
                                  hipStream_t stream, const void *varlen_meta = nullptr,
                                  float *seq_states = nullptr);
hipError_t launch_onepass_varlen_prep(const int *cu_seqlens, int nseq, int seqlen, int nheads,
                                      int dstate, void *meta, float *seq_states,
                                      hipStream_t stream);

// Stages 2 and 3 in one kernel (bf16 only; used when state_passing_fused()):
// writes chunk_init (bf16) and final_state (nullable) directly, without the
// per-chunk float32 states. Reads dA_cumsum and delta (stage 1's outputs).
bool state_passing_fused(int batch, int nheads, bool bf16);
// reverse (backward): the adjoint pass (x = dy, B = C, init = dfinal; chunk_init
// receives the gradient of the state leaving each chunk, final_state G_0).
hipError_t launch_chunk_state_passing(const void *x, const void *B, const float *dA_cumsum,
                                      const float *delta, const float *init, int batch,
                                      int seqlen, int nheads, int ngroups, int dstate, int chunk,
                                      void *chunk_init, float *final_state, hipStream_t stream,
                                      bool reverse = false);

// chunk_init is written in the MFMA operand type of the forward's dtype
// (bf16 when bf16 is true, else float32). reverse (backward): the adjoint pass,
// from init = dfinal over the chunks in reverse (see state_passing.hip).
hipError_t launch_state_passing(const float *states, const float *dA_cumsum, const float *init,
                                const int *seg, int batch, int seqlen, int nheads, int dstate, int chunk,
                                bool bf16, void *chunk_init, float *final_state,
                                hipStream_t stream, bool reverse = false);

size_t chunk_cb_bytes(int batch, int seqlen, int ngroups, int chunk, bool bf16);

hipError_t launch_chunk_cb(const void *B, const void *C, int batch, int seqlen, int ngroups,
                           int dstate, int chunk, bool bf16, void *cb, hipStream_t stream);

// The bf16 path forms C B^T itself (reads B, ignores cb); the float path reads
// the C B^T tiles of launch_chunk_cb (reads cb, ignores B).
bool chunk_scan_reads_cb(bool bf16);

hipError_t launch_chunk_scan(const void *x, const float *delta, const float *dA_cumsum, const void *B,
                             const void *C, const void *cb, const float *D, const void *chunk_init,
                             const int *seg, int batch, int seqlen, int nheads, int ngroups, int dstate, int chunk,
                             bool bf16, void *y, hipStream_t stream);

// Packed sequences (batch 1): seg of every token position (nC*Q ints) from
// cu_seqlens [nseq + 1]; and each sequence's state after its last token,
// seq_states [nseq][H][P][N] float32, from the stage outputs (chunk_init in the
// operand type of the forward's dtype).
hipError_t launch_varlen_seg(const int *cu_seqlens, int nseq, int seqlen, int chunk, int *seg,
                             hipStream_t stream);
hipError_t launch_varlen_final_states(const void *x, const void *B, const float *delta,
                                      const float *dA_cumsum, const int *cu_seqlens,
                                      const int *seg, const void *chunk_init, int nseq,
                                      int seqlen, int nheads, int ngroups, int dstate, int chunk,
                                      bool bf16, float *seq_states, hipStream_t stream);

// ---- backward (chunk_bwd.hip)
// Chunk length the backward runs with (0: unsupported) and its head blocks.
int bwd_chunk(int dstate, bool bf16);
int bwd_head_blocks(int batch, int seqlen, int nheads, int ngroups, int chunk);

struct BwdArgs {
    const void *x, *dy, *B, *C;
    const float *dA_cumsum, *delta, *D;
    const void *chunk_init, *grad_next;  // operand type: H_c and the adjoint G_{c+1}
    int batch, seqlen, nheads, ngroups, dstate, chunk, nblk;
    bool bf16;
    void *dx;
    float *ds, *dw;                 // [Bt][H][nC*Q]
    float *dB_part, *dC_part;       // [nblk][Bt][L][G][N]
    float *dD_part;                 // [Bt][nC][H]
};
hipError_t launch_chunk_bwd(const BwdArgs &a, hipStream_t stream);
// out0, out1 (input dtype, count elements each, count a multiple of 4) = the
// sums over nblk of part0[k][count], part1[k][count], in one launch
hipError_t launch_bwd_reduce(const float *part0, const float *part1, int nblk, size_t count,
                             bool bf16, void *out0, void *out1, hipStream_t stream);
hipError_t launch_bwd_dt(const void *dt, const float *A, const float *ds, const float *dw,
                         int batch, int seqlen, int nheads, int chunk, bool bf16,
                         const DtOpts &opts, void *ddt, float *dA_part, float *dbias_part,
                         hipStream_t stream);
// out[j][h] = sum_i part[j][i][h], i < nbc, for the j < n (at most 3) whose out[j] is
// not NULL, in one launch
hipError_t launch_bwd_head_sum(const float *const *part, float *const *out, int n, int nbc,
                               int nheads, hipStream_t stream);

// State-size padding (pad.hip): the N the kernels run with for dstate (the
// smallest of 16, 32, 64, 128, 256 not below it; 0 above 256), and a copy of
// `rows` rows of src_cols elements into rows of dst_cols elements, zero-filled
// past src_cols or cut to dst_cols (both column counts times elem_bytes must
// be multiples of 16; src and dst 16-byte aligned).
int kernel_dstate(int dstate);
hipError_t launch_pad_rows(const void *src, void *dst, size_t rows, int src_cols, int dst_cols,
                           int elem_bytes, hipStream_t stream);

// dstate: any multiple of 16 up to 256 (the kernel for 16, 32, 64, 128, 256
// keeps the state's rows in lanes that share them by powers of two; the other
// sizes reduce each row's products through LDS).
hipError_t launch_decode_step(float *state, const void *x, const void *dt, const float *A,
                              const void *B, const void *C, const float *D, int batch, int nheads,
                              int ngroups, int dstate, bool bf16, const DtOpts &opts, void *y,
                              hipStream_t stream);

// ---- normalisation (norm.hip)
// Rows of `width` elements; x and z rows `x_stride`, `z_stride` elements
// apart, every other tensor dense. residual / z / bias / mean / rstd nullable.
struct NormArgs {
    const void *x, *residual, *z;
    size_t x_stride, z_stride;
    const float *weight, *bias;
    long long rows;
    int width, rms;
    float eps;
    void *y, *residual_out;
    float *mean, *rstd;
};
hipError_t launch_norm_fwd(const NormArgs &a, bool bf16, bool res_bf16, hipStream_t stream);
// mean NULL: the root-mean-square form. part: norm_bwd_part_bytes of scratch.
struct NormBwdArgs {
    const void *dy, *x, *z, *dresidual;
    size_t x_stride, z_stride;
    const float *weight, *mean, *rstd;
    long long rows;
    int width;
    void *dx, *dresidual_in, *dz;
    float *dweight, *dbias, *part;
};
size_t norm_bwd_part_bytes(long long rows, int width, bool bf16, bool want_db);
hipError_t launch_norm_bwd(const NormBwdArgs &a, bool bf16, bool x_bf16, hipStream_t stream);
// out[c] = sum over k < n of part[k][c], c < cols, in a fixed order; columns
// below `first` go to out0, the others to out1. More than kColsumRows rows are first
// summed to kColsumChunks of them where `spare` has room for those: few columns
// would leave all rows to few workgroups (convolution backward, 1048576 tokens of 16
// channels: 115 us in one pass, 36 in two).
constexpr int kColsumRows = 2048, kColsumChunks = 64;
// Whether the launches fit a grid (fewer than 2^32 lanes): to be asked before anything
// that they sum up is enqueued.
bool colsum_grid_ok(int n, long long cols, bool spare);
hipError_t launch_colsum(const float *part, int n, long long cols, long long first, float *out0,
                         float *out1, hipStream_t stream, float *spare = nullptr);

// ---- short causal convolution (conv.hip)
// The channel axis cut into `n` parts (1 to 3) that live in tensors of their
// own, each dense [rows][count[i]]; first[i] is the part's first channel.
struct ConvParts {
    int n, first[3], count[3];
    void *ptr[3];
};
struct ConvArgs {
    const void *x, *init;         // init [Bt][W-1][K], nullable
    size_t x_batch, x_row;        // strides in elements
    const float *weight, *bias;   // [K][W], [K] (nullable)
    const int *cu_seqlens;        // packed sequences (batch 1), or NULL
    int nseq, batch, seqlen, channels, width, silu;
    ConvParts y;
    void *final_state;            // [Bt or nseq][W-1][K], nullable
};
hipError_t launch_conv_fwd(const ConvArgs &a, bool bf16, hipStream_t stream);
struct ConvBwdArgs {
    const void *x, *init, *dfinal;
    size_t x_batch, x_row;
    const float *weight, *bias;
    int batch, seqlen, channels, width, silu;
    ConvParts dy;
    void *dx, *dinit;
    float *dweight, *dbias, *part;  // part: conv_bwd_part_bytes of scratch
};
size_t conv_bwd_part_bytes(int batch, int seqlen, int channels, int width);
// Whether every launch of launch_conv_bwd fits a grid.
bool conv_bwd_grid_ok(int batch, int seqlen, int channels, int width, const ConvParts &dy);
hipError_t launch_conv_bwd(const ConvBwdArgs &a, bool bf16, hipStream_t stream);
hipError_t launch_conv_step(void *state, const void *x, size_t x_row, const float *weight,
                            const float *bias, int batch, int channels, int width, int silu,
                            const ConvParts &y, bool bf16, hipStream_t stream);

// ---- selective scan (selective.hip, selective_bwd.hip)
// Strides in elements between sequences and tokens; channels (and a token's
// [G][N] of B and C) are dense. x, dt, z [Bt][L][E], B, C [Bt][L][G][N].
struct SelArgs {
    const void *x, *dt, *z, *B, *C;   // z nullable
    size_t x_batch, x_token, dt_batch, dt_token, z_batch, z_token, B_batch, B_token, C_batch,
        C_token;
    const float *A, *D;               // [E][N], [E] (nullable)
    const float *init;                // [Bt][E][N], nullable
    DtOpts opts;                      // bias [E]; no zero-order hold
    int batch, seqlen, channels, ngroups, dstate;
    int units, whole;                 // workgroups of all sequences; the first so many uncut
    int segs, seg_len;                // the others' segments of the token axis
    float *bc;                        // B and C as the kernels read them: scratch
    float *seg_state, *seg_sum;       // [Bt][segs - 1][E * NK], [Bt][segs - 1][E]: scratch
    void *y;                          // [Bt][L][E] dense
    float *final_state;               // [Bt][E][N], nullable
    // the backward's: states before every so many tokens (selective_keep_tokens)
    int keeps;                        // of them per sequence
    float *keep_state, *keep_sum;     // [Bt][keeps][E * NK], [Bt][keeps][E]
    const void *dy;                   // [Bt][L][E] dense
    const float *dfinal;              // [Bt][E][N], nullable
    float *seg_adj;                   // [Bt][segs - 1][E * NK]: segments 1 .. segs - 1
};
// The state size the kernels hold (4, 8, 16, 32 or 64; 0: not supported) and
// the workgroups one sequence's channels take.
int selective_kernel_dstate(int dstate);
int selective_blocks(int channels, int ngroups, int dstate);
struct SelPlan {
    int units, whole, segs, seg_len;
    size_t seg_floats;  // of seg_state
};
size_t selective_bc_floats(int batch, int seqlen, int ngroups, int dstate);
SelPlan selective_plan(int batch, int seqlen, int channels, int ngroups, int dstate);
hipError_t launch_selective_fwd(const SelArgs &a, bool bf16, hipStream_t stream);
// The backward's first pass: fills seg_state, seg_sum, seg_adj, keep_state, keep_sum.
hipError_t launch_selective_keep(const SelArgs &a, bool bf16, hipStream_t stream);
int selective_keep_tokens(int dstate);
// One token: the token strides and init are not read.
hipError_t launch_selective_step(const SelArgs &a, float *state, bool bf16, hipStream_t stream);

struct SelBwdArgs {
    SelArgs f;                  // the forward's inputs; y, final_state unused
    float *dbc_part;            // selective_dbc_floats: every workgroup's dB and dC
    float *dA_part;             // [Bt][segs][E][N]
    float *de_part;             // [Bt][segs][dD, dbias][E]
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *ddt_bias, *dinit;  // dD, ddt_bias, dinit nullable
};
SelPlan selective_bwd_plan(int batch, int seqlen, int channels, int ngroups, int dstate);
size_t selective_dbc_floats(int batch, int seqlen, int channels, int ngroups, int dstate);
// Whether every launch of launch_selective_bwd fits a grid (beside the layout of B and C).
bool selective_bwd_grid_ok(int batch, int seqlen, int channels, int ngroups, int dstate, int segs);
hipError_t launch_selective_bwd(const SelBwdArgs &a, bool bf16, hipStream_t stream);

}  // namespace ssd
