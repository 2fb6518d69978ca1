/*
 * mamba_layer.h -- C ABI of the layer operators around the scan on MI355X
 * (gfx950): the short causal convolution in front of it, the selective scan
 * whose decay differs for each channel and state, and the gated group norm
 * behind it. Each has a forward and a backward pass; the two with a state also
 * have a step of one token. They live in the library of mimo_bwd_fwd.h, with
 * its status codes, mimo_last_error() and MIMO_DTYPE_* codes.
 *
 * Sequences. n sequences are given dense, [n, S, ...], or packed along one
 * token axis, [S, ...] with S the total and cu_seqlens [n + 1] int32 on the
 * device: sequence i holds the tokens [cu_seqlens[i], cu_seqlens[i+1]), which
 * may be none; cu_seqlens[0] = 0, not decreasing, at most S. The values are not
 * read on the host. Values outside these rules give wrong results but no access
 * outside the tensors. Tokens behind the last sequence are not read; their
 * outputs are left as they were, or zero where zero_tail is set.
 *
 * Tensors. A mamba_rows is a tensor with a batch and a token axis (strides in
 * elements; the batch stride is not used when packed) whose inner axes are
 * dense. Everything else is dense, row-major. Data tensors share one dtype
 * (MIMO_DTYPE_BF16, _FP16 or _FP32); parameters, the scan's state and their
 * gradients are fp32. All arithmetic is fp32, rounded once when stored. Outputs,
 * gradients and the workspace must not overlap any input or each other.
 *
 * Limits, MIMO_ERR_UNSUPPORTED beyond them: 65535 sequences or rows of a step, S up to
 * 2^30, 2^20 channels, 1024 groups of the scan, 65535 groups and 2^31 groups of rows of
 * the norm, 2^32 threads along an axis of a kernel's grid.
 *
 * Ownership, asynchrony and errors as in mimo_bwd_fwd.h: the caller owns every
 * buffer; nothing is allocated; the call returns once its kernels are queued on
 * `stream`; on error nothing has been queued. A workspace's contents do not
 * matter on entry; calls that may overlap need workspaces of their own. Its size
 * goes by the sizes, by which optional pointers are NULL and by the alignment of
 * the tensors, so the query takes the arguments of the call (without workspace).
 * Sums run in a fixed order: equal inputs give equal bits.
 *
 * The backward scan's workspace, in bytes, with channel tiles of B = 128 channels
 * for N <= 8, 64 up to 32, 32 up to 64 and 16 up to 128, t = ceil(D / G / B) of
 * them in a group, and chunks of C = 16 to 128 tokens (fewer where there is less
 * to do; a whole sequence of up to 128 tokens where two chunks would hold it):
 *   partial sums of db and dc: 8 N G t a token;
 *   sums of a chunk: 4 D (N + 2), and where chunks follow each other in a sequence
 *     4 D (N + 1) more; n ceil(S / C) chunks, packed S / C + n + 1;
 *   states at every sixteenth token but a chunk's first: 4 D (N + 1) each;
 *     n (ceil(S / 16) - ceil(S / C)) of them, packed S (C / 16 - 1) / C + n.
 * Each packed sequence thus costs about 3 states [D, N] beside its tokens.
 */
#ifndef MAMBA_LAYER_H
#define MAMBA_LAYER_H

#include "mimo_bwd_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mamba_rows {
    const void *data;
    int64_t batch_stride, token_stride;
} mamba_rows;

#define MAMBA_CONV_MIN_TAPS 2
#define MAMBA_CONV_MAX_TAPS 8
#define MAMBA_SCAN_MAX_STATE 128
#define MAMBA_NORM_MAX_WIDTH 8192

/*
 * Short causal convolution, one filter of W taps per channel. With e the
 * sequence behind its W - 1 rows of state (zeros where initial_state is NULL):
 *   pre[t] = bias + sum_k weight[:,k] * e[t + k];  out = silu(pre) or pre.
 * state (optional) receives the last W - 1 rows of e.
 *   x, out [.., D]; weight [D, W]; bias [D] or NULL; states [n, W-1, D] (data dtype)
 */
typedef struct mamba_conv_fwd_args {
    int64_t n, S, D;
    int32_t W, dtype, silu, zero_tail;
    const int32_t *cu_seqlens;    /* NULL: dense */
    mamba_rows x;
    const float *weight, *bias;
    const void *initial_state;    /* optional */
    void *out;
    void *state;                  /* optional */
} mamba_conv_fwd_args;
mimo_status mamba_conv_fwd(const mamba_conv_fwd_args *args, void *stream);

/* Gradients of sum(out * dout) + sum(state * dstate). dx [.., D] and
 * dinitial_state in the data dtype, dweight [D, W] and dbias [D] fp32; dbias,
 * dinitial_state and dstate are optional. Tokens behind the last sequence get dx = 0. */
typedef struct mamba_conv_bwd_args {
    int64_t n, S, D;
    int32_t W, dtype, silu, reserved;
    const int32_t *cu_seqlens;
    mamba_rows dout, x;
    const float *weight, *bias;
    const void *initial_state;    /* optional */
    const void *dstate;           /* optional */
    void *dx;
    float *dweight, *dbias;
    void *dinitial_state;
    void *workspace;              /* mamba_conv_bwd_workspace_size() bytes, 256-byte aligned */
    size_t workspace_bytes;
} mamba_conv_bwd_args;
mimo_status mamba_conv_bwd_workspace_size(const mamba_conv_bwd_args *args, size_t *bytes);
mimo_status mamba_conv_bwd(const mamba_conv_bwd_args *args, void *stream);

/* One token for each of n rows: x, out [n, D]; state [slots, W-1, D] (slot_stride
 * elements from slot to slot), updated in place. Row i uses slot indices[i] (i
 * when NULL, then n <= slots). A row whose index is outside [0, slots) is
 * skipped: its output is zero. Rows with the same index are taken in row order,
 * as consecutive tokens of one sequence. */
typedef struct mamba_conv_step_args {
    int64_t n, D, slots, slot_stride, x_stride;
    int32_t W, dtype, silu, reserved;
    const void *x;
    void *state;
    const float *weight, *bias;
    const int32_t *indices;       /* optional */
    void *out;
} mamba_conv_step_args;
mimo_status mamba_conv_step(const mamba_conv_step_args *args, void *stream);

/*
 * Selective scan. For channel d of group g = d / (D / G) and state n:
 *   dt'   = dt + dt_bias, through softplus where asked
 *   h[t]  = exp(dt'[t] a[d,n]) h[t-1] + dt'[t] u[t] b[t,g,n]
 *   y[t]  = sum_n c[t,g,n] h[t] + d[d] u[t];   out = y * silu(z), or y without z
 * from h = initial_state (zeros where NULL); state (optional) receives the last h.
 * Infinities come out as the formulas give them, but da may be NaN where a state is
 * infinite. Long sequences are cut into chunks whose factors exp(dt' a) are multiplied
 * over up to 32768 tokens before they meet a state: a product below fp32's range turns
 * an infinite state into NaN, and one above it (steps that let the state grow, dt' a > 0)
 * a state or an adjoint of zero.
 *   u, dt, z, out [.., D]; a [D, N]; b, c [.., G, N]; d, dt_bias [D] or NULL;
 *   states [n, D, N] fp32. N <= MAMBA_SCAN_MAX_STATE, D a multiple of G.
 */
typedef struct mamba_scan_fwd_args {
    int64_t n, S, D, G, N;
    int32_t dtype, dt_softplus, zero_tail, reserved;
    const int32_t *cu_seqlens;
    mamba_rows u, dt, b, c;
    mamba_rows z;                 /* data NULL: no gate */
    const float *a, *d, *dt_bias;
    const float *initial_state;   /* optional */
    void *out;
    float *state;                 /* optional */
    void *workspace;              /* mamba_scan_fwd_workspace_size() bytes, 256-byte aligned */
    size_t workspace_bytes;
} mamba_scan_fwd_args;
mimo_status mamba_scan_fwd_workspace_size(const mamba_scan_fwd_args *args, size_t *bytes);
mimo_status mamba_scan_fwd(const mamba_scan_fwd_args *args, void *stream);

/* Gradients of sum(out * dout) + sum(state * dstate). du, ddt, dz [.., D] and db,
 * dc [.., G, N] in the data dtype; da [D, N], dd, ddt_bias [D] and dinitial_state
 * fp32. dz is required iff z is given; dd, ddt_bias, dinitial_state and dstate are
 * optional. Tokens behind the last sequence get zero gradients. */
typedef struct mamba_scan_bwd_args {
    int64_t n, S, D, G, N;
    int32_t dtype, dt_softplus, reserved0, reserved1;
    const int32_t *cu_seqlens;
    mamba_rows dout, u, dt, b, c;
    mamba_rows z;                 /* data NULL: no gate */
    const float *a, *d, *dt_bias;
    const float *initial_state, *dstate;
    void *du, *ddt, *db, *dc, *dz;
    float *da, *dd, *ddt_bias, *dinitial_state;
    void *workspace;              /* mamba_scan_bwd_workspace_size() bytes, 256-byte aligned */
    size_t workspace_bytes;
} mamba_scan_bwd_args;
mimo_status mamba_scan_bwd_workspace_size(const mamba_scan_bwd_args *args, size_t *bytes);
mimo_status mamba_scan_bwd(const mamba_scan_bwd_args *args, void *stream);

/* One token for each of n rows: u, dt, z, out [n, D]; b, c [n, G, N]; state [slots,
 * D, N] fp32 (slot_stride elements from slot to slot), updated in place. Slots and
 * indices as for mamba_conv_step. Here batch_stride is the row stride. */
typedef struct mamba_scan_step_args {
    int64_t n, D, G, N, slots, slot_stride;
    int32_t dtype, dt_softplus;
    mamba_rows u, dt, b, c;
    mamba_rows z;                 /* data NULL: no gate */
    const float *a, *d, *dt_bias;
    float *state;
    const int32_t *indices;       /* optional */
    void *out;
} mamba_scan_step_args;
mimo_status mamba_scan_step(const mamba_scan_step_args *args, void *stream);

/*
 * Gated group norm over the channels of each row, channels last, G groups of
 * D / G channels (at most MAMBA_NORM_MAX_WIDTH). With v = x * silu(z) (z given,
 * gate_after = 0) or x, m = mean(v) (center) or 0 over the group:
 *   p = (v - m) / sqrt(mean((v - m)^2) + eps) * weight + bias
 *   out = p * silu(z) (z given, gate_after = 1), silu(p) (silu), or p.
 * rows x, z, out [rows, D] (row strides in elements); silu excludes z.
 */
typedef struct mamba_norm_fwd_args {
    int64_t rows, D, G;
    int64_t x_stride, z_stride;
    int32_t dtype, center, gate_after, silu;
    float eps;
    int32_t reserved;
    const void *x, *z;            /* z optional */
    const float *weight, *bias;   /* bias optional */
    void *out;
} mamba_norm_fwd_args;
mimo_status mamba_norm_fwd(const mamba_norm_fwd_args *args, void *stream);

/* Gradients of sum(out * dout): dx, dz [rows, D] in the data dtype, dweight and
 * dbias [D] fp32. dz is required iff z is given, dbias iff bias is. */
typedef struct mamba_norm_bwd_args {
    int64_t rows, D, G;
    int64_t dout_stride, x_stride, z_stride;
    int32_t dtype, center, gate_after, silu;
    float eps;
    int32_t reserved;
    const void *dout, *x, *z;
    const float *weight, *bias;
    void *dx, *dz;
    float *dweight, *dbias;
    void *workspace;              /* mamba_norm_bwd_workspace_size() bytes, 256-byte aligned */
    size_t workspace_bytes;
} mamba_norm_bwd_args;
mimo_status mamba_norm_bwd_workspace_size(const mamba_norm_bwd_args *args, size_t *bytes);
mimo_status mamba_norm_bwd(const mamba_norm_bwd_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_LAYER_H */
