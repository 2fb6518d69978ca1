/*
 * mamba_layer.h -- C ABI of the layer operators around the scan on MI355X
 * (gfx950): the short causal convolution in front of it, the selective scan
 * whose decay differs for each channel and state, the gated linear recurrence, and
 * the gated group norm behind it; and what lies between blocks, the addition to
 * the residual stream with its norm. Each has a forward and a backward pass;
 * those with a state also have a step of one token. They live in the library of mimo_bwd_fwd.h, with
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
 * the norms, 2^32 threads along an axis of a kernel's grid.
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

/*
 * Gated linear recurrence, one state a channel:
 *   l[t]  = -rate * softplus(decay[d]) * sigmoid(r[t] + r_bias[d])
 *   h[t]  = exp(l[t]) h[t-1] + sqrt(1 - exp(2 l[t])) * sigmoid(i[t] + i_bias[d]) * x[t]
 *   out   = h * silu(z), or h without z
 * from h = initial_state (zeros where NULL); state (optional) receives the last h.
 * Long sequences are cut into chunks whose factors exp(l) are multiplied before they
 * meet a state: a product below fp32's range turns an infinite state into NaN. A decay
 * below -87 counts as none (its softplus is below fp32's range), and so does rate *
 * softplus(decay) below 8e-39: nothing is forgotten or enters.
 *   x, r, i, z, out [.., D]; decay, r_bias, i_bias [D] (the biases optional); states
 *   [n, D] fp32. rate is not negative; rate * softplus(decay) beyond 1e29 counts as
 *   some 1e30. Token strides: 0 to MAMBA_RECUR_MAX_STRIDE elements (forward and backward;
 *   not used where S = 1).
 * Blocks of the forward pass wait for those in front of them, with a limit: where
 * cu_seqlens decreases, a call may take some tenths of a second and leave NaN; its
 * status, given before it runs, is MIMO_OK. Nothing else reaches the limit.
 * Workspace, in bytes, with chunks of C tokens: dense 128 forward and 64 backward, packed
 * 64 and 32, or 32 and 16 where S / n < 64; n ceil(S / C) chunks, packed S / C + n + 1.
 *   forward: 8 D for each chunk and for every C / 4 of them, none where S <= C
 *   backward: 12 D for each chunk, 24 D where S > C
 */
#define MAMBA_RECUR_MAX_STRIDE (1 << 26)
typedef struct mamba_recur_fwd_args {
    int64_t n, S, D;
    int32_t dtype, zero_tail;
    float rate;
    int32_t reserved;
    const int32_t *cu_seqlens;
    mamba_rows x, r, i;
    mamba_rows z;                 /* data NULL: no gate */
    const float *decay, *r_bias, *i_bias;
    const float *initial_state;   /* optional */
    void *out;
    float *state;                 /* optional */
    void *workspace;              /* mamba_recur_fwd_workspace_size() bytes, 256-byte aligned */
    size_t workspace_bytes;
} mamba_recur_fwd_args;
mimo_status mamba_recur_fwd_workspace_size(const mamba_recur_fwd_args *args, size_t *bytes);
mimo_status mamba_recur_fwd(const mamba_recur_fwd_args *args, void *stream);

/* Gradients of sum(out * dout) + sum(state * dstate). dx, dr, di, dz [.., D] in the
 * data dtype; ddecay, dr_bias, di_bias [D] and dinitial_state fp32. dz is required iff
 * z is given, dr_bias iff r_bias is, di_bias iff i_bias is; dinitial_state and dstate
 * are optional. Where exp(l) = 1 nothing of x enters, and the gradients are those of the
 * limit (no part of r, decay or their biases). Tokens behind the last sequence get zero
 * gradients. */
typedef struct mamba_recur_bwd_args {
    int64_t n, S, D;
    int32_t dtype, reserved0;
    float rate;
    int32_t reserved1;
    const int32_t *cu_seqlens;
    mamba_rows dout, x, r, i;
    mamba_rows z;                 /* data NULL: no gate */
    const float *decay, *r_bias, *i_bias;
    const float *initial_state, *dstate;
    void *dx, *dr, *di, *dz;
    float *ddecay, *dr_bias, *di_bias, *dinitial_state;
    void *workspace;              /* mamba_recur_bwd_workspace_size() bytes, 256-byte aligned */
    size_t workspace_bytes;
} mamba_recur_bwd_args;
mimo_status mamba_recur_bwd_workspace_size(const mamba_recur_bwd_args *args, size_t *bytes);
mimo_status mamba_recur_bwd(const mamba_recur_bwd_args *args, void *stream);

/* One token for each of n rows: x, r, i, z, out [n, D]; state [slots, D] fp32
 * (slot_stride elements from slot to slot), updated in place. Slots and indices as for
 * mamba_conv_step. Here batch_stride is the row stride. */
typedef struct mamba_recur_step_args {
    int64_t n, D, slots, slot_stride;
    int32_t dtype, reserved;
    float rate;
    int32_t reserved1;
    mamba_rows x, r, i;
    mamba_rows z;                 /* data NULL: no gate */
    const float *decay, *r_bias, *i_bias;
    float *state;
    const int32_t *indices;       /* optional */
    void *out;
} mamba_recur_step_args;
mimo_status mamba_recur_step(const mamba_recur_step_args *args, void *stream);

/*
 * Addition to the residual stream and root-mean-square norm of the sum, by rows:
 *   v = dropout(x) + residual (or dropout(x));  y = v / sqrt(mean(v^2) + eps) * weight
 * The norm takes v before it is rounded to `sum`. The stream (residual, sum, and their
 * gradients) has the data dtype, or fp32 where wide is set. A square of v beyond fp32's
 * range (|v| > 1.8e19) makes the row's norm infinite; with eps = 0, a row of zeros, or of
 * squares below that range, has the norm zero and gives NaN and infinities.
 *
 * Dropout: an element is dropped, whatever its value, where its 16 bits are below
 * `drop`, and multiplied by 65536 / (65536 - drop) elsewhere. The bits of the columns
 * 8 c .. 8 c + 7 of row k are the four words of Philox4x32 with ten rounds (J. Salmon
 * et al., "Parallel random numbers: as easy as 1, 2, 3", 2011), low halves first, for
 * the counter (c, k, low word, high word of seed[1]) and the key (low word, high word
 * of seed[0]); seed lies on the device, so that a captured call takes new numbers. No
 * mask is stored: the backward pass draws the bits again.
 *
 * out: y in the data dtype (MAMBA_OUT_SAME), or in 8 bits with scales, y = q * scale:
 * q in e4m3 (no infinities, largest 448) or whole numbers from -127 to 127, rounded to
 * nearest even; a scale for every `block` columns (32, 64, 128 or 256; the last block may
 * be short), or for the row (0). scale = max(largest |y|, 2^-100) / (448 or 127); where a
 * block holds a value that is not finite its scale is NaN, and q NaN (e4m3) or 0.
 *   x [rows, D] (row stride in elements), residual likewise; sum, out [rows, D] dense;
 *   weight [D]; scale [rows, ceil(D / block)] or [rows]. D <= MAMBA_ADD_NORM_MAX_WIDTH.
 *   sum is optional where nothing is added or dropped and the stream has the data dtype.
 */
#define MAMBA_ADD_NORM_MAX_WIDTH 16384
#define MAMBA_OUT_SAME 0
#define MAMBA_OUT_E4M3 1
#define MAMBA_OUT_INT8 2
typedef struct mamba_add_norm_fwd_args {
    int64_t rows, D;
    int64_t x_stride, residual_stride;
    int32_t dtype, wide, out_kind, block;
    int32_t drop;                 /* of 65536; 0: none */
    float eps;
    const void *x, *residual;     /* residual optional */
    const int64_t *seed;          /* [2], required where drop is not 0 */
    const float *weight;
    void *sum, *out;
    float *scale;                 /* required unless MAMBA_OUT_SAME */
} mamba_add_norm_fwd_args;
mimo_status mamba_add_norm_fwd(const mamba_add_norm_fwd_args *args, void *stream);

/* Gradients of sum(y * dout) + sum(sum * dsum), from the sum: with dv the gradient of v,
 * dx = dropout's factor * dv in the data dtype (that of dout), dresidual = dv in the
 * stream's, dweight [D] fp32. dsum and dresidual are optional. */
typedef struct mamba_add_norm_bwd_args {
    int64_t rows, D;
    int64_t dout_stride, sum_stride, dsum_stride;
    int32_t dtype, wide;
    int32_t drop;
    float eps;
    const void *dout, *sum, *dsum;
    const int64_t *seed;
    const float *weight;
    void *dx, *dresidual;
    float *dweight;
    void *workspace;              /* mamba_add_norm_bwd_workspace_size() bytes, 256-byte aligned */
    size_t workspace_bytes;
} mamba_add_norm_bwd_args;
mimo_status mamba_add_norm_bwd_workspace_size(const mamba_add_norm_bwd_args *args, size_t *bytes);
mimo_status mamba_add_norm_bwd(const mamba_add_norm_bwd_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_LAYER_H */
