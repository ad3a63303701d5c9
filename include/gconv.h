/*
 * gconv.h -- C ABI of the grouped 2-D convolution library for AMD MI355X
 * (gfx950). Channels-first (NCHW) float32.
 *
 * The operation ("[Feature request] Groups support for SpatialConvolutionMM",
 * the opening definition of groups): the C input planes and the K output
 * planes are each split into `groups` contiguous blocks, and output block g
 * is computed from input block g only. With Cg = C/groups and Kg = K/groups:
 *
 *   y[n,k,ho,wo] = bias[k] + sum_{c<Cg, i<kh, j<kw}
 *                  w[k,c,i,j] * x[n, g*Cg + c, ho*stride_h - pad_h + i*dil_h,
 *                                               wo*stride_w - pad_w + j*dil_w]
 *
 * with g = k / Kg, x read as 0 outside [0,H) x [0,W) (zero padding), and no
 * kernel flip (cross-correlation: a kernel-sized input gives exactly the
 * Linear layer on the flattened input, as "SpatialConvolution running in
 * fully-connected mode is very slow, even with R4" relies on).
 *
 * Tensor layouts (all dense, row-major, float32, device memory):
 *   x, dx  [N, C, H, W]
 *   w, dw  [K, C/groups, kh, kw]    (K * C/groups filter planes)
 *   bias, db [K]
 *   y, dy  [N, K, Ho, Wo],  Ho = floor((H + pad_h + pad_h_end - dil_h*(kh-1) - 1)/stride_h) + 1
 *                           (likewise Wo), pad_h_end = pad_h + pad_h_extra
 * or, with layout = GCONV_LAYOUT_NHWC (channels last, the layout the
 * DLPrimitives Blog measures oneDNN fastest in), x, dx [N, H, W, C] and
 * y, dy [N, Ho, Wo, K]; w, dw and the bias keep their layouts.
 *
 * Ownership and execution. The caller owns every buffer; the library never
 * allocates device memory. Every op is enqueued on the caller's HIP stream
 * (`stream` is a hipStream_t; NULL means the default stream) and returns once
 * its kernels are enqueued. Inputs are read only. Outputs are overwritten in
 * full (gradWeight and gradBias are not accumulated into); outputs must not
 * overlap any input. Results are deterministic: the same inputs on the same
 * device give bit-identical outputs (no floating-point atomics).
 *
 * Empty batch. N == 0 is valid: forward and gradInput write nothing, and
 * gradWeight and gradBias are set to 0 (sums over no images). Pointers to
 * tensors with no elements may be NULL.
 *
 * Errors. Every function returns a gconv_status. Descriptor and argument
 * errors are detected on the host before anything is enqueued, and nothing
 * is written. GCONV_ERR_HIP reports a failed launch. gconv_last_error()
 * gives a readable detail of the calling thread's last failure (e.g. which
 * dimension does not divide by groups).
 */
#ifndef GCONV_H
#define GCONV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Convolution descriptor. K is the total number of output planes, not the
 * per-group count. The fields follow the constructor the clnn issue quotes
 * (nInputPlane, nOutputPlane, kW, kH, dW, dH, padW, padH, groups), plus
 * batch, input extent and dilation. Valid when N >= 0, C,H,W,K,kh,kw >= 1,
 * stride >= 1, dil >= 1, pad >= 0, pad + pad_extra >= 0, groups >= 1,
 * layout a gconv_layout,
 * C % groups == 0, K % groups == 0 and Ho, Wo >= 1 ("Support groups in
 * DenseConvDims": the channel counts must agree with the tensors and with the
 * group split).
 *
 * Asymmetric padding (DLPrimitives Blog, "TensorFlow": TensorFlow's "same"
 * padding can put one more zero row or column at the end of an axis than at
 * its start, which cuDNN cannot express). pad_h / pad_w are the zero rows at
 * the top and columns at the left; the bottom and right get pad_h +
 * pad_h_extra and pad_w + pad_w_extra. The end padding only sets Ho and Wo;
 * no padded copy of x is made. A zero-initialised pad_*_extra gives the
 * symmetric padding of the formula above.
 */
typedef struct gconv_desc {
    int64_t N, C, H, W;
    int64_t K;
    int64_t kh, kw;
    int64_t stride_h, stride_w;
    int64_t pad_h, pad_w;
    int64_t dil_h, dil_w;
    int64_t groups;
    int64_t pad_h_extra, pad_w_extra;  /* end padding minus start padding (0: symmetric) */
    int64_t layout;                    /* gconv_layout of x, dx, y, dy (0: NCHW) */
} gconv_desc;

/*
 * Activation layout. NHWC: a 1x1 stride-1 unpadded layer with one group is
 * one GEMM over the N*H*W rows (the fully-connected path, no reordering);
 * gradBias sums the [N*Ho*Wo, K] rows of dy directly; depthwise layers (one
 * channel per group, 3x3 or 5x5) run on channels-last kernels of their own
 * (gradWeight there when C % 4 == 0 and no family is forced; x and dy that
 * are not 16-byte aligned take 4-byte loads). Every other NHWC op
 * reorders its NHWC inputs to NCHW in the workspace, runs the NCHW kernels
 * there and reorders the NHWC outputs back (the MFMA implicit-GEMM forward
 * and gradInput store y and dx channels-last themselves), so
 * gconv_workspace_size() then includes those copies (x and y for the forward
 * pass, dy and dx for gradInput, x and dy for gradWeight).
 */
typedef enum gconv_layout {
    GCONV_LAYOUT_NCHW = 0,
    GCONV_LAYOUT_NHWC = 1
} gconv_layout;

typedef enum gconv_status {
    GCONV_OK = 0,
    GCONV_ERR_NULL = 1,        /* a required pointer is NULL */
    GCONV_ERR_SHAPE = 2,       /* a dimension < 1, a bad stride/pad/dilation, or Ho/Wo < 1 */
    GCONV_ERR_GROUPS = 3,      /* C or K not divisible by groups */
    GCONV_ERR_WORKSPACE = 4,   /* workspace smaller than gconv_workspace_size(), or misaligned */
    GCONV_ERR_HIP = 5,         /* a HIP runtime call or kernel launch failed */
    GCONV_ERR_UNSUPPORTED = 6, /* valid descriptor the forced path cannot run */
    GCONV_ERR_ARG = 7          /* other bad argument, e.g. an output overlapping an input */
} gconv_status;

typedef enum gconv_op {
    GCONV_OP_FWD = 0,
    GCONV_OP_BWD_DATA = 1,
    GCONV_OP_BWD_FILTER = 2,
    GCONV_OP_BWD_BIAS = 3
} gconv_op;

/* Kernel families the dispatcher routes between. */
typedef enum gconv_path {
    GCONV_PATH_AUTO = 0,       /* the dispatcher's own choice (default) */
    GCONV_PATH_DIRECT = 1,     /* general direct kernels: any valid descriptor */
    GCONV_PATH_SMALLGROUP = 2, /* few channels per group: HBM-bound 4x4x1-MFMA kernels */
    GCONV_PATH_IGEMM = 3,      /* fp32-MFMA implicit GEMM, groups in the grid */
    GCONV_PATH_FC = 4,         /* kernel == input: plain fp32-MFMA GEMM */
    GCONV_PATH_POINTWISE = 5   /* 1x1, stride 1, no padding: one fp32-MFMA GEMM per
                                  (image, group), gradWeight split over images */
} gconv_path;

/*
 * Output extent of the descriptor: the floor rule above, which fits every
 * shape the pages print ("Support groups in DenseConvDims": a 3x3 kernel
 * takes the 28x28 grouped benchmark input to 26x26; "SpatialConvolution
 * running in fully-connected mode is very slow, even with R4": a 6x6 kernel
 * on a 6x6 input gives the 1x1 output MatConvNet's gradient shape shows).
 * Writes *Ho and *Wo and returns GCONV_OK, or returns the descriptor's error
 * status (GCONV_ERR_SHAPE when the dilated kernel exceeds the padded input)
 * and writes nothing. Host only; launches nothing.
 */
int gconv_output_dims(const gconv_desc* d, int64_t* Ho, int64_t* Wo);

/*
 * Bytes of device workspace `op` (a gconv_op) needs for this descriptor (0
 * when none), written to *bytes. Pass at least this much to the op, 16-byte
 * aligned (GCONV_ERR_WORKSPACE otherwise); the workspace may be NULL when 0.
 * The contents need no initialisation and are scratch after the call. The
 * size comes back through *bytes so that an invalid descriptor or op can
 * return its status (GCONV_ERR_SHAPE, GCONV_ERR_GROUPS, GCONV_ERR_ARG) rather
 * than a size a caller might allocate. Host only.
 */
int gconv_workspace_size(const gconv_desc* d, int op, size_t* bytes);

/*
 * Forward pass (updateOutput in the clnn issue): y = conv(x, w) + bias.
 * `bias` may be NULL (no bias); otherwise bias[k] is added to every element
 * of output plane k (DLPrimitives Blog, "Pointwise Broadcast Reduce": the
 * [C] bias broadcast over [B,C,H,W]). One launch covers every group.
 */
int gconv_fwd(const gconv_desc* d, const float* x, const float* w, const float* bias, float* y,
              void* workspace, size_t workspace_bytes, void* stream);

/* Element-wise activations the forward pass can apply in its epilogue. */
typedef enum gconv_epilogue {
    GCONV_EPILOGUE_NONE = 0,   /* y = conv(x, w) + bias */
    GCONV_EPILOGUE_RELU = 1    /* y = max(conv(x, w) + bias, 0); NaN becomes 0 */
} gconv_epilogue;

/*
 * Forward pass with an element-wise activation applied to each output as it
 * is stored, after the bias (DLPrimitives Blog, "Pointwise Broadcast Reduce":
 * element-wise operations over the conv's output, broadcast over [B,C,H,W]),
 * so the activation costs no extra pass over y. Same arguments as gconv_fwd
 * plus `epilogue`, a gconv_epilogue; any other value is GCONV_ERR_ARG.
 * gconv_fwd is gconv_fwd_ex with GCONV_EPILOGUE_NONE.
 */
int gconv_fwd_ex(const gconv_desc* d, const float* x, const float* w, const float* bias, int epilogue,
                 float* y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * gradInput (updateGradInput in the clnn issue): dx = d<y,dy>/dx, the exact
 * adjoint of the forward map. dx[n, g*Cg+c, h, w] sums w[k,c,i,j] *
 * dy[n,k,ho,wo] over the k of group g and the taps (i, j) whose window
 * position (ho, wo) reads (h, w); input pixels no window reads get 0.
 */
int gconv_bwd_data(const gconv_desc* d, const float* dy, const float* w, float* dx,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * gradWeight (the weight half of accGradParameters in the clnn issue):
 * dw[k,c,i,j] = sum_{n,ho,wo} dy[n,k,ho,wo] * x[n, g*Cg+c, h(ho,i), w(wo,j)].
 * Overwrites dw. Uses the workspace for split reductions.
 */
int gconv_bwd_filter(const gconv_desc* d, const float* x, const float* dy, float* dw,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * gradWeight without a workspace argument and without allocating, for callers
 * that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc). Same arguments, results
 * and errors as gconv_bwd_filter, whose kernels it runs; what that call keeps
 * in the workspace (split partials, channels-last copies) goes to a static
 * device array of 64 MiB instead, one per device, held until the process
 * ends. A descriptor that needs more (gconv_workspace_size) returns
 * GCONV_ERR_WORKSPACE before anything is enqueued. The stream must belong to
 * the current device (GCONV_ERR_ARG otherwise); the array's device address is
 * looked up on the first call on each device. Nothing in the array needs to
 * start at zero: every call writes what it reads. All calls on one device
 * share the array, so calls that overlap on one device (concurrent streams,
 * or threads) race and give wrong results; serialise them.
 */
int gconv_bwd_filter_static(const gconv_desc* d, const float* x, const float* dy, float* dw, void* stream);

/*
 * gradBias: db[k] = sum_{n,ho,wo} dy[n,k,ho,wo] (DLPrimitives Blog,
 * "Pointwise Broadcast Reduce": the sum of dy over dims 0, 2 and 3).
 * Only N, K, Ho, Wo and the layout of the descriptor matter. Overwrites db.
 */
int gconv_bwd_bias(const gconv_desc* d, const float* dy, float* db, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * Kernel family the dispatcher would run `op` on for this descriptor
 * (gradBias is one reduction for every shape and reports GCONV_PATH_DIRECT).
 */
int gconv_select_path(const gconv_desc* d, int op, int* path);

/*
 * Force every later call in this process onto one kernel family (for
 * cross-checking each family against the others); GCONV_PATH_AUTO restores
 * the dispatcher's choice. A forced family that cannot run a descriptor
 * makes that call return GCONV_ERR_UNSUPPORTED. Not meant for concurrent use.
 */
int gconv_set_path_override(int path);

const char* gconv_status_string(int status);

/*
 * Readable detail of the calling thread's last failed call, "" after a call
 * that succeeded ("Support groups in DenseConvDims" adds a channel check so
 * that a bad group split gets a clear message: here, e.g., "input channels
 * C=10 not divisible by groups=3"). The string is owned by the library and
 * stays valid until the thread's next call into it.
 */
const char* gconv_last_error(void);

/* Library version: major*10000 + minor*100 + patch. */
int gconv_version(void);

/* ---- sequence operators ---------------------------------------------------
 *
 * Operators that stand next to 1x1 convolutions in sequence models: linear
 * attention with a decay for each head, the gated norm around a block, and
 * the orthogonalised update of a weight gradient. The conventions above hold
 * (the caller owns every buffer, the stream, determinism, errors before
 * anything is enqueued); tensors have one of two element types.
 */
typedef enum gconv_dtype {
    GCONV_F32 = 0,
    GCONV_BF16 = 1
} gconv_dtype;

/*
 * Linear attention with a decay for each head. For a sequence of L tokens and
 * a head h with lambda = exp(log_decay[h]), a state S (dk x dv, float32) that
 * starts at initial_state (0 if that is NULL) takes in every token and then
 * answers its query:
 *
 *   S_t = lambda S_{t-1} + k_t v_t^T        o_t = scale q_t S_t
 *
 * so that o_t = scale (sum_{j<=t} lambda^(t-j) (q_t . k_j) v_j
 *                      + lambda^(t+1) q_t S_init), t from 0, and the final state is S_{L-1}.
 * An infinity or a NaN in a later token does not reach an earlier one.
 *
 * Heads: q, o have `heads`; k, v have `kv_heads`, each shared by
 * heads / kv_heads consecutive heads. States are per q head.
 * Sequences: with packed == 0, `sequences` of `tokens` each. With packed != 0
 * the tokens of all sequences follow one another, `tokens` in all, and
 * cu_seqlens (int32, device memory, sequences + 1 values from 0 to `tokens`,
 * not decreasing) says where each begins; a sequence may be empty. Tokens
 * before the first and after the last sequence (padding) are not read; their
 * outputs and gradients are 0.
 * Strides are in elements: [0] between sequences (not read when packed), [1]
 * between tokens, [2] between heads; the last axis is contiguous. Outputs
 * are dense, [sequences, tokens, heads, d] or [tokens, heads, d].
 * dk, dv from 1 to 128. log_decay [heads] float32; -infinity (no memory) and
 * values above 0 (growth) are valid. States [sequences, heads, dk, dv]
 * float32, dense. Up to 65536 heads, 2^30 tokens and as many sequences x heads
 * as launches take (2^20 - 1 with dk and dv above 64, 2^22 - 1 with both up to
 * 64, 2^24 - 1 one token at a time); GCONV_ERR_UNSUPPORTED beyond.
 */
typedef struct gconv_linattn_desc {
    int64_t dtype;              /* gconv_dtype of q, k, v, o and their gradients */
    int64_t packed;
    int64_t sequences, tokens;
    int64_t heads, kv_heads;
    int64_t dk, dv;
    int64_t q_stride[3], k_stride[3], v_stride[3];
    int64_t do_stride[3];       /* of the gradient of o; read by gconv_linattn_bwd only */
    double scale;
} gconv_linattn_desc;

typedef enum gconv_linattn_op {
    GCONV_LINATTN_FWD = 0,
    GCONV_LINATTN_BWD = 1
} gconv_linattn_op;

/* Bytes of workspace `op` (a gconv_linattn_op) needs, 16-byte aligned. */
int gconv_linattn_workspace_size(const gconv_linattn_desc* d, int op, size_t* bytes);

/* o and the final states of whole sequences. initial_state and final_state may be NULL. */
int gconv_linattn_fwd(const gconv_linattn_desc* d, const void* q, const void* k, const void* v, const float* log_decay,
                      const int32_t* cu_seqlens, const float* initial_state, void* o, float* final_state,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients for the gradient dout of o and d_final_state of the final state
 * (NULL: 0): dq, dk, dv (dense, of the inputs' type; those of a shared head
 * are summed over the heads that share it) and d_initial_state (may be NULL).
 * initial_state as in the forward pass.
 */
int gconv_linattn_bwd(const gconv_linattn_desc* d, const void* dout, const void* q, const void* k, const void* v,
                      const float* log_decay, const int32_t* cu_seqlens, const float* initial_state,
                      const float* d_final_state, void* dq, void* dk, void* dv, float* d_initial_state,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token of each of `sequences` sequences (packed and tokens are 0): takes
 * the token into the state, in place, and answers its query. state is a pool
 * of num_slots states [num_slots, heads, dk, dv]; sequence i uses number
 * slots[i] (int32, device memory), or i where slots is NULL. Slots of one call
 * must differ. A slot outside 0..num_slots-1 (say, -1 for an idle row) gives
 * o = 0 and touches no state. Strides [1] are not read.
 */
int gconv_linattn_step(const gconv_linattn_desc* d, const void* q, const void* k, const void* v, const float* log_decay,
                       float* state, const int32_t* slots, int64_t num_slots, void* o, void* stream);

/*
 * The norms before and after a block, with its gate and its residual scale:
 *
 *   y = x + scale * act(gate) * rmsnorm(b) * w_post      h = rmsnorm(y) * w_pre
 *   rmsnorm(v) = v / sqrt(mean(v^2) + eps) over the last axis (`dim`)
 *
 * b is what the block gave, x the residual stream, h the next block's input.
 * x, gate, scale, w_pre (and with it h) may be absent. h is taken from y
 * before y is rounded to its type. Tensors [sequences, tokens, dim], strides
 * in elements ([0] between sequences, [1] between tokens, the last axis
 * contiguous); a gate of GCONV_GATE_SEQUENCE is one row for each sequence.
 * Weights [dim] of the same type; outputs dense. dim up to 8192.
 */
typedef enum gconv_gate {
    GCONV_GATE_NONE = 0,
    GCONV_GATE_FULL = 1,      /* a gate for every element of b */
    GCONV_GATE_SEQUENCE = 2   /* a row of gates for each sequence */
} gconv_gate;

typedef enum gconv_act {
    GCONV_ACT_NONE = 0,       /* act(z) = z */
    GCONV_ACT_SIGMOID = 1,    /* 1 / (1 + exp(-z)) */
    GCONV_ACT_SILU = 2        /* z / (1 + exp(-z)) */
} gconv_act;

typedef struct gconv_normgate_desc {
    int64_t dtype;            /* gconv_dtype of every tensor and weight */
    int64_t sequences, tokens, dim;
    int64_t gate, act;        /* gconv_gate, gconv_act */
    int64_t x_stride[2], b_stride[2], gate_stride[2];
    int64_t dy_stride[2], dh_stride[2];  /* read by gconv_normgate_bwd only */
    double eps;
} gconv_normgate_desc;

/* Bytes of workspace gconv_normgate_bwd needs, 16-byte aligned (the forward pass needs none). */
int gconv_normgate_workspace_size(const gconv_normgate_desc* d, size_t* bytes);

int gconv_normgate_fwd(const gconv_normgate_desc* d, const void* x, const void* b, const void* gate, const void* w_post,
                       const void* scale, const void* w_pre, void* y, void* h, void* stream);

/*
 * Gradients for dy of y and dh of h (given exactly when w_pre is). dx, db and
 * a full gate's dgate are dense; dgate of a gate for each sequence is
 * [sequences, dim], summed over its tokens (0 without tokens, so it is given
 * then too). The weights' gradients are summed over all rows in float32 and
 * rounded once. dx may be NULL; the others are given exactly when their inputs
 * are.
 */
int gconv_normgate_bwd(const gconv_normgate_desc* d, const void* dy, const void* dh, const void* x, const void* b, const void* gate,
                       const void* w_post, const void* scale, const void* w_pre, void* dx, void* db, void* dgate, void* dw_post,
                       void* dscale, void* dw_pre, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The orthogonalised update of a weight gradient. Each group's gradient, the
 * filters / groups x inner matrix U (inner: C/groups * kh * kw), is scaled to
 * X = U / (norm(U) + eps) in the Frobenius norm and sent through `steps`
 * rounds of the Newton-Schulz iteration
 *
 *   X <- a X + (b A + c A^2) X,  A = X X^T,  (a, b, c) = (3.4445, -4.7750, 2.0315)
 *
 * (of the transposed matrix where U has more rows than columns), after which
 * its singular values lie around 1. u [filters][inner] dense, of either type;
 * out [filters][inner] in bfloat16, 8-byte aligned. The iterates are rounded
 * to fp16 between products, whose sums are float32. Relative in the norm, and
 * besides the output's own rounding, the result is within 5e-3 of the exact one
 * up to seven rounds and 7e-3 at eight, for gradients of any rank with sides of
 * 64 or more whose roundings are independent (some 1.5e-3 for a random one of
 * full rank, 3e-3 for one of low rank). At worst, for a constant gradient, all
 * of whose entries are rounded the same way, or for a side of 2 or 3, it is
 * 1.5e-2 after five rounds and 6e-2 after eight. Each further round enlarges the
 * noise in the directions that a gradient of low rank does not have up to 3.4445
 * times: rank one is 5e-2 off at ten rounds and by half at twelve, as it is when
 * all is kept in float32. Full rank is within 3e-2 at twenty. A group that
 * holds an infinity or a NaN gives NaN, and the other groups their own
 * results. A group's matrix, its longer side padded to 64, holds up to 2^29
 * elements, and neither side is above 2^24.
 */
typedef struct gconv_ortho_desc {
    int64_t dtype;            /* gconv_dtype of u */
    int64_t filters, inner;
    int64_t groups;
    int64_t steps;            /* 1 to 1000 */
    double eps;
} gconv_ortho_desc;

/* Bytes of workspace gconv_orthogonalize needs, 16-byte aligned. */
int gconv_orthogonalize_workspace_size(const gconv_ortho_desc* d, size_t* bytes);

int gconv_orthogonalize(const gconv_ortho_desc* d, const void* u, void* out, void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * The short causal convolution of each channel over its last `taps` tokens:
 *
 *   y_t = act(bias + sum_j w[.][j] x_{t-taps+1+j})
 *
 * x, y [sequences, tokens, dim] (x with strides in elements, [0] between
 * sequences, [1] between tokens, the last axis contiguous; y dense), w
 * [dim, taps], bias [dim] or NULL, all of one type. The taps - 1 inputs before
 * a sequence's first are initial_state [sequences, taps - 1, dim] (NULL: 0),
 * the oldest first; final_state (may be NULL) is the last taps - 1 inputs of
 * initial_state and sequence together. Packed sequences as in linear
 * attention. taps 1 to 8, dim up to 2^24.
 */
typedef struct gconv_shortconv_desc {
    int64_t dtype;              /* gconv_dtype of every tensor, weight and state */
    int64_t packed;
    int64_t sequences, tokens;
    int64_t dim, taps;
    int64_t act;                /* gconv_act */
    int64_t x_stride[2];
    int64_t dy_stride[2];       /* read by gconv_shortconv_bwd only */
} gconv_shortconv_desc;

/* Bytes of workspace gconv_shortconv_bwd needs, 16-byte aligned (the forward pass needs none). */
int gconv_shortconv_workspace_size(const gconv_shortconv_desc* d, size_t* bytes);

int gconv_shortconv_fwd(const gconv_shortconv_desc* d, const void* x, const void* w, const void* bias, const int32_t* cu_seqlens,
                        const void* initial_state, void* y, void* final_state, void* stream);

/*
 * Gradients for dy of y and d_final_state of the final state (NULL: 0): dx
 * (dense), dw, dbias (given exactly when bias is) and d_initial_state (may be
 * NULL). The weights' are summed over all tokens in float32 and rounded once.
 */
int gconv_shortconv_bwd(const gconv_shortconv_desc* d, const void* dy, const void* x, const void* w, const void* bias,
                        const int32_t* cu_seqlens, const void* initial_state, const void* d_final_state, void* dx, void* dw, void* dbias,
                        void* d_initial_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token x [sequences, dim] of each sequence (packed and tokens are 0), in
 * place on a pool of states [num_slots, taps - 1, dim]; slots as in
 * gconv_linattn_step. Strides [1] are not read.
 */
int gconv_shortconv_step(const gconv_shortconv_desc* d, const void* x, const void* w, const void* bias, void* state, const int32_t* slots,
                         int64_t num_slots, void* y, void* stream);

/*
 * The selective state space scan: a recurrence of `states` numbers for each
 * channel, whose decay and inputs depend on the token.
 *
 *   s_t = softplus(dt_t + dt_bias)      (s_t = dt_t + dt_bias without softplus)
 *   h_t = exp(s_t a) h_{t-1} + s_t u_t b_t
 *   y_t = (c_t . h_t + skip u_t) silu(gate_t)
 *
 * u, dt, gate, y [sequences, tokens, dim]; b, c [sequences, tokens, groups,
 * states], shared by the dim / groups channels of a group; strides in elements
 * ([0] between sequences, [1] between tokens, [2] between groups, the last
 * axis contiguous), outputs dense. a [dim, states], skip, dt_bias [dim]
 * float32; a of -infinity is valid and any below -2e38 counts as it: no memory
 * after a step above 1e-36, all of it after one of 0, and no gradient of the
 * decay. gate, skip and dt_bias may be NULL (1, 0 and 0 in their place).
 * States [sequences, dim, states] float32, dense; initial_state (NULL: 0) and
 * final_state may be NULL. Packed sequences as in linear attention. states up
 * to 64, dim up to 2^20, 2^31 tokens of all sequences together (2^30 of one).
 */
typedef struct gconv_scan_desc {
    int64_t dtype;              /* gconv_dtype of u, dt, b, c, gate, y and their gradients */
    int64_t packed;
    int64_t sequences, tokens;
    int64_t dim, states, groups;
    int64_t softplus;
    int64_t u_stride[2], dt_stride[2], gate_stride[2];
    int64_t b_stride[3], c_stride[3];
    int64_t dy_stride[2];       /* read by gconv_scan_bwd only */
} gconv_scan_desc;

typedef enum gconv_scan_op {
    GCONV_SCAN_FWD = 0,
    GCONV_SCAN_BWD = 1
} gconv_scan_op;

/* Bytes of workspace `op` (a gconv_scan_op) needs, 16-byte aligned. */
int gconv_scan_workspace_size(const gconv_scan_desc* d, int op, size_t* bytes);

int gconv_scan_fwd(const gconv_scan_desc* d, const void* u, const void* dt, const float* a, const void* b, const void* c, const float* skip,
                   const void* gate, const float* dt_bias, const int32_t* cu_seqlens, const float* initial_state, void* y,
                   float* final_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients for dy of y and d_final_state of the final state (NULL: 0): du,
 * ddt, db, dc, dgate of the inputs' type, dense; da, dskip, ddt_bias summed
 * over all tokens in float32; d_initial_state may be NULL. dskip, dgate and
 * ddt_bias are given exactly when their inputs are.
 *
 * The workspace holds the states before every eighth token and sums over 64
 * channels each of db and dc: about 0.76 bytes for each token, channel and state
 * (up to three times as many where sequences or groups are short), 0.41 GB for
 * 4 x 2048 tokens of 4096 x 16, 25 GB for 65536 of 8192 x 64.
 */
int gconv_scan_bwd(const gconv_scan_desc* d, const void* dy, const void* u, const void* dt, const float* a, const void* b, const void* c,
                   const float* skip, const void* gate, const float* dt_bias, const int32_t* cu_seqlens, const float* initial_state,
                   const float* d_final_state, void* du, void* ddt, float* da, void* db, void* dc, float* dskip, void* dgate,
                   float* ddt_bias, float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token of each sequence (packed and tokens are 0), in place on a pool of
 * states [num_slots, dim, states]; slots as in gconv_linattn_step. Strides [1]
 * are not read.
 */
int gconv_scan_step(const gconv_scan_desc* d, const void* u, const void* dt, const float* a, const void* b, const void* c,
                    const float* skip, const void* gate, const float* dt_bias, float* state, const int32_t* slots, int64_t num_slots,
                    void* y, void* stream);

/* Whole numbers that name tokens. */
typedef enum gconv_index {
    GCONV_I32 = 0,
    GCONV_I64 = 1
} gconv_index;

/*
 * The embedding of tokens: y[n][t] = scale table[ids[n][t]]. ids [sequences,
 * tokens] dense, of type `index`; table [rows, dim], y [sequences, tokens,
 * dim] dense. An id outside 0..rows-1 (say, -1 for padding) gives 0 and has no
 * gradient. rows up to 2^31 - 1, dim up to 2^24, 2^30 ids.
 */
typedef struct gconv_embed_desc {
    int64_t dtype;              /* gconv_dtype of table, y and their gradients */
    int64_t index;              /* gconv_index of ids */
    int64_t sequences, tokens;
    int64_t rows, dim;
    int64_t dy_stride[2];       /* in elements, between sequences and tokens; read by gconv_embed_bwd only */
    double scale;
} gconv_embed_desc;

/* Bytes of workspace gconv_embed_bwd needs, 16-byte aligned (the forward pass needs none). */
int gconv_embed_workspace_size(const gconv_embed_desc* d, size_t* bytes);

int gconv_embed_fwd(const gconv_embed_desc* d, const void* table, const void* ids, void* y, void* stream);

/*
 * dtable [rows, dim], dense, for dy of y: each row the sum over its tokens in
 * float32, rounded once; rows without tokens are 0. The order of the sums is
 * fixed by the ids: that of the tokens, for rows with many of them by slices
 * whose sums are then added up, so equal calls give equal results.
 */
int gconv_embed_bwd(const gconv_embed_desc* d, const void* dy, const void* ids, void* dtable, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * Softmax cross entropy of tokens against a vocabulary, without keeping the
 * logits: z = scale h w^T, and for each token
 *
 *   lse = log sum_v exp(z_v)        loss = lse - z_target
 *
 * h [sequences, tokens, dim] (strides in elements, [0] between sequences, [1]
 * between tokens, the last axis contiguous), w [vocab, dim] dense (16-byte
 * aligned where it is bfloat16 and dim a multiple of 64), targets, loss and
 * lse [sequences, tokens] dense; targets of type `index`, loss and lse
 * float32. A token whose target is outside 0..vocab-1 does not count: its loss
 * is 0 (its lse is given) and it has no gradient. bfloat16 products are summed
 * in float32; float32 ones are made of bfloat16 parts, to float32's accuracy,
 * and an infinity in float32 h or w gives NaN. dim up to 2^20, vocab up to
 * 2^30, 2^30 tokens.
 */
typedef struct gconv_xent_desc {
    int64_t dtype;              /* gconv_dtype of h, w and their gradients */
    int64_t index;              /* gconv_index of targets */
    int64_t sequences, tokens;
    int64_t vocab, dim;
    int64_t h_stride[2];
    double scale;
} gconv_xent_desc;

typedef enum gconv_xent_op {
    GCONV_XENT_FWD = 0,
    GCONV_XENT_BWD = 1
} gconv_xent_op;

/* Bytes of workspace `op` (a gconv_xent_op) needs, 16-byte aligned. */
int gconv_xent_workspace_size(const gconv_xent_desc* d, int op, size_t* bytes);

int gconv_xent_fwd(const gconv_xent_desc* d, const void* h, const void* w, const void* targets, float* loss, float* lse, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * Gradients for dloss of loss and dlse of lse (NULL: 0), [sequences, tokens]
 * float32 dense, given the forward pass's lse: dh [sequences, tokens, dim] and
 * dw, dense, of the inputs' type. The logits' gradient is rounded to bfloat16
 * for the products that follow where h and w are bfloat16, but for the target's
 * entry, whose rounding is made up for: by what it left in float32 for dh, and
 * for dw by the sums of that times h over a target's tokens, taken in float32
 * and rounded to bfloat16 (2^-9 of a rest that is 2^-9 of the entry at most).
 */
int gconv_xent_bwd(const gconv_xent_desc* d, const float* dloss, const float* dlse, const void* h, const void* w, const void* targets,
                   const float* lse, void* dh, void* dw, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GCONV_H */
