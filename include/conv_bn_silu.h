/*
 * conv_bn_silu.h -- C ABI of the fused conv2d -> BatchNorm -> SiLU layer for
 * NVIDIA GB300 (sm_103a).
 *
 * The layer computes, per output pixel and output channel k,
 *
 *     y = SiLU(conv2d(x, W) * scale[k] + bias[k]),   SiLU(z) = z * sigmoid(z),
 *
 * as one kernel that reads x once and writes y once: the BatchNorm multiply/add
 * and the SiLU are applied to the convolution's output tile while it is still
 * on chip ("Fusing an Epilogue", kernels book, sections "The problem",
 * "What an epilogue is" and "The shape of it").
 *
 * Conventions shared by every entry point:
 *   - Layouts: x is NHWC [n][h][w][c] bf16; W is KRSC [c_out][r][s][c] bf16
 *     (for each output channel, the filter taps row by row, channels
 *     innermost); y is NHWC [n][ho][wo][c_out] bf16; every tensor dense.
 *   - The convolution is a cross-correlation with zero padding, dilation 1 and
 *     groups 1; ho = (h + 2*pad_h - r)/stride_h + 1 (floor), likewise wo.
 *   - Pointers named device are CUDA device (or managed) memory owned by the
 *     caller.  The library keeps no reference to them after a call returns and
 *     never frees or reallocates them.  Inputs are never written.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     are asynchronous: they validate, enqueue and return.
 *   - Every function returns a cbs_status.  Invalid arguments return an error
 *     without launching anything.  A fault inside a kernel surfaces at the
 *     caller's next synchronisation, like any CUDA launch; a pipeline wait
 *     that exceeded its time bound inside a kernel is reported by
 *     conv_bn_silu_check().
 *   - Thread safety: all entry points may be called from several host threads.
 */
#ifndef CONV_BN_SILU_H
#define CONV_BN_SILU_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum cbs_status {
    CBS_OK = 0,
    CBS_ERR_INVALID_ARG = 1, /* null pointer, dim <= 0, stride < 1, pad < 0, ho/wo < 1, eps < 0 */
    CBS_ERR_MISALIGNED = 2,  /* a device pointer is not 16-byte aligned */
    CBS_ERR_UNSUPPORTED = 3, /* the requested algorithm cannot run this shape */
    CBS_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed; see conv_bn_silu_last_cuda_error() */
    CBS_ERR_TIMEOUT = 5      /* a kernel's pipeline wait ran past its bound and the kernel gave up */
} cbs_status;

/* Kernel choice for conv_bn_silu_forward_algo(). */
typedef enum cbs_algo {
    CBS_ALGO_AUTO = 0,    /* pick by shape (what conv_bn_silu_forward does) */
    CBS_ALGO_TCGEN05 = 1, /* implicit GEMM on the tcgen05 tensor cores, TMA-fed, TMEM accumulator */
    CBS_ALGO_DIRECT = 2   /* CUDA-core direct convolution, one output pixel per thread; any shape */
} cbs_algo;

/*
 * BatchNorm fold, run once per layer at load time.
 *   scale[k] = gamma[k] / sqrt(var[k] + eps),  bias[k] = beta[k] - mean[k] * scale[k]
 * The fusion page treats BN as one multiply and one add per element, with a
 * scale and a bias per output channel ("Fusing an Epilogue", sections "The
 * problem" and "The shape of it"); this is the inference-mode fold with running
 * statistics.  Computed in double precision, rounded once to float.
 *   gamma, beta, mean, var : device, float32 [c_out]
 *   eps                    : >= 0 and finite
 *   scale, bias            : device, float32 [c_out], written; must not overlap the inputs
 * c_out == 0 is a no-op.  var + eps <= 0 yields NaN/Inf in scale (not checked).
 */
int conv_bn_silu_fold(const float *gamma, const float *beta, const float *mean, const float *var,
                      float eps, int c_out, float *scale, float *bias, void *stream);

/*
 * The same fold for several layers in one launch (a network's layers at load
 * time, or every layer of a step): layer i's arguments and results are those
 * of conv_bn_silu_fold with layers[i]'s fields; the results are bit-identical.
 *   layers   : host array of n_layers descriptors, read during the call only
 *   n_layers : >= 0; 0 is a no-op.  Layers with c_out == 0 are skipped.
 * Every layer is validated before anything is launched (the first invalid
 * one decides the status).  Output arrays of different layers must not
 * overlap each other or any input.
 */
typedef struct cbs_fold_layer {
    const float *gamma, *beta, *mean, *var; /* device, float32 [c_out] */
    float eps;                              /* >= 0 and finite */
    int c_out;
    float *scale, *bias;                    /* device, float32 [c_out], written */
} cbs_fold_layer;

int conv_bn_silu_fold_batch(const cbs_fold_layer *layers, int n_layers, void *stream);

/*
 * Fused forward pass: y = SiLU(conv2d(x, W) * scale + bias).
 * ("Fusing an Epilogue", section "The shape of it": the K loop accumulates
 * the output tile; while it is still on chip, a per-channel multiply-add
 * and then SiLU are applied, and the tile is stored once; section "Three
 * kernels for one operation": convolution as a GEMM on the tensor cores.)
 *   x     : device, bf16 NHWC [n][h][w_in][c]
 *   w     : device, bf16 KRSC [c_out][r][s][c]
 *   scale : device, float32 [c_out]  (from conv_bn_silu_fold, or any per-channel multiplier)
 *   bias  : device, float32 [c_out]
 *   y     : device, bf16 NHWC [n][ho][wo][c_out], written; must not overlap x, w, scale or bias
 * All device pointers must be 16-byte aligned.  n == 0 or c_out == 0 is a
 * no-op.  The result is bf16 rounded to nearest even from an fp32
 * accumulator; it is deterministic (no atomics, fixed reduction order).
 * Kernels: the tcgen05 implicit GEMM when c % 16 == 0 and c_out % 8 == 0,
 * the thin-input tcgen05 kernel for 3x3 filters over 1, 3 or 4 channels,
 * otherwise the CUDA-core direct kernel.
 * Host work and memory held by the library, which this and every other
 * forward entry point (except conv_bn_silu_forward_noalloc) may do:
 *   - The first call of a shape on a set of buffers encodes TMA descriptors
 *     (host driver calls; cached for later calls), and the first launch of a
 *     kernel on a device sets its shared-memory limit.
 *   - Plans that split K loops between CTAs (cbs_plan_info.stream_k == 1,
 *     e.g. the 32x20x20x512 -> 512 3x3 layer) keep fp32 partial tiles in a
 *     scratch buffer the library holds, one per (device, stream).  The first
 *     such call on a stream allocates it with cudaMalloc (an implicit device
 *     synchronisation) and zeroes its flags with cudaMemsetAsync on `stream`;
 *     a later call that needs a larger buffer first synchronises `stream`,
 *     frees the old buffer and allocates a new one.  The buffers are kept
 *     until the process exits.  Make each such shape's first call on a stream
 *     before capturing that stream into a CUDA graph.
 *   - At most 64 (device, stream) pairs can hold such a buffer: a stream-K
 *     call on a 65th returns CBS_ERR_UNSUPPORTED (nothing is launched).
 *     conv_bn_silu_forward_noalloc needs none of this.
 */
int conv_bn_silu_forward(const void *x, const void *w, const float *scale, const float *bias,
                         void *y, int n, int h, int w_in, int c, int c_out, int r, int s,
                         int stride_h, int stride_w, int pad_h, int pad_w, void *stream);

/* As conv_bn_silu_forward, with the kernel chosen by `algo` (a cbs_algo).
 * Returns CBS_ERR_UNSUPPORTED when that kernel cannot run this shape. */
int conv_bn_silu_forward_algo(const void *x, const void *w, const float *scale, const float *bias,
                              void *y, int n, int h, int w_in, int c, int c_out, int r, int s,
                              int stride_h, int stride_w, int pad_h, int pad_w, int algo,
                              void *stream);

/*
 * Allocation-free variant of conv_bn_silu_forward (CBS_ALGO_AUTO), for callers
 * that may not allocate device memory: code running under a framework's own
 * caching allocator or a fixed memory budget, real-time loops where
 * cudaMalloc's implicit synchronisation is not acceptable, or hosts that hand
 * out only pre-sized buffers.  The fusion page has no counterpart to this; it
 * is a deployment convenience of this library.
 * Same arguments, layouts, results and errors as conv_bn_silu_forward, and
 * the same plan: where the plan splits K loops between CTAs (stream-K), the
 * partial tiles go to a fixed 20 MiB device array inside the library instead
 * of a library-allocated buffer, so the result is bit-identical to
 * conv_bn_silu_forward's.  A split that would need more than 20 MiB (see
 * cbs_plan_info.workspace_bytes; on a 152-SM GB300 every split fits) runs
 * whole tiles per CTA instead, which need no scratch: same values within the
 * layer's tolerance, not necessarily bit-identical.  Nothing is allocated by
 * any call, and no memory is held per stream.
 *   - The first call on a device looks up that array's device address (once
 *     per device, with that device current); make that first call before any
 *     stream capture.
 *   - Every call shares the one array per device and clears its ready flags
 *     first (an asynchronous memset on `stream`): calls whose kernels overlap
 *     on the GPU, e.g. on two streams, race and may produce wrong results.
 *     Serialise them on one stream.
 */
int conv_bn_silu_forward_noalloc(const void *x, const void *w, const float *scale, const float *bias,
                                 void *y, int n, int h, int w_in, int c, int c_out, int r, int s,
                                 int stride_h, int stride_w, int pad_h, int pad_w, void *stream);

/* Activation applied by conv_bn_act_forward after the BN multiply/add. */
typedef enum cbs_activation {
    CBS_ACT_SILU = 0,     /* z * sigmoid(z): the layer of conv_bn_silu_forward */
    CBS_ACT_IDENTITY = 1, /* z: BN (or a plain per-channel bias add) without activation */
    CBS_ACT_RELU = 2      /* max(z, 0) */
} cbs_activation;

/*
 * The fused layer with another epilogue.  "Fusing an Epilogue", section "What
 * an epilogue is": work that touches each output element once and needs no
 * neighbours (an activation, a bias add, a scaling) belongs in the epilogue of
 * the kernel that produced the element; a residual add of a tensor shaped like
 * y meets the same rule.
 *   y = act(conv2d(x, W) * scale + bias) [+ residual]
 * Arguments as conv_bn_silu_forward (the same kernels, chosen the same way), plus
 *   residual   : device, bf16 NHWC [n][ho][wo][c_out], or NULL for none; added
 *                after the activation, in fp32, before the one bf16 rounding.
 *                It may be y itself (an in-place add) but must not otherwise
 *                overlap y.  16-byte aligned.
 *   activation : a cbs_activation; anything else returns CBS_ERR_INVALID_ARG.
 * A plain per-channel bias (no BN) is scale = 1, bias = b with CBS_ACT_IDENTITY.
 * CBS_ACT_SILU with residual NULL computes exactly what conv_bn_silu_forward does.
 */
int conv_bn_act_forward(const void *x, const void *w, const float *scale, const float *bias,
                        const void *residual, void *y, int n, int h, int w_in, int c, int c_out, int r,
                        int s, int stride_h, int stride_w, int pad_h, int pad_w, int activation,
                        void *stream);

/*
 * conv_bn_act_forward with a narrower output: y is fp8 e4m3 (1 sign, 4 exponent
 * bits with bias 7, 3 mantissa bits; largest finite value 448, no infinities),
 * one byte per element, NHWC [n][ho][wo][c_out].  Each value is rounded once,
 * from the fp32 epilogue result to the nearest e4m3 (ties to even), saturating
 * to +-448 ("Fusing an Epilogue", section "What an epilogue is": casts to a
 * narrower dtype are epilogue work).  No residual.  The tensor-core path needs
 * c_out % 16 == 0 (16-byte rows) and takes the same tiles as the bf16 layer;
 * other shapes run on the direct kernel.
 */
int conv_bn_act_forward_fp8(const void *x, const void *w, const float *scale, const float *bias, void *y,
                            int n, int h, int w_in, int c, int c_out, int r, int s, int stride_h, int stride_w,
                            int pad_h, int pad_w, int activation, void *stream);

/*
 * Unfused comparator: the same layer as the three-kernel sequence that the
 * fusion replaces -- the convolution writes t1 to memory, a BatchNorm kernel
 * reads t1 and writes t2, a SiLU kernel reads t2 and writes y ("Fusing an
 * Epilogue", kernels book, section "The problem": each step a round trip
 * through memory; section "When not to fuse": measure the fused kernel
 * against the sequence it replaces).  It exists to be measured against
 * conv_bn_silu_forward, not to be used in its place.
 *   t1 = bf16(conv2d(x, W))            (the forward kernel with the epilogue reduced to the cast)
 *   t2 = bf16(t1 * scale[k] + bias[k])
 *   y  = bf16(SiLU(t2))
 * Arguments as conv_bn_silu_forward, plus
 *   t1, t2 : device, bf16 NHWC [n][ho][wo][c_out] each, written (caller-owned
 *            scratch; must not overlap each other or any other argument)
 * y differs from conv_bn_silu_forward's by the two extra bf16 roundings of
 * t1 and t2.  Three kernels are enqueued on `stream`.
 */
int conv_bn_silu_forward_unfused(const void *x, const void *w, const float *scale, const float *bias,
                                 void *t1, void *t2, void *y, int n, int h, int w_in, int c, int c_out,
                                 int r, int s, int stride_h, int stride_w, int pad_h, int pad_w,
                                 void *stream);

/* The comparator's BatchNorm step on its own, over `count` bf16 elements of
 * an NHWC tensor with c_out channels (count % c_out == 0, count <= 2^40):
 *   t2[i] = bf16(t1[i] * scale[i mod c_out] + bias[i mod c_out]), fp32 arithmetic.
 * t1, t2: device bf16 [count]; scale, bias: device float32 [c_out]; all
 * 16-byte aligned; t2 must not overlap the inputs.  count == 0 is a no-op. */
int conv_bn_silu_bn_apply(const void *t1, const float *scale, const float *bias, void *t2,
                          long long count, int c_out, void *stream);

/* The comparator's SiLU step on its own: y[i] = bf16(SiLU(t2[i])) over `count`
 * bf16 elements (count <= 2^40), SiLU(z) = z * sigmoid(z) in fp32 ("Fusing
 * an Epilogue", section "The problem": SiLU is x times sigmoid of x).
 * t2, y: device bf16 [count], 16-byte aligned, not overlapping. */
int conv_bn_silu_silu_apply(const void *t2, void *y, long long count, void *stream);

/* Output spatial size of the convolution; host only, touches no GPU.
 * ho = (h + 2*pad_h - r)/stride_h + 1, wo likewise; CBS_ERR_INVALID_ARG when
 * either would be < 1 or an argument is out of range. */
int conv_bn_silu_output_dims(int h, int w_in, int r, int s, int stride_h, int stride_w,
                             int pad_h, int pad_w, int *ho, int *wo);

/* What conv_bn_silu_forward_algo would launch for this shape; host only. */
typedef struct cbs_plan_info {
    int algo;         /* cbs_algo actually selected (never CBS_ALGO_AUTO) */
    int block_m;      /* output pixels per tile */
    int block_n;      /* output channels per tile */
    int block_k;      /* reduction depth (channels) per pipeline stage */
    int stages;       /* shared-memory pipeline depth (0 for the direct kernel) */
    int tiles;        /* output tiles */
    int grid;         /* CTAs launched */
    int threads;      /* threads per CTA */
    int smem_bytes;   /* dynamic shared memory per CTA */
    int k_iters;      /* pipeline steps per tile */
    int stream_k;     /* 1 when the K steps of all tiles are split evenly over the grid */
    int swap_ab;      /* 1 when the GEMM runs transposed: channels on the MMA's M side, pixels on N */
    int cluster;      /* CTAs per cluster: 2 when CTA pairs run the 2-CTA MMA, each holding half of every weight tile */
    long long workspace_bytes; /* library-held scratch for stream-K partial tiles (0 if none) */
    int balanced;     /* swap_ab only: 1 when each CTA takes an equal run of 32-pixel chunks (units of at
                         most 256 pixels) instead of whole 256-pixel tiles */
    int weights_resident; /* swap_ab only: 1 when each CTA keeps its 128-channel weight tile in tensor
                             memory for the whole kernel and streams only x (units of block_m pixels) */
    int row_boxes;    /* swap_ab only: 1 when x is loaded in boxes of whole output rows (units of
                         block_m pixels = whole rows of one image) instead of im2col boxes */
} cbs_plan_info;

/* Fills `info` for the given shape, algorithm and SM count (sm_count > 0;
 * pass the device's multiprocessor count).  Host only, touches no GPU. */
int conv_bn_silu_plan(int n, int h, int w_in, int c, int c_out, int r, int s, int stride_h,
                      int stride_w, int pad_h, int pad_w, int algo, int sm_count,
                      cbs_plan_info *info);

/*
 * Overrides of the planner's choices, for measuring the alternatives on a
 * given shape ("Fusing an Epilogue", section "Three kernels for one
 * operation": which kernel and tile run is a threshold somebody measures and
 * writes down).  -1 (block_n: 0) leaves that choice to the planner.
 */
typedef struct cbs_plan_request {
    int algo;     /* cbs_algo */
    int swap_ab;  /* -1, or 0: pixel-major tiles, 1: channel-major tiles (swap AB: 128 channels x 256 pixels) */
    int stream_k; /* -1, or 0: whole tiles per CTA, 1: K steps split evenly over the grid */
    int pair;     /* -1, or 0: single CTAs, 1: 2-CTA pairs (256-wide pixel-major tiles with stream-K only) */
    int block_n;  /* 0, or 16/32/64/128/256 output channels per pixel-major tile */
    long long wait_timeout_ns; /* 0: the default bound (2 s) on every pipeline wait of the tcgen05
                                  kernel; > 0: that bound instead.  A kernel whose wait runs out
                                  records it, stops, waits for its own copies in flight, frees its
                                  tensor memory and returns: conv_bn_silu_check then reports
                                  CBS_ERR_TIMEOUT, and later calls run normally.  (A bound of a
                                  few nanoseconds makes the waits run out on purpose: the watchdog
                                  test.)  Ignored by the other kernels. */
    int balanced; /* -1, or (channel-major tiles only) 0: whole 256-pixel tiles dealt round-robin,
                     1: each CTA an equal run of 32-pixel chunks */
    int weights_resident; /* -1, or 0: weights loaded with every tile, 1: the weight tile resident in
                             tensor memory (channel-major tiles, bf16 output without a residual, when
                             the tile fits next to two accumulators) */
    int row_boxes;        /* -1, or (channel-major tiles, bf16 output without a residual) 1: x loaded in
                             boxes of whole output rows (W divisible by the stride, equal strides, up
                             to 256 output columns), 0: im2col boxes */
} cbs_plan_request;

/* conv_bn_silu_plan with overrides.  CBS_ERR_INVALID_ARG for an out-of-range
 * field; CBS_ERR_UNSUPPORTED when the kernel cannot run the combination on
 * this shape (e.g. stream-K with shares shorter than one tile, pairs without
 * stream-K, any tcgen05 override on the thin-input or direct kernels). */
int conv_bn_silu_plan_request(int n, int h, int w_in, int c, int c_out, int r, int s, int stride_h,
                              int stride_w, int pad_h, int pad_w, const cbs_plan_request *req, int sm_count,
                              cbs_plan_info *info);

/* conv_bn_silu_forward_algo with overrides (req->algo replaces `algo`); the
 * same result within the layer's tolerance, whatever the tiling. */
int conv_bn_silu_forward_request(const void *x, const void *w, const float *scale, const float *bias,
                                 void *y, int n, int h, int w_in, int c, int c_out, int r, int s,
                                 int stride_h, int stride_w, int pad_h, int pad_w, const cbs_plan_request *req,
                                 void *stream);

/*
 * ---------------------------------------------------------------------------
 * Token-wise operators: layer norm and root-mean-square norm with their gradients,
 * rows quantised to 8-bit integers, and the linear layer over such rows.  A pixel of an NHWC tensor is
 * a row of its channels, so they run on the same activations as the layers
 * above ([n*h*w][c]), and on tokens [tokens][c].
 *
 * Conventions, besides those at the top:
 *   - A matrix is given by a pointer, its number of rows, and the distance of
 *     its rows in elements; elements of one row are adjacent.  Inputs may have
 *     any distance >= 0 (0: every row the same memory), outputs at least
 *     their width.  Pointers need only be aligned to their element; rows that
 *     are 16-byte aligned throughout run on wider loads and stores (8-bit rows
 *     on 4-byte boundaries nearly as fast).  Input rows off those boundaries
 *     are read in whole aligned words of up to 16 bytes, of which each holds
 *     at least a byte of the row.
 *   - The norms, their gradients and the quantisation take up to 2^40 rows of 1 to 2^29
 *     channels; wider rows are CBS_ERR_INVALID_ARG.
 *   - dtype is a cbs_dtype and goes for every activation of the call; parameters,
 *     statistics and scales are float32, as the folded scale and bias are.
 *   - Outputs must not overlap inputs, workspaces or each other.
 *   - No call allocates.  Where a workspace is asked for, its size comes from
 *     the call's *_workspace function; it needs no initialisation, holds nothing
 *     between calls, and belongs to one call at a time.
 *   - Results are deterministic: no atomics, every sum in a fixed order for one
 *     GPU model and one set of arguments.
 */

/* Element type of activations. */
typedef enum cbs_dtype {
    CBS_DTYPE_F32 = 0,
    CBS_DTYPE_BF16 = 1,
    CBS_DTYPE_F16 = 2
} cbs_dtype;

/*
 * Layer norm of each row over its c channels:
 *   mean = sum x / c,  var = sum (x - mean)^2 / c,  rstd = 1 / sqrt(var + eps)
 *   y = (x - mean) * rstd * gamma + beta
 *   x, y  : device, dtype [rows][c], row distances x_stride and y_stride
 *   gamma : device, float32 [c], or NULL for 1;  beta : likewise, or NULL for 0
 *   eps   : >= 0 and finite (with eps == 0 a row whose variance comes out 0 gives NaN)
 *   stats : device, float32 [2][rows], written with mean, then rstd (what
 *           conv_bn_silu_layer_norm_backward needs), or NULL
 * Computed in fp32 with the variance summed around the mean; y rounded once.
 * (A constant row whose sum fp32 holds has its value as its mean, and beta as y.)
 * rows == 0 is a no-op; c >= 1.
 */
int conv_bn_silu_layer_norm(const void *x, long long x_stride, const float *gamma, const float *beta, float eps,
                            void *y, long long y_stride, float *stats, long long rows, int c, int dtype,
                            void *stream);

/*
 * Gradient of conv_bn_silu_layer_norm.  With h = (x - mean) * rstd and g = dy * gamma,
 *   dx = rstd * (g - sum_c(g)/c - h * sum_c(g*h)/c)
 *   dgamma = sum over rows of dy * h,  dbeta = sum over rows of dy
 *   dy, x, dx     : device, dtype [rows][c], row distances *_stride
 *   gamma         : as in the forward call, or NULL for 1
 *   stats         : device, float32 [2][rows], written by the forward call
 *   dgamma, dbeta : device, float32 [c], written (not added to)
 *   workspace     : device, 16-byte aligned, at least
 *                   conv_bn_silu_layer_norm_backward_workspace(rows, c) bytes
 * rows == 0 leaves dgamma and dbeta zero.
 */
int conv_bn_silu_layer_norm_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                     const float *gamma, const float *stats, void *dx, long long dx_stride,
                                     float *dgamma, float *dbeta, long long rows, int c, int dtype,
                                     void *workspace, long long workspace_bytes, void *stream);

/* Workspace of conv_bn_silu_layer_norm_backward on the current device in bytes;
 * -1 for arguments out of range or when no device answers. */
long long conv_bn_silu_layer_norm_backward_workspace(long long rows, int c);

/*
 * Rows quantised to 8-bit integers with one scale each:
 *   most = max(max_c |x|, 2^-100),  scale = most / 127,  q = round(x * (127 / most))
 * rounded to nearest even, so q * scale is x within half a step and q is in
 * [-127, 127].  A row holding a NaN or an infinity gets q = 0 and a scale that is
 * not finite, so that whatever is computed from it is NaN.
 *   x         : device, dtype [rows][c];  q : device, int8 [rows][c], written
 *   row_scale : device, float32 [rows], written
 */
int conv_bn_silu_quantize_rows(const void *x, long long x_stride, void *q, long long q_stride, float *row_scale,
                               long long rows, int c, int dtype, void *stream);

/* conv_bn_silu_layer_norm and conv_bn_silu_quantize_rows in one pass: the
 * normalised values are quantised in fp32, without being rounded to dtype first. */
int conv_bn_silu_layer_norm_quantize(const void *x, long long x_stride, const float *gamma, const float *beta,
                                     float eps, void *q, long long q_stride, float *row_scale, long long rows,
                                     int c, int dtype, void *stream);

/*
 * Root-mean-square norm of each row over its c channels, after the residual's addition:
 *   total = x + residual, rounded to dtype (residual NULL: total is x, and nothing is written)
 *   rstd = 1 / sqrt(sum total^2 / c + eps),  y = total * rstd * gamma
 *   x, residual, total, y : device, dtype [rows][c], row distances *_stride; total is written
 *           and may be residual itself (the same pointer and distance)
 *   gamma : device, float32 [c], or NULL for 1
 *   eps   : >= 0 and finite (with eps == 0 a row whose squares fp32 holds as zeros gives NaN)
 *   rstd  : device, float32 [rows], written (what conv_bn_silu_rms_norm_backward needs), or NULL
 * The norm is of the rounded total.  Computed in fp32, y rounded once; a row whose sum of squares
 * leaves fp32, at magnitudes from 2^64 / sqrt(c) on, gives zeros.
 * rows == 0 is a no-op; c >= 1.
 */
int conv_bn_silu_rms_norm(const void *x, long long x_stride, const void *residual, long long residual_stride,
                          const float *gamma, float eps, void *total, long long total_stride, void *y,
                          long long y_stride, float *rstd, long long rows, int c, int dtype, void *stream);

/* conv_bn_silu_rms_norm and conv_bn_silu_quantize_rows in one pass: the normalised values are
 * quantised in fp32, without being rounded to dtype first.  y may be NULL: it is written only
 * for callers that need the rows in dtype as well (adapters beside the int8 linear layer). */
int conv_bn_silu_rms_norm_quantize(const void *x, long long x_stride, const void *residual,
                                   long long residual_stride, const float *gamma, float eps, void *total,
                                   long long total_stride, void *y, long long y_stride, void *q,
                                   long long q_stride, float *row_scale, float *rstd, long long rows, int c,
                                   int dtype, void *stream);

/*
 * Gradient of conv_bn_silu_rms_norm.  With h = x * rstd and g = dy * gamma,
 *   dx = rstd * (g - h * sum_c(g * h) / c) [+ residual]
 *   dgamma = sum over rows of dy * h
 *   dy, x, dx : device, dtype [rows][c], row distances *_stride; x is what the forward call
 *               normalised (its total, where it had a residual)
 *   gamma     : as in the forward call, or NULL for 1
 *   rstd      : device, float32 [rows], written by the forward call
 *   residual  : device, dtype [rows][c], or NULL: the gradient that arrives at x past the norm,
 *               added in fp32 before the one rounding.  It may be dx itself.
 *   dgamma    : device, float32 [c], written (not added to)
 *   workspace : device, 16-byte aligned, at least
 *               conv_bn_silu_rms_norm_backward_workspace(rows, c) bytes
 * dx is the gradient of x and of the forward call's residual alike.
 * rows == 0 leaves dgamma zero.
 */
int conv_bn_silu_rms_norm_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                   const float *gamma, const float *rstd, const void *residual,
                                   long long residual_stride, void *dx, long long dx_stride, float *dgamma,
                                   long long rows, int c, int dtype, void *workspace, long long workspace_bytes,
                                   void *stream);

/* Workspace of conv_bn_silu_rms_norm_backward on the current device in bytes; -1 for arguments
 * out of range or when no device answers. */
long long conv_bn_silu_rms_norm_backward_workspace(long long rows, int c);

/*
 * Low-rank adapters of many requests beside a linear layer.  Row i has adapter g = index[i], or
 * none where index[i] is outside [0, adapters):
 *   hidden[i] = A_g x[i],  y[i] = base[i] + scale[g] * B_g hidden[i]      (without one: y[i] = base[i])
 *   x      : device, dtype [m][k];  index : device, int32 [m], in any order
 *   a, b   : device, dtype [adapters][rank][k] and [adapters][n][rank], dense
 *   scale  : device, float32 [adapters], or NULL for 1
 *   base   : device, dtype [m][n], or NULL for 0 (the linear layer's output).  It may be y itself,
 *            whose rows without an adapter are then left as they are
 *   y      : device, dtype [m][n], written
 *   hidden : device, float32 [m][rank], written (what conv_bn_silu_linear_adapters_backward needs;
 *            zeros without an adapter), or NULL
 *   workspace : device, 16-byte aligned, at least conv_bn_silu_linear_adapters_workspace(...)
 *               bytes; NULL when that is 0
 * Sums in fp32; with 16-bit activations hidden goes to the second product in two parts of their
 * type (f16 after a power of two a row), which keep 2^-16 (bf16) or 2^-22 of it, and y is rounded
 * once.  float32 activations are products of two-part 19-bit floats, to some 2^-21 of their terms.
 * What is computed from a value that is not finite is not finite, but may be NaN where the formula
 * gives an infinity, as may what is computed from one within 2^-8 of the largest float32.
 * m <= 2^20; 1 <= k, n <= 2^22; 1 <= rank <= 128; 1 <= adapters <= 4096.  m == 0 is a no-op.
 * Finding the rows of each adapter takes a time with the square of m, 0.15 ms for 2^18 rows and 2.1 for
 * 2^20: where that shows beside the products, calls of fewer rows are faster.
 * Adapters of lower rank than the others are padded with zeros.
 */
int conv_bn_silu_linear_adapters(const void *x, long long x_stride, const int *index, const void *a, const void *b,
                                 const float *scale, const void *base, long long base_stride, void *y,
                                 long long y_stride, float *hidden, long long m, int k, int n, int rank,
                                 int adapters, int dtype, void *workspace, long long workspace_bytes, void *stream);

/*
 * Gradients of conv_bn_silu_linear_adapters:
 *   dhidden[i] = B_g^T dy[i],  dx[i] = base[i] + scale[g] * A_g^T dhidden[i]   (without an adapter: base[i])
 *   da_g = scale[g] * sum over the rows of g of dhidden x^T,  db_g likewise of dy hidden^T
 *   dy, x, index, a, b, scale : of the forward call
 *   hidden : device, float32 [m][rank], written by the forward call
 *   base   : device, dtype [m][k], or NULL for 0: the gradient that x has from elsewhere.  It may be dx itself
 *   dx     : device, dtype [m][k], written; neither dy nor x, which are read again behind it
 *   da, db : device, float32 [adapters][rank][k] and [adapters][n][rank], written (zeros for adapters
 *            without rows)
 * The gradient of base is dy itself.  Sizes as in the forward call; m == 0 leaves da and db zero.
 */
int conv_bn_silu_linear_adapters_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                          const int *index, const void *a, const void *b, const float *scale,
                                          const float *hidden, const void *base, long long base_stride, void *dx,
                                          long long dx_stride, float *da, float *db, long long m, int k, int n,
                                          int rank, int adapters, int dtype, void *workspace,
                                          long long workspace_bytes, void *stream);

/* Workspaces of the two calls on the current device in bytes; -1 for sizes out of range or when
 * no device answers. */
long long conv_bn_silu_linear_adapters_workspace(long long m, int k, int n, int rank, int adapters);
long long conv_bn_silu_linear_adapters_backward_workspace(long long m, int k, int n, int rank, int adapters);

/*
 * AdamW step of `count` tensors, each in place:
 *   g' = grad_scale * grad,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *   param = param - (lr decay param + lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps))
 * in fp32, the parameter rounded once to its type.  Elements of a tensor are adjacent.
 *   state_bits 32: m and v are float32 [n].
 *   state_bits 8 : m and v hold 8-bit floats (e4m3) [n], each times the scale of its block of 256
 *                  elements: m, and the square root of v.  A block's scale is its largest magnitude
 *                  (2^-100 at least) / 448.  A value goes to one of the two around it: to
 *                  floor(|value| / distance + u) * distance with u in [0, 1) from the mixed bits of
 *                  (element + step * 0x9E3779B9) modulo 2^32, so the same step gives the same bits
 *                  again; where v is not 0 its root is held as 2^-9 of the scale at least.  The odds keep the
 *                  mean of a value that is rounded, not of v over many steps: under steady gradients
 *                  the held roots spread by 12 to 17 % of themselves, and v is 3 to 6 % larger than
 *                  in 32 bits (where beta2 = 0.999 leaves roots a spread of 1.6 %).  A block with a
 *                  gradient that is not finite has NaN for its m.  Zeros everywhere are the initial state.
 * What the step writes (parameters, moments, scales) may overlap neither another of these nor a
 * gradient or a number that it reads: CBS_ERR_INVALID_ARG.  Gradients may overlap each other.
 * Pointers are aligned to their element, and those aligned to 8 elements (float32 to 32 bytes) run
 * on wide loads and stores.
 */
typedef struct cbs_adamw_tensor {
    void *param;             /* device, param_dtype [n] */
    const void *grad;        /* device, grad_dtype [n] */
    void *exp_avg;           /* m */
    void *exp_avg_sq;        /* v, or its square root in 8 bits */
    float *exp_avg_scale;    /* device, float32 [(n + 255) / 256]; 8 bits only */
    float *exp_avg_sq_scale; /* likewise */
    long long n;             /* 0 <= n <= 2^40 */
    int param_dtype, grad_dtype; /* cbs_dtype */
} cbs_adamw_tensor;

typedef struct cbs_adamw_options {
    double lr, beta1, beta2, eps, weight_decay; /* finite; 0 <= beta < 1, eps >= 0.  In 64 bits, so that
                                                   1 - beta keeps its bits */
    double grad_scale;
    long long step;                /* >= 1: the number of this step, counted from 1 */
    const float *lr_device;        /* not NULL: read on the device in place of lr, grad_scale, step */
    const float *grad_scale_device;
    const long long *step_device;
    int state_bits;                /* 8 or 32 */
} cbs_adamw_options;

int conv_bn_silu_adamw_step(const cbs_adamw_tensor *tensors, int count, const cbs_adamw_options *options,
                            void *stream);

/*
 * Linear layer over 8-bit integers, scales for each row (token) and output channel:
 *   y[m][n] = act( (sum_k a[m][k] * w[n][k]) * (a_scale[m] * w_scale[n]) + bias[n] ) [+ residual[m][n]]
 *   a        : device, int8 [m][k];  w : device, int8 [n][k] (a 1x1 filter's KRSC)
 *   a_scale  : device, float32 [m];  w_scale : device, float32 [n]
 *   bias     : device, float32 [n], or NULL
 *   residual : device, out_dtype [m][n], or NULL; added after the activation, in
 *              fp32, before the one rounding.  It may be y itself.
 *   y        : device, out_dtype [m][n], written
 *   activation : a cbs_activation;  out_dtype : a cbs_dtype
 *   workspace  : device, 16-byte aligned, at least
 *                conv_bn_silu_linear_int8_workspace(...) bytes; NULL when that is 0
 * Sums are of integers: in 32-bit integers, or in fp32 on the tensor cores, which is
 * exact while partial sums stay below 2^24 and rounds beyond.  k <= 131071, n <= 2^22,
 * m < 2^31, and y of at most 2^43 elements.
 * SiLU is within 5 units in the last place of fp32 where the output is float32, and -0
 * below -88.7; where it is 16-bit, within some 1.2 |z| such units, which the rounding of
 * the output hides, and -0 below -87.3.
 * m == 0 or n == 0 is a no-op; k == 0 gives act(bias) + residual.
 * A pipeline wait that runs out is reported by conv_bn_silu_check.
 */
int conv_bn_silu_linear_int8(const void *a, long long a_stride, const void *w, long long w_stride,
                             const float *a_scale, const float *w_scale, const float *bias, const void *residual,
                             long long residual_stride, void *y, long long y_stride, long long m, int n, int k,
                             int activation, int out_dtype, void *workspace, long long workspace_bytes,
                             void *stream);

/* Workspace of conv_bn_silu_linear_int8 on the current device in bytes for these sizes, whatever
 * the pointers and row distances; -1 for sizes out of range or when no device answers. */
long long conv_bn_silu_linear_int8_workspace(long long m, int n, int k);

/* The kernels of conv_bn_silu_linear_int8. */
typedef enum cbs_linear_kernel {
    CBS_LINEAR_FEW = 0,    /* few rows: the weights streamed once past integer dot products */
    CBS_LINEAR_TILE = 1,   /* small products: one launch on the integer matrix instruction */
    CBS_LINEAR_RING = 2,   /* one operand streamed through TMA and widened into tensor memory */
    CBS_LINEAR_STREAM = 3, /* one operand streamed through registers and widened into shared memory */
    CBS_LINEAR_GEMM = 4    /* both operands widened first, then a tensor-core product */
} cbs_linear_kernel;

/* What conv_bn_silu_linear_int8 launches for these sizes. */
typedef struct cbs_linear_plan {
    int kernel;         /* cbs_linear_kernel */
    int turned;         /* RING and STREAM: 1 when a is the streamed operand in place of w */
    int tile_rows;      /* of an output tile */
    int tile_channels;
    int align;          /* bytes that the kernel takes rows of a and w to start at multiples of: 16, 4 or 1 */
    int k_steps;        /* steps of K in a tile */
    int tiles;
    int workers;        /* CTAs, or CTA pairs, that share the tiles */
} cbs_linear_plan;

/* Fills `plan` for m, n and k as in conv_bn_silu_linear_int8 and the device's SM count; align is the largest of
 * 16, 4 and 1 that the addresses and row distances of a and w are multiples of.  For rows at least k apart (RING has
 * no form for rows that overlap, which run as STREAM); all zeros where m or n is 0.  Host only, touches no GPU. */
int conv_bn_silu_linear_int8_plan(long long m, int n, int k, int align, int sm_count, cbs_linear_plan *plan);

/* Synchronises `stream`, then reads and clears the library's device error word.
 * Returns CBS_ERR_TIMEOUT if any kernel since the last check gave up on a
 * pipeline wait, CBS_ERR_CUDA if the synchronisation failed, else CBS_OK. */
int conv_bn_silu_check(void *stream);

/* Short English text for a cbs_status value (static storage, never NULL). */
const char *conv_bn_silu_status_string(int status);

/* The cudaError_t behind the calling thread's most recent CBS_ERR_CUDA (0 if none). */
int conv_bn_silu_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* CONV_BN_SILU_H */
