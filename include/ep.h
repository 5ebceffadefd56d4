/*
 * transformer_epilogue_gb300 — C ABI of the fused transformer-block epilogue ops
 * (SkipLayerNormalization, BiasSoftmax, BiasAdd, QuickGelu, GroupNorm and
 * BiasDropout, the last two with their gradients; an RMS norm to 8 bits and a
 * matrix product with its epilogue, with their gradients) for one NVIDIA GB300
 * (sm_103a) GPU.
 *
 * The ops are the com.microsoft ONNX Runtime contrib ops whose definitions are
 * given by the manifest pages "com.microsoft.SkipLayerNormalization",
 * "com.microsoft.BiasSoftmax", "com.microsoft.BiasAdd" and
 * "com.microsoft.QuickGelu" (sections `description`, `inputs`, `outputs`,
 * `attributes`, `derive`).  Each entry point below cites the section that
 * defines what it computes.  GroupNorm and BiasDropout are ops of the same
 * contrib family that have no manifest page; their declarations state the whole
 * definition.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are dense, contiguous, row-major device buffers of element type T
 *    (ep_dtype); every pointer is a device pointer owned by the caller.  The
 *    library allocates nothing and frees nothing.
 *  - Every call is asynchronous: it validates on the host, enqueues its kernel(s)
 *    on `stream` and returns without synchronising.  Outputs are valid once the
 *    stream reaches that point.  A NULL stream is the legacy default stream.
 *  - Kernels are launched as programmatic dependents of the work before them in
 *    the stream (CUDA programmatic dependent launch): their blocks may be
 *    scheduled while that work drains, but no block reads or writes global
 *    memory before every kernel ahead of it in the stream has completed, so the
 *    ordering seen by the caller is ordinary stream order.  Calls may be
 *    captured into CUDA graphs (a workspace must then outlive the graph).
 *  - All validation happens before anything is enqueued.  A contract violation
 *    returns EP_ERR_INVALID_ARG, a legal op this library does not implement
 *    (another element type, an unsupported rank) returns EP_ERR_UNSUPPORTED, a
 *    call without the workspace it needs returns EP_ERR_WORKSPACE, and
 *    a launch error reported by the CUDA runtime returns EP_ERR_CUDA.  On any
 *    non-OK status nothing has been enqueued, except for EP_ERR_CUDA (the
 *    runtime's state is then whatever the failing launch left).  ep_last_error()
 *    gives a message for the calling thread's last non-OK status.
 *  - Empty tensors (numel 0) return EP_OK without launching anything; their
 *    pointers may be NULL.  (Sums over them, dgamma, dbeta and dbias, are set
 *    to 0 on the stream.)
 *  - Pointers must be aligned to sizeof(T).  16-byte alignment is not
 *    required: it selects the 128-bit vector path (BiasAdd and QuickGelu also
 *    when X, skip and Y share one offset within 16 bytes), and other alignments
 *    take a scalar path computing the same function (the results agree within
 *    the ops' tolerances).
 *  - An output may alias an input exactly (same address, same size: in place).
 *    Any other overlap between an output and another operand is rejected.
 *  - Counts and offsets are 64-bit.
 *  - Arithmetic is float32 for every element type; float16 and bfloat16
 *    results are rounded once, to nearest-even, when stored.
 */
#ifndef TRANSFORMER_EPILOGUE_EP_H
#define TRANSFORMER_EPILOGUE_EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream; the same type as cudaStream_t (struct CUstream_st*). */
typedef struct CUstream_st* ep_stream_t;

/* Element type T.  The manifests' typeConstraints list float32 and float16
 * (typeConstraints of all four manifests); the op schemas also allow
 * bfloat16, which the WebGPU package leaves out (QuickGelu and
 * SkipLayerNormalization `description`) and this library implements. */
typedef enum { EP_F32 = 0, EP_F16 = 1, EP_BF16 = 2 } ep_dtype;

typedef enum {
  EP_OK = 0,
  EP_ERR_INVALID_ARG = 1,   /* shape, attribute, pointer or overlap contract violated   */
  EP_ERR_UNSUPPORTED = 2,   /* legal for the op, not implemented here (dtype, rank)     */
  EP_ERR_WORKSPACE = 3,     /* a needed workspace is NULL, too small, misaligned or overlapping */
  EP_ERR_CUDA = 4           /* the CUDA runtime reported an error for a launch          */
} ep_status;

/* Message for the calling thread's last non-OK status ("" if none).  The string
 * belongs to the library and stays valid until the thread's next call. */
const char* ep_last_error(void);

/* Name of a status code, e.g. "EP_ERR_INVALID_ARG". */
const char* ep_status_name(ep_status s);

/* Number of kernels this library has enqueued in this process (all threads). */
uint64_t ep_kernel_launch_count(void);

/* Version of this ABI (incremented on any incompatible change). */
int ep_abi_version(void);

/* Failure detection.  Every shared-memory barrier wait in the staged kernels
 * is bounded (1 s); a wait that runs out is counted on the device, the kernel
 * stops its remaining work without leaving copies in flight, and the affected
 * outputs are not written.  ep_pipeline_timeouts() adds up those counts on the
 * current device into *count (0 when nothing timed out) and, if clear != 0,
 * resets them.  It synchronises with the device.  No op definition covers
 * this; it exists because the library's kernels wait on barriers. */
ep_status ep_pipeline_timeouts(uint64_t* count, int clear);

/* Self-test of that mechanism: launches a one-CTA kernel on `stream` whose
 * barrier wait is set up to run out (it expects 16 bytes that no copy
 * delivers) with a limit of timeout_us microseconds (1..1000000), waits for the
 * stream, and stores in *timeouts_seen how many timed-out waits the library
 * counted meanwhile (1 expected).  The kernel returns normally after the
 * limit; the device stays usable.  EP_ERR_INVALID_ARG for a limit out of
 * range or a NULL timeouts_seen. */
ep_status ep_selftest_bounded_wait(uint32_t timeout_us, uint64_t* timeouts_seen, ep_stream_t stream);

/*
 * SkipLayerNormalization
 *   com.microsoft.SkipLayerNormalization manifest: `description`, `inputs`,
 *   `outputs`, `attributes.epsilon`, `derive.rank2CoreContract`,
 *   `derive.broadcastSkipShapeOk`.
 *
 *   s = (input + skip) + bias          (float32, in this order; bias optional)
 *   input_skip_bias_sum = T(s)         (optional output)
 *   mu = mean(s), var = mean((s-mu)^2) over the last (hidden) axis, population
 *   output = (s - mu) / sqrt(var + epsilon) * gamma + beta   (beta optional)
 *
 * input      [in_rank dims], in_rank 2 (rows, H) or 3 (N, S, H); H > 0.
 * skip       rank 2: the shape of input.  rank-3 input: the shape of input,
 *            (1, S, H) or (S, H); row r of input uses skip row r mod skipRows,
 *            skipRows = numel(skip) / H.
 * gamma      H elements (required).  beta, bias: H elements or NULL.
 * epsilon    >= 0 (the op's default is 9.999999960041972e-13, float32 1e-12).
 * output     shape of input.
 * input_skip_bias_sum   shape of input, or NULL.
 *
 * Errors: EP_ERR_UNSUPPORTED for a dtype other than EP_F32/EP_F16/EP_BF16 or a rank
 * other than 2/3; EP_ERR_INVALID_ARG for a non-positive H, a skip shape not
 * listed above, a negative or NaN epsilon, a NULL required pointer, a
 * misaligned pointer or an overlap other than exact in-place aliasing.
 */
ep_status ep_skip_layer_norm(ep_dtype t,
                             const void* input, const int64_t* in_shape, int in_rank,
                             const void* skip, const int64_t* skip_shape, int skip_rank,
                             const void* gamma, const void* beta, const void* bias,
                             float epsilon,
                             void* output, void* input_skip_bias_sum,
                             ep_stream_t stream);

/*
 * SkipLayerNormalization with the RMS form and the per-row statistics.
 *   The manifests' SkipLayerNormalization shaders carry a `simplified` flag
 *   (always false in the package; the RMS form of the contrib op family,
 *   SkipSimplifiedLayerNormalization), and the op's `description` names the
 *   training-statistics outputs it does not implement.  This entry point adds
 *   both to ep_skip_layer_norm (same arguments, layout and errors otherwise):
 *
 * simplified   0: as ep_skip_layer_norm.  1: RMS form, no mean subtraction:
 *              output = s / sqrt(mean(s^2) + epsilon) * gamma (+ beta)
 *              (beta is normally NULL in this form).
 * mean         NULL, or numel(input)/H float32 values: the mean of each row's s
 *              (0 when simplified).
 * inv_std_dev  NULL, or numel(input)/H float32 values: 1/sqrt(var + epsilon)
 *              (1/sqrt(mean(s^2) + epsilon) when simplified).
 * The float32 outputs must be 4-byte aligned and overlap no other operand.
 */
ep_status ep_skip_layer_norm_ex(ep_dtype t,
                                const void* input, const int64_t* in_shape, int in_rank,
                                const void* skip, const int64_t* skip_shape, int skip_rank,
                                const void* gamma, const void* beta, const void* bias,
                                float epsilon, int simplified,
                                void* output, void* input_skip_bias_sum,
                                float* mean, float* inv_std_dev,
                                ep_stream_t stream);

/*
 * BiasSoftmax
 *   com.microsoft.BiasSoftmax manifest: `description`, `attributes.axis`,
 *   `attributeDescriptions.is_inner_broadcast`, `derive` (axisNorm, batchCount,
 *   blockSize, biasBlockCount, biasContract).
 *
 *   axisN = axis < 0 ? axis + rank : axis           (0 <= axisN < rank)
 *   batchCount = prod(shape[0:axisN]); blockSize = prod(shape[axisN:rank])
 *   biasRows = bias_numel / blockSize; innerRepeat = batchCount / biasRows
 *   bias row of data row r: r / innerRepeat if is_inner_broadcast != 0,
 *                           r % biasRows    otherwise
 *   output[r, :] = softmax(data[r, :] + bias[bias row, :])
 *
 * data, output  `rank` dims given by `shape` (1 <= rank <= 16).
 * bias          bias_numel elements; only its element count matters.
 * The biasContract must hold: bias_numel % blockSize == 0,
 * 0 < biasRows <= batchCount and batchCount % biasRows == 0, or data and bias
 * are both empty.
 * workspace     device scratch for rows too long to keep on chip (the split-row
 *               path); ep_bias_softmax_workspace_size() gives the bytes needed
 *               (0 when the row path is taken; then workspace may be NULL).
 *               16-byte aligned; its contents on entry do not matter.
 *
 * Errors: EP_ERR_INVALID_ARG for an axis out of range, a violated biasContract,
 * NULL/misaligned pointers or overlaps; EP_ERR_WORKSPACE when the split-row
 * path needs more than workspace_bytes or workspace is NULL/misaligned.
 */
ep_status ep_bias_softmax(ep_dtype t,
                          const void* data, const int64_t* shape, int rank,
                          const void* bias, int64_t bias_numel,
                          int axis, int is_inner_broadcast,
                          void* output,
                          void* workspace, size_t workspace_bytes,
                          ep_stream_t stream);

/* Workspace bytes ep_bias_softmax needs for this dtype, shape and axis (0 if
 * none).  Returns 0 as well for arguments ep_bias_softmax would reject. */
size_t ep_bias_softmax_workspace_size(ep_dtype t, const int64_t* shape, int rank, int axis);

/*
 * BiasSoftmax without a caller-provided workspace.
 *   The op definition has no counterpart to this entry point: it is a variant
 *   of ep_bias_softmax for callers that cannot allocate device memory, e.g. a
 *   plugin or engine whose device memory is all reserved at start-up, code
 *   running inside an allocator or memory-pool callback, or a loop that cannot
 *   afford the device-wide synchronisation cudaMalloc/cudaFree may cause.  Such
 *   callers have no way to provide the scratch the split-row path needs.
 *
 * Same arguments, results and errors as ep_bias_softmax, minus the workspace.
 * The split-row scratch comes from a fixed 1 MiB device array inside the
 * library (held by every device that loads the library until process exit),
 * so rows * ceil(blockSize / chunk) must not exceed 131072 when blockSize >
 * 16384, with chunk = 4096 for float32 and 8192 for float16/bfloat16; larger shapes
 * return EP_ERR_WORKSPACE before anything is enqueued.
 * Rows of up to 16384 elements need no scratch and have no such limit.
 * This entry point allocates nothing.
 *
 * The first call on a device that needs the scratch looks up its device
 * address (cudaGetSymbolAddress, with that device current); make that first
 * call before any stream capture.  All calls share the one array, which keeps
 * the previous call's contents: every entry a call reads is written earlier in
 * the same call, so nothing needs clearing, but calls that may overlap on the
 * GPU (other streams, other threads) race on the array and must be ordered by
 * the caller.
 */
ep_status ep_bias_softmax_noalloc(ep_dtype t,
                                  const void* data, const int64_t* shape, int rank,
                                  const void* bias, int64_t bias_numel,
                                  int axis, int is_inner_broadcast,
                                  void* output, ep_stream_t stream);

/*
 * BiasAdd
 *   com.microsoft.BiasAdd manifest: `description`, `inputs`, `outputs`.
 *
 *   Y[n, s, c] = (X[n, s, c] + bias[c]) + skip[n, s, c]
 *
 * shape   3 dims (N, S, C) of X, skip and Y; bias has C elements.
 * For float32 the three-term sum is compensated (error-free two-sums), so Y
 * is within one rounding of the exact sum even under cancellation.
 *
 * Errors: EP_ERR_INVALID_ARG for negative dims, NULL/misaligned pointers or
 * overlaps.
 */
ep_status ep_bias_add(ep_dtype t, const void* X, const int64_t* shape,
                      const void* bias, const void* skip, void* Y,
                      ep_stream_t stream);

/*
 * QuickGelu
 *   com.microsoft.QuickGelu manifest: `description`, `attributes.alpha`.
 *
 *   Y = X * sigmoid(alpha * X)       elementwise over numel elements
 *
 * alpha   the op's default is 1.702.
 *
 * Errors: EP_ERR_INVALID_ARG for numel < 0, NULL/misaligned pointers or
 * overlaps.
 */
ep_status ep_quick_gelu(ep_dtype t, const void* X, int64_t numel, float alpha,
                        void* Y, ep_stream_t stream);

/* Activation of GroupNorm (the contrib op's `activation` attribute). */
typedef enum {
  EP_ACT_NONE = 0,
  EP_ACT_SILU = 1,
  /* of the matrix product alone */
  EP_ACT_RELU = 2,
  EP_ACT_QUICK_GELU = 3,
  EP_ACT_GELU = 4,
  EP_ACT_FAST_GELU = 5
} ep_activation;

/*
 * GroupNorm
 *   The GroupNorm op of the com.microsoft contrib family with channels_last = 1.
 *   The channels of X form `groups` groups of D = C / groups neighbours; per
 *   sample n and group g, over its S * D values:
 *
 *   mu = mean(X), var = mean((X - mu)^2)          (population)
 *   u[n, s, c] = (X[n, s, c] - mu) / sqrt(var + epsilon) * gamma[c] + beta[c]
 *   Y = u (EP_ACT_NONE) or u * sigmoid(u) (EP_ACT_SILU)
 *
 * shape        3 dims (N, S, C) of X and Y; S is the product of the spatial
 *              sizes (1: a norm over each token's groups of channels).  C is at
 *              most 2^24.
 * gamma        C elements (required).  beta: C elements or NULL.
 * groups       > 0, divides C.
 * epsilon      >= 0 (the op's default is 1e-5).
 * mean, inv_std_dev   NULL, or N * groups float32 values: mu and
 *              1/sqrt(var + epsilon), which ep_group_norm_grad takes.
 * workspace    device scratch of ep_group_norm_workspace_size() bytes, or where X
 *              and Y start on 16-byte boundaries of
 *              ep_group_norm_workspace_size_aligned() (may be NULL when that is 0:
 *              small samples and tokens), 16-byte aligned; its contents on entry
 *              do not matter.  Calls that may overlap on the GPU (other streams,
 *              concurrently replayed graphs) need one each.
 * Y may be X.  Of an empty tensor nothing is written, mean and inv_std_dev
 * included.
 *
 * Errors: EP_ERR_UNSUPPORTED for another dtype or C > 2^24; EP_ERR_INVALID_ARG
 * for negative dims, groups that do not divide C, a negative or NaN epsilon, another
 * activation, NULL/misaligned pointers or overlaps; EP_ERR_WORKSPACE.
 */
ep_status ep_group_norm(ep_dtype t, const void* X, const int64_t* shape,
                        const void* gamma, const void* beta,
                        int64_t groups, float epsilon, int activation,
                        void* Y, float* mean, float* inv_std_dev,
                        void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* Workspace bytes ep_group_norm needs, for operands at any address or on 16-byte
 * boundaries (never more); 0 as well for arguments it rejects.  They depend on
 * the arguments alone. */
size_t ep_group_norm_workspace_size(ep_dtype t, const int64_t* shape, int64_t groups);
size_t ep_group_norm_workspace_size_aligned(ep_dtype t, const int64_t* shape, int64_t groups);

/*
 * Gradient of ep_group_norm.
 *   With h = (X - mean) * inv_std_dev, u = h * gamma + beta, s = sigmoid(u):
 *
 *   du = dY (EP_ACT_NONE) or dY * s * (1 + u * (1 - s)) (EP_ACT_SILU)
 *   dbeta[c] = sum over n, s of du,  dgamma[c] = sum over n, s of du * h
 *   dX = inv_std_dev * (du * gamma - m1 - h * m2),
 *   m1 = mean over the group of du * gamma, m2 of du * gamma * h
 *
 * dY, X, dX    (N, S, C).  dX may be dY or X.
 * gamma, beta, groups, activation   as in the forward call (beta NULL if it was).
 * mean, inv_std_dev   N * groups float32 values, as ep_group_norm wrote them.
 * dgamma, dbeta   C elements of T each, or NULL where not wanted.  The sums
 *              are float32 in a fixed order (the same call gives the same
 *              bits), rounded once: a float16 sum beyond 65504 is infinite.  Of an
 *              empty tensor they are set to 0.
 * workspace    ep_group_norm_grad_workspace_size() bytes, or where dY, X and dX start
 *              on 16-byte boundaries ..._aligned(), as for ep_group_norm.
 *
 * Errors: as ep_group_norm.
 */
ep_status ep_group_norm_grad(ep_dtype t, const void* dY, const void* X, const int64_t* shape,
                             const void* gamma, const void* beta, int64_t groups, int activation,
                             const float* mean, const float* inv_std_dev,
                             void* dX, void* dgamma, void* dbeta,
                             void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* Workspace bytes ep_group_norm_grad needs, as for ep_group_norm. */
size_t ep_group_norm_grad_workspace_size(ep_dtype t, const int64_t* shape, int64_t groups);
size_t ep_group_norm_grad_workspace_size_aligned(ep_dtype t, const int64_t* shape, int64_t groups);

/*
 * BiasDropout
 *   The BiasDropout op of the com.microsoft contrib family, with its mask a
 *   function of the element's index instead of an output:
 *
 *   Y[i] = residual[i] + keep(i) * (X[i] + bias[i mod C]) / (1 - ratio)
 *   keep(i) = word(i) < K,  K = round((1 - ratio) * 2^32), but 1 at least
 *             (a ratio within 2^-33 of 1 keeps the word 0)
 *   word(i) = 32-bit word number i mod 4 of Philox4x32-10 (Salmon, Moraes, Dror
 *             and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011)
 *             with the counter words (i/4 low, i/4 high, offset low, offset
 *             high) and the key words (seed low, seed high)
 *
 *   i is the flat index in X.  The same seed, offset and shape give the same
 *   mask in every call, whatever the element type, and in the gradient; each
 *   dropout of a step takes an offset (or seed) of its own.
 *
 * X, Y         `rank` dims given by `shape` (1 <= rank <= 16), C the last.
 * bias         C elements or NULL.  residual: the shape of X, or NULL.
 * ratio        0 <= ratio < 1; 0 keeps everything.
 * offset_device   NULL, or a device pointer to a 64-bit number that is added
 *              to offset (modulo 2^64) when the kernel runs: a captured graph
 *              draws another mask on each replay if the number is changed in
 *              between.
 * A dropped element is the residual (or 0) whatever X holds there, infinities
 * and NaN included.  Y may be X or residual.
 *
 * Errors: EP_ERR_UNSUPPORTED for another dtype or rank > 16; EP_ERR_INVALID_ARG
 * for negative dims, a ratio outside [0, 1), NULL/misaligned pointers or
 * overlaps.
 */
ep_status ep_bias_dropout(ep_dtype t, const void* X, const int64_t* shape, int rank,
                          const void* bias, const void* residual,
                          double ratio, uint64_t seed, uint64_t offset, const uint64_t* offset_device,
                          void* Y, ep_stream_t stream);

/*
 * Gradient of ep_bias_dropout (that of the residual is dY itself).
 *
 *   dX[i] = keep(i) * dY[i] / (1 - ratio),  dbias[c] = sum over rows of dX[., c]
 *
 * ratio, seed, offset, offset_device   as in the forward call (*offset_device
 *              too must still hold the forward call's number).
 * dX           the shape of dY; may be dY.
 * dbias        C elements of T, or NULL.  The sum is float32, over the values
 *              before they are rounded to T, in a fixed order, rounded once (beyond
 *              65504 a float16 sum is infinite).
 *              Of an empty tensor it is set to 0.
 * workspace    with dbias: ep_bias_dropout_grad_workspace_size() bytes, 16-byte
 *              aligned; its contents on entry do not matter.  Calls that may
 *              overlap on the GPU need one each.
 *
 * Errors: as ep_bias_dropout; EP_ERR_WORKSPACE.
 */
ep_status ep_bias_dropout_grad(ep_dtype t, const void* dY, const int64_t* shape, int rank,
                               double ratio, uint64_t seed, uint64_t offset, const uint64_t* offset_device,
                               void* dX, void* dbias,
                               void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* Workspace bytes ep_bias_dropout_grad needs for dbias; 0 as well for
 * arguments it rejects. */
size_t ep_bias_dropout_grad_workspace_size(ep_dtype t, const int64_t* shape, int rank);

/*
 * MX8: rows held in 8 bits (the OCP microscaling format MXFP8 with E4M3 elements)
 *
 *   32 consecutive elements of a row (its last group may be shorter) share one
 *   E8M0 scale: a byte b that stands for 2^(b - 127), 255 for NaN.
 *     b = max(1, ceil(log2(amax / 448)) + 127),  amax = the group's largest magnitude
 *     q = E4M3(x * 2^(127 - b)), rounded to nearest even;  value = q * 2^(b - 127)
 *   Nothing saturates (|x| 2^(127 - b) <= 448).  A NaN becomes a NaN element; an
 *   infinity, which E4M3 lacks, makes its group's scale NaN (all its values read NaN).
 *   (rows, H) values are rows * H bytes of elements and rows * ceil(H / 32) bytes of
 *   scales, both dense.  The format comes from the OCP Microscaling Formats
 *   specification; no op definition covers these entry points.
 *
 * ep_quantize_mx8     X (`rank` dims, rows along the last) of T -> Q, scales.
 * ep_dequantize_mx8   Q, scales -> Y of T: exact, but where a value lies beyond T's
 *                     range (float16: infinite from 65520 on; float32 and bfloat16 from
 *                     2^128 on) or is subnormal in it (rounded).
 *
 * Errors: EP_ERR_UNSUPPORTED for another dtype, rank > 16, a last dimension H over
 * 2^31 - 512 or rows * ceil(H / 256) over 2^33; EP_ERR_INVALID_ARG for negative dims,
 * rank 0, NULL/misaligned pointers or any overlap.
 */
ep_status ep_quantize_mx8(ep_dtype t, const void* X, const int64_t* shape, int rank,
                          void* Q, uint8_t* scales, ep_stream_t stream);
ep_status ep_dequantize_mx8(ep_dtype t, const void* Q, const uint8_t* scales, const int64_t* shape, int rank,
                            void* Y, ep_stream_t stream);

/*
 * RMS norm with the residual's addition and an output in MX8: what
 * ep_skip_layer_norm_ex computes in its simplified form, ready for an 8-bit
 * product (the contrib op family's SkipSimplifiedLayerNormalization).
 *
 *   s = (input + skip) + bias           (float32, in this order; skip and bias optional)
 *   input_skip_bias_sum = T(s)          (optional output)
 *   inv = 1 / sqrt(mean(s^2) + epsilon) over the last axis (a float32 sum, in an order fixed
 *         by the shape and by which operands start on 16-byte boundaries)
 *   Q, scales = MX8(s * inv * gamma)    (of the float32 values: not rounded to T before)
 *
 * input, skip   `rank` dims (1 <= rank <= 16); skip has input's shape, or is NULL.
 * gamma         H elements (required), H > 0 the last dimension; bias: H elements or NULL.
 * inv_std_dev   NULL, or one float32 a row.
 * input_skip_bias_sum   NULL, or the shape of input; may be input or skip.
 *
 * Errors: as ep_quantize_mx8; EP_ERR_INVALID_ARG also for H = 0, a negative or NaN
 * epsilon or an overlap other than the above.
 */
ep_status ep_skip_rms_norm_mx8(ep_dtype t, const void* input, const int64_t* shape, int rank,
                               const void* skip, const void* gamma, const void* bias, float epsilon,
                               void* Q, uint8_t* scales, void* input_skip_bias_sum, float* inv_std_dev,
                               ep_stream_t stream);

/*
 * Gradient of the RMS norm (of ep_skip_rms_norm_mx8, the rounding to 8 bits taken
 * as the identity, and of ep_skip_layer_norm_ex in its simplified form).
 *
 *   u = dY * gamma,  h = s * inv
 *   dX = inv * (u - h * mean(u * h)) + dsum    (the gradient of input and of skip)
 *   dgamma = sum over rows of dY * h,  dbias = sum over rows of dX
 *
 * s             input_skip_bias_sum as the forward call left it; inv_std_dev its float32 statistic.
 * dsum          the gradient that reaches input_skip_bias_sum by other ways (the residual stream), or NULL.
 * dX            the shape of dY; may be dY, s or dsum.
 * dgamma, dbias H elements of T, or NULL: float32 sums of the unrounded values, rounded once
 *               (float16: infinite from 65520 on).  Of no rows they are set to 0.  The order of all
 *               sums is fixed by the shape and by which operands start on 16-byte boundaries.
 * workspace     ep_skip_rms_norm_grad_workspace_size() bytes, 16-byte aligned; its contents
 *               on entry do not matter.  Calls that may overlap on the GPU need one each.
 *
 * Errors: as ep_skip_rms_norm_mx8; EP_ERR_WORKSPACE.
 */
ep_status ep_skip_rms_norm_grad(ep_dtype t, const void* dY, const void* input_skip_bias_sum, const int64_t* shape,
                                int rank, const void* gamma, const float* inv_std_dev, const void* dsum,
                                void* dX, void* dgamma, void* dbias,
                                void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* Workspace bytes ep_skip_rms_norm_grad needs; 0 as well for arguments it rejects. */
size_t ep_skip_rms_norm_grad_workspace_size(ep_dtype t, const int64_t* shape, int rank);

/*
 * Matrix product with bias, activation and residual in its epilogue
 *
 *   z = A W^T + bias,  Y = act(z) + residual
 *
 * A             (M, K) row-major; W (N, K) row-major (a row for each output channel).
 *               ep_matmul_bias_act: of T; ep_matmul_bias_act_mx8: E4M3 elements with
 *               A_scales (M, ceil(K / 32)) and W_scales (N, ceil(K / 32)), see MX8 above.
 * t             T, EP_F16 or EP_BF16: bias, residual, Y and Z (and A and W of the first form).
 * bias          N elements, or NULL.  residual: (M, N), or NULL.
 * activation    EP_ACT_NONE; EP_ACT_SILU z s(z); EP_ACT_RELU; EP_ACT_QUICK_GELU z s(alpha z);
 *               EP_ACT_GELU z Phi(z) (the error function); EP_ACT_FAST_GELU its tanh form
 *               z s(2 sqrt(2/pi) (z + 0.044715 z^3)).  s(x) = 1 / (1 + e^-x).  At z = -infinity
 *               the last five are 0, EP_ACT_QUICK_GELU where alpha > 0: with alpha < 0 it is
 *               0 at +infinity and -infinity at -infinity, with alpha = 0 NaN at both.
 *               Results of theirs below 2^-100 in magnitude may be 0.
 *               alpha: of EP_ACT_QUICK_GELU alone (the QuickGelu op's default is 1.702), finite.
 * Y             (M, N); may be residual.
 * Z             NULL, or the pre-activation as the gradient wants it: (M, N) of T, or with
 *               Z_scales (M, ceil(N / 32)) in MX8.
 * Products are exact, sums float32 (in an order that depends on the shape alone),
 * each result rounded once.
 * workspace     ep_matmul_bias_act_workspace_size() bytes, 16-byte aligned: rows of K
 *               elements that are no multiple of 16 bytes, or operands that do not start on
 *               16-byte boundaries, are copied to where they are; large 8-bit products
 *               arrange their scales in it.  Calls that may overlap on the GPU need one each.
 * K = 0 gives z = bias.
 *
 * Errors: EP_ERR_UNSUPPORTED for another dtype, M, N or K over 2^31 - 512 or operands
 * over 2^40 elements; EP_ERR_INVALID_ARG for negative sizes, an unknown activation, an infinite or NaN
 * alpha, missing or misaligned pointers, Z_scales without Z, or an overlap of an output
 * other than Y exactly residual; EP_ERR_WORKSPACE.
 */
ep_status ep_matmul_bias_act(ep_dtype t, const void* A, const void* W, int64_t M, int64_t N, int64_t K,
                             const void* bias, const void* residual, int activation, float alpha,
                             void* Y, void* Z, uint8_t* Z_scales,
                             void* workspace, size_t workspace_bytes, ep_stream_t stream);
ep_status ep_matmul_bias_act_mx8(ep_dtype t, const void* A, const uint8_t* A_scales,
                                 const void* W, const uint8_t* W_scales, int64_t M, int64_t N, int64_t K,
                                 const void* bias, const void* residual, int activation, float alpha,
                                 void* Y, void* Z, uint8_t* Z_scales,
                                 void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* Workspace bytes of the two (mx8 != 0: of the second).  aligned16 != 0: A and W
 * start on 16-byte boundaries.  0 where none is needed, and for arguments they reject. */
size_t ep_matmul_bias_act_workspace_size(int mx8, int64_t M, int64_t N, int64_t K, int aligned16);

/*
 * Gradient of ep_matmul_bias_act (that of the residual is dY itself), from what
 * the forward pass kept in T or in MX8.
 *
 *   dz = dY * act'(Z),  dA = dz W,  dW = dz^T A,  dbias = sum over rows of dz
 *
 * A             (M, K) of T, or with A_scales in MX8 (its values are taken in T for dW).
 * W             (N, K) of T.
 * Z             as the forward call left it: (M, N) of T, or with Z_scales in MX8.
 *               Not read (and may be NULL) with EP_ACT_NONE.
 * dA, dW, dbias (M, K), (N, K) and N elements of T, or NULL where not wanted.  dz is rounded
 *               to T in front of the products of dA and dW (not of dbias); sums are float32,
 *               rounded once (float16: infinite from 65520 on).
 *               Sums over no rows (M = 0, or N = 0 for dA) are set to 0.
 * workspace     ep_matmul_bias_act_grad_workspace_size() bytes, 16-byte aligned (dz and the
 *               operands that are copied).  Calls that may overlap on the GPU need one each.
 *
 * Errors: as ep_matmul_bias_act; no output may overlap another operand.
 */
ep_status ep_matmul_bias_act_grad(ep_dtype t, const void* dY, const void* A, const uint8_t* A_scales,
                                  const void* W, const void* Z, const uint8_t* Z_scales,
                                  int64_t M, int64_t N, int64_t K, int activation, float alpha,
                                  void* dA, void* dW, void* dbias,
                                  void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* Its workspace bytes.  a_mx8: A comes with A_scales; aligned16: dY, W and a
 * 16-bit A start on 16-byte boundaries.  0 as well for arguments it rejects. */
size_t ep_matmul_bias_act_grad_workspace_size(int64_t M, int64_t N, int64_t K, int activation, int a_mx8,
                                              int aligned16);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* TRANSFORMER_EPILOGUE_EP_H */
