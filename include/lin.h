/*
 * lin.h - C ABI of a GB300 (sm_103a) library for the transformer linear layer
 *
 *     Y = act(X . W^T + bias)
 *
 * X is M x K row-major (one row per token / batch vector), W is N x K
 * row-major ("out x in", the way PyTorch stores a linear layer's weight), Y
 * is M x N row-major. Output (m, n) is the inner product of row m of X and
 * row n of W ("One multiply, one RTX 5090, eight kernels", section "The
 * multiply"). The bias (length N, optional) and the activation are applied in
 * the store of the product ("Writing a CUDA matmul that catches cuBLAS",
 * sections "The bias add did not need to exist" and "The residual and GELU go
 * the same way"). The activation is the identity or the tanh form of GELU,
 * 0.5 s (1 + tanh(sqrt(2/pi) (s + 0.044715 s^3))), applied to (sum + bias).
 *
 * All pointers to X, W, bias and Y are DEVICE pointers on the context's
 * device, owned by the caller. Every call is asynchronous on the given CUDA
 * stream (a cudaStream_t passed as void*, NULL = legacy default stream) and
 * returns after the work is enqueued; no call synchronises except
 * lin_check_device. No call ever computes on the host: when the GPU path
 * cannot run the call returns an error.
 *
 * Status codes: 0 on success, a negative LIN_ERR_* otherwise; lin_strerror
 * gives a message. No C++ exception crosses this boundary.
 */
#ifndef LIN_H
#define LIN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LIN_ABI_VERSION 1

#if defined(__GNUC__)
#define LIN_API __attribute__((visibility("default")))
#else
#define LIN_API
#endif

/* Arithmetic of the multiply.
 * FP32: fp32 X, W, Y; fp32 fused multiply-add on the CUDA cores (exact fp32
 *       products, fp32 sums) - the path of the sgemm ladder ("Writing a CUDA
 *       matmul that catches cuBLAS", "Kernel 8: the loop was shaped wrong").
 * TF32: fp32 X, W, Y; tensor-core products of the operands' TF32 parts with
 *       fp32 accumulation ("Writing a CUDA matmul that catches cuBLAS",
 *       "Kernel 9: the silicon I had not touched").
 * BF16: bf16 X, W, Y; fp32 bias; tensor-core bf16 products with fp32
 *       accumulation, output rounded to nearest-even bf16 ("One multiply, one
 *       RTX 5090, eight kernels", "From 748 to 29 microseconds"). */
typedef enum {
    LIN_PREC_FP32 = 0,
    LIN_PREC_TF32 = 1,
    LIN_PREC_BF16 = 2
} lin_precision;

/* Activation applied after the bias. */
typedef enum {
    LIN_EPI_NONE = 0,
    LIN_EPI_GELU_TANH = 1
} lin_epilogue;

typedef enum {
    LIN_OK = 0,
    LIN_ERR_ARG = -1,            /* NULL pointer, negative size, unknown enum, Y aliasing an input */
    LIN_ERR_ALIGN = -2,          /* X or W not 16-byte aligned, or K * element size not a multiple of 16 */
    LIN_ERR_WORKSPACE = -3,      /* an explicit plan needs more workspace than the context holds */
    LIN_ERR_CUDA = -4,           /* a CUDA runtime call or kernel launch failed */
    LIN_ERR_DEVICE_TIMEOUT = -5, /* a kernel gave up a bounded wait and skipped its work */
    LIN_ERR_UNSUPPORTED = -6     /* the plan's kernel cannot run this shape / precision */
} lin_status;

/* Kernels a plan can name. */
typedef enum {
    LIN_KERNEL_NONE = 0,   /* M == 0 or N == 0: nothing to do */
    LIN_KERNEL_FILL = 1,   /* K == 0: Y = act(bias) (or act(0)) */
    LIN_KERNEL_SKINNY = 2, /* M <= 16, BF16: W stream on the tensor cores, split-K in a cluster (no workspace) */
    LIN_KERNEL_FFMA = 3,   /* FP32: register-tiled FFMA, optional split-K */
    LIN_KERNEL_TC = 4,     /* TF32 / BF16: TMA + tcgen05 + TMEM, fused epilogue */
    LIN_KERNEL_GEMV = 5    /* FP32 / TF32 M <= 8, BF16 M <= 4 (the table: BF16 one row only): one pass over W in fp32 FMAs */
} lin_kernel;

/* One launch configuration, chosen by the dispatch table or given explicitly.
 * splits > 1 is split-K: each CTA sums one range of K into the workspace and
 * the last CTA to finish a tile adds the ranges in fixed order (0, 1, ...),
 * so results are bitwise repeatable ("Optimizing a GPT-2-class transformer on
 * a GPU", Act I, split-K combined by a fixed-order reduction). */
typedef struct {
    int kernel;   /* lin_kernel */
    int variant;  /* kernel-specific tile configuration id. TC: 0, 1, 2 = one CTA
                   * per 128 x 256 / 128 / 192 tile; 3, 4, 5 = SM pairs (2-CTA
                   * clusters issuing cta_group::2 MMAs) per 256 x 256 / 128 / 192
                   * tile. SKINNY and FFMA: see the kernels' sources. */
    int bm, bn, bk;
    int splits;   /* >= 1 */
    int stages;   /* shared-memory pipeline depth (TC), 0 otherwise */
    int grid_x, grid_y, grid_z; /* TC: grid_z = K splits (1 = none; the splits of a tile
                                 * are added in order by the last one to finish) */
    int threads;
    long long workspace_bytes; /* bytes of context workspace the launch uses */
} lin_plan;

typedef struct lin_ctx lin_ctx; /* opaque; owned by the library */

/* Create a context on CUDA device `device`. Allocates `max_workspace_bytes`
 * of device workspace (0 = a default of 64 MiB) for split-K partial sums and
 * tile counters, plus one device status word. Returns LIN_ERR_CUDA when the
 * device cannot be used. *out is NULL on failure. */
LIN_API int lin_create(lin_ctx** out, int device, size_t max_workspace_bytes);

/* Free a context and its workspace (synchronises the device first). NULL is
 * accepted. */
LIN_API int lin_destroy(lin_ctx* ctx);

/* Y = act(X . W^T + bias), chosen kernel per the dispatch table.
 *   M, N, K   : sizes, each >= 0 (M == 0 or N == 0 does nothing; K == 0 gives
 *               Y = act(bias) or act(0)).
 *   X         : M x K row-major; fp32 for FP32/TF32, bf16 for BF16.
 *   W         : N x K row-major (out x in), same element type as X.
 *   bias      : N fp32 values, or NULL for no bias.
 *   Y         : M x N row-major; fp32 for FP32/TF32, bf16 for BF16. Must not
 *               overlap X, W or bias.
 *   epilogue  : lin_epilogue.   precision : lin_precision.
 *   stream    : cudaStream_t (as void*).
 * X and W must be 16-byte aligned and K * element size a multiple of 16
 * (LIN_ERR_ALIGN otherwise); bias 4-byte aligned; Y aligned to its element.
 * One context must not run two calls at the same time (they share the
 * workspace): use one context per stream.
 * Back-to-back calls: with LIN_OPT_EARLY_START at 2 (off by default; see
 * that option for when it is safe), a call whose inputs (X, W, bias) overlap
 * none of the outputs that earlier calls on the same stream may still write is
 * launched as a programmatic dependent of the previous call, reads its inputs
 * before that call's kernel has finished and writes Y only after it. For such a
 * call the built-in plan may also drop its K split (the skinny kernel's cluster split, the
 * tensor-core K split, an FFMA split over a short K), so that consecutive
 * independent calls fill the SMs together; see LIN_OPT_ADAPTIVE_PLANS.
 * lin_plan_query returns the plan of an isolated call. */
LIN_API int lin_forward(lin_ctx* ctx, int M, int N, int K, const void* X, const void* W,
                const float* bias, void* Y, int epilogue, int precision, void* stream);

/* Y = act(X . W^T + bias) + R: the residual add in the GEMM's store
 * ("Optimizing a GPT-2-class transformer on a GPU", Act II, rung 10, where
 * the bias, the activation and the residual add stop being kernels of their
 * own; "Writing a CUDA matmul that catches cuBLAS", "The residual and GELU go
 * the same way"). A
 * transformer block's x = x + proj(h) is this call with R = Y = x.
 *   R : M x N row-major, Y's element type; added after the activation, in
 *       fp32, with one rounding of the sum to Y's type. R may be Y itself (in
 *       place) and must otherwise not overlap Y; NULL is LIN_ERR_ARG (use
 *       lin_forward). Aligned to its element.
 * Everything else as lin_forward (same dispatch, installed plans included). */
LIN_API int lin_forward_residual(lin_ctx* ctx, int M, int N, int K, const void* X, const void* W,
                                 const float* bias, const void* R, void* Y, int epilogue, int precision,
                                 void* stream);

/* LayerNorm fold ("Optimizing a GPT-2-class transformer on a GPU", Act II,
 * rung 10: since LayerNorm's scale and shift reach the output only through
 * the linear layer after it, they can be moved into that layer's weight and
 * bias once, ahead of time, in double). With
 * LN(x) = gamma * xhat + beta, xhat = (x - mean) / sqrt(var + eps):
 *   W LN(x) + bias = W_out xhat + bias_out,
 *   W_out[n][k] = W[n][k] * gamma[k],  bias_out[n] = bias[n] + sum_k W[n][k] * beta[k].
 *   W        : N x K fp32 (device), the layer's weight (out x in).
 *   bias     : N fp32 or NULL (zero).   gamma : K fp32.   beta : K fp32 or NULL (zero).
 *   W_out    : N x K in the storage type of `precision` (fp32 for FP32/TF32,
 *              bf16 for BF16); may be W itself for fp32 storage (in place).
 *   bias_out : N fp32; may be bias itself.
 * Products and the sum (ascending k) in double; each output rounded once to
 * nearest even. Other overlaps: LIN_ERR_ARG; pointers aligned to their
 * elements (LIN_ERR_ALIGN). Asynchronous on `stream`. */
LIN_API int lin_fold_layernorm(lin_ctx* ctx, int N, int K, const float* W, const float* bias, const float* gamma,
                               const float* beta, void* W_out, float* bias_out, int precision, void* stream);

/* Same, with an explicit launch configuration (for tuning and for tests that
 * must reach one kernel). The plan is validated; LIN_ERR_UNSUPPORTED if its
 * kernel cannot run the shape, LIN_ERR_WORKSPACE if it needs more workspace
 * than the context holds. */
LIN_API int lin_forward_plan(lin_ctx* ctx, const lin_plan* plan, int M, int N, int K, const void* X,
                     const void* W, const float* bias, void* Y, int epilogue, int precision,
                     void* stream);

/* The dispatch table, on the host only (no GPU needed): the plan lin_forward
 * would use for this shape on a device with `sm_count` SMs and a workspace of
 * `workspace_bytes`. Returns LIN_ERR_ARG for invalid sizes or enums. */
LIN_API int lin_plan_query(int sm_count, int M, int N, int K, int precision, int epilogue,
                   size_t workspace_bytes, lin_plan* out);

/* Check a plan against a shape on the host (no GPU needed): LIN_OK when
 * lin_forward_plan would accept it in a context with `workspace_bytes` of
 * workspace, else the status it would return (LIN_ERR_UNSUPPORTED: the kernel
 * cannot run this shape / precision with this grid; LIN_ERR_WORKSPACE; or
 * LIN_ERR_ARG for a NULL plan, negative sizes or an unknown precision).
 * Limits that depend on the device (stream-K CTAs at most one per SM) are
 * checked when the call is launched. */
LIN_API int lin_plan_check(const lin_plan* plan, int M, int N, int K, int precision, size_t workspace_bytes);

/* Fill *out with the default plan of a kernel family for a shape (host only),
 * for sweeps: kernel = lin_kernel, variant = tile configuration, splits = 0
 * lets the table choose the split. For LIN_KERNEL_TC, splits counts CTAs
 * instead: >= 0 CTAs walking whole tiles (0 = one per SM); -1 stream-K with
 * one CTA per SM; -c (c >= 2) stream-K with c CTAs (single-CTA variants, at
 * least one tile per CTA; the plan's splits is then 2 and it needs workspace
 * for one 128 x BN fp32 slot per CTA). For LIN_KERNEL_GEMV, splits is the
 * CTA count (0 = as many as fit at once). Returns LIN_ERR_UNSUPPORTED when the
 * kernel cannot run the shape. */
LIN_API int lin_plan_make(int sm_count, int kernel, int variant, int splits, int M, int N, int K,
                  int precision, lin_plan* out);

/* ---- Backward (training) ----
 * The backward pass of the same layer ("Writing a CUDA matmul that catches
 * cuBLAS", the backward transpose cases: dX = dY W^T and dW = dY^T X for a
 * weight stored in x out; here W is stored out x in):
 *   dZ = dY * act'(Z)           (lin_gelu_backward, or dZ = dY for no activation)
 *   dX = dZ . W      (M x K)    (lin_backward_data)
 *   dW = dZ^T . X    (N x K)    (lin_backward_weight, with db = sum over rows of dZ)
 * Operands are in the precision's input type and results in its output type
 * (bf16 for LIN_PREC_BF16, fp32 otherwise; db is always fp32). BF16 runs on
 * the tensor cores with the transposes folded into the operands' shared-memory
 * layout (nothing is transposed in memory); FP32 and TF32 run exact fp32
 * FFMAs. Results are bitwise repeatable. Calls are asynchronous on `stream`
 * and follow lin_forward's early-start rules. */

/* dX (M x K) = dZ (M x N) . W (N x K), all row-major. dZ, W and dX 16-byte
 * aligned; K * element size a multiple of 16; for BF16 also N * 2 (the rows
 * of dZ are read by TMA). dX must not overlap dZ or W. N == 0 gives zeros. */
LIN_API int lin_backward_data(lin_ctx* ctx, int M, int N, int K, const void* dZ, const void* W, void* dX,
                              int precision, void* stream);

/* dW (N x K) = dZ^T . X (dZ: M x N, X: M x K), and db[n] = sum_m dZ[m][n]
 * in fp32 when db is not NULL (two passes over fixed row chunks, in order;
 * uses the context workspace: LIN_ERR_WORKSPACE when it is too small). The
 * alignment rules of lin_backward_data apply to dZ, X and dW; db is 4-byte
 * aligned. M == 0 gives zeros. */
LIN_API int lin_backward_weight(lin_ctx* ctx, int M, int N, int K, const void* dZ, const void* X, void* dW,
                                float* db, int precision, void* stream);

/* dZ = dY * gelu'(Z) elementwise over `count` values, Z the pre-activation
 * (act's input) of the forward; the slope of the tanh form used by the
 * forward. dZ may be dY (in place) but not Z. */
LIN_API int lin_gelu_backward(lin_ctx* ctx, long long count, const void* dY, const void* Z, void* dZ,
                              int precision, void* stream);

/* dX carried through the previous layer's GELU in the same pass: when this
 * layer's input was X = gelu(Zp) (Zp the previous layer's pre-activation),
 *   dZp = (dZ . W) * gelu'(Zp)      (M x K),
 * i.e. lin_backward_data followed by lin_gelu_backward, with the slope
 * applied in the GEMM's store instead of a second pass over M x K.
 *   Zp : M x K row-major in the precision's storage type; dZp may be Zp
 *        itself (in place) and must otherwise not overlap it.
 * Everything else as lin_backward_data. */
LIN_API int lin_backward_data_gelu(lin_ctx* ctx, int M, int N, int K, const void* dZ, const void* W,
                                   const void* Zp, void* dZp, int precision, void* stream);

/* Measured dispatch ("Optimizing a GPT-2-class transformer on a GPU", Act II:
 * route each shape to its measured winner). Install `plan` as the context's
 * choice for lin_forward calls with exactly these sizes, precision and
 * epilogue (checked like lin_forward_plan; LIN_ERR_UNSUPPORTED or
 * LIN_ERR_WORKSPACE when it cannot run the shape in this context; a refused
 * plan leaves any earlier entry in place). A NULL plan removes the entry
 * (LIN_OK whether or not there was one). The plan is copied; entries are
 * guarded by a lock, so installing while another thread calls lin_forward is
 * safe. lin_forward consults these entries before the
 * built-in table and runs an installed plan as given (no adaptive change for
 * back-to-back calls). The Python package's autotuner measures candidates and
 * installs winners through this call. */
LIN_API int lin_set_plan_override(lin_ctx* ctx, int M, int N, int K, int precision, int epilogue,
                                  const lin_plan* plan);

/* Remove every installed plan of the context. */
LIN_API int lin_clear_plan_overrides(lin_ctx* ctx);

/* Synchronise `stream`, read and clear the context's device status word.
 * Returns LIN_ERR_DEVICE_TIMEOUT if any kernel since the last check gave up
 * a bounded wait (its output is then incomplete), LIN_ERR_CUDA on a CUDA
 * error, LIN_OK otherwise. */
LIN_API int lin_check_device(lin_ctx* ctx, void* stream);

/* Context options (lin_set_option).
 * LIN_OPT_PROGRAMMATIC_LAUNCH (default 1): calls are launched as programmatic
 *   dependents of the previous kernel on their stream: a call's CTAs may start
 *   on SMs as the previous kernel's CTAs leave them, set up (barriers, tensor
 *   memory, descriptors) and ask the L2 cache to fetch their first operand
 *   tiles, and then wait (griddepcontrol.wait) until that kernel has finished
 *   and its writes are visible before they read anything. An L2 prefetch
 *   returns no data to the kernel and L2 is where all writes meet, so this
 *   changes no result whatever the previous kernel writes. 0 = plain stream
 *   order (the CTAs start only after all earlier work has finished).
 * LIN_OPT_EARLY_START (default 0): which operands may be READ before the
 *   previous kernel on the stream has finished (needs programmatic launch).
 *   0: none; every call reads its operands only after all earlier work on the
 *      stream, like any stream-ordered library.
 *   1: W and bias may be read before that kernel has finished. X is read, and
 *      Y written, only after it.
 *   2: as 1, and X may be read early too.
 *   The library only sees its own calls: it drops the early reads of W / bias
 *   (and X) by itself when they overlap the previous library call's output on
 *   that stream, and a call whose early reads would touch what an older call may
 *   still be writing is launched in plain stream order. It cannot see other work. Use 1 only when no other work on
 *   the stream writes the next call's W or bias between two library calls (an
 *   optimizer step does), and 2 only when nothing but library calls write its X
 *   either (a framework kernel that produces X, such as a layernorm, does).
 *   With 2, a call that overlaps an independent predecessor may also narrow its
 *   plan (LIN_OPT_ADAPTIVE_PLANS).
 * LIN_OPT_ADAPTIVE_PLANS (default 1): a call that overlaps an independent
 *   predecessor on its stream (early start level 2) may drop
 *   the K split of its built-in plan: the neighbouring call then fills the SMs
 *   the split would. A split changes the order of the fp32 sums, so with this
 *   option on, the last bits of a result can depend on the call before it on
 *   the stream (never beyond the precision's tolerance). 0 = the plan of a
 *   call depends only on its sizes, precision and epilogue, so identical
 *   inputs give identical bits whatever ran before. Installed plans
 *   (lin_set_plan_override) and lin_forward_plan are never adapted. */
typedef enum {
    LIN_OPT_EARLY_START = 1,
    LIN_OPT_ADAPTIVE_PLANS = 2,
    LIN_OPT_PROGRAMMATIC_LAUNCH = 3
} lin_option;

/* The plan of the last call launched through this context (host value, no
 * GPU call): lin_forward may refine the dispatch table's plan for a call that
 * overlaps its predecessor. LIN_ERR_ARG if ctx or out is NULL; a context with
 * no call yet reports LIN_KERNEL_NONE. */
LIN_API int lin_ctx_last_plan(const lin_ctx* ctx, lin_plan* out);

/* Set a context option. LIN_ERR_ARG for an unknown option or value. */
LIN_API int lin_set_option(lin_ctx* ctx, int option, long long value);

/* SM count and device ordinal of a context (host values, no GPU call). */
LIN_API int lin_ctx_info(const lin_ctx* ctx, int* device, int* sm_count, size_t* workspace_bytes);

/* Throughput probe of the exact-fp32 FMA pipe (the roofline of the FFMA
 * kernels; the pages derive their fp32 peak from unit counts and the clock,
 * "Writing a CUDA matmul that catches cuBLAS", opening section). Launches, on
 * `stream`, the context's SM count x 4 CTAs of 256 threads, each thread
 * running 8 independent fmaf chains for iters x 16 steps, and nothing else;
 * *flops (if not NULL) receives the FLOPs launched (2 per fmaf). The caller
 * times the launch (CUDA events on `stream`). `out`: a device float the
 * kernel writes only in a case that cannot occur, which keeps the chains
 * live. Returns LIN_ERR_ARG for iters < 1 or a NULL out. */
LIN_API int lin_probe_ffma(lin_ctx* ctx, int iters, float* out, double* flops, void* stream);

/* Static message for a status code. */
LIN_API const char* lin_strerror(int status);

/* LIN_ABI_VERSION of the loaded library. */
LIN_API int lin_abi_version(void);

/* Kernel timeline (measurement aid; "One multiply, one RTX 5090, eight
 * kernels", "Where the time goes", times parts of a kernel separately to see
 * where its time goes). In the separate timeline build of this library
 * (compiled with -DLIN_TIMELINE), the tcgen05 kernel and the skinny kernel
 * record %globaltimer nanoseconds at fixed points of each CTA's schedule into
 * device arrays of LIN_TIMELINE_CTAS x LIN_TIMELINE_SLOTS unsigned 64-bit
 * values (0 = point not reached):
 *   kernel LIN_KERNEL_TC, record = blockIdx.x: [0] set up, [1] producer past
 *     its dependency wait, [2] teardown; for work item j < 32: [8 + 4j] MMAs
 *     start (accumulator free), [8 + 4j + 1] last MMA and commit issued,
 *     [8 + 4j + 2] epilogue warp 2 sees the accumulator, [8 + 4j + 3]
 *     epilogue warp 2 done, [136 + j] epilogue warp 9 done;
 *   kernel LIN_KERNEL_SKINNY, records in the order CTAs start (consecutive
 *     launches follow one another): [0] set up, [1] producer past its
 *     dependency wait, [2] MMAs complete, [3] done, [16 + i] stage i landed;
 *   kernel LIN_TIMELINE_ATTENTION (lin_attention_forward), record =
 *     blockIdx.x: [0] set up, [1] producer past its dependency wait, [2]
 *     teardown; for the CTA's work item n < 16, at 8 + 10n + k: k = 0 Q copy
 *     issued, 1 first K/V copy issued, 2 MMA warp saw the first K/V land, 3
 *     first S MMAs committed, 4 softmax warp 2 saw the first S, 5 it released
 *     the last P, 6 last P.V MMAs committed, 7 softmax warp 2 saw the last
 *     P.V, 8 softmax warp 2 stored its rows, 9 softmax warp 9 stored its rows.
 * lin_timeline copies the first `bytes` of that kernel's array to `host_dst`
 * (synchronously; both NULL/0 to skip the copy), then zeroes the array (and
 * the skinny record counter) if `clear` is non-zero. A stamped launch is
 * identical to the library build's in everything else. Returns
 * LIN_ERR_UNSUPPORTED in the library build, LIN_ERR_ARG for another kernel
 * id or a NULL/non-zero mismatch of host_dst and bytes. */
#define LIN_TIMELINE_ATTENTION 16
#define LIN_TIMELINE_CTAS 1024
#define LIN_TIMELINE_SLOTS 192
LIN_API int lin_timeline(int kernel, void* host_dst, size_t bytes, int clear);

/* Size of the fixed device array behind lin_forward_fp32_static. */
#define LIN_STATIC_SCRATCH_BYTES (8u << 20)

/* The pages have no counterpart to this entry point; it exists for callers
 * that cannot allocate device memory when they run the layer, for example:
 * - runtimes that reserve all device memory for their own pool at start-up
 *   and treat any other allocation as a failure;
 * - latency-critical paths where an allocation could block on the device or
 *   fail under memory pressure;
 * - plug-ins that are handed device pointers but no allocator.
 *
 * Y = act(X . W^T + bias) in fp32 on the CURRENT device, with the same
 * kernel and split-K choice as lin_forward(..., LIN_PREC_FP32, ...) (the FFMA
 * kernel, or the GEMV for M <= 8, which needs no scratch), but with no
 * context. It calls no cudaMalloc or cudaFree: the split-K counters and
 * partial sums live in one fixed array of LIN_STATIC_SCRATCH_BYTES (8 MiB),
 * a static device variable of this library that every GPU which loads the
 * library holds until the process exits. Arguments, layouts and alignment
 * rules are those of lin_forward; X, W, bias and Y are caller-owned device
 * pointers.
 *
 * Limits and caveats:
 * - The split is the one lin_forward would take, so the result is bitwise
 *   that of lin_forward. A shape whose split needs more scratch than the
 *   array holds returns LIN_ERR_WORKSPACE (nothing is launched); the split
 *   fills the SMs, so its scratch grows with the SM count (about 5 MB on 152
 *   SMs) and not with the shape.
 * - The first call on a device (and the first after that device's context
 *   was created anew) looks up the array's device address; make that first
 *   call before any stream capture.
 * - Every call shares the one array, and the array keeps the last call's
 *   contents. The call zeroes the counters it uses on `stream` before its
 *   kernel.
 * - Calls whose kernels overlap on the GPU (other streams, or other threads
 *   without ordering) race on the array: order them on one stream. */
LIN_API int lin_forward_fp32_static(int M, int N, int K, const float* X, const float* W,
                                    const float* bias, float* Y, int epilogue, void* stream);

/* Fused self-attention forward, the step between the qkv projection and the
 * output projection ("Writing a CUDA matmul that catches cuBLAS", section
 * "Fusing attention: the score matrix never exists": q, k and v are read
 * straight from the projection's output, a running row max and sum replace
 * the stored score matrix, and causality is the loop bound). For sequence b,
 * head h and query token i:
 *   s_ij  = (q_i . k_j) * scale over the visible keys j (j <= i when causal,
 *           all j < T otherwise),
 *   out[b*T + i][h*64 + d] = sum_j exp(s_ij - m_i) v_j[d] / l_i,
 *   m_i = max_j s_ij, l_i = sum_j exp(s_ij - m_i),
 *   lse[(b*H + h)*T + i] = m_i + log(l_i)            (when lse is not NULL).
 *   qkv : DEVICE, (B*T) x 3C bf16 row-major, C = H*D; token t of sequence b is
 *         row b*T + t, holding q, k, v at column offsets 0, C, 2C and head h
 *         at h*D within each (the layout of the qkv linear layer's output).
 *   out : DEVICE, (B*T) x C bf16 row-major (the output projection's input);
 *         must not overlap qkv or lse.
 *   lse : DEVICE fp32 B x H x T, or NULL (the softmax statistics a backward
 *         pass rebuilds the probabilities from).
 *   D   : head width; 64 only (LIN_ERR_UNSUPPORTED otherwise).
 *   causal: 1 (decoder attention) or 0.
 *   scale: softmax scale > 0; 0 selects 1/sqrt(D).
 * Arithmetic: bf16 q, k products accumulated in fp32 on the tensor cores,
 * softmax in fp32 (base-2 exponent of the scaled scores, hardware ex2),
 * probabilities rounded to bf16 for the product with v (fp32 accumulation),
 * output rounded to nearest-even bf16. qkv and out must be 16-byte aligned
 * (LIN_ERR_ALIGN), lse 4-byte aligned; B*T < 2^31. B, T or H == 0: nothing to
 * do. Asynchronous on `stream`; launched as a programmatic dependent of the
 * previous kernel (when LIN_OPT_PROGRAMMATIC_LAUNCH is on) but reads qkv and
 * writes out / lse only after that kernel has finished (before that it only
 * asks the L2 cache for its first tiles, which returns no data to the
 * kernel). LIN_ERR_UNSUPPORTED also when the library was compiled so that
 * the kernel holds fewer registers a thread than its warp-specialised
 * register split needs (it then launches nothing). */
LIN_API int lin_attention_forward(lin_ctx* ctx, int B, int T, int H, int D, const void* qkv, void* out, float* lse,
                                  int causal, float scale, void* stream);

/* Backward pass of lin_attention_forward, in its layouts: the probabilities are
 * rebuilt from the forward's lse, so nothing of size T x T reaches memory.
 *   s_ij = (q_i . k_j) * scale,  p_ij = exp(s_ij - lse_i) (0 where masked),
 *   delta_i = dout_i . out_i,    dp_ij = dout_i . v_j,
 *   ds_ij = p_ij (dp_ij - delta_i),
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,
 *   dv_j = sum_i p_ij dout_i.
 *   qkv  : (B*T) x 3C bf16, the forward's input.
 *   out  : (B*T) x C bf16, the forward's output.   lse : B x H x T fp32, its lse
 *          (-inf marks a query that sees no key: it contributes nothing).
 *   dout : (B*T) x C bf16, the gradient of out.
 *   dqkv : (B*T) x 3C bf16, written whole; must not overlap the inputs.
 *   B, T, H, D, causal, scale as in the forward; a scale below 2^-100 or above
 *   2^100 is refused (LIN_ERR_ARG): lse / scale has to be finite in fp32.
 * Arithmetic: bf16 products accumulated in fp32 on the tensor cores; p and ds
 * in fp32, each rounded once to bf16 for the products that take it; sums in
 * fp32, each gradient rounded once. The sums' order is fixed by the sizes, the
 * SM count and the workspace, so results repeat bit for bit. Uses the context
 * workspace (up to about 256 bytes a head and token per partial sum of dq;
 * heads that do not fit at once go in several launches; LIN_ERR_WORKSPACE
 * when not even one head fits: the default workspace holds one of 246000
 * tokens). Key blocks add to a partial sum of dq in turn; a larger workspace
 * gives more partial sums, and less waiting, up to one for every key block of a
 * head that runs at the same time. A wait is only for a block that runs already,
 * whatever SMs other streams hold. A NaN or infinity in a token's row of qkv may
 * reach the gradients of all tokens in its block of 128 of the sequence, also
 * across the causal mask (0 times NaN in the products); one in dout their dk and
 * dv. out of a query that sees no key is not used. qkv, out, dout and dqkv must
 * be 16-byte aligned (LIN_ERR_ALIGN), lse 4-byte aligned. Asynchronous on
 * `stream`; reads and writes only after the previous kernel on the stream has
 * finished. */
LIN_API int lin_attention_backward(lin_ctx* ctx, int B, int T, int H, int D, const void* qkv, const void* out,
                                   const float* lse, const void* dout, void* dqkv, int causal, float scale,
                                   void* stream);

/* ---- Operators on the LM head's logits ----
 * R rows of V logits, row r at logits + r * ld elements (ld >= V: a padded
 * vocabulary's columns are neither read nor written), z_rj below. Element
 * types are named by lin_dtype. tau > 0 is a temperature: probabilities are
 * softmax(z / tau). Maxima, sums and statistics are held in fp32, the
 * differences from a row's maximum are formed before they are scaled (but see
 * lin_distill_backward, which is given lse), and results do not depend on the
 * order in which blocks run (identical inputs give identical bits). A NaN or
 * +inf among a row's logits makes that row's results NaN; -inf is a token that
 * cannot occur (probability 0).
 * Pointers are DEVICE pointers aligned to their elements (LIN_ERR_ALIGN).
 * LIN_ERR_ARG: a NULL that is not allowed, a negative size, ld < V, an
 * unknown type, tau not positive and finite (or so small that log2(e) / tau is
 * not finite in fp32), or an output that overlaps an input or another output
 * (except as said). LIN_ERR_UNSUPPORTED: V > 2^30 or
 * R > 2^27. R == 0 does nothing; V == 0 with rows is LIN_ERR_ARG. No
 * workspace. Launched like lin_forward, as a programmatic dependent that reads
 * and writes only after the previous kernel on the stream has finished. */
typedef enum {
    LIN_TYPE_FP32 = 0,
    LIN_TYPE_BF16 = 1,
    LIN_TYPE_INT32 = 2,
    LIN_TYPE_INT64 = 3
} lin_dtype;

/* Log probabilities of given tokens, with the distribution's entropy and its
 * top alternatives:
 *   lse_r     = log sum_j exp(z_rj / tau)
 *   logprob_r = z_r,token_r / tau - lse_r
 *   entropy_r = - sum_j p_rj log p_rj          (nats, p = exp(z / tau - lse))
 *   top_ids[r * top + i]     : the i-th largest logit's index; equal values
 *                              (zeros of either sign are equal) by the lowest
 *                              index, NaN ranked with -inf
 *   top_logprob[r * top + i] : its log probability
 *   logits_type : LIN_TYPE_FP32 or LIN_TYPE_BF16.
 *   tokens : R of LIN_TYPE_INT32 or LIN_TYPE_INT64 (tokens_type), or NULL
 *            (with logprob NULL). A negative token gives logprob 0 (no token
 *            here), one >= V gives NaN.
 *   logprob, entropy, lse : R fp32 each; entropy and lse may be NULL, logprob
 *            if and only if tokens is.
 *   top    : 0 to 64, at most V; with 0 both top outputs are ignored.
 * A row whose logits are all -inf: lse and log probabilities -inf, entropy 0. */
LIN_API int lin_token_logprobs(lin_ctx* ctx, int R, int V, const void* logits, long long ld, int logits_type,
                               const void* tokens, int tokens_type, float tau, int top, float* logprob,
                               float* entropy, float* lse, float* top_logprob, int* top_ids, void* stream);

/* Distillation towards a teacher's top logits. Row r has K entries: token
 * ids[r * K + i] with the teacher's logit (or log probability: a constant
 * added to a row changes nothing) teacher[r * K + i]. Entries with a negative
 * id are padding. With
 *   q = softmax(teacher / tau) over the row's entries,
 *   p = softmax(z / tau) over the row's V logits,
 *   loss_r = tau^2 sum_i q_i (log q_i - log p_id(i)),
 *   dz_rj  = g_r tau (p_rj - sum of the q_i with id(i) = j),
 * g_r being the gradient that reaches loss_r. Entries may repeat a token. A
 * row without entries (or whose teacher logits are all -inf) has loss 0 and
 * gradient 0, and so has the gradient where g_r = 0, whatever the logits are.
 * An id >= V makes its row's loss and gradient NaN. Logits that are all -inf
 * leave p undefined: NaN, in a row with entries (the gradient: and weight).
 *   ids     : R x K, LIN_TYPE_INT32 or LIN_TYPE_INT64 (ids_type), 0 <= K <= 256.
 *   teacher : R x K, LIN_TYPE_FP32 or LIN_TYPE_BF16 (teacher_type). */

/* loss (R fp32) and, if not NULL, lse (R fp32, log sum exp(z / tau): what
 * lin_distill_backward needs). */
LIN_API int lin_distill_forward(lin_ctx* ctx, int R, int V, int K, const void* logits, long long ld, int logits_type,
                                const void* ids, int ids_type, const void* teacher, int teacher_type, float tau,
                                float* loss, float* lse, void* stream);

/* dlogits (R rows of V, ldd apart, in the logits' type, one rounding) from the
 * forward's lse of the same logits and tau, and grad_loss (R fp32: g). Where
 * |lse| is at most 512 (bf16 logits) or 64 (fp32), p = exp(z / tau - lse): the
 * rounding of lse moves the row's p by up to 2^-23 |lse| relative, 2^-14 and
 * 2^-17 at most. Past that lse has lost the digits that p needs, and the row's
 * maximum and sum are computed again, at the cost of another read of the row.
 * dlogits may be the logits themselves (in place, with ldd == ld). Fast when dlogits and logits start
 * at the same offset within 16 bytes and (ld - ldd) * element size is a
 * multiple of 16; right for any. */
LIN_API int lin_distill_backward(lin_ctx* ctx, int R, int V, int K, const void* logits, long long ld, int logits_type,
                                 const void* ids, int ids_type, const void* teacher, int teacher_type, float tau,
                                 const float* lse, const float* grad_loss, void* dlogits, long long ldd,
                                 void* stream);

/* Both in one pass over the logits, for a loss whose weights are known before
 * it is computed: weight (R fp32, NULL = 1) is g, loss (not weighted) may be
 * NULL. dlogits as above. */
LIN_API int lin_distill_forward_backward(lin_ctx* ctx, int R, int V, int K, const void* logits, long long ld,
                                         int logits_type, const void* ids, int ids_type, const void* teacher,
                                         int teacher_type, float tau, const float* weight, float* loss,
                                         void* dlogits, long long ldd, void* stream);

/* ---- Rotary positions, and serving from a paged cache ---- */

/* Rotary positions of (part of) a head: pair i < dim / 2 of a token at position p
 * turns by the angle p f_i. Pairs are elements (i, i + dim / 2) or (2i, 2i + 1) of
 * the head's first dim elements; the rest of the head does not rotate. */
typedef enum {
    LIN_ROTARY_HALF = 0,         /* element i with i + dim / 2 */
    LIN_ROTARY_INTERLEAVED = 1   /* element 2i with 2i + 1 */
} lin_rotary_layout;

typedef struct {
    int dim;                           /* elements that rotate: even, 0 to the head's width */
    int layout;                        /* lin_rotary_layout */
    float scale;                       /* factor on the rotated elements (1 = none): finite */
    const unsigned long long* turns;   /* DEVICE, dim / 2: f_i / (2 pi) mod 1 in units of 2^-64 */
} lin_rotary;

/* turns[i] (host) from frequencies[i] (host, radians per position, finite): the
 * fixed-point form that lin_rotary holds on the device, off by at most 0.6 of its unit
 * for frequencies up to 2^40 in size. The kernels multiply it by the position modulo 2^64, which
 * is p times the entry modulo one turn, without rounding, for any 64-bit position p: the angle
 * is off by at most |p| 2^-62 radians. */
LIN_API int lin_rotary_turns(const double* frequencies, int n, unsigned long long* turns);

/* y = x with every head rotated by its row's position. Row n, head h at
 * x + n * ldx + h * D and y + n * ldy + h * D (elements; ldx, ldy >= H * D).
 *   x, y      : LIN_TYPE_FP32 or LIN_TYPE_BF16 (type), DEVICE. y may be x (with ldy == ldx);
 *               otherwise no row's heads of y may lie over x's. Rows of equal stride may
 *               interleave (column ranges of one matrix).
 *   positions : N of LIN_TYPE_INT32 or LIN_TYPE_INT64 (positions_type), any value.
 *   D         : 1 to 1024. H up to 65535 (more where heads are narrow), H * D up to 2^27, ldx and
 *               ldy up to 2^30; LIN_ERR_UNSUPPORTED beyond.
 * Angles, cosines and products in fp32 (from the exact product of position and table entry), one rounding to
 * the type. A NaN or infinity reaches its own pair only. Fast when addresses and
 * strides are multiples of 16 bytes and the pairs fill them; right for any. No workspace. Reads and writes only
 * after the previous kernel on the stream has finished. */
LIN_API int lin_rotary_forward(lin_ctx* ctx, int N, int H, int D, const void* x, long long ldx, void* y, long long ldy,
                               int type, const void* positions, int positions_type, const lin_rotary* rotary,
                               void* stream);

/* Its gradient: dx from dy, the rotation by the negative angle (and the same scale). */
LIN_API int lin_rotary_backward(lin_ctx* ctx, int N, int H, int D, const void* dy, long long lddy, void* dx,
                                long long lddx, int type, const void* positions, int positions_type,
                                const lin_rotary* rotary, void* stream);

/* A paged cache of keys and values, bf16. Slot s of head h of page g starts at element
 * g * page_stride + h * head_stride + s * token_stride of k, and of v, head_dim
 * consecutive elements. */
typedef struct {
    void* k;                  /* DEVICE, 16-byte aligned */
    void* v;
    int pages;                /* at least 1 */
    int page_size;            /* tokens a page holds: a power of two, 8 to 4096 */
    int heads;                /* key (and value) heads */
    int head_dim;             /* 64 or 128 */
    long long page_stride;    /* elements; multiples of 8 (16 bytes), each head's row of a slot apart */
    long long head_stride;
    long long token_stride;
} lin_kv_cache;

/* A batch of sequences whose new tokens are rows of packed matrices, one sequence
 * after the other. The arrays are on the DEVICE and are read when the kernels run, so a captured graph
 * follows them. */
typedef struct {
    int sequences;            /* at most 2^30, for attention 2^24 */
    int tokens;               /* rows of the packed matrices; for attention at most 2^28 */
    const int* q_start;       /* sequences + 1: sequence b's new tokens are rows q_start[b] to q_start[b + 1] - 1; ascending */
    const int* kv_len;        /* sequences: tokens that sequence b has in the cache, the new ones included */
    const int* block_table;   /* sequence b's tokens i * page_size .. lie in page block_table[b * table_stride + i] */
    int table_pages;          /* entries of a sequence that may be read: at most 2^30 / page_size */
    long long table_stride;   /* >= table_pages */
} lin_kv_batch;

/* Write the new tokens' keys and values into the cache. Row n, the i-th new token of
 * sequence b (i = n - q_start[b]), goes to the place of position
 *   p = kv_len[b] - (q_start[b + 1] - q_start[b]) + i.
 * With a rotary plan (not NULL) keys are rotated on the way, by p or by
 * positions[n], and queries too: q_out = q rotated.
 *   q, q_out : tokens x H heads of head_dim, bf16, rows ldq and ldqo elements apart; q_out
 *              may be q (ldqo == ldq). Both NULL (H 0): keys and values only. Without a
 *              rotary plan they must be.
 *   k, v     : tokens x cache->heads heads of head_dim, bf16, rows ldk and ldv apart.
 *              H * head_dim up to 2^27, all row strides up to 2^30 (LIN_ERR_UNSUPPORTED beyond).
 *   positions: NULL, or one per row (LIN_TYPE_INT32 or LIN_TYPE_INT64), used for the rotation only.
 * Rows of no sequence are left out: nothing is written for them. A token whose
 * position lies outside the table, or whose table entry is not a page of the cache, is not
 * stored (its q_out is written). Two tokens with the same place: what lies there
 * afterwards is a mixture of both (16 bytes of the one or the other). q_start has to ascend; whatever the arrays hold, nothing outside the
 * operands is read or written. Columns of one matrix (a qkv
 * projection's output) are fine as q, k, v and q_out; nothing else may overlap an output. */
LIN_API int lin_cache_append(lin_ctx* ctx, const lin_kv_cache* cache, const lin_kv_batch* batch, int H, const void* q,
                             long long ldq, void* q_out, long long ldqo, const void* k, long long ldk, const void* v,
                             long long ldv, const void* positions, int positions_type, const lin_rotary* rotary,
                             void* stream);

/* Attention of the batch's new tokens over the paged cache (which holds their own keys
 * and values already, see lin_cache_append). Row n, the i-th of the n_b new tokens of sequence b, at
 * position p = kv_len[b] - n_b + i, query head h, reading key head g = h / (H / heads):
 *   s_j = (q_nh . K_bgj) scale   for the keys j that it sees: j <= p when causal, else all
 *         j < kv_len[b]           (a cross attention's encoder states)
 *   out[n * ldo + h * head_dim ..] = sum_j exp(s_j - m) V_bgj / sum_j exp(s_j - m),  m = max_j s_j
 *   lse[n * H + h] = log sum_j exp(s_j)            (when lse is not NULL)
 * A row that sees no key (an empty sequence, or one that holds fewer keys than it has new tokens)
 * has out 0 and lse -inf; so has one whose scores are all -inf. Rows of no sequence are
 * left as they were. kv_len is taken as 0 below 0, and up to table_pages * page_size; what lies on a page that is
 * none of the cache's reads as zeros. Whatever the arrays hold, nothing outside the
 * operands is read or written.
 *   q, out : tokens x H heads of head_dim, bf16, 16-byte aligned, rows ldq and ldo apart (multiples of 8, up to 2^30).
 *   H      : a multiple of cache->heads, at most 128 times as many, and at most 65535.
 *   scale  : 2^-100 to 2^100; 0 selects 1/sqrt(head_dim).
 *   max_new: about how many new tokens the longest sequence has (0: as many as the average); it picks the
 *            kernel, and any value gives right results. The average of a long prompt among single tokens can pick the one
 *            for few tokens, which reads the prompt's keys once per 16 rows (63 single tokens and a prompt of 900, 12 heads
 *            of 64: 161 us instead of 138).
 *   workspace: DEVICE, 16-byte aligned, of lin_paged_attention_workspace's size for the same max_new: parts of
 *            items that several blocks share. NULL: the context's own (LIN_ERR_WORKSPACE when it is too
 *            small); calls that may run at the same time, captured ones included, need one each, and so do calls that
 *            several threads make at once, on one stream too (a call enqueues two kernels, one right after the other).
 * Arithmetic: bf16 products summed in fp32, softmax in fp32, probabilities rounded to bf16 for the product with V,
 * one rounding of the output. Sums are split by the lengths and the device alone: results repeat bit
 * for bit. A NaN or infinity in a key or value that some row of a sequence's new tokens sees may
 * reach all of that sequence's rows; slots that no row sees may hold anything. Reads and writes
 * only after the previous kernel on the stream has finished. Waits inside the kernels end after about a second
 * (lin_check_device then reports it): none lasts nearly as long, unless one block has more than 10^8 keys of one
 * head and tile to itself. */
LIN_API int lin_paged_attention(lin_ctx* ctx, const lin_kv_cache* cache, const lin_kv_batch* batch, int H, const void* q,
                                long long ldq, void* out, long long ldo, float* lse, int causal, float scale,
                                int max_new, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that such a call needs (host only; batch may be NULL when max_new is given). */
LIN_API int lin_paged_attention_workspace(const lin_ctx* ctx, const lin_kv_cache* cache, const lin_kv_batch* batch,
                                          int H, int max_new, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* LIN_H */
