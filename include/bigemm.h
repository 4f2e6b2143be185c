/*
 * bigemm.h -- C ABI of the broadcast / implicit-GEMM convolution library for
 * one NVIDIA GB300 GPU (sm_103a).
 *
 * Operations (the sources that define them):
 *
 *  conv2d   NCHW 2-D convolution, as computed by topi.nn.conv2d_nchw in
 *           "Tuning High Performance Convolution on NVIDIA GPUs" (TVM v0.5
 *           autotvm tutorial), Step 1 (compute declaration, inlined padding):
 *             out[n,f,y,x] = sum_{rc<CI/groups, ry<KH, rx<KW}
 *                              pad(data)[n, g*CI/groups + rc, y*s+ry, x*s+rx]
 *                              * kernel[f, rc, ry, rx]
 *           with g = f / (CO/groups), pad() = `padding` zeros on every side,
 *           dilation 1, Ho = floor((H + 2*padding - KH)/stride) + 1 (Wo alike).
 *           The tutorial's template signature (N, H, W, CO, CI, KH, KW, stride,
 *           padding) gives the argument order of conv2d_nchw_plan.
 *  epilogue The per-channel broadcast of "[CINN] Add the TileBroadcastTactic
 *           for NCHW broadcast" (PaddlePaddle PR 70092), Introduction and
 *           Example, applied to the conv sum before the store:
 *             out[n,f,y,x] = op(acc[n,f,y,x] + bias[f]).
 *  bcast    The same PR's broadcast on its own:
 *             out[n,c,h,w] = op(var[c]),  [1,C,1,1] => [N,C,H,W],
 *           with the channel value computed once per channel block.
 *  plan     A timed choice among a few kernel tilings per shape, the analogue
 *           of the tutorial's Step 2 (tuning with a measure option of repeated
 *           timed runs, keeping the best record for the workload).
 *
 * Conventions for every entry point:
 *  * Tensors are contiguous and in the caller's DEVICE memory (pointers from
 *    cudaMalloc / torch): data [N,CI,H,W] (NCHW), kernel [CO,CI/groups,KH,KW]
 *    (OIHW), bias/var [C] fp32, out [N,CO,Ho,Wo] (NCHW).  The caller owns
 *    them; the library never frees or retains them past the call.
 *  * `stream` is a cudaStream_t (NULL = the legacy default stream).  Runs are
 *    asynchronous on it; only conv2d_nchw_plan with search=1 synchronises.
 *  * Every function returns a bigemm_status; none aborts or exits.  Shapes,
 *    dtypes and alignment are checked before any launch.  A launch failure
 *    returns BIGEMM_ERR_CUDA.  Kernels bound every wait; a wait that runs out
 *    sets a sticky device flag read by bigemm_last_device_error().
 *  * Plans own their scratch memory (packed operands, split-K partial sums),
 *    allocated by conv2d_nchw_plan and freed by conv2d_nchw_plan_destroy.
 *    Two runs of one plan must not overlap on the GPU (they share scratch).
 */
#ifndef BIGEMM_H
#define BIGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* MXF8 (the transformer-layer operators below alone): e4m3 elements with one
 * power-of-two scale (E8M0) per 32 elements of a row, kept apart. */
typedef enum { BIGEMM_F32 = 0, BIGEMM_F16 = 1, BIGEMM_BF16 = 2, BIGEMM_MXF8 = 3 } bigemm_dtype;

/* Fused epilogue: out = acc (NONE), acc + bias[f] (BIAS),
 * exp(acc + bias[f]) (BIAS_EXP), 1/sqrt(acc + bias[f] + eps) (BIAS_RSQRT),
 * 1/(acc + bias[f]) (BIAS_RECIP, the div of the CINN broadcast page's complex
 * ops: div, exp, rsqrt), max(acc + bias[f], 0) (BIAS_RELU, add + ReLU). */
typedef enum {
    BIGEMM_EPI_NONE = 0,
    BIGEMM_EPI_BIAS = 1,
    BIGEMM_EPI_BIAS_EXP = 2,
    BIGEMM_EPI_BIAS_RSQRT = 3,
    BIGEMM_EPI_BIAS_RECIP = 4,
    BIGEMM_EPI_BIAS_RELU = 5
} bigemm_epilogue;

typedef enum {
    BIGEMM_OK = 0,
    BIGEMM_ERR_INVALID_ARG = 1,   /* bad shape, null pointer, misaligned buffer   */
    BIGEMM_ERR_UNSUPPORTED = 2,   /* valid conv this library does not implement  */
    BIGEMM_ERR_CUDA = 3,          /* a CUDA runtime / driver call failed         */
    BIGEMM_ERR_TIMEOUT = 4,       /* a bounded device wait ran out               */
    BIGEMM_ERR_NO_CANDIDATE = 5   /* plan search found no runnable kernel        */
} bigemm_status;

/* Broadcast ops: out = var[c] (COPY), exp(var[c]) (EXP),
 * 1/sqrt(fp32(var[c] + eps)) (RSQRT), 1/var[c] (RECIP). */
typedef enum {
    BIGEMM_BC_COPY = 0,
    BIGEMM_BC_EXP = 1,
    BIGEMM_BC_RSQRT = 2,
    BIGEMM_BC_RECIP = 3
} bigemm_bcast_op;

/* Kernel families a plan can hold. */
typedef enum {
    BIGEMM_KIND_AUTO = 0,
    BIGEMM_KIND_UMMA = 1,         /* tcgen05 implicit GEMM (TF32 / FP16 / BF16)  */
    BIGEMM_KIND_SIMT = 2,         /* direct FP32-FMA conv (any shape, depthwise) */
} bigemm_kind;

typedef struct bigemm_plan_s *bigemm_plan;   /* opaque, library-owned */

/* Optional overrides for conv2d_nchw_plan_ex; zero fields mean "choose". */
typedef struct {
    int kind;       /* bigemm_kind                                              */
    int tile_n;     /* UMMA: output channels per tile, 16..256 step 16           */
    int split_k;    /* UMMA: number of K slices (>= 1)                          */
    int stages;     /* UMMA: shared-memory pipeline depth (2..8)                */
    int box_w;      /* UMMA: output pixels per tile along W (with box_h)        */
    int box_h;      /* UMMA: output rows per tile (box_w*box_h*boxes = 128);
                       SIMT depthwise: output rows per block of the staged-band
                       kernel (selects it over the streaming kernel)            */
    int mode;       /* UMMA operand-A mode: 1 channels-last boxes per tap,
                       2 NCHW read in place (1x1, stride 1, 16-bit),
                       3 one halo box per channel block (stride 1),
                       4 mode 1 over a subsampled copy (1x1, pad 0, stride > 1:
                         only the pixels the conv reads are packed),
                       5 mode 3 with the images stacked, pad zero rows apart,
                         so that one 16-row tile spans several small images,
                       6 NCHW read in place for a 1x1, stride-2, unpadded conv
                         (16-bit, H even, 2*W*element size a multiple of 16
                         bytes): TMA brings the even input rows, and warps of
                         the kernel keep the even pixels, so no packed copy is
                         made.
                       7 mode 1 with im2col tiles (K x K > 1, stride 1 or 2):
                         a tile is 128 consecutive output pixels of the
                         flattened N x Ho x Wo, across rows and images, and
                         each tap's operand is one TMA im2col load over the
                         channels-last copy (box_w and box_h are ignored;
                         outputs are written from registers).
                       With kind = SIMT it names the kernel instead: 1 tiled
                       (groups = 1) or naive, 2 depthwise staged band (box_h
                       rows per block), 3 depthwise streaming (box_h = 2, 4
                       or 8 rows per thread), 4 depthwise whole planes
                       (H, W <= 32, one or two planes per warp), 5 depthwise
                       small planes (stride 1, square 3/5/7 kernel, pad K/2,
                       outputs at most 16 wide and 32 tall; each thread
                       computes a box_h x 8 block of outputs, box_h = 2 or 4,
                       0 meaning 4), 6 depthwise bands of rows (square 3/5/7
                       kernel, pad K/2, stride 1 or 2, input rows whose bytes
                       are a multiple of 16 and at most 512; 4 x 8 outputs
                       per thread).
                       Other values: INVALID_ARG.                               */
    int resident_b; /* UMMA: 1 keeps the weights resident in shared memory --
                       halo modes: one output-channel tile must cover CO and
                       every tap must fit; other modes: split_k 1, and every K
                       block of one output-channel tile must fit (each block
                       keeps one tile) -- -1 streams them, 0 chooses            */
    int epi_warps;  /* UMMA modes 1, 2 and 4 with tile_n = 128: 16 runs four
                       epilogue warps per TMEM lane quadrant (576 threads per
                       block) instead of two (8); 0 chooses; other values:
                       INVALID_ARG                                              */
    int cta_pair;   /* UMMA modes 3 and 5 with resident weights, tile_n 64 or
                       128, split_k 1: 1 runs clusters of two blocks that share
                       each MMA (M = 256 pixels, each block holding half of the
                       weights), -1 single blocks, 0 chooses; other values:
                       INVALID_ARG                                              */
} bigemm_plan_options;

/*
 * conv2d_nchw_plan -- validate a conv shape and pick the kernel that runs it.
 *   N,H,W      batch and input spatial size (N >= 1, H, W >= 1)
 *   CO, CI     output / input channels; groups = 1, or groups = CI = CO
 *              (depthwise)
 *   KH, KW     kernel size; stride >= 1, padding >= 0 (dilation is 1)
 *   in_dtype   type of data and kernel: F32 (TF32 tensor cores or FP32 FMA),
 *              F16 or BF16 (fp32 accumulation)
 *   out_dtype  type of out (F32, F16 or BF16)
 *   epi        fused epilogue (bias is then required at run time)
 *   search     0: heuristic choice, no launch; 1: time every valid candidate
 *              with CUDA events on `stream` (synchronises) and keep the best
 *   out_plan   receives the plan; free it with conv2d_nchw_plan_destroy.
 * Errors: INVALID_ARG (Ho or Wo <= 0, bad groups, null out_plan),
 * UNSUPPORTED (e.g. depthwise with a channel multiplier), CUDA,
 * NO_CANDIDATE.  Plans are cached per (shape, dtypes, epilogue, device);
 * each call still returns a fresh handle.
 */
bigemm_status conv2d_nchw_plan(int N, int H, int W, int CO, int CI, int KH, int KW,
                               int stride, int padding, int groups,
                               bigemm_dtype in_dtype, bigemm_dtype out_dtype,
                               bigemm_epilogue epi, int search,
                               void *stream, bigemm_plan *out_plan);

/* As conv2d_nchw_plan, with optional overrides (opts may be NULL).  A forced
 * choice that cannot run this shape returns UNSUPPORTED.  Forced plans are
 * not cached. */
bigemm_status conv2d_nchw_plan_ex(int N, int H, int W, int CO, int CI, int KH, int KW,
                                  int stride, int padding, int groups,
                                  bigemm_dtype in_dtype, bigemm_dtype out_dtype,
                                  bigemm_epilogue epi, int search,
                                  const bigemm_plan_options *opts,
                                  void *stream, bigemm_plan *out_plan);

/*
 * conv2d_nchw_run -- run a plan on `stream`.
 *   data   [N,CI,H,W] device, in_dtype, 16-byte aligned
 *   kernel [CO,CI/groups,KH,KW] device, in_dtype, 16-byte aligned
 *   bias   [CO] fp32 device, or NULL when the plan's epilogue is NONE
 *   eps    added inside rsqrt for BIAS_RSQRT, ignored otherwise
 *   out    [N,CO,Ho,Wo] device, out_dtype, 16-byte aligned; fully written
 * Errors: INVALID_ARG (null or misaligned pointer, missing bias), CUDA.
 */
bigemm_status conv2d_nchw_run(bigemm_plan plan, const void *data, const void *kernel,
                              const float *bias, float eps, void *out, void *stream);

/* Free the plan and its scratch (synchronises with the device first). */
bigemm_status conv2d_nchw_plan_destroy(bigemm_plan plan);

/* Write a one-line JSON description of the plan (kernel, tiles, split-K,
 * launches per run, scratch bytes, search records) into buf (NUL-terminated,
 * truncated to len).  Returns INVALID_ARG for a NULL plan or buffer. */
bigemm_status conv2d_nchw_plan_describe(bigemm_plan plan, char *buf, size_t len);

/*
 * bcast_nchw_run -- out[n,c,h,w] = op(var[c]) for all n < N, h < H, w < W.
 *   var  [C] fp32 device; out [N,C,H,W] device of out_dtype (F32/F16/BF16).
 *   op   bigemm_bcast_op; eps is used by RSQRT only.
 * Errors: INVALID_ARG (N, C, H or W < 1, null pointer, bad op/dtype), CUDA.
 */
bigemm_status bcast_nchw_run(int N, int C, int H, int W, int op, const float *var, float eps,
                             void *out, bigemm_dtype out_dtype, void *stream);

/*
 * bcast_run -- the general form, out[b0,p,b1] = op(var[p]) for b0 < B0,
 * p < P, b1 < B1: any broadcast [1,P,1] => [B0,P,B1] after fusing adjacent axes
 * of the same kind, the last axis broadcast ("[CINN] Add the TileBroadcastTactic
 * for NCHW broadcast", PaddlePaddle PR 70092, Introduction).  The NCHW case is
 * B0 = N, P = C, B1 = H*W.  Long rows (B1 * element size >= 1 KB) run the
 * per-channel kernel of bcast_nchw_run; shorter rows a kernel whose threads
 * each own a fixed 16-byte piece of the P*B1 run and repeat it down B0.
 *   var  [P] fp32 device; out [B0,P,B1] device of out_dtype (F32/F16/BF16),
 *        aligned to its element size (16-byte alignment takes vector stores).
 *   op   bigemm_bcast_op; eps is used by RSQRT only.
 * Errors: INVALID_ARG (a size < 1, null pointer, bad op/dtype, misaligned
 * output), UNSUPPORTED (P*B1 > 2^31 - 1), CUDA.
 */
bigemm_status bcast_run(int B0, int P, int B1, int op, const float *var, float eps, void *out,
                        bigemm_dtype out_dtype, void *stream);

/* The same broadcast written the way a generic fused-loop schedule does it:
 * one flat loop over all N*C*H*W outputs, each recomputing op(var[c]) from
 * its own index.  Kept to measure the per-channel mapping against it. */
bigemm_status bcast_nchw_run_flat(int N, int C, int H, int W, int op, const float *var,
                                  float eps, void *out, bigemm_dtype out_dtype, void *stream);

/*
 * conv2d_nchw_run_noalloc -- the same convolution for callers that cannot
 * allocate device memory: code that runs where cudaMalloc is forbidden or
 * would break a memory budget someone else fixed, and so can neither create a
 * plan (plans own cudaMalloc'd scratch) nor lend the library a workspace.
 * The sources have no counterpart of this call; it exists for those callers.
 *
 * It runs the channels-last tensor-core kernel (the packed-operand path with
 * split-K when the tiles alone leave SMs idle) with every scratch byte in one
 * fixed array in the library's own device memory: 16 MiB (16777216 bytes),
 * held on every GPU that loads the library until the process exits.  The
 * scratch a shape needs is
 *   r(N*H*W*Ch*e) + r(CO*KH*KW*cip*e) + S*N*CO*Ho*Wo*4 bytes,
 * where r() rounds up to 256, e is the input element size, Ch = CI rounded up
 * to 16/e, cip = CI rounded up to 128/e, and S is the number of K slices.
 * S = 1 unless the pixel tiles times the channel tiles cover less than half
 * the SMs; then S is lowered, down to 1, until the partial sums fit.  Shapes
 * whose data and kernel copies alone exceed 16 MiB return
 * BIGEMM_ERR_UNSUPPORTED before any launch.
 *
 * Arguments and layouts are those of conv2d_nchw_plan + conv2d_nchw_run with
 * groups = 1 (data [N,CI,H,W], kernel [CO,CI,KH,KW], bias [CO] fp32, out
 * [N,CO,Ho,Wo], device pointers owned by the caller, 16-byte aligned;
 * stride <= 8).  timeout_flag is an optional device int the kernels set to 4
 * (BIGEMM_ERR_TIMEOUT) if a bounded device wait runs out (the caller clears
 * it); when NULL the kernels raise the library's sticky device flag instead,
 * which bigemm_last_device_error() reports and bigemm_clear_device_error()
 * clears.  That flag is a file-scope device variable too, not an allocation.
 *
 * The call allocates nothing: no cudaMalloc, cudaFree or allocating library
 * routine.  The first call on a device looks up the device address of the
 * scratch array (cudaGetSymbolAddress, with that device current), so make
 * that first call before any stream capture.  Every call on a device shares
 * the one array and leaves its contents behind; calls whose kernels overlap on
 * the GPU (different streams, or several host threads) race on it and must be
 * ordered by the caller.  Errors: INVALID_ARG (bad shape, dtype, epilogue,
 * null or misaligned pointer, missing bias), UNSUPPORTED (scratch above the
 * limit, stride > 8), CUDA.
 */
bigemm_status conv2d_nchw_run_noalloc(int N, int H, int W, int CO, int CI, int KH, int KW,
                                      int stride, int padding, bigemm_dtype in_dtype,
                                      bigemm_dtype out_dtype, bigemm_epilogue epi,
                                      const void *data, const void *kernel, const float *bias,
                                      float eps, void *out, int *timeout_flag, void *stream);

/* ------------------------------------------------ transformer-layer operators
 *
 * Matrices are row-major in device memory, rows `ld` elements apart (ld at
 * least the row's length), each base on a boundary of its element size.  Rows
 * on 16-byte boundaries take the fast paths; any other alignment is served too.
 * The calls keep no state and allocate nothing; they are asynchronous on `stream`, and calls may overlap on different streams.  rows
 * or M = 0 is a call that does nothing.
 *
 * MXF8 matrices: e4m3 elements, and a buffer of scales (16-byte aligned,
 * bigemm_mx_scale_bytes(rows, cols) bytes): the byte `code` of element (r, k)
 * stands for 2^(code - 127) and is at
 *   ((r/128) * ceil(cols/128) + k/128) * 512 + (r%32)*16 + ((r%128)/32)*4 + (k%128)/32.
 * Writers use the smallest power of two s >= 2^-127 with amax <= 448 s over the
 * group's 32 elements and round each element / s to nearest even; a group with
 * a NaN or an infinity gets code 255 and NaN elements.  They write the codes of
 * every group of the rows' last 128-column block (0 past the last column), and
 * leave the codes of rows past the last alone.  Readers ignore those rows' codes
 * and expect finite codes (not 255) in groups past the last column.
 */
typedef enum {
    BIGEMM_ACT_NONE = 0,
    BIGEMM_ACT_RELU = 1,
    BIGEMM_ACT_GELU = 2,        /* 0.5 z (1 + erf(z / sqrt 2))                          */
    BIGEMM_ACT_GELU_TANH = 3,   /* 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))      */
    BIGEMM_ACT_SILU = 4         /* z / (1 + exp(-z))                                    */
} bigemm_act;

typedef enum {
    BIGEMM_COMBINE_NONE = 0,
    BIGEMM_COMBINE_ADD = 1,     /* + other: the residual                                */
    BIGEMM_COMBINE_MUL = 2      /* * other: the other half of a gated layer             */
} bigemm_combine;

/*
 * matmul_run -- out[m,n] = combine(act(sum_k x[m,k] w[n,k] + bias[n]), other[m,n])
 *   x [M,K], w [N,K] of in_dtype (F16 or BF16), fp32 sums; bias [N] fp32 or NULL
 *   other [M,N] of other_dtype (F32, F16, BF16), read unless combine is NONE; it
 *   may be out itself (same type and rows)
 *   out [M,N] of out_dtype (F32, F16, BF16), rounded once.  For F32, and for an MXF8
 *   output, at most 512 products at a time (2048 of MXF8 operands) are summed in
 *   the tensor core, the rest in fp32 adds.
 *   workspace: matmul_workspace_bytes of device memory on a 16-byte boundary,
 *   the call's until it is done; NULL where that is 0.
 * Errors: INVALID_ARG (a size, null or misaligned pointer, short ld, bad enum, a
 * workspace that is too small), UNSUPPORTED (in_dtype F32; a size above 2^30 or 2^31 tiles), CUDA.
 */
bigemm_status matmul_run(int M, int N, int K, bigemm_dtype in_dtype, const void *x, int64_t ldx,
                         const void *w, int64_t ldw, const float *bias, int act, int combine,
                         bigemm_dtype other_dtype, const void *other, int64_t ldother,
                         bigemm_dtype out_dtype, void *out, int64_t ldo, void *workspace,
                         uint64_t workspace_bytes, void *stream);

/*
 * matmul_mx_run -- the same product of MXF8 matrices x [M,K] and w [N,K] with
 * their scales.  out_dtype F32, F16, BF16 (out_scale NULL), or MXF8: e4m3 into
 * out and its scales into out_scale.
 */
bigemm_status matmul_mx_run(int M, int N, int K, const void *x, int64_t ldx, const void *x_scale,
                            const void *w, int64_t ldw, const void *w_scale, const float *bias,
                            int act, int combine, bigemm_dtype other_dtype, const void *other,
                            int64_t ldother, bigemm_dtype out_dtype, void *out, int64_t ldo,
                            void *out_scale, void *workspace, uint64_t workspace_bytes,
                            void *stream);

/* Bytes of workspace that a product of these operands (in_dtype F16, BF16 or
 * MXF8) needs: for a copy of each whose rows are off the 16-byte grid, rows on
 * it; 0 where none is. */
uint64_t matmul_workspace_bytes(int M, int N, int K, bigemm_dtype in_dtype, const void *x,
                                int64_t ldx, const void *w, int64_t ldw);

/*
 * matmul_gated_run -- the two products of a gated layer in one kernel:
 *   g = x w_gate^T + bias_gate,  u = x w_up^T + bias_up,  out = act(g) * u
 *   x [M,K], w_gate and w_up [N,K], out [M,N] of dtype (F16 or BF16); bias_gate,
 *   bias_up [N] fp32, each or NULL; fp32 sums, out rounded once (g and u are not
 *   rounded on the way to it)
 *   one tensor-core accumulator, which cuts each addition short, takes sums of up to
 *   32768 products (terms of one sign come out 2e-4 too small at that length, 2e-5 at
 *   4096); longer K is summed in pieces of 512
 *   gate, up [M,N] of dtype, each or NULL (not wanted): receive g and u, each rounded
 *   once, which matmul_gated_backward_run takes.  out, gate and up are buffers of their own
 *   workspace: matmul_gated_workspace_bytes of device memory on a 16-byte boundary,
 *   the call's until it is done; NULL where that is 0.
 * Errors: as matmul_run.
 */
bigemm_status matmul_gated_run(int M, int N, int K, bigemm_dtype dtype, const void *x, int64_t ldx,
                               const void *w_gate, int64_t ldw_gate, const void *w_up,
                               int64_t ldw_up, const float *bias_gate, const float *bias_up, int act,
                               void *out, int64_t ldo, void *gate, int64_t ldgate, void *up,
                               int64_t ldup, void *workspace, uint64_t workspace_bytes,
                               void *stream);

/* Bytes of workspace that it needs: for a copy of each operand whose rows are off the
 * 16-byte grid; 0 where none is. */
uint64_t matmul_gated_workspace_bytes(int M, int N, int K, const void *x, int64_t ldx,
                                      const void *w_gate, int64_t ldw_gate, const void *w_up,
                                      int64_t ldw_up);

/*
 * matmul_backward_run -- gradients of out = x w^T + bias, of dout [M,N], that of out:
 *   dx [M,K] = dout w,  dw [N,K] = dout^T x,  dbias [N] = sum over tokens of dout
 *   all but dbias (fp32, or NULL: not wanted) of dtype (F16 or BF16); fp32 sums, of at
 *   most 32768 products in a tensor-core accumulator (as in matmul_gated_run) and the
 *   shares of longer ones added in fp32; each output rounded once; the sums' order does
 *   not depend on timing.  M = 0 writes zeros to dw and dbias.  The outputs are buffers of
 *   their own.
 *   workspace: matmul_backward_workspace_bytes of device memory on a 16-byte boundary,
 *   the call's until it is done.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype F32; a size above 2^30), CUDA.
 */
bigemm_status matmul_backward_run(int M, int N, int K, bigemm_dtype dtype, const void *dout,
                                  int64_t lddout, const void *x, int64_t ldx, const void *w,
                                  int64_t ldw, void *dx, int64_t lddx, void *dw, int64_t lddw,
                                  float *dbias, void *workspace, uint64_t workspace_bytes,
                                  void *stream);
uint64_t matmul_backward_workspace_bytes(int M, int N, int K, const void *dout, int64_t lddout,
                                         const void *x, int64_t ldx, const void *w, int64_t ldw);

/*
 * matmul_gated_backward_run -- gradients of matmul_gated_run, of dout [M,N], that of out,
 * and gate and up (g and u) as that call kept them:
 *   dg = dout u act'(g),  du = dout act(g)   in fp32, then rounded to dtype, which the
 *   tensor core takes (F16: infinite past 65504, fewer bits below 6e-5)
 *   dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x
 *   dbias_gate, dbias_up [N] fp32, each or NULL: sums over tokens of dg and du, not rounded
 *   (act' of relu is 0 at 0.)  Otherwise as matmul_backward_run.
 */
bigemm_status matmul_gated_backward_run(int M, int N, int K, bigemm_dtype dtype, const void *dout,
                                        int64_t lddout, const void *x, int64_t ldx,
                                        const void *w_gate, int64_t ldw_gate, const void *w_up,
                                        int64_t ldw_up, const void *gate, int64_t ldgate,
                                        const void *up, int64_t ldup, int act, void *dx,
                                        int64_t lddx, void *dw_gate, int64_t lddw_gate, void *dw_up,
                                        int64_t lddw_up, float *dbias_gate, float *dbias_up,
                                        void *workspace, uint64_t workspace_bytes, void *stream);
uint64_t matmul_gated_backward_workspace_bytes(int M, int N, int K, const void *x, int64_t ldx,
                                               const void *w_gate, int64_t ldw_gate,
                                               const void *w_up, int64_t ldw_up);

/*
 * rmsnorm_run -- h = x + residual; out = h * rsqrt(mean(h^2) + eps) * weight,
 * row by row over `cols` columns, in fp32 from the inputs to one rounding of
 * each output.
 *   x, residual (NULL: none), sum_out (NULL: not wanted; receives h; it may be
 *   x or residual itself) of in_dtype (F32, F16, BF16); weight [cols] fp32 or
 *   NULL (ones); out of in_dtype, F32, or MXF8 (then out_scale, else NULL)
 * Errors: INVALID_ARG, UNSUPPORTED (another out_dtype; cols above 2^30), CUDA.
 */
bigemm_status rmsnorm_run(int rows, int cols, bigemm_dtype in_dtype, const void *x, int64_t ldx,
                          const void *residual, int64_t ldr, const float *weight, float eps,
                          void *sum_out, int64_t lds, bigemm_dtype out_dtype, void *out, int64_t ldo,
                          void *out_scale, void *stream);

/*
 * layernorm_run -- h = x + residual; out = (h - mean(h)) * rsqrt(var(h) + eps) *
 * weight + bias, row by row over `cols` columns, var the mean square of h - mean(h);
 * in fp32 from the inputs to one rounding of each output.
 *   x, residual (NULL: none), sum_out (NULL: not wanted; receives h) of in_dtype (F32,
 *   F16, BF16); weight, bias [cols] fp32, each or NULL (ones, zeros); out of in_dtype,
 *   F32, or MXF8 (then out_scale, else NULL).  sum_out, and out of in_dtype, may be x or
 *   residual itself (same rows); outputs share no memory with anything else
 *   mean, rstd [rows] fp32, each or NULL (not wanted): of h before it is rounded,
 *   what layernorm_backward_run takes
 * Errors: INVALID_ARG, UNSUPPORTED (another out_dtype; cols above 2^30), CUDA.
 */
bigemm_status layernorm_run(int rows, int cols, bigemm_dtype in_dtype, const void *x, int64_t ldx,
                            const void *residual, int64_t ldr, const float *weight,
                            const float *bias, float eps, void *sum_out, int64_t lds,
                            bigemm_dtype out_dtype, void *out, int64_t ldo, void *out_scale,
                            float *mean, float *rstd, void *stream);

/*
 * layernorm_backward_run -- gradients of out = (x - mean) * rstd * weight + bias, of
 * dout, that of out.  With xh = (x - mean) rstd and g = dout * weight, mean over k:
 *   dx = rstd (g - mean(g) - xh mean(g xh)) + dsum
 *   dweight[k] = sum over rows of dout xh,  dbias[k] = sum over rows of dout
 * in fp32, dx rounded once; the sums' order does not depend on timing.
 *   dout, x (the normed rows: h where there was a residual), dsum (NULL: none; the
 *   gradient that reaches h along the residual stream) and dx of dtype (F32, F16,
 *   BF16); dx may be dout, x or dsum itself (same rows); outputs share no memory with
 *   anything else
 *   mean, rstd [rows] of the forward pass; weight [cols] or NULL (ones); dweight,
 *   dbias [cols], all fp32.  rows = 0 writes zeros to dweight and dbias.
 *   workspace: norm_backward_workspace_bytes of device memory on a 16-byte boundary,
 *   the call's until it is done.
 * Errors: INVALID_ARG, UNSUPPORTED (cols above 2^30), CUDA.
 */
bigemm_status layernorm_backward_run(int rows, int cols, bigemm_dtype dtype, const void *dout,
                                     int64_t lddout, const void *x, int64_t ldx, const float *mean,
                                     const float *rstd, const float *weight, const void *dsum,
                                     int64_t lddsum, void *dx, int64_t lddx, float *dweight,
                                     float *dbias, void *workspace, uint64_t workspace_bytes,
                                     void *stream);

/*
 * rmsnorm_backward_run -- gradients of out = x * rstd * weight, rstd = rsqrt(mean(x^2)
 * + eps), found again from x.  With xh = x rstd and g = dout * weight:
 *   dx = rstd (g - xh mean(g xh)) + dsum,  dweight[k] = sum over rows of dout xh
 * Otherwise as layernorm_backward_run.
 */
bigemm_status rmsnorm_backward_run(int rows, int cols, bigemm_dtype dtype, const void *dout,
                                   int64_t lddout, const void *x, int64_t ldx, const float *weight,
                                   float eps, const void *dsum, int64_t lddsum, void *dx,
                                   int64_t lddx, float *dweight, void *workspace,
                                   uint64_t workspace_bytes, void *stream);

/* Bytes of workspace that either norm's gradients need. */
uint64_t norm_backward_workspace_bytes(int rows, int cols);

/* mx_quantize_run -- a matrix of in_dtype (F32, F16, BF16) as MXF8. */
bigemm_status mx_quantize_run(int rows, int cols, bigemm_dtype in_dtype, const void *x, int64_t ldx,
                              void *out, int64_t ldo, void *scale, void *stream);

/* Bytes of the scales of a rows x cols MXF8 matrix (0 if a size is below 1). */
uint64_t bigemm_mx_scale_bytes(int rows, int cols);

/* Human-readable text of a status code (static storage). */
const char *bigemm_status_string(bigemm_status s);

/* Sticky device-side flag: BIGEMM_ERR_TIMEOUT once any kernel's bounded wait
 * ran out on the current device (planned runs, broadcasts, and
 * conv2d_nchw_run_noalloc calls given no timeout_flag), else BIGEMM_OK.
 * Synchronises the device.  The flag is a file-scope device variable of the
 * library (one per device, zero at load), so reading it allocates nothing. */
bigemm_status bigemm_last_device_error(void);

/* Clear the sticky device flag (synchronises the device). */
bigemm_status bigemm_clear_device_error(void);

/* Upper bound, in nanoseconds, of every device-side wait of later launches
 * (default 2e9).  Values below 1000 are raised to 1000. */
bigemm_status bigemm_set_wait_timeout_ns(uint64_t ns);

/* Launch one block that waits on a barrier nothing will complete, bounded by
 * timeout_ns; the host then sees BIGEMM_ERR_TIMEOUT from
 * bigemm_last_device_error().  Exercises the timeout path without a fault. */
bigemm_status bigemm_debug_wait_timeout(uint64_t timeout_ns, void *stream);

/* Per-kernel timing with CUDA events recorded around each launch on its
 * stream.  enable(1) starts recording (and clears old records). */
typedef struct {
    char name[48];
    int launches;
    double total_ms;
} bigemm_kernel_time;

bigemm_status bigemm_profile_enable(int on);
/* Synchronises, then fills up to max entries; *count receives the number of
 * distinct kernels.  Records stay until the next enable(1). */
bigemm_status bigemm_profile_read(bigemm_kernel_time *out, int max, int *count);

/* Library version string. */
const char *bigemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BIGEMM_H */
