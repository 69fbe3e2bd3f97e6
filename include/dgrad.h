/*
 * dgrad.h -- C ABI of libdgrad, a B200 (sm_100a) engine for convolution
 * backward-data ("dgrad"): dX = dgrad(dY, W) on NHWC activations.
 *
 * Operation.  For a forward convolution with dilation 1, stride S, per-axis
 * padding (pad_h, pad_w) and output extents
 *     Ho = floor((H + 2*pad_h - KH) / S) + 1,   Wo = floor((W + 2*pad_w - KW) / S) + 1
 * ("channel-packed and large-filter depthwise dgrad", Technical Details,
 * per-axis padding: Wo uses PAD_W), dgrad is the adjoint of the forward map in
 * its input:
 *     dX[n,h,w,c] = sum over (ho,wo,k,r,s) with h = ho*S - pad_h + r and
 *                   w = wo*S - pad_w + s of dY[n,ho,wo,k] * Wt(k,r,s,c).
 * Two shape classes are served:
 *   - pointwise: 1x1 filter, stride 1, no padding, one group.  dX[M,C] =
 *     dY[M,K] . W[K,C] with M = N*H*W, dY offset m*K + k, W offset k*C + c and
 *     dX offset m*C + c ("add the pointwise fast path dgrad was missing",
 *     Technical Details and the fast-path commit message);
 *   - depthwise: groups = C = K (depth multiplier 1), W[KH][KW][C].  Stride 1
 *     runs as a correlation of dY with the 180-degree rotated filter at padding
 *     KH-1-pad_h rows and KW-1-pad_w columns, filters up to 64 a side, square or
 *     not; stride > 1 runs as a row-streaming kernel whose accumulator rows sit
 *     in circular slots (registers, or a shared-memory ring) ("channel-packed and large-filter
 *     depthwise dgrad", Technical Details: rotated-filter dgrad and the
 *     channel-packed row-streaming dgrad).
 *
 * Layouts (all dense, channels innermost, no padding between rows):
 *     dY  [N][Ho][Wo][K]      dX [N][H][W][C]
 *     W   pointwise [K][C];   depthwise [KH][KW][C]
 * Element type: DGRAD_F32 (float in, float out), DGRAD_BF16 (bf16 in, bf16 out)
 * or DGRAD_F16 (f16 in, f16 out).  Accumulation is always fp32; a 16-bit dX is
 * rounded once, to nearest even.
 *
 * Memory and streams.  Every pointer is device memory the caller owns (for
 * example a PyTorch CUDA tensor's data pointer) on the current device.  Calls
 * enqueue work on `stream` (a cudaStream_t; NULL is the legacy default stream)
 * and return without synchronising; the library allocates no device memory per
 * call.  dX is written in full (never accumulated into), so it needs no zeroing.
 * Alignment: every base pointer 16-byte aligned, and K and C multiples of 8
 * (bf16, f16) or 4 (f32), so that every channel row starts on 16 bytes.
 *
 * Errors.  Arguments are validated on the host before anything is launched; a
 * rejected call launches nothing and leaves dX untouched.  A launch failure is
 * reported as DGRAD_ERR_CUDA (the CUDA error is kept for dgrad_last_cuda_error).
 * Kernels never trap: a device-side wait that runs past its limit sets a status
 * word and the kernel returns; dgrad_check_status reports it.
 */
#ifndef DGRAD_H
#define DGRAD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Problem geometry (the pages' DirectConvProblem: extents, filter, stride and
 * per-axis padding; "channel-packed and large-filter depthwise dgrad",
 * Technical Details, per-axis padding).  H, W are dX's spatial extents; C is
 * dX's channel count and K dY's.  Dilation is 1.  pad_w == -1 means "same as
 * pad_h" (the pages' sentinel); any other negative value is invalid. */
typedef struct {
    int64_t N, H, W, C, K;
    int32_t KH, KW, stride;
    int32_t pad_h, pad_w;
} dgrad_problem_t;

/* Element type of dY, W and dX (one type for all three).  DGRAD_F16 is served by
 * every entry point: dgrad_pointwise, its split-K variants, dgrad_dense,
 * dgrad_grouped and dgrad_depthwise_tc run tcgen05 MMAs on f16 operands with
 * fp32 accumulation; dgrad_depthwise widens f16 to fp32 on load and uses fp32
 * FMAs.  DGRAD_F32 is served by dgrad_pointwise, dgrad_depthwise, layer norm and
 * dropout only. */
typedef enum { DGRAD_F32 = 0, DGRAD_BF16 = 1, DGRAD_F16 = 2 } dgrad_dtype_t;

/* Depthwise kernel choice.  AUTO: rotated-filter for stride 1, row-streaming
 * otherwise.  ROTATED requires stride 1.  ROWSTREAM serves any stride (at
 * stride 1 it is a cross-check of the rotated-filter kernel). */
typedef enum { DGRAD_DW_AUTO = 0, DGRAD_DW_ROTATED = 1, DGRAD_DW_ROWSTREAM = 2 } dgrad_dw_mode_t;

typedef enum {
    DGRAD_OK = 0,
    DGRAD_ERR_INVALID = 1,      /* null pointer, non-positive extent, pad_w < -1, Ho or Wo < 1 ... */
    DGRAD_ERR_UNSUPPORTED = 2,  /* valid geometry this entry point does not serve */
    DGRAD_ERR_ALIGNMENT = 3,    /* base pointer or channel row not 16-byte aligned */
    DGRAD_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed */
    DGRAD_ERR_TIMEOUT = 5,      /* a kernel gave up waiting (reported by dgrad_check_status) */
    DGRAD_ERR_BOUNDS = 6        /* libdgrad_debug.so only: a store index check failed (dgrad_check_status) */
} dgrad_status_t;

/* Pointwise dgrad, dX[M,C] = dY[M,K] . W[K,C] with M = N*H*W.
 * Requires KH = KW = 1, stride 1, pad_h = pad_w = 0 (else DGRAD_ERR_UNSUPPORTED;
 * the pointwise page's shape class).  DGRAD_BF16 runs on the tcgen05 tensor
 * cores (TMA-fed shared-memory tiles, fp32 accumulators in tensor memory);
 * DGRAD_F16 runs on them through the tap kernel of dgrad_grouped (one 1x1 tap);
 * DGRAD_F32 runs as an fp32 FMA kernel (no reduced-precision inputs). */
dgrad_status_t dgrad_pointwise(const dgrad_problem_t* prob, dgrad_dtype_t dtype,
                               const void* dY, const void* W, void* dX, void* stream);

/* Split-K pointwise dgrad for problems with few output tiles (small M = N*H*W,
 * long K): each 128 x 128 tile's K-loop is split into `splits` ranges that run
 * on different SMs; partial tiles are written as fp32 to `workspace` and then
 * summed in split order (deterministic: no atomics, nothing to zero) and
 * rounded once to bf16 (or f16) into dX.  Same shape class and layouts as
 * dgrad_pointwise; DGRAD_BF16 or DGRAD_F16 (else DGRAD_ERR_UNSUPPORTED).  The pages'
 * implicit-GEMM dgrad has a split-K mode ("add the pointwise fast path dgrad
 * was missing", review-fix commit: split-K sub-GEMMs, dX accumulated
 * atomically).
 * splits: 1 .. 64, or 0 to let the library choose one that fills the GPU.
 * workspace: caller-owned device memory, 16-byte aligned, at least the size
 * dgrad_pointwise_splitk_workspace reports for the same problem and splits;
 * its contents on entry do not matter and are clobbered.  Too small or null:
 * DGRAD_ERR_INVALID. */
dgrad_status_t dgrad_pointwise_splitk(const dgrad_problem_t* prob, dgrad_dtype_t dtype, int splits,
                                      const void* dY, const void* W, void* dX,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes dgrad_pointwise_splitk needs for `splits` (0: the automatic
 * choice, which is returned in *splits_used when that pointer is non-null).
 * Queries the current device's SM count for the automatic choice. */
dgrad_status_t dgrad_pointwise_splitk_workspace(const dgrad_problem_t* prob, int splits, size_t* bytes,
                                                int* splits_used);

/* ---- A variant for callers that cannot allocate (no counterpart on the
 * pages: their kernels take whatever workspace their host framework gives). ---- */

/* Size of the fixed split-K scratch buffer built into the library: 8 MiB, one
 * buffer per device. */
#define DGRAD_SPLITK_SCRATCH_BYTES ((size_t)8 << 20)

/* dgrad_pointwise_splitk with no workspace argument: the fp32 partial tiles go
 * to a fixed buffer of DGRAD_SPLITK_SCRATCH_BYTES that is part of the
 * library's device image (CUDA reserves it when it loads the library's code on
 * a device), so the call allocates nothing: no cudaMalloc, no framework
 * allocator.  It serves callers that have no workspace to pass and must not
 * allocate at call time, for example a plugin or callback running inside a
 * framework that owns all device memory, or code that runs while a caching
 * allocator is reclaiming memory and so cannot call back into it.
 * Same shape class, dtype, layouts, kernels and results as
 * dgrad_pointwise_splitk with the same split count.
 * splits: 1 .. 64, or 0 for the automatic count, lowered as far as needed for
 * the partial tiles to fit the buffer.  When the partial tiles still need more
 * than DGRAD_SPLITK_SCRATCH_BYTES (splits * M * C * 4 bytes, M = N*H*W; with
 * splits 0, even one split's M * C * 4), the call returns
 * DGRAD_ERR_UNSUPPORTED and launches nothing.
 * Nothing in the buffer has to start at zero and nothing clears it: each split
 * writes its whole partial tile before the reduction reads it.
 * Set-up: the first call on each device (with that device current) looks up
 * the buffer's device address and keeps it for the life of the process; make
 * that first call before any stream capture begins.  The kept address belongs
 * to the device's primary context: resetting the device (cudaDeviceReset) or
 * calling from another context is not supported.
 * Races: there is ONE buffer per device.  Calls whose work may overlap on the
 * same device (issued to different streams, or from several host threads
 * without ordering between their streams) write the same buffer and corrupt
 * each other's results.  Calls ordered on one stream are safe. */
dgrad_status_t dgrad_pointwise_splitk_noalloc(const dgrad_problem_t* prob, dgrad_dtype_t dtype, int splits,
                                              const void* dY, const void* W, void* dX, void* stream);

/* Grouped dgrad: `groups` groups, each of K/groups dY and C/groups dX channels,
 * any KH x KW filter and stride, on the tcgen05 tensor cores; W is
 * [KH][KW][K][C/groups] (tap-major; each tap holds, for every dY channel k, the
 * C/groups filter values of k's group).  A 1x1 filter is the pages' grouped
 * pointwise dgrad (per-group output channel base and a C/groups W stride; "add
 * the pointwise fast path dgrad was missing", Technical Details).  Each group
 * runs as its own set of phase GEMMs, as in dgrad_dense.  groups must divide K
 * and C (else DGRAD_ERR_INVALID); K/groups and C/groups multiples of 8 (else
 * DGRAD_ERR_ALIGNMENT); DGRAD_BF16 or DGRAD_F16; other limits as dgrad_dense. */
dgrad_status_t dgrad_grouped(const dgrad_problem_t* prob, int64_t groups, dgrad_dtype_t dtype, const void* dY,
                             const void* W, void* dX, void* stream);

/* Dense (ungrouped, groups = 1) dgrad with a KH x KW filter and any stride, on
 * the tcgen05 tensor cores; W is [KH][KW][K][C] (tap-major: each tap is a
 * pointwise [K][C] matrix).  The pages' main dgrad engine decomposes a strided
 * dgrad by output phase into stride*stride sub-GEMMs ("add the pointwise fast
 * path dgrad was missing", Technical Details); here each phase's GEMM sums, over
 * the phase's taps, products of a shifted window of dY (K deep) with that tap's
 * [K][C] matrix, so no im2col buffer is built.  DGRAD_BF16 or DGRAD_F16 (else
 * DGRAD_ERR_UNSUPPORTED); KH, KW, stride <= 64; K and C multiples of 8; padding
 * any value >= 0 that leaves Ho, Wo >= 1. */
dgrad_status_t dgrad_dense(const dgrad_problem_t* prob, dgrad_dtype_t dtype, const void* dY, const void* W, void* dX,
                           void* stream);

/* Depthwise dgrad (groups = C; requires K == C, else DGRAD_ERR_UNSUPPORTED).
 * Rotated-filter mode requires stride 1, KH and KW <= 64 and
 * 0 <= pad_h <= KH-1, 0 <= pad_w <= KW-1 (the rotated padding KH-1-pad_h and
 * KW-1-pad_w is then non-negative).  Row-streaming requires KH, KW <= 64,
 * stride <= 8, 0 <= pad_h <= KH-1 and 0 <= pad_w <= KW-1.  Any element type:
 * 16-bit inputs are widened to fp32 on load and dX is rounded once. */
dgrad_status_t dgrad_depthwise(const dgrad_problem_t* prob, dgrad_dtype_t dtype,
                               dgrad_dw_mode_t mode,
                               const void* dY, const void* W, void* dX, void* stream);

/* Stride-1 depthwise dgrad on the tensor cores, for large filters.  Each
 * channel's plane is a sum of GEMMs, one per filter line along the shorter
 * filter side, whose other operand is the banded (Toeplitz) matrix of that
 * filter line along the longer side: the implicit-GEMM formulation of the
 * rotated-filter correlation ("channel-packed and large-filter depthwise
 * dgrad", Technical Details: rotated-filter dgrad; the pages sent large filters
 * through an implicit-GEMM path before the FP32 rotated-filter kernel).  The
 * MMAs run in bf16 (or f16) with fp32 accumulation (tcgen05), so results equal
 * those of dgrad_depthwise up to fp32 summation order.
 * Requirements: DGRAD_BF16 or DGRAD_F16, stride 1, K == C, KH and KW <= 64,
 * 0 <= pad_h <= KH-1, 0 <= pad_w <= KW-1, N, H, W <= 65535; else
 * DGRAD_ERR_UNSUPPORTED (also when the filter is too large for the tile plan).
 * workspace: caller-owned device memory, 16-byte aligned, at least the size
 * dgrad_depthwise_tc_workspace reports; it holds dY and dX as per-channel planes
 * (channel-outermost copies of both); its contents on entry do not matter.
 * Three kernels run in order on `stream`: dY to planes, the tensor-core kernel,
 * planes to dX. */
dgrad_status_t dgrad_depthwise_tc(const dgrad_problem_t* prob, dgrad_dtype_t dtype, const void* dY, const void* W,
                                  void* dX, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes dgrad_depthwise_tc needs (0 for an empty batch); returns the
 * same refusals as dgrad_depthwise_tc for the problem (host only). */
dgrad_status_t dgrad_depthwise_tc_workspace(const dgrad_problem_t* prob, size_t* bytes);

/* ---- The residual branch around the gradients: x + dropout(f(layernorm(x))).
 * No counterpart on the pages: these are the operators a training program runs on
 * the same channel rows between its calls of the entry points above. Rows are the
 * N*H*W positions of an NHWC tensor (or tokens): M rows of C channels, dense.
 * Base pointers 16-byte aligned (fp32 statistics: 4-byte); unlike the gradients
 * above, layer norm and dropout take any C or n >= 1: rows that do not start on
 * 16 bytes run on the 16-byte vectors inside them and single elements at their ends
 * (rows too long for registers: on single elements).  Ranges an output shares with another
 * argument are refused (DGRAD_ERR_INVALID) except where one is named below.
 * Results repeat bit for bit: no atomics, sums in a fixed order, fp32 throughout
 * and one rounding to the element type at the end (the gated block's gradients: two, see
 * there).  M (or n) of 0 is a no-op, and
 * sets gradients that are sums over rows to zero. ---- */

/* Layer norm over C channels:
 *     mean = sum(x)/C,  rstd = 1/sqrt(sum((x - mean)^2)/C + eps),
 *     Y = (x - mean)*rstd*gamma + beta.
 * All element types (gamma, beta and Y have X's).  gamma or beta null: ones, zeros.
 * mean, rstd (fp32, M each, either may be null) are what the backward pass needs.
 * Y may be X.  eps finite and >= 0 (at eps 0 a constant row gives NaN, or what rounding
 * leaves of its differences).  C <= 65536, M < 2^31 (else DGRAD_ERR_UNSUPPORTED). */
dgrad_status_t dgrad_layernorm_forward(int64_t M, int64_t C, dgrad_dtype_t dtype, double eps, const void* X,
                                       const void* gamma, const void* beta, void* Y, float* mean, float* rstd,
                                       void* stream);

/* Its gradients, with n = (x - mean)*rstd and q = dY*gamma:
 *     dX = rstd*(q - sum(q)/C - n*sum(q*n)/C),
 *     dgamma = sum over rows of dY*n,  dbeta = sum over rows of dY.
 * dgamma or dbeta null: not computed.  dX may be dY or X.  workspace (16-byte
 * aligned, at least dgrad_layernorm_backward_workspace bytes; contents do not
 * matter and are clobbered) is needed when dgamma or dbeta is wanted; too small or
 * null then: DGRAD_ERR_INVALID.  Two calls that may overlap need a workspace each. */
dgrad_status_t dgrad_layernorm_backward(int64_t M, int64_t C, dgrad_dtype_t dtype, const void* dY, const void* X,
                                        const void* gamma, const float* mean, const float* rstd, void* dX,
                                        void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* Workspace bytes dgrad_layernorm_backward needs (host only, no CUDA call). */
dgrad_status_t dgrad_layernorm_backward_workspace(int64_t M, int64_t C, dgrad_dtype_t dtype, size_t* bytes);

/* The activations: silu g/(1 + exp(-g)); gelu g*P(g) with the normal
 * distribution P (exact) or its tanh form g*(1 + tanh(sqrt(2/pi)*(g + 0.044715 g^3)))/2;
 * relu max(g, 0); sigmoid 1/(1 + exp(-g)); none g (group norm only). */
typedef enum {
    DGRAD_ACT_SILU = 0, DGRAD_ACT_GELU = 1, DGRAD_ACT_GELU_TANH = 2, DGRAD_ACT_RELU = 3, DGRAD_ACT_SIGMOID = 4,
    DGRAD_ACT_NONE = 5
} dgrad_act_t;

/* Gated pointwise block in one kernel: two 1x1 projections of C to F channels, the
 * activation and the product,
 *     Z = [G | U] = X . W^T  (M x 2F),   H = act(G)*U  (M x F),
 * X [M][C], W [2F][C] (rows 0..F-1 the gate's, rows F..2F-1 the other projection's: a
 * pointwise filter with 2F output channels), H [M][F].  H comes from the fp32
 * accumulators.  Z [M][2F], rounded to the element type, is what the backward pass
 * takes; null: not kept.  DGRAD_BF16 or DGRAD_F16 (else DGRAD_ERR_UNSUPPORTED) on the
 * tcgen05 tensor cores; up to 32 rows run on kernels that stream W once.  C and F
 * multiples of 8 (else DGRAD_ERR_ALIGNMENT); C <= 65536, F <= 32768, M <= 2^30 (else
 * DGRAD_ERR_UNSUPPORTED).  H and Z overlap nothing. */
dgrad_status_t dgrad_gated_forward(int64_t M, int64_t C, int64_t F, dgrad_dtype_t dtype, dgrad_act_t act,
                                   const void* X, const void* W, void* H, void* Z, void* stream);

/* Its gradients from dH [M][F], X, the kept Z and W:
 *     dZ = [dH*U*act'(G) | dH*act(G)],   dX = dZ . W,   dW = dZ^T . X.
 * dX or dW null: not computed (X is then needed for dW only, W for dX only; both null:
 * DGRAD_ERR_INVALID).  dZ is computed in fp32 and rounded to the element type, the
 * operand type of both products (M*F <= 4096: it stays fp32); in f16 times a power of
 * two, undone in the fp32 sums, where its largest finite value lies beyond 65504 or below 2^-10
 * (values under 2^-29 of that one are then held to 2^-39 of it).  The rounding of dZ makes the
 * gradients' error about 1.4 times that of one rounding.  An infinite pre-activation (an f16 Z
 * that overflowed) gives NaN where the formulas multiply it by zero, as silu and both gelus do:
 * in its row of dX and its rows of dW.  Types and limits as dgrad_gated_forward.
 * workspace (16-byte aligned, at least dgrad_gated_backward_workspace bytes; contents
 * do not matter and are clobbered) holds dZ and fp32 partial sums; too small or null:
 * DGRAD_ERR_INVALID.  Two calls that may overlap need a workspace each.  dX, dW and
 * the workspace overlap nothing. */
dgrad_status_t dgrad_gated_backward(int64_t M, int64_t C, int64_t F, dgrad_dtype_t dtype, dgrad_act_t act,
                                    const void* dH, const void* X, const void* Z, const void* W, void* dX, void* dW,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes dgrad_gated_backward needs (host only, no CUDA call). */
dgrad_status_t dgrad_gated_backward_workspace(int64_t M, int64_t C, int64_t F, size_t* bytes);

/* Group norm over NHWC samples with an activation.  X is [N][S][C], S positions (H*W) of C
 * channels; a group is C/G adjacent channels of a sample at all positions, m = S*C/G values:
 *     mean = sum(x)/m,  rstd = 1/sqrt(sum((x - mean)^2)/m + eps),
 *     z = (x - mean)*rstd*gamma + beta,  Y = act(z).
 * All element types (gamma, beta [C] and Y have X's).  gamma or beta null: ones, zeros.
 * mean, rstd (fp32, [N][G] each, either may be null) are what the backward pass needs.
 * Y may be X.  eps finite and >= 0 (at eps 0 a constant group gives NaN).  G divides C (else
 * DGRAD_ERR_INVALID).  A group that holds an infinity or NaN becomes NaN, and so do its mean and rstd;
 * one whose squares pass fp32's range has rstd 0, and one whose sums do (m times its largest magnitude
 * 3.4e38 or more) has that or becomes NaN.  C <= 65536, N*S and N*G <= 2^30 (else
 * DGRAD_ERR_UNSUPPORTED).  N or S of 0: nothing but mean and rstd is
 * written, and those are NaN (sums over no values).  workspace: at least
 * dgrad_groupnorm_forward_workspace bytes (0 for sizes that need none; it may be null then), 16-byte
 * aligned, as for layer norm's gradients. */
dgrad_status_t dgrad_groupnorm_forward(int64_t N, int64_t S, int64_t C, int64_t G, dgrad_dtype_t dtype, double eps,
                                       dgrad_act_t act, const void* X, const void* gamma, const void* beta, void* Y,
                                       float* mean, float* rstd, void* workspace, size_t workspace_bytes,
                                       void* stream);

/* Its gradients, with n = (x - mean)*rstd, dz = dY*act'(z) and q = dz*gamma (z is formed again
 * from x, the statistics, gamma and beta):
 *     dX = rstd*(q - sum(q)/m - n*sum(q*n)/m) with the sums over the group,
 *     dgamma = sum over samples and positions of dz*n,  dbeta = the same of dz.
 * relu's derivative is 0 where z, every operation rounded to fp32 in the order
 * ((x - mean)*rstd)*gamma + beta, is 0.  dgamma or dbeta null: not computed.  dX may be dY or X.
 * N or S of 0: dgamma and dbeta are set to zero.  workspace: at least
 * dgrad_groupnorm_backward_workspace bytes.  Two calls that may overlap need a workspace each. */
dgrad_status_t dgrad_groupnorm_backward(int64_t N, int64_t S, int64_t C, int64_t G, dgrad_dtype_t dtype,
                                        dgrad_act_t act, const void* dY, const void* X, const void* gamma,
                                        const void* beta, const float* mean, const float* rstd, void* dX,
                                        void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* Workspace bytes the two need (host only, no CUDA call; 0 for N or S of 0). */
dgrad_status_t dgrad_groupnorm_forward_workspace(int64_t N, int64_t S, int64_t C, int64_t G, dgrad_dtype_t dtype,
                                                 size_t* bytes);
dgrad_status_t dgrad_groupnorm_backward_workspace(int64_t N, int64_t S, int64_t C, int64_t G, dgrad_dtype_t dtype,
                                                  size_t* bytes);

/* Dropout of n elements with no stored mask: Y = keep ? X*scale : 0, plus residual
 * when it is not null.  Element i of block b = i/8 draws 16 bits of Philox-4x32-10
 * (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) at counter
 * (low word of b, high word of b, low word of offset, high word of offset) and key
 * (low word of seed, high word of seed): word (i % 8)/2, its low half for even i.  It
 * is kept where the draw is >= t = round(65536*p) (ties to even) and scale is
 * 65536/(65536 - t); 0 <= p <= 1 is thus rounded to a multiple of 2^-16, and p = 1
 * drops everything, p <= 2^-17 nothing.  A dropped element does not enter the result (an
 * infinity or NaN in X leaves no trace there).  Give every call its own (seed, offset); the backward
 * pass takes its forward's.  Both are taken when the call is made: a call captured into a graph
 * draws the same mask in every replay.  All element types; Y may be X or residual. n <= 2^48. */
dgrad_status_t dgrad_dropout_forward(int64_t n, dgrad_dtype_t dtype, double p, uint64_t seed, uint64_t offset,
                                     const void* X, const void* residual, void* Y, void* stream);

/* Its gradient, dX = keep ? dY*scale : 0 (the residual's gradient is dY itself).
 * dX may be dY. */
dgrad_status_t dgrad_dropout_backward(int64_t n, dgrad_dtype_t dtype, double p, uint64_t seed, uint64_t offset,
                                      const void* dY, void* dX, void* stream);

/* ---- The optimizer's step over all parameters at once, and the norm of their gradients.
 * No counterpart on the pages.  Lists of tensors are host arrays, read while the call is
 * made: a call captured into a graph keeps its tensors' addresses.  Tensors of 0 elements are
 * allowed (their pointers are not looked at). Pointers are aligned to their elements; those on
 * 16 bytes (8-bit codes: 4) are read four elements at a time.  One launch takes up to 380
 * tensors (norms: 1600). ---- */

/* One tensor: param [n] of the parameters' type, grad [n] (null: the tensor is left as it is),
 * the states m and v, and an fp32 master copy (null: none; for all tensors or none).
 * 32-bit states: m, v fp32 [n]; m_max and v_max are not used.
 * 8-bit states: blocks of 256 elements share m_max and v_max (fp32, ceil(n/256) each); m holds
 * int8 codes -127 .. 127 for m = c|c|/127^2 m_max, v uint8 codes for v = (c/255)^4 v_max.  All
 * zero: a fresh state. */
typedef struct {
    void* param;
    const void* grad;
    void* m;
    void* v;
    float* master;
    float* m_max;
    float* v_max;
    int64_t n;
} dgrad_adamw_tensor_t;

/* A step's scalars.  step: t, counted from 1.  lr_device, step_device (one fp32, one int64; null:
 * lr and step): read by the kernels, so that a captured step follows them.  grad_scale (one
 * fp32 in device memory, null: 1): every gradient is multiplied by it; if it is no finite
 * number the step changes nothing (parameters, states and maxima).  state_bits: 32 or 8.
 * stochastic (8 bits only): codes are rounded by the random bits of (seed, offset), as below. */
typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;
    const float* lr_device;
    const int64_t* step_device;
    const float* grad_scale;
    int32_t state_bits, stochastic;
    uint64_t seed, offset;
} dgrad_adamw_t;

/* The AdamW step, with g = grad_scale*grad:
 *     m' = beta1 m + (1 - beta1) g,   v' = beta2 v + (1 - beta2) g g,
 *     p' = p (1 - lr weight_decay) - lr (m'/(1 - beta1^t)) / (sqrt(v'/(1 - beta2^t)) + eps),
 * (a t below 1 or an lr that is no finite number, read from device memory, leaves the step out as a
 * grad_scale does), all in fp32; p is the master copy where there is one (both are written), and is rounded once
 * to the parameter's type.  param_type: any; grad_type: the same or DGRAD_F32.
 * 8-bit states enter p' unrounded.  Their codes are defined by fp32 operations, each rounded
 * (in the order written: m' = beta1*m + (1-beta1)*g, v' = beta2*v + ((1-beta2)*g)*g), so that
 * they can be reproduced bit for bit: with M the block's largest |m'|, k = 2^64 where M < 2^-60,
 * 2^-64 where M > 2^60, else 1, and w = (|m'| k) ((1/(M k)) 127^2), low is the largest c with
 * c*c <= w, and c = low + 1 if (w - low^2) 65536 > ((low+1)^2 - low^2) draw, else low, at most
 * 127; draw is 32768 (the nearer value), or with `stochastic` 16 random bits.  v likewise with 255, c^4 = (c*c)*(c*c)
 * and V the largest v', where a v' above 0 has a code of at least 1.  The random bits are those
 * of Philox-4x32-10 at counter (b, offset), key seed (as for dropout): with every tensor rounded up to 256 elements,
 * element i of the whole list takes word i % 4 of b = i/4, the low half for m, the high half for v.
 * An infinity or NaN in a gradient makes the states of its 256 elements NaN (8 bits), or its own (32).
 * count 0: no-op.  beta1, beta2 in [0, 1); eps >= 0; finite scalars; step >= 1 (unless
 * step_device), else DGRAD_ERR_INVALID.  A master copy of fp32 parameters: DGRAD_ERR_UNSUPPORTED.
 * The written ranges must lie apart from each other and from the gradients; dgrad_adamw_check
 * looks at that, once for a list. */
dgrad_status_t dgrad_adamw_step(int64_t count, const dgrad_adamw_tensor_t* tensors, dgrad_dtype_t param_type,
                                dgrad_dtype_t grad_type, const dgrad_adamw_t* opt, void* stream);

/* Host only: the checks of dgrad_adamw_step on the tensors, and DGRAD_ERR_INVALID where a written
 * range shares a byte with another range of the list. */
dgrad_status_t dgrad_adamw_check(int64_t count, const dgrad_adamw_tensor_t* tensors, dgrad_dtype_t param_type,
                                 dgrad_dtype_t grad_type, int32_t state_bits);

/* What 8-bit states stand for: m_out[i], v_out[i] (host arrays of fp32 device pointers, n elements each,
 * apart from everything else), each operation rounded: m = ((c|c|) (1/127^2)) m_max,
 * v = (c^4 (1/255^4)) v_max. */
dgrad_status_t dgrad_adamw_moments(int64_t count, const dgrad_adamw_tensor_t* tensors, float* const* m_out,
                                   float* const* v_out, void* stream);

/* The norm over all elements of the tensors grads[i] (n[i] elements, one type):
 *     out[0] = sqrt(sum of squares),  out[1] = min(1, max_norm/(out[0] + 1e-6)),
 * fp32 in device memory; squares and sums are formed in 64 bits.  out[1] is the step's grad_scale;
 * it is NaN where the norm is no finite number, so that the step is left out.  max_norm >= 0 (it may be
 * infinite: out[1] = 1).  count 0: a norm of 0.  workspace: 16-byte aligned, at least
 * dgrad_grad_norm_workspace bytes; two calls that may overlap need one each. */
dgrad_status_t dgrad_grad_norm(int64_t count, const void* const* grads, const int64_t* n, dgrad_dtype_t dtype,
                               double max_norm, float* out, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes dgrad_grad_norm needs for a list of count tensors (host only). */
dgrad_status_t dgrad_grad_norm_workspace(int64_t count, size_t* bytes);

/* Output extents of the forward convolution the problem describes (host only,
 * no CUDA call).  Returns DGRAD_ERR_INVALID for an invalid problem. */
dgrad_status_t dgrad_out_dims(const dgrad_problem_t* prob, int64_t* Ho, int64_t* Wo);

/* Synchronise `stream`, then report (and clear) the device status word of the
 * current device: DGRAD_ERR_TIMEOUT if any kernel gave up waiting since the
 * last check, DGRAD_ERR_BOUNDS if (in the debug build, libdgrad_debug.so, built
 * from the same sources with -DDGRAD_DEBUG) a hand-indexed store fell outside
 * its output buffer and was skipped, DGRAD_ERR_CUDA if the stream reported an
 * error, else DGRAD_OK. */
dgrad_status_t dgrad_check_status(void* stream);

/* Static, human-readable text for a status code. */
const char* dgrad_status_string(dgrad_status_t status);

/* The last CUDA error code the library saw on this thread (0 if none). */
int dgrad_last_cuda_error(void);

/* ---- Diagnostics (no counterpart on the pages; they support testing and
 * measurement of the entry points above). ---- */

/* Enqueue one small kernel whose bounded wait is made to run out: it waits on a
 * barrier nothing completes for `limit_cycles` SM cycles (0 .. 2e9), then
 * records a timeout in the status word exactly as the dgrad kernels do and
 * returns.  dgrad_check_status then reports DGRAD_ERR_TIMEOUT and clears it.
 * Used to test the failure path without faulting or hanging the GPU. */
dgrad_status_t dgrad_selftest_timeout(long long limit_cycles, void* stream);

/* Enqueue an fp32 FMA-rate probe: `blocks` CTAs of 256 threads, each thread
 * running `iters` rounds of 16 independent FMAs (packed != 0: as 8 fma.rn.f32x2).
 * Work = blocks * 256 * iters * 16 FMAs.  `sink` is a device buffer of at least
 * `blocks` floats that keeps the work live (normally left untouched). */
dgrad_status_t dgrad_fma_probe(int blocks, int iters, int packed, float* sink, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DGRAD_H */
