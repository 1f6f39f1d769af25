/*
 * linear_amd.h -- C ABI of the MI355X (gfx950) FP16 linear layer.
 *
 *     proj[m,n] = FP16( sum_k x[m,k] * weight[n,k] )     products exact, FP32 accumulation
 *     y[m,n]    = FP16( FP32(proj[m,n]) + FP32(b[n]) )
 *
 * This is the computation and numerical contract of "tensor programs, part 1":
 * the PyTorch line y = torch.matmul(x, weight.T) + b and Figure 1.1 (the weight
 * transpose is a view, the projection is rounded before the bias add), the
 * contraction formula of section "One Program and One Numerical Contract" and its
 * two requirements (FP32 accumulation of unrounded products in any order; the
 * projection rounded to FP16 before the bias addition, output FP16), and the
 * Inductor capture's epilogue (both operands widened to f32, added, rounded to
 * f16).  The weight is contracted in its stored [N, K] order with no transposed or
 * widened copy, as "The Graph IR" op table describes a dense contraction
 * (DenseContraction).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Binary16 values are passed as uint16_t words (their IEEE 754 bit patterns).
 *  - x is [M, K] with row stride ldx >= K, weight is [N, K] with row stride
 *    ldw >= K (the [out_features, in_features] layout), y is [M, N] with row
 *    stride ldy >= N; strides are in elements, the inner stride is 1.  b is [N],
 *    contiguous.
 *  - All data pointers are DEVICE pointers owned by the caller.  The library
 *    neither allocates, frees nor keeps them after the call returns.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL means the default stream)
 *    and the call returns without synchronising.  Results are visible after the
 *    stream is synchronised.  A call enqueues kernel launches only (one or a few:
 *    a column split of a large GEMM, see linear_plan, the indexed call's routing
 *    pass, the parts of a gradient), no allocation, copy or memset, so it can be
 *    captured into a HIP graph (the first call of an epilogue program with an
 *    activation on a device excepted, see below).
 *  - Only y[m, n] for m < M, n < N is written; stride padding is never touched.
 *  - Rounding is IEEE round-to-nearest-even with subnormals kept (no flush to
 *    zero) and overflow to infinity; the empty sum (K == 0) is +0.
 *  - For given shapes, the bias call and the bias-less call use the same
 *    summation order, so y of the bias call equals FP16(FP32(p) + FP32(b)) where
 *    p is the bias-less result, bit for bit.  Reruns are bit-identical.
 *  - Every argument error is detected on the host before anything is enqueued;
 *    y is then untouched.  No exception or abort crosses this ABI.
 *  - Limits: M, N, K < 2^31; ldx, ldw < 2^22 and ldy < 2^31 elements.
 *    A launch holds fewer than 2^32 threads: outputs of more than 2^25 columns are
 *    computed in parts, and a call that needs a larger launch all the same (some 2^29
 *    rows) returns LINEAR_E_LAUNCH.
 *  - Fast path: x and weight 16-byte aligned, ldx, ldw and K multiples of 8.
 *    Any other layout is accepted and runs a slower element-wise loader.
 */
#ifndef LINEAR_AMD_H
#define LINEAR_AMD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Status codes.  Every entry point returns one: a call the library cannot run is
 * refused with a typed error before anything is enqueued, never a crash or an
 * abort, as the pages' builder refuses ill-formed ops with a typed error rather
 * than a panic ("Tracing a Model", section "The Builder and Traced handles";
 * "The Graph IR", section "Graph structure": shapes and dtypes are checked when
 * an op is added).
 */
#define LINEAR_OK         0
#define LINEAR_E_NULL     1  /* a required pointer is NULL (only when the output is non-empty) */
#define LINEAR_E_SHAPE    2  /* M, N or K negative, or beyond the limits above */
#define LINEAR_E_STRIDE   3  /* ldx < K, ldw < K, ldy < N, or a stride beyond its limit */
#define LINEAR_E_ALIAS    4  /* y's byte range overlaps x, weight or b */
#define LINEAR_E_PATH     5  /* unknown path selector */
#define LINEAR_E_DEVICE   6  /* no usable gfx950 device current, or a HIP query failed */
#define LINEAR_E_LAUNCH   7  /* a kernel launch failed; linear_last_hip_error() has the HIP code */
#define LINEAR_E_EPILOGUE 8  /* epilogue program: step count outside 0..LINEAR_EPI_MAX_STEPS or an unknown step */
#define LINEAR_E_CAPTURE  9  /* the first activation epilogue on a device was called under stream capture */
#define LINEAR_E_WORKSPACE 10 /* workspace misaligned or smaller than the call's linear_*_workspace_bytes */
#define LINEAR_E_SCRATCH  11  /* linear_f16_indexed_noalloc: the call needs more than LINEAR_NOALLOC_SCRATCH_BYTES */
#define LINEAR_E_VALUE    12  /* unknown activation or tensor type, or a negative or NaN max_norm */
#define LINEAR_E_MEMORY   13  /* linear_grad_clip: no host memory for the overlap check */

/*
 * Path selectors for linear_f16_ex / linear_f16_plan.  The path and the tile are
 * chosen on the host from the static shapes before any launch: the op table
 * treats GEMV and GEMM as one MatMul op specialised when the call is planned, and
 * shapes are inferred on the host ("The Graph IR", op table, MatMul row, and
 * section "Host-side shape inference").  AUTO is that specialisation; the forced
 * paths give results within the same contract.
 */
#define LINEAR_PATH_AUTO   0  /* M <= 16: skinny path; otherwise the MFMA tiled GEMM */
#define LINEAR_PATH_GEMM   1  /* force the MFMA tiled GEMM (any M) */
#define LINEAR_PATH_SKINNY 2  /* force the weight-streaming skinny path (any M, 16 rows per block;
                                 at M == 1 with the fast-path layout, no epilogue program, one group
                                 and K <= 32768: one wave per weight row, 4 rows per block) */

/*
 * y = FP16(FP16(x . weight^T) + b).  See the conventions above.
 * M == 0 or N == 0 is a successful no-op (pointers may then be NULL).
 * Returns LINEAR_OK or one of the LINEAR_E_* codes.
 */
int32_t linear_f16(const uint16_t* x, int64_t ldx,
                   const uint16_t* weight, int64_t ldw,
                   const uint16_t* b,
                   uint16_t* y, int64_t ldy,
                   int64_t M, int64_t N, int64_t K,
                   void* stream);

/*
 * The projection alone: y = FP16(x . weight^T), no bias.  Same conventions.
 */
int32_t linear_f16_nobias(const uint16_t* x, int64_t ldx,
                          const uint16_t* weight, int64_t ldw,
                          uint16_t* y, int64_t ldy,
                          int64_t M, int64_t N, int64_t K,
                          void* stream);

/*
 * linear_f16 with an explicit path (LINEAR_PATH_*) and an optional bias
 * (b == NULL computes the projection alone).  Every path gives results within
 * the same contract; forcing one lets tests exercise both on every shape.
 */
int32_t linear_f16_ex(const uint16_t* x, int64_t ldx,
                      const uint16_t* weight, int64_t ldw,
                      const uint16_t* b,
                      uint16_t* y, int64_t ldy,
                      int64_t M, int64_t N, int64_t K,
                      int32_t path, void* stream);

/*
 * The unrounded FP32 sums: y[m,n] = sum_k x[m,k] * weight[n,k] accumulated in FP32
 * (products exact), stored as float with row stride ldy (elements).  No rounding,
 * no bias.  This is the op table's DenseContraction with an f32 output ("The
 * Graph IR", op table) and the rank-local partial product that a K-split tensor
 * parallel layer all-reduces before rounding and adding the bias ("Model and
 * Distributed IR", section "Boundary between the layers"; rounding per rank would
 * break the projection-rounding requirement).  Same conventions otherwise; path
 * as in linear_f16_ex.  Fast path additionally needs y 16-byte aligned.
 */
int32_t linear_f16_f32out(const uint16_t* x, int64_t ldx,
                          const uint16_t* weight, int64_t ldw,
                          float* y, int64_t ldy,
                          int64_t M, int64_t N, int64_t K,
                          int32_t path, void* stream);

/*
 * The same layer with bfloat16 x, weight, b and y (words are the upper halves of
 * binary32): FP32 accumulation, the projection rounded to bfloat16 (round to
 * nearest even) before the bias, then y = BF16(FP32(proj) + FP32(b[n])).  This
 * is the BF16 form of the contraction epilogue ("The Graph IR", op table:
 * ContractionEpilogue, a BF16 head rounds to BF16 before the first epilogue step;
 * Cast to bf16 rounds to bf16 precision).  bfloat16 x bfloat16 products are exact
 * in FP32 unless they leave its normal range.  Conventions, status codes, paths
 * and limits as for the binary16 entry points.
 */
int32_t linear_bf16(const uint16_t* x, int64_t ldx,
                    const uint16_t* weight, int64_t ldw,
                    const uint16_t* b,
                    uint16_t* y, int64_t ldy,
                    int64_t M, int64_t N, int64_t K,
                    void* stream);

int32_t linear_bf16_nobias(const uint16_t* x, int64_t ldx,
                           const uint16_t* weight, int64_t ldw,
                           uint16_t* y, int64_t ldy,
                           int64_t M, int64_t N, int64_t K,
                           void* stream);

int32_t linear_bf16_ex(const uint16_t* x, int64_t ldx,
                       const uint16_t* weight, int64_t ldw,
                       const uint16_t* b,
                       uint16_t* y, int64_t ldy,
                       int64_t M, int64_t N, int64_t K,
                       int32_t path, void* stream);

/* The unrounded FP32 sums for bfloat16 operands (see linear_f16_f32out). */
int32_t linear_bf16_f32out(const uint16_t* x, int64_t ldx,
                           const uint16_t* weight, int64_t ldw,
                           float* y, int64_t ldy,
                           int64_t M, int64_t N, int64_t K,
                           int32_t path, void* stream);

/*
 * Multi-step contraction epilogue ("The Graph IR", op table: ContractionEpilogue,
 * whose extra inputs are the bias, a residual and so on: the head contraction's
 * result keeps its dtype and every step rounds through it), with the activation
 * compositions of "Tracing a Model" (the gated feed-forward section: SiLU as
 * x / (1 + exp(-x)) over Neg, Exp, Add and Div; the tanh GeLU in the same
 * sigmoid form, x / (1 + exp(-2 sqrt(2/pi) (x + 0.044715 x^3))); the exact GeLU
 * (x (1 + erf(x / sqrt 2))) * 0.5 on the Erf primitive).
 *
 *     t = RNE_E( sum_k x[m,k] * weight[n,k] )          the projection, as linear_*_nobias
 *     for each step s: t = step_s(t)                    each result rounded to E
 *     y[m,n] = t
 *
 * Steps (op[s]):
 *   LINEAR_EPI_BIAS       t + bias[n]
 *   LINEAR_EPI_RESIDUAL   t + residual[m * ldr + n]
 *   LINEAR_EPI_MUL        t * mul[m * ldm + n]     (the gate product of a gated feed-forward)
 *   LINEAR_EPI_SILU, LINEAR_EPI_GELU_TANH, LINEAR_EPI_GELU_ERF
 * Every primitive of a step (each Add, Mul, Div, Neg, Exp, Erf of a composition,
 * left to right, x^3 as (x*x)*x) returns its exact result rounded to E, round to
 * nearest even; the constants 1, 0.5, 0.044715, -2 sqrt(2/pi) and 1/sqrt 2 are
 * E values (their real value rounded to E).  IEEE special values propagate
 * (e.g. SiLU of -inf is NaN: -inf / inf).
 *
 * bias, residual and mul are device words of the call's element type, caller
 * owned; each is read only by the steps that name it and may be NULL otherwise.
 * y may be the residual itself (same pointer, ldr == ldy: y = ... + y in place);
 * any other overlap of y with an input is LINEAR_E_ALIAS.  The program is read
 * when the call is made (the struct may be reused right after the call returns).
 * The activation steps use tables the library builds on the device at the first
 * such call per device and element type: that call waits for the build on
 * `stream`, and made under stream capture it returns LINEAR_E_CAPTURE with
 * nothing enqueued.  With no steps the call is linear_*_nobias; with the single
 * step LINEAR_EPI_BIAS it gives the bits of linear_*.
 */
#define LINEAR_EPI_MAX_STEPS 8
#define LINEAR_EPI_BIAS      1
#define LINEAR_EPI_RESIDUAL  2
#define LINEAR_EPI_MUL       3
#define LINEAR_EPI_SILU      4
#define LINEAR_EPI_GELU_TANH 5
#define LINEAR_EPI_GELU_ERF  6

typedef struct linear_epilogue {
    int32_t nsteps;                        /* 0 .. LINEAR_EPI_MAX_STEPS */
    int32_t op[LINEAR_EPI_MAX_STEPS];      /* LINEAR_EPI_*, applied in index order */
    const uint16_t* bias;                  /* [N] */
    const uint16_t* residual;              /* [M, N], row stride ldr >= N */
    int64_t ldr;
    const uint16_t* mul;                   /* [M, N], row stride ldm >= N */
    int64_t ldm;
} linear_epilogue;

int32_t linear_f16_epilogue(const uint16_t* x, int64_t ldx,
                            const uint16_t* weight, int64_t ldw,
                            const linear_epilogue* epilogue,
                            uint16_t* y, int64_t ldy,
                            int64_t M, int64_t N, int64_t K,
                            int32_t path, void* stream);

/* The same with bfloat16 x, weight, epilogue inputs and y. */
int32_t linear_bf16_epilogue(const uint16_t* x, int64_t ldx,
                             const uint16_t* weight, int64_t ldw,
                             const linear_epilogue* epilogue,
                             uint16_t* y, int64_t ldy,
                             int64_t M, int64_t N, int64_t K,
                             int32_t path, void* stream);

/*
 * Grouped contraction ("The Graph IR", op table: GroupedDenseContraction): a
 * [G*N, K] weight read in place as G blocks of N rows against a [G, M, K]
 * activation, giving [G, M, N]:
 *
 *     y[g, m, n] = RNE_E( sum_k x[g, m, k] * weight[g*N + n, k] )   (+ b[g*N + n] as in linear_*)
 *
 * x: group g at x + g * sx, rows with stride ldx (sx in elements, >= 0; slices may
 * overlap, they are only read); weight: [G*N, K] with row stride ldw; b: [G*N] or
 * NULL (NULL: the projection alone); y: group g at y + g * sy, row stride ldy,
 * sy >= (M-1)*ldy + N so that groups write disjoint outputs.  Element type,
 * rounding, bias epilogue, paths, reruns and errors as for linear_f16_ex (G up to
 * 65535); each group is exactly linear_f16_ex on its slices.  The _f32out forms
 * return the unrounded FP32 sums (the op table gives this contraction an f32
 * output).  The op table's f32 activation is read here in the weight's element
 * type: the MFMA path multiplies 16-bit operands.
 */
int32_t linear_f16_grouped(const uint16_t* x, int64_t ldx, int64_t sx,
                           const uint16_t* weight, int64_t ldw,
                           const uint16_t* b,
                           uint16_t* y, int64_t ldy, int64_t sy,
                           int64_t G, int64_t M, int64_t N, int64_t K,
                           int32_t path, void* stream);
int32_t linear_bf16_grouped(const uint16_t* x, int64_t ldx, int64_t sx,
                            const uint16_t* weight, int64_t ldw,
                            const uint16_t* b,
                            uint16_t* y, int64_t ldy, int64_t sy,
                            int64_t G, int64_t M, int64_t N, int64_t K,
                            int32_t path, void* stream);
int32_t linear_f16_grouped_f32out(const uint16_t* x, int64_t ldx, int64_t sx,
                                  const uint16_t* weight, int64_t ldw,
                                  float* y, int64_t ldy, int64_t sy,
                                  int64_t G, int64_t M, int64_t N, int64_t K,
                                  int32_t path, void* stream);
int32_t linear_bf16_grouped_f32out(const uint16_t* x, int64_t ldx, int64_t sx,
                                   const uint16_t* weight, int64_t ldw,
                                   float* y, int64_t ldy, int64_t sy,
                                   int64_t G, int64_t M, int64_t N, int64_t K,
                                   int32_t path, void* stream);

/*
 * Indexed contraction ("The Graph IR", op table: IndexedMatMul; "Tracing a
 * Model", section "Mixture-of-experts routing": each row contracts against its
 * own expert, the expert tables read in place):
 *
 *     y[m, n] = RNE_E( sum_k x[m, k] * w[idx[m], k, n] )      (FP32 accumulation)
 *
 * x: [M, K], row stride ldx >= K.  w: E expert tables of [K, N] (k first, n
 * contiguous): element (e, k, n) at w[e * sw + k * ldw + n], ldw >= N,
 * sw >= K * ldw.  idx: [M] device int32.  y: [M, N], row stride ldy >= N.  A row
 * whose idx lies outside [0, E) has no expert and its outputs are left untouched.
 * Only rows m < M and columns n < N are written; reruns are bit-identical.
 * E up to 65535; M, N, K < 2^31.  The _f32out forms store the unrounded sums.
 *
 * workspace: device memory of at least linear_indexed_workspace_bytes(E, M)
 * bytes, 16-byte aligned, owned by the caller, overwritten by the call (it holds
 * the row-to-expert binning) and free again once the call's work on `stream`
 * has finished; two calls in flight at once need two workspaces.
 *
 * Errors as for linear_f16_ex (y or the workspace overlapping x, w, idx or each
 * other is LINEAR_E_ALIAS; a NULL workspace is LINEAR_E_NULL, a short or
 * misaligned one LINEAR_E_WORKSPACE); E == 0, M == 0 or N == 0 is a successful
 * no-op that touches nothing.
 */
int64_t linear_indexed_workspace_bytes(int64_t E, int64_t M);   /* -1 if E or M is out of range */
int32_t linear_f16_indexed(const uint16_t* x, int64_t ldx,
                           const uint16_t* w, int64_t ldw, int64_t sw,
                           const int32_t* idx,
                           uint16_t* y, int64_t ldy,
                           int64_t E, int64_t M, int64_t N, int64_t K,
                           void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_bf16_indexed(const uint16_t* x, int64_t ldx,
                            const uint16_t* w, int64_t ldw, int64_t sw,
                            const int32_t* idx,
                            uint16_t* y, int64_t ldy,
                            int64_t E, int64_t M, int64_t N, int64_t K,
                            void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_f16_indexed_f32out(const uint16_t* x, int64_t ldx,
                                  const uint16_t* w, int64_t ldw, int64_t sw,
                                  const int32_t* idx,
                                  float* y, int64_t ldy,
                                  int64_t E, int64_t M, int64_t N, int64_t K,
                                  void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_bf16_indexed_f32out(const uint16_t* x, int64_t ldx,
                                   const uint16_t* w, int64_t ldw, int64_t sw,
                                   const int32_t* idx,
                                   float* y, int64_t ldy,
                                   int64_t E, int64_t M, int64_t N, int64_t K,
                                   void* workspace, int64_t workspace_bytes, void* stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): linear_f16_indexed
 * without the workspace argument.  Same arguments otherwise, same kernels, same
 * results bit for bit, same errors, except that the row-to-expert binning goes
 * into a scratch array of LINEAR_NOALLOC_SCRATCH_BYTES that the library holds in
 * device memory (one per GPU, from the first such call on that GPU until the
 * process ends).  A call whose binning needs more, i.e.
 * linear_indexed_workspace_bytes(E, M) > LINEAR_NOALLOC_SCRATCH_BYTES (about
 * 200,000 rows at a few experts), returns LINEAR_E_SCRATCH with nothing
 * enqueued.  The call allocates nothing and frees nothing; nothing in the
 * scratch array needs clearing between calls (each call's routing pass writes
 * every word its kernels read).  All such calls on one GPU share that GPU's
 * array: two of them in flight at once on that GPU (on different streams, or
 * captured graphs replayed concurrently) race and may give wrong results; calls
 * in one stream's order are safe.
 */
#define LINEAR_NOALLOC_SCRATCH_BYTES (1 << 20)
int32_t linear_f16_indexed_noalloc(const uint16_t* x, int64_t ldx,
                                   const uint16_t* w, int64_t ldw, int64_t sw,
                                   const int32_t* idx,
                                   uint16_t* y, int64_t ldy,
                                   int64_t E, int64_t M, int64_t N, int64_t K,
                                   void* stream);

/*
 * The gated feed-forward block: both projections, the activation and the product
 * ("Tracing a Model", the gated feed-forward section), in one kernel:
 *
 *     g[m, n] = sum_k x[m, k] * wg[n, k]        u[m, n] = sum_k x[m, k] * wu[n, k]
 *     h[m, n] = RNE_E( act(g[m, n]) * u[m, n] )
 *
 * act: LINEAR_EPI_SILU, LINEAR_EPI_GELU_TANH or LINEAR_EPI_GELU_ERF (any other
 * code is LINEAR_E_VALUE).  The sums are FP32; the activation and the product are
 * taken in FP32 on the unrounded sums and rounded once (unlike an epilogue
 * program, whose every primitive rounds to E).  exp, erfc and the reciprocal are
 * FP32 approximations within a few FP32 ulps.
 *
 * x: [M, K]; wg, wu: [N, K] each with its own row stride (the two halves of one
 * [2N, K] weight are wg = w, wu = w + N * ldw).  h: [M, N].  gate and up: [M, N]
 * or NULL; where given, RNE_E(g) and RNE_E(u) are stored there for the backward
 * call.  Outputs may not overlap the inputs or each other (LINEAR_E_ALIAS); columns
 * of their own in rows of one stride do not (gate and up in one [M, 2N] matrix).
 * M == 0 or N == 0 is a no-op; K == 0 gives +0 (act(0) * 0).  M, N and K of this
 * and the gradients' calls are at most 2^31 - 65536, row strides below 2^31.
 *
 * workspace: linear_gated_forward_workspace_bytes(M, N, K) bytes of device memory,
 * 16-byte aligned, owned by the caller, overwritten, free again once the call's work
 * on `stream` has finished (two calls in flight at once need two).  It is 0 (and workspace may be NULL) where K is a multiple
 * of 8 and for a few rows; otherwise it holds copies of the operands with padded rows.
 */
int64_t linear_gated_forward_workspace_bytes(int64_t M, int64_t N, int64_t K);   /* -1 if out of range */
int32_t linear_f16_gated(const uint16_t* x, int64_t ldx,
                         const uint16_t* wg, int64_t ldwg,
                         const uint16_t* wu, int64_t ldwu,
                         int32_t act,
                         uint16_t* h, int64_t ldh,
                         uint16_t* gate, int64_t ldgate,
                         uint16_t* up, int64_t ldup,
                         int64_t M, int64_t N, int64_t K,
                         void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_bf16_gated(const uint16_t* x, int64_t ldx,
                          const uint16_t* wg, int64_t ldwg,
                          const uint16_t* wu, int64_t ldwu,
                          int32_t act,
                          uint16_t* h, int64_t ldh,
                          uint16_t* gate, int64_t ldgate,
                          uint16_t* up, int64_t ldup,
                          int64_t M, int64_t N, int64_t K,
                          void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The gated block's gradients, from dh [M, N] and the projections gate and up
 * [M, N] that the forward call stored:
 *
 *     dg = RNE_E( c * dh * u * act'(g) ) / c     du = RNE_E( c * dh * act(g) ) / c      (FP32 inside)
 *     dx[m, k]  = RNE_E( sum_n dg[m, n] * wg[n, k] + du[m, n] * wu[n, k] )
 *     dwg[n, k] = RNE_E( sum_m dg[m, n] * x[m, k] )      dwu likewise from du
 *
 * dg and du are rounded to E because they are the matrix unit's operands (up to 32
 * rows they are kept as two words, so that only the outputs' own rounding is left).
 * In bfloat16 c is 1.  In binary16 c is the power of two that brings the largest
 * finite |dg| or |du| of the call to 2^14 .. 2^15, and the products' FP32 sums are
 * divided by it: whatever the gradients' size none overflows, and those down to 2^-28
 * of the largest keep the type's relative precision (smaller ones are off by up to
 * 2^-39 of the largest).
 *
 * dx may be NULL (not wanted; the weights are then not read), and dwg and dwu may both
 * be NULL (x is then not read); one of the two groups must be given, unless M or N is
 * 0.  N == 0 gives dx = +0, M == 0 gives dwg = dwu = +0.  N is at most 2^30 - 64 (dg and
 * du share rows).  Fast path of dx: both weights with one row stride (16-byte aligned,
 * as everywhere); weights of two strides run the slower element-wise loader.
 *
 * workspace: linear_gated_workspace_bytes(M, N, K) bytes of device memory (it
 * holds dg and du, partial sums, and copies of operands of odd widths), 16-byte
 * aligned, owned by the caller, overwritten, free again once the call's work on
 * `stream` has finished; two calls in flight at once need two workspaces.  It may
 * not overlap any other argument.
 */
int64_t linear_gated_workspace_bytes(int64_t M, int64_t N, int64_t K);   /* -1 if out of range */
int32_t linear_f16_gated_backward(const uint16_t* dh, int64_t lddh,
                                  const uint16_t* x, int64_t ldx,
                                  const uint16_t* wg, int64_t ldwg,
                                  const uint16_t* wu, int64_t ldwu,
                                  const uint16_t* gate, int64_t ldgate,
                                  const uint16_t* up, int64_t ldup,
                                  int32_t act,
                                  uint16_t* dx, int64_t lddx,
                                  uint16_t* dwg, int64_t lddwg,
                                  uint16_t* dwu, int64_t lddwu,
                                  int64_t M, int64_t N, int64_t K,
                                  void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_bf16_gated_backward(const uint16_t* dh, int64_t lddh,
                                   const uint16_t* x, int64_t ldx,
                                   const uint16_t* wg, int64_t ldwg,
                                   const uint16_t* wu, int64_t ldwu,
                                   const uint16_t* gate, int64_t ldgate,
                                   const uint16_t* up, int64_t ldup,
                                   int32_t act,
                                   uint16_t* dx, int64_t lddx,
                                   uint16_t* dwg, int64_t lddwg,
                                   uint16_t* dwu, int64_t lddwu,
                                   int64_t M, int64_t N, int64_t K,
                                   void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The layer's gradients, from dy [M, N]:
 *
 *     _backward_input:   dx[m, k] = RNE_E( sum_n dy[m, n] * weight[n, k] )
 *     _backward_weight:  dw[n, k] = RNE_E( sum_m dy[m, n] * x[m, k] )
 *                        db[n]    = RNE_E( sum_m dy[m, n] )         (db may be NULL)
 *
 * FP32 sums, rounded once; operands are read in place, no transposed copies.
 * The projection's rounding and the bias addition's are taken as the identity,
 * as usual for gradients.  The _f32out forms store the unrounded FP32 sums in dw
 * and db (floats), or with accumulate != 0 add them to what dw and db hold
 * (gradients summed over several batches).  N == 0 gives dx = +0; M == 0 gives
 * dw = db = +0 (or leaves them, when accumulating).  Reruns are bit-identical.
 * The matrix unit aligns a product by its words' exponents, and a binary16 subnormal's
 * is that of 2^-14: sums of products with subnormal words are as precise as if those
 * words' magnitude were 2^-14, which only the _f32out forms can show.
 *
 * workspace: linear_backward_workspace_bytes(M, N, K) bytes of device memory for
 * any of these calls, 16-byte aligned; ownership and overlaps as for the gated
 * block's.
 */
int64_t linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);   /* -1 if out of range */
int32_t linear_f16_backward_input(const uint16_t* dy, int64_t lddy,
                                  const uint16_t* weight, int64_t ldw,
                                  uint16_t* dx, int64_t lddx,
                                  int64_t M, int64_t N, int64_t K,
                                  void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_bf16_backward_input(const uint16_t* dy, int64_t lddy,
                                   const uint16_t* weight, int64_t ldw,
                                   uint16_t* dx, int64_t lddx,
                                   int64_t M, int64_t N, int64_t K,
                                   void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_f16_backward_weight(const uint16_t* dy, int64_t lddy,
                                   const uint16_t* x, int64_t ldx,
                                   uint16_t* dw, int64_t lddw, uint16_t* db,
                                   int64_t M, int64_t N, int64_t K,
                                   void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_bf16_backward_weight(const uint16_t* dy, int64_t lddy,
                                    const uint16_t* x, int64_t ldx,
                                    uint16_t* dw, int64_t lddw, uint16_t* db,
                                    int64_t M, int64_t N, int64_t K,
                                    void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_f16_backward_weight_f32out(const uint16_t* dy, int64_t lddy,
                                          const uint16_t* x, int64_t ldx,
                                          float* dw, int64_t lddw, float* db, int32_t accumulate,
                                          int64_t M, int64_t N, int64_t K,
                                          void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_bf16_backward_weight_f32out(const uint16_t* dy, int64_t lddy,
                                           const uint16_t* x, int64_t ldx,
                                           float* dw, int64_t lddw, float* db, int32_t accumulate,
                                           int64_t M, int64_t N, int64_t K,
                                           void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The global norm of a set of gradients, and clipping by it.
 *
 *     linear_grad_norm:  norm[0] = FP32( sqrt( sum over all tensors and elements of g^2 ) )
 *     linear_grad_clip:  out = RNE( g * s ),  s = min(1, max_norm / (norm[0] + 1e-6)) in FP32
 *
 * Squares are taken and summed in FP64 in a fixed order, so the sum of finite
 * gradients does not overflow and reruns are bit-identical; the norm itself does where
 * it passes FLT_MAX.  A NaN norm makes every output NaN; an infinite one (an infinite
 * gradient, or finite ones past FLT_MAX together) makes s zero, so finite gradients
 * zero and infinite ones NaN, or, with an infinite max_norm, every output NaN.  The two calls are apart so
 * that a sharded caller can combine norms in between.
 *
 * Tensors are [rows, cols] with row stride ld (elements; a vector is one row, whose
 * ld is not read), of any mix of types, any alignment; cols up to 2^46, rows and ld
 * below 2^31.  The arrays of linear_tensor are host memory, read during the call.
 * out == NULL clips in place; else out[i] has grads[i]'s shape and type and is
 * grads[i] itself or overlaps no tensor of the call (LINEAR_E_ALIAS, judged by the
 * range from a tensor's first word to its last: columns of one matrix overlap); a
 * tensor listed twice may not be clipped in place.  norm is device memory.  count up to
 * LINEAR_GRAD_MAX_TENSORS; count == 0 gives norm 0.  max_norm: not negative or NaN
 * (LINEAR_E_VALUE).
 *
 * workspace of linear_grad_norm: linear_grad_workspace_bytes(count) bytes, 16-byte
 * aligned, as above.
 */
#define LINEAR_TYPE_F16  0
#define LINEAR_TYPE_BF16 1
#define LINEAR_TYPE_F32  2
#define LINEAR_GRAD_MAX_TENSORS 65536

typedef struct linear_tensor {
    void* data;
    int64_t rows, cols, ld;
    int64_t type;            /* LINEAR_TYPE_* */
} linear_tensor;

int64_t linear_grad_workspace_bytes(int64_t count);   /* -1 if out of range */
int32_t linear_grad_norm(const linear_tensor* grads, int64_t count, float* norm,
                         void* workspace, int64_t workspace_bytes, void* stream);
int32_t linear_grad_clip(const linear_tensor* grads, const linear_tensor* out, int64_t count,
                         const float* norm, float max_norm, void* stream);

/* Which kernels a call would launch: the host-side plan of "The Graph IR" (op
 * table, MatMul row: GEMV versus GEMM chosen at plan time; section "Host-side
 * shape inference").  Enqueues nothing and touches no device memory; the tile
 * rules count the compute units of the current device when a gfx950 is current
 * (a partitioned part has fewer), else those of a whole MI355X (256).
 * A GEMM call whose largest tiles would leave a last wave of workgroups at most
 * half full over the GPU's CUs is split by output columns into two launches of
 * the same kernel family: columns [0, split_n) in whole waves of the first tile,
 * columns [split_n, N) with the tile chosen for that part alone. */
typedef struct linear_plan {
    int32_t path;       /* LINEAR_PATH_GEMM or LINEAR_PATH_SKINNY */
    int32_t tile_m;     /* output rows (m) per workgroup */
    int32_t tile_n;     /* output columns (n) per workgroup */
    int32_t tile_k;     /* K elements per main-loop stage (GEMM), per wave step (skinny) or per wave
                           load (skinny at M == 1: tile_m 1, tile_n 4) */
    int32_t threads;    /* threads per workgroup */
    int32_t vector_io;  /* 1: 16-byte loads; 0: element-wise loader */
    int64_t grid;       /* workgroups launched (the first launch when split) */
    int64_t split_n;    /* 0: one launch; else the first column of the second launch */
    int32_t tile_m2;    /* the second launch's tile (0 when not split) */
    int32_t tile_n2;
    int64_t grid2;      /* the second launch's workgroups (0 when not split) */
    int32_t stages;     /* GEMM: slices of tile_k K in its LDS ring (0 for the skinny path) */
} linear_plan;

/*
 * Fill *plan for a call with these shapes, strides, alignments and path, after
 * the same validation as linear_f16_ex (device pointers are only inspected for
 * alignment, never dereferenced).  Returns LINEAR_OK or a LINEAR_E_* code.
 */
int32_t linear_f16_plan(const uint16_t* x, int64_t ldx,
                        const uint16_t* weight, int64_t ldw,
                        const uint16_t* b,
                        uint16_t* y, int64_t ldy,
                        int64_t M, int64_t N, int64_t K,
                        int32_t path, linear_plan* plan);

/*
 * How a gated backward call of these sizes forms its products (host only, 16-byte
 * aligned layouts; it depends on the sizes alone): the tiles of dx and of the pair dwg,
 * dwu, the sets of workgroups that share a contraction (splits), and, where the output
 * columns from split_c on are a second launch, that launch's tile.  joint: both
 * products run in one launch.  Returns LINEAR_OK, LINEAR_E_SHAPE or LINEAR_E_NULL.
 */
typedef struct linear_product_plan {
    int32_t tile_m, tile_n;   /* output rows and columns per workgroup */
    int32_t stages;           /* slices of 64 contraction indices in a workgroup's LDS ring */
    int32_t sets;             /* sets of waves that share a tile's slices */
    int32_t splits;
    int32_t tile_m2, tile_n2; /* the second launch's tile (0: one launch) */
    int64_t split_c;          /* its first column (0: one launch) */
} linear_product_plan;
typedef struct linear_gated_plan {
    linear_product_plan dx, dw;
    int32_t joint;
    int32_t two_words;        /* dg and du are kept as two words each (up to 32 rows) */
} linear_gated_plan;
int32_t linear_gated_backward_plan(int64_t M, int64_t N, int64_t K, linear_gated_plan* plan);

/* Static English text for a status code (never NULL). */
const char* linear_status_string(int32_t status);

/* The hipError_t of the last LINEAR_E_DEVICE / LINEAR_E_LAUNCH on this thread (0 if none). */
int32_t linear_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_AMD_H */
