/*
 * t3.h -- C ABI of the ternary-weight x int8 GEMM library for GB300 (sm_103a).
 *
 * Three integer products of a ternary-weight layer and the packer of its
 * weights.  All results are exact int32; there is no rounding, no scale and no
 * tolerance on this path.
 *
 * Sources (web pages, cited by title and section):
 *   [fwd] "t27c PTX backend: ternary x int8 GEMM kernel emitted by a .t27 spec
 *         (int8 mma.sync), ptx-run glue", section "What this adds": C = A x W
 *         with int8 A and ternary W held as 2-bit codes, each decoded as
 *         (c & 1) - ((c >> 1) & 1), i.e. 0 -> 0, 1 -> +1, 2 -> -1, 3 -> 0.
 *   [bwd] "spec(igla): hslm_bwd_ptx -- HSLM backward dX and dW as int8
 *         tensor-core PTX written by t27", kernel 1 (dX = dY x W^T, W ternary
 *         in the same code layout) and kernel 2 (dW = X^T x dY summed over
 *         rows, int32 accumulation, reduction length <= 131071).
 *
 * Layouts (all row-major and densely packed, no row padding):
 *   A  int8  [M][K]          activations
 *   Wp uint8 [N][ceil(K/4)]  packed weights: the code of W[k][n] is at bits
 *                            2*(k%4) of byte k/4 of row n; positions k >= K of
 *                            the last byte of a row are ignored by every call.
 *   C  int32 [M][N]          forward output
 *   dY int8  [M][N]          output gradient
 *   dX int32 [M][K]          input gradient
 *   dW int32 [K][N]          weight gradient
 *
 * Ownership and threading:
 *   - The caller owns every buffer.  The GEMM calls take DEVICE pointers (any
 *     memory the current device can read/write), enqueue their work on
 *     `stream` and return without waiting; the results are ready once the
 *     stream reaches that point.  The library allocates no device memory per
 *     call.
 *   - Outputs are overwritten, never accumulated into.
 *   - A call whose output is empty (no rows or no columns) does nothing and
 *     returns T3_OK.  A call whose reduction is empty (K = 0 for the forward,
 *     N = 0 for dX, M = 0 for dW) writes zeros to its output.
 *   - Argument errors are reported before anything is launched; nothing is
 *     written then.  After T3_ECUDA (a launch or attribute call failed) the
 *     contents of the output are undefined: a call that queues a zeroing
 *     kernel before its product may have queued it already.  No C++
 *     exception crosses this interface and the device code never traps.
 *   - Calls may be made from several host threads; each call is independent.
 *   - Per-device state (the device error word's address, kernel attributes,
 *     the no-alloc buffer's address) is resolved once per device and process.
 *     It does not survive cudaDeviceReset: do not call the library on a device
 *     again in a process that reset it.
 */
#ifndef T3_H_
#define T3_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream (the same type as cudaStream_t / CUstream); NULL is the
 * legacy default stream. */
typedef struct CUstream_st* t3_stream_t;

typedef enum {
  T3_OK = 0,
  T3_EINVAL = -1,     /* null pointer with a non-empty shape, negative size   */
  T3_EVALUE = -2,     /* t3_pack_ternary: a weight outside {-1, 0, +1}        */
  T3_EOVERFLOW = -3,  /* a reduction too long for an exact int32 result       */
  T3_ECUDA = -4,      /* a CUDA runtime/driver call failed (launch, attribute) */
  T3_ETIMEOUT = -5,   /* a bounded device-side wait gave up (see below)       */
  T3_EDEVICE = -6     /* no usable sm_103 device for this call               */
} t3_status;

/*
 * t3_pack_ternary -- [fwd] "What this adds" (the 2-bit weight codes).
 *   w   HOST int8 [K][N], every value in {-1, 0, +1} (W as it appears in A x W)
 *   wp  HOST uint8 [N][ceil(K/4)], written in full: code 1 for +1, 2 for -1,
 *       0 for 0 and for the pad positions k >= K.
 * Synchronous, host memory only.  Returns T3_EVALUE and writes nothing when a
 * value is outside {-1, 0, +1}; T3_EINVAL for negative sizes or null pointers.
 */
int t3_pack_ternary(const int8_t* w, uint8_t* wp, int64_t K, int64_t N);

/*
 * t3_pack_ternary_device -- the same packing as t3_pack_ternary, on the device.
 *   w   DEVICE int8 [K][N]; wp DEVICE uint8 [N][ceil(K/4)], written in full
 *       (pad codes 0).  Both are owned by the caller.
 * Asynchronous on `stream`.  A value outside {-1, 0, +1} packs as code 0 and
 * records (9 << 8) | 6 in the device error word: t3_last_device_error then
 * returns T3_EVALUE.  Returns T3_EINVAL, without launching, for negative
 * sizes, null pointers (with K, N > 0) or sizes above 2^31 - 1; K or N = 0 is
 * a no-op.  Training changes W every step: this keeps the packing on the GPU.
 */
int t3_pack_ternary_device(const int8_t* w, uint8_t* wp, int64_t K, int64_t N,
                           t3_stream_t stream);

/*
 * t3_gemm_fwd -- [fwd]: C[m][n] = sum_{k<K} A[m][k] * W[k][n].
 *   A [M][K], Wp [N][ceil(K/4)], C [M][N] (layouts above), device pointers.
 * Exact for every input when K <= 16777215 (|A W| <= 128 K fits int32);
 * larger K returns T3_EOVERFLOW.  M <= 32 takes the small-M path, which is
 * bound by reading the packed weights: one or two rows (and up to eight when
 * Wp is at most 4 MB) run on the CUDA cores (byte-permute decode, dp4a), the
 * rest on the tensor cores.  Either way it enqueues one kernel on `stream` as
 * a programmatic dependent of the work before it, so that its launch and set-
 * up overlap that work's end; it reads A and Wp and writes C only after all
 * earlier work on `stream` has completed.
 * For M > 32, when whole output tiles would leave most of the GPU idle over a
 * long reduction (few tiles, many reduction stages) and A and Wp are
 * TMA-addressable, the reduction of the last tiles is split over the whole
 * GPU: the call then enqueues the same pair of kernels, the first zeroing the
 * rows of C that the split part adds into.
 * Small products (M*N*K at most the limit of t3_set_small_product_limit,
 * 2^29 by default, when a row stride or base of A or Wp is not a multiple of
 * 4 bytes, else at most an eighth of it; for M <= 32 only when Wp's rows are
 * not 16-byte multiples on a 16-byte boundary)
 * run on the CUDA cores instead: 64 x 64 output tiles, the reduction split
 * over CTAs that add atomically onto a zeroed C when the tiles are few (a
 * cudaMemsetAsync and one kernel, both on `stream`, in stream order), any
 * alignment of A, Wp and C.
 */
int t3_gemm_fwd(const int8_t* A, const uint8_t* Wp, int32_t* C, int64_t M, int64_t N,
                int64_t K, t3_stream_t stream);

/*
 * t3_gemm_bwd_dx -- [bwd] kernel 1: dX[m][k] = sum_{n<N} dY[m][n] * W[k][n].
 *   dY [M][N], Wp [N][ceil(K/4)] (the forward's packed weights), dX [M][K].
 * Exact for every input when N <= 16777215; larger N returns T3_EOVERFLOW.
 * Long reductions over few output tiles are split as in t3_gemm_fwd (M > 32),
 * with a zeroing kernel before the product.  Small products run on the CUDA
 * cores as in t3_gemm_fwd.
 */
int t3_gemm_bwd_dx(const int8_t* dY, const uint8_t* Wp, int32_t* dX, int64_t M, int64_t N,
                   int64_t K, t3_stream_t stream);

/*
 * t3_gemm_bwd_dw -- [bwd] kernel 2: dW[k][n] = sum_{m<M} A[m][k] * dY[m][n].
 *   A [M][K], dY [M][N], dW [K][N].
 * int8 x int8 products reach 16384, so the reduction is exact in int32 only
 * for M <= 131071 (the pages' bound); larger M returns T3_EOVERFLOW.
 * It enqueues two kernels on `stream`: one that zeroes dW and one that adds
 * 1024-row partial sums into it; the second may start before the first ends
 * (programmatic dependent launch) but touches dW only after it, and the first
 * touches dW only after all earlier work on `stream`.  Small products run on
 * the CUDA cores as in t3_gemm_fwd.
 */
int t3_gemm_bwd_dw(const int8_t* A, const int8_t* dY, int32_t* dW, int64_t M, int64_t N,
                   int64_t K, t3_stream_t stream);

/*
 * t3_quantize_rows_bf16 -- the step before the products: bf16 activations to
 * int8 with one scale per row.  The second page feeds its int8 kernels from
 * quantized tensors and names per-row scales for dX but gives no quantizer;
 * this is symmetric absmax per row:
 *   amax = max_k |x[m][k]|, row_scale[m] = amax / 127, inv = 127 / amax
 *   (each a float division rounded to nearest),
 *   q[m][k] = rint(x[m][k] * inv)  (product rounded to a float, then to the
 *   nearest integer, ties to even), clamped to [-127, 127];
 *   a row of zeros gives q = 0 and row_scale = 0.
 *   x DEVICE bf16 [M][K] (bit patterns), q DEVICE int8 [M][K], row_scale
 *   DEVICE float [M]; all owned by the caller.  Finite inputs; a product
 *   0 * inf (amax so small that 127 / amax overflows) counts as 0.
 * Asynchronous on `stream`.  M = 0 is a no-op; K = 0 writes row_scale = 0.
 */
int t3_quantize_rows_bf16(const void* x, int8_t* q, float* row_scale, int64_t M, int64_t K,
                          t3_stream_t stream);

/*
 * t3_gemm_fwd_bf16 -- the row quantizer fused into the forward product: the
 * same result as t3_quantize_rows_bf16(X, q, row_scale) followed by
 * t3_gemm_fwd(q, Wp, C), without writing q.  A first kernel takes each row's
 * absolute maximum and writes
 *   row_scale[m] = amax / 127 and row_inv[m] = 127 / amax   (0 and 0 for a
 *   zero row; the divisions of t3_quantize_rows_bf16),
 * then the forward pair pipeline reads X as bf16 tiles and its converters
 * quantize them (q = rint(x * row_inv[m]), ties to even) on their way to the
 * tensor core:
 *   C[m][n] = sum_k q[m][k] * W[k][n]     (exact int32, as t3_gemm_fwd).
 *   X DEVICE bf16 [M][K] (bit patterns), Wp DEVICE [N][ceil(K/4)], C DEVICE
 *   int32 [M][N], row_scale and row_inv DEVICE float [M]; caller-owned.
 * The fused kernel takes M > 32, K a multiple of 64 and X, Wp 16-byte aligned
 * (bf16 and packed rows TMA can address); any other shape returns T3_EINVAL
 * without launching (quantize, then multiply, instead).  N = 0 computes the
 * scales only; K = 0 writes zero scales and a zero C.  Asynchronous on
 * `stream`.  Finite inputs, as for t3_quantize_rows_bf16.
 */
int t3_gemm_fwd_bf16(const void* X, const uint8_t* Wp, int32_t* C, float* row_scale,
                     float* row_inv, int64_t M, int64_t N, int64_t K, t3_stream_t stream);

/*
 * Scaled outputs -- the step after the products in "spec(igla): hslm_bwd_ptx
 * -- HSLM backward dX and dW as int8 tensor-core PTX written by t27": the
 * host rescales the integer results (dX by a scale per row; dW by scales per
 * column of X and of dY, i.e. per row and per column of dW), and the products
 * also have "+=" forms.  For an exact int32 result x[r][c]:
 *   y = ((float)x * row_scale[r]) * col_scale[c]
 * with each conversion and product rounded to the nearest float (ties to
 * even); a NULL scale vector stands for ones.  The output kind decides what
 * is written: T3_OUT_F32 stores y (float), T3_OUT_BF16 stores y rounded to
 * bf16 (nearest, ties to even), T3_OUT_F32_ADD sets out = out + y (float, one
 * rounding).  Scale vectors are device float arrays, owned by the caller.
 */
enum { T3_OUT_F32 = 0, T3_OUT_BF16 = 1, T3_OUT_F32_ADD = 2 };

/*
 * t3_dequant_i32 -- out[r][c] from x [rows][cols] (DEVICE int32) as above;
 *   out DEVICE [rows][cols] float or bf16; row_scale [rows], col_scale [cols].
 * x and out may be the same buffer for T3_OUT_F32 only (else T3_EINVAL).
 * Asynchronous on `stream`; rows or cols = 0 is a no-op.
 */
int t3_dequant_i32(const int32_t* x, void* out, int64_t rows, int64_t cols,
                   const float* row_scale, const float* col_scale, int out_kind,
                   t3_stream_t stream);

/*
 * t3_gemm_fwd_scaled, t3_gemm_bwd_dx_scaled, t3_gemm_bwd_dw_scaled -- the
 * products of t3_gemm_fwd / t3_gemm_bwd_dx / t3_gemm_bwd_dw with the scaled
 * output above, same operands, sizes, validation and overflow rules:
 *   fwd: C [M][N],  row_scale [M], col_scale [N];
 *   dX:  dX [M][K], row_scale [M], col_scale [K];
 *   dW:  dW [K][N], row_scale [K] (X's column scales), col_scale [N] (dY's).
 * The forward (M > 32) and dX apply the scales in the epilogue of their
 * pair pipeline when the reduction is at most 65536 long and the output rows
 * are 16-byte aligned; otherwise, and always for dW, they compute the exact
 * int32 product first and then run t3_dequant_i32.  That product goes to
 * `workspace` (DEVICE int32 with the output's rows x cols, caller-owned) or,
 * for T3_OUT_F32 when `workspace` is NULL, into the output buffer, converted
 * in place; T3_OUT_BF16 and T3_OUT_F32_ADD return T3_EINVAL there without a
 * workspace.  The result is the same on every path.
 */
int t3_gemm_fwd_scaled(const int8_t* A, const uint8_t* Wp, void* C, int64_t M, int64_t N,
                       int64_t K, const float* row_scale, const float* col_scale, int out_kind,
                       int32_t* workspace, t3_stream_t stream);
int t3_gemm_bwd_dx_scaled(const int8_t* dY, const uint8_t* Wp, void* dX, int64_t M, int64_t N,
                          int64_t K, const float* row_scale, const float* col_scale, int out_kind,
                          int32_t* workspace, t3_stream_t stream);
int t3_gemm_bwd_dw_scaled(const int8_t* A, const int8_t* dY, void* dW, int64_t M, int64_t N,
                          int64_t K, const float* row_scale, const float* col_scale, int out_kind,
                          int32_t* workspace, t3_stream_t stream);

/*
 * t3_gemm_bwd_dw_scaled_noalloc -- t3_gemm_bwd_dw_scaled whose int32
 * intermediate lives in a fixed buffer inside the library instead of a
 * caller workspace, so that neither the call nor the caller allocates device
 * memory for it.  The pages have no counterpart: it serves callers that
 * cannot provide a workspace (bf16 and "+=" outputs need one).
 *   The buffer holds 8,388,608 int32 entries (32 MiB) per device: K * N above
 *   that returns T3_EINVAL before any CUDA call.  Nothing in it has to start
 *   at zero (the dW product writes all of its K x N block first).
 *   Races: every call on a device shares the buffer, so two calls must not
 *   overlap on one device -- not on different streams, and not from several
 *   host threads without ordering; each call's stream order alone protects
 *   only calls on that stream.
 *   The first call on each device resolves the buffer's address
 *   (cudaGetSymbolAddress); make that call outside any stream capture.  The
 *   address, like all per-device state, is not valid after cudaDeviceReset.
 *   Residency: the buffer sits in a module of its own.  With CUDA's lazy
 *   module loading (the default) a device reserves its 32 MiB at the first
 *   call of this function there and keeps it until the process exits; the
 *   other entry points do not load that module.  With eager loading
 *   (CUDA_MODULE_LOADING=EAGER) every device reserves it when the library's
 *   modules load.
 * Arguments, sizes, results and other errors are those of
 * t3_gemm_bwd_dw_scaled.
 */
int t3_gemm_bwd_dw_scaled_noalloc(const int8_t* A, const int8_t* dY, void* dW, int64_t M,
                                  int64_t N, int64_t K, const float* row_scale,
                                  const float* col_scale, int out_kind, t3_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The operators around the products of a ternary layer: the norm that feeds
 * them, the recurrence between them, and the product with its epilogue.  The
 * pages have no counterpart; each formula stands with its declaration.
 *
 * Element types of activations (`dtype`): T3_OUT_F32 (float) or T3_OUT_BF16.
 * Gains, biases, scales, statistics and states are float.  Arithmetic is
 * float, with one rounding per output element.  Results do not change from call
 * to call (no atomics; sums are added in a fixed order).
 *
 * A matrix [rows][cols] with a stride `ld*` (in elements) has its row r at
 * base + r * ld*; an output's stride is at least its columns, an input's may be
 * anything from 0 up.  Without a stride a matrix is dense.  Rows whose base
 * and stride are multiples of 16 bytes go fastest; any others are taken too.
 * Outputs must not overlap inputs or each other except where a call says so.
 * All of these calls are asynchronous on `stream`, take device pointers
 * and allocate nothing.
 */

/*
 * t3_rmsnorm_quant -- residual add, root-mean-square norm and int8 rows, one
 * pass over each row:
 *   s = x + residual, rounded to `dtype` (s = x when residual is NULL),
 *   rstd[r] = 1 / sqrt(mean_c(s^2) + eps),   y = s * rstd[r] * gamma[c],
 *   row_scale[r] = max_c |y| / 127,
 *   q = rint(u * (127 / max_c |u|)) with u = s * gamma (a float product), ties
 *   to even, clamped to [-127, 127]; y / row_scale up to rounding.  Where 127 /
 *   max_c |u| would pass the float range (below 3.7e-37) u counts 2^64 times.
 * q [rows][cols] (dense) and row_scale are what the products take.  gamma [cols]
 * NULL stands for ones.  sum_out (stride lds) receives s, the residual stream, and may be
 * x's or residual's buffer with the same stride; rstd is kept for the
 * gradient; either may be NULL.  A row of zeros gives q = 0 and row_scale = 0.  A row
 * with an element of u that is not finite, or whose squares overflow a float
 * sum, gets row_scale = NaN and q = 0, so that whatever is computed from it shows it.
 * Rows of up to 16384 columns (8192 for the gradient) are kept in registers;
 * longer ones are read element by element, two or three times, and take five to
 * six times as long per element.  Odd rows keep 16-byte accesses where all arrays, the
 * codes too, lie alike to 16-byte boundaries, as dense ones of fresh buffers do; a
 * padded stride beside the dense codes, or a view that begins at an odd row, does not
 * (bf16 8000 x 729: 16 us for 11; the gradient has no codes and keeps them).
 * T3_EINVAL: negative sizes or strides, lds < cols, a null x, q or row_scale
 * with a non-empty shape, eps not a positive finite float, an unknown dtype.
 * rows = 0 is a no-op; cols = 0 writes row_scale = 0 and rstd = 1 / sqrt(eps).
 */
int t3_rmsnorm_quant(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                     const float* gamma, float eps, int8_t* q, float* row_scale, float* rstd,
                     void* sum_out, int64_t lds, int64_t rows, int64_t cols, int dtype,
                     t3_stream_t stream);

/*
 * t3_rmsnorm_bwd -- the gradient of t3_rmsnorm_quant with the rounding to int8
 * passed straight through.  dy is the gradient of y, dsum (may be NULL) that of s
 * itself (the residual stream):
 *   n = dy * gamma,
 *   dx = rstd * (n - s * rstd^2 * mean_c(n * s)) + dsum,
 *   dgamma[c] = sum_r dy * s * rstd          (skipped when dgamma is NULL).
 * dx is the gradient of x and of residual alike.  s and rstd are the forward's.
 * dx may be dy's or dsum's buffer with the same stride.  workspace:
 * DEVICE floats, at least t3_colsum_workspace(rows, cols) of them, needed
 * (not zeroed) when dgamma is given.  rows = 0 writes dgamma = 0.
 */
int t3_rmsnorm_bwd(const void* dy, int64_t lddy, const void* s, int64_t lds, const float* rstd,
                   const float* gamma, const void* dsum, int64_t lddsum, void* dx, int64_t lddx,
                   float* dgamma, int64_t rows, int64_t cols, int dtype, float* workspace,
                   t3_stream_t stream);

/* Floats of workspace the column sums over [rows][cols] need (0 for empty or
 * invalid sizes); the same on every device. */
int64_t t3_colsum_workspace(int64_t rows, int64_t cols);

/*
 * t3_gated_scan_fwd -- the gated linear recurrence of `batch` sequences of
 * `length` tokens and `width` channels, element by element:
 *   a_t = sigmoid(gate_t),   h_t = a_t * h'_{t-1} + (1 - a_t) * cand_t,
 *   h'_{t-1} = h_{t-1}, or 0 where resets[b][t] is not 0 (a document starts);
 *   h_{-1} = h0 (NULL: zeros).
 * gate, cand, h: token t of sequence b is row b * length + t of a matrix with
 * `width` columns and the given stride.  h0, h_last float [batch][width]; resets
 * uint8 [batch][length] or NULL.  h_last (may be NULL, may be h0's buffer) receives the
 * float state after the last token, so single tokens (length = 1) advance
 * a state in place.  A token whose 1 - a_t is exactly 0 (gate = +inf, or one
 * beyond the float range of sigmoid) leaves the state as it is whatever cand
 * holds, NaN included.  The step is taken as h' + (1 - a_t) (cand_t - h'), which keeps a
 * long memory: where a state or a candidate that counts is infinite, or their
 * difference passes the float range, the state is infinite or NaN from there on.  None
 * of that passes a reset, in either direction.  length = 0 copies h0 to h_last.
 * T3_EINVAL: negative sizes or strides, sizes above 2^31 - 1, ldh < width, a
 * null gate, cand or h with a non-empty shape, an unknown dtype.
 */
int t3_gated_scan_fwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc,
                      const float* h0, const uint8_t* resets, void* h, int64_t ldh, float* h_last,
                      int64_t batch, int64_t length, int64_t width, int dtype, t3_stream_t stream);

/*
 * t3_gated_scan_bwd -- the gradient of t3_gated_scan_fwd.  dh is the gradient
 * of h, dh_last (may be NULL) that of h_last; h is the forward's output:
 *   G_t = dh_t + a_{t+1} G_{t+1} (without the second term where t + 1 resets;
 *         dh_last joins at the last token),
 *   dcand_t = (1 - a_t) G_t,  dgate_t = G_t (h'_{t-1} - cand_t) a_t (1 - a_t),
 *   dh0 = a_0 G_0 (0 where token 0 resets; dh0 may be NULL).
 * h'_{t-1} is read from h as it was stored (token 0's from h0): with bf16 rows its rounding adds up to
 * 2^-8 |G_t h'_{t-1}| a_t (1 - a_t) to dgate, and nothing to dcand and dh0.
 * From token to token a G is taken as G - (1 - a) G, off by a rounding of G however small a
 * is; dh0 = a_0 G_0 keeps its own relative precision.
 */
int t3_gated_scan_bwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const void* h,
                      int64_t ldh, const void* dh, int64_t lddh, const float* h0,
                      const uint8_t* resets, const float* dh_last, void* dgate, int64_t lddg,
                      void* dcand, int64_t lddc, float* dh0, int64_t batch, int64_t length,
                      int64_t width, int dtype, t3_stream_t stream);

/* Activations: T3_ACT_RELU2 is max(z, 0)^2, T3_ACT_SILU z sigmoid(z), T3_ACT_GELU
 * the tanh form z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2. */
enum { T3_ACT_NONE = 0, T3_ACT_RELU = 1, T3_ACT_RELU2 = 2, T3_ACT_SILU = 3, T3_ACT_GELU = 4 };

/*
 * t3_gemm_fwd_act -- the forward product with the rest of a layer in its
 * epilogue.  For the exact int32 x = A . W of t3_gemm_fwd:
 *   z = (x * row_scale[m]) * col_scale[n] + bias[n],
 *   C = act(z) + residual,   pre = z.
 * row_scale [M], col_scale [N], bias [N] (float), residual [M][N] and pre
 * [M][N] (the output's type) may each be NULL: ones, ones, zeros, zeros, not
 * written.  pre is what t3_act_bwd takes.  out_kind: T3_OUT_F32 or T3_OUT_BF16.  K = 0
 * takes x = 0.  C, residual and pre must be different buffers, and workspace
 * another one than a bf16 C (T3_EINVAL).  One kernel does it all for one or two
 * rows (and up to eight when Wp is at most 4 MB), for M > 32 where A, Wp, C,
 * residual and pre have rows of whole 16-byte pieces on 16-byte boundaries and K
 * <= 65536, and for small products of many tiles.  Otherwise the int32 product
 * is taken first, into `workspace` (DEVICE int32 [M][N]) or, for T3_OUT_F32
 * without one, into C; T3_OUT_BF16 returns T3_EINVAL there without a
 * workspace (t3_gemm_fwd_act_workspace tells).  scratch (DEVICE, 16-byte aligned, may be NULL) of at least
 * t3_gemm_fwd_act_scratch(M, N, K) bytes makes products with M > 32 and odd
 * rows several times faster: they are laid out aligned there first.
 * Sizes and overflow rules are those of t3_gemm_fwd_scaled.
 */
int t3_gemm_fwd_act(const int8_t* A, const uint8_t* Wp, void* C, int64_t M, int64_t N, int64_t K,
                    const float* row_scale, const float* col_scale, const float* bias, int act,
                    const void* residual, void* pre, int out_kind, int32_t* workspace, void* scratch,
                    int64_t scratch_bytes, t3_stream_t stream);

/* Bytes of scratch that t3_gemm_fwd_act can use for a product of these sizes: 0
 * where its rows are whole 16-byte pieces anyway. */
int64_t t3_gemm_fwd_act_scratch(int64_t M, int64_t N, int64_t K);
/* The same under the present limit of small products (t3_set_small_product_limit):
 * 0, too, for those, which the CUDA cores take as they lie. */
int64_t t3_gemm_fwd_act_scratch_now(int64_t M, int64_t N, int64_t K);
/* int32 entries of workspace that t3_gemm_fwd_act takes for these arguments and this
 * much scratch (16-byte aligned): M * N, or 0 where a call without one works; a
 * negative status where the device cannot be asked. */
int64_t t3_gemm_fwd_act_workspace(const int8_t* A, const uint8_t* Wp, const void* C, int64_t M, int64_t N,
                                  int64_t K, const void* residual, const void* pre, int out_kind,
                                  int64_t scratch_bytes);

/*
 * t3_act_bwd -- the gradient of that epilogue: for dy, the gradient of C, and
 * z, the forward's pre, both dense [rows][cols] of `dtype`:
 *   dz = dy * act'(z),   dbias[c] = sum_r dz   (before dz is rounded).
 * dz (may be dy's buffer) or dbias may be NULL; z may be NULL for T3_ACT_NONE.
 * dz is what t3_quantize_rows_bf16 and the backward products take; the
 * residual's gradient is dy itself.  workspace: at least
 * t3_colsum_workspace(rows, cols) floats when dbias is given.  rows = 0
 * writes dbias = 0.
 */
int t3_act_bwd(const void* dy, const void* z, int act, void* dz, float* dbias, int64_t rows,
               int64_t cols, int dtype, float* workspace, t3_stream_t stream);

/* A static, human-readable name for a status code (never NULL). */
const char* t3_status_string(int status);

/*
 * t3_last_device_error -- every pipeline wait inside the kernels is bounded
 * (about two seconds of device time).  A wait that runs out makes its kernel
 * stop early, leaving its output incomplete, and records a code in a
 * per-device error word instead of hanging the GPU.  This call synchronizes
 * `stream`, returns T3_ETIMEOUT if the word is set (T3_OK otherwise) and
 * clears it; T3_EVALUE instead when the code is the device packer's invalid
 * value.  *detail, when not NULL, receives the recorded code (0 if none):
 * bits 0-7 the role (1 producer, 2 converter, 3 MMA issuer, 4 epilogue,
 * 5 pair forwarder gave up; 6 an input value was invalid; 7 a CTA gave up
 * waiting for its cluster), bits 8-15 the kernel (4 small-M fwd;
 * 5 fwd, 6 dX, 7 dW on CTA pairs; 9 the device packer; 10 the wait self-test
 * below; 11 the gated recurrence).
 */
int t3_last_device_error(t3_stream_t stream, int32_t* detail);

/*
 * t3_set_small_product_limit -- the route of t3_gemm_fwd, t3_gemm_bwd_dx and
 * t3_gemm_bwd_dw (and of their scaled forms' int32 pass): products of at most
 * `macs` multiply-adds (M*N*K) run on the CUDA cores when an operand's rows
 * are not 4-byte aligned (stride or base not a multiple of 4 bytes), of at
 * most macs / 8 when they all are; larger ones on the tensor cores.  Default
 * 2^29 (536870912); 0 sends every product to the tensor cores; negative
 * values count as 0.  Process-wide, for every device;
 * a call racing with products on other threads may see either route, and
 * both give the same exact result.  Returns the previous limit.  Host only:
 * no CUDA call, no error.
 */
int64_t t3_set_small_product_limit(int64_t macs);

/*
 * t3_selftest_wait_timeout -- exercises the bounded-wait path above without
 * any fault: one CTA waits on a pipeline barrier that nothing completes, with
 * the kernels' own wait loop but a limit of `limit_ns` nanoseconds of device
 * time instead of two seconds.  The wait gives up, records (10 << 8) | 2 in
 * the error word (unless a code is already there) and the kernel returns, so
 * the next t3_last_device_error reports T3_ETIMEOUT with that detail and the
 * device stays usable.  The pages have no counterpart: this is a check of the
 * library's failure reporting.  limit_ns must lie in [1000, 2e9], else
 * T3_EINVAL; asynchronous on `stream`.
 */
int t3_selftest_wait_timeout(int64_t limit_ns, t3_stream_t stream);
/* The same for the wait of the recurrence's CTAs on their cluster, which records
 * (11 << 8) | 7. */
int t3_selftest_scan_wait_timeout(int64_t limit_ns, t3_stream_t stream);

/* Library version as major*10000 + minor*100 + patch. */
int t3_version(void);

#ifdef __cplusplus
}
#endif

#endif /* T3_H_ */
