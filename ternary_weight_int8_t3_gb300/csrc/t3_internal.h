// t3_internal.h -- declarations shared by the library's translation units.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include "t3_act.cuh"
#include "t3_common.cuh"
#include "t3_tc2.cuh"
#include "t3_tc2_dw.cuh"

namespace t3 {

// Tensor maps for 2-D row-major matrices (row stride = cols elements).  They
// return false, leaving *map zeroed, when TMA cannot be used (base or row
// stride not 16-byte aligned, or the driver refuses).
bool make_u8_map_tiled(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld,
                       int box_rows, int box_cols, bool swizzle128 = false);
bool make_i32_map_tiled(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                        int box_rows, int box_cols, bool swizzle128);

// CTA-pair pipeline for the forward and dX products.  With a split schedule
// (p.dp_tiles below the tile count) the rows the stream-K pieces add into must
// have been zeroed by launch_zero_pdl just before on `s`.
int launch_tc2_fwd(const tc2::Params& p, const CUtensorMap& ma, const CUtensorMap& mw,
                   const CUtensorMap& mo, int grid, cudaStream_t s);
int launch_tc2_dx(const tc2::Params& p, const CUtensorMap& ma, const CUtensorMap& mw,
                  const CUtensorMap& mo, int grid, cudaStream_t s);
// The same kernels' launch attributes, set once per device (launch_tc2_* call
// these too); the split schedule calls them before it queues its zeroing grid.
int prepare_tc2_fwd();
int prepare_tc2_dx();

// The forward on bf16 activations quantized in the pair pipeline's converters
// (tc2::kModeBf16; p.row_inv holds the rows' inverse scales).
int launch_tc2_fwd_bf16(const tc2::Params& p, const CUtensorMap& ma, const CUtensorMap& mw,
                        const CUtensorMap& mo, int grid, cudaStream_t s);

// The forward with the whole epilogue of a layer (tc2::kModeAct; p.epi, out_kind
// f32 or bf16): operands by TMA, whole tiles, one exact chunk, bulk stores; `more`
// describes p.epi.pre and p.epi.residual where those are set.
int launch_tc2_fwd_act(const tc2::Params& p, const CUtensorMap& ma, const CUtensorMap& mw,
                       const CUtensorMap& mo, const tc2::ActMaps& more, int grid, cudaStream_t s);

// Two forwards with their product in the epilogue (tc2::kModeGlu; p.glu): mw maps the gate's weights,
// `more` the other's and p.glu.pre where those are set.
int launch_tc2_fwd_glu(const tc2::Params& p, const CUtensorMap& ma, const CUtensorMap& mw,
                       const CUtensorMap& mo, const tc2::GluMaps& more, int grid, cudaStream_t s);

// Zeroes out[0, n) on `s` as a programmatic dependent of the work before it:
// it waits for that work to complete, then lets the next grid launch early.
int launch_zero_pdl(int32_t* out, int64_t n, int sms, cudaStream_t s);

// CTA-pair pipeline for dW (A, dY and dW all TMA-able).  Adds onto dW, which
// launch_zero_pdl has cleared just before on `s`; launched as its programmatic
// dependent.
int launch_dw2(const dw2::Params& p, const CUtensorMap& ma, const CUtensorMap& mdy,
               const CUtensorMap& mo, int grid, cudaStream_t s);

// Device packer: int8 w [K][N] -> Wp [N][ceil(K/4)] on `s`; a value outside
// {-1, 0, +1} packs as 0 and records (9 << 8) | 6 in *err.
int launch_pack_device(const int8_t* w, uint8_t* wp, int64_t K, int64_t N, int sms, int* err,
                       cudaStream_t s);

// bf16 x [M][K] -> int8 q [M][K] and a float scale per row (absmax), on `s`.
int launch_quant_rows(const void* x, int8_t* q, float* scale, int64_t M, int64_t K, int sms,
                      cudaStream_t s);

// The row quantizer's scales only: scale = amax / 127 and inv = 127 / amax per
// row of bf16 x [M][K] (0 and 0 for a zero row), on `s`.
int launch_row_scales(const void* x, float* scale, float* inv, int64_t M, int64_t K, int sms,
                      cudaStream_t s);

// out[r][c] = scaled int32 x[r][c] (T3_OUT_* kind), on `s`.
int launch_dequant(const int32_t* x, void* out, int64_t rows, int64_t cols, const float* row_scale,
                   const float* col_scale, int kind, int sms, cudaStream_t s);

// Forward for M <= 8 on the CUDA cores (t3_gemv.cu); T3_EINVAL, with nothing
// launched, when A's copy would not fit its shared-memory budget.
int launch_gemv_fwd(const int8_t* A, const uint8_t* Wp, int32_t* C, int64_t M, int64_t N,
                    int64_t K, int sms, cudaStream_t s);
// Whether it takes these rows.
bool gemv_fits(int64_t M, int64_t N, int64_t K);
// The same with the epilogue in the kernel that ends each sum.
int launch_gemv_fwd_act(const int8_t* A, const uint8_t* Wp, void* C, const EpilogueArgs& e, int kind,
                        int64_t M, int64_t N, int64_t K, int sms, cudaStream_t s);

// The same with two weights over one A.
int launch_gemv_fwd_glu(const int8_t* A, const uint8_t* Wg, const uint8_t* Wu, void* C, const GluArgs& e, int kind,
                        int64_t M, int64_t N, int64_t K, int sms, cudaStream_t s);

// The three products on the CUDA cores for small problems, any alignment
// (t3_small.cu): op 1 C = A.W (x = A, wp = Wp), 2 dX = dY.Wᵀ (x = dY, wp = Wp),
// 3 dW = Aᵀ.dY (x = A, y = dY); int32 output, written whole (zeroed first
// when the reduction is split over CTAs).
int launch_small(int op, const int8_t* x, const int8_t* y, const uint8_t* wp, int32_t* out,
                 int64_t M, int64_t N, int64_t K, int sms, cudaStream_t s);

// The forward of launch_small with the epilogue in its kernel; not where the tiles
// are so few that splitting the reduction is faster (small_act_fits).  launch_few_act
// splits it over a CTA's warps, unless it is too long for that (few_act_fits).
bool small_act_fits(int64_t M, int64_t N, int sms);
bool few_act_fits(int64_t M, int64_t N, int64_t K, int sms);
int launch_small_act(const int8_t* A, const uint8_t* Wp, void* C, const EpilogueArgs& e, int kind, int64_t M,
                     int64_t N, int64_t K, cudaStream_t s);
int launch_few_act(const int8_t* A, const uint8_t* Wp, void* C, const EpilogueArgs& e, int kind, int64_t M,
                   int64_t N, int64_t K, cudaStream_t s);

// The same two with two weights over one A; the fits take twice the columns.
int launch_small_glu(const int8_t* A, const uint8_t* Wg, const uint8_t* Wu, void* C, const GluArgs& e, int kind,
                     int64_t M, int64_t N, int64_t K, cudaStream_t s);
int launch_few_glu(const int8_t* A, const uint8_t* Wg, const uint8_t* Wu, void* C, const GluArgs& e, int kind,
                   int64_t M, int64_t N, int64_t K, cudaStream_t s);

// Small-M forward (M <= 32) on the tensor cores.
int launch_skinny_fwd(const int8_t* A, const uint8_t* Wp, int32_t* C, int64_t M, int64_t N,
                      int64_t K, int sms, int* err, cudaStream_t s);

// Partial rows of the column sums (norm and epilogue gradients): at most so
// many, so that a workspace's size does not depend on the device.
constexpr int kMaxColParts = 1216;

// out[c] = the sum of partial[0 .. parts)[c], added in a fixed order, on `s`.
int launch_col_finish(const float* partial, int parts, int64_t cols, float* out, cudaStream_t s);
// The same over partial rows of 2 cols floats: the first cols sums to out, the others to out2.
int launch_col_finish2(const float* partial, int parts, int64_t cols, float* out, float* out2, cudaStream_t s);

// Residual add, root-mean-square norm, int8 rows with a scale each, and its
// gradient (t3_norm.cu); dtype T3_OUT_F32 or T3_OUT_BF16.
int launch_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                    float eps, int8_t* q, float* row_scale, float* rstd, void* sum_out, int64_t lds,
                    int64_t rows, int64_t cols, int dtype, int sms, cudaStream_t s);
int launch_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t lds, const float* rstd,
                    const float* gamma, const void* dsum, int64_t lddsum, void* dx, int64_t lddx,
                    float* dgamma, int64_t rows, int64_t cols, int dtype, float* workspace, int sms,
                    cudaStream_t s);

// The same for the layer norm (t3_layernorm.cu).
int launch_layernorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                         const float* beta, float eps, int8_t* q, float* row_scale, float* mean, float* rstd,
                         void* sum_out, int64_t lds, int64_t rows, int64_t cols, int dtype, int sms,
                         cudaStream_t s);
int launch_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t lds, const float* mean,
                         const float* rstd, const float* gamma, const void* dsum, int64_t lddsum, void* dx,
                         int64_t lddx, float* dgamma, float* dbeta, int64_t rows, int64_t cols, int dtype,
                         float* workspace, int sms, cudaStream_t s);

// The gated recurrence over sequences and its gradient (t3_scan.cu).
int launch_scan_fwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const float* h0,
                    const uint8_t* resets, void* h, int64_t ldh, float* h_last, int64_t batch,
                    int64_t length, int64_t width, int dtype, int* err, cudaStream_t s);
int launch_scan_bwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const void* h,
                    int64_t ldh, const void* dh, int64_t lddh, const float* h0, const uint8_t* resets,
                    const float* dh_last, void* dgate, int64_t lddg, void* dcand, int64_t lddc,
                    float* dh0, int64_t batch, int64_t length, int64_t width, int dtype, int* err,
                    cudaStream_t s);

// What follows a product (EpilogueArgs) on its int32 result x with row stride
// ldx (t3_epilogue.cu); x may be out's buffer for T3_OUT_F32 (ldx = cols).
int launch_epilogue(const int32_t* x, int64_t ldx, void* out, const EpilogueArgs& e, int64_t rows, int64_t cols,
                    int kind, int sms, cudaStream_t s);

// Lays byte rows out 16-byte aligned: rows of len bytes (dense) to rows of pitch
// bytes (a multiple of 16, so is the destination), zeros behind each row and in
// rows rows .. rows2.  Two arrays in one launch; a may be null.
int launch_align_rows(const uint8_t* a, int64_t rows_a, int64_t len_a, uint8_t* a2, int64_t rows_a2, int64_t pitch_a,
                      const uint8_t* b, int64_t rows_b, int64_t len_b, uint8_t* b2, int64_t rows_b2, int64_t pitch_b,
                      cudaStream_t s);

// dz = dy act'(z) and its column sums.
int launch_act_bwd(const void* dy, const void* z, int act, void* dz, float* dbias, int64_t rows,
                   int64_t cols, int dtype, float* workspace, int sms, cudaStream_t s);

// What follows two products (GluArgs) on their int32 results, with row stride ldx
// (t3_glu.cu).
int launch_glu_epilogue(const int32_t* gate, const int32_t* up, int64_t ldx, void* out, const GluArgs& e, int64_t rows,
                        int64_t cols, int kind, int sms, cudaStream_t s);

// dgate = dy up act'(gate), dup = dy act(gate), and their column sums.
int launch_glu_bwd(const void* dy, const void* gate, const void* up, int act, void* dgate, void* dup,
                   float* dgate_bias, float* dup_bias, int64_t rows, int64_t cols, int dtype, float* workspace,
                   int sms, cudaStream_t s);

// The recurrence's wait between CTAs, run out on purpose (t3_selftest_scan_wait_timeout).
int launch_scan_wait_selftest(int* err, uint64_t limit_ns, cudaStream_t s);

}  // namespace t3
