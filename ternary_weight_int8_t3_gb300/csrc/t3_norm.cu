// t3_norm.cu -- the root-mean-square norm in front of a product: the residual
// added on the way in, int8 rows with one scale each on the way out, and the
// gradient of it.
//
// What it computes, for a row of `cols` elements with a float gain gamma:
//   s = x + r, rounded once to the rows' type (the residual stream it is kept in)
//   rstd = 1 / sqrt(mean(s^2) + eps),   y = s rstd gamma
//   row_scale = max|y| / 127,           q = rint(y / row_scale) in [-127, 127]
// With u = s gamma the norm cancels in q: q = rint(u * (127 / max|u|)), and
// row_scale = max|u| rstd / 127.  So both reductions (the sum of squares and
// max|u|) are taken in one pass over the row, and q does not depend on the
// order of the sum.  Backward, with the rounding passed straight through and
// n = dy gamma:
//   dx = rstd (n - s rstd^2 mean(n s)) + dsum,   dgamma = sum over rows of dy s rstd
//
// How, and what bounds it: t3_norm.cuh.
//
// Measured (GB300, with residual; bytes of the formulas over the time, of the measured
// 6784 GB/s): bf16 forward 16384 x 1280 26.3 us (82 %), 16384 x 3456 63 us (92 %), 1 x
// 8192 2.9 us; backward 33 us (75 %) and 82 us (82 %).  Float 16384 x 1280 49 us (82 %)
// and 60 us (83 %), 16384 x 3456 121 us (90 %) and 152 us (88 %), although every float
// instantiation of the backward and the widest of the forward spill 28 to 136 bytes a thread.
// Odd widths: 1782 x 729 float 5.8 us forward, 10.9 us backward; 8000 x 729 bf16 without
// residual 11.3 and 14.6 us, forward 16.3 where the codes lie differently to the rows.
// Wide rows (bf16 without residual): 4096 x 16384 forward 56 us, 16392 columns 312 us;
// backward 8192 columns 46 us, 12288 285 us: past the registers every element is a
// load of its own, and dy and s are read three times.
#include "t3_norm.cuh"

namespace t3 {

int launch_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                    float eps, int8_t* q, float* row_scale, float* rstd, void* sum_out, int64_t lds,
                    int64_t rows, int64_t cols, int dtype, int sms, cudaStream_t s) {
  const nm::FwdArgs p{x,   residual, ldx,       ldr,     lds,  gamma,   nullptr, eps,
                      q,   row_scale, nullptr,  rstd,    sum_out, rows, cols};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(x, ldx, es) && nm::vec_rows(residual, ldr, es) &&
                   nm::vec_rows(sum_out, lds, es) && vec::aligned(q, v) &&
                   (!gamma || vec::aligned(gamma, 16));
  // rows that are alike; their codes, too, then lie to boundaries of v bytes as they do to v elements
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(residual, ldr, x, ldx, es, v) &&
                   nm::alike_rows(sum_out, lds, x, ldx, es, v) && reinterpret_cast<uintptr_t>(x) % es == 0 &&
                   (reinterpret_cast<uintptr_t>(x) / es - reinterpret_cast<uintptr_t>(q)) % v == 0 && (ldx - cols) % v == 0;
  if (dtype == T3_OUT_BF16)
    return vec   ? nm::fwd_vec<vec::bf16, 8, 4, false, false>(p, sms, s)
           : odd ? nm::fwd_vec<vec::bf16, 8, 4, true, false>(p, sms, s)
                 : nm::fwd_vec<vec::bf16, 1, 32, false, false>(p, sms, s);
  return vec   ? nm::fwd_vec<float, 4, 4, false, false>(p, sms, s)
         : odd ? nm::fwd_vec<float, 4, 4, true, false>(p, sms, s)
               : nm::fwd_vec<float, 1, 32, false, false>(p, sms, s);
}

int launch_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t lds, const float* rstd,
                    const float* gamma, const void* dsum, int64_t lddsum, void* dx, int64_t lddx,
                    float* dgamma, int64_t rows, int64_t cols, int dtype, float* workspace, int sms,
                    cudaStream_t s) {
  const nm::BwdArgs p{dy,   x,     dsum, lddy, lds,  lddsum, lddx, nullptr, rstd, gamma, dx, dgamma ? workspace : nullptr,
                      nullptr, cols, rows, cols, 0};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(dy, lddy, es) && nm::vec_rows(x, lds, es) &&
                   nm::vec_rows(dsum, lddsum, es) && nm::vec_rows(dx, lddx, es) &&
                   (!gamma || vec::aligned(gamma, 16));
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(x, lds, dy, lddy, es, v) &&
                   nm::alike_rows(dsum, lddsum, dy, lddy, es, v) && nm::alike_rows(dx, lddx, dy, lddy, es, v);
  int parts = 0, st;
  if (dtype == T3_OUT_BF16)
    st = vec   ? nm::bwd_vec<vec::bf16, 8, 4, false, false>(p, dgamma, nullptr, sms, &parts, s)
         : odd ? nm::bwd_vec<vec::bf16, 8, 4, true, false>(p, dgamma, nullptr, sms, &parts, s)
               : nm::bwd_vec<vec::bf16, 1, 32, false, false>(p, dgamma, nullptr, sms, &parts, s);
  else
    st = vec   ? nm::bwd_vec<float, 4, 4, false, false>(p, dgamma, nullptr, sms, &parts, s)
         : odd ? nm::bwd_vec<float, 4, 4, true, false>(p, dgamma, nullptr, sms, &parts, s)
               : nm::bwd_vec<float, 1, 32, false, false>(p, dgamma, nullptr, sms, &parts, s);
  if (st != T3_OK || !dgamma || parts == 1) return st;
  return launch_col_finish(workspace, parts, cols, dgamma, s);
}

}  // namespace t3
