// t3_layernorm.cu -- the layer norm in front of a product: the residual added on the
// way in, int8 rows with one scale each on the way out, and the gradient of it.
//
// What it computes, for a row of `cols` elements with float gains gamma and shifts beta:
//   s = x + r, rounded once to the rows' type (the residual stream it is kept in)
//   mean = sum(s) / cols,   rstd = 1 / sqrt(sum((s - mean)^2) / cols + eps)
//   y = (s - mean) rstd gamma + beta
//   row_scale = max|y| / 127,   q = rint(y * (127 / max|y|)) in [-127, 127]
// The squares are taken of differences from a mean, never as sum(s^2) - mean^2, so that a row
// far from zero keeps its deviation: each warp takes its own mean and its squares from that, and
// the warps' moments join exactly (cta_moments).  With a shift, max|y| needs the
// deviation first, so a row is reduced twice, with a barrier each.  Backward, with the rounding passed
// straight through, h = (s - mean) rstd and n = dy gamma:
//   dx = rstd (n - mean(n) - h mean(n h)) + dsum
//   dgamma = sum over rows of dy h,   dbeta = sum over rows of dy
//
// How, and what bounds it: t3_norm.cuh.
#include "t3_norm.cuh"

namespace t3 {

int launch_layernorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                         const float* beta, float eps, int8_t* q, float* row_scale, float* mean, float* rstd,
                         void* sum_out, int64_t lds, int64_t rows, int64_t cols, int dtype, int sms,
                         cudaStream_t s) {
  const nm::FwdArgs p{x, residual,  ldx,  ldr,  lds,     gamma, beta, eps,
                      q, row_scale, mean, rstd, sum_out, rows,  cols};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(x, ldx, es) && nm::vec_rows(residual, ldr, es) &&
                   nm::vec_rows(sum_out, lds, es) && vec::aligned(q, v) && (!gamma || vec::aligned(gamma, 16));
  // rows that are alike; their codes, too, then lie to boundaries of v bytes as they do to v elements
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(residual, ldr, x, ldx, es, v) &&
                   nm::alike_rows(sum_out, lds, x, ldx, es, v) && reinterpret_cast<uintptr_t>(x) % es == 0 &&
                   (reinterpret_cast<uintptr_t>(x) / es - reinterpret_cast<uintptr_t>(q)) % v == 0 && (ldx - cols) % v == 0;
  if (dtype == T3_OUT_BF16)
    return vec   ? nm::fwd_vec<vec::bf16, 8, 4, false, true>(p, sms, s)
           : odd ? nm::fwd_vec<vec::bf16, 8, 4, true, true>(p, sms, s)
                 : nm::fwd_vec<vec::bf16, 1, 32, false, true>(p, sms, s);
  return vec   ? nm::fwd_vec<float, 4, 4, false, true>(p, sms, s)
         : odd ? nm::fwd_vec<float, 4, 4, true, true>(p, sms, s)
               : nm::fwd_vec<float, 1, 32, false, true>(p, sms, s);
}

int launch_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t lds, const float* mean,
                         const float* rstd, const float* gamma, const void* dsum, int64_t lddsum, void* dx,
                         int64_t lddx, float* dgamma, float* dbeta, int64_t rows, int64_t cols, int dtype,
                         float* workspace, int sms, cudaStream_t s) {
  // both sums: a partial row holds dgamma's columns and then dbeta's
  const int64_t ldp = dgamma && dbeta ? 2 * cols : cols;
  const nm::BwdArgs p{dy, x, dsum, lddy, lds, lddsum, lddx, mean, rstd, gamma, dx, dgamma ? workspace : nullptr,
                      dbeta ? workspace + (dgamma ? cols : 0) : nullptr, ldp, rows, cols, 0};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(dy, lddy, es) && nm::vec_rows(x, lds, es) &&
                   nm::vec_rows(dsum, lddsum, es) && nm::vec_rows(dx, lddx, es) &&
                   (!gamma || vec::aligned(gamma, 16));
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(x, lds, dy, lddy, es, v) &&
                   nm::alike_rows(dsum, lddsum, dy, lddy, es, v) && nm::alike_rows(dx, lddx, dy, lddy, es, v);
  int parts = 0, st;
  if (dtype == T3_OUT_BF16)
    st = vec   ? nm::bwd_vec<vec::bf16, 8, 4, false, true>(p, dgamma, dbeta, sms, &parts, s)
         : odd ? nm::bwd_vec<vec::bf16, 8, 4, true, true>(p, dgamma, dbeta, sms, &parts, s)
               : nm::bwd_vec<vec::bf16, 1, 32, false, true>(p, dgamma, dbeta, sms, &parts, s);
  else
    st = vec   ? nm::bwd_vec<float, 4, 4, false, true>(p, dgamma, dbeta, sms, &parts, s)
         : odd ? nm::bwd_vec<float, 4, 4, true, true>(p, dgamma, dbeta, sms, &parts, s)
               : nm::bwd_vec<float, 1, 32, false, true>(p, dgamma, dbeta, sms, &parts, s);
  if (st != T3_OK || (!dgamma && !dbeta) || parts == 1) return st;
  if (dgamma && dbeta) return launch_col_finish2(workspace, parts, cols, dgamma, dbeta, s);
  return launch_col_finish(workspace, parts, cols, dgamma ? dgamma : dbeta, s);
}

}  // namespace t3
