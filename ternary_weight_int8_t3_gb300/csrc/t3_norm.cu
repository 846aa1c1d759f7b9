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
// What bounds it: memory.  A row is read once and written once.  A persistent
// grid of one wave takes rows in turn; a thread's columns are the same in every
// row, so their gains (and, backward, their sums of dgamma) stay in registers, and the
// next row's operands are loaded while this one is reduced and written.  Many
// rows take 16 elements a thread forward and 8 backward (8 and 8 where rows
// go element by element: arrays whose rows lie differently to 16-byte boundaries), few rows as few as 1024 threads
// allow, for the shortest time to one row; rows longer than the registers
// hold are read twice.  Backward, narrow rows share a CTA in groups of warps that
// meet at barriers of their own.  dgamma: each CTA adds its groups' sums in turn,
// writes one partial row, and a second small kernel adds the partial rows in a
// fixed order.
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
namespace nm {

using namespace vec;

struct FwdArgs {
  const void *x, *residual;
  int64_t ldx, ldr, lds;
  const float* gamma;
  float eps;
  int8_t* q;
  float *row_scale, *rstd;
  void* sum_out;
  int64_t rows, cols;
};

struct BwdArgs {
  const void *dy, *s, *dsum;
  int64_t lddy, lds, lddsum, lddx;
  const float *rstd, *gamma;
  void* dx;
  float* partial;  // [gridDim.x][cols], null without dgamma
  int64_t rows, cols;
  int groups;      // row groups a CTA (norm_bwd_kernel)
};

// One thread: the row's scale (NaN where it is not finite) and rstd.
__device__ __forceinline__ void put_scales(const FwdArgs& p, int64_t row, float ssq, float amax) {
  const float rstd =
      __fdiv_rn(1.0f, __fsqrt_rn(p.cols > 0 ? __fdiv_rn(ssq, static_cast<float>(p.cols)) + p.eps : p.eps));
  const bool finite = ssq < __int_as_float(0x7f800000) && amax < __int_as_float(0x7f800000);
  p.row_scale[row] = finite ? __fdiv_rn(__fmul_rn(amax, rstd), 127.0f) : __int_as_float(0x7fffffff);
  if (p.rstd) p.rstd[row] = rstd;
}

template <class T, int VEC, int NV, bool kOdd>
__global__ void __launch_bounds__(fwd_threads(NV * VEC)) norm_fwd_kernel(const FwdArgs p) {
  __shared__ float sm[2][64];
  const int lanes = blockDim.x, cols = static_cast<int>(p.cols);
  const Columns<T, VEC, kOdd> at(p.x, blockIdx.x * p.ldx, cols, threadIdx.x);
  launch_dependents();
  grid_dependency_wait();
  // this thread's columns: their gains, and the next row's operands, which are on
  // their way while this row is reduced and written
  float g[NV][VEC];
  float ge = 1.0f;
  Raw<T, VEC> xr[NV], rr[NV];
  Raw<T, 1> xe = zero<T, 1>(), re = zero<T, 1>();
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = static_cast<const T*>(p.residual) + row * p.ldr;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + static_cast<int>(v * lanes + threadIdx.x) * VEC;
      xr[v] = zero<T, VEC>();
      rr[v] = zero<T, VEC>();
      if (k < at.end && row < p.rows) {
        xr[v] = load<T, VEC>(x + k);
        if (p.residual) rr[v] = load<T, VEC>(r + k);
      }
    }
    if constexpr (kOdd) {
      if (at.has && row < p.rows) {
        xe = load<T, 1>(x + at.one);
        if (p.residual) re = load<T, 1>(r + at.one);
      }
    }
  };
  fetch(blockIdx.x);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int k = at.head + static_cast<int>(v * lanes + threadIdx.x) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[v][j] = 1.0f;
    if (p.gamma && k < at.end) {
      if constexpr (kOdd) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[v][j] = __ldg(p.gamma + k + j);
      } else {
        load_floats<VEC>(p.gamma + k, g[v]);
      }
    }
  }
  if (kOdd && p.gamma && at.has) ge = __ldg(p.gamma + at.one);
  int phase = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, phase ^= 1) {
    T* so = static_cast<T*>(p.sum_out) + row * p.lds;
    float u[NV][VEC], ssq = 0.0f, amax = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + static_cast<int>(v * lanes + threadIdx.x) * VEC;
      float s[VEC], t[VEC];
      to_float(xr[v], s);
      if (p.residual) {
        to_float(rr[v], t);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[j] += t[j];
      }
      const Raw<T, VEC> w = from_float(s, T());
      to_float(w, s);
      if (p.sum_out && k < at.end) store<T, VEC>(so + k, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        ssq = fmaf(s[j], s[j], ssq);
        u[v][j] = __fmul_rn(s[j], g[v][j]);
        amax = max_nan(amax, fabsf(u[v][j]));
      }
    }
    float ue = 0.0f;
    if constexpr (kOdd) {
      float se[1], te[1];
      to_float(xe, se);
      if (p.residual) {
        to_float(re, te);
        se[0] += te[0];
      }
      const Raw<T, 1> w = from_float(se, T());
      to_float(w, se);
      if (at.has) {
        if (p.sum_out) store<T, 1>(so + at.one, w);
        ssq = fmaf(se[0], se[0], ssq);
        ue = __fmul_rn(se[0], ge);
        amax = max_nan(amax, fabsf(ue));
      }
    }
    fetch(row + gridDim.x);
    cta_reduce(ssq, amax, sm[phase]);
    float up;
    const float inv = inverse_of(ssq, amax, up);
    if (threadIdx.x == 0) put_scales(p, row, ssq, amax);
    int8_t* q = p.q + row * p.cols;
    // u * inv within [-127, 127]: not for rows that are not finite (codes 0) nor small ones
    const bool plain = inv > 0.0f && up == 1.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + static_cast<int>(v * lanes + threadIdx.x) * VEC;
      if (k >= at.end) break;
      if constexpr (VEC == 1) {
        q[k] = static_cast<int8_t>(quant(u[v][0], inv, up));
      } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int j = 0; j < VEC / 4; ++j) {
          if (plain) {
            w[j] = quant4(u[v][4 * j], u[v][4 * j + 1], u[v][4 * j + 2], u[v][4 * j + 3], inv);
          } else {
            w[j] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[j] |= static_cast<uint32_t>(quant(u[v][4 * j + i], inv, up) & 0xFF) << (8 * i);
          }
        }
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(q + k) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(q + k) = w[0];
      }
    }
    if (kOdd && at.has) q[at.one] = static_cast<int8_t>(quant(ue, inv, up));
  }
}

// Rows longer than the registers hold: one CTA a row, read twice (the second
// time from sum_out where it is written).
template <class T>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const FwdArgs p) {
  __shared__ float sm[2][64];
  int phase = 0;
  launch_dependents();
  grid_dependency_wait();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, phase ^= 1) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = static_cast<const T*>(p.residual) + row * p.ldr;
    T* so = static_cast<T*>(p.sum_out) + row * p.lds;
    auto sum_at = [&](int64_t k) {
      float a[1], b[1];
      to_float(load<T, 1>(x + k), a);
      if (!p.residual) return a[0];
      to_float(load<T, 1>(r + k), b);
      return round_to(a[0] + b[0], T());
    };
    float ssq = 0.0f, amax = 0.0f;
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      const float s[1] = {sum_at(k)};
      if (p.sum_out) store<T, 1>(so + k, from_float(s, T()));
      ssq = fmaf(s[0], s[0], ssq);
      amax = max_nan(amax, fabsf(p.gamma ? __fmul_rn(s[0], __ldg(p.gamma + k)) : s[0]));
    }
    cta_reduce(ssq, amax, sm[phase]);
    float up;
    const float inv = inverse_of(ssq, amax, up);
    if (threadIdx.x == 0) put_scales(p, row, ssq, amax);
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float s[1];
      if (p.sum_out)
        to_float(load<T, 1>(so + k), s);  // this thread wrote it (it may lie over x or residual)
      else
        s[0] = sum_at(k);
      p.q[row * p.cols + k] =
          static_cast<int8_t>(quant(p.gamma ? __fmul_rn(s[0], __ldg(p.gamma + k)) : s[0], inv, up));
    }
  }
}

// kOne: the CTA is one group; else it has p.groups of them in 256 threads.
template <class T, int VEC, int NV, bool kOne, bool kOdd>
__global__ void __launch_bounds__(kOne ? bwd_threads(NV * VEC) : 256, kOne ? 1 : 3) norm_bwd_kernel(const BwdArgs p) {
  __shared__ float sm[2][32];
  extern __shared__ __align__(16) float sums[];  // [cols], with more than one group
  const int groups = kOne ? 1 : p.groups;
  const int lanes = blockDim.x / groups, cols = static_cast<int>(p.cols);
  const int group = kOne ? 0 : threadIdx.x / lanes, t = threadIdx.x - group * lanes, warps = lanes >> 5;
  const int64_t each = static_cast<int64_t>(gridDim.x) * groups;
  const Columns<T, VEC, kOdd> at(p.dy, (static_cast<int64_t>(blockIdx.x) * groups + group) * p.lddy, cols, t);
  launch_dependents();
  grid_dependency_wait();
  // this thread's columns: gains, sums, and the next row's operands
  float g[NV][VEC], acc[NV][VEC], next_rstd = 0.0f;
  float ge = 1.0f, acce = 0.0f;
  Raw<T, VEC> dyr[NV], sr[NV], dr[NV];
  Raw<T, 1> dye = zero<T, 1>(), se = zero<T, 1>(), de = zero<T, 1>();
  auto fetch = [&](int64_t row) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* sp = static_cast<const T*>(p.s) + row * p.lds;
    const T* ds = static_cast<const T*>(p.dsum) + row * p.lddsum;
    if (row < p.rows) next_rstd = p.rstd[row];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + (v * lanes + t) * VEC;
      dyr[v] = zero<T, VEC>();
      sr[v] = zero<T, VEC>();
      dr[v] = zero<T, VEC>();
      if (k < at.end && row < p.rows) {
        dyr[v] = load<T, VEC>(dy + k);
        sr[v] = load<T, VEC>(sp + k);
        if (p.dsum) dr[v] = load<T, VEC>(ds + k);
      }
    }
    if constexpr (kOdd) {
      if (at.has && row < p.rows) {
        dye = load<T, 1>(dy + at.one);
        se = load<T, 1>(sp + at.one);
        if (p.dsum) de = load<T, 1>(ds + at.one);
      }
    }
  };
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
  fetch(first);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int k = at.head + (v * lanes + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      g[v][j] = 1.0f;
      acc[v][j] = 0.0f;
    }
    if (p.gamma && k < at.end) {
      if constexpr (kOdd) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[v][j] = __ldg(p.gamma + k + j);
      } else {
        load_floats<VEC>(p.gamma + k, g[v]);
      }
    }
  }
  if (kOdd && p.gamma && at.has) ge = __ldg(p.gamma + at.one);
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  int phase = 0;
  for (int64_t row = first; row < p.rows; row += each, phase ^= 1) {
    const float rstd = next_rstd;
    float n[NV][VEC], s[NV][VEC], dot = 0.0f;
    Raw<T, VEC> d[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      to_float(dyr[v], n[v]);
      to_float(sr[v], s[v]);
      d[v] = dr[v];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s[v][j] *= rstd;
        acc[v][j] = fmaf(n[v][j], s[v][j], acc[v][j]);
        n[v][j] *= g[v][j];
        dot = fmaf(n[v][j], s[v][j], dot);
      }
    }
    float ne[1] = {}, sse[1] = {}, ye[1] = {};
    if constexpr (kOdd) {  // zeros where the thread has none
      to_float(dye, ne);
      to_float(se, sse);
      to_float(de, ye);
      sse[0] *= rstd;
      acce = fmaf(ne[0], sse[0], acce);
      ne[0] *= ge;
      dot = fmaf(ne[0], sse[0], dot);
    }
    fetch(row + each);
    dot = group_sum(dot, sm[phase] + group * warps, t >> 5, warps, 1 + group);
    const float c = dot * inv_cols;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + (v * lanes + t) * VEC;
      if (k >= at.end) break;
      float y[VEC];
      to_float(d[v], y);
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[j] = fmaf(rstd, fmaf(-c, s[v][j], n[v][j]), y[j]);
      store<T, VEC>(dx + k, from_float(y, T()));
    }
    if (kOdd && at.has) {
      ye[0] = fmaf(rstd, fmaf(-c, sse[0], ne[0]), ye[0]);
      store<T, 1>(dx + at.one, from_float(ye, T()));
    }
  }
  if (!p.partial) return;
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.cols;
  if constexpr (kOdd) {  // element by element, and then in order
    for (int i = 0; i < groups; ++i) {
      if (group == i) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int k = at.head + (v * lanes + t) * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (k < at.end) sums[k + j] = (i ? sums[k + j] : 0.0f) + acc[v][j];
        }
        if (at.has) sums[at.one] = (i ? sums[at.one] : 0.0f) + acce;
      }
      __syncthreads();
    }
    for (int k = threadIdx.x; k < cols; k += blockDim.x) out[k] = sums[k];
  } else {
    // the groups add their sums in turn; the last one writes
    for (int i = 0; i < groups - 1; ++i) {
      if (group == i) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int k = at.head + (v * lanes + t) * VEC;
          if (k < cols) add_floats<VEC>(sums + k, sums + k, i > 0, acc[v], true);
        }
      }
      __syncthreads();
    }
    if (group != groups - 1) return;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + (v * lanes + t) * VEC;
      if (k < cols) add_floats<VEC>(out + k, sums + k, groups > 1, acc[v], wide);
    }
  }
}

// Long rows: dx with the row read twice; the column sums come from
// norm_dgamma_kernel, which runs first (dx may lie over dy or dsum).
template <class T>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const BwdArgs p) {
  __shared__ float sm[2][64];
  int phase = 0;
  launch_dependents();
  grid_dependency_wait();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, phase ^= 1) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* sp = static_cast<const T*>(p.s) + row * p.lds;
    const T* ds = static_cast<const T*>(p.dsum) + row * p.lddsum;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    const float rstd = p.rstd[row];
    float dot = 0.0f;
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float a[1], s[1];
      to_float(load<T, 1>(dy + k), a);
      to_float(load<T, 1>(sp + k), s);
      dot = fmaf(p.gamma ? a[0] * __ldg(p.gamma + k) : a[0], s[0], dot);
    }
    {
      float unused = 0.0f;
      cta_reduce(dot, unused, sm[phase]);
    }
    const float c = rstd * (dot * rstd / static_cast<float>(p.cols));
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float a[1], s[1], d[1] = {0.0f};
      to_float(load<T, 1>(dy + k), a);
      to_float(load<T, 1>(sp + k), s);
      if (p.dsum) to_float(load<T, 1>(ds + k), d);
      d[0] = fmaf(rstd, fmaf(-c, s[0], p.gamma ? a[0] * __ldg(p.gamma + k) : a[0]), d[0]);
      store<T, 1>(dx + k, from_float(d, T()));
    }
  }
}

// Partial column sums of dy s rstd: a CTA takes 32 columns (one a lane) and
// every gridDim.x / tiles-th block of rows; its 8 warps take rows in turn.
template <class T>
__global__ void __launch_bounds__(256) norm_dgamma_kernel(const BwdArgs p, int parts) {
  __shared__ float sm[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % parts;
  const int64_t k = static_cast<int64_t>(blockIdx.x / parts) * 32 + lane;
  launch_dependents();
  grid_dependency_wait();
  float acc = 0.0f;
  if (k < p.cols)
    for (int64_t row = part * 8 + warp; row < p.rows; row += static_cast<int64_t>(parts) * 8) {
      float a[1], s[1];
      to_float(load<T, 1>(static_cast<const T*>(p.dy) + row * p.lddy + k), a);
      to_float(load<T, 1>(static_cast<const T*>(p.s) + row * p.lds + k), s);
      acc = fmaf(a[0], s[0] * p.rstd[row], acc);
    }
  sm[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && k < p.cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sm[w][lane];
    p.partial[static_cast<int64_t>(part) * p.cols + k] = t;
  }
}

// ----------------------------------------------------------------- routing

// Forward: few rows take the fewest elements a thread, many rows 16 or more.
template <class T, int VEC, int MAXNV, bool kOdd>
int fwd_vec(const FwdArgs& p, int sms, cudaStream_t s) {
  const bool many = p.rows >= 2 * static_cast<int64_t>(sms);
  int threads = 0;
  const int nv = pick<VEC, MAXNV>((p.cols + VEC - 1) / VEC, many ? (VEC > 1 ? 16 : 8) : 1, fwd_threads,
                                &threads);
  // one wave of resident CTAs (64 registers a thread)
  int64_t grid = static_cast<int64_t>(sms) * (threads > 512 ? 1 : 1024 / (threads > 0 ? threads : 1024));
  if (nv == 0) grid = 2ll * sms;
  if (grid > p.rows) grid = p.rows;
  if (kOdd && nv) grid = alike<VEC>(grid, p.rows, p.ldx, 1);
  if (nv == MAXNV / 4) return launch(norm_fwd_kernel<T, VEC, MAXNV / 4, kOdd>, grid, threads, 0, s, 1, p);
  if (nv == MAXNV / 2) return launch(norm_fwd_kernel<T, VEC, MAXNV / 2, kOdd>, grid, threads, 0, s, 1, p);
  if (nv == MAXNV) return launch(norm_fwd_kernel<T, VEC, MAXNV, kOdd>, grid, threads, 0, s, 1, p);
  return launch(norm_fwd_long_kernel<T>, grid, 1024, 0, s, 1, p);
}

// Backward: many rows take 8 elements a thread (more only where the row would not
// fit a CTA).
template <class T, int VEC, int MAXNV, bool kOdd>
int bwd_vec(BwdArgs p, float* dgamma, int sms, int* parts, cudaStream_t s) {
  const bool many = p.rows >= 2 * static_cast<int64_t>(sms);
  int threads = 0;
  const int nv = pick<VEC, MAXNV>((p.cols + VEC - 1) / VEC, many ? 8 : 1, bwd_threads, &threads);
  int64_t grid = 2ll * sms;
  if (nv) {
    // narrow rows: two groups or more in 256 threads, three such CTAs an SM;
    // else a CTA a row, as many as the registers hold
    p.groups = many && nv * VEC == 8 ? 256 / threads : 1;
    if (p.groups < 1) p.groups = 1;
    const bool one = p.groups == 1;
    const int room = (one ? bwd_threads(nv * VEC) : 768) / (threads * p.groups);
    grid = static_cast<int64_t>(sms) * room;
    const int64_t need = (p.rows + p.groups - 1) / p.groups;
    if (grid > need) grid = need;
    if (grid > kMaxColParts) grid = kMaxColParts;
    if (kOdd) grid = alike<VEC>(grid, p.rows, p.lddy, p.groups);
    *parts = static_cast<int>(grid);
    if (grid == 1 && p.partial) p.partial = dgamma;  // one part is the sum itself
    const size_t sums = kOdd || !one ? static_cast<size_t>(p.cols) * sizeof(float) : 0;
    if (!one)
      return launch(norm_bwd_kernel<T, VEC, 8 / VEC, false, kOdd>, grid, threads * p.groups, sums, s, 1, p);
    if (nv == MAXNV / 4) return launch(norm_bwd_kernel<T, VEC, MAXNV / 4, true, kOdd>, grid, threads, sums, s, 1, p);
    if (nv == MAXNV / 2) return launch(norm_bwd_kernel<T, VEC, MAXNV / 2, true, kOdd>, grid, threads, sums, s, 1, p);
    return launch(norm_bwd_kernel<T, VEC, MAXNV, true, kOdd>, grid, threads, sums, s, 1, p);
  }
  if (p.partial) {
    const int64_t tiles = (p.cols + 31) / 32;
    const int64_t n = (p.rows + 7) / 8 < 16 ? (p.rows + 7) / 8 : 16;
    *parts = static_cast<int>(n);
    if (n == 1) p.partial = dgamma;
    const int st = launch(norm_dgamma_kernel<T>, tiles * n, 256, 0, s, 1, p, *parts);
    if (st != T3_OK) return st;
  }
  if (grid > p.rows) grid = p.rows;
  return launch(norm_bwd_long_kernel<T>, grid, 1024, 0, s, 1, p);
}

}  // namespace nm

int launch_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                    float eps, int8_t* q, float* row_scale, float* rstd, void* sum_out, int64_t lds,
                    int64_t rows, int64_t cols, int dtype, int sms, cudaStream_t s) {
  const nm::FwdArgs p{x, residual, ldx, ldr, lds, gamma, eps, q, row_scale, rstd, sum_out, rows, cols};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(x, ldx, es) && nm::vec_rows(residual, ldr, es) &&
                   nm::vec_rows(sum_out, lds, es) && vec::aligned(q, v) &&
                   (!gamma || vec::aligned(gamma, 16));
  // rows that are alike; their codes, too, then lie to boundaries of v bytes as they do to v elements
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(residual, ldr, x, ldx, es, v) &&
                   nm::alike_rows(sum_out, lds, x, ldx, es, v) && reinterpret_cast<uintptr_t>(x) % es == 0 &&
                   (reinterpret_cast<uintptr_t>(x) / es - reinterpret_cast<uintptr_t>(q)) % v == 0 && (ldx - cols) % v == 0;
  if (dtype == T3_OUT_BF16)
    return vec   ? nm::fwd_vec<vec::bf16, 8, 4, false>(p, sms, s)
           : odd ? nm::fwd_vec<vec::bf16, 8, 4, true>(p, sms, s)
                 : nm::fwd_vec<vec::bf16, 1, 32, false>(p, sms, s);
  return vec   ? nm::fwd_vec<float, 4, 4, false>(p, sms, s)
         : odd ? nm::fwd_vec<float, 4, 4, true>(p, sms, s)
               : nm::fwd_vec<float, 1, 32, false>(p, sms, s);
}

int launch_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t lds, const float* rstd,
                    const float* gamma, const void* dsum, int64_t lddsum, void* dx, int64_t lddx,
                    float* dgamma, int64_t rows, int64_t cols, int dtype, float* workspace, int sms,
                    cudaStream_t s) {
  const nm::BwdArgs p{dy, x, dsum, lddy, lds, lddsum, lddx, rstd, gamma, dx, dgamma ? workspace : nullptr,
                      rows, cols};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(dy, lddy, es) && nm::vec_rows(x, lds, es) &&
                   nm::vec_rows(dsum, lddsum, es) && nm::vec_rows(dx, lddx, es) &&
                   (!gamma || vec::aligned(gamma, 16));
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(x, lds, dy, lddy, es, v) &&
                   nm::alike_rows(dsum, lddsum, dy, lddy, es, v) && nm::alike_rows(dx, lddx, dy, lddy, es, v);
  int parts = 0, st;
  if (dtype == T3_OUT_BF16)
    st = vec   ? nm::bwd_vec<vec::bf16, 8, 4, false>(p, dgamma, sms, &parts, s)
         : odd ? nm::bwd_vec<vec::bf16, 8, 4, true>(p, dgamma, sms, &parts, s)
               : nm::bwd_vec<vec::bf16, 1, 32, false>(p, dgamma, sms, &parts, s);
  else
    st = vec   ? nm::bwd_vec<float, 4, 4, false>(p, dgamma, sms, &parts, s)
         : odd ? nm::bwd_vec<float, 4, 4, true>(p, dgamma, sms, &parts, s)
               : nm::bwd_vec<float, 1, 32, false>(p, dgamma, sms, &parts, s);
  if (st != T3_OK || !dgamma || parts == 1) return st;
  return launch_col_finish(workspace, parts, cols, dgamma, s);
}

}  // namespace t3
