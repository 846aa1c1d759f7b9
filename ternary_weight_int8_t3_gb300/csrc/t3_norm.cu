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
// What bounds it: memory.  A row is read once, kept in registers between the
// reductions and the output, and written once.  Rows of up to 1024 elements
// (512 floats) take one warp, longer ones a CTA whose threads each hold one, two
// or four 16-byte vectors; rows that 16-byte vectors cannot address (odd
// widths, strides or bases) go element by element; rows longer than the
// registers hold are read twice.  dgamma: each CTA of a persistent grid holds
// its columns' sums in registers over all its rows, writes one partial row,
// and a second small kernel adds the partial rows in a fixed order.
#include "t3_vec.cuh"

namespace t3 {
namespace nm {

using namespace vec;

constexpr int kWarpRows = 8;  // rows per CTA where a warp takes a row

// Threads a CTA may have when each holds EPT elements of a row: up to 16384
// elements a row forward (one float an element is kept) and 8192 backward (the
// gain, the column sum and three operands), within 64 to 128 registers a thread.
constexpr int fwd_threads(int ept) { return ept <= 16 ? 1024 : 16384 / ept; }
constexpr int bwd_threads(int ept) { return ept <= 8 ? 1024 : 8192 / ept; }

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
};

__device__ __forceinline__ int quant(float u, float inv) {
  const int q = __float2int_rn(__fmul_rn(u, inv));  // NaN (0 * inf) gives 0
  return q > 127 ? 127 : (q < -127 ? -127 : q);
}

// A row's two results from its reductions.  Elements that are not finite, or
// whose squares overflow the sum, make the row's scale NaN and its codes 0.
struct RowScale {
  float rstd, scale, inv;
};
__device__ __forceinline__ RowScale row_scale_of(float ssq, float amax, float eps, int64_t cols) {
  RowScale o;
  o.rstd = __fdiv_rn(1.0f, __fsqrt_rn(cols > 0 ? __fdiv_rn(ssq, static_cast<float>(cols)) + eps : eps));
  const bool finite = ssq < __int_as_float(0x7f800000) && amax < __int_as_float(0x7f800000);
  if (!finite) {
    o.scale = __int_as_float(0x7fffffff);
    o.inv = 0.0f;
  } else {
    o.scale = __fdiv_rn(__fmul_rn(amax, o.rstd), 127.0f);
    o.inv = amax > 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
  }
  return o;
}

// Sum of `a` and NaN-keeping maximum of `b` over the CTA's threads; `sm` holds
// 64 floats and alternates between two areas from call to call, so one barrier
// a call is enough.
__device__ __forceinline__ void cta_reduce(float& a, float& b, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  a = warp_sum(a);
  b = warp_max_nan(b);
  if (warps == 1) return;
  if (lane == 0) {
    sm[warp] = a;
    sm[32 + warp] = b;
  }
  __syncthreads();
  a = warp_sum(lane < warps ? sm[lane] : 0.0f);
  b = warp_max_nan(lane < warps ? sm[32 + lane] : 0.0f);
}

template <class T, int VEC, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : fwd_threads(NV * VEC)) norm_fwd_kernel(const FwdArgs p) {
  __shared__ float sm[2][64];
  const int lanes = kWarp ? 32 : blockDim.x;
  const int tid = kWarp ? (threadIdx.x & 31) : threadIdx.x;
  const int per = kWarp ? kWarpRows : 1;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int phase = 0;
  launch_dependents();
  grid_dependency_wait();
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per + (kWarp ? threadIdx.x >> 5 : 0); row < p.rows;
       row += step, phase ^= 1) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = static_cast<const T*>(p.residual) + row * p.ldr;
    T* so = static_cast<T*>(p.sum_out) + row * p.lds;
    Raw<T, VEC> xr[NV], rr[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = (v * lanes + tid) * VEC;
      xr[v] = zero<T, VEC>();
      rr[v] = zero<T, VEC>();
      if (k < p.cols) {
        xr[v] = load<T, VEC>(x + k);
        if (p.residual) rr[v] = load<T, VEC>(r + k);
      }
    }
    float u[NV][VEC];
    float ssq = 0.0f, amax = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = (v * lanes + tid) * VEC;
      float s[VEC], g[VEC];
      to_float(xr[v], s);
      if (p.residual) {
        to_float(rr[v], g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[j] = round_to(s[j] + g[j], T());
      }
      if (k < p.cols) {
        if (p.sum_out) store<T, VEC>(so + k, from_float(s, T()));
        if (p.gamma) load_floats<VEC>(p.gamma + k, g);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        ssq = fmaf(s[j], s[j], ssq);
        u[v][j] = p.gamma && k < p.cols ? __fmul_rn(s[j], g[j]) : s[j];
        amax = max_nan(amax, fabsf(u[v][j]));
      }
    }
    if constexpr (kWarp) {
      ssq = warp_sum(ssq);
      amax = warp_max_nan(amax);
    } else {
      cta_reduce(ssq, amax, sm[phase]);
    }
    const RowScale o = row_scale_of(ssq, amax, p.eps, p.cols);
    if (tid == 0) {
      p.row_scale[row] = o.scale;
      if (p.rstd) p.rstd[row] = o.rstd;
    }
    int8_t* q = p.q + row * p.cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = (v * lanes + tid) * VEC;
      if (k >= p.cols) break;
      uint32_t w[(VEC + 3) / 4] = {};
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        w[j / 4] |= static_cast<uint32_t>(quant(u[v][j], o.inv) & 0xFF) << (8 * (j & 3));
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(q + k) = make_uint2(w[0], w[1]);
      else if constexpr (VEC == 4)
        *reinterpret_cast<uint32_t*>(q + k) = w[0];
      else
        q[k] = static_cast<int8_t>(w[0]);
    }
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
    const RowScale o = row_scale_of(ssq, amax, p.eps, p.cols);
    if (threadIdx.x == 0) {
      p.row_scale[row] = o.scale;
      if (p.rstd) p.rstd[row] = o.rstd;
    }
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float s[1];
      if (p.sum_out)
        to_float(load<T, 1>(so + k), s);  // this thread wrote it (it may lie over x or residual)
      else
        s[0] = sum_at(k);
      p.q[row * p.cols + k] =
          static_cast<int8_t>(quant(p.gamma ? __fmul_rn(s[0], __ldg(p.gamma + k)) : s[0], o.inv));
    }
  }
}

template <class T, int VEC, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : bwd_threads(NV * VEC)) norm_bwd_kernel(const BwdArgs p) {
  __shared__ float sm[2][64];
  extern __shared__ float sums[];  // kWarp: [cols], the CTA's column sums
  const int lanes = kWarp ? 32 : blockDim.x;
  const int tid = kWarp ? (threadIdx.x & 31) : threadIdx.x;
  const int warp = threadIdx.x >> 5;
  const int per = kWarp ? kWarpRows : 1;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int phase = 0;
  float g[NV][VEC], acc[NV][VEC];
  launch_dependents();
  grid_dependency_wait();
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int k = (v * lanes + tid) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      g[v][j] = 1.0f;
      acc[v][j] = 0.0f;
    }
    if (p.gamma && k < p.cols) load_floats<VEC>(p.gamma + k, g[v]);
  }
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per + (kWarp ? warp : 0); row < p.rows;
       row += step, phase ^= 1) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* sp = static_cast<const T*>(p.s) + row * p.lds;
    const T* ds = static_cast<const T*>(p.dsum) + row * p.lddsum;
    Raw<T, VEC> dyr[NV], sr[NV], dr[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = (v * lanes + tid) * VEC;
      dyr[v] = zero<T, VEC>();
      sr[v] = zero<T, VEC>();
      dr[v] = zero<T, VEC>();
      if (k < p.cols) {
        dyr[v] = load<T, VEC>(dy + k);
        sr[v] = load<T, VEC>(sp + k);
        if (p.dsum) dr[v] = load<T, VEC>(ds + k);
      }
    }
    const float rstd = p.rstd[row];
    float dot = 0.0f, unused = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float a[VEC], s[VEC];
      to_float(dyr[v], a);
      to_float(sr[v], s);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dot = fmaf(a[j] * g[v][j], s[j], dot);
        acc[v][j] = fmaf(a[j], s[j] * rstd, acc[v][j]);
      }
    }
    if constexpr (kWarp)
      dot = warp_sum(dot);
    else
      cta_reduce(dot, unused, sm[phase]);
    // rstd s bounded by sqrt(cols) / |s|: scale before squaring
    const float c = rstd * (dot * rstd * inv_cols);
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = (v * lanes + tid) * VEC;
      if (k >= p.cols) break;
      float a[VEC], s[VEC], d[VEC];
      to_float(dyr[v], a);
      to_float(sr[v], s);
      to_float(dr[v], d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] = fmaf(rstd, fmaf(-c, s[j], a[j] * g[v][j]), d[j]);
      store<T, VEC>(dx + k, from_float(d, T()));
    }
  }
  if (!p.partial) return;
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.cols;
  if constexpr (kWarp) {
    // the CTA's warps add their sums in turn, in a fixed order
    for (int w = 0; w < kWarpRows; ++w) {
      if (warp == w) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int k = (v * lanes + tid) * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (k + j < p.cols) sums[k + j] = (w ? sums[k + j] : 0.0f) + acc[v][j];
        }
      }
      __syncthreads();
    }
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) out[k] = sums[k];
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = (v * lanes + tid) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (k + j < p.cols) out[k + j] = acc[v][j];
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
    float dot = 0.0f, unused = 0.0f;
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float a[1], s[1];
      to_float(load<T, 1>(dy + k), a);
      to_float(load<T, 1>(sp + k), s);
      dot = fmaf(p.gamma ? a[0] * __ldg(p.gamma + k) : a[0], s[0], dot);
    }
    cta_reduce(dot, unused, sm[phase]);
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

// How a row of `units` vectors is dealt to threads.  Many rows (two an SM or
// more): a warp a row up to MAXNV vectors a lane, else the fewest vectors a
// thread that leave the CTA at 256 threads, so that several CTAs an SM overlap
// their barriers.  Few rows: the fewest vectors a thread that fit a CTA, for
// the shortest time to one row.
struct Shape {
  bool warp;
  int nv, threads;
};

template <int VEC, int MAXNV>
bool pick(int64_t units, int64_t rows, int sms, int (*max_threads)(int), Shape& s) {
  const bool many = rows >= 2 * static_cast<int64_t>(sms);
  s.warp = many && units <= 32 * MAXNV;
  if (s.warp) {
    s.nv = units <= 32 * (MAXNV / 4) ? MAXNV / 4 : units <= 32 * (MAXNV / 2) ? MAXNV / 2 : MAXNV;
    s.threads = 32 * kWarpRows;
    return true;
  }
  for (int pass = many ? 0 : 1; pass < 2; ++pass)
    for (s.nv = MAXNV / 4; s.nv <= MAXNV; s.nv *= 2) {
      const int64_t t = (units + s.nv - 1) / s.nv;
      if (t <= (pass ? max_threads(s.nv * VEC) : 256)) {
        s.threads = t > 0 ? static_cast<int>((t + 31) / 32 * 32) : 32;
        return true;
      }
    }
  return false;
}

template <class T, int VEC, int NV>
int fwd_nv(const FwdArgs& p, const Shape& sh, int sms, cudaStream_t s) {
  const int64_t per = sh.warp ? kWarpRows : 1;
  int64_t grid = (p.rows + per - 1) / per;
  const int64_t cap = static_cast<int64_t>(sms) * (2048 / sh.threads) * 4;
  if (grid > cap) grid = cap;
  return sh.warp ? launch(norm_fwd_kernel<T, VEC, NV, true>, grid, sh.threads, 0, s, 1, p)
                 : launch(norm_fwd_kernel<T, VEC, NV, false>, grid, sh.threads, 0, s, 1, p);
}

template <class T, int VEC, int MAXNV>
int fwd_vec(const FwdArgs& p, int sms, cudaStream_t s) {
  Shape sh;
  if (!pick<VEC, MAXNV>((p.cols + VEC - 1) / VEC, p.rows, sms, fwd_threads, sh)) {
    const int64_t grid = p.rows < 4 * sms ? p.rows : 4 * sms;
    return launch(norm_fwd_long_kernel<T>, grid, 1024, 0, s, 1, p);
  }
  if (sh.nv == MAXNV / 4) return fwd_nv<T, VEC, MAXNV / 4>(p, sh, sms, s);
  if (sh.nv == MAXNV / 2) return fwd_nv<T, VEC, MAXNV / 2>(p, sh, sms, s);
  return fwd_nv<T, VEC, MAXNV>(p, sh, sms, s);
}

template <class T, int VEC, int NV>
int bwd_nv(const BwdArgs& p, const Shape& sh, int sms, int max_parts, int* parts, cudaStream_t s) {
  const int64_t per = sh.warp ? kWarpRows : 1;
  int64_t grid = (p.rows + per - 1) / per;
  int64_t cap = static_cast<int64_t>(sms) * 3;
  if (cap > max_parts) cap = max_parts;
  if (grid > cap) grid = cap;
  *parts = static_cast<int>(grid);
  const size_t smem = sh.warp ? static_cast<size_t>(p.cols) * 4 : 0;
  return sh.warp ? launch(norm_bwd_kernel<T, VEC, NV, true>, grid, sh.threads, smem, s, 1, p)
                 : launch(norm_bwd_kernel<T, VEC, NV, false>, grid, sh.threads, 0, s, 1, p);
}

template <class T, int VEC, int MAXNV>
int bwd_vec(const BwdArgs& p, int sms, int max_parts, int* parts, cudaStream_t s) {
  Shape sh;
  if (!pick<VEC, MAXNV>((p.cols + VEC - 1) / VEC, p.rows, sms, bwd_threads, sh)) {
    if (p.partial) {
      const int64_t tiles = (p.cols + 31) / 32;
      int64_t n = (p.rows + 7) / 8;
      if (n > 16) n = 16;
      if (n > max_parts) n = max_parts;
      *parts = static_cast<int>(n);
      const int st = launch(norm_dgamma_kernel<T>, tiles * n, 256, 0, s, 1, p, *parts);
      if (st != T3_OK) return st;
    }
    const int64_t grid = p.rows < 4 * sms ? p.rows : 4 * sms;
    return launch(norm_bwd_long_kernel<T>, grid, 1024, 0, s, 1, p);
  }
  if (sh.nv == MAXNV / 4) return bwd_nv<T, VEC, MAXNV / 4>(p, sh, sms, max_parts, parts, s);
  if (sh.nv == MAXNV / 2) return bwd_nv<T, VEC, MAXNV / 2>(p, sh, sms, max_parts, parts, s);
  return bwd_nv<T, VEC, MAXNV>(p, sh, sms, max_parts, parts, s);
}

bool vec_rows(const void* p, int64_t ld, int esize) {
  return !p || (aligned(p, 16) && (ld * esize) % 16 == 0);
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
  if (dtype == T3_OUT_BF16)
    return vec ? nm::fwd_vec<vec::bf16, 8, 4>(p, sms, s) : nm::fwd_vec<vec::bf16, 1, 32>(p, sms, s);
  return vec ? nm::fwd_vec<float, 4, 4>(p, sms, s) : nm::fwd_vec<float, 1, 32>(p, sms, s);
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
  int parts = 0, st;
  if (dtype == T3_OUT_BF16)
    st = vec ? nm::bwd_vec<vec::bf16, 8, 4>(p, sms, kMaxColParts, &parts, s)
             : nm::bwd_vec<vec::bf16, 1, 32>(p, sms, kMaxColParts, &parts, s);
  else
    st = vec ? nm::bwd_vec<float, 4, 4>(p, sms, kMaxColParts, &parts, s)
             : nm::bwd_vec<float, 1, 32>(p, sms, kMaxColParts, &parts, s);
  if (st != T3_OK || !dgamma) return st;
  return launch_col_finish(workspace, parts, cols, dgamma, s);
}

}  // namespace t3
