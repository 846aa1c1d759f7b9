// t3_norm.cuh -- the kernels of the norms in front of a product (t3_norm.cu: root mean
// square; t3_layernorm.cu: mean and deviation): the residual added on the way in, int8
// rows with one scale each on the way out, and the gradient.  What each computes and what
// was measured stands in those two files; here is what they share.
//
// What bounds them: memory.  A row is read once and written once.  A persistent
// grid of one wave takes rows in turn; a thread's columns are the same in every
// row, so their gains (and, backward, their column sums) stay in registers, and the
// next row's operands are loaded while this one is reduced and written.  Many
// rows take 16 elements a thread forward and 8 backward (8 and 8 where rows
// go element by element: arrays whose rows lie differently to 16-byte boundaries), few rows as few as 1024 threads
// allow, for the shortest time to one row; rows longer than the registers
// hold are read again from memory.  Backward, narrow rows share a CTA in groups of warps that
// meet at barriers of their own.  Column sums: each CTA adds its groups' sums in turn,
// writes one partial row, and a second small kernel adds the partial rows in a
// fixed order.
#pragma once
#include "t3_vec.cuh"

namespace t3 {
namespace nm {

using namespace vec;

// Threads a CTA may have when each holds EPT elements of a row: up to 16384
// elements a row forward (one float an element is kept) and 8192 backward (the
// gain, the column sum and three operands), within 64 to 128 registers a thread.
constexpr int fwd_threads(int ept) { return ept <= 16 ? 1024 : 16384 / ept; }
// Columns from which vectors that begin inside a row pay (bf16, forward and
// backward: 8000 x 1001 13.8 and 20.6 us, element by element 24.1 and 46.7; 16000 x 243
// 11.0 and 12.7, 13.3 and 26.6).
constexpr int64_t kOddCols = 64;
constexpr int bwd_threads(int ept) { return ept <= 8 ? 1024 : 8192 / ept; }
// The layer norm keeps a second column sum an element: half the threads at 8 elements, so
// that they have 128 registers.
constexpr int layer_bwd_threads(int ept) { return ept <= 4 ? 1024 : ept <= 8 ? 512 : 8192 / ept; }

struct FwdArgs {
  const void *x, *residual;
  int64_t ldx, ldr, lds;
  const float *gamma, *beta;  // beta, mean: the layer norm
  float eps;
  int8_t* q;
  float *row_scale, *mean, *rstd;
  void* sum_out;
  int64_t rows, cols;
};

struct BwdArgs {
  const void *dy, *s, *dsum;
  int64_t lddy, lds, lddsum, lddx;
  const float *mean, *rstd, *gamma;
  void* dx;
  // partial rows of the column sums of dy s rstd (null without dgamma) and, in the layer
  // norm, of dy (null without dbeta), ldp floats from row to row
  float *partial, *partial_dy;
  int64_t ldp;
  int64_t rows, cols;
  int groups;      // row groups a CTA (norm_bwd_kernel)
};

// Rows whose largest element is below kSmallRow are quantized 2^64 times larger, since 127 /
// max|u| would pass the float range; a power of two changes no rounding.
constexpr float kSmallRow = 7.888609e-31f;  // 2^-100
constexpr float kSmallUp = 18446744073709551616.0f;

__device__ __forceinline__ int quant(float u, float inv, float up) {
  const int q = __float2int_rn(__fmul_rn(__fmul_rn(u, up), inv));  // NaN (of a row that is not finite) gives 0
  return q > 127 ? 127 : (q < -127 ? -127 : q);
}

// 127 / max|u up|, or 0 for a row of zeros or one that is not finite: an element
// of u is not, or the squares overflow their sum.
__device__ __forceinline__ float inverse_of(float ssq, float amax, float& up) {
  const bool finite = ssq < __int_as_float(0x7f800000) && amax < __int_as_float(0x7f800000);
  up = amax < kSmallRow ? kSmallUp : 1.0f;
  return finite && amax > 0.0f ? __fdiv_rn(127.0f, __fmul_rn(amax, up)) : 0.0f;
}

// One thread: the row's scale (NaN where it is not finite) and rstd.
__device__ __forceinline__ void put_scales(const FwdArgs& p, int64_t row, float ssq, float amax) {
  const float rstd =
      __fdiv_rn(1.0f, __fsqrt_rn(p.cols > 0 ? __fdiv_rn(ssq, static_cast<float>(p.cols)) + p.eps : p.eps));
  const bool finite = ssq < __int_as_float(0x7f800000) && amax < __int_as_float(0x7f800000);
  p.row_scale[row] = finite ? __fdiv_rn(__fmul_rn(amax, rstd), 127.0f) : __int_as_float(0x7fffffff);
  if (p.rstd) p.rstd[row] = rstd;
}

// The same for the layer norm: m2 the sum of squared deviations from the mean, amax = max|y|.
__device__ __forceinline__ void put_layer_scales(const FwdArgs& p, int64_t row, float mean, float m2, float rstd,
                                                 float amax) {
  const bool finite = m2 < __int_as_float(0x7f800000) && amax < __int_as_float(0x7f800000);
  p.row_scale[row] = finite ? __fdiv_rn(amax, 127.0f) : __int_as_float(0x7fffffff);
  if (p.mean) p.mean[row] = mean;
  if (p.rstd) p.rstd[row] = rstd;
}

__device__ __forceinline__ float deviation(const FwdArgs& p, float m2) {
  return __fdiv_rn(1.0f, __fsqrt_rn(p.cols > 0 ? __fdiv_rn(m2, static_cast<float>(p.cols)) + p.eps : p.eps));
}

// Four codes of four floats u * inv that lie in [-127, 127]: adding 1.5 * 2^23
// rounds to the nearest integer, ties to even, into the low bits.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t x = __float_as_uint(__fadd_rn(__fmul_rn(a, inv), kMagic));
  const uint32_t y = __float_as_uint(__fadd_rn(__fmul_rn(b, inv), kMagic));
  const uint32_t z = __float_as_uint(__fadd_rn(__fmul_rn(c, inv), kMagic));
  const uint32_t w = __float_as_uint(__fadd_rn(__fmul_rn(d, inv), kMagic));
  return prmt(prmt(x, y, 0x0040u), prmt(z, w, 0x0040u), 0x5410u);
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
  if (warps <= 4) {  // reading them all beats five more shuffles of each
    a = sm[0];
    b = sm[32];
    for (int i = 1; i < warps; ++i) {
      a += sm[i];
      b = max_nan(b, sm[32 + i]);
    }
    return;
  }
  a = warp_sum(lane < warps ? sm[lane] : 0.0f);
  b = warp_max_nan(lane < warps ? sm[32 + lane] : 0.0f);
}

// NaN-keeping maximum over the CTA's threads; `sm` holds 32 floats that no one reads any more.
__device__ __forceinline__ float cta_max(float b, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  b = warp_max_nan(b);
  if (warps == 1) return b;
  if (lane == 0) sm[warp] = b;
  __syncthreads();
  if (warps <= 4) {
    b = sm[0];
    for (int i = 1; i < warps; ++i) b = max_nan(b, sm[i]);
    return b;
  }
  return warp_max_nan(lane < warps ? sm[lane] : 0.0f);
}

// A row's mean and sum of squared deviations from the warps' own (mean m of n elements,
// sum m2 of squared deviations from m), with one barrier: the deviations of the whole are
// m2 plus n (m - mean)^2 of every warp, and no square is taken of anything but a difference from a
// mean.  counts: every warp's n; sm holds 64 floats that no one reads any more.
__device__ __forceinline__ void cta_moments(float& m, float& m2, const float* counts, float inv_cols, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (warps == 1) return;
  if (lane == 0) {
    sm[warp] = m;
    sm[32 + warp] = m2;
  }
  __syncthreads();
  if (warps <= 4) {
    m = 0.0f;
    for (int i = 0; i < warps; ++i) m = fmaf(counts[i], sm[i], m);
    m *= inv_cols;
    m2 = 0.0f;
    for (int i = 0; i < warps; ++i) {
      const float d = sm[i] - m;
      m2 += fmaf(counts[i] * d, d, sm[32 + i]);
    }
    return;
  }
  const float n = lane < warps ? counts[lane] : 0.0f, own = lane < warps ? sm[lane] : 0.0f;
  m = warp_sum(n * own) * inv_cols;
  const float d = own - m;
  m2 = warp_sum(lane < warps ? fmaf(n * d, d, sm[32 + lane]) : 0.0f);
}

// The sum of `a` over a group of `warps` warps, which meets at barrier `bar`;
// `sm` holds a float for each of its warps and alternates from call to call.
__device__ __forceinline__ float group_sum(float a, float* sm, int warp, int warps, int bar) {
  const int lane = threadIdx.x & 31;
  a = warp_sum(a);
  if (warps == 1) return a;
  if (lane == 0) sm[warp] = a;
  named_bar_sync(bar, 32 * warps);
  if (warps <= 4) {
    a = sm[0];
    for (int i = 1; i < warps; ++i) a += sm[i];
    return a;
  }
  return warp_sum(lane < warps ? sm[lane] : 0.0f);
}

// Two sums at once; `sm` holds two floats for each warp of the group.
__device__ __forceinline__ void group_sum2(float& a, float& b, float* sm, int warp, int warps, int bar) {
  const int lane = threadIdx.x & 31;
  a = warp_sum(a);
  b = warp_sum(b);
  if (warps == 1) return;
  if (lane == 0) {
    sm[warp] = a;
    sm[warps + warp] = b;
  }
  named_bar_sync(bar, 32 * warps);
  if (warps <= 4) {
    a = sm[0];
    b = sm[warps];
    for (int i = 1; i < warps; ++i) {
      a += sm[i];
      b += sm[warps + i];
    }
    return;
  }
  a = warp_sum(lane < warps ? sm[lane] : 0.0f);
  b = warp_sum(lane < warps ? sm[warps + lane] : 0.0f);
}

// Rows that do not begin on 16-byte boundaries (kOdd): the vectors begin on the first
// boundary in the row, and the few elements in front of them and behind them go one to
// a thread.  A CTA's rows are a multiple of VEC apart in memory, so that a thread's columns
// stay the same.
template <class T, int VEC, bool kOdd>
struct Columns {
  int head = 0, end;  // the vectors' columns
  int one = 0;        // this thread's single column
  bool has = false;   // whether it has one
  // a row begins `at` elements from p; `t` numbers the threads that share it
  __device__ __forceinline__ Columns(const void* p, int64_t at, int cols, int t) : end(cols) {
    if constexpr (kOdd) {
      const uint64_t lead = (reinterpret_cast<uintptr_t>(p) / sizeof(T) + static_cast<uint64_t>(at)) % VEC;
      head = min(static_cast<int>((VEC - lead) % VEC), cols);
      end = head + (cols - head) / VEC * VEC;
      one = t < head ? t : end + t - head;
      has = one < cols;
    }
  }
};

// kLayer: the layer norm, whose row is reduced twice (its mean and deviation, then max|y|).
template <class T, int VEC, int NV, bool kOdd, bool kLayer>
__global__ void __launch_bounds__(fwd_threads(NV * VEC)) norm_fwd_kernel(const FwdArgs p) {
  __shared__ float sm[2][64];
  __shared__ float counts[kLayer ? 32 : 1];
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
  // kLayer: shifts of this thread's columns, and how many elements its warp has
  float shift[kLayer ? NV : 1][VEC], shifte = 0.0f, count = 0.0f, inv_count = 0.0f;
  const float inv_cols = kLayer && cols > 0 ? __fdiv_rn(1.0f, static_cast<float>(cols)) : 0.0f;
  if constexpr (kLayer) {
    int mine = kOdd && at.has ? 1 : 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + static_cast<int>(v * lanes + threadIdx.x) * VEC;
      if (k < at.end) mine += VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) shift[v][j] = p.beta && k < at.end ? __ldg(p.beta + k + j) : 0.0f;
    }
    if (kOdd && p.beta && at.has) shifte = __ldg(p.beta + at.one);
    count = static_cast<float>(__reduce_add_sync(0xffffffffu, mine));
    inv_count = count > 0.0f ? __fdiv_rn(1.0f, count) : 0.0f;
    if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = count;
    __syncthreads();
  }
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
        if constexpr (kLayer) {
          u[v][j] = s[j];
          ssq += s[j];  // zeros where the thread has no columns
        } else {
          ssq = fmaf(s[j], s[j], ssq);
          u[v][j] = __fmul_rn(s[j], g[v][j]);
          amax = max_nan(amax, fabsf(u[v][j]));
        }
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
        if constexpr (kLayer) {
          ue = se[0];
          ssq += ue;
        } else {
          ssq = fmaf(se[0], se[0], ssq);
          ue = __fmul_rn(se[0], ge);
          amax = max_nan(amax, fabsf(ue));
        }
      }
    }
    fetch(row + gridDim.x);
    if constexpr (kLayer) {
      float mean = warp_sum(ssq) * inv_count, m2 = 0.0f;  // the warp's own
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = at.head + static_cast<int>(v * lanes + threadIdx.x) * VEC;
        if (k >= at.end) break;
#pragma unroll
        for (int j = 0; j < VEC; ++j) m2 = fmaf(u[v][j] - mean, u[v][j] - mean, m2);
      }
      if (kOdd && at.has) m2 = fmaf(ue - mean, ue - mean, m2);
      m2 = warp_sum(m2);
      cta_moments(mean, m2, counts, inv_cols, sm[0]);
      const float rstd = deviation(p, m2);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = at.head + static_cast<int>(v * lanes + threadIdx.x) * VEC;
        if (k >= at.end) break;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          u[v][j] = fmaf(__fmul_rn(u[v][j] - mean, rstd), g[v][j], shift[v][j]);
          amax = max_nan(amax, fabsf(u[v][j]));
        }
      }
      if (kOdd && at.has) {
        ue = fmaf(__fmul_rn(ue - mean, rstd), ge, shifte);
        amax = max_nan(amax, fabsf(ue));
      }
      amax = cta_max(amax, sm[1]);
      if (threadIdx.x == 0) put_layer_scales(p, row, mean, m2, rstd, amax);
      ssq = m2;
    } else {
      cta_reduce(ssq, amax, sm[phase]);
      if (threadIdx.x == 0) put_scales(p, row, ssq, amax);
    }
    float up;
    const float inv = inverse_of(ssq, amax, up);
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
// The layer norm reads it two times more, for the mean and for the deviation.
template <class T, bool kLayer>
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
    float ssq = 0.0f, amax = 0.0f, mean = 0.0f, rstd = 0.0f;
    // kLayer: the element of a row that is normalized; behind the first pass the sum is read
    // where it was written, by the thread that wrote it
    auto y_at = [&](int64_t k) {
      float s[1];
      if (p.sum_out)
        to_float(load<T, 1>(so + k), s);
      else
        s[0] = sum_at(k);
      return fmaf(__fmul_rn(s[0] - mean, rstd), p.gamma ? __ldg(p.gamma + k) : 1.0f, p.beta ? __ldg(p.beta + k) : 0.0f);
    };
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      const float s[1] = {sum_at(k)};
      if (p.sum_out) store<T, 1>(so + k, from_float(s, T()));
      if constexpr (kLayer) {
        ssq += s[0];
      } else {
        ssq = fmaf(s[0], s[0], ssq);
        amax = max_nan(amax, fabsf(p.gamma ? __fmul_rn(s[0], __ldg(p.gamma + k)) : s[0]));
      }
    }
    cta_reduce(ssq, amax, sm[phase]);
    if constexpr (kLayer) {
      mean = __fdiv_rn(ssq, static_cast<float>(p.cols));
      ssq = 0.0f;
      for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
        float s[1];
        if (p.sum_out)
          to_float(load<T, 1>(so + k), s);
        else
          s[0] = sum_at(k);
        ssq = fmaf(s[0] - mean, s[0] - mean, ssq);
      }
      cta_reduce(ssq, amax, sm[phase ^= 1]);
      rstd = deviation(p, ssq);
      for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) amax = max_nan(amax, fabsf(y_at(k)));
      float unused = 0.0f;
      cta_reduce(unused, amax, sm[phase ^= 1]);
      if (threadIdx.x == 0) put_layer_scales(p, row, mean, ssq, rstd, amax);
    } else {
      if (threadIdx.x == 0) put_scales(p, row, ssq, amax);
    }
    float up;
    const float inv = inverse_of(ssq, amax, up);
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      if constexpr (kLayer) {
        p.q[row * p.cols + k] = static_cast<int8_t>(quant(y_at(k), inv, up));
        continue;
      }
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

// to = (add ? from : 0) + v, in 16-byte pieces where there are some and `to` allows
// them (`wide`): a thread's elements one by one would touch 32 sectors a warp and
// store (40 x 8192: 4 us for the partial sums).
template <int VEC>
__device__ __forceinline__ void add_floats(float* to, const float* from, bool add, const float (&v)[VEC], bool wide) {
  float y[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) y[j] = v[j];
  if constexpr (VEC % 4 == 0) {
    if (add) {
#pragma unroll
      for (int j = 0; j < VEC; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(from + j);
        y[j] = f.x + y[j];
        y[j + 1] = f.y + y[j + 1];
        y[j + 2] = f.z + y[j + 2];
        y[j + 3] = f.w + y[j + 3];
      }
    }
    if (wide) {
#pragma unroll
      for (int j = 0; j < VEC; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
      return;
    }
  } else if (add) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) y[j] = from[j] + y[j];
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) to[j] = y[j];
}

// kOne: the CTA is one group; else it has p.groups of them in 256 threads.
// kLayer: the layer norm, with two sums a row and two a column.
template <class T, int VEC, int NV, bool kOne, bool kOdd, bool kLayer>
__global__ void __launch_bounds__(kOne ? (kLayer ? layer_bwd_threads(NV * VEC) : bwd_threads(NV * VEC)) : 256, kOne ? 1 : 3)
    norm_bwd_kernel(const BwdArgs p) {
  __shared__ float sm[2][kLayer ? 64 : 32];
  extern __shared__ __align__(16) float sums[];  // [cols], with more than one group
  const int groups = kOne ? 1 : p.groups;
  const int lanes = blockDim.x / groups, cols = static_cast<int>(p.cols);
  const int group = kOne ? 0 : threadIdx.x / lanes, t = threadIdx.x - group * lanes, warps = lanes >> 5;
  const int64_t each = static_cast<int64_t>(gridDim.x) * groups;
  const Columns<T, VEC, kOdd> at(p.dy, (static_cast<int64_t>(blockIdx.x) * groups + group) * p.lddy, cols, t);
  launch_dependents();
  grid_dependency_wait();
  // this thread's columns: gains, sums, and the next row's operands
  float g[NV][VEC], acc[NV][VEC], next_rstd = 0.0f, next_mean = 0.0f;
  float accd[kLayer ? NV : 1][VEC], accde = 0.0f;  // kLayer: the sums of dy
  float ge = 1.0f, acce = 0.0f;
  Raw<T, VEC> dyr[NV], sr[NV], dr[NV];
  Raw<T, 1> dye = zero<T, 1>(), se = zero<T, 1>(), de = zero<T, 1>();
  auto fetch = [&](int64_t row) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* sp = static_cast<const T*>(p.s) + row * p.lds;
    const T* ds = static_cast<const T*>(p.dsum) + row * p.lddsum;
    if (row < p.rows) next_rstd = p.rstd[row];
    if (kLayer && row < p.rows) next_mean = p.mean[row];
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
      if constexpr (kLayer) accd[v][j] = 0.0f;
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
    const float rstd = next_rstd, mean = next_mean;
    float n[NV][VEC], s[NV][VEC], dot = 0.0f, total = 0.0f;  // total: kLayer, the sum of n
    Raw<T, VEC> d[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      to_float(dyr[v], n[v]);
      to_float(sr[v], s[v]);
      d[v] = dr[v];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if constexpr (kLayer) {  // dy is zero where the thread has no columns
          s[v][j] -= mean;
          accd[v][j] += n[v][j];
        }
        s[v][j] *= rstd;
        acc[v][j] = fmaf(n[v][j], s[v][j], acc[v][j]);
        n[v][j] *= g[v][j];
        if constexpr (kLayer) total += n[v][j];
        dot = fmaf(n[v][j], s[v][j], dot);
      }
    }
    float ne[1] = {}, sse[1] = {}, ye[1] = {};
    if constexpr (kOdd) {  // zeros where the thread has none
      to_float(dye, ne);
      to_float(se, sse);
      to_float(de, ye);
      if constexpr (kLayer) {
        sse[0] -= mean;
        accde += ne[0];
      }
      sse[0] *= rstd;
      acce = fmaf(ne[0], sse[0], acce);
      ne[0] *= ge;
      if constexpr (kLayer) total += ne[0];
      dot = fmaf(ne[0], sse[0], dot);
    }
    fetch(row + each);
    if constexpr (kLayer)
      group_sum2(dot, total, sm[phase] + 2 * group * warps, t >> 5, warps, 1 + group);
    else
      dot = group_sum(dot, sm[phase] + group * warps, t >> 5, warps, 1 + group);
    const float c = dot * inv_cols, level = kLayer ? total * inv_cols : 0.0f;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = at.head + (v * lanes + t) * VEC;
      if (k >= at.end) break;
      float y[VEC];
      to_float(d[v], y);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        y[j] = fmaf(rstd, fmaf(-c, s[v][j], kLayer ? n[v][j] - level : n[v][j]), y[j]);
      store<T, VEC>(dx + k, from_float(y, T()));
    }
    if (kOdd && at.has) {
      ye[0] = fmaf(rstd, fmaf(-c, sse[0], kLayer ? ne[0] - level : ne[0]), ye[0]);
      store<T, 1>(dx + at.one, from_float(ye, T()));
    }
  }
  auto emit = [&](float* out, const float (&a)[NV][VEC], float ae) {
    if constexpr (kOdd) {  // element by element, and then in order
      for (int i = 0; i < groups; ++i) {
        if (group == i) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int k = at.head + (v * lanes + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
              if (k < at.end) sums[k + j] = (i ? sums[k + j] : 0.0f) + a[v][j];
          }
          if (at.has) sums[at.one] = (i ? sums[at.one] : 0.0f) + ae;
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
            if (k < cols) add_floats<VEC>(sums + k, sums + k, i > 0, a[v], true);
          }
        }
        __syncthreads();
      }
      if (group != groups - 1) return;
      const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = at.head + (v * lanes + t) * VEC;
        if (k < cols) add_floats<VEC>(out + k, sums + k, groups > 1, a[v], wide);
      }
    }
  };
  if (p.partial) emit(p.partial + static_cast<int64_t>(blockIdx.x) * p.ldp, acc, acce);
  if constexpr (kLayer) {
    if (p.partial && p.partial_dy) __syncthreads();  // the first sums have been read
    if (p.partial_dy) emit(p.partial_dy + static_cast<int64_t>(blockIdx.x) * p.ldp, accd, accde);
  }
}

// Long rows: dx with the row read twice; the column sums come from
// norm_dgamma_kernel, which runs first (dx may lie over dy or dsum).
template <class T, bool kLayer>
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
    const float rstd = p.rstd[row], mean = kLayer ? p.mean[row] : 0.0f;
    float dot = 0.0f, total = 0.0f;
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float a[1], s[1];
      to_float(load<T, 1>(dy + k), a);
      to_float(load<T, 1>(sp + k), s);
      if constexpr (kLayer) s[0] -= mean;
      const float n = p.gamma ? a[0] * __ldg(p.gamma + k) : a[0];
      if constexpr (kLayer) total += n;
      dot = fmaf(n, s[0], dot);
    }
    {
      float unused = 0.0f;
      cta_reduce(dot, unused, sm[phase]);
      unused = 0.0f;
      if constexpr (kLayer) cta_reduce(total, unused, sm[phase ^= 1]);
    }
    const float c = rstd * (dot * rstd / static_cast<float>(p.cols)), level = total / static_cast<float>(p.cols);
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float a[1], s[1], d[1] = {0.0f};
      to_float(load<T, 1>(dy + k), a);
      to_float(load<T, 1>(sp + k), s);
      if (p.dsum) to_float(load<T, 1>(ds + k), d);
      const float n = p.gamma ? a[0] * __ldg(p.gamma + k) : a[0];
      if constexpr (kLayer)
        d[0] = fmaf(rstd, fmaf(-c, s[0] - mean, n - level), d[0]);
      else
        d[0] = fmaf(rstd, fmaf(-c, s[0], n), d[0]);
      store<T, 1>(dx + k, from_float(d, T()));
    }
  }
}

// Partial column sums of dy s rstd: a CTA takes 32 columns (one a lane) and
// every gridDim.x / tiles-th block of rows; its 8 warps take rows in turn.
template <class T, bool kLayer>
__global__ void __launch_bounds__(256) norm_dgamma_kernel(const BwdArgs p, int parts) {
  __shared__ float sm[kLayer ? 16 : 8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % parts;
  const int64_t k = static_cast<int64_t>(blockIdx.x / parts) * 32 + lane;
  launch_dependents();
  grid_dependency_wait();
  float acc = 0.0f, accd = 0.0f;
  if (k < p.cols)
    for (int64_t row = part * 8 + warp; row < p.rows; row += static_cast<int64_t>(parts) * 8) {
      float a[1], s[1];
      to_float(load<T, 1>(static_cast<const T*>(p.dy) + row * p.lddy + k), a);
      to_float(load<T, 1>(static_cast<const T*>(p.s) + row * p.lds + k), s);
      if constexpr (kLayer) {
        s[0] -= p.mean[row];
        accd += a[0];
      }
      acc = fmaf(a[0], s[0] * p.rstd[row], acc);
    }
  sm[warp][lane] = acc;
  if constexpr (kLayer) sm[8 + warp][lane] = accd;
  __syncthreads();
  if (warp < (kLayer ? 2 : 1) && k < p.cols) {  // warp 1: the sums of dy
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sm[8 * warp + w][lane];
    float* out = warp ? p.partial_dy : p.partial;
    if (out) out[static_cast<int64_t>(part) * p.ldp + k] = t;
  }
}

// ----------------------------------------------------------------- routing

// The fewest vectors a thread (MAXNV / 4, / 2 or MAXNV) that make at least
// `least` elements and fit a CTA.
template <int VEC, int MAXNV>
int pick(int64_t units, int least, int (*max_threads)(int), int* threads) {
  for (int nv = MAXNV / 4; nv <= MAXNV; nv *= 2) {
    if (nv * VEC < least && nv < MAXNV) continue;
    const int64_t t = (units + nv - 1) / nv;
    if (t <= max_threads(nv * VEC)) {
      *threads = t > 0 ? static_cast<int>((t + 31) / 32 * 32) : 32;
      return nv;
    }
  }
  return 0;
}

// Forward: few rows take the fewest elements a thread, many rows 16 or more.
// kOdd: as many CTAs as keep their rows' boundaries alike.
template <int VEC>
int64_t alike(int64_t grid, int64_t rows, int64_t ld, int groups) {
  if (grid * groups >= rows) return grid;  // a row each
  int64_t m = VEC;
  for (int64_t step = ld * groups; m > 1 && step % 2 == 0; step /= 2) m /= 2;
  return grid / m * m;
}

template <class T, int VEC, int MAXNV, bool kOdd, bool kLayer>
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
  if (nv == MAXNV / 4) return launch(norm_fwd_kernel<T, VEC, MAXNV / 4, kOdd, kLayer>, grid, threads, 0, s, 1, p);
  if (nv == MAXNV / 2) return launch(norm_fwd_kernel<T, VEC, MAXNV / 2, kOdd, kLayer>, grid, threads, 0, s, 1, p);
  if (nv == MAXNV) return launch(norm_fwd_kernel<T, VEC, MAXNV, kOdd, kLayer>, grid, threads, 0, s, 1, p);
  return launch(norm_fwd_long_kernel<T, kLayer>, grid, 1024, 0, s, 1, p);
}

// Backward: many rows take 8 elements a thread (more only where the row would not
// fit a CTA).
// One part is the sums themselves: it goes where they are wanted.
template <class T, int VEC, int MAXNV, bool kOdd, bool kLayer>
int bwd_vec(BwdArgs p, float* dgamma, float* dbeta, int sms, int* parts, cudaStream_t s) {
  int (*const most)(int) = kLayer ? layer_bwd_threads : bwd_threads;
  const bool many = p.rows >= 2 * static_cast<int64_t>(sms);
  int threads = 0;
  const int nv = pick<VEC, MAXNV>((p.cols + VEC - 1) / VEC, many ? 8 : 1, most, &threads);
  int64_t grid = 2ll * sms;
  if (nv) {
    // narrow rows: two groups or more in 256 threads, three such CTAs an SM;
    // else a CTA a row, as many as the registers hold
    p.groups = many && nv * VEC == 8 ? 256 / threads : 1;
    if (p.groups < 1) p.groups = 1;
    const bool one = p.groups == 1;
    const int room = (one ? most(nv * VEC) : 768) / (threads * p.groups);
    grid = static_cast<int64_t>(sms) * room;
    const int64_t need = (p.rows + p.groups - 1) / p.groups;
    if (grid > need) grid = need;
    if (grid > kMaxColParts) grid = kMaxColParts;
    if (kOdd) grid = alike<VEC>(grid, p.rows, p.lddy, p.groups);
    *parts = static_cast<int>(grid);
    if (grid == 1 && p.partial) p.partial = dgamma;
    if (grid == 1 && p.partial_dy) p.partial_dy = dbeta;
    const size_t sums = kOdd || !one ? static_cast<size_t>(p.cols) * sizeof(float) : 0;
    if (!one)
      return launch(norm_bwd_kernel<T, VEC, 8 / VEC, false, kOdd, kLayer>, grid, threads * p.groups, sums, s, 1, p);
    if (nv == MAXNV / 4) return launch(norm_bwd_kernel<T, VEC, MAXNV / 4, true, kOdd, kLayer>, grid, threads, sums, s, 1, p);
    if (nv == MAXNV / 2) return launch(norm_bwd_kernel<T, VEC, MAXNV / 2, true, kOdd, kLayer>, grid, threads, sums, s, 1, p);
    return launch(norm_bwd_kernel<T, VEC, MAXNV, true, kOdd, kLayer>, grid, threads, sums, s, 1, p);
  }
  if (p.partial || p.partial_dy) {
    const int64_t tiles = (p.cols + 31) / 32;
    const int64_t n = (p.rows + 7) / 8 < 16 ? (p.rows + 7) / 8 : 16;
    *parts = static_cast<int>(n);
    if (n == 1 && p.partial) p.partial = dgamma;
    if (n == 1 && p.partial_dy) p.partial_dy = dbeta;
    const int st = launch(norm_dgamma_kernel<T, kLayer>, tiles * n, 256, 0, s, 1, p, *parts);
    if (st != T3_OK) return st;
  }
  if (grid > p.rows) grid = p.rows;
  return launch(norm_bwd_long_kernel<T, kLayer>, grid, 1024, 0, s, 1, p);
}

inline bool vec_rows(const void* p, int64_t ld, int esize) {
  return !p || (aligned(p, 16) && (ld * esize) % 16 == 0);
}

// Whether the rows of `p` lie to 16-byte boundaries as those of `q` do (elements of
// `esize` bytes, `v` of them in 16).
inline bool alike_rows(const void* p, int64_t ld, const void* q, int64_t ldq, int esize, int v) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return !p || (a % esize == 0 && b % esize == 0 && (a - b) / esize % v == 0 && (ld - ldq) % v == 0);
}

}  // namespace nm
}  // namespace t3

