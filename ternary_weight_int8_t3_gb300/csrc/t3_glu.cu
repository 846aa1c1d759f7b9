// t3_glu.cu -- what follows the two products of a gated feed-forward block: scales, biases,
// the gate's activation and the product of both, and the gradient of that.
//
// What it computes, for exact int32 products x_g and x_u over one A:
//   z_i = (x_i row_scale) scale_i + bias_i,  pre_i = z_i,  out = act(z_g) z_u
// and backward, for the gradient dy of out:
//   dgate = dy z_u act'(z_g),   dup = dy act(z_g),
//   dgate_bias[c] = sum over rows of dgate,   dup_bias[c] = sum over rows of dup
// Everything is float until the one rounding of each output.  Most products end in
// their own epilogue; the kernel here serves those that leave int32 results (few rows over
// many weights, unaligned operands).
//
// What bounds it: memory (forward 8 bytes in and 2 to 12 out per element, backward three
// reads and two writes).  Backward, a lane holds eight neighbouring columns (four floats, or one
// where rows are not 16-byte vectors) and a CTA's eight warps take rows in turn, so that the
// column sums stay in registers over all rows of the CTA; the CTA writes one partial
// row, and a second kernel adds the partial rows in a fixed order.  Measured, bf16: backward 16384 x 3456 107 us
// (5.3 TB/s), 4096 x 3456 27.5; forward behind the two products of 27 x 8192 x 8192 2 of 26 us.
#include <algorithm>

#include "t3_vec.cuh"

namespace t3 {
namespace gl {

using namespace vec;

struct Args {
  const int32_t *gate, *up;
  int64_t ldx;
  void* out;
  GluArgs e;
  int64_t rows, cols, tiles;
};

// A thread holds VEC columns (their scales and biases in registers) and takes
// every gridDim / tiles-th row.
template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(256) glu_epilogue_kernel(const Args p) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x % p.tiles) * 256 + threadIdx.x) * VEC;
  const int64_t step = gridDim.x / p.tiles;
  launch_dependents();
  grid_dependency_wait();
  if (c >= p.cols) return;
  float cs[2][VEC], bias[2][VEC];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      cs[i][j] = p.e.scale[i] ? __ldg(p.e.scale[i] + c + j) : 1.0f;
      bias[i][j] = p.e.bias[i] ? __ldg(p.e.bias[i] + c + j) : 0.0f;
    }
  }
#pragma unroll 2
  for (int64_t r = blockIdx.x / p.tiles; r < p.rows; r += step) {
    const int64_t at = r * p.cols + c;
    const float rs = p.e.row_scale ? __ldg(p.e.row_scale + r) : 1.0f;
    float z[2][VEC];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t* x = (i ? p.up : p.gate) + r * p.ldx + c;
      if constexpr (VEC == 4) {
        const int4 v = *reinterpret_cast<const int4*>(x);
        z[i][0] = __int2float_rn(v.x);
        z[i][1] = __int2float_rn(v.y);
        z[i][2] = __int2float_rn(v.z);
        z[i][3] = __int2float_rn(v.w);
      } else {
        z[i][0] = __int2float_rn(x[0]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) z[i][j] = __fadd_rn(__fmul_rn(__fmul_rn(z[i][j], rs), cs[i][j]), bias[i][j]);
      if (p.e.pre[i]) store<T, VEC>(static_cast<T*>(p.e.pre[i]) + at, from_float(z[i], T()));
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) z[0][j] = __fmul_rn(act<ACT>(z[0][j]), z[1][j]);
    store<T, VEC>(static_cast<T*>(p.out) + at, from_float(z[0], T()));
  }
}

// act(z) and act'(z) from one exponential.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& value, float& slope) {
  if constexpr (ACT == T3_ACT_SILU) {
    const Logistic s = logistic(z);
    value = z * s.pos;
    slope = s.slope == 0.0f ? s.pos : fmaf(z, s.slope, s.pos);  // far out: no infinity times zero
  } else if constexpr (ACT == T3_ACT_GELU) {
    const float z2 = z * z;
    const Logistic s = logistic(kGeluC * z * fmaf(kGeluA, z2, 1.0f));
    value = z * s.pos;
    slope = s.slope == 0.0f ? s.pos : fmaf(z * s.slope, kGeluC * fmaf(3.0f * kGeluA, z2, 1.0f), s.pos);
  } else {
    value = act<ACT>(z);
    slope = act_slope<ACT>(z);
  }
}

struct BwdArgs {
  const void *dy, *gate, *up;
  void *dgate, *dup;
  // partial rows of the column sums (null without one), ldp floats from row to row
  float* partial[2];
  int64_t ldp;
  int64_t rows, cols;
  int parts;
};

constexpr int kUnroll = 2;  // rows a warp has in flight

template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(256) glu_bwd_kernel(const BwdArgs p) {
  __shared__ float sm[2][8][32 * VEC + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % p.parts;
  const int64_t c = (static_cast<int64_t>(blockIdx.x / p.parts) * 32 + lane) * VEC;
  const T* dy = static_cast<const T*>(p.dy);
  const T* gate = static_cast<const T*>(p.gate);
  const T* up = static_cast<const T*>(p.up);
  T* dgate = static_cast<T*>(p.dgate);
  T* dup = static_cast<T*>(p.dup);
  float acc[2][VEC] = {};
  launch_dependents();
  grid_dependency_wait();
  // this part's rows: an equal contiguous share, its warps in turn
  const int64_t r0 = p.rows * part / p.parts, r1 = p.rows * (part + 1) / p.parts;
  if (c < p.cols)
    for (int64_t r = r0 + warp; r < r1; r += 8 * kUnroll) {
      Raw<T, VEC> a[kUnroll], g[kUnroll], u[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        a[i] = zero<T, VEC>();
        g[i] = zero<T, VEC>();
        u[i] = zero<T, VEC>();
        if (r + 8 * i < r1) {
          a[i] = load<T, VEC>(dy + (r + 8 * i) * p.cols + c);
          g[i] = load<T, VEC>(gate + (r + 8 * i) * p.cols + c);
          u[i] = load<T, VEC>(up + (r + 8 * i) * p.cols + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        float d[VEC], z[VEC], o[VEC];
        to_float(a[i], d);
        to_float(g[i], z);
        to_float(u[i], o);
        if (r + 8 * i < r1) {  // zeros behind the last row would meet act(0) and its slope alike, at a cost
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float value, slope;
            act_both<ACT>(z[j], value, slope);
            o[j] = d[j] * o[j] * slope;
            d[j] *= value;
            acc[0][j] += o[j];
            acc[1][j] += d[j];
          }
          if (dgate) store<T, VEC>(dgate + (r + 8 * i) * p.cols + c, from_float(o, T()));
          if (dup) store<T, VEC>(dup + (r + 8 * i) * p.cols + c, from_float(d, T()));
        }
      }
    }
  if (!p.partial[0] && !p.partial[1]) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) sm[i][warp][lane * VEC + j] = acc[i][j];
  __syncthreads();
  for (int k = threadIdx.x; k < 2 * 32 * VEC; k += 256) {
    const int i = k / (32 * VEC), at = k - i * 32 * VEC;
    const int64_t col = static_cast<int64_t>(blockIdx.x / p.parts) * 32 * VEC + at;
    if (p.partial[i] && col < p.cols) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += sm[i][w][at];
      p.partial[i][static_cast<int64_t>(part) * p.ldp + col] = t;
    }
  }
}

template <class T, int VEC>
int epilogue_act(Args p, int sms, cudaStream_t s) {
  p.tiles = (p.cols + 256 * VEC - 1) / (256 * VEC);
  // about eight CTAs an SM
  const int64_t groups = std::min<int64_t>(p.rows, std::max<int64_t>(1, 8ll * sms / p.tiles));
  const int64_t grid = p.tiles * groups;
  switch (p.e.act) {
    case T3_ACT_RELU: return launch(glu_epilogue_kernel<T, VEC, T3_ACT_RELU>, grid, 256, 0, s, 1, p);
    case T3_ACT_RELU2: return launch(glu_epilogue_kernel<T, VEC, T3_ACT_RELU2>, grid, 256, 0, s, 1, p);
    case T3_ACT_SILU: return launch(glu_epilogue_kernel<T, VEC, T3_ACT_SILU>, grid, 256, 0, s, 1, p);
    case T3_ACT_GELU: return launch(glu_epilogue_kernel<T, VEC, T3_ACT_GELU>, grid, 256, 0, s, 1, p);
    default: return launch(glu_epilogue_kernel<T, VEC, T3_ACT_NONE>, grid, 256, 0, s, 1, p);
  }
}

// One part writes the column sums themselves.
template <class T, int VEC>
int bwd_act(BwdArgs p, int act, float* const (&sums)[2], int sms, int* parts, cudaStream_t s) {
  const int64_t tiles = (p.cols + 32 * VEC - 1) / (32 * VEC);
  // at most four CTAs an SM, each with at least one round of rows a warp
  const int64_t n = std::max<int64_t>(
      1, std::min<int64_t>({4ll * sms / tiles, (p.rows + 8 * kUnroll - 1) / (8 * kUnroll), kMaxColParts}));
  p.parts = *parts = static_cast<int>(n);
  for (int i = 0; i < 2; ++i)
    if (n == 1 && sums[i]) p.partial[i] = sums[i];
  const int64_t grid = tiles * n;
  switch (act) {
    case T3_ACT_RELU: return launch(glu_bwd_kernel<T, VEC, T3_ACT_RELU>, grid, 256, 0, s, 1, p);
    case T3_ACT_RELU2: return launch(glu_bwd_kernel<T, VEC, T3_ACT_RELU2>, grid, 256, 0, s, 1, p);
    case T3_ACT_SILU: return launch(glu_bwd_kernel<T, VEC, T3_ACT_SILU>, grid, 256, 0, s, 1, p);
    case T3_ACT_GELU: return launch(glu_bwd_kernel<T, VEC, T3_ACT_GELU>, grid, 256, 0, s, 1, p);
    default: return launch(glu_bwd_kernel<T, VEC, T3_ACT_NONE>, grid, 256, 0, s, 1, p);
  }
}

}  // namespace gl

int launch_glu_epilogue(const int32_t* gate, const int32_t* up, int64_t ldx, void* out, const GluArgs& e, int64_t rows,
                        int64_t cols, int kind, int sms, cudaStream_t s) {
  const gl::Args p{gate, up, ldx, out, e, rows, cols, 0};
  const int64_t es = kind == T3_OUT_BF16 ? 8 : 16;
  const bool vec4 = cols % 4 == 0 && ldx % 4 == 0 && vec::aligned(gate, 16) && vec::aligned(up, 16) &&
                    vec::aligned(out, es) && vec::aligned(e.pre[0], es) && vec::aligned(e.pre[1], es);
  if (kind == T3_OUT_BF16)
    return vec4 ? gl::epilogue_act<vec::bf16, 4>(p, sms, s) : gl::epilogue_act<vec::bf16, 1>(p, sms, s);
  return vec4 ? gl::epilogue_act<float, 4>(p, sms, s) : gl::epilogue_act<float, 1>(p, sms, s);
}

int launch_glu_bwd(const void* dy, const void* gate, const void* up, int act, void* dgate, void* dup,
                   float* dgate_bias, float* dup_bias, int64_t rows, int64_t cols, int dtype, float* workspace,
                   int sms, cudaStream_t s) {
  float* const sums[2] = {dgate_bias, dup_bias};
  const bool both = dgate_bias && dup_bias;
  const gl::BwdArgs p{dy, gate, up, dgate, dup,
                      {dgate_bias ? workspace : nullptr, dup_bias ? workspace + (both ? cols : 0) : nullptr},
                      both ? 2 * cols : cols, rows, cols, 0};
  const int v = dtype == T3_OUT_BF16 ? 8 : 4;
  const bool vec = cols % v == 0 && vec::aligned(dy, 16) && vec::aligned(gate, 16) && vec::aligned(up, 16) &&
                   vec::aligned(dgate, 16) && vec::aligned(dup, 16);
  int parts = 0, st;
  if (dtype == T3_OUT_BF16)
    st = vec ? gl::bwd_act<vec::bf16, 8>(p, act, sums, sms, &parts, s)
             : gl::bwd_act<vec::bf16, 1>(p, act, sums, sms, &parts, s);
  else
    st = vec ? gl::bwd_act<float, 4>(p, act, sums, sms, &parts, s) : gl::bwd_act<float, 1>(p, act, sums, sms, &parts, s);
  if (st != T3_OK || (!dgate_bias && !dup_bias) || parts == 1) return st;
  if (both) return launch_col_finish2(workspace, parts, cols, dgate_bias, dup_bias, s);
  return launch_col_finish(workspace, parts, cols, dgate_bias ? dgate_bias : dup_bias, s);
}

}  // namespace t3
