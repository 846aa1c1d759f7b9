// t3_epilogue.cu -- what follows a ternary product in a layer: scales, bias,
// activation and residual, and the gradient of the activation with the
// bias's column sums.
//
// What it computes, for an exact int32 product x:
//   z = (x row_scale) col_scale + bias,  pre = z,  out = act(z) + residual
// and backward, for the gradient dy of act(z):
//   dz = dy act'(z),   dbias[c] = sum over rows of dz[r][c]
// Everything is float until the one rounding of each output.  Most products
// apply the forward part in their own epilogue; the kernel here serves those
// that leave an int32 result (split reductions, unaligned operands).
//
// What bounds it: memory (forward 4 bytes in and 2 to 8 out per element,
// backward two reads and a write).  Backward, a lane holds eight neighbouring
// columns (four floats, or one where rows are not 16-byte vectors) and a CTA's
// eight warps take rows in turn, so that the column sums stay in registers
// over all rows of the CTA; the CTA writes one partial row, and a second
// kernel adds the partial rows in a fixed order.
//
// Measured (GB300, of the measured 6784 GB/s): backward with the bias's sums,
// bf16, 4096 x 3456 16.3 us (77 %), 16384 x 3456 54.9 us (91 %).  Laying out
// odd rows for the CTA pairs costs about 3 us at 129 x 4001 and 1500 x 1001 bytes.
#include "t3_vec.cuh"

namespace t3 {
namespace ep {

using namespace vec;

struct Args {
  const int32_t* x;
  int64_t ldx;
  void* out;
  EpilogueArgs e;
  int64_t rows, cols, tiles;
};

// A thread holds VEC columns (their scales and biases in registers) and takes
// every gridDim / tiles-th row.
template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(256) epilogue_kernel(const Args p) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x % p.tiles) * 256 + threadIdx.x) * VEC;
  const int64_t step = gridDim.x / p.tiles;
  launch_dependents();
  grid_dependency_wait();
  if (c >= p.cols) return;
  float cs[VEC], bias[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    cs[j] = 1.0f;
    bias[j] = 0.0f;
  }
  if (p.e.col_scale) load_floats<VEC>(p.e.col_scale + c, cs);
  if (p.e.bias) load_floats<VEC>(p.e.bias + c, bias);
#pragma unroll 2
  for (int64_t r = blockIdx.x / p.tiles; r < p.rows; r += step) {
    const int64_t at = r * p.cols + c;
    const float rs = p.e.row_scale ? __ldg(p.e.row_scale + r) : 1.0f;
    float y[VEC], t[VEC] = {};
    if constexpr (VEC == 4) {
      const int4 v = *reinterpret_cast<const int4*>(p.x + r * p.ldx + c);
      y[0] = __int2float_rn(v.x);
      y[1] = __int2float_rn(v.y);
      y[2] = __int2float_rn(v.z);
      y[3] = __int2float_rn(v.w);
    } else {
      y[0] = __int2float_rn(p.x[r * p.ldx + c]);
    }
    if (p.e.residual) to_float(load<T, VEC>(static_cast<const T*>(p.e.residual) + at), t);
#pragma unroll
    for (int j = 0; j < VEC; ++j) y[j] = __fadd_rn(__fmul_rn(__fmul_rn(y[j], rs), cs[j]), bias[j]);
    if (p.e.pre) store<T, VEC>(static_cast<T*>(p.e.pre) + at, from_float(y, T()));
#pragma unroll
    for (int j = 0; j < VEC; ++j) y[j] = __fadd_rn(act<ACT>(y[j]), t[j]);
    store<T, VEC>(static_cast<T*>(p.out) + at, from_float(y, T()));
  }
}

// Rows of `len` bytes, one after the other at any alignment, to rows of `pitch`
// bytes (a multiple of 16), zeros behind each and in rows from `rows` to `rows2`.
struct AlignArgs {
  const uint8_t* src;
  int64_t rows, len;
  uint8_t* dst;
  int64_t rows2, pitch;
};

// Bytes [at, at + 16) of the array [0, end): whole words where they lie inside.
__device__ __forceinline__ uint4 gather16(const uint8_t* src, int64_t at, int64_t end) {
  const uint64_t a = reinterpret_cast<uint64_t>(src) + at;
  const int sh = static_cast<int>(a & 3) * 8;
  const int64_t w = at - (sh >> 3);  // the aligned word's offset
  uint32_t x[5];
  if (w >= 0 && w + 20 <= end) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(a & ~3ull);
#pragma unroll
    for (int i = 0; i < 5; ++i) x[i] = __ldg(p + i);
  } else {
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      x[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t o = w + 4 * i + j;
        if (o >= 0 && o < end) x[i] |= static_cast<uint32_t>(__ldg(src + o)) << (8 * j);
      }
    }
  }
  return make_uint4(__funnelshift_r(x[0], x[1], sh), __funnelshift_r(x[1], x[2], sh),
                    __funnelshift_r(x[2], x[3], sh), __funnelshift_r(x[3], x[4], sh));
}

__global__ void __launch_bounds__(256) align_rows_kernel(const AlignArgs a, const AlignArgs b, int64_t blocks_a) {
  const bool first = blockIdx.x < blocks_a;
  const AlignArgs& p = first ? a : b;
  launch_dependents();
  grid_dependency_wait();
  const int64_t i = (blockIdx.x - (first ? 0 : blocks_a)) * 256 + threadIdx.x;
  const int64_t each = p.pitch / 16, r = i / each, c = (i - r * each) * 16;
  if (r >= p.rows2) return;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (r < p.rows && c < p.len) {
    v = gather16(p.src, r * p.len + c, p.rows * p.len);
    const int64_t left = p.len - c;  // bytes of this row
    if (left < 16) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = left >= 4 * j + 4 ? w[j] : left <= 4 * j ? 0u : w[j] & (0xFFFFFFFFu >> (8 * (4 * j + 4 - left)));
    }
  }
  *reinterpret_cast<uint4*>(p.dst + r * p.pitch + c) = v;
}

struct BwdArgs {
  const void *dy, *z;
  void* dz;
  float* partial;  // [parts][cols] or null
  int64_t rows, cols;
  int parts;
};

constexpr int kUnroll = 4;  // rows a warp has in flight

template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(256) act_bwd_kernel(const BwdArgs p) {
  __shared__ float sm[8][32 * VEC + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % p.parts;
  const int64_t c = (static_cast<int64_t>(blockIdx.x / p.parts) * 32 + lane) * VEC;
  const T* dy = static_cast<const T*>(p.dy);
  const T* z = static_cast<const T*>(p.z);
  T* dz = static_cast<T*>(p.dz);
  float acc[VEC] = {};
  launch_dependents();
  grid_dependency_wait();
  // this part's rows: an equal contiguous share, its warps in turn
  const int64_t r0 = p.rows * part / p.parts, r1 = p.rows * (part + 1) / p.parts;
  if (c < p.cols)
    for (int64_t r = r0 + warp; r < r1; r += 8 * kUnroll) {
      Raw<T, VEC> a[kUnroll], b[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        a[i] = zero<T, VEC>();
        b[i] = zero<T, VEC>();
        if (r + 8 * i < r1) {
          a[i] = load<T, VEC>(dy + (r + 8 * i) * p.cols + c);
          if (ACT != T3_ACT_NONE) b[i] = load<T, VEC>(z + (r + 8 * i) * p.cols + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        float d[VEC], t[VEC];
        to_float(a[i], d);
        to_float(b[i], t);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          if (ACT != T3_ACT_NONE) d[j] *= act_slope<ACT>(t[j]);
          acc[j] += d[j];
        }
        if (dz && r + 8 * i < r1) store<T, VEC>(dz + (r + 8 * i) * p.cols + c, from_float(d, T()));
      }
    }
  if (!p.partial) return;
#pragma unroll
  for (int j = 0; j < VEC; ++j) sm[warp][lane * VEC + j] = acc[j];
  __syncthreads();
  for (int k = threadIdx.x; k < 32 * VEC; k += 256) {
    const int64_t col = static_cast<int64_t>(blockIdx.x / p.parts) * 32 * VEC + k;
    if (col < p.cols) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += sm[w][k];
      p.partial[static_cast<int64_t>(part) * p.cols + col] = t;
    }
  }
}

// 32 columns a CTA, its 32 warps take the partial rows in turn.
__global__ void __launch_bounds__(1024) col_finish_kernel(const float* partial, int parts, int64_t cols,
                                                          float* out) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  launch_dependents();
  grid_dependency_wait();
  float acc = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int r = warp; r < parts; r += 32) acc += partial[static_cast<int64_t>(r) * cols + c];
  }
  sm[warp][lane] = acc;
  __syncthreads();
  const float t = warp_sum(sm[lane][warp]);  // warp w: column w's 32 sums
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && col < cols) out[col] = t;
}

template <class T, int VEC>
int epilogue_act(Args p, int sms, cudaStream_t s) {
  p.tiles = (p.cols + 256 * VEC - 1) / (256 * VEC);
  // about eight CTAs an SM
  int64_t groups = 8ll * sms / p.tiles > 1 ? 8ll * sms / p.tiles : 1;
  if (groups > p.rows) groups = p.rows;
  const int64_t grid = p.tiles * groups;
  switch (p.e.act) {
    case T3_ACT_RELU: return launch(epilogue_kernel<T, VEC, T3_ACT_RELU>, grid, 256, 0, s, 1, p);
    case T3_ACT_RELU2: return launch(epilogue_kernel<T, VEC, T3_ACT_RELU2>, grid, 256, 0, s, 1, p);
    case T3_ACT_SILU: return launch(epilogue_kernel<T, VEC, T3_ACT_SILU>, grid, 256, 0, s, 1, p);
    case T3_ACT_GELU: return launch(epilogue_kernel<T, VEC, T3_ACT_GELU>, grid, 256, 0, s, 1, p);
    default: return launch(epilogue_kernel<T, VEC, T3_ACT_NONE>, grid, 256, 0, s, 1, p);
  }
}

// One part writes the column sums themselves.
template <class T, int VEC>
int act_bwd_act(BwdArgs p, int act, float* dbias, int sms, int* parts, cudaStream_t s) {
  const int64_t tiles = (p.cols + 32 * VEC - 1) / (32 * VEC);
  // at most four CTAs an SM (one wave: a few CTAs more would double the time),
  // each with at least one round of rows a warp
  int64_t n = 4ll * sms / tiles > 1 ? 4ll * sms / tiles : 1;
  const int64_t most = (p.rows + 8 * kUnroll - 1) / (8 * kUnroll);
  if (n > most) n = most;
  if (n > kMaxColParts) n = kMaxColParts;
  p.parts = *parts = static_cast<int>(n);
  if (n == 1 && dbias) p.partial = dbias;
  const int64_t grid = tiles * n;
  switch (act) {
    case T3_ACT_RELU: return launch(act_bwd_kernel<T, VEC, T3_ACT_RELU>, grid, 256, 0, s, 1, p);
    case T3_ACT_RELU2: return launch(act_bwd_kernel<T, VEC, T3_ACT_RELU2>, grid, 256, 0, s, 1, p);
    case T3_ACT_SILU: return launch(act_bwd_kernel<T, VEC, T3_ACT_SILU>, grid, 256, 0, s, 1, p);
    case T3_ACT_GELU: return launch(act_bwd_kernel<T, VEC, T3_ACT_GELU>, grid, 256, 0, s, 1, p);
    default: return launch(act_bwd_kernel<T, VEC, T3_ACT_NONE>, grid, 256, 0, s, 1, p);
  }
}

}  // namespace ep

int launch_align_rows(const uint8_t* a, int64_t rows_a, int64_t len_a, uint8_t* a2, int64_t rows_a2, int64_t pitch_a,
                      const uint8_t* b, int64_t rows_b, int64_t len_b, uint8_t* b2, int64_t rows_b2, int64_t pitch_b,
                      cudaStream_t s) {
  const ep::AlignArgs x{a, rows_a, len_a, a2, a ? rows_a2 : 0, pitch_a}, y{b, rows_b, len_b, b2, rows_b2, pitch_b};
  const int64_t blocks_a = a ? (rows_a2 * (pitch_a / 16) + 255) / 256 : 0;
  const int64_t blocks_b = (rows_b2 * (pitch_b / 16) + 255) / 256;
  return vec::launch(ep::align_rows_kernel, blocks_a + blocks_b, 256, 0, s, 1, x, y, blocks_a);
}

int launch_epilogue(const int32_t* x, int64_t ldx, void* out, const EpilogueArgs& e, int64_t rows, int64_t cols,
                    int kind, int sms, cudaStream_t s) {
  const ep::Args p{x, ldx, out, e, rows, cols, 0};
  const int64_t es = kind == T3_OUT_BF16 ? 8 : 16;
  const bool vec4 = cols % 4 == 0 && ldx % 4 == 0 && vec::aligned(x, 16) && vec::aligned(out, es) &&
                    vec::aligned(e.pre, es) && vec::aligned(e.residual, es) &&
                    vec::aligned(e.col_scale, 16) && vec::aligned(e.bias, 16);
  if (kind == T3_OUT_BF16)
    return vec4 ? ep::epilogue_act<vec::bf16, 4>(p, sms, s) : ep::epilogue_act<vec::bf16, 1>(p, sms, s);
  return vec4 ? ep::epilogue_act<float, 4>(p, sms, s) : ep::epilogue_act<float, 1>(p, sms, s);
}

int launch_col_finish(const float* partial, int parts, int64_t cols, float* out, cudaStream_t s) {
  return vec::launch(ep::col_finish_kernel, (cols + 31) / 32, 1024, 0, s, 1, partial, parts, cols, out);
}

int launch_act_bwd(const void* dy, const void* z, int act, void* dz, float* dbias, int64_t rows,
                   int64_t cols, int dtype, float* workspace, int sms, cudaStream_t s) {
  const ep::BwdArgs p{dy, z, dz, dbias ? workspace : nullptr, rows, cols, 0};
  const int v = dtype == T3_OUT_BF16 ? 8 : 4;
  const bool vec = cols % v == 0 && vec::aligned(dy, 16) && vec::aligned(z, 16) && vec::aligned(dz, 16);
  int parts = 0, st;
  if (dtype == T3_OUT_BF16)
    st = vec ? ep::act_bwd_act<vec::bf16, 8>(p, act, dbias, sms, &parts, s)
             : ep::act_bwd_act<vec::bf16, 1>(p, act, dbias, sms, &parts, s);
  else
    st = vec ? ep::act_bwd_act<float, 4>(p, act, dbias, sms, &parts, s)
             : ep::act_bwd_act<float, 1>(p, act, dbias, sms, &parts, s);
  if (st != T3_OK || !dbias || parts == 1) return st;
  return launch_col_finish(workspace, parts, cols, dbias, s);
}

}  // namespace t3
