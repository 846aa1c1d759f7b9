// t3_norm.cuh -- what the norms in front of a product share (t3_norm.cu: root mean square,
// t3_layernorm.cu: mean and deviation): int8 codes of a row, reductions over a CTA and over
// groups of its warps, the columns of rows on any boundary, partial column sums, and the
// choice of threads.
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

// As many CTAs as keep their rows' boundaries alike.
template <int VEC>
int64_t alike(int64_t grid, int64_t rows, int64_t ld, int groups) {
  if (grid * groups >= rows) return grid;  // a row each
  int64_t m = VEC;
  for (int64_t step = ld * groups; m > 1 && step % 2 == 0; step /= 2) m /= 2;
  return grid / m * m;
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
