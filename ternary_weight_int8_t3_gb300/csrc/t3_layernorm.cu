// t3_layernorm.cu -- the layer norm in front of a product: the residual added on the
// way in, int8 rows with one scale each on the way out, and the gradient of it.
//
// What it computes, for a row of `cols` elements with float gains gamma and shifts beta:
//   s = x + r, rounded once to the rows' type (the residual stream it is kept in)
//   mean = sum(s) / cols,   rstd = 1 / sqrt(sum((s - mean)^2) / cols + eps)
//   y = (s - mean) rstd gamma + beta
//   row_scale = max|y| / 127,   q = rint(y * (127 / max|y|)) in [-127, 127]
// The squares are taken of differences from a mean, never as sum(s^2) - mean^2, so that a row
// far from zero keeps its deviation: each warp takes its own mean and its squares from that, with the sum of
// the differences themselves, which tells how far that mean is from the right one.  So the warps' moments
// join without the error of a float sum over the row (cta_moments): the mean is rounded once at its own size,
// and a row of equal elements has no deviation.  With a shift, max|y| needs the
// deviation first, so a row is reduced twice, with a barrier each.  Backward, with the rounding passed
// straight through, h = (s - mean) rstd and n = dy gamma:
//   dx = rstd (n - mean(n) - h mean(n h)) + dsum
//   dgamma = sum over rows of dy h,   dbeta = sum over rows of dy
//
// What bounds it: memory; a row is read once and written once.  A persistent grid of one
// wave takes rows in turn; a thread's columns are the same in every row, so their gains,
// shifts and column sums stay in registers.  A row spends longer between its load and its end than
// under the root mean square (two reductions instead of one), so one row ahead is too little:
// rows that are 16-byte vectors come through a ring of kAhead + 1 rows in shared
// memory, which each thread fills by asynchronous copies of its own columns and reads back
// alone, so that it needs no barrier.  Operands whose rows lie differently to 16-byte boundaries, and
// rows longer than a CTA holds, go element by element and are read again from memory for every
// pass.  Column sums as in t3_norm.cu: partial rows, added in a fixed order.
//
// Measured (replays of a graph, the kernel's own bytes).  bf16 with residual and shift: 16384 x 1280 forward 28 us (5.3 TB/s),
// 16384 x 3456 66 (6.0) and 99 backward (4.6: two thirds of the issue slots and of the memory's rate), 4096 x 8192 43 and 64, 4096 x
// 16384 87, 1 x 8192 4.8.  float: 16384 x 1280 52 and 57, 8192 x 3456 64 and 75, 1782 x 729 5.8 and 14.
#include <algorithm>

#include "t3_norm.cuh"

namespace t3 {
namespace ln {

using namespace vec;
using namespace nm;

constexpr int kAhead = 2;  // rows on their way while one is reduced, where shared memory holds as many

struct FwdArgs {
  const void* from[2];  // x, the residual
  int64_t ld[2], lds;
  int64_t skip[2], lds_skip, q_skip;  // elements from one row of a CTA's to the next
  const float *gamma, *beta;
  float eps;
  int8_t* q;
  float *row_scale, *mean, *rstd;
  void* sum_out;
  int64_t rows, cols;
  int ahead;  // rows on their way, 0 to kAhead
};

struct BwdArgs {
  const void* from[3];  // dy, s, dsum
  int64_t ld[3], lddx;
  int64_t skip[3], dx_skip;  // elements from one row of a group's to the next
  const float *mean, *rstd, *gamma;
  void* dx;
  // partial rows of the sums of dy h (null without dgamma) and of dy (null without
  // dbeta), ldp floats from row to row
  float *partial, *partial_dy;
  int64_t ldp;
  int64_t rows, cols;
  int groups;  // row groups a CTA
  int ahead;
};

__device__ __forceinline__ bool row_finite(float m2, float amax) {
  return m2 < __int_as_float(0x7f800000) && amax < __int_as_float(0x7f800000);
}

// One thread: what is kept of a row.  m2: the sum of squared deviations.
__device__ __forceinline__ void put_row(const FwdArgs& p, int64_t row, float mean, float m2, float rstd, float amax) {
  p.row_scale[row] = row_finite(m2, amax) ? __fmul_rn(amax, 1.0f / 127.0f) : __int_as_float(0x7fffffff);
  if (p.mean) p.mean[row] = mean;
  if (p.rstd) p.rstd[row] = rstd;
}

// 1 / sqrt: the hardware's approximation, 2 ulp.
__device__ __forceinline__ float deviation(const FwdArgs& p, float m2, float inv_cols) {
  return rsqrtf(fmaf(m2, inv_cols, p.eps));
}

// 127 / max|y up| (a reciprocal of 1 ulp), or 0 for a row of zeros or one that is not finite.
__device__ __forceinline__ float inverse_row(float m2, float amax, float& up) {
  up = amax < kSmallRow ? kSmallUp : 1.0f;
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(__fmul_rn(amax, up)));
  return row_finite(m2, amax) && amax > 0.0f ? 127.0f * r : 0.0f;
}

// Elements in pairs, so that a packed instruction takes the place of two: the kernels are bound by
// their instructions as much as by memory (16384 x 1280 forward took 41 us element by element).
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 wide(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void pairs(const Raw<bf16, 8>& r, float2 (&f)[4]) {
  f[0] = wide(r.v.x);
  f[1] = wide(r.v.y);
  f[2] = wide(r.v.z);
  f[3] = wide(r.v.w);
}
__device__ __forceinline__ void pairs(const Raw<float, 4>& r, float2 (&f)[2]) {
  f[0] = make_float2(r.v.x, r.v.y);
  f[1] = make_float2(r.v.z, r.v.w);
}
__device__ __forceinline__ Raw<bf16, 8> narrow(const float2 (&f)[4], bf16) {
  Raw<bf16, 8> r;
  r.v = make_uint4(pack(f[0].x, f[0].y), pack(f[1].x, f[1].y), pack(f[2].x, f[2].y), pack(f[3].x, f[3].y));
  return r;
}
__device__ __forceinline__ Raw<float, 4> narrow(const float2 (&f)[2], float) {
  Raw<float, 4> r;
  r.v = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  return r;
}
// a + b rounded once to the type.  (A float sum of two bf16 that is not exact is nowhere near the middle between
// two bf16, so rounding it a second time would give the same.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ Raw<bf16, 8> sum(const Raw<bf16, 8>& a, const Raw<bf16, 8>& b) {
  Raw<bf16, 8> r;
  r.v = make_uint4(add_bf16x2(a.v.x, b.v.x), add_bf16x2(a.v.y, b.v.y), add_bf16x2(a.v.z, b.v.z), add_bf16x2(a.v.w, b.v.w));
  return r;
}
__device__ __forceinline__ Raw<float, 4> sum(const Raw<float, 4>& a, const Raw<float, 4>& b) {
  Raw<float, 4> r;
  r.v = make_float4(a.v.x + b.v.x, a.v.y + b.v.y, a.v.z + b.v.z, a.v.w + b.v.w);
  return r;
}
template <class T>
__device__ __forceinline__ Raw<T, 1> sum(const Raw<T, 1>& a, const Raw<T, 1>& b) {
  float x[1], y[1];
  to_float(a, x);
  to_float(b, y);
  x[0] += y[0];
  return from_float(x, T());
}

// max(m, |a|, |b|) that keeps a NaN.
__device__ __forceinline__ float absmax(float m, float2 f) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(f.x), "f"(f.y));
  return r;
}

// NaN-keeping maximum of magnitudes over a warp, one instruction.
__device__ __forceinline__ float warp_absmax(float v) {
  float r;
  asm("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The same over the CTA; `sm` holds 32 floats that no one reads any more.
__device__ __forceinline__ float cta_absmax(float b, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  b = warp_absmax(b);
  if (warps == 1) return b;
  if (lane == 0) sm[warp] = b;
  __syncthreads();
  return warp_absmax(lane < warps ? sm[lane] : 0.0f);
}

// How many of a row's elements each warp has.
struct Counts {
  int head, end, cols, lanes;
  template <int VEC, int NV>
  __device__ __forceinline__ float of(int warp) const {
    int n = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) n += min(max(end - head - (v * lanes + 32 * warp) * VEC, 0), 32 * VEC);
    const int single = head + cols - end - 32 * warp;  // those outside the vectors go one to a thread
    return static_cast<float>(n + min(max(single, 0), 32));
  }
};

// The sum of n squared differences from a mean that lies `off` from some value near it, from the sum m2 of the
// squared differences from that value and `rest` of the differences themselves: m2 - 2 off rest + n off^2.
__device__ __forceinline__ float about(float m2, float rest, float n, float off) {
  return fmaf(off, fmaf(n, off, -2.0f * rest), m2);
}
// A sum of squares is not below zero for its roundings (a NaN stays).
__device__ __forceinline__ float no_less(float m2) { return max_nan(m2, 0.0f); }

// Two sums over a warp at the shuffles of one: a's in lanes 0 to 15, b's in the others.
__device__ __forceinline__ float warp_sum_halves(float a, float b) {
  const bool upper = threadIdx.x & 16;
  float x = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
  for (int i = 8; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
  return x;
}

// A row's mean and sum of squared deviations from the warps' own (a mean m of n elements as a float sum has
// it, and the sum m2 of squared differences from it), with one barrier.  The means are added as
// differences from the first one and with how far each is from the right one, so that only the last addition rounds at
// their own size; no square is taken of anything but a difference from a mean.  n: the count of warp
// `lane`; sm holds 96 floats that no one reads any more, the last 32 of them by now the sums of each warp's
// differences from its mean.
__device__ __forceinline__ void cta_moments(float& m, float& m2, float n, float inv_cols, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) {
    sm[warp] = m;
    sm[32 + warp] = m2;
  }
  __syncthreads();
  const bool has = lane < warps;
  const float own = has ? sm[lane] : 0.0f, own2 = has ? sm[32 + lane] : 0.0f, rest = has ? sm[64 + lane] : 0.0f;
  const float first = sm[0];
  m = fmaf(warp_sum(fmaf(n, own - first, rest)), inv_cols, first);  // n is 0 behind the last warp
  m2 = no_less(warp_sum(about(own2, rest, n, m - own)));
}

// Two sums over a group of `warps` warps, which meets at barrier `bar`; `sm` holds two floats
// for each of its warps and alternates from call to call.
__device__ __forceinline__ void group_sums(float& a, float& b, float* sm, int warp, int warps, int bar) {
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

__device__ __forceinline__ void copy16_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

// A thread's columns of a row's operand: NV vectors of 16 bytes and, in odd rows, a single element.
template <class T, int VEC, int NV>
struct Piece {
  Raw<T, VEC> v[NV];
  Raw<T, 1> one;
};

// The operands of the rows to come.  The vectors: a ring of ahead + 1 rows in shared
// memory, a slot a thread, operand and vector; the single elements a row ahead in registers.
template <class T, int VEC, int NV, bool kOdd, int kOperands>
struct Rows {
  static_assert(sizeof(T) * VEC == 16, "slots of 16 bytes");
  const T* from[kOperands];  // this thread's first column of the next row to fetch; null: zeros
  int left;                  // rows of this CTA's or group's still to fetch
  Columns<T, VEC, kOdd> at;
  int column0, end, stride;  // this thread's vectors: column0, column0 + stride, ... below end
  uint8_t* mine;             // this thread's first slot
  int pitch, stage, ahead;   // bytes from slot to slot of a row, and of a row
  int put = 0, take = 0;
  Raw<T, 1> next[kOperands];

  // t: this thread's number among the `lanes` of its row, `threads` those of the CTA
  __device__ __forceinline__ Rows(const void* const (&base)[kOperands], const int64_t (&ld)[kOperands], int64_t rows,
                                  int64_t first, int64_t step, int cols, int t, int lanes, int threads, uint4* ring,
                                  int ahead_)
      : at(base[0], first * ld[0], cols, t) {
    left = first < rows ? static_cast<int>((rows - first + step - 1) / step) : 0;
    column0 = at.head + t * VEC;
    stride = lanes * VEC;
    end = at.end;
#pragma unroll
    for (int i = 0; i < kOperands; ++i)
      from[i] = base[i] ? static_cast<const T*>(base[i]) + first * ld[i] + column0 : nullptr;
    mine = reinterpret_cast<uint8_t*>(ring) + threadIdx.x * 16;
    pitch = threads * 16;
    stage = kOperands * NV * pitch;
    ahead = ahead_;
  }
  __device__ __forceinline__ int column(int v) const { return column0 + v * stride; }
  // the next row's operands on their way, as the newest of the ring
  __device__ __forceinline__ void fetch(const int64_t (&skip)[kOperands]) {
    if (left > 0) {
      uint8_t* to = mine + put;
#pragma unroll
      for (int i = 0; i < kOperands; ++i)
        if (from[i]) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
            if (column(v) < end) copy16_async(to + (i * NV + v) * pitch, from[i] + v * stride);
          from[i] += skip[i];
        }
    }
    --left;
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = put == ahead * stage ? 0 : put + stage;
  }
  // the single elements of row `row`, read by their address in the kernel's parameters (pointers
  // kept from row to row would take registers that the odd kernels do not have)
  template <class Args>
  __device__ __forceinline__ void fetch_near(const Args& p, int64_t row) {
    if constexpr (kOdd) {
#pragma unroll
      for (int i = 0; i < kOperands; ++i) {
        next[i] = zero<T, 1>();
        if (p.from[i] && at.has && row < p.rows)
          next[i] = load<T, 1>(static_cast<const T*>(p.from[i]) + row * p.ld[i] + at.one);
      }
    }
  }
  template <class Args>
  __device__ __forceinline__ void start(const Args& p, int64_t row) {
    fetch_near(p, row);
    for (int i = 0; i < ahead; ++i) fetch(p.skip);
  }
  // this row's operands; those of a later one follow
  template <class Args>
  __device__ __forceinline__ void operands(const Args& args, int64_t row_behind, Piece<T, VEC, NV> (&p)[kOperands]) {
    fetch(args.skip);
    if (ahead == 2)
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (ahead == 1)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    const uint8_t* out = mine + take;
#pragma unroll
    for (int i = 0; i < kOperands; ++i) {
      if constexpr (kOdd) p[i].one = next[i];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        p[i].v[v] = zero<T, VEC>();
        if (from[i] && column(v) < end)
          p[i].v[v].v = *reinterpret_cast<const decltype(p[i].v[v].v)*>(out + (i * NV + v) * pitch);
      }
    }
    take = take == ahead * stage ? 0 : take + stage;
    fetch_near(args, row_behind);
  }
};
static_assert(kAhead == 2, "the waits in operands()");

// Threads a CTA may have forward: 80 registers at 16 elements.
constexpr int front_threads(int ept) { return ept <= 8 ? 1024 : ept <= 16 ? 768 : 16384 / ept; }

template <class T, int VEC, int NV, bool kOdd>
__global__ void __launch_bounds__(front_threads(NV * VEC)) layer_fwd_kernel(const FwdArgs p) {
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float sm[4][32], count[2][32];
  constexpr int P = VEC / 2;
  const int cols = static_cast<int>(p.cols), tid = threadIdx.x, lanes = blockDim.x;
  Rows<T, VEC, NV, kOdd, 2> rows(p.from, p.ld, p.rows, blockIdx.x, gridDim.x, cols, tid, lanes,
                                 lanes, ring, p.ahead);
  const Columns<T, VEC, kOdd>& at = rows.at;
  launch_dependents();
  grid_dependency_wait();
  rows.start(p, blockIdx.x);
  // this thread's columns: their gains and shifts
  float2 g[NV][P], b[NV][P];
  float ge = 1.0f, be = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int k = rows.column(v);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      g[v][j] = both(1.0f);
      b[v][j] = both(0.0f);
      if (k < rows.end) {
        if (p.gamma) g[v][j] = make_float2(__ldg(p.gamma + k + 2 * j), __ldg(p.gamma + k + 2 * j + 1));
        if (p.beta) b[v][j] = make_float2(__ldg(p.beta + k + 2 * j), __ldg(p.beta + k + 2 * j + 1));
      }
    }
  }
  if (kOdd && at.has) {
    if (p.gamma) ge = __ldg(p.gamma + at.one);
    if (p.beta) be = __ldg(p.beta + at.one);
  }
  const Counts counts{at.head, at.end, cols, lanes};
  const int lane = tid & 31;
  // the warps' counts and their reciprocals (in registers they cost spills)
  if (tid < 32) {
    const float n = lane < lanes >> 5 ? counts.of<VEC, NV>(lane) : 0.0f;
    count[0][lane] = n;
    count[1][lane] = n > 0.0f ? __fdiv_rn(1.0f, n) : 0.0f;
  }
  __syncthreads();
  const float inv_cols = cols > 0 ? __fdiv_rn(1.0f, static_cast<float>(cols)) : 0.0f;
  T* so = static_cast<T*>(p.sum_out) + blockIdx.x * p.lds + rows.column0;
  int8_t* q = p.q + blockIdx.x * p.cols + rows.column0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, so += p.lds_skip, q += p.q_skip) {
    Piece<T, VEC, NV> in[2];
    rows.operands(p, row + gridDim.x, in);
    float2 u[NV][P], total = both(0.0f);
    float ue = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (p.from[1]) in[0].v[v] = sum(in[0].v[v], in[1].v[v]);
      if (p.sum_out && rows.column(v) < rows.end) store<T, VEC>(so + v * rows.stride, in[0].v[v]);
      pairs(in[0].v[v], u[v]);
#pragma unroll
      for (int j = 0; j < P; ++j) total = __fadd2_rn(total, u[v][j]);  // zeros where the thread has no columns
    }
    float first = total.x + total.y;
    if constexpr (kOdd) {
      if (p.from[1]) in[0].one = sum(in[0].one, in[1].one);
      if (at.has) {
        if (p.sum_out) store<T, 1>(so + (at.one - rows.column0), in[0].one);
        float x1[1];
        to_float(in[0].one, x1);
        ue = x1[0];
        first += ue;
      }
    }
    // How far a warp's mean is from the right one: the sum of the differences from it.  bf16 elements that are alike
    // enough for it to matter have few bits in common units, so that their float sum is exact and tells.
    constexpr bool kSums = sizeof(T) == 2;
    first = warp_sum(first);
    float mean = first * count[1][tid >> 5];  // the warp's own
    if (kSums && lane == 0) sm[2][tid >> 5] = fmaf(-count[0][tid >> 5], mean, first);
    float2 square = both(0.0f), diff = both(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (rows.column(v) < rows.end) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float2 d = __fadd2_rn(u[v][j], both(-mean));
          square = __ffma2_rn(d, d, square);
          if (!kSums) diff = __fadd2_rn(diff, d);
        }
      }
    float m2 = square.x + square.y, rest = diff.x + diff.y;
    if (kOdd && at.has) {
      m2 = fmaf(ue - mean, ue - mean, m2);
      if (!kSums) rest += ue - mean;
    }
    if (kSums) {
      m2 = warp_sum(m2);
    } else {
      m2 = warp_sum_halves(m2, rest);
      if (lane == 16) sm[2][tid >> 5] = m2;
      m2 = __shfl_sync(0xffffffffu, m2, 0);
    }
    cta_moments(mean, m2, count[0][lane], inv_cols, sm[0]);
    const float rstd = deviation(p, m2, inv_cols);
    float amax = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (rows.column(v) < rows.end) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          u[v][j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(u[v][j], both(-mean)), both(rstd)), g[v][j], b[v][j]);
          amax = absmax(amax, u[v][j]);
        }
      }
    if (kOdd && at.has) {
      ue = fmaf(__fmul_rn(ue - mean, rstd), ge, be);
      amax = absmax(amax, make_float2(ue, 0.0f));
    }
    amax = cta_absmax(amax, sm[3]);
    if (tid == 0) put_row(p, row, mean, m2, rstd, amax);
    float up;
    const float inv = inverse_row(m2, amax, up);
    // y * inv within [-127, 127]: not for rows that are not finite (codes 0) nor small ones
    if (inv > 0.0f && up == 1.0f) {
      const float2 magic = both(12582912.0f);  // rounds to the nearest integer, into the low bits
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (rows.column(v) < rows.end) {
          uint32_t w[P];
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const float2 t = __fadd2_rn(__fmul2_rn(u[v][j], both(inv)), magic);
            w[j] = prmt(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040u);
          }
          if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(q + v * rows.stride) = make_uint2(prmt(w[0], w[1], 0x5410u), prmt(w[2], w[3], 0x5410u));
          else
            *reinterpret_cast<uint32_t*>(q + v * rows.stride) = prmt(w[0], w[1], 0x5410u);
        }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (rows.column(v) < rows.end) {
#pragma unroll
          for (int j = 0; j < P; ++j) {
            q[v * rows.stride + 2 * j] = static_cast<int8_t>(quant(u[v][j].x, inv, up));
            q[v * rows.stride + 2 * j + 1] = static_cast<int8_t>(quant(u[v][j].y, inv, up));
          }
        }
    }
    if (kOdd && at.has) q[at.one - rows.column0] = static_cast<int8_t>(quant(ue, inv, up));
  }
}

// Sums of `a` over the CTA's threads for the long rows; `sm` alternates between two areas
// from call to call.
__device__ __forceinline__ float cta_sum(float a, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  a = warp_sum(a);
  if (lane == 0) sm[warp] = a;
  __syncthreads();
  return warp_sum(lane < warps ? sm[lane] : 0.0f);
}

// Other rows: one CTA a row, read once a pass (mean, deviation, max|y|, codes), behind
// the first from sum_out where it is written.
template <class T>
__global__ void __launch_bounds__(1024) layer_fwd_long_kernel(const FwdArgs p) {
  __shared__ float sm[4][32];
  launch_dependents();
  grid_dependency_wait();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.from[0]) + row * p.ld[0];
    const T* r = static_cast<const T*>(p.from[1]) + row * p.ld[1];
    T* so = static_cast<T*>(p.sum_out) + row * p.lds;
    auto sum_at = [&](int64_t k) {
      float a[1], b[1];
      to_float(load<T, 1>(x + k), a);
      if (!p.from[1]) return a[0];
      to_float(load<T, 1>(r + k), b);
      return round_to(a[0] + b[0], T());
    };
    auto again = [&](int64_t k) {  // this thread wrote it (it may lie over x or residual)
      if (!p.sum_out) return sum_at(k);
      float s[1];
      to_float(load<T, 1>(so + k), s);
      return s[0];
    };
    float total = 0.0f, rest = 0.0f, m2 = 0.0f, amax = 0.0f;
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      const float s[1] = {sum_at(k)};
      if (p.sum_out) store<T, 1>(so + k, from_float(s, T()));
      total += s[0];
    }
    const float inv_cols = __fdiv_rn(1.0f, static_cast<float>(p.cols));
    const float near = cta_sum(total, sm[0]) * inv_cols;  // the mean but for its sum's roundings
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      const float d = again(k) - near;
      rest += d;
      m2 = fmaf(d, d, m2);
    }
    rest = cta_sum(rest, sm[3]);
    m2 = cta_sum(m2, sm[1]);
    const float mean = fmaf(rest, inv_cols, near);
    m2 = no_less(about(m2, rest, static_cast<float>(p.cols), mean - near));
    const float rstd = deviation(p, m2, inv_cols);
    auto y_at = [&](int64_t k) {
      return fmaf(__fmul_rn(again(k) - mean, rstd), p.gamma ? __ldg(p.gamma + k) : 1.0f,
                  p.beta ? __ldg(p.beta + k) : 0.0f);
    };
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) amax = absmax(amax, make_float2(y_at(k), 0.0f));
    amax = cta_absmax(amax, sm[2]);
    if (threadIdx.x == 0) put_row(p, row, mean, m2, rstd, amax);
    float up;
    const float inv = inverse_row(m2, amax, up);
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x)
      p.q[row * p.cols + k] = static_cast<int8_t>(quant(y_at(k), inv, up));
  }
}

// Threads a CTA may have backward, two column sums an element.  bf16 rows want warps (72
// registers at 8 elements: 16384 x 3456 100 us, with 128 registers and half the warps 107), float rows, which are nearer to the
// memory's rate, registers to have more loads in flight (8192 x 3456 76 us with 128, 112 with 72).
template <int VEC>
constexpr int back_threads(int ept) { return ept <= 4 ? 1024 : ept <= 8 ? (VEC == 8 ? 896 : 512) : 8192 / ept; }
constexpr int kBackCtas = 3;  // CTAs of 256 threads an SM, where several row groups share one

// kOne: the CTA is one group; else it has p.groups of them in 256 threads.
template <class T, int VEC, int NV, bool kOne, bool kOdd>
__global__ void __launch_bounds__(kOne ? back_threads<VEC>(NV * VEC) : 256, kOne ? 1 : kBackCtas) layer_bwd_kernel(const BwdArgs p) {
  __shared__ float sm[2][64];
  extern __shared__ __align__(16) uint4 ring[];
  // behind the rows the column sums are joined where the ring was
  float* sums = reinterpret_cast<float*>(ring);  // [cols], with more than one group or odd rows
  const int groups = kOne ? 1 : p.groups;
  const int lanes = blockDim.x / groups, cols = static_cast<int>(p.cols);
  const int group = kOne ? 0 : threadIdx.x / lanes, t = threadIdx.x - group * lanes, warps = lanes >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  constexpr int P = VEC / 2;
  Rows<T, VEC, NV, kOdd, 3> rows(p.from, p.ld, p.rows, first, step, cols, t, lanes,
                                 blockDim.x, ring, p.ahead);
  const Columns<T, VEC, kOdd>& at = rows.at;
  launch_dependents();
  grid_dependency_wait();
  rows.start(p, first);
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (first < p.rows) {
    next_mean = p.mean[first];
    next_rstd = p.rstd[first];
  }
  // this thread's columns: gains and sums
  float2 g[NV][P], acc[NV][P], accd[NV][P];
  float ge = 1.0f, acce = 0.0f, accde = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int k = rows.column(v);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      g[v][j] = both(1.0f);
      if (p.gamma && k < rows.end)
        g[v][j] = make_float2(__ldg(p.gamma + k + 2 * j), __ldg(p.gamma + k + 2 * j + 1));
      acc[v][j] = both(0.0f);
      accd[v][j] = both(0.0f);
    }
  }
  if (kOdd && p.gamma && at.has) ge = __ldg(p.gamma + at.one);
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  T* dx = static_cast<T*>(p.dx) + first * p.lddx + rows.column0;
  int phase = 0;
  for (int64_t row = first; row < p.rows; row += step, phase ^= 1, dx += p.dx_skip) {
    const float mean = next_mean, rstd = next_rstd;
    Piece<T, VEC, NV> in[3];
    rows.operands(p, row + step, in);
    if (row + step < p.rows) {
      next_mean = p.mean[row + step];
      next_rstd = p.rstd[row + step];
    }
    float2 n[NV][P], h[NV][P], dot2 = both(0.0f), total2 = both(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      pairs(in[0].v[v], n[v]);
      pairs(in[1].v[v], h[v]);
#pragma unroll
      for (int j = 0; j < P; ++j) {  // dy is zero where the thread has no columns
        h[v][j] = __fmul2_rn(__fadd2_rn(h[v][j], both(-mean)), both(rstd));
        accd[v][j] = __fadd2_rn(accd[v][j], n[v][j]);
        acc[v][j] = __ffma2_rn(n[v][j], h[v][j], acc[v][j]);
        n[v][j] = __fmul2_rn(n[v][j], g[v][j]);
        total2 = __fadd2_rn(total2, n[v][j]);
        dot2 = __ffma2_rn(n[v][j], h[v][j], dot2);
      }
    }
    float dot = dot2.x + dot2.y, total = total2.x + total2.y;
    float n1[1] = {}, h1[1] = {}, y1[1] = {};
    if constexpr (kOdd) {
      to_float(in[0].one, n1);
      to_float(in[1].one, h1);
      to_float(in[2].one, y1);
      h1[0] = (h1[0] - mean) * rstd;
      accde += n1[0];
      acce = fmaf(n1[0], h1[0], acce);
      n1[0] *= ge;
      total += n1[0];
      dot = fmaf(n1[0], h1[0], dot);
    }
    group_sums(dot, total, sm[phase] + 2 * group * warps, t >> 5, warps, 1 + group);
    const float c = -dot * inv_cols, level = -total * inv_cols;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (rows.column(v) < rows.end) {
        float2 y[P];
        pairs(in[2].v[v], y);
#pragma unroll
        for (int j = 0; j < P; ++j)
          y[j] = __ffma2_rn(both(rstd), __ffma2_rn(both(c), h[v][j], __fadd2_rn(n[v][j], both(level))), y[j]);
        store<T, VEC>(dx + v * rows.stride, narrow(y, T()));
      }
    if (kOdd && at.has) {
      y1[0] = fmaf(rstd, fmaf(c, h1[0], n1[0] + level), y1[0]);
      store<T, 1>(dx + (at.one - rows.column0), from_float(y1, T()));
    }
  }
  if (!p.partial && !p.partial_dy) return;
  if (!kOne || kOdd) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // no thread has rows in the ring any more
  }
  auto emit = [&](float* out, const float2 (&pair)[NV][P], float ae) {
    float a[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[v][j] = j & 1 ? pair[v][j / 2].y : pair[v][j / 2].x;
    if constexpr (kOdd) {  // element by element, and then in order
      for (int i = 0; i < groups; ++i) {
        if (group == i) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int k = rows.column(v);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
              if (k < at.end) sums[k + j] = (i ? sums[k + j] : 0.0f) + a[v][j];
          }
          if (at.has) sums[at.one] = (i ? sums[at.one] : 0.0f) + ae;
        }
        __syncthreads();
      }
      for (int k = threadIdx.x; k < cols; k += blockDim.x) out[k] = sums[k];
      __syncthreads();
    } else {
      // the groups add their sums in turn; the last one writes
      for (int i = 0; i < groups; ++i) {
        if (group == i) {
          const bool last = i == groups - 1, wide = !last || (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int k = rows.column(v);
            if (k < cols) add_floats<VEC>((last ? out : sums) + k, sums + k, i > 0, a[v], wide);
          }
        }
        if (!kOne) __syncthreads();
      }
    }
  };
  if (p.partial) emit(p.partial + static_cast<int64_t>(blockIdx.x) * p.ldp, acc, acce);
  if (p.partial_dy) emit(p.partial_dy + static_cast<int64_t>(blockIdx.x) * p.ldp, accd, accde);
}

// Other rows: dx with the row read twice; the column sums come from layer_sums_kernel, which
// runs first (dx may lie over dy or dsum).
template <class T>
__global__ void __launch_bounds__(1024) layer_bwd_long_kernel(const BwdArgs p) {
  __shared__ float sm[2][2][32];
  int phase = 0;
  launch_dependents();
  grid_dependency_wait();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, phase ^= 1) {
    const T* dy = static_cast<const T*>(p.from[0]) + row * p.ld[0];
    const T* sp = static_cast<const T*>(p.from[1]) + row * p.ld[1];
    const T* ds = static_cast<const T*>(p.from[2]) + row * p.ld[2];
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float dot = 0.0f, total = 0.0f;
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float a[1], s[1];
      to_float(load<T, 1>(dy + k), a);
      to_float(load<T, 1>(sp + k), s);
      const float n = p.gamma ? a[0] * __ldg(p.gamma + k) : a[0];
      total += n;
      dot = fmaf(n, (s[0] - mean) * rstd, dot);
    }
    dot = cta_sum(dot, sm[phase][0]);
    total = cta_sum(total, sm[phase][1]);
    const float c = dot / static_cast<float>(p.cols), level = total / static_cast<float>(p.cols);
    for (int64_t k = threadIdx.x; k < p.cols; k += blockDim.x) {
      float a[1], s[1], d[1] = {0.0f};
      to_float(load<T, 1>(dy + k), a);
      to_float(load<T, 1>(sp + k), s);
      if (p.from[2]) to_float(load<T, 1>(ds + k), d);
      const float n = p.gamma ? a[0] * __ldg(p.gamma + k) : a[0];
      d[0] = fmaf(rstd, fmaf(-c, (s[0] - mean) * rstd, n - level), d[0]);
      store<T, 1>(dx + k, from_float(d, T()));
    }
  }
}

// Partial column sums of dy h and dy: a CTA takes 32 columns (one a lane) and every
// gridDim.x / tiles-th block of rows; its 8 warps take rows in turn.
template <class T>
__global__ void __launch_bounds__(256) layer_sums_kernel(const BwdArgs p, int parts) {
  __shared__ float sm[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % parts;
  const int64_t k = static_cast<int64_t>(blockIdx.x / parts) * 32 + lane;
  launch_dependents();
  grid_dependency_wait();
  float acc = 0.0f, accd = 0.0f;
  if (k < p.cols)
    for (int64_t row = part * 8 + warp; row < p.rows; row += static_cast<int64_t>(parts) * 8) {
      float a[1], s[1];
      to_float(load<T, 1>(static_cast<const T*>(p.from[0]) + row * p.ld[0] + k), a);
      to_float(load<T, 1>(static_cast<const T*>(p.from[1]) + row * p.ld[1] + k), s);
      acc = fmaf(a[0], (s[0] - p.mean[row]) * p.rstd[row], acc);
      accd += a[0];
    }
  sm[0][warp][lane] = acc;
  sm[1][warp][lane] = accd;
  __syncthreads();
  float* out = warp == 0 ? p.partial : p.partial_dy;
  if (warp < 2 && out && k < p.cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sm[warp][w][lane];
    out[static_cast<int64_t>(part) * p.ldp + k] = t;
  }
}

// ----------------------------------------------------------------- routing

constexpr int kSmemSm = 216 << 10;  // of an SM's shared memory, what rings may fill
constexpr int kSmemCta = 200 << 10;

// Bytes of a ring over a CTA's rows of `row` bytes, and how far ahead it runs: not further than the
// CTA has rows, nor than its shared memory holds (12288 floats and their residual: one row ahead).
int ring_of(int row, int64_t rows_each, int* ahead) {
  *ahead = kAhead;
  while (*ahead > 0 && (*ahead >= rows_each || (*ahead + 1) * row > kSmemCta)) --*ahead;
  return (*ahead + 1) * row;
}

template <auto Fn>
int launch_ring(int64_t grid, int threads, size_t smem, cudaStream_t s, const FwdArgs& p) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return T3_EDEVICE;
  const int st = allow_smem<Fn>(dev, kSmemCta);
  return st == T3_OK ? launch(Fn, grid, threads, smem, s, 1, p) : st;
}
template <auto Fn>
int launch_ring(int64_t grid, int threads, size_t smem, cudaStream_t s, const BwdArgs& p) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return T3_EDEVICE;
  const int st = allow_smem<Fn>(dev, kSmemCta);
  return st == T3_OK ? launch(Fn, grid, threads, smem, s, 1, p) : st;
}

// Threads of a CTA that reads its row again, some four elements each, and CTAs of a wave.
int other_threads(int64_t cols) { return cols >= 4096 ? 1024 : cols > 128 ? static_cast<int>((cols / 4 + 31) / 32 * 32) : 32; }
int64_t other_grid(int64_t rows, int64_t cols, int sms) {
  return std::min<int64_t>(rows, static_cast<int64_t>(sms) * std::min(1024 / other_threads(cols), 16));
}

template <class T>
int fwd_other(const FwdArgs& p, int sms, cudaStream_t s) {
  return launch(layer_fwd_long_kernel<T>, other_grid(p.rows, p.cols, sms), other_threads(p.cols), 0, s, 1, p);
}

// Forward: few rows take the fewest elements a thread, many rows 16 or more.
template <class T, int VEC, bool kOdd>
int fwd_vec(FwdArgs p, int sms, cudaStream_t s) {
  const bool many = p.rows >= 2 * static_cast<int64_t>(sms);
  int threads = 0;
  const int nv = pick<VEC, 4>((p.cols + VEC - 1) / VEC, many ? (VEC == 8 ? 16 : 8) : 1, front_threads, &threads);
  if (nv == 0) return fwd_other<T>(p, sms, s);
  // one wave of resident CTAs (80 registers a thread)
  const int smem = ring_of(2 * nv * threads * 16, (p.rows + sms - 1) / sms, &p.ahead);
  const int64_t each = std::max(1, std::min(front_threads(nv * VEC) / threads, kSmemSm / (smem + 1024)));
  int64_t grid = std::min<int64_t>(p.rows, sms * each);
  if (kOdd) grid = alike<VEC>(grid, p.rows, p.ld[0], 1);
  for (int i = 0; i < 2; ++i) p.skip[i] = grid * p.ld[i];
  p.lds_skip = grid * p.lds;
  p.q_skip = grid * p.cols;
  if (nv == 1) return launch_ring<layer_fwd_kernel<T, VEC, 1, kOdd>>(grid, threads, smem, s, p);
  if (nv == 2) return launch_ring<layer_fwd_kernel<T, VEC, 2, kOdd>>(grid, threads, smem, s, p);
  return launch_ring<layer_fwd_kernel<T, VEC, 4, kOdd>>(grid, threads, smem, s, p);
}

template <class T>
int bwd_other(BwdArgs p, float* dgamma, float* dbeta, int sms, int* parts, cudaStream_t s) {
  if (p.partial || p.partial_dy) {
    const int64_t tiles = (p.cols + 31) / 32;
    // some four CTAs an SM, each with at least a block of rows
    const int64_t n = std::max<int64_t>(1, std::min<int64_t>({(p.rows + 7) / 8, 4ll * sms / tiles, kMaxColParts}));
    *parts = static_cast<int>(n);
    if (n == 1 && p.partial) p.partial = dgamma;
    if (n == 1 && p.partial_dy) p.partial_dy = dbeta;
    const int st = launch(layer_sums_kernel<T>, tiles * n, 256, 0, s, 1, p, *parts);
    if (st != T3_OK) return st;
  }
  return launch(layer_bwd_long_kernel<T>, other_grid(p.rows, p.cols, sms), other_threads(p.cols), 0, s, 1, p);
}

// Backward: many rows take 8 elements a thread (more only where the row would not
// fit a CTA).  One part is the sums themselves: it goes where they are wanted.
template <class T, int VEC, bool kOdd>
int bwd_vec(BwdArgs p, float* dgamma, float* dbeta, int sms, int* parts, cudaStream_t s) {
  const bool many = p.rows >= 2 * static_cast<int64_t>(sms);
  int threads = 0;
  const int nv = pick<VEC, 4>((p.cols + VEC - 1) / VEC, many ? 8 : 1, back_threads<VEC>, &threads);
  if (nv == 0) return bwd_other<T>(p, dgamma, dbeta, sms, parts, s);
  // narrow rows: two groups or more in 256 threads, kBackCtas such CTAs an SM;
  // else a CTA a row, as many as the registers hold
  p.groups = many && nv * VEC == 8 ? std::max(1, 256 / threads) : 1;
  const bool one = p.groups == 1;
  int smem = ring_of(3 * nv * threads * p.groups * 16, (p.rows + sms - 1) / sms, &p.ahead);
  if ((kOdd || !one) && smem < p.cols * 4) smem = static_cast<int>(p.cols) * 4;
  const int room = (one ? back_threads<VEC>(nv * VEC) : 256 * kBackCtas) / (threads * p.groups);
  const int64_t each = std::max(1, std::min(room, kSmemSm / (smem + 1024)));
  int64_t grid = std::min<int64_t>({sms * each, (p.rows + p.groups - 1) / p.groups, kMaxColParts});
  if (kOdd) grid = alike<VEC>(grid, p.rows, p.ld[0], p.groups);
  for (int i = 0; i < 3; ++i) p.skip[i] = grid * p.groups * p.ld[i];
  p.dx_skip = grid * p.groups * p.lddx;
  *parts = static_cast<int>(grid);
  if (grid == 1 && p.partial) p.partial = dgamma;
  if (grid == 1 && p.partial_dy) p.partial_dy = dbeta;
  if (!one)
    return launch_ring<layer_bwd_kernel<T, VEC, 8 / VEC, false, kOdd>>(grid, threads * p.groups, smem, s, p);
  if (nv == 1) return launch_ring<layer_bwd_kernel<T, VEC, 1, true, kOdd>>(grid, threads, smem, s, p);
  if (nv == 2) return launch_ring<layer_bwd_kernel<T, VEC, 2, true, kOdd>>(grid, threads, smem, s, p);
  return launch_ring<layer_bwd_kernel<T, VEC, 4, true, kOdd>>(grid, threads, smem, s, p);
}

}  // namespace ln

int launch_layernorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                         const float* beta, float eps, int8_t* q, float* row_scale, float* mean, float* rstd,
                         void* sum_out, int64_t lds, int64_t rows, int64_t cols, int dtype, int sms,
                         cudaStream_t s) {
  const ln::FwdArgs p{{x, residual}, {ldx, ldr}, lds,     {}, 0, 0, gamma, beta, eps, q,
                      row_scale,     mean,       rstd,    sum_out, rows, cols, 0};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(x, ldx, es) && nm::vec_rows(residual, ldr, es) &&
                   nm::vec_rows(sum_out, lds, es) && vec::aligned(q, v);
  // rows that are alike; their codes, too, then lie to boundaries of v bytes as they do to v elements
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(residual, ldr, x, ldx, es, v) &&
                   nm::alike_rows(sum_out, lds, x, ldx, es, v) && reinterpret_cast<uintptr_t>(x) % es == 0 &&
                   (reinterpret_cast<uintptr_t>(x) / es - reinterpret_cast<uintptr_t>(q)) % v == 0 && (ldx - cols) % v == 0;
  if (dtype == T3_OUT_BF16)
    return vec   ? ln::fwd_vec<vec::bf16, 8, false>(p, sms, s)
           : odd ? ln::fwd_vec<vec::bf16, 8, true>(p, sms, s)
                 : ln::fwd_other<vec::bf16>(p, sms, s);
  return vec   ? ln::fwd_vec<float, 4, false>(p, sms, s)
         : odd ? ln::fwd_vec<float, 4, true>(p, sms, s)
               : ln::fwd_other<float>(p, sms, s);
}

int launch_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t lds, const float* mean,
                         const float* rstd, const float* gamma, const void* dsum, int64_t lddsum, void* dx,
                         int64_t lddx, float* dgamma, float* dbeta, int64_t rows, int64_t cols, int dtype,
                         float* workspace, int sms, cudaStream_t s) {
  // both sums: a partial row holds dgamma's columns and then dbeta's
  const int64_t ldp = dgamma && dbeta ? 2 * cols : cols;
  const ln::BwdArgs p{{dy, x, dsum}, {lddy, lds, lddsum}, lddx, {}, 0, mean, rstd, gamma, dx, dgamma ? workspace : nullptr,
                      dbeta ? workspace + (dgamma ? cols : 0) : nullptr, ldp, rows, cols, 0, 0};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4, v = 16 / es;
  const bool vec = cols % v == 0 && nm::vec_rows(dy, lddy, es) && nm::vec_rows(x, lds, es) &&
                   nm::vec_rows(dsum, lddsum, es) && nm::vec_rows(dx, lddx, es);
  const bool odd = !vec && cols >= nm::kOddCols && nm::alike_rows(x, lds, dy, lddy, es, v) &&
                   nm::alike_rows(dsum, lddsum, dy, lddy, es, v) && nm::alike_rows(dx, lddx, dy, lddy, es, v);
  int parts = 0, st;
  if (dtype == T3_OUT_BF16)
    st = vec   ? ln::bwd_vec<vec::bf16, 8, false>(p, dgamma, dbeta, sms, &parts, s)
         : odd ? ln::bwd_vec<vec::bf16, 8, true>(p, dgamma, dbeta, sms, &parts, s)
               : ln::bwd_other<vec::bf16>(p, dgamma, dbeta, sms, &parts, s);
  else
    st = vec   ? ln::bwd_vec<float, 4, false>(p, dgamma, dbeta, sms, &parts, s)
         : odd ? ln::bwd_vec<float, 4, true>(p, dgamma, dbeta, sms, &parts, s)
               : ln::bwd_other<float>(p, dgamma, dbeta, sms, &parts, s);
  if (st != T3_OK || (!dgamma && !dbeta) || parts == 1) return st;
  if (dgamma && dbeta) return launch_col_finish2(workspace, parts, cols, dgamma, dbeta, s);
  return launch_col_finish(workspace, parts, cols, dgamma ? dgamma : dbeta, s);
}

}  // namespace t3
