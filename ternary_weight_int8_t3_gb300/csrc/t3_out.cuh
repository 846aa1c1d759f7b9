// t3_out.cuh -- where the kernels that end a sum in registers put it: into the
// int32 output, or through a layer's epilogue (EpilogueArgs) into f32 or bf16.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "t3.h"
#include "t3_act.cuh"

namespace t3 {

// `ahead` loads what the epilogue of C[m][n] needs before the sum is taken, so
// that those loads are not on the end of the kernel; `put` ends the sum of the
// element at `at` = m N + n.
struct OutI32 {
  int32_t* C;
  struct Ahead {};
  __device__ __forceinline__ Ahead ahead(int64_t, int64_t, int64_t) const { return {}; }
  __device__ __forceinline__ void put(int64_t at, int32_t acc, const Ahead&) const { C[at] = acc; }
};

template <class T>
struct OutAct {
  T* C;
  EpilogueArgs e;
  struct Ahead {
    float rs, cs, bias, res;
  };
  static __device__ __forceinline__ float value(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ __forceinline__ Ahead ahead(int64_t m, int64_t n, int64_t N) const {
    return {e.row_scale ? __ldg(e.row_scale + m) : 1.0f, e.col_scale ? __ldg(e.col_scale + n) : 1.0f,
            e.bias ? __ldg(e.bias + n) : 0.0f,
            e.residual ? value(static_cast<const T*>(e.residual) + m * N + n) : 0.0f};
  }
  static __device__ __forceinline__ void write(float* p, float y) { *p = y; }
  static __device__ __forceinline__ void write(__nv_bfloat16* p, float y) { *p = __float2bfloat16_rn(y); }
  __device__ __forceinline__ void put(int64_t at, int32_t acc, const Ahead& a) const {
    float y = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(acc), a.rs), a.cs), a.bias);
    if (e.pre) write(static_cast<T*>(e.pre) + at, y);
    switch (e.act) {
      case T3_ACT_RELU: y = vec::act<T3_ACT_RELU>(y); break;
      case T3_ACT_RELU2: y = vec::act<T3_ACT_RELU2>(y); break;
      case T3_ACT_SILU: y = vec::act<T3_ACT_SILU>(y); break;
      case T3_ACT_GELU: y = vec::act<T3_ACT_GELU>(y); break;
      default: break;
    }
    write(C + at, __fadd_rn(y, a.res));  // the same bits on every route
  }
};

}  // namespace t3
