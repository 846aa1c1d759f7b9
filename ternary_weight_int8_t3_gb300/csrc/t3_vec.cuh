// t3_vec.cuh -- what the row, sequence and epilogue kernels share: element
// types (float, bf16) loaded and stored as vectors of floats, reductions over a
// warp, and the launch that lets a
// kernel's set-up overlap the end of the work before it.
#pragma once
#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>

#include "t3.h"
#include "t3_act.cuh"
#include "t3_internal.h"

namespace t3 {
namespace vec {

using bf16 = __nv_bfloat16;

// VEC elements of T as they lie in memory: 16 bytes, 4 bytes or one element.
template <class T, int VEC> struct Raw;
template <> struct Raw<bf16, 8> { uint4 v; };
template <> struct Raw<float, 4> { float4 v; };
template <> struct Raw<bf16, 4> { uint2 v; };
template <> struct Raw<bf16, 2> { uint32_t v; };
template <> struct Raw<float, 2> { float2 v; };
template <> struct Raw<bf16, 1> { uint16_t v; };
template <> struct Raw<float, 1> { float v; };

template <class T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load(const T* p) {
  Raw<T, VEC> r;
  r.v = *reinterpret_cast<const decltype(r.v)*>(p);
  return r;
}

template <class T, int VEC>
__device__ __forceinline__ Raw<T, VEC> zero() {
  Raw<T, VEC> r;
  r.v = {};
  return r;
}

__device__ __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xFFFF0000u);
}

__device__ __forceinline__ void to_float(const Raw<bf16, 8>& r, float (&f)[8]) {
  unpack(r.v.x, f[0], f[1]);
  unpack(r.v.y, f[2], f[3]);
  unpack(r.v.z, f[4], f[5]);
  unpack(r.v.w, f[6], f[7]);
}
__device__ __forceinline__ void to_float(const Raw<bf16, 4>& r, float (&f)[4]) {
  unpack(r.v.x, f[0], f[1]);
  unpack(r.v.y, f[2], f[3]);
}
__device__ __forceinline__ void to_float(const Raw<bf16, 2>& r, float (&f)[2]) { unpack(r.v, f[0], f[1]); }
__device__ __forceinline__ void to_float(const Raw<bf16, 1>& r, float (&f)[1]) {
  f[0] = __uint_as_float(static_cast<uint32_t>(r.v) << 16);
}
__device__ __forceinline__ void to_float(const Raw<float, 4>& r, float (&f)[4]) {
  f[0] = r.v.x;
  f[1] = r.v.y;
  f[2] = r.v.z;
  f[3] = r.v.w;
}
__device__ __forceinline__ void to_float(const Raw<float, 2>& r, float (&f)[2]) {
  f[0] = r.v.x;
  f[1] = r.v.y;
}
__device__ __forceinline__ void to_float(const Raw<float, 1>& r, float (&f)[1]) { f[0] = r.v; }

// Two floats rounded to bf16 (nearest, ties to even), `lo` in the low half.
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ Raw<bf16, 8> from_float(const float (&f)[8], bf16) {
  Raw<bf16, 8> r;
  r.v = make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
  return r;
}
__device__ __forceinline__ Raw<bf16, 4> from_float(const float (&f)[4], bf16) {
  Raw<bf16, 4> r;
  r.v = make_uint2(pack(f[0], f[1]), pack(f[2], f[3]));
  return r;
}
__device__ __forceinline__ Raw<bf16, 2> from_float(const float (&f)[2], bf16) {
  Raw<bf16, 2> r;
  r.v = pack(f[0], f[1]);
  return r;
}
__device__ __forceinline__ Raw<bf16, 1> from_float(const float (&f)[1], bf16) {
  Raw<bf16, 1> r;
  r.v = static_cast<uint16_t>(pack(f[0], 0.0f) & 0xFFFFu);
  return r;
}
__device__ __forceinline__ Raw<float, 4> from_float(const float (&f)[4], float) {
  Raw<float, 4> r;
  r.v = make_float4(f[0], f[1], f[2], f[3]);
  return r;
}
__device__ __forceinline__ Raw<float, 2> from_float(const float (&f)[2], float) {
  Raw<float, 2> r;
  r.v = make_float2(f[0], f[1]);
  return r;
}
__device__ __forceinline__ Raw<float, 1> from_float(const float (&f)[1], float) {
  Raw<float, 1> r;
  r.v = f[0];
  return r;
}

template <class T, int VEC>
__device__ __forceinline__ void store(T* p, const Raw<T, VEC>& r) {
  *reinterpret_cast<decltype(r.v)*>(p) = r.v;
}

// A float as it reads back after being stored as T.
__device__ __forceinline__ float round_to(float x, float) { return x; }
__device__ __forceinline__ float round_to(float x, bf16) { return __bfloat162float(__float2bfloat16_rn(x)); }

// VEC floats from a float array (16-byte loads where VEC allows; the array is
// 16-byte aligned there).
template <int VEC>
__device__ __forceinline__ void load_floats(const float* p, float (&f)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p) + j);
      f[4 * j] = v.x;
      f[4 * j + 1] = v.y;
      f[4 * j + 2] = v.z;
      f[4 * j + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = __ldg(p + j);
  }
}

// max that keeps a NaN of either side (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Launches `fn` as a programmatic dependent of the work before it on `s`: the
// kernel calls grid_dependency_wait() before it touches memory.  cluster > 1:
// that many CTAs per cluster.
template <class... Params, class... Args>
int launch(void (*fn)(Params...), int64_t grid, int threads, size_t smem, cudaStream_t s, int cluster,
           Args... args) {
  if (grid < 1 || grid > 2147483647) return T3_EINVAL;  // more CTAs than a grid holds
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, fn, static_cast<Params>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return T3_ECUDA;
  }
  return T3_OK;
}

constexpr int kMaxCluster = 8;  // CTAs a cluster, the portable limit

// Host queries in front of a launch.  One that fails is not kept, and takes its
// error out of the runtime's record: other calls end by looking there.

// Dynamic shared memory of `Fn`, set once per device.
template <auto Fn>
int allow_smem(int dev, int bytes) {
  static std::atomic<bool> done[64];
  if (!done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(Fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
      cudaGetLastError();
      return T3_ECUDA;
    }
    done[dev].store(true, std::memory_order_release);
  }
  return T3_OK;
}

// How many clusters of c CTAs of `Fn` are resident at once, asked once per device.
template <auto Fn>
int max_clusters(int dev, int c, int threads, size_t smem) {
  static std::atomic<int> cache[64][kMaxCluster + 1];  // the answer + 1
  int n = cache[dev][c].load(std::memory_order_acquire);
  if (n > 0) return n - 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(c);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, Fn, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cache[dev][c].store(n + 1, std::memory_order_release);
  return n;
}

__host__ inline bool aligned(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

}  // namespace vec
}  // namespace t3
