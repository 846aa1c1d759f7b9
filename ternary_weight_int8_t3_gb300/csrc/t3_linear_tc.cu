// t3_linear_tc.cu -- linear attention by chunks: which calls it takes, and its launch (the kernels are in
// t3_linear_tc.cuh).
#include <cudaTypedefs.h>

#include <cstring>

#include "t3_internal.h"
#include "t3_linear.cuh"

namespace t3 {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace lin {

constexpr int kChunk = 128;

// One pass for heads of up to DK and DV elements (t3_linear_tc.cuh).
template <int DK, int DV>
int run_tc(const Args& p, bool reverse, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int* err,
           cudaStream_t s);

// Rows of a head's 64 columns and 128 tokens of [batch][length][heads][d], 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* map, const void* base, const Args& p, int64_t ld, int d) {
  std::memset(map, 0, sizeof(*map));
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.heads), static_cast<cuuint64_t>(p.length),
                        static_cast<cuuint64_t>(p.pairs / p.heads)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(ld) * 2,
                           static_cast<cuuint64_t>(p.length) * ld * 2};
  cuuint32_t box[4] = {64, 1, kChunk, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace lin

// More tokens than one block of the other kernel takes as fast; rows and heads that TMA can address, and
// outputs that take 16-byte stores.
bool linear_tc_fits(const lin::Args& p, int dtype) {
  auto rows = [](const void* base, int64_t ld) { return vec::aligned(base, 16) && ld % 8 == 0; };
  return dtype == T3_OUT_BF16 && p.length > 16 && p.dk % 8 == 0 && p.dv % 8 == 0 && rows(p.q, p.ldq) &&
         rows(p.k, p.ldk) && rows(p.v, p.ldv) && rows(p.o, p.ldo) && p.ldq >= p.heads * p.dk &&
         p.ldk >= p.heads * p.dk && p.ldv >= p.heads * p.dv &&
         p.length * std::max(p.ldq, std::max(p.ldk, p.ldv)) < (int64_t{1} << 38);
}

int launch_linear_tc(lin::Args p, bool reverse, float* workspace, int sms, int* err, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!lin::make_map(&mq, p.q, p, p.ldq, p.dk) || !lin::make_map(&mk, p.k, p, p.ldk, p.dk) ||
      !lin::make_map(&mv, p.v, p, p.ldv, p.dv))
    return T3_ECUDA;
  p.blocks = (p.length + lin::kChunk - 1) / lin::kChunk;
  const int st = lin::cut(&p, sms, workspace, s);
  if (st != T3_OK) return st;
  if (p.dk <= 64)
    return p.dv <= 64 ? lin::run_tc<64, 64>(p, reverse, mq, mk, mv, err, s) : lin::run_tc<64, 128>(p, reverse, mq, mk, mv, err, s);
  return p.dv <= 64 ? lin::run_tc<128, 64>(p, reverse, mq, mk, mv, err, s) : lin::run_tc<128, 128>(p, reverse, mq, mk, mv, err, s);
}

}  // namespace t3
