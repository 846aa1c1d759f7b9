// t3_linear_tc_64_128.cu -- linear attention by chunks for heads of up to 64 (q, k) and 128 (v) elements.
#include "t3_linear_tc.cuh"

namespace t3 {
namespace lin {
T3_LINEAR_TC(64, 128);
}  // namespace lin
}  // namespace t3
