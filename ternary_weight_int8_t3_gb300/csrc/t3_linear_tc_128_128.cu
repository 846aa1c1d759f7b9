// t3_linear_tc_128_128.cu -- linear attention by chunks for heads of up to 128 (q, k) and 128 (v) elements.
#include "t3_linear_tc.cuh"

namespace t3 {
namespace lin {
T3_LINEAR_TC(128, 128);
}  // namespace lin
}  // namespace t3
