// attend_4w1.cu -- attention over a cache of 4 bits: queries and weights in two pieces, 8 rows.
#include "attend_mma.cuh"

namespace lp {

cudaError_t attend_4w1(const AttendArgs& a, int block, cudaStream_t stream) {
  return attend_mma<4, true, 1>(a, block, stream);
}

}  // namespace lp
