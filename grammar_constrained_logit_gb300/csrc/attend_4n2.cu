// attend_4n2.cu -- attention over a cache of 4 bits: queries and weights in one piece, 16 rows.
#include "attend_mma.cuh"

namespace lp {

cudaError_t attend_4n2(const AttendArgs& a, int block, cudaStream_t stream) {
  return attend_mma<4, false, 2>(a, block, stream);
}

}  // namespace lp
